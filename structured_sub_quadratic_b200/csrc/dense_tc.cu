// Exact softmax attention on the tensor cores: bf16, d a multiple of 8 up to
// 128 (the TMA boxes of 64 or 128 channels fill the rest with zeros), rows of
// 16-byte alignment in any strides.
#include "dense.cuh"

#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>

#include "launch.cuh"
#include "tc_ptx.cuh"
#include "timing.cuh"

namespace monarch {
namespace {

using namespace tc;

constexpr int kTile = 128;           // rows and keys of a tile = UMMA M = TMEM lanes
constexpr int kChunk = kTile * 128;  // 128 rows x 64 bf16, 128-byte swizzled
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_ns() - t0 > kWaitLimitNs) break;
}

// One arrival for the warp, after the tcgen05 loads and stores of its lanes
// (an arrival per thread would queue 32 updates of one word in shared memory,
// whose bandwidth the products need).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// 16-byte unit u (channels 8u ..) of row r of a tile of swizzled 64-channel chunks.
__device__ __forceinline__ uint4* row_unit(uint8_t* tile, int r, int u) {
  return reinterpret_cast<uint4*>(tile + (u >> 3) * kChunk + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

// 2^x of a pair on the FMA pipe, beside the exponential unit (16 results a
// clock and SM, which a d = 64 tile keeps busier than its products do the
// tensor cores): x = n + f with n the nearest integer (x + 1.5 2^23 has it in
// its low bits), 2^f by the polynomial of least relative error on [-1/2, 1/2]
// (degree 5, by Remez exchange: 7e-8, 2e-7 in fp32, as the unit's), n added to
// the exponent.  Hidden keys, at -inf, give 2^-149, which bf16 rounds to 0 and
// a sum does not feel; what lies between 2^-127 and 2^-126 is only known to be
// below 2^-126.  A NaN is lost here (at the clamp, and the exponent's sum would
// turn one into a number): the row's maximum and other exponentials keep it.
__device__ __forceinline__ float2 exp2_fma(float2 x) {
  x.x = fmaxf(x.x, -127.f);
  x.y = fmaxf(x.y, -127.f);
  const float2 big = make_float2(12582912.f, 12582912.f);
  const float2 y = add2(x, big);
  const float2 n = add2(y, make_float2(-12582912.f, -12582912.f));
  const float2 f = add2(x, make_float2(-n.x, -n.y));
  auto both = [](float c) { return make_float2(c, c); };
  float2 p = fma2(both(1.3276472454890609e-3f), f, both(9.675540961325169e-3f));
  p = fma2(p, f, both(5.550713092088699e-2f));
  p = fma2(p, f, both(2.4022120237350464e-1f));
  p = fma2(p, f, both(6.931469440460205e-1f));
  p = fma2(p, f, both(1.0000001192092896f));
  return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(y.x) << 23)),
                     __int_as_float(__float_as_int(p.y) + (__float_as_int(y.y) << 23)));
}

// One 128-row tile of a (B, H, N, d) tensor, D channels: D / 64 boxes.  A
// broadcast head or batch has one entry in the map (mul 0).
struct TileMap {
  CUtensorMap map;
  int h_mul, b_mul;
};

template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const TileMap& m, uint64_t* bar, int row,
                                          int h, int b) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    tma_load_4d(dst + c * kChunk, &m.map, bar, c * 64, row, h * m.h_mul, b * m.b_mul);
}

// The products below are issued by a whole warp (one lane elected).

// Wait of the whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

__device__ __forceinline__ void warp_commit(uint64_t* bar) {
  if (elect_one()) mma_commit(bar);
}

// D[tmem] = A B^T over D channels: A a tile, B a tile or its first N rows,
// both K-major in shared memory.
template <int D, int N = kTile>
__device__ __forceinline__ void mma_nt(uint32_t tmem, uint64_t a, uint64_t b) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * kChunk + (kk & 3) * 32) >> 4;
    if (elect_one())
      mma_bf16_ss(tmem, a + off, b + off, idesc_bf16(kTile, N, false), kk > 0 ? 1u : 0u);
  }
}

// D[tmem] (+)= W X: W 128 x 64 bf16 in TMEM, X 64 rows of a tile, D channels.
template <int D>
__device__ __forceinline__ void mma_ts64(uint32_t tmem, uint32_t w_tmem, uint64_t x,
                                         bool accumulate) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
    if (elect_one())
      mma_bf16_ts(tmem, w_tmem + kk * 8, x + ((kk * 16 * 128) >> 4), idesc_bf16(kTile, D, true),
                  accumulate || kk > 0 ? 1u : 0u);
}

// 64 columns of this thread's lane.
__device__ __forceinline__ void load_half(uint32_t taddr, float (&x)[64]) {
  float t[2][32];
  tmem_ld32(taddr, t[0]);
  tmem_ld32(taddr + 32, t[1]);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 64; ++e) x[e] = t[e >> 5][e & 31];
}

// Row r of a D-wide accumulator times `f`, as bf16, into a swizzled tile;
// zeros where nothing was accumulated (the columns hold anything) or `keep`
// is false.
template <int D>
__device__ __forceinline__ void accumulator_row(uint8_t* tile, int r, uint32_t taddr, float f,
                                                bool any, bool keep = true) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    if (any) {
      tmem_ld32(taddr + c * 32, o);
      tmem_wait_ld();
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = any && keep ? o[e] * f : 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *row_unit(tile, r, c * 4 + u) =
          make_uint4(pack_bf16x2(o[8 * u], o[8 * u + 1]), pack_bf16x2(o[8 * u + 2], o[8 * u + 3]),
                     pack_bf16x2(o[8 * u + 4], o[8 * u + 5]),
                     pack_bf16x2(o[8 * u + 6], o[8 * u + 7]));
  }
}

// ---------------------------------------------------------------------------
// Forward.  A CTA has two 128-row tiles of queries at d > 64, one at d <= 64
// (where two CTAs share an SM: their softmaxes drift apart, which those of one
// CTA's tiles do not, 12 heads of 16384 keys 1075 -> 1022 us), a warpgroup each
// with a thread per row.  They walk the keys 64 at a time in one pass.  S has
// two buffers a tile, so that S of step u + 2 is issued right behind P V of step
// u and the softmaxes never wait for a product that has not long begun (with one
// 128-key buffer, the chain softmax, P V, S took 3450 clocks per 256 x 128
// scores at d = 128, against 2070 of products).  O stays in TMEM under a running
// maximum that only moves when it grows by more than 2^8 (probabilities then
// reach 256, exact in the exponents of P's bf16 and of the fp32 sum), so
// rescaling O is rare.  A score of NaN or +inf makes the maximum NaN, and with
// it the row's exponentials, sum and result.  P overwrites S, rounded to bf16 as
// the result is, and is the A operand of P V.  Bound: the exponential unit and
// the FMA pipe at d = 64 (12 heads of 16384 in 1047 us between idle times, 790
// TFLOP/s, and 1127 in a pass among others, 730), the products at d = 128, 12
// heads of 4680 in 139 us (0.97 PFLOP/s).
// Warps: four of softmax per tile, one of TMA, one of products.
// ---------------------------------------------------------------------------
constexpr int kStep = 64;  // keys of a step

template <int D>
struct FwdLayout {
  static constexpr int kCh = D / 64, kStages = D == 128 ? 2 : 3;
  static constexpr int kTileBytes = kCh * kChunk;
  static constexpr int kTiles = D == 128 ? 2 : 1;  // 128-row tiles of a CTA
  static constexpr int kThreads = kTiles * kTile + 64, kTmaWarp = kTiles * 4;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kTiles * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kBarOff = kVOff + kStages * kTileBytes;
  static constexpr int kBytes = kBarOff + 32 * 8;
  // TMEM columns: S of tile t and buffer y at 128 t + 64 y, then O of tile t
  static constexpr uint32_t kTmemCols = kTiles * 256, kOCol = kTiles * kTile;
  // of 16 pairs of exponentials, those on the FMA pipe
  static constexpr int kFmaPairs = D == 64 ? 4 : 0;
  static_assert(kBytes * (3 - kTiles) <= 226 * 1024, "shared memory");
};

struct FwdArgs {
  float* lse;
  DenseProblem pb;
  int tiles;  // CTAs along the queries of a head
  int* status;
  KeySplit split;
};

template <int D>
__global__ void __launch_bounds__(FwdLayout<D>::kThreads, 3 - FwdLayout<D>::kTiles)
    dense_fwd_tc_kernel(const __grid_constant__ TileMap mq, const __grid_constant__ TileMap mk,
                        const __grid_constant__ TileMap mv, const __grid_constant__ TileMap mo,
                        const __grid_constant__ FwdArgs a) {
  using L = FwdLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // swizzled tiles need 1024-B alignment: report, never fault
    if (tid == 0) atomicExch(a.status, 2);
    return;
  }
  const DenseProblem& pb = a.pb;
  // causal: the longest tiles first, over all heads; else head by head
  const int split = blockIdx.x % a.split.splits, unit = blockIdx.x / a.split.splits;
  int tile, bh;
  if (pb.causal) {
    bh = unit % (pb.B * pb.H);
    tile = a.tiles - 1 - unit / (pb.B * pb.H);
  } else {
    tile = unit % a.tiles;
    bh = unit / a.tiles;
  }
  const int k0 = split * a.split.per * kTile;  // first key of this CTA's range
  const int h = bh % pb.H, b = bh / pb.H, hk = h / (pb.H / pb.Hkv);
  const int q0 = tile * L::kTiles * kTile;
  const int len = dense_len(pb, b);
  // steps of each row tile in the range, key tiles, and the last one's rows
  // up to the length
  int nt[2] = {0, 0};
#pragma unroll
  for (int t = 0; t < L::kTiles; ++t) {
    const int r0 = q0 + t * kTile;
    const int keys = r0 < pb.Nq ? dense_visible(pb, len, min(r0 + kTile, pb.Nq) - 1) - k0 : 0;
    nt[t] = min((max(keys, 0) + kStep - 1) / kStep, a.split.per * 2);
  }
  const int steps = max(nt[0], nt[1]), n = (steps + 1) / 2;
  const int tail = k0 + n * kTile > len && len < pb.Nk ? len - k0 - (n - 1) * kTile : kTile;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* q_full = bars;       // [2]
  uint64_t* s_full = bars + 2;   // [2][2]: S of a step, and P V of the one two before
  uint64_t* p_full = bars + 6;   // [2][2]: P of a step (a softmax may be one step ahead)
  uint64_t* k_full = bars + 10;  // [stages]
  uint64_t* k_empty = bars + 13;
  uint64_t* v_full = bars + 16;
  uint64_t* v_empty = bars + 19;
  uint64_t* v_tail = bars + 22;
  uint64_t* drain = bars + 23;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 24);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 25);
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full + t, 1);
      mbar_init(s_full + 2 * t, 1);
      mbar_init(s_full + 2 * t + 1, 1);
      mbar_init(p_full + 2 * t, 4);
      mbar_init(p_full + 2 * t + 1, 4);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, 1);
    }
    mbar_init(v_tail, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == L::kTmaWarp + 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  if (a.split.splits > 1) pdl_launch_dependents();  // the join

  if (warp == L::kTmaWarp) {
    // ---- TMA: Q, then K and V tile by tile ----
    bool ok = true;
    int kt = 0, vt = 0;  // tiles issued
    if (lane == 0) {
      tma_prefetch_desc(&mq.map);
      tma_prefetch_desc(&mk.map);
      tma_prefetch_desc(&mv.map);
      for (int t = 0; t < L::kTiles; ++t)
        if (q0 + t * kTile < pb.Nq) {
          mbar_arrive_expect_tx(q_full + t, L::kTileBytes);
          load_tile<D>(smem + L::kQOff + t * L::kTileBytes, mq, q_full + t, q0 + t * kTile, h, b);
        }
      for (int j = 0; j < n; ++j) {
        const int st = j % L::kStages;
        const uint32_t par = (j / L::kStages - 1) & 1;
        if (j >= L::kStages && !(ok = mbar_wait(k_empty + st, par, abort_flag, a.status))) break;
        mbar_arrive_expect_tx(k_full + st, L::kTileBytes);
        load_tile<D>(smem + L::kKOff + st * L::kTileBytes, mk, k_full + st, k0 + j * kTile, hk,
                     b);
        kt = j + 1;
        if (j >= L::kStages && !(ok = mbar_wait(v_empty + st, par, abort_flag, a.status))) break;
        mbar_arrive_expect_tx(v_full + st, L::kTileBytes);
        load_tile<D>(smem + L::kVOff + st * L::kTileBytes, mv, v_full + st, k0 + j * kTile, hk,
                     b);
        vt = j + 1;
      }
    }
    __syncwarp();
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok && n > 0 && tail < kTile) {
      // values past the length may hold anything (0 x NaN): zeros in their place
      const int st = (n - 1) % L::kStages;
      if (mbar_wait(v_full + st, ((n - 1) / L::kStages) & 1, abort_flag, a.status)) {
        uint8_t* sv = smem + L::kVOff + st * L::kTileBytes;
        for (int x = lane; x < (kTile - tail) * L::kCh * 8; x += 32)
          *row_unit(sv, tail + x / (L::kCh * 8), x % (L::kCh * 8)) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_tail);
      }
    }
    if (lane == 0 && *abort_flag) {  // wait (bounded) for the loads in flight
      for (int t = 0; t < L::kTiles; ++t)
        if (q0 + t * kTile < pb.Nq) drain_bar(q_full + t, 0);
      for (int s = 0; s < L::kStages; ++s) {
        if (kt > s) drain_bar(k_full + s, ((kt - 1 - s) / L::kStages) & 1);
        if (vt > s) drain_bar(v_full + s, ((vt - 1 - s) / L::kStages) & 1);
      }
    }
  } else if (warp == L::kTmaWarp + 1) {
    // ---- MMA issue ----
    if (n > 0) {
      const uint64_t dq = desc_kmajor(smem_u32(smem + L::kQOff));
      const uint64_t dk = desc_kmajor(smem_u32(smem + L::kKOff));
      const uint64_t dv = desc_mnmajor(smem_u32(smem + L::kVOff), kChunk);
      constexpr uint64_t kTileStep = L::kTileBytes >> 4, kHalf = (kStep * 128) >> 4;
      auto issue_s = [&](int t, int y, int st) {
        mma_nt<D, kStep>(tmem + t * kTile + y * kStep, dq + t * kTileStep,
                         dk + st * kTileStep + y * kHalf);
      };
      bool ok = warp_wait(k_full, 0, abort_flag, a.status);
#pragma unroll
      for (int t = 0; t < L::kTiles; ++t)
        if (ok && nt[t] > 0 && (ok = warp_wait(q_full + t, 0, abort_flag, a.status))) {
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (y < nt[t]) {
              issue_s(t, y, 0);
              warp_commit(s_full + 2 * t + y);
            }
        }
      if (ok) warp_commit(k_empty);
      int st = 0, ph = 0;  // stage and phase of key tile j
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j) {
        const int s1 = st + 1 == L::kStages ? 0 : st + 1, ph1 = s1 ? ph : ph ^ 1;
        if (!(ok = warp_wait(v_full + st, ph, abort_flag, a.status))) break;
        if (j + 1 == n && tail < kTile && !(ok = warp_wait(v_tail, 0, abort_flag, a.status))) break;
        if (j + 1 < n && !(ok = warp_wait(k_full + s1, ph1, abort_flag, a.status))) break;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int t = 0; t < L::kTiles; ++t) {
            const int u = 2 * j + y;
            if (!ok || u >= nt[t] || !(ok = warp_wait(p_full + 2 * t + y, j & 1, abort_flag, a.status)))
              continue;
            tc_fence_after();
            mma_ts64<D>(tmem + L::kOCol + t * D, tmem + t * kTile + y * kStep,
                        dv + st * kTileStep + y * kHalf, u > 0);
            // the products of one thread run in order, so S overwrites P once
            // P V has read it
            if (u + 2 < nt[t]) issue_s(t, y, s1);
            warp_commit(s_full + 2 * t + y);
          }
        if (!ok) break;
        warp_commit(v_empty + st);
        if (j + 1 < n) warp_commit(k_empty + s1);
        st = s1;
        ph = ph1;
      }
      if (__any_sync(0xffffffffu, *abort_flag != 0)) {
        warp_commit(drain);
        drain_bar(drain, 0);
      }
    }
  } else {
    // ---- softmax: thread = row r of tile t ----
    const int t = warp >> 2, r = tid & (kTile - 1);
    const int r0 = q0 + t * kTile, row = r0 + r;
    const int nj = nt[t];
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + t * kTile + lane_off, to = tmem + L::kOCol + t * D + lane_off;
    // of the range: keys that this row, and every row of the tile, sees
    const int vis = dense_visible(pb, len, row) - k0;
    const int all = dense_visible(pb, len, r0) - k0;
    const float sl = pb.scale * kLog2e;
    const float2 sl2 = make_float2(sl, sl);
    float m = -INFINITY, z = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int u = 0; u < nj; ++u) {
      uint64_t* full = s_full + 2 * t + (u & 1);
      if (!(ok = mbar_wait(full, (u >> 1) & 1, abort_flag, a.status))) break;
      tc_fence_after();
      float s[64];
      load_half(ts + (u & 1) * kStep, s);
      if ((u + 1) * kStep > all) {
        const int lim = vis - u * kStep;
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e >= lim) s[e] = -INFINITY;
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = max3_nan(c ? s[16 * c] : m, s[16 * c], s[16 * c + 1]);
#pragma unroll
        for (int e = 2; e < 16; e += 2) mx[c] = max3_nan(mx[c], s[16 * c + e], s[16 * c + e + 1]);
      }
      float mn = max3_nan(mx[0], mx[1], max3_nan(mx[2], mx[3], mx[3]));
      if (mn == INFINITY) mn = NAN;
      if (u == 0) {
        m = mn;
      } else if (__any_sync(0xffffffffu, m != mn && !((mn - m) * sl <= 8.f))) {
        // O as step u - 1 leaves it: its P V is behind the other buffer's next phase
        if (!(ok = mbar_wait(s_full + 2 * t + (~u & 1), ((u + 1) >> 1) & 1, abort_flag, a.status)))
          break;
        tc_fence_after();
        const float f = m == mn ? 1.f : ex2((m - mn) * sl);
        z *= f;
        m = mn;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(to + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
          tmem_st32(to + c * 32, o);
        }
      }
      const float base = m == -INFINITY ? 0.f : -m * sl;
      const float2 base2 = make_float2(base, base);
      float2 zs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 x = fma2(make_float2(s[c * 32 + 2 * e], s[c * 32 + 2 * e + 1]), sl2, base2);
          if ((e + 1) * L::kFmaPairs / 16 > e * L::kFmaPairs / 16)  // spread over the 16
            x = exp2_fma(x);
          else
            x = make_float2(ex2(x.x), ex2(x.y));
          zs[e & 1] = add2(zs[e & 1], x);
          pk[e] = pack_bf16x2(x.x, x.y);
        }
        tmem_st16(ts + (u & 1) * kStep + c * 16, pk);
      }
      tmem_wait_st();
      warp_arrive(p_full + 2 * t + (u & 1));
      const float2 zz = add2(zs[0], zs[1]);
      z += zz.x + zz.y;
    }
    if (r0 < pb.Nq) {
      // O / z to the tile of Q (read by every S of the tile), then one TMA store
      uint8_t* so = smem + L::kQOff + t * L::kTileBytes;
      if (ok) ok = mbar_wait(q_full + t, 0, abort_flag, a.status);
      if (ok && nj > 0)  // P V of the last step
        ok = mbar_wait(s_full + 2 * t + (~nj & 1), ((nj + 1) >> 1) & 1, abort_flag, a.status);
      tc_fence_after();
      const bool any = m != -INFINITY;  // a visible key, not all of them at -inf
      if (ok && a.split.splits > 1) {
        if (row < pb.Nq) {
          const long at = (((long)split * pb.B + b) * pb.H + h) * pb.Nq + row;
          a.split.mz[at] = make_float2(m * sl, any ? z : 0.f);
        }
        if (nj > 0) {
          float* po = a.split.o + ((((long)split * pb.B + b) * pb.H + h) * pb.Nq + row) * pb.d;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld32(to + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if (any && row < pb.Nq && c * 32 + e < pb.d)
                *reinterpret_cast<float4*>(po + c * 32 + e) =
                    make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
      } else if (ok) {
        accumulator_row<D>(so, r, to, 1.f / z, nj > 0, any);
        if (row < pb.Nq)
          a.lse[((long)b * pb.H + h) * pb.Nq + row] =
              any ? (m * sl + log2f(z)) * kLn2 : -INFINITY;
        fence_proxy_async_smem();
      }
      named_barrier(1 + t, kTile);
      if (r == 0 && ok && a.split.splits == 1 && !*abort_flag) {
        for (int c = 0; c < L::kCh; ++c)
          if (c * 64 < pb.d) tma_store_4d(&mo.map, so + c * kChunk, c * 64, r0, h, b);
        bulk_commit();
        bulk_wait_read<0>();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == L::kTmaWarp + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Backward.  The probabilities are recomputed from q, k and lse; delta is the
// row sum of dO O, from one form of it or another (kExactTiles).  Two kernels,
// so that no sum needs atomics: one owns a tile of keys and walks the queries
// (dK, dV: four products a tile), the other a tile of queries and walks the keys
// (dQ: three).  In both, eight warps hold the score tile with two threads per
// TMEM lane (64 columns each: warps 0-3 the first, 4-7 the second half), warp 8
// issues TMA and warp 9 the products.  P and dS are rounded to bf16 as operands,
// half a step each like the results; every sum is fp32.  Bound: the products and
// the chain score, exponential, product between them; 12 heads of 4680 x 128: dK
// and dV 240 us (1.12 PFLOP/s of their products), dQ 177 us (1.14).
// ---------------------------------------------------------------------------
struct BwdArgs {
  const float* lse;
  float* delta;
  DenseProblem pb;
  int tiles;  // 128-row tiles of a head
  int* status;
};

constexpr int kBwdThreads = 320;

// delta = row sum of dO O = row sum of P (dO V^T).  O is rounded to bf16, and
// where the values share a large part, which dO V^T - delta cancels, its
// rounding is most of dQ and dK (values of 256 or 258: all of them); with few
// keys it shows for any values (36 causal keys: error 2.8e-3 of dQ and dK
// against 2.4e-3, of which the roundings of dS and of the result are the rest).
// So tiles of queries that see up to 512 keys take the second form, whatever the
// length of the tensors that their sequence shares, at the price of two more
// products (five in dQ, for three) and a second walk over their keys (32 x 12
// heads of 197 x 64: 108 us, in a kernel of its own 122; 16 x 12 causal heads of
// 640 x 64, most of whose tiles are short: 163 us, with the first form 148);
// longer tiles take the first.
constexpr int kExactTiles = 4;

// The 64 columns of a thread as bf16 pairs, over its own half of a score tile.
__device__ __forceinline__ void store_half(uint32_t taddr, const float (&x)[64]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(x[c * 32 + 2 * e], x[c * 32 + 2 * e + 1]);
    tmem_st16(taddr + c * 16, pk);
  }
}

// D[tmem] (+)= W X, W's columns 0-63 and 64-127 as store_half left them.
template <int D>
__device__ __forceinline__ void mma_halves(uint32_t tmem, uint32_t w, uint64_t x,
                                           bool accumulate) {
#pragma unroll
  for (int kk = 0; kk < kTile / 16; ++kk)
    if (elect_one())
      mma_bf16_ts(tmem, w + (kk >> 2) * 64 + (kk & 3) * 8, x + ((kk * 16 * 128) >> 4),
                idesc_bf16(kTile, D, true), accumulate || kk > 0 ? 1u : 0u);
}

template <int D>
struct BwdLayout {
  static constexpr int kCh = D / 64, kStages = 2;
  static constexpr int kTileBytes = kCh * kChunk;
  static constexpr int kAOff = 0;                      // the two tiles that stay
  static constexpr int kBOff = kAOff + kTileBytes;
  static constexpr int kXOff = kBOff + kTileBytes;     // the two that are streamed
  static constexpr int kYOff = kXOff + kStages * kTileBytes;
  static constexpr int kRowOff = kYOff + kStages * kTileBytes;  // float [stages][2][128]
  static constexpr int kBarOff = kRowOff + kStages * 2 * kTile * 4;
  static constexpr int kBytes = kBarOff + 32 * 8;
  // S and dP (P and dS over them), then the accumulators
  static constexpr uint32_t kTmemCols = 512, kDPCol = 128, kAccCol = 256;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// dK and dV of 128 keys of a key/value head.  With keys as the rows:
//   S^T = K Q^T, P^T = exp(scale S^T - lse), dV += P^T dO,
//   dP^T = V dO^T, dS^T = P^T (dP^T - delta), dK += dS^T Q (times scale).
// P^T and dS^T are written over S^T and dP^T and read as A operands, so
// exponentials of one tile run beside dK and dP of the tile before, and dS
// beside dV and the next S.  The query heads of the group follow one another
// in the same accumulators.
template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    dense_dkv_tc_kernel(const __grid_constant__ TileMap mq, const __grid_constant__ TileMap mk,
                        const __grid_constant__ TileMap mv, const __grid_constant__ TileMap mg,
                        const __grid_constant__ TileMap mdk, const __grid_constant__ TileMap mdv,
                        const __grid_constant__ BwdArgs a) {
  using L = BwdLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) atomicExch(a.status, 2);
    return;
  }
  const DenseProblem& pb = a.pb;
  // causal: the first keys, which most queries see, first
  const int heads = pb.B * pb.Hkv;
  const int tile = pb.causal ? blockIdx.x / heads : blockIdx.x % a.tiles;
  const int bh = pb.causal ? blockIdx.x % heads : blockIdx.x / a.tiles;
  const int hk = bh % pb.Hkv, b = bh / pb.Hkv, group = pb.H / pb.Hkv;
  const int k0 = tile * kTile, shift = pb.Nk - pb.Nq;
  const int len = dense_len(pb, b);
  const int first = pb.causal ? max(0, k0 - shift) / kTile : 0;  // query tile
  const int per = k0 < len ? max(0, (pb.Nq + kTile - 1) / kTile - first) : 0;
  const int n = per * group;

  float* rows = reinterpret_cast<float*>(smem + L::kRowOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;   // [stages]
  uint64_t* q_empty = bars + 3;
  uint64_t* g_full = bars + 5;   // [stages]: dO
  uint64_t* g_empty = bars + 7;
  uint64_t* row_full = bars + 9;  // [stages]: lse and delta (free with Q's slot)
  uint64_t* s_full = bars + 11;
  uint64_t* dp_full = bars + 12;
  uint64_t* p_full = bars + 13;
  uint64_t* ds_full = bars + 14;
  uint64_t* done = bars + 15;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 17);
  if (tid == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(q_full + s, 1);
      mbar_init(q_empty + s, 1);
      mbar_init(g_full + s, 1);
      mbar_init(g_empty + s, 1);
      mbar_init(row_full + s, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_full, 8);
    mbar_init(ds_full, 8);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp == 8) {
    // ---- TMA: K and V, then Q and dO tile by tile with lse and delta ----
    int qs = 0, gs = 0;  // tiles issued
    if (lane == 0 && n > 0) {
      mbar_arrive_expect_tx(kv_full, 2 * L::kTileBytes);
      load_tile<D>(smem + L::kAOff, mk, kv_full, k0, hk, b);
      load_tile<D>(smem + L::kBOff, mv, kv_full, k0, hk, b);
    }
    int h = hk * group, q0 = first * kTile;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      const uint32_t par = ((i >> 1) - 1) & 1;
      // the row statistics are under way before the tile's slots are free
      const long at = ((long)b * pb.H + h) * pb.Nq;
      float l2[4], dl[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        // a row outside the tensor or without keys: exp(S - inf) = 0
        const int row = q0 + x * 32 + lane;
        const bool live = row < pb.Nq && dense_visible(pb, len, row) > 0;
        l2[x] = live ? dense_lse2(__ldg(a.lse + at + row)) : INFINITY;
        dl[x] = live ? __ldg(a.delta + at + row) : 0.f;
      }
      if (i >= 2 && !warp_wait(g_empty + st, par, abort_flag, a.status)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(g_full + st, L::kTileBytes);
        load_tile<D>(smem + L::kYOff + st * L::kTileBytes, mg, g_full + st, q0, h, b);
      }
      gs = i + 1;
      if (i >= 2 && !warp_wait(q_empty + st, par, abort_flag, a.status)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full + st, L::kTileBytes);
        load_tile<D>(smem + L::kXOff + st * L::kTileBytes, mq, q_full + st, q0, h, b);
      }
      qs = i + 1;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        rows[st * 256 + x * 32 + lane] = l2[x];
        rows[st * 256 + kTile + x * 32 + lane] = dl[x];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(row_full + st);
      q0 += kTile;
      if (q0 >= pb.Nq) {
        q0 = first * kTile;
        ++h;
      }
    }
    if (lane == 0 && n > 0 && *abort_flag) {  // wait (bounded) for the loads in flight
      drain_bar(kv_full, 0);
      for (int s = 0; s < L::kStages; ++s) {
        if (qs > s) drain_bar(q_full + s, ((qs - 1 - s) >> 1) & 1);
        if (gs > s) drain_bar(g_full + s, ((gs - 1 - s) >> 1) & 1);
      }
    }
  } else if (warp == 9) {
    // ---- MMA issue ----
    if (n > 0) {
      const uint64_t dk = desc_kmajor(smem_u32(smem + L::kAOff));
      const uint64_t dv = desc_kmajor(smem_u32(smem + L::kBOff));
      const uint64_t xk = desc_kmajor(smem_u32(smem + L::kXOff));
      const uint64_t yk = desc_kmajor(smem_u32(smem + L::kYOff));
      const uint64_t xm = desc_mnmajor(smem_u32(smem + L::kXOff), kChunk);
      const uint64_t ym = desc_mnmajor(smem_u32(smem + L::kYOff), kChunk);
      constexpr uint64_t kStep = L::kTileBytes >> 4;
      bool ok = warp_wait(kv_full, 0, abort_flag, a.status) &&
                warp_wait(q_full, 0, abort_flag, a.status);
      if (ok) {
        mma_nt<D>(tmem, dk, xk);
        warp_commit(s_full);
        ok = warp_wait(g_full, 0, abort_flag, a.status);
      }
      if (ok) {
        mma_nt<D>(tmem + L::kDPCol, dv, yk);
        warp_commit(dp_full);
      }
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int st = i & 1, s1 = st ^ 1;
        const uint32_t ph1 = ((i + 1) >> 1) & 1;
        const bool more = i + 1 < n;
        if (more && !(ok = warp_wait(q_full + s1, ph1, abort_flag, a.status))) break;
        if (!(ok = warp_wait(p_full, i & 1, abort_flag, a.status))) break;
        tc_fence_after();
        mma_halves<D>(tmem + L::kAccCol, tmem, ym + st * kStep, i > 0);
        warp_commit(g_empty + st);
        if (more) {  // (in order: over P once dV has read it)
          mma_nt<D>(tmem, dk, xk + s1 * kStep);
          warp_commit(s_full);
          if (!(ok = warp_wait(g_full + s1, ph1, abort_flag, a.status))) break;
        }
        if (!(ok = warp_wait(ds_full, i & 1, abort_flag, a.status))) break;
        tc_fence_after();
        mma_halves<D>(tmem + L::kAccCol + D, tmem + L::kDPCol, xm + st * kStep, i > 0);
        warp_commit(q_empty + st);
        if (more) {
          mma_nt<D>(tmem + L::kDPCol, dv, yk + s1 * kStep);
          warp_commit(dp_full);
        }
      }
      warp_commit(done);
      if (__any_sync(0xffffffffu, *abort_flag != 0)) drain_bar(done, 0);
    }
  } else {
    // ---- thread = key r, 64 query columns ----
    const int half = warp >> 2, r = tid & (kTile - 1), key = k0 + r;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + half * 64, tp = ts + L::kDPCol;
    const float sl = pb.scale * kLog2e;
    const float2 sl2 = make_float2(sl, sl);
    bool ok = true;
    int q0 = first * kTile;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      const float* lse2 = rows + st * 256 + half * 64;
      const float* delta = lse2 + kTile;
      if (!(ok = mbar_wait(row_full + st, (i >> 1) & 1, abort_flag, a.status))) break;
      if (!(ok = mbar_wait(s_full, i & 1, abort_flag, a.status))) break;
      tc_fence_after();
      float p[64];
      load_half(ts, p);
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
        const float4 l = *reinterpret_cast<const float4*>(lse2 + e);
        const float2 u = fma2(make_float2(p[e], p[e + 1]), sl2, make_float2(-l.x, -l.y));
        const float2 w = fma2(make_float2(p[e + 2], p[e + 3]), sl2, make_float2(-l.z, -l.w));
        p[e] = ex2(u.x);
        p[e + 1] = ex2(u.y);
        p[e + 2] = ex2(w.x);
        p[e + 3] = ex2(w.y);
      }
      // the first column whose query sees this key, and the end of the queries:
      // the zeros behind them times an infinite key are NaN (two selections; one
      // over both ends slows every tile, 12 heads of 4680 238 -> 269 us)
      const int lo = (key >= len ? kTile : pb.causal ? key - shift - q0 : 0) - half * 64;
      const int hi = pb.Nq - q0 - half * 64;
      const bool masked = k0 + kTile > len || (pb.causal && k0 + kTile - 1 > q0 + shift);
      if (masked) {
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e < lo) p[e] = 0.f;
      }
      if (hi < 64) {
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e >= hi) p[e] = 0.f;
      }
      store_half(ts, p);
      tmem_wait_st();
      warp_arrive(p_full);
      if (!(ok = mbar_wait(dp_full, i & 1, abort_flag, a.status))) break;
      tc_fence_after();
      float d[64];
      load_half(tp, d);
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
        const float4 l = *reinterpret_cast<const float4*>(delta + e);
        d[e] = p[e] * (d[e] - l.x);
        d[e + 1] = p[e + 1] * (d[e + 1] - l.y);
        d[e + 2] = p[e + 2] * (d[e + 2] - l.z);
        d[e + 3] = p[e + 3] * (d[e + 3] - l.w);
      }
      if (masked) {  // what lies past the length may be NaN: selected away, not multiplied
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e < lo) d[e] = 0.f;
      }
      if (hi < 64) {
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e >= hi) d[e] = 0.f;
      }
      store_half(tp, d);
      tmem_wait_st();
      warp_arrive(ds_full);
      q0 = q0 + kTile < pb.Nq ? q0 + kTile : first * kTile;
    }
    if (ok && n > 0) ok = mbar_wait(done, 0, abort_flag, a.status);
    tc_fence_after();
    // dV (warps 0-3) and dK (warps 4-7) through the tiles of K and V; a tile
    // that no query sees gets zeros
    uint8_t* so = smem + (half ? L::kBOff : L::kAOff);
    if (ok) {
      accumulator_row<D>(so, r, tmem + lane_off + L::kAccCol + half * D, half ? pb.scale : 1.f,
                         n > 0);
      fence_proxy_async_smem();
    }
    named_barrier(1 + half, kTile);
    if (r == 0 && ok && !*abort_flag) {
      for (int c = 0; c < L::kCh; ++c)
        if (c * 64 < pb.d)
          tma_store_4d(half ? &mdk.map : &mdv.map, so + c * kChunk, c * 64, k0, hk, b);
      bulk_commit();
      bulk_wait_read<0>();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// dQ of 128 queries of a head: dQ = scale sum over the key tiles of dS K,
// dS = P (dO V^T - delta).  P stays in registers, so the next S starts as soon
// as this one is read, and runs beside its exponentials.
// TWICE: a first walk over the same tiles sums delta from P (dO V^T) and leaves
// it for dK and dV, too.
struct DqTile {
  int h, b, hk, q0, len, n, tail;  // n key tiles, the last with `tail` rows up to the length
};

template <int D, bool TWICE>
__device__ __forceinline__ void dq_tile(uint8_t* smem, uint32_t tmem, const TileMap& mq,
                                        const TileMap& mk, const TileMap& mv, const TileMap& mg,
                                        const TileMap& mdq, const BwdArgs& a, const DqTile& x,
                                        int warp) {
  using L = BwdLayout<D>;
  const int tid = threadIdx.x, lane = tid & 31;
  const DenseProblem& pb = a.pb;
  const int n = x.n, q0 = x.q0, steps = TWICE ? 2 * n : n;
  auto key_tile_of = [&](int j) { return TWICE && j >= n ? j - n : j; };
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* qg_full = bars;
  uint64_t* k_full = bars + 1;   // [stages]
  uint64_t* v_full = bars + 3;
  uint64_t* k_empty = bars + 5;
  uint64_t* v_empty = bars + 7;
  uint64_t* k_tail = bars + 9;
  uint64_t* s_full = bars + 10;
  uint64_t* s_read = bars + 11;
  uint64_t* dp_full = bars + 12;
  uint64_t* ds_full = bars + 13;
  uint64_t* done = bars + 14;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 16);

  if (warp == 8) {
    // ---- TMA: Q and dO, then K and V tile by tile ----
    bool ok = true;
    int kt = 0, vt = 0;
    if (lane == 0 && n > 0) {
      mbar_arrive_expect_tx(qg_full, 2 * L::kTileBytes);
      load_tile<D>(smem + L::kAOff, mq, qg_full, q0, x.h, x.b);
      load_tile<D>(smem + L::kBOff, mg, qg_full, q0, x.h, x.b);
      for (int j = 0; j < steps; ++j) {
        const int st = j & 1, row = key_tile_of(j) * kTile;
        const uint32_t par = ((j >> 1) - 1) & 1;
        if (j >= 2 && !(ok = mbar_wait(k_empty + st, par, abort_flag, a.status))) break;
        mbar_arrive_expect_tx(k_full + st, L::kTileBytes);
        load_tile<D>(smem + L::kXOff + st * L::kTileBytes, mk, k_full + st, row, x.hk, x.b);
        kt = j + 1;
        if (j >= 2 && !(ok = mbar_wait(v_empty + st, par, abort_flag, a.status))) break;
        mbar_arrive_expect_tx(v_full + st, L::kTileBytes);
        load_tile<D>(smem + L::kYOff + st * L::kTileBytes, mv, v_full + st, row, x.hk, x.b);
        vt = j + 1;
      }
    }
    __syncwarp();
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok && n > 0 && x.tail < kTile) {
      // keys past the length may hold anything (0 x NaN): zeros in their place
      // (a first walk selects their products away)
      const int st = (steps - 1) & 1;
      if (mbar_wait(k_full + st, ((steps - 1) >> 1) & 1, abort_flag, a.status)) {
        uint8_t* sk = smem + L::kXOff + st * L::kTileBytes;
        for (int y = lane; y < (kTile - x.tail) * L::kCh * 8; y += 32)
          *row_unit(sk, x.tail + y / (L::kCh * 8), y % (L::kCh * 8)) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_tail);
      }
    }
    if (lane == 0 && n > 0 && *abort_flag) {
      drain_bar(qg_full, 0);
      for (int s = 0; s < L::kStages; ++s) {
        if (kt > s) drain_bar(k_full + s, ((kt - 1 - s) >> 1) & 1);
        if (vt > s) drain_bar(v_full + s, ((vt - 1 - s) >> 1) & 1);
      }
    }
  } else if (warp == 9) {
    // ---- MMA issue ----
    if (n > 0) {
      const uint64_t dq = desc_kmajor(smem_u32(smem + L::kAOff));
      const uint64_t dg = desc_kmajor(smem_u32(smem + L::kBOff));
      const uint64_t xk = desc_kmajor(smem_u32(smem + L::kXOff));
      const uint64_t yk = desc_kmajor(smem_u32(smem + L::kYOff));
      const uint64_t xm = desc_mnmajor(smem_u32(smem + L::kXOff), kChunk);
      constexpr uint64_t kStep = L::kTileBytes >> 4;
      auto key_tile = [&](int j) {
        return warp_wait(k_full + (j & 1), (j >> 1) & 1, abort_flag, a.status) &&
               (j + 1 < steps || x.tail == kTile || warp_wait(k_tail, 0, abort_flag, a.status));
      };
      bool ok = warp_wait(qg_full, 0, abort_flag, a.status) && key_tile(0);
      if (ok) {
        mma_nt<D>(tmem, dq, xk);
        warp_commit(s_full);
        ok = warp_wait(v_full, 0, abort_flag, a.status);
      }
      if (ok) {
        mma_nt<D>(tmem + L::kDPCol, dg, yk);
        warp_commit(dp_full);
        warp_commit(v_empty);
      }
#pragma unroll 1
      for (int j = 0; j < steps && ok; ++j) {
        const int st = j & 1, s1 = st ^ 1;
        const bool more = j + 1 < steps;
        if (more) {
          if (!(ok = key_tile(j + 1) && warp_wait(s_read, j & 1, abort_flag, a.status))) break;
          tc_fence_after();
          mma_nt<D>(tmem, dq, xk + s1 * kStep);
          warp_commit(s_full);
          if (!(ok = warp_wait(v_full + s1, ((j + 1) >> 1) & 1, abort_flag, a.status))) break;
        }
        if (!(ok = warp_wait(ds_full, j & 1, abort_flag, a.status))) break;
        tc_fence_after();
        if (!TWICE || j >= n)
          mma_halves<D>(tmem + L::kAccCol, tmem + L::kDPCol, xm + st * kStep, key_tile_of(j) > 0);
        warp_commit(k_empty + st);
        if (more) {  // (in order: over dS once dQ has read it)
          mma_nt<D>(tmem + L::kDPCol, dg, yk + s1 * kStep);
          warp_commit(dp_full);
          warp_commit(v_empty + s1);
        }
      }
      warp_commit(done);
      if (__any_sync(0xffffffffu, *abort_flag != 0)) drain_bar(done, 0);
    }
  } else {
    // ---- thread = query r, 64 key columns ----
    const int half = warp >> 2, r = tid & (kTile - 1), row = q0 + r;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + half * 64, tp = ts + L::kDPCol;
    const int vis = dense_visible(pb, x.len, row), all = dense_visible(pb, x.len, q0);
    const long at = ((long)x.b * pb.H + x.h) * pb.Nq + row;
    const bool live = row < pb.Nq && vis > 0;
    const float lse2 = live ? dense_lse2(__ldg(a.lse + at)) : INFINITY;
    const float sl = pb.scale * kLog2e;
    const float2 sl2 = make_float2(sl, sl), base2 = make_float2(-lse2, -lse2);
    // d = P (dO V^T - delta) of step j, hidden keys zero; P and dP are read
    auto weights = [&](int j, float2 nd2, float (&d)[64]) -> bool {
      if (!mbar_wait(s_full, j & 1, abort_flag, a.status)) return false;
      tc_fence_after();
      float p[64];
      load_half(ts, p);
      warp_arrive(s_read);
#pragma unroll
      for (int e = 0; e < 64; e += 2) {
        const float2 u = fma2(make_float2(p[e], p[e + 1]), sl2, base2);
        p[e] = ex2(u.x);
        p[e + 1] = ex2(u.y);
      }
      if (!mbar_wait(dp_full, j & 1, abort_flag, a.status)) return false;
      tc_fence_after();
      load_half(tp, d);
#pragma unroll
      for (int e = 0; e < 64; e += 2) {
        const float2 u = mul2(make_float2(p[e], p[e + 1]),
                              add2(make_float2(d[e], d[e + 1]), nd2));
        d[e] = u.x;
        d[e + 1] = u.y;
      }
      const int k0 = key_tile_of(j) * kTile;
      if (k0 + kTile > all) {  // hidden keys, whatever the products hold
        const int lim = vis - k0 - half * 64;
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e >= lim) d[e] = 0.f;
      }
      return true;
    };
    bool ok = true;
    float delta = 0.f;
    if (TWICE) {
      float sum = 0.f;
      for (int j = 0; j < n; ++j) {
        float d[64];
        if (!(ok = weights(j, make_float2(0.f, 0.f), d))) break;
#pragma unroll
        for (int e = 0; e < 64; ++e) sum += d[e];
        warp_arrive(ds_full);
      }
      float* rows = reinterpret_cast<float*>(smem + L::kRowOff);
      rows[half * kTile + r] = sum;
      named_barrier(2, 2 * kTile);
      delta = rows[r] + rows[kTile + r];
      if (half == 0 && ok && row < pb.Nq) a.delta[at] = delta;
    } else if (live) {
      delta = __ldg(a.delta + at);
    }
    const float2 nd2 = make_float2(-delta, -delta);
    for (int j = TWICE ? n : 0; j < steps && ok; ++j) {
      float d[64];
      if (!(ok = weights(j, nd2, d))) break;
      store_half(tp, d);
      tmem_wait_st();
      warp_arrive(ds_full);
    }
    if (ok && n > 0) ok = mbar_wait(done, 0, abort_flag, a.status);
    tc_fence_after();
    if (half == 0) {
      uint8_t* so = smem + L::kAOff;
      if (ok) {
        accumulator_row<D>(so, r, tmem + lane_off + L::kAccCol, pb.scale, n > 0);
        fence_proxy_async_smem();
      }
      named_barrier(1, kTile);
      if (r == 0 && ok && !*abort_flag) {
        for (int c = 0; c < L::kCh; ++c)
          if (c * 64 < pb.d) tma_store_4d(&mdq.map, so + c * kChunk, c * 64, q0, x.h, x.b);
        bulk_commit();
        bulk_wait_read<0>();
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    dense_dq_tc_kernel(const __grid_constant__ TileMap mq, const __grid_constant__ TileMap mk,
                       const __grid_constant__ TileMap mv, const __grid_constant__ TileMap mg,
                       const __grid_constant__ TileMap mdq, const __grid_constant__ BwdArgs a) {
  using L = BwdLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) atomicExch(a.status, 2);
    return;
  }
  const DenseProblem& pb = a.pb;
  const int heads = pb.B * pb.H;
  const int tile = pb.causal ? a.tiles - 1 - blockIdx.x / heads : blockIdx.x % a.tiles;
  const int bh = pb.causal ? blockIdx.x % heads : blockIdx.x / a.tiles;
  DqTile x;
  x.h = bh % pb.H;
  x.b = bh / pb.H;
  x.hk = x.h / (pb.H / pb.Hkv);
  x.q0 = tile * kTile;
  x.len = dense_len(pb, x.b);
  x.n = (dense_visible(pb, x.len, min(x.q0 + kTile, pb.Nq) - 1) + kTile - 1) / kTile;
  x.tail = x.n * kTile > x.len && x.len < pb.Nk ? x.len - (x.n - 1) * kTile : kTile;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 15);
  if (tid == 0) {
    for (int i = 0; i < 15; ++i)  // (as dq_tile names them)
      mbar_init(bars + i, i == 11 || i == 13 ? 8 : 1);
    *reinterpret_cast<volatile int*>(bars + 16) = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  if (x.n <= kExactTiles)
    dq_tile<D, true>(smem, tmem, mq, mk, mv, mg, mdq, a, x, warp);
  else
    dq_tile<D, false>(smem, tmem, mq, mk, mv, mg, mdq, a, x, warp);
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// Map of a (B, H, N, d) tensor with boxes of 128 rows x 64 channels.
bool make_tile_map(TileMap* m, const void* base, const HeadStrides& s, int B, int H, int N,
                   int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  // a stride of 0 (one entry, or a broadcast) never enters an address
  m->h_mul = s.h != 0;
  m->b_mul = s.b != 0;
  const cuuint64_t row = (cuuint64_t)(s.n ? s.n : d) * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)(s.h ? H : 1),
                              (cuuint64_t)(s.b ? B : 1)};
  const cuuint64_t str[3] = {row, s.h ? (cuuint64_t)s.h * 2 : row, s.b ? (cuuint64_t)s.b * 2 : row};
  const cuuint32_t box[4] = {64, kTile, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(&m->map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, str, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Ranges of the keys: as many as fill the CTA slots of the SMs (where the
// queries alone leave half of them empty or more), of at least four tiles:
// fewer do not pay for writing and reading a range's result.
KeySplit split_keys(const DenseProblem& pb) {
  const int tiles = pb.d <= 64 ? FwdLayout<64>::kTiles : FwdLayout<128>::kTiles;
  const long ctas = (long)((pb.Nq + tiles * kTile - 1) / (tiles * kTile)) * pb.H * pb.B;
  return split_of(pb, (pb.Nk + kTile - 1) / kTile, ctas, (3 - tiles) * (long)num_sms(), 4);
}

template <int D>
cudaError_t forward_d(const TileMap& mq, const TileMap& mk, const TileMap& mv, const TileMap& mo,
                      bf16* out, FwdArgs a, cudaStream_t stream, int* launches) {
  using L = FwdLayout<D>;
  cudaError_t e = allow_smem<dense_fwd_tc_kernel<D>>(L::kBytes);
  if (e != cudaSuccess) return e;
  a.tiles = (a.pb.Nq + L::kTiles * kTile - 1) / (L::kTiles * kTile);
  const unsigned grid = (unsigned)a.tiles * a.pb.H * a.pb.B * a.split.splits;
  e = timed_launch("dense_fwd_tc", stream, launches, [&] {
    dense_fwd_tc_kernel<D><<<grid, L::kThreads, L::kBytes, stream>>>(mq, mk, mv, mo, a);
  });
  if (e != cudaSuccess || a.split.splits == 1) return e;
  return dense_join<bf16>(out, a.lse, a.pb, a.split, stream, launches);
}

template <int D>
cudaError_t backward_d(const TileMap& mq, const TileMap& mk, const TileMap& mv, const TileMap& mg,
                       const TileMap& mdq, const TileMap& mdk, const TileMap& mdv, BwdArgs a,
                       cudaStream_t stream, int* launches) {
  using L = BwdLayout<D>;
  cudaError_t e;
  auto dq = [&] {
    if ((e = allow_smem<dense_dq_tc_kernel<D>>(L::kBytes)) != cudaSuccess) return e;
    a.tiles = (a.pb.Nq + kTile - 1) / kTile;
    return timed_launch("dense_dq_tc", stream, launches, [&] {
      dense_dq_tc_kernel<D><<<(unsigned)a.tiles * a.pb.H * a.pb.B, kBwdThreads, L::kBytes,
                              stream>>>(mq, mk, mv, mg, mdq, a);
    });
  };
  auto dkv = [&] {
    if ((e = allow_smem<dense_dkv_tc_kernel<D>>(L::kBytes)) != cudaSuccess) return e;
    a.tiles = (a.pb.Nk + kTile - 1) / kTile;
    return timed_launch("dense_dkv_tc", stream, launches, [&] {
      dense_dkv_tc_kernel<D><<<(unsigned)a.tiles * a.pb.Hkv * a.pb.B, kBwdThreads, L::kBytes,
                               stream>>>(mq, mk, mv, mg, mdk, mdv, a);
    });
  };
  // dQ first where its short tiles give delta; else last, for dK and dV behind
  // it take up to 7% longer (12 heads of 4680: 240 us, behind dQ 242 to 261,
  // with where the tensors lie)
  const bool dq_first = a.pb.Nk <= kExactTiles * kTile || a.pb.causal || a.pb.k_lens;
  if ((e = dq_first ? dq() : dkv()) != cudaSuccess) return e;
  return dq_first ? dkv() : dq();
}

}  // namespace

bool dense_tc_rows(const void* p, const HeadStrides& s, int N, int d) {
  constexpr long kTop = 1L << 38;  // map strides end at 2^40 bytes
  return d % 8 == 0 && d <= 128 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && s.b % 8 == 0 &&
         s.h % 8 == 0 && s.n % 8 == 0 && (N == 1 || s.n >= d) && s.b < kTop && s.h < kTop &&
         s.n < kTop;
}

size_t dense_tc_workspace_bytes(const DenseProblem& pb) {
  if (pb.d % 8 || pb.d > 128 || pb.Nq == 0 || pb.Nk == 0) return 0;
  return split_bytes(pb, split_keys(pb));
}

cudaError_t dense_tc_forward(const bf16* q, const bf16* k, const bf16* v, bf16* out, float* lse,
                             const DenseProblem& pb, float* workspace, int* status,
                             cudaStream_t stream, int* launches) {
  TileMap mq, mk, mv, mo;
  if (!make_tile_map(&mq, q, pb.q, pb.B, pb.H, pb.Nq, pb.d) ||
      !make_tile_map(&mk, k, pb.k, pb.B, pb.Hkv, pb.Nk, pb.d) ||
      !make_tile_map(&mv, v, pb.v, pb.B, pb.Hkv, pb.Nk, pb.d) ||
      !make_tile_map(&mo, out, pb.out, pb.B, pb.H, pb.Nq, pb.d))
    return cudaErrorInvalidValue;
  FwdArgs a = {};
  a.lse = lse;
  a.pb = pb;
  a.status = status;
  a.split = split_keys(pb);
  place_split(pb, workspace, &a.split);
  return pb.d <= 64 ? forward_d<64>(mq, mk, mv, mo, out, a, stream, launches)
                    : forward_d<128>(mq, mk, mv, mo, out, a, stream, launches);
}

cudaError_t dense_tc_backward(const bf16* q, const bf16* k, const bf16* v, const bf16* out,
                              const float* lse, const bf16* dout, bf16* dq, bf16* dk, bf16* dv,
                              float* delta, const DenseProblem& pb, int* status,
                              cudaStream_t stream, int* launches) {
  TileMap mq, mk, mv, mg, mdq, mdk, mdv;
  if (!make_tile_map(&mq, q, pb.q, pb.B, pb.H, pb.Nq, pb.d) ||
      !make_tile_map(&mk, k, pb.k, pb.B, pb.Hkv, pb.Nk, pb.d) ||
      !make_tile_map(&mv, v, pb.v, pb.B, pb.Hkv, pb.Nk, pb.d) ||
      !make_tile_map(&mg, dout, pb.dout, pb.B, pb.H, pb.Nq, pb.d) ||
      !make_tile_map(&mdq, dq, pb.dq, pb.B, pb.H, pb.Nq, pb.d) ||
      !make_tile_map(&mdk, dk, pb.dk, pb.B, pb.Hkv, pb.Nk, pb.d) ||
      !make_tile_map(&mdv, dv, pb.dv, pb.B, pb.Hkv, pb.Nk, pb.d))
    return cudaErrorInvalidValue;
  if (pb.Nk > kExactTiles * kTile) {  // some tiles may be longer
    const cudaError_t e = dense_delta<bf16>(out, dout, delta, pb, stream, launches);
    if (e != cudaSuccess) return e;
  }
  const BwdArgs a = {lse, delta, pb, 0, status};
  return pb.d <= 64
             ? backward_d<64>(mq, mk, mv, mg, mdq, mdk, mdv, a, stream, launches)
             : backward_d<128>(mq, mk, mv, mg, mdq, mdk, mdv, a, stream, launches);
}

}  // namespace monarch
