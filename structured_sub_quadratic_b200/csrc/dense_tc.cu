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

// 16-byte unit u (channels 8u ..) of row r of a tile of swizzled 64-channel chunks.
__device__ __forceinline__ uint4* row_unit(uint8_t* tile, int r, int u) {
  return reinterpret_cast<uint4*>(tile + (u >> 3) * kChunk + r * 128 + (((u & 7) ^ (r & 7)) << 4));
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

// D[tmem] (+)= A B^T over D channels, both tiles K-major in shared memory.
template <int D>
__device__ __forceinline__ void mma_nt(uint32_t tmem, uint64_t a, uint64_t b) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * kChunk + (kk & 3) * 32) >> 4;
    mma_bf16_ss(tmem, a + off, b + off, idesc_bf16(kTile, kTile, false), kk > 0 ? 1u : 0u);
  }
}

// D[tmem] (+)= W X: W 128 x 128 bf16 in TMEM, X a tile of 128 rows x D channels.
template <int D>
__device__ __forceinline__ void mma_ts(uint32_t tmem, uint32_t w_tmem, uint64_t x,
                                       bool accumulate) {
#pragma unroll
  for (int kk = 0; kk < kTile / 16; ++kk)
    mma_bf16_ts(tmem, w_tmem + kk * 8, x + ((kk * 16 * 128) >> 4), idesc_bf16(kTile, D, true),
                accumulate || kk > 0 ? 1u : 0u);
}

// ---------------------------------------------------------------------------
// Forward.  One CTA per 256 queries of a head: two 128-row tiles whose
// softmaxes (one warpgroup each, a thread per row) and products alternate, so
// that one tile's S = Q K^T and O += P V run while the other's exponentials
// do.  One pass over the keys: O stays in TMEM under a running maximum that
// only moves when it grows by more than 2^8 (probabilities then reach 256,
// exact in the bf16 of P as well as in the fp32 sum), so rescaling O is rare.
// P overwrites S in TMEM and is the A operand of P V.
// Warps: 0-3 and 4-7 softmax of tile 0 and 1, 8 TMA, 9 MMA.
// ---------------------------------------------------------------------------
template <int D>
struct FwdLayout {
  static constexpr int kCh = D / 64, kStages = D == 128 ? 2 : 3;
  static constexpr int kTileBytes = kCh * kChunk;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kBarOff = kVOff + kStages * kTileBytes;
  static constexpr int kBytes = kBarOff + 32 * 8;
  static constexpr uint32_t kTmemCols = 512, kOCol = 256;  // S 0, S 1, then O 0, O 1
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct FwdArgs {
  float* lse;
  DenseProblem pb;
  int tiles;  // 256-row tiles of a head
  int* status;
};

constexpr int kFwdThreads = 320;

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
    dense_fwd_tc_kernel(const __grid_constant__ TileMap mq, const __grid_constant__ TileMap mk,
                        const __grid_constant__ TileMap mv, const __grid_constant__ TileMap mo,
                        const __grid_constant__ FwdArgs a) {
  using L = FwdLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // swizzled tiles need 1024-B alignment: report, never fault
    if (tid == 0) atomicExch(a.status, 2);
    return;
  }
  const DenseProblem& pb = a.pb;
  // causal: the longest tiles first, over all heads; else head by head
  int tile, bh;
  if (pb.causal) {
    bh = blockIdx.x % (pb.B * pb.H);
    tile = a.tiles - 1 - blockIdx.x / (pb.B * pb.H);
  } else {
    tile = blockIdx.x % a.tiles;
    bh = blockIdx.x / a.tiles;
  }
  const int h = bh % pb.H, b = bh / pb.H, hk = h / (pb.H / pb.Hkv);
  const int q0 = tile * 2 * kTile;
  const int len = dense_len(pb, b);
  // key tiles of the two row tiles, and the last one's rows past the length
  int nt[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int r0 = q0 + t * kTile;
    nt[t] = r0 < pb.Nq
                ? (dense_visible(pb, len, min(r0 + kTile, pb.Nq) - 1) + kTile - 1) / kTile
                : 0;
  }
  const int n = max(nt[0], nt[1]);
  const int tail = n * kTile > len && len < pb.Nk ? len - (n - 1) * kTile : kTile;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* q_full = bars;         // [2]
  uint64_t* s_full = bars + 2;     // [2]
  uint64_t* p_full = bars + 4;     // [2]
  uint64_t* o_full = bars + 6;     // [2]
  uint64_t* k_full = bars + 8;     // [stages]
  uint64_t* k_empty = bars + 11;
  uint64_t* v_full = bars + 14;
  uint64_t* v_empty = bars + 17;
  uint64_t* v_tail = bars + 20;
  uint64_t* drain = bars + 21;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 22);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 23);
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full + t, 1);
      mbar_init(s_full + t, 1);
      mbar_init(p_full + t, kTile);
      mbar_init(o_full + t, 1);
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
  if (warp == 9) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    // ---- TMA: Q, then K and V tile by tile ----
    bool ok = true;
    int kt = 0, vt = 0;  // tiles issued
    if (lane == 0) {
      tma_prefetch_desc(&mq.map);
      tma_prefetch_desc(&mk.map);
      tma_prefetch_desc(&mv.map);
      for (int t = 0; t < 2; ++t)
        if (q0 + t * kTile < pb.Nq) {
          mbar_arrive_expect_tx(q_full + t, L::kTileBytes);
          load_tile<D>(smem + L::kQOff + t * L::kTileBytes, mq, q_full + t, q0 + t * kTile, h, b);
        }
      for (int j = 0; j < n; ++j) {
        const int st = j % L::kStages;
        const uint32_t par = (j / L::kStages - 1) & 1;
        if (j >= L::kStages && !(ok = mbar_wait(k_empty + st, par, abort_flag, a.status))) break;
        mbar_arrive_expect_tx(k_full + st, L::kTileBytes);
        load_tile<D>(smem + L::kKOff + st * L::kTileBytes, mk, k_full + st, j * kTile, hk, b);
        kt = j + 1;
        if (j >= L::kStages && !(ok = mbar_wait(v_empty + st, par, abort_flag, a.status))) break;
        mbar_arrive_expect_tx(v_full + st, L::kTileBytes);
        load_tile<D>(smem + L::kVOff + st * L::kTileBytes, mv, v_full + st, j * kTile, hk, b);
        vt = j + 1;
      }
    }
    __syncwarp();
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok && tail < kTile) {
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
      for (int t = 0; t < 2; ++t)
        if (q0 + t * kTile < pb.Nq) drain_bar(q_full + t, 0);
      for (int s = 0; s < L::kStages; ++s) {
        if (kt > s) drain_bar(k_full + s, ((kt - 1 - s) / L::kStages) & 1);
        if (vt > s) drain_bar(v_full + s, ((vt - 1 - s) / L::kStages) & 1);
      }
    }
  } else if (warp == 9) {
    // ---- MMA issue ----
    if (lane == 0 && n > 0) {
      uint64_t dq[2], dk[L::kStages], dv[L::kStages];
      for (int t = 0; t < 2; ++t)
        dq[t] = desc_kmajor(smem_u32(smem + L::kQOff + t * L::kTileBytes));
      for (int s = 0; s < L::kStages; ++s) {
        dk[s] = desc_kmajor(smem_u32(smem + L::kKOff + s * L::kTileBytes));
        dv[s] = desc_mnmajor(smem_u32(smem + L::kVOff + s * L::kTileBytes), kChunk);
      }
      bool ok = mbar_wait(k_full, 0, abort_flag, a.status);
      for (int t = 0; t < 2 && ok; ++t)
        if (nt[t] > 0 && (ok = mbar_wait(q_full + t, 0, abort_flag, a.status))) {
          mma_nt<D>(tmem + t * kTile, dq[t], dk[0]);
          mma_commit(s_full + t);
        }
      if (ok) mma_commit(k_empty);
      int st = 0, ph = 0;  // stage and phase of tile j
      for (int j = 0; j < n && ok; ++j) {
        const int s1 = st + 1 == L::kStages ? 0 : st + 1, ph1 = s1 ? ph : ph ^ 1;
        ok = mbar_wait(v_full + st, ph, abort_flag, a.status) &&
             (j + 1 < n || tail == kTile || mbar_wait(v_tail, 0, abort_flag, a.status));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || j >= nt[t]) continue;
          if (!(ok = mbar_wait(p_full + t, j & 1, abort_flag, a.status))) continue;
          tc_fence_after();
          mma_ts<D>(tmem + L::kOCol + t * D, tmem + t * kTile, dv[st], j > 0);
          if (j + 1 < nt[t]) {
            // the products of one thread run in order: S overwrites P once P V has read it
            if (!(ok = mbar_wait(k_full + s1, ph1, abort_flag, a.status))) continue;
            mma_nt<D>(tmem + t * kTile, dq[t], dk[s1]);
            mma_commit(s_full + t);  // also: P V of tile j is done
          } else {
            mma_commit(o_full + t);
          }
        }
        if (ok) {
          mma_commit(v_empty + st);
          if (j + 1 < n) mma_commit(k_empty + s1);
        }
        st = s1;
        ph = ph1;
      }
      if (*abort_flag) {
        mma_commit(drain);
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
    const int vis = dense_visible(pb, len, row);
    const int all = dense_visible(pb, len, r0);  // keys that every row of the tile sees
    const float sl = pb.scale * kLog2e;
    float m = -INFINITY, z = 0.f;
    bool ok = true;
    for (int j = 0; j < nj; ++j) {
      if (!(ok = mbar_wait(s_full + t, j & 1, abort_flag, a.status))) break;
      tc_fence_after();
      float s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, s[c]);
      tmem_wait_ld();
      if ((j + 1) * kTile > all) {
        const int lim = vis - j * kTile;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e >= lim) s[c][e] = -INFINITY;
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = fmaxf(s[c][0], s[c][1]);
#pragma unroll
        for (int e = 2; e < 32; e += 2) mx[c] = max3(mx[c], s[c][e], s[c][e + 1]);
      }
      const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
      if (j == 0) {
        m = mn;
      } else if (__any_sync(0xffffffffu, (mn - m) * sl > 8.f)) {
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
      const float2 sl2 = make_float2(sl, sl), base2 = make_float2(base, base);
      float2 zs = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float2 x = fma2(make_float2(s[c][e], s[c][e + 1]), sl2, base2);
          x.x = ex2(x.x);
          x.y = ex2(x.y);
          zs = add2(zs, x);
          pk[e / 2] = pack_bf16x2(x.x, x.y);
        }
        tmem_st16(ts + c * 16, pk);
      }
      z += zs.x + zs.y;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full + t);
    }
    if (r0 < pb.Nq) {
      // O / z to the tile of Q (read by every S of the tile), then one TMA store
      uint8_t* so = smem + L::kQOff + t * L::kTileBytes;
      if (ok) ok = mbar_wait(q_full + t, 0, abort_flag, a.status);
      if (ok && nj > 0) ok = mbar_wait(o_full + t, 0, abort_flag, a.status);
      tc_fence_after();
      const bool any = vis > 0;
      const float inv = 1.f / z;
      if (ok) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          if (nj > 0) {
            tmem_ld32(to + c * 32, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = any ? o[e] * inv : 0.f;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *row_unit(so, r, c * 4 + u) =
                make_uint4(pack_bf16x2(o[8 * u], o[8 * u + 1]),
                           pack_bf16x2(o[8 * u + 2], o[8 * u + 3]),
                           pack_bf16x2(o[8 * u + 4], o[8 * u + 5]),
                           pack_bf16x2(o[8 * u + 6], o[8 * u + 7]));
        }
        if (row < pb.Nq)
          a.lse[((long)b * pb.H + h) * pb.Nq + row] =
              any ? (m * sl + log2f(z)) * kLn2 : -INFINITY;
        fence_proxy_async_smem();
      }
      named_barrier(1 + t, kTile);
      if (r == 0 && ok && !*abort_flag) {
        for (int c = 0; c < L::kCh; ++c)
          if (c * 64 < pb.d) tma_store_4d(&mo.map, so + c * kChunk, c * 64, r0, h, b);
        bulk_commit();
        bulk_wait_read<0>();
      }
    }
  }
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

template <int D>
cudaError_t forward_d(const TileMap& mq, const TileMap& mk, const TileMap& mv, const TileMap& mo,
                      const FwdArgs& a, cudaStream_t stream, int* launches) {
  using L = FwdLayout<D>;
  const cudaError_t e = cudaFuncSetAttribute(
      dense_fwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)a.tiles * a.pb.H * a.pb.B;
  return timed_launch("dense_fwd_tc", stream, launches, [&] {
    dense_fwd_tc_kernel<D><<<grid, kFwdThreads, L::kBytes, stream>>>(mq, mk, mv, mo, a);
  });
}

}  // namespace

bool dense_tc_rows(const void* p, const HeadStrides& s, int N, int d) {
  constexpr long kTop = 1L << 38;  // map strides end at 2^40 bytes
  return d % 8 == 0 && d <= 128 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && s.b % 8 == 0 &&
         s.h % 8 == 0 && s.n % 8 == 0 && (N == 1 || s.n >= d) && s.b < kTop && s.h < kTop &&
         s.n < kTop;
}

cudaError_t dense_tc_forward(const bf16* q, const bf16* k, const bf16* v, bf16* out, float* lse,
                             const DenseProblem& pb, int* status, cudaStream_t stream,
                             int* launches) {
  TileMap mq, mk, mv, mo;
  if (!make_tile_map(&mq, q, pb.q, pb.B, pb.H, pb.Nq, pb.d) ||
      !make_tile_map(&mk, k, pb.k, pb.B, pb.Hkv, pb.Nk, pb.d) ||
      !make_tile_map(&mv, v, pb.v, pb.B, pb.Hkv, pb.Nk, pb.d) ||
      !make_tile_map(&mo, out, pb.out, pb.B, pb.H, pb.Nq, pb.d))
    return cudaErrorInvalidValue;
  const FwdArgs a = {lse, pb, (pb.Nq + 2 * kTile - 1) / (2 * kTile), status};
  return pb.d <= 64 ? forward_d<64>(mq, mk, mv, mo, a, stream, launches)
                    : forward_d<128>(mq, mk, mv, mo, a, stream, launches);
}

}  // namespace monarch
