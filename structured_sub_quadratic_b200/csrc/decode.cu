// Exact softmax attention of one new token per sequence over a paged cache.
//
// The cache of a sequence is a list of pages; key j sits in row j % page_size
// of page table[b][j / page_size].  The keys are cut into chunks that CTAs
// take independently, each for the query heads that share its key/value head
// (so the cache is read once); a chunk gives its own maximum, sum and
// unnormalised output, and a second launch joins the chunks in order (no
// atomics).  One pass: every warp walks its tiles of a chunk under a running
// maximum, and the four warps of the CTA are joined in shared memory.
// Bound: the bytes of the cache.
#include "dense.cuh"

#include <math.h>

#include <algorithm>

#include "launch.cuh"
#include "tc_ptx.cuh"
#include "timing.cuh"

namespace monarch {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = 16;  // query heads of a CTA on the tensor cores (M of the product)

struct Split {
  int chunk;   // keys per chunk
  int chunks;  // chunks of the longest sequence that the table allows
};

// Chunks that fill the two CTA slots of each SM, of 128 keys at least (fewer do
// not fill the loads in flight of a CTA).  Where a chunk is then still longer
// than 1024 keys, up to four waves of CTAs, for lengths differ (12 to 32 waves
// measured the same); shorter chunks lose to the start of a CTA, about 3 us (32
// sequences of 1000 keys over 8 heads: 27 us in whole sequences, 40 us in
// chunks of 256).  Up to 256 keys are one chunk, whose CTA writes the result
// itself (12 heads of 250 keys: 5.8 us, in two chunks and a join 6.4; of 500
// keys 9.1 and 6.4).
Split make_split(const DecodeProblem& pb) {
  const long top = (long)pb.max_pages * pb.page_size;
  const long units = (long)pb.B * pb.Hkv * ((pb.H / pb.Hkv + kRows - 1) / kRows);
  long n = std::max(1L, std::min((top + 127) / 128, 2L * num_sms() / units));
  if (top > 1024 * n) n = std::max(n, std::min((top + 1023) / 1024, 8L * num_sms() / units));
  if (top <= 256) n = 1;
  Split s;
  s.chunk = (int)(((top + n - 1) / n + 127) / 128 * 128);
  s.chunk = std::max(s.chunk, 128);
  s.chunks = (int)std::max(1L, (top + s.chunk - 1) / s.chunk);
  return s;
}

struct Parts {
  float2* ml;  // [chunk][b][h]: maximum in log2 units, sum
  float* o;    // [chunk][b][h][d], unnormalised
};

// One CTA's share: heads [h0, h0 + nh) of sequence b over keys [j0, j1).
struct Share {
  int b, hk, h0, nh, c, j0, j1;
};

__device__ __forceinline__ Share share_of(const DecodeProblem& pb, const Split& sp, int heads,
                                          int* status) {
  const int group = pb.H / pb.Hkv, hgs = (group + heads - 1) / heads;
  Share s;
  // heads first: where a token's heads lie side by side, they are read together
  int x = blockIdx.x;
  const int hg = x % hgs;
  x /= hgs;
  s.hk = x % pb.Hkv;
  x /= pb.Hkv;
  s.c = x % sp.chunks;
  s.b = x / sp.chunks;
  s.h0 = s.hk * group + hg * heads;
  s.nh = min(heads, (s.hk + 1) * group - s.h0);
  const int n = __ldg(pb.lens + s.b), top = pb.max_pages * pb.page_size;
  if (n < 0 || n > top) atomicCAS(status, 0, MONARCH_DEVICE_BAD_INDEX_FLAG);
  s.j0 = s.c * sp.chunk;
  s.j1 = min(min(max(n, 0), top), s.j0 + sp.chunk);
  return s;
}

// Page and row of key j, page -1 where there is none (its score is masked) or it
// lies outside the cache (which is recorded; the key and value are zeros).
__device__ __forceinline__ int2 place(const DecodeProblem& pb, const Share& s, int j,
                                      int* status) {
  if (j >= s.j1) return make_int2(-1, 0);
  const int p = j / pb.page_size;
  int page = __ldg(pb.table + (long)s.b * pb.max_pages + p);
  if (page < 0 || page >= pb.n_pages) {
    atomicCAS(status, 0, MONARCH_DEVICE_BAD_INDEX_FLAG);
    page = -1;
  }
  return make_int2(page, j - p * pb.page_size);
}

// The four warps' results (m, z per head and o[head][channel], in shared
// memory, warps `o_step` floats apart) joined and written: as a part, or as
// the result itself where one chunk holds every sequence.
template <typename T>
__device__ __forceinline__ void join_warps(const float (*m)[kRows], const float (*z)[kRows],
                                           const float* o, int o_step, int pitch,
                                           const DecodeProblem& pb, const Split& sp,
                                           const Share& s, Parts part, T* out, float* lse) {
  const long row0 = (long)s.b * pb.H + s.h0;
  for (int x = threadIdx.x; x < s.nh * pb.d; x += kThreads) {
    const int h = x / pb.d, e = x % pb.d;
    float mm = m[0][h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, m[w][h]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float zz = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(m[w][h] - base);
      zz = fmaf(z[w][h], f, zz);
      acc = fmaf(o[w * o_step + h * pitch + e], f, acc);
    }
    if (sp.chunks == 1) {  // (zz 0: every key scores -inf, as if there were none)
      out[s.b * pb.out_b + (s.h0 + h) * pb.out_h + e] = from_f32<T>(zz == 0.f ? 0.f : acc / zz);
      if (e == 0) lse[row0 + h] = (mm + log2f(zz)) * kLn2;
    } else {
      const long at = (long)s.c * pb.B * pb.H + row0 + h;
      part.o[at * pb.d + e] = acc;
      if (e == 0) part.ml[at] = make_float2(mm, zz);
    }
  }
}

// An empty sequence's only chunk.
template <typename T>
__device__ __forceinline__ void write_empty(const DecodeProblem& pb, const Share& s, T* out,
                                            float* lse) {
  for (int x = threadIdx.x; x < s.nh * pb.d; x += kThreads) {
    const int h = x / pb.d, e = x % pb.d;
    out[s.b * pb.out_b + (s.h0 + h) * pb.out_h + e] = from_f32<T>(0.f);
    if (e == 0) lse[(long)s.b * pb.H + s.h0 + h] = -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// bf16 rows of 16-byte alignment, d a multiple of 8 up to 128: 16 heads by 8
// keys products (the heads padded to 16 rows; the tensor cores have room to
// spare beside the loads).  Each warp streams its own tiles of 16 (d > 64) or
// 32 keys through three 8 KB slots by 16-byte asynchronous copies, without
// any barrier between the warps.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DP>
struct MmaTile {
  static constexpr int kKeys = 2048 / DP, kUnits = DP / 8;  // 16-byte units of a row
  static constexpr int kHalf = kKeys * DP * 2;              // bytes of K (or V) of a tile
  static constexpr int kStages = 3, kWarpBytes = kStages * 2 * kHalf;
  static constexpr int kPitch = DP + 4;
  static_assert(kRows * kPitch * 4 <= kWarpBytes, "the result reuses the warp's slots");
};

// WIDE: more than 8 heads (else rows 8-15 of the products are padding, and
// their softmax is left out).
template <int DP, bool WIDE>
__global__ void __launch_bounds__(kThreads)
    decode_mma_kernel(const bf16* __restrict__ q, const bf16* __restrict__ kc,
                      const bf16* __restrict__ vc, Parts part, bf16* __restrict__ out,
                      float* __restrict__ lse, DecodeProblem pb, Split sp, int* status) {
  using L = MmaTile<DP>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm[kWarps][kRows], sz[kWarps][kRows];
  if (sp.chunks > 1) tc::pdl_launch_dependents();  // the join
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Share s = share_of(pb, sp, kRows, status);
  if (s.j0 >= s.j1) {  // the join reads no chunk from the length on
    if (sp.chunks == 1) write_empty(pb, s, out, lse);
    return;
  }
  uint8_t* ring = smem + warp * L::kWarpBytes;
  const uint32_t ring32 = tc::smem_u32(ring);
  const int g = lane >> 2, t4 = lane & 3;
  // Q as A operands: rows g and g + 8 (heads), channels 16 kk + 2 t4 and + 8
  uint32_t qa[DP / 16][4];
  {
    const bf16* q0 = q + s.b * pb.q_b + s.h0 * pb.q_h;
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int h = g + (x & 1) * 8, e = kk * 16 + (x >> 1) * 8 + t4 * 2;
        qa[kk][x] = h < s.nh && e < pb.d
                        ? __ldg(reinterpret_cast<const unsigned int*>(q0 + h * pb.q_h + e))
                        : 0u;
      }
  }
  const int n = max(0, ((s.j1 - s.j0 + L::kKeys - 1) / L::kKeys - warp + kWarps - 1) / kWarps);
  auto tile_key = [&](int i) { return s.j0 + (warp + i * kWarps) * L::kKeys; };
  // Tiles start at multiples of their size: where pages hold whole tiles, one
  // entry of the table places a tile, and lanes step by a fixed stride.
  const bool whole = pb.page_size % L::kKeys == 0;
  auto lookup = [&](int i) {  // of the tile's first key, or of key `lane` of it
    return i < n ? place(pb, s, tile_key(i) + (whole ? 0 : lane & (L::kKeys - 1)), status)
                 : make_int2(-1, 0);
  };
  constexpr int kCopies = L::kKeys * L::kUnits / 32, kStep = 32 / L::kUnits;
  const int lr = lane / L::kUnits, lu = lane % L::kUnits;  // row and unit of the first copy
  const bf16* k0 = kc + s.hk * pb.k_h + lu * 8;
  const bf16* v0 = vc + s.hk * pb.v_h + lu * 8;
  const bool in_row = lu * 8 < pb.d;
  auto fetch = [&](int i, int2 at) {
    if (i < n) {
      const uint32_t dst = ring32 + (i % L::kStages) * 2 * L::kHalf;
      const int left = s.j1 - tile_key(i);
      if (whole && left >= L::kKeys && at.x >= 0) {
        const bf16* ks = k0 + at.x * pb.k_page + (at.y + lr) * pb.k_n;
        const bf16* vs = v0 + at.x * pb.v_page + (at.y + lr) * pb.v_n;
#pragma unroll
        for (int x = 0; x < kCopies; ++x) {
          const int r = x * kStep + lr;
          const uint32_t o = dst + r * DP * 2 + ((lu ^ (r & 7)) << 4);
          copy16(o, in_row ? ks : kc, in_row);
          copy16(o + L::kHalf, in_row ? vs : vc, in_row);
          ks += kStep * pb.k_n;
          vs += kStep * pb.v_n;
        }
      } else {
#pragma unroll 1
        for (int x = 0; x < kCopies; ++x) {
          const int r = x * kStep + lr;
          const int page = whole ? (r < left ? at.x : -1) : __shfl_sync(0xffffffffu, at.x, r);
          const int row = whole ? at.y + r : __shfl_sync(0xffffffffu, at.y, r);
          const bool there = page >= 0 && in_row;
          const uint32_t o = dst + r * DP * 2 + ((lu ^ (r & 7)) << 4);
          copy16(o, there ? k0 + page * pb.k_page + row * pb.k_n : kc, there);
          copy16(o + L::kHalf, there ? v0 + page * pb.v_page + row * pb.v_n : vc, there);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float o[DP / 8][4];
#pragma unroll
  for (int x = 0; x < DP / 8; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y) o[x][y] = 0.f;
  // heads g and g + 8: maximum of the raw products, sum
  float m0 = -INFINITY, m1 = -INFINITY, z0 = 0.f, z1 = 0.f;
  const float sl = pb.scale * kLog2e;
#pragma unroll
  for (int i = 0; i < L::kStages - 1; ++i) fetch(i, lookup(i));
  int2 next = lookup(L::kStages - 1);
  for (int i = 0; i < n; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 2) : "memory");
    __syncwarp();  // tile i is there for every lane, and tile i - 1 is read
    fetch(i + L::kStages - 1, next);
    next = lookup(i + L::kStages);
    const uint32_t sk = ring32 + (i % L::kStages) * 2 * L::kHalf, sv = sk + L::kHalf;
    const int left = s.j1 - tile_key(i);
    float c[L::kKeys / 8][4];
#pragma unroll
    for (int x = 0; x < L::kKeys / 8; ++x) {
#pragma unroll
      for (int y = 0; y < 4; ++y) c[x][y] = 0.f;
      const int r = x * 8 + (lane & 7);
#pragma unroll
      for (int kk = 0; kk < DP / 16; kk += 2) {  // four 8-channel blocks of 8 keys
        uint32_t kb[4];
        ldsm4(kb, sk + r * DP * 2 + (((kk * 2 + (lane >> 3)) ^ (r & 7)) << 4));
        mma16816(c[x], qa[kk], kb[0], kb[1]);
        mma16816(c[x], qa[kk + 1], kb[2], kb[3]);
      }
    }
    if (left < L::kKeys) {
#pragma unroll
      for (int x = 0; x < L::kKeys / 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (x * 8 + t4 * 2 + (y & 1) >= left) c[x][y] = -INFINITY;
    }
    float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
    for (int x = 0; x < L::kKeys / 8; ++x) {
      a0 = tc::max3(a0, c[x][0], c[x][1]);
      if (WIDE) a1 = tc::max3(a1, c[x][2], c[x][3]);
    }
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, x));
      if (WIDE) a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, x));
    }
    // The running maximum moves when it grows by 2^8 or more: weights then
    // reach 256, exact in bf16's and fp32's exponents.  The weights are rounded
    // to bf16 as operands of the product with V, half a step each like the result
    // (up to 8192 keys: error 2.3e-3 of it, 1.7e-3 from its own rounding alone);
    // their sum is of the unrounded ones.
    if (__any_sync(0xffffffffu, (a0 - m0) * sl > 8.f || (WIDE && (a1 - m1) * sl > 8.f))) {
      const float n0 = fmaxf(m0, a0), n1 = fmaxf(m1, a1);
      const float f0 = m0 == n0 ? 1.f : tc::ex2((m0 - n0) * sl);
      const float f1 = m1 == n1 ? 1.f : tc::ex2((m1 - n1) * sl);
      m0 = n0;
      m1 = n1;
      z0 *= f0;
      z1 *= f1;
#pragma unroll
      for (int x = 0; x < DP / 8; ++x) {
        o[x][0] *= f0;
        o[x][1] *= f0;
        if (WIDE) {
          o[x][2] *= f1;
          o[x][3] *= f1;
        }
      }
    }
    const float b0 = m0 == -INFINITY ? 0.f : -m0 * sl, b1 = m1 == -INFINITY ? 0.f : -m1 * sl;
#pragma unroll
    for (int kk = 0; kk < L::kKeys / 16; ++kk) {
      uint32_t pa[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float* cc = c[kk * 2 + x];
        const float p0 = tc::ex2(fmaf(cc[0], sl, b0)), p1 = tc::ex2(fmaf(cc[1], sl, b0));
        z0 += p0 + p1;
        pa[2 * x] = tc::pack_bf16x2(p0, p1);
        pa[2 * x + 1] = 0u;
        if (WIDE) {
          const float p2 = tc::ex2(fmaf(cc[2], sl, b1)), p3 = tc::ex2(fmaf(cc[3], sl, b1));
          z1 += p2 + p3;
          pa[2 * x + 1] = tc::pack_bf16x2(p2, p3);
        }
      }
      const int r = kk * 16 + (lane & 15);
#pragma unroll
      for (int x = 0; x < DP / 8; x += 2) {  // 16 keys by two 8-channel blocks
        uint32_t vb[4];
        ldsm4_trans(vb, sv + r * DP * 2 + (((x + (lane >> 4)) ^ (r & 7)) << 4));
        mma16816(o[x], pa, vb[0], vb[1]);
        mma16816(o[x + 1], pa, vb[2], vb[3]);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int x = 1; x < 4; x <<= 1) {
    z0 += __shfl_xor_sync(0xffffffffu, z0, x);
    z1 += __shfl_xor_sync(0xffffffffu, z1, x);
  }
  if (t4 == 0) {
    sm[warp][g] = m0 * sl;
    sm[warp][g + 8] = m1 * sl;
    sz[warp][g] = z0;
    sz[warp][g + 8] = z1;
  }
  float* so = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int x = 0; x < DP / 8; ++x) {
    const int e = x * 8 + t4 * 2;
    *reinterpret_cast<float2*>(so + g * L::kPitch + e) = make_float2(o[x][0], o[x][1]);
    *reinterpret_cast<float2*>(so + (g + 8) * L::kPitch + e) = make_float2(o[x][2], o[x][3]);
  }
  __syncthreads();
  join_warps<bf16>(sm, sz, reinterpret_cast<const float*>(smem), L::kWarpBytes / 4, L::kPitch, pb,
                   sp, s, part, out, lse);
}

// ---------------------------------------------------------------------------
// Every other case, in fp32 on the CUDA cores: a lane holds CH = DP / 32
// channels of a row, GH heads and KT keys at a time.  The KT x GH dot
// products are summed over the lanes by halving (each step leaves a lane half
// of the values it had), about one shuffle a product.
// ---------------------------------------------------------------------------
template <typename T, int CH>
__device__ __forceinline__ void load_channels(float (&x)[CH], const T* p, int e, int d, bool vec) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < CH; i += 2) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(p + e + i));
        x[i] = v.x;
        x[i + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH; i += 2) {
        const uint32_t v = __ldg(reinterpret_cast<const unsigned int*>(p + e + i));
        x[i] = __uint_as_float(v << 16);
        x[i + 1] = __uint_as_float(v & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) x[i] = e + i < d ? to_f32(p[e + i]) : 0.f;
  }
}

template <typename T, int CH>
__device__ __forceinline__ void load_vector(float (&x)[CH], const T* p) {
  if constexpr (sizeof(T) == 4 && CH >= 4) {
#pragma unroll
    for (int i = 0; i < CH; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      x[i] = v.x;
      x[i + 1] = v.y;
      x[i + 2] = v.z;
      x[i + 3] = v.w;
    }
  } else {
    load_channels<T, CH>(x, p, 0, CH, true);
  }
}

template <typename T, int DP, int GH, int KT>
__global__ void __launch_bounds__(kThreads)
    decode_simt_kernel(const T* __restrict__ q, const T* __restrict__ kc,
                       const T* __restrict__ vc, Parts part, T* __restrict__ out,
                       float* __restrict__ lse, DecodeProblem pb, Split sp, bool vec,
                       int* status) {
  constexpr int CH = DP / 32, kVals = KT * GH;
  static_assert(kVals <= 32 && (kVals & (kVals - 1)) == 0, "dot products of a tile");
  __shared__ float sm[kWarps][kRows], sz[kWarps][kRows];
  __shared__ float so[kWarps][GH][DP + 4];
  if (sp.chunks > 1) tc::pdl_launch_dependents();  // the join
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * CH;
  const Share s = share_of(pb, sp, GH, status);
  if (s.j0 >= s.j1) {
    if (sp.chunks == 1) write_empty(pb, s, out, lse);
    return;
  }
  const float sl = pb.scale * kLog2e;
  float qr[GH][CH], o[GH][CH], m[GH], z[GH];
#pragma unroll
  for (int h = 0; h < GH; ++h) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      qr[h][i] = h < s.nh && e0 + i < pb.d
                     ? to_f32(q[s.b * pb.q_b + (s.h0 + h) * pb.q_h + e0 + i]) * sl
                     : 0.f;
      o[h][i] = 0.f;
    }
    m[h] = -INFINITY;
    z[h] = 0.f;
  }
  const T *k0 = kc + s.hk * pb.k_h, *v0 = vc + s.hk * pb.v_h;
  for (int t0 = s.j0 + warp * KT; t0 < s.j1; t0 += kWarps * KT) {
    const int2 at = place(pb, s, t0 + lane % KT, status);
    float k[KT][CH], v[KT][CH];
#pragma unroll
    for (int y = 0; y < KT; ++y) {
      const int page = __shfl_sync(0xffffffffu, at.x, y), row = __shfl_sync(0xffffffffu, at.y, y);
#pragma unroll
      for (int i = 0; i < CH; ++i) k[y][i] = v[y][i] = 0.f;
      if (page >= 0 && e0 < pb.d) {
        const T* kr = k0 + page * pb.k_page + row * pb.k_n;
        const T* vr = v0 + page * pb.v_page + row * pb.v_n;
        if (vec) {
          load_vector<T, CH>(k[y], kr + e0);
          load_vector<T, CH>(v[y], vr + e0);
        } else {
          load_channels<T, CH>(k[y], kr, e0, pb.d, false);
          load_channels<T, CH>(v[y], vr, e0, pb.d, false);
        }
      }
    }
    float w[kVals];  // product of key y and head h at y * GH + h
#pragma unroll
    for (int y = 0; y < KT; ++y)
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) a = fmaf(qr[h][i], k[y][i], a);
        w[y * GH + h] = a;
      }
    // value x ends on the lanes whose top bits spell it, highest bit first
    int bit = 16;
#pragma unroll
    for (int left = kVals; left > 1; left >>= 1, bit >>= 1) {
      const bool up = lane & bit;
#pragma unroll
      for (int x = 0; x < left / 2; ++x) {
        const float keep = up ? w[x + left / 2] : w[x], give = up ? w[x] : w[x + left / 2];
        w[x] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
      }
    }
#pragma unroll
    for (; bit > 0; bit >>= 1) w[0] += __shfl_xor_sync(0xffffffffu, w[0], bit);
    constexpr int kStep = 32 / kVals;  // lanes of a value
    const int mine = lane / kStep;
    float sc = t0 + mine / GH < s.j1 ? w[0] : -INFINITY;
    // maximum of each head over the keys: lanes GH * kStep apart
    float mt = sc;
#pragma unroll
    for (int x = GH * kStep; x < 32; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
    float base[GH];
#pragma unroll
    for (int h = 0; h < GH; ++h) {
      const float mn = fmaxf(m[h], __shfl_sync(0xffffffffu, mt, h * kStep));
      base[h] = mn == -INFINITY ? 0.f : mn;
      if (mn > m[h]) {
        const float f = exp2f(m[h] - base[h]);
        z[h] *= f;
#pragma unroll
        for (int i = 0; i < CH; ++i) o[h][i] *= f;
        m[h] = mn;
      }
    }
    float mb = base[0];
#pragma unroll
    for (int h = 1; h < GH; ++h)
      if (mine % GH == h) mb = base[h];
    const float p = exp2f(sc - mb);
#pragma unroll
    for (int y = 0; y < KT; ++y)
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        const float a = __shfl_sync(0xffffffffu, p, (y * GH + h) * kStep);
        z[h] += a;
#pragma unroll
        for (int i = 0; i < CH; ++i) o[h][i] = fmaf(a, v[y][i], o[h][i]);
      }
  }
#pragma unroll
  for (int h = 0; h < GH; ++h) {
#pragma unroll
    for (int i = 0; i < CH; ++i) so[warp][h][e0 + i] = o[h][i];
    if (lane == 0) {
      sm[warp][h] = m[h];
      sz[warp][h] = z[h];
    }
  }
  __syncthreads();
  join_warps<T>(sm, sz, &so[0][0][0], GH * (DP + 4), DP + 4, pb, sp, s, part, out, lse);
}

// One CTA of eight warps per (b, h): the chunks' results weighted by
// exp2(m - max); a warp sums every eighth chunk, then the warps are summed.
constexpr int kJoinWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps)
    decode_join_kernel(T* __restrict__ out, float* __restrict__ lse, Parts part,
                       DecodeProblem pb, Split sp) {
  __shared__ float sm[kJoinWarps], sz[kJoinWarps];
  __shared__ float sa[kJoinWarps][256];
  tc::pdl_wait();
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = row / pb.H, h = row % pb.H;
  const int len = min(max(__ldg(pb.lens + b), 0), pb.max_pages * pb.page_size);
  const int n = (len + sp.chunk - 1) / sp.chunk;
  const long step = (long)pb.B * pb.H;
  float m = -INFINITY;
  for (int c = tid; c < n; c += 32 * kJoinWarps) m = fmaxf(m, part.ml[c * step + row].x);
  m = warp_max(m);
  if (lane == 0) sm[warp] = m;
  __syncthreads();
  m = warp_max(sm[lane % kJoinWarps]);
  const float base = m == -INFINITY ? 0.f : m;
  float acc[8], z = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int c = warp; c < n; c += kJoinWarps) {
    const float2 ml = part.ml[c * step + row];
    const float* p = part.o + (c * step + row) * pb.d;
    const float f = exp2f(ml.x - base);
    z = fmaf(ml.y, f, z);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 32 + lane < pb.d) acc[i] = fmaf(p[i * 32 + lane], f, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sa[warp][i * 32 + lane] = acc[i];
  if (lane == 0) sz[warp] = z;
  __syncthreads();
  float zz = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) zz += sz[w];
  if (tid < pb.d) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) a += sa[w][tid];
    out[b * pb.out_b + h * pb.out_h + tid] = from_f32<T>(zz == 0.f ? 0.f : a / zz);
  }
  if (tid == 0) lse[row] = (m + log2f(zz)) * kLn2;  // (-inf without keys)
}

bool rows_allow(const void* p, std::initializer_list<long> strides, long elements, size_t elt) {
  if (reinterpret_cast<uintptr_t>(p) % (elements * elt)) return false;
  for (long s : strides)
    if (s % elements) return false;
  return true;
}

template <int DP, bool WIDE>
cudaError_t launch_mma(const bf16* q, const bf16* k, const bf16* v, bf16* out, float* lse,
                       const DecodeProblem& pb, const Split& sp, Parts part, int* status,
                       cudaStream_t stream, int* launches) {
  const int smem = kWarps * MmaTile<DP>::kWarpBytes;
  const cudaError_t e = allow_smem<decode_mma_kernel<DP, WIDE>>(smem);
  if (e != cudaSuccess) return e;
  const int hgs = (pb.H / pb.Hkv + kRows - 1) / kRows;
  const unsigned grid = (unsigned)((long)sp.chunks * hgs * pb.Hkv * pb.B);
  return timed_launch("decode_mma", stream, launches, [&] {
    decode_mma_kernel<DP, WIDE>
        <<<grid, kThreads, smem, stream>>>(q, k, v, part, out, lse, pb, sp, status);
  });
}

template <typename T, int DP, int GH, int KT>
cudaError_t launch_simt(const T* q, const T* k, const T* v, T* out, float* lse,
                        const DecodeProblem& pb, const Split& sp, Parts part, int* status,
                        cudaStream_t stream, int* launches) {
  constexpr long CH = DP / 32, kVec = CH * sizeof(T) > 16 ? 16 / sizeof(T) : CH;
  const bool vec = pb.d % CH == 0 && rows_allow(k, {pb.k_page, pb.k_h, pb.k_n}, kVec, sizeof(T)) &&
                   rows_allow(v, {pb.v_page, pb.v_h, pb.v_n}, kVec, sizeof(T));
  const int hgs = (pb.H / pb.Hkv + GH - 1) / GH;
  const unsigned grid = (unsigned)((long)sp.chunks * hgs * pb.Hkv * pb.B);
  return timed_launch("decode_simt", stream, launches, [&] {
    decode_simt_kernel<T, DP, GH, KT><<<grid, kThreads, 0, stream>>>(q, k, v, part, out, lse, pb,
                                                                    sp, vec, status);
  });
}

// One head, or up to four heads of a group at a time; eight keys, and four
// where a lane holds eight channels.
template <typename T>
cudaError_t launch_simt_dp(const T* q, const T* k, const T* v, T* out, float* lse,
                           const DecodeProblem& pb, const Split& sp, Parts part, int* status,
                           cudaStream_t stream, int* launches) {
  const bool one = pb.H == pb.Hkv;
#define MONARCH_DECODE(DP, GH, KT) \
  launch_simt<T, DP, GH, KT>(q, k, v, out, lse, pb, sp, part, status, stream, launches)
  if (pb.d <= 64) return one ? MONARCH_DECODE(64, 1, 8) : MONARCH_DECODE(64, 4, 8);
  if (pb.d <= 128) return one ? MONARCH_DECODE(128, 1, 8) : MONARCH_DECODE(128, 4, 8);
  return one ? MONARCH_DECODE(256, 1, 4) : MONARCH_DECODE(256, 4, 4);
#undef MONARCH_DECODE
}

}  // namespace

size_t decode_workspace_bytes(const DecodeProblem& pb) {
  const Split sp = make_split(pb);
  return sp.chunks == 1 ? 0 : (size_t)sp.chunks * pb.B * pb.H * (pb.d + 2) * sizeof(float);
}

template <typename T>
cudaError_t decode_forward(const T* q, const T* k, const T* v, T* out, float* lse,
                           const DecodeProblem& pb, float* ws, int* status, cudaStream_t stream,
                           int* launches) {
  const Split sp = make_split(pb);
  Parts part = {reinterpret_cast<float2*>(ws), nullptr};
  if (sp.chunks > 1) part.o = ws + 2 * (size_t)sp.chunks * pb.B * pb.H;
  cudaError_t e;
  bool mma = false;
  if constexpr (sizeof(T) == 2) {
    mma = pb.d % 8 == 0 && pb.d <= 128 && rows_allow(q, {pb.q_b, pb.q_h}, 8, 2) &&
          rows_allow(k, {pb.k_page, pb.k_h, pb.k_n}, 8, 2) &&
          rows_allow(v, {pb.v_page, pb.v_h, pb.v_n}, 8, 2);
    if (mma) {
      const bool wide = pb.H / pb.Hkv > 8;
      const auto launch = pb.d <= 64 ? (wide ? launch_mma<64, true> : launch_mma<64, false>)
                                     : (wide ? launch_mma<128, true> : launch_mma<128, false>);
      e = launch(q, k, v, out, lse, pb, sp, part, status, stream, launches);
    }
  }
  if (!mma) e = launch_simt_dp<T>(q, k, v, out, lse, pb, sp, part, status, stream, launches);
  if (e != cudaSuccess || sp.chunks == 1) return e;
  return timed_launch("decode_join", stream, launches, [&] {
    return launch_pdl(decode_join_kernel<T>, dim3(pb.B * pb.H), dim3(32 * kJoinWarps), 0,
                      stream, out, lse, part, pb, sp);
  });
}

template cudaError_t decode_forward<float>(const float*, const float*, const float*, float*,
                                           float*, const DecodeProblem&, float*, int*,
                                           cudaStream_t, int*);
template cudaError_t decode_forward<bf16>(const bf16*, const bf16*, const bf16*, bf16*, float*,
                                          const DecodeProblem&, float*, int*, cudaStream_t, int*);

}  // namespace monarch
