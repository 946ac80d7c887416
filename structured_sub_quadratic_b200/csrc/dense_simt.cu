// Exact softmax attention on the CUDA cores, forward and backward, in fp32:
// fp32 tensors (whose bar rules out TF32), and the bf16 shapes that the
// tensor-core kernels do not take (d above 128 or not a multiple of 8,
// unaligned rows).
//
// A CTA owns a tile of ROWS rows (queries, or keys in the dK, dV kernel) and
// walks tiles of COLS of the other axis, both widened to fp32 in shared
// memory.  Of its 4 ROWS threads, thread (ty, tx) holds rows ty + ROWS/4 i
// (i < 4) and columns tx + 16 j of each score tile, and columns 4 tx + 64 c of
// each d-wide accumulator.  Bound: the FFMA pipe, fed by float4 shared loads
// (rows padded by 4 floats, conflict-free) in packed pairs of channels.
#include "dense.cuh"

#include <math.h>

#include "launch.cuh"
#include "tc_ptx.cuh"
#include "timing.cuh"

namespace monarch {
namespace {

constexpr int kDeltaThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 load4<bf16>(const bf16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
template <>
__device__ __forceinline__ void store4<bf16>(bf16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// Rows [r0, r0 + BT) of one head into shared memory as fp32, rows from n on
// and channels from d on zero.  vec: rows allow four-element loads and
// d % 4 == 0.
template <typename T, int BT, int DP, int THREADS>
__device__ __forceinline__ void load_tile(float* dst, const T* src, long stride, int r0, int n,
                                          int d, bool vec) {
  constexpr int kPitch = DP + 4, kEach = BT * (DP / 4) / THREADS;
  static_assert(BT * (DP / 4) % THREADS == 0, "whole loads per thread");
#pragma unroll 8
  for (int i = 0; i < kEach; ++i) {
    const int x = i * THREADS + (int)threadIdx.x, r = x / (DP / 4), c = x % (DP / 4) * 4;
    float* to = dst + r * kPitch + c;
    const bool there = r0 + r < n && c < d;
    const T* p = src + (there ? (long)(r0 + r) * stride + c : 0);
    if (sizeof(T) == 4 && vec) {  // straight to shared memory, all of a tile in flight
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(to)),
                   "l"(p), "r"(there ? 16 : 0)
                   : "memory");
      continue;
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (there) {
      if (vec) {
        v = load4(p);
      } else {
        v.x = to_f32(p[0]);
        if (c + 1 < d) v.y = to_f32(p[1]);
        if (c + 2 < d) v.z = to_f32(p[2]);
        if (c + 3 < d) v.w = to_f32(p[3]);
      }
    }
    *reinterpret_cast<float4*>(to) = v;
  }
}

// Every tile that this thread's load_tile calls asked for is there, for all
// threads of the CTA.
__device__ __forceinline__ void tiles_arrived() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ void store_row4(T* p, float4 v, int c, int d, bool vec) {
  if (c >= d) return;
  if (vec) {
    store4(p + c, v);
  } else {
    p[c] = from_f32<T>(v.x);
    if (c + 1 < d) p[c + 1] = from_f32<T>(v.y);
    if (c + 2 < d) p[c + 2] = from_f32<T>(v.z);
    if (c + 3 < d) p[c + 3] = from_f32<T>(v.w);
  }
}

// acc[i][j] = A[ty + ROWS/4 i] . B[tx + 16 j] over DP channels; even and odd
// channels are summed apart (one packed instruction for both).
template <int ROWS, int COLS, int DP>
__device__ __forceinline__ void scores(const float* A, const float* B, int ty, int tx,
                                       float (&acc)[4][COLS / 16]) {
  constexpr int J = COLS / 16, kPitch = DP + 4;
  float2 s[4][J];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) s[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int c = 0; c < DP; c += 4) {
    float4 a[4], b[J];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = *reinterpret_cast<const float4*>(A + (ty + ROWS / 4 * i) * kPitch + c);
#pragma unroll
    for (int j = 0; j < J; ++j)
      b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * kPitch + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        s[i][j] = tc::fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), s[i][j]);
        s[i][j] = tc::fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), s[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[i][j] = s[i][j].x + s[i][j].y;
}

// acc[i][c] += sum_k W[ty + ROWS/4 i][k] X[k][4 tx + 64 c ..].
template <int ROWS, int COLS, int DP>
__device__ __forceinline__ void accumulate(const float* W, const float* X, int ty, int tx,
                                           float4 (&acc)[4][DP / 64]) {
  constexpr int kPitch = DP + 4, kWPitch = COLS + 4;
#pragma unroll 2
  for (int k = 0; k < COLS; k += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = *reinterpret_cast<const float4*>(W + (ty + ROWS / 4 * i) * kWPitch + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        const float4 x =
            *reinterpret_cast<const float4*>(X + (k + kk) * kPitch + 4 * tx + 64 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
          const float2 s2 = make_float2(s, s);
          const float2 lo = tc::fma2(s2, make_float2(x.x, x.y), make_float2(acc[i][c].x, acc[i][c].y));
          const float2 hi = tc::fma2(s2, make_float2(x.z, x.w), make_float2(acc[i][c].z, acc[i][c].w));
          acc[i][c] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
      }
  }
}

// Keys past the length may hold anything: load_tile puts zeros in their
// place, and their scores are masked by selection.

template <typename T, int DP, int ROWS, int COLS>
__global__ void __launch_bounds__(4 * ROWS)
    dense_fwd_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                     T* __restrict__ out, float* __restrict__ lse, DenseProblem pb, bool vec) {
  constexpr int J = COLS / 16, kThreads = 4 * ROWS;
  extern __shared__ __align__(16) float smf[];
  float* sQ = smf;
  float* sK = sQ + ROWS * (DP + 4);
  float* sV = sK + COLS * (DP + 4);
  float* sP = sV + COLS * (DP + 4);  // [query][key]
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int tiles = (pb.Nq + ROWS - 1) / ROWS, bh = blockIdx.x / tiles;
  const int q0 = (int)(blockIdx.x % tiles) * ROWS, h = bh % pb.H, b = bh / pb.H;
  const int hk = h / (pb.H / pb.Hkv);
  const int len = dense_len(pb, b);
  const T* qb = q + b * pb.q.b + h * pb.q.h;
  const T* kb = k + b * pb.k.b + hk * pb.k.h;
  const T* vb = v + b * pb.v.b + hk * pb.v.h;
  load_tile<T, ROWS, DP, kThreads>(sQ, qb, pb.q.n, q0, pb.Nq, pb.d, vec);
  int vis[4];
  float m[4], z[4];
  float4 o[4][DP / 64];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + ty + ROWS / 4 * i;
    vis[i] = row < pb.Nq ? dense_visible(pb, len, row) : 0;
    m[i] = -INFINITY;
    z[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int end = dense_visible(pb, len, min(q0 + ROWS, pb.Nq) - 1);  // keys of the last row
  const float sl = pb.scale * kLog2e;
  for (int k0 = 0; k0 < end; k0 += COLS) {
    __syncthreads();
    load_tile<T, COLS, DP, kThreads>(sK, kb, pb.k.n, k0, len, pb.d, vec);
    load_tile<T, COLS, DP, kThreads>(sV, vb, pb.v.n, k0, len, pb.d, vec);
    tiles_arrived();
    float s[4][J];
    scores<ROWS, COLS, DP>(sQ, sK, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        s[i][j] = k0 + tx + 16 * j < vis[i] ? s[i][j] * sl : -INFINITY;
        mt = fmaxf(mt, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
      const float mn = fmaxf(m[i], mt);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float corr = exp2f(m[i] - base);
      float zt = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float p = exp2f(s[i][j] - base);
        zt += p;
        sP[(ty + ROWS / 4 * i) * (COLS + 4) + tx + 16 * j] = p;
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) zt += __shfl_xor_sync(0xffffffffu, zt, x);
      z[i] = z[i] * corr + zt;
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        o[i][c].x *= corr;
        o[i][c].y *= corr;
        o[i][c].z *= corr;
        o[i][c].w *= corr;
      }
    }
    __syncthreads();
    accumulate<ROWS, COLS, DP>(sP, sV, ty, tx, o);
  }
  tiles_arrived();  // (a CTA without keys still has its queries in flight)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + ty + ROWS / 4 * i;
    if (row >= pb.Nq) continue;
    const float inv = vis[i] > 0 ? 1.f / z[i] : 0.f;
    T* ob = out + b * pb.out.b + h * pb.out.h + (long)row * pb.out.n;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      const float4 t = make_float4(o[i][c].x * inv, o[i][c].y * inv, o[i][c].z * inv,
                                   o[i][c].w * inv);
      store_row4(ob, t, 4 * tx + 64 * c, pb.d, vec);
    }
    if (tx == 0)
      lse[((long)b * pb.H + h) * pb.Nq + row] =
          vis[i] > 0 ? (m[i] + log2f(z[i])) * kLn2 : -INFINITY;
  }
}

// delta = the row sum of dO O, `lanes` (a power of two) lanes a row.  CHUNKS:
// 16 bytes a lane at a time, four rows' in flight; else element by element.
template <typename T, bool CHUNKS>
__global__ void __launch_bounds__(kDeltaThreads)
    dense_delta_kernel(const T* __restrict__ out, const T* __restrict__ dout,
                       float* __restrict__ delta, DenseProblem pb, int lanes) {
  constexpr int E = CHUNKS ? 16 / (int)sizeof(T) : 1, kRows = 4;
  const int per = kDeltaThreads / lanes, lane = threadIdx.x % lanes;
  const long total = (long)pb.B * pb.H * pb.Nq;
  const long row0 = (long)blockIdx.x * per * kRows + threadIdx.x / lanes;
  float s[kRows];
  const T *o[kRows], *g[kRows];
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    const long row = min(row0 + x * per, total - 1);
    const int i = (int)(row % pb.Nq), bh = (int)(row / pb.Nq), h = bh % pb.H, b = bh / pb.H;
    o[x] = out + b * pb.out.b + h * pb.out.h + i * pb.out.n;
    g[x] = dout + b * pb.dout.b + h * pb.dout.h + i * pb.dout.n;
    s[x] = 0.f;
  }
  for (int c = lane * E; c < pb.d; c += lanes * E) {
    if constexpr (CHUNKS) {
      uint4 a[kRows], w[kRows];
#pragma unroll
      for (int x = 0; x < kRows; ++x) {
        a[x] = __ldg(reinterpret_cast<const uint4*>(o[x] + c));
        w[x] = __ldg(reinterpret_cast<const uint4*>(g[x] + c));
      }
#pragma unroll
      for (int x = 0; x < kRows; ++x)
#pragma unroll
        for (int e = 0; e < E; ++e)
          s[x] = fmaf(to_f32(reinterpret_cast<const T*>(&a[x])[e]),
                      to_f32(reinterpret_cast<const T*>(&w[x])[e]), s[x]);
    } else {
#pragma unroll
      for (int x = 0; x < kRows; ++x) s[x] = fmaf(to_f32(o[x][c]), to_f32(g[x][c]), s[x]);
    }
  }
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    for (int y = lanes / 2; y > 0; y >>= 1) s[x] += __shfl_xor_sync(0xffffffffu, s[x], y);
    if (lane == 0 && row0 + x * per < total) delta[row0 + x * per] = s[x];
  }
}

// dK and dV of a tile of keys: every query head of the group and every query
// tile that sees the keys, in order.
//   P = exp(S - lse), dV = P^T dO, dS = P (dO V^T - delta), dK = scale dS^T Q
template <typename T, int DP, int ROWS, int COLS>
__global__ void __launch_bounds__(4 * ROWS)
    dense_dkv_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                     const float* __restrict__ lse, const float* __restrict__ delta,
                     const T* __restrict__ dout, T* __restrict__ dk, T* __restrict__ dv,
                     DenseProblem pb, bool vec) {
  constexpr int J = COLS / 16, kThreads = 4 * ROWS;
  extern __shared__ __align__(16) float smf[];
  float* sK = smf;
  float* sV = sK + ROWS * (DP + 4);
  float* sQ = sV + ROWS * (DP + 4);
  float* sG = sQ + COLS * (DP + 4);
  float* sP = sG + COLS * (DP + 4);  // [key][query]
  float* sS = sP + ROWS * (COLS + 4);
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int tiles = (pb.Nk + ROWS - 1) / ROWS, bh = blockIdx.x / tiles;
  const int k0 = (int)(blockIdx.x % tiles) * ROWS, hk = bh % pb.Hkv, b = bh / pb.Hkv;
  const int len = dense_len(pb, b), group = pb.H / pb.Hkv;
  load_tile<T, ROWS, DP, kThreads>(sK, k + b * pb.k.b + hk * pb.k.h, pb.k.n, k0, len, pb.d, vec);
  load_tile<T, ROWS, DP, kThreads>(sV, v + b * pb.v.b + hk * pb.v.h, pb.v.n, k0, len, pb.d, vec);
  float4 ak[4][DP / 64], av[4][DP / 64];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) ak[i][c] = av[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  // the first query that sees key k0
  const int qfirst = pb.causal ? max(0, k0 - (pb.Nk - pb.Nq)) / COLS * COLS : 0;
  const float sl = pb.scale * kLog2e;
  if (k0 < len) {
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
      const T* qb = q + b * pb.q.b + h * pb.q.h;
      const T* gb = dout + b * pb.dout.b + h * pb.dout.h;
      const long row0 = ((long)b * pb.H + h) * pb.Nq;
      for (int q0 = qfirst; q0 < pb.Nq; q0 += COLS) {
        __syncthreads();
        load_tile<T, COLS, DP, kThreads>(sQ, qb, pb.q.n, q0, pb.Nq, pb.d, vec);
        load_tile<T, COLS, DP, kThreads>(sG, gb, pb.dout.n, q0, pb.Nq, pb.d, vec);
        tiles_arrived();
        float s[4][J], dp[4][J];
        scores<ROWS, COLS, DP>(sK, sQ, ty, tx, s);
        scores<ROWS, COLS, DP>(sV, sG, ty, tx, dp);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int row = q0 + tx + 16 * j;
          const bool ok = row < pb.Nq;
          const int vis = ok ? dense_visible(pb, len, row) : 0;
          const float l2 = ok ? __ldg(lse + row0 + row) * kLog2e : 0.f;
          const float dl = ok ? __ldg(delta + row0 + row) : 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = ty + ROWS / 4 * i, at = key * (COLS + 4) + tx + 16 * j;
            const bool see = k0 + key < vis;
            const float p = see ? exp2f(fmaf(s[i][j], sl, -l2)) : 0.f;
            sP[at] = p;
            sS[at] = see ? p * (dp[i][j] - dl) : 0.f;
          }
        }
        __syncthreads();
        accumulate<ROWS, COLS, DP>(sP, sG, ty, tx, av);
        accumulate<ROWS, COLS, DP>(sS, sQ, ty, tx, ak);
      }
    }
  }
  tiles_arrived();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = k0 + ty + ROWS / 4 * i;
    if (row >= pb.Nk) continue;
    T* kr = dk + b * pb.dk.b + hk * pb.dk.h + (long)row * pb.dk.n;
    T* vr = dv + b * pb.dv.b + hk * pb.dv.h + (long)row * pb.dv.n;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      const float4 t = make_float4(ak[i][c].x * pb.scale, ak[i][c].y * pb.scale,
                                   ak[i][c].z * pb.scale, ak[i][c].w * pb.scale);
      store_row4(kr, t, 4 * tx + 64 * c, pb.d, vec);
      store_row4(vr, av[i][c], 4 * tx + 64 * c, pb.d, vec);
    }
  }
}

// dQ of a tile of queries: dQ = scale dS K over the tiles of visible keys.
template <typename T, int DP, int ROWS, int COLS>
__global__ void __launch_bounds__(4 * ROWS)
    dense_dq_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                    const float* __restrict__ lse, const float* __restrict__ delta,
                    const T* __restrict__ dout, T* __restrict__ dq, DenseProblem pb, bool vec) {
  constexpr int J = COLS / 16, kThreads = 4 * ROWS;
  extern __shared__ __align__(16) float smf[];
  float* sQ = smf;
  float* sG = sQ + ROWS * (DP + 4);
  float* sK = sG + ROWS * (DP + 4);
  float* sV = sK + COLS * (DP + 4);
  float* sS = sV + COLS * (DP + 4);  // [query][key]
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int tiles = (pb.Nq + ROWS - 1) / ROWS, bh = blockIdx.x / tiles;
  const int q0 = (int)(blockIdx.x % tiles) * ROWS, h = bh % pb.H, b = bh / pb.H;
  const int hk = h / (pb.H / pb.Hkv);
  const int len = dense_len(pb, b);
  const T* kb = k + b * pb.k.b + hk * pb.k.h;
  const T* vb = v + b * pb.v.b + hk * pb.v.h;
  load_tile<T, ROWS, DP, kThreads>(sQ, q + b * pb.q.b + h * pb.q.h, pb.q.n, q0, pb.Nq, pb.d, vec);
  load_tile<T, ROWS, DP, kThreads>(sG, dout + b * pb.dout.b + h * pb.dout.h, pb.dout.n, q0, pb.Nq, pb.d, vec);
  int vis[4];
  float l2[4], dl[4];
  float4 acc[4][DP / 64];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + ty + ROWS / 4 * i;
    const bool ok = row < pb.Nq;
    const long at = ((long)b * pb.H + h) * pb.Nq + row;
    vis[i] = ok ? dense_visible(pb, len, row) : 0;
    l2[i] = ok ? __ldg(lse + at) * kLog2e : 0.f;
    dl[i] = ok ? __ldg(delta + at) : 0.f;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int end = dense_visible(pb, len, min(q0 + ROWS, pb.Nq) - 1);
  const float sl = pb.scale * kLog2e;
  for (int k0 = 0; k0 < end; k0 += COLS) {
    __syncthreads();
    load_tile<T, COLS, DP, kThreads>(sK, kb, pb.k.n, k0, len, pb.d, vec);
    load_tile<T, COLS, DP, kThreads>(sV, vb, pb.v.n, k0, len, pb.d, vec);
    tiles_arrived();
    float s[4][J], dp[4][J];
    scores<ROWS, COLS, DP>(sQ, sK, ty, tx, s);
    scores<ROWS, COLS, DP>(sG, sV, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const bool see = k0 + tx + 16 * j < vis[i];
        const float p = exp2f(fmaf(s[i][j], sl, -l2[i]));
        sS[(ty + ROWS / 4 * i) * (COLS + 4) + tx + 16 * j] = see ? p * (dp[i][j] - dl[i]) : 0.f;
      }
    __syncthreads();
    accumulate<ROWS, COLS, DP>(sS, sK, ty, tx, acc);
  }
  tiles_arrived();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + ty + ROWS / 4 * i;
    if (row >= pb.Nq) continue;
    T* qr = dq + b * pb.dq.b + h * pb.dq.h + (long)row * pb.dq.n;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      const float4 t = make_float4(acc[i][c].x * pb.scale, acc[i][c].y * pb.scale,
                                   acc[i][c].z * pb.scale, acc[i][c].w * pb.scale);
      store_row4(qr, t, 4 * tx + 64 * c, pb.d, vec);
    }
  }
}

bool rows_allow_four(const void* p, const HeadStrides& s, size_t elt) {
  return (reinterpret_cast<uintptr_t>(p) % (4 * elt)) == 0 && s.b % 4 == 0 && s.h % 4 == 0 &&
         s.n % 4 == 0;
}

// Rows of a CTA: 64 read each streamed tile half as often, 32 where 64 would
// leave the SMs fewer than four CTAs each.
inline bool few(long rows, long heads) { return (rows + 63) / 64 * heads < 4L * num_sms(); }

template <typename T, int DP, int ROWS, int COLS>
cudaError_t forward_rows(const T* q, const T* k, const T* v, T* out, float* lse,
                         const DenseProblem& pb, bool vec, cudaStream_t stream, int* launches) {
  constexpr int smem =
      ((ROWS + 2 * COLS) * (DP + 4) + ROWS * (COLS + 4)) * (int)sizeof(float);
  constexpr auto kernel = dense_fwd_kernel<T, DP, ROWS, COLS>;
  cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((pb.Nq + ROWS - 1) / ROWS) * pb.H * pb.B;
  return timed_launch("dense_fwd_simt", stream, launches, [&] {
    kernel<<<grid, 4 * ROWS, smem, stream>>>(q, k, v, out, lse, pb, vec);
  });
}

template <typename T, int DP, int COLS>
cudaError_t forward_dp(const T* q, const T* k, const T* v, T* out, float* lse,
                       const DenseProblem& pb, bool vec, cudaStream_t stream, int* launches) {
  return few(pb.Nq, (long)pb.H * pb.B)
             ? forward_rows<T, DP, 32, COLS>(q, k, v, out, lse, pb, vec, stream, launches)
             : forward_rows<T, DP, 64, COLS>(q, k, v, out, lse, pb, vec, stream, launches);
}

template <typename T, int DP, int ROWS, int COLS>
cudaError_t dkv_rows(const T* q, const T* k, const T* v, const float* lse, const float* delta,
                     const T* dout, T* dk, T* dv, const DenseProblem& pb, bool vec,
                     cudaStream_t stream, int* launches) {
  constexpr int smem =
      (2 * (ROWS + COLS) * (DP + 4) + 2 * ROWS * (COLS + 4)) * (int)sizeof(float);
  constexpr auto kernel = dense_dkv_kernel<T, DP, ROWS, COLS>;
  cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((pb.Nk + ROWS - 1) / ROWS) * pb.Hkv * pb.B;
  return timed_launch("dense_dkv_simt", stream, launches, [&] {
    kernel<<<grid, 4 * ROWS, smem, stream>>>(q, k, v, lse, delta, dout, dk, dv, pb, vec);
  });
}

template <typename T, int DP, int ROWS, int COLS>
cudaError_t dq_rows(const T* q, const T* k, const T* v, const float* lse, const float* delta,
                    const T* dout, T* dq, const DenseProblem& pb, bool vec, cudaStream_t stream,
                    int* launches) {
  constexpr int smem =
      (2 * (ROWS + COLS) * (DP + 4) + ROWS * (COLS + 4)) * (int)sizeof(float);
  constexpr auto kernel = dense_dq_kernel<T, DP, ROWS, COLS>;
  cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((pb.Nq + ROWS - 1) / ROWS) * pb.H * pb.B;
  return timed_launch("dense_dq_simt", stream, launches, [&] {
    kernel<<<grid, 4 * ROWS, smem, stream>>>(q, k, v, lse, delta, dout, dq, pb, vec);
  });
}

// TALL: rows of a CTA where there are many.
template <typename T, int DP, int TALL, int COLS>
cudaError_t backward_dp(const T* q, const T* k, const T* v, const float* lse, const float* delta,
                        const T* dout, T* dq, T* dk, T* dv, const DenseProblem& pb, bool vec,
                        cudaStream_t stream, int* launches) {
  cudaError_t e = cudaSuccess;
  if (pb.Nk > 0)
    e = few(pb.Nk, (long)pb.Hkv * pb.B)
            ? dkv_rows<T, DP, 32, COLS>(q, k, v, lse, delta, dout, dk, dv, pb, vec, stream,
                                        launches)
            : dkv_rows<T, DP, TALL, COLS>(q, k, v, lse, delta, dout, dk, dv, pb, vec, stream,
                                          launches);
  if (e == cudaSuccess && pb.Nq > 0)
    e = few(pb.Nq, (long)pb.H * pb.B)
            ? dq_rows<T, DP, 32, COLS>(q, k, v, lse, delta, dout, dq, pb, vec, stream, launches)
            : dq_rows<T, DP, TALL, COLS>(q, k, v, lse, delta, dout, dq, pb, vec, stream,
                                         launches);
  return e;
}

}  // namespace

template <typename T>
cudaError_t dense_simt_forward(const T* q, const T* k, const T* v, T* out, float* lse,
                               const DenseProblem& pb, cudaStream_t stream, int* launches) {
  if (pb.Nq == 0) return cudaSuccess;
  const bool vec = pb.d % 4 == 0 && rows_allow_four(q, pb.q, sizeof(T)) &&
                   rows_allow_four(k, pb.k, sizeof(T)) && rows_allow_four(v, pb.v, sizeof(T)) &&
                   rows_allow_four(out, pb.out, sizeof(T));
  if (pb.d <= 64) return forward_dp<T, 64, 64>(q, k, v, out, lse, pb, vec, stream, launches);
  if (pb.d <= 128) return forward_dp<T, 128, 64>(q, k, v, out, lse, pb, vec, stream, launches);
  return forward_dp<T, 256, 32>(q, k, v, out, lse, pb, vec, stream, launches);
}

template <typename T>
cudaError_t dense_delta(const T* out, const T* dout, float* delta, const DenseProblem& pb,
                        cudaStream_t stream, int* launches) {
  const long rows = (long)pb.B * pb.H * pb.Nq;
  if (rows == 0) return cudaSuccess;
  constexpr int E = 16 / (int)sizeof(T);
  bool chunks = pb.d % E == 0;
  const void* p[2] = {out, dout};
  const HeadStrides st[2] = {pb.out, pb.dout};
  for (int x = 0; x < 2; ++x)
    chunks = chunks && (reinterpret_cast<uintptr_t>(p[x]) & 15u) == 0 && st[x].b % E == 0 &&
             st[x].h % E == 0 && st[x].n % E == 0;
  const int units = chunks ? pb.d / E : pb.d;
  int lanes = 1;
  while (lanes < 32 && lanes < units) lanes *= 2;
  const long each = kDeltaThreads / lanes * 4;
  const unsigned blocks = (unsigned)((rows + each - 1) / each);
  return timed_launch("dense_delta", stream, launches, [&] {
    if (chunks)
      dense_delta_kernel<T, true><<<blocks, kDeltaThreads, 0, stream>>>(out, dout, delta, pb,
                                                                        lanes);
    else
      dense_delta_kernel<T, false><<<blocks, kDeltaThreads, 0, stream>>>(out, dout, delta, pb,
                                                                         lanes);
  });
}

template <typename T>
cudaError_t dense_simt_backward(const T* q, const T* k, const T* v, const T* out,
                                const float* lse, const T* dout, T* dq, T* dk, T* dv,
                                float* delta, const DenseProblem& pb, cudaStream_t stream,
                                int* launches) {
  bool vec = pb.d % 4 == 0;
  const void* p[7] = {q, k, v, dout, dq, dk, dv};
  const HeadStrides s[7] = {pb.q, pb.k, pb.v, pb.dout, pb.dq, pb.dk, pb.dv};
  for (int x = 0; x < 7; ++x) vec = vec && rows_allow_four(p[x], s[x], sizeof(T));
  cudaError_t e = dense_delta<T>(out, dout, delta, pb, stream, launches);
  if (e != cudaSuccess) return e;
  if (pb.d <= 64)
    return backward_dp<T, 64, 64, 64>(q, k, v, lse, delta, dout, dq, dk, dv, pb, vec, stream,
                                  launches);
  if (pb.d <= 128)
    return backward_dp<T, 128, 64, 64>(q, k, v, lse, delta, dout, dq, dk, dv, pb, vec, stream,
                                   launches);
  // four 64-row tiles of 256 channels exceed shared memory
  return backward_dp<T, 256, 32, 32>(q, k, v, lse, delta, dout, dq, dk, dv, pb, vec, stream,
                                 launches);
}

template cudaError_t dense_simt_forward<float>(const float*, const float*, const float*, float*,
                                               float*, const DenseProblem&, cudaStream_t, int*);
template cudaError_t dense_simt_forward<bf16>(const bf16*, const bf16*, const bf16*, bf16*,
                                              float*, const DenseProblem&, cudaStream_t, int*);
template cudaError_t dense_simt_backward<float>(const float*, const float*, const float*,
                                                const float*, const float*, const float*, float*,
                                                float*, float*, float*, const DenseProblem&,
                                                cudaStream_t, int*);
template cudaError_t dense_simt_backward<bf16>(const bf16*, const bf16*, const bf16*, const bf16*,
                                               const float*, const bf16*, bf16*, bf16*, bf16*,
                                               float*, const DenseProblem&, cudaStream_t, int*);
template cudaError_t dense_delta<float>(const float*, const float*, float*, const DenseProblem&,
                                        cudaStream_t, int*);
template cudaError_t dense_delta<bf16>(const bf16*, const bf16*, float*, const DenseProblem&,
                                       cudaStream_t, int*);

}  // namespace monarch
