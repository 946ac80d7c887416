// Exact softmax attention in fp32, forward and backward: fp32 tensors, and the
// bf16 shapes that the tcgen05 kernels do not take (d above 128 or not a
// multiple of 8, unaligned rows).
//
// The fp32 bar (1e-4 relative, 1e-6 in practice) rules out TF32 products, and
// FFMA products were bound by shared memory at half the FFMA rate (four rows
// by four columns a thread: one 16-byte load per eight multiply-adds).  So
// each fp32 operand is split into two TF32 values, x = hi + lo + r with |r|
// below 2^-21 |x|, and a product is three TF32 products, hi hi + hi lo + lo hi
// (what is left out is below 2^-21 of it).  Tensor cores truncate their sums:
// two steps of 8 are summed there from zero and added to the fp32 accumulator
// in the FMA pipe, rounded to nearest.
//
// A CTA owns a tile of ROWS rows (queries, or keys in the dK, dV kernel) and
// walks tiles of COLS of the other axis, both widened to fp32 in shared memory
// (rows padded by 4 floats: fragment loads touch all banks once).  Two warps
// share 16 rows, each with half of a tile's columns and sums of its own, which
// are joined at the end: one warp a row block leaves an SM five warps at 12
// heads of 1024 rows, and the kernels wait for their own instructions.  Score
// fragments become the A operands of the second products in registers, with
// the columns of a block of 8 in the order 0 2 4 6 1 3 5 7.
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

// Two neighbouring channels c, c + 1 of a row.
template <typename T>
__device__ __forceinline__ void store_pair(T* p, float x, float y, int c, int d, bool vec) {
  if (c >= d) return;
  if (vec) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>(p + c) = make_float2(x, y);
    else
      *reinterpret_cast<uint32_t*>(p + c) = tc::pack_bf16x2(x, y);
  } else {
    p[c] = from_f32<T>(x);
    if (c + 1 < d) p[c + 1] = from_f32<T>(y);
  }
}

struct Split {
  uint32_t hi, lo;
};

// hi: x cut to TF32's 11 significant bits; lo: the rest, rounded to them when
// the product drops its last 13 bits.
__device__ __forceinline__ Split split(float x) {
  const uint32_t hi = __float_as_uint(x) & 0xffffe000u;
  return {hi, __float_as_uint(x - __uint_as_float(hi)) + 0x1000u};
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An A operand of 16 rows by 8, split.
struct SplitA {
  uint32_t hi[4], lo[4];
  __device__ __forceinline__ void set(int i, float x) {
    const Split s = split(x);
    hi[i] = s.hi;
    lo[i] = s.lo;
  }
};

// t[n] += A B_n for a group of blocks of B, whose two elements `b` gives:
// product by product over all blocks, so that none waits for the one before.
template <int kGroup, typename F>
__device__ __forceinline__ void mma_split(float (&t)[kGroup][4], const SplitA& a, F&& b) {
  Split s[kGroup][2];
#pragma unroll
  for (int n = 0; n < kGroup; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) s[n][x] = split(b(n, x));
#pragma unroll
  for (int n = 0; n < kGroup; ++n) mma_tf32(t[n], a.lo, s[n][0].hi, s[n][1].hi);
#pragma unroll
  for (int n = 0; n < kGroup; ++n) mma_tf32(t[n], a.hi, s[n][0].lo, s[n][1].lo);
#pragma unroll
  for (int n = 0; n < kGroup; ++n) mma_tf32(t[n], a.hi, s[n][0].hi, s[n][1].hi);
}

template <int N>
__device__ __forceinline__ void clear(float (&acc)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[n][x] = 0.f;
}

// acc[n] = A's 16 rows . rows 8 n .. of B, over DP channels (A: the warp's
// first row).  A thread holds rows lane / 4 (+ 8), columns 2 (lane % 4) (+ 1).
template <int COLS, int DP>
__device__ __forceinline__ void scores(const float* A, const float* B, float (&acc)[COLS / 8][4]) {
  constexpr int kPitch = DP + 4, kGroup = COLS >= 32 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const float* a0 = A + lane / 4 * kPitch + lane % 4;
  const float* b0 = B + lane / 4 * kPitch + lane % 4;
#pragma unroll
  for (int n = 0; n < COLS / 8; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[n][x] = 0.f;
#pragma unroll 1
  for (int c = 0; c < DP; c += 16) {
    SplitA a[2];
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int x = 0; x < 4; ++x) a[y].set(x, a0[(x & 1) * 8 * kPitch + c + y * 8 + (x >> 1) * 4]);
#pragma unroll
    for (int n0 = 0; n0 < COLS / 8; n0 += kGroup) {
      float t[kGroup][4];
      clear(t);
#pragma unroll
      for (int y = 0; y < 2; ++y)
        mma_split(t, a[y], [&](int n, int x) {
          return b0[(n0 + n) * 8 * kPitch + c + y * 8 + x * 4];
        });
#pragma unroll
      for (int n = 0; n < kGroup; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[n0 + n][x] += t[n][x];
    }
  }
}

// acc[n] += W X over COLS rows of X: W as scores left it, X's channels 8 n ..
// from `X` on.
template <int COLS, int DP, int N>
__device__ __forceinline__ void accumulate(const float (&w)[COLS / 8][4], const float* X,
                                           float (&acc)[N][4]) {
  constexpr int kPitch = DP + 4, kGroup = 4;
  const int lane = threadIdx.x & 31;
  const float* b0 = X + lane % 4 * 2 * kPitch + lane / 4;
#pragma unroll
  for (int k = 0; k < COLS / 8; k += 2) {
    SplitA a[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      a[y].set(0, w[k + y][0]);
      a[y].set(1, w[k + y][2]);
      a[y].set(2, w[k + y][1]);
      a[y].set(3, w[k + y][3]);
    }
#pragma unroll
    for (int n0 = 0; n0 < N; n0 += kGroup) {
      float t[kGroup][4];
      clear(t);
#pragma unroll
      for (int y = 0; y < 2; ++y)
        mma_split(t, a[y], [&](int n, int x) {
          return b0[((k + y) * 8 + x) * kPitch + (n0 + n) * 8];
        });
#pragma unroll
      for (int n = 0; n < kGroup; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[n0 + n][x] += t[n][x];
    }
  }
}

// A warp's 16 rows of an accumulator to shared memory, and from there.
template <int DP, int N>
__device__ __forceinline__ float2* pair_of(float* rows, int i, int n) {
  const int lane = threadIdx.x & 31;
  return reinterpret_cast<float2*>(rows + (lane / 4 + 8 * i) * (DP + 4) + n * 8 + lane % 4 * 2);
}

template <int DP, int N>
__device__ __forceinline__ void put_rows(float* rows, const float (&acc)[N][4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n)
      *pair_of<DP, N>(rows, i, n) = make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
}

template <int DP, int N>
__device__ __forceinline__ void add_rows(float* rows, float (&acc)[N][4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float2 x = *pair_of<DP, N>(rows, i, n);
      acc[n][2 * i] += x.x;
      acc[n][2 * i + 1] += x.y;
    }
}

// The sums of the warps that share 16 rows, in order, in the first of them.
template <int WAYS, int DP, int N>
__device__ __forceinline__ void join_ways(int way, float* rows, float (&acc)[N][4]) {
#pragma unroll 1
  for (int w = 1; w < WAYS; ++w) {
    if (way == w) put_rows<DP>(rows, acc);
    __syncthreads();
    if (way == 0) add_rows<DP>(rows, acc);
    __syncthreads();
  }
}

// Keys past the length may hold anything: load_tile puts zeros in their
// place, and their scores are masked by selection.

template <typename T, int DP, int ROWS, int COLS>
__global__ void __launch_bounds__(4 * ROWS)
    dense_fwd_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                     T* __restrict__ out, float* __restrict__ lse, DenseProblem pb, KeySplit split,
                     bool vec) {
  constexpr int kThreads = 4 * ROWS, kHalf = COLS / 2, N = kHalf / 8;
  extern __shared__ __align__(16) float smf[];
  float* sQ = smf;
  float* sK = sQ + ROWS * (DP + 4);
  float* sV = sK + COLS * (DP + 4);
  __shared__ float other_m[ROWS], other_z[ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp / 2 * 16, wc = warp % 2 * kHalf;  // first row and column
  if (split.splits > 1) tc::pdl_launch_dependents();  // the join
  const int range = blockIdx.x % split.splits, unit = blockIdx.x / split.splits;
  const int tiles = (pb.Nq + ROWS - 1) / ROWS, bh = unit / tiles;
  const int q0 = unit % tiles * ROWS, h = bh % pb.H, b = bh / pb.H;
  const int hk = h / (pb.H / pb.Hkv);
  const int len = dense_len(pb, b);
  const T* qb = q + b * pb.q.b + h * pb.q.h;
  const T* kb = k + b * pb.k.b + hk * pb.k.h;
  const T* vb = v + b * pb.v.b + hk * pb.v.h;
  load_tile<T, ROWS, DP, kThreads>(sQ, qb, pb.q.n, q0, pb.Nq, pb.d, vec);
  int vis[2];  // of rows lane / 4 and + 8 of the warp
  float m[2] = {-INFINITY, -INFINITY}, z[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = q0 + wr + lane / 4 + 8 * i;
    vis[i] = row < pb.Nq ? dense_visible(pb, len, row) : 0;
  }
  float o[DP / 8][4];
  clear(o);
  // keys of the range that the last row sees
  const int first = range * split.per * COLS;
  const int end = min(dense_visible(pb, len, min(q0 + ROWS, pb.Nq) - 1), first + split.per * COLS);
  const float sl = pb.scale * kLog2e;
#pragma unroll 1
  for (int k0 = first; k0 < end; k0 += COLS) {
    __syncthreads();
    load_tile<T, COLS, DP, kThreads>(sK, kb, pb.k.n, k0, len, pb.d, vec);
    load_tile<T, COLS, DP, kThreads>(sV, vb, pb.v.n, k0, len, pb.d, vec);
    tiles_arrived();
    float s[N][4];
    scores<kHalf, DP>(sQ + wr * (DP + 4), sK + wc * (DP + 4), s);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mt = -INFINITY;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float& y = s[n][2 * i + x];
          y = k0 + wc + n * 8 + lane % 4 * 2 + x < vis[i] ? y * sl : -INFINITY;
          mt = fmaxf(mt, y);
        }
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
      const float mn = fmaxf(m[i], mt), base = mn == -INFINITY ? 0.f : mn;
      const float corr = exp2f(m[i] - base);
      m[i] = mn;
      z[i] *= corr;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float& y = s[n][2 * i + x];
          y = exp2f(y - base);
          z[i] += y;  // this thread's keys; the row is summed at the end
        }
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        o[n][2 * i] *= corr;
        o[n][2 * i + 1] *= corr;
      }
    }
    accumulate<kHalf, DP>(s, sV + wc * (DP + 4), o);
  }
  tiles_arrived();  // (a CTA without keys still has its queries in flight)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    z[i] += __shfl_xor_sync(0xffffffffu, z[i], 1);
    z[i] += __shfl_xor_sync(0xffffffffu, z[i], 2);
  }
  // the second warp's half of the keys, over the queries
  float* rows = sQ + wr * (DP + 4);
  if (wc > 0) {
    put_rows<DP>(rows, o);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane % 4 == 0) {
        other_m[wr + lane / 4 + 8 * i] = m[i];
        other_z[wr + lane / 4 + 8 * i] = z[i];
      }
  }
  __syncthreads();
  if (wc > 0) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = q0 + wr + lane / 4 + 8 * i;
    if (row >= pb.Nq) continue;
    const float m1 = other_m[row - q0], mn = fmaxf(m[i], m1), base = mn == -INFINITY ? 0.f : mn;
    const float f0 = exp2f(m[i] - base), f1 = exp2f(m1 - base);
    const float sum = z[i] * f0 + other_z[row - q0] * f1;
    const bool any = sum != 0.f;  // a visible key, not all of them at -inf
    const bool whole = split.splits == 1;
    const float inv = whole ? 1.f / sum : 1.f;
    const long at = (((long)range * pb.B + b) * pb.H + h) * pb.Nq + row;
    T* ob = out + b * pb.out.b + h * pb.out.h + (long)row * pb.out.n;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      const float2 p = *pair_of<DP, DP / 8>(rows, i, n);
      const float x = (o[n][2 * i] * f0 + p.x * f1) * inv;
      const float y = (o[n][2 * i + 1] * f0 + p.y * f1) * inv;
      const int c = n * 8 + lane % 4 * 2;
      if (whole)
        store_pair(ob, any ? x : 0.f, any ? y : 0.f, c, pb.d, vec);
      else if (any)
        store_pair(split.o + at * pb.d, x, y, c, pb.d, pb.d % 4 == 0);
    }
    if (lane % 4) continue;
    if (whole)
      lse[((long)b * pb.H + h) * pb.Nq + row] = any ? (mn + log2f(sum)) * kLn2 : -INFINITY;
    else
      split.mz[at] = make_float2(mn, any ? sum : 0.f);
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
// WAYS warps share 16 keys and a tile's queries.  Of 256 channels, whose two
// sums do not fit a warp's registers, two warps take half each (CHANNELS), over
// all queries.
template <typename T, int DP, int ROWS, int COLS, int WAYS, bool CHANNELS>
__global__ void __launch_bounds__(2 * ROWS * WAYS)
    dense_dkv_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                     const float* __restrict__ lse, const float* __restrict__ delta,
                     const T* __restrict__ dout, T* __restrict__ dk, T* __restrict__ dv,
                     DenseProblem pb, bool vec) {
  constexpr int kThreads = 2 * ROWS * WAYS, kOwn = CHANNELS ? COLS : COLS / WAYS, N = kOwn / 8;
  constexpr int kPart = CHANNELS ? DP / 2 : DP;
  extern __shared__ __align__(16) float smf[];
  float* sK = smf;
  float* sV = sK + ROWS * (DP + 4);
  float* sQ = sV + ROWS * (DP + 4);
  float* sG = sQ + COLS * (DP + 4);
  __shared__ float row_l2[COLS], row_dl[COLS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // first row, column and channel
  const int wr = warp / WAYS * 16, way = warp % WAYS, wc = CHANNELS ? 0 : way * kOwn;
  const int part = CHANNELS ? way * kPart : 0;
  const int tiles = (pb.Nk + ROWS - 1) / ROWS, bh = blockIdx.x / tiles;
  const int k0 = (int)(blockIdx.x % tiles) * ROWS, hk = bh % pb.Hkv, b = bh / pb.Hkv;
  const int len = dense_len(pb, b), group = pb.H / pb.Hkv;
  load_tile<T, ROWS, DP, kThreads>(sK, k + b * pb.k.b + hk * pb.k.h, pb.k.n, k0, len, pb.d, vec);
  load_tile<T, ROWS, DP, kThreads>(sV, v + b * pb.v.b + hk * pb.v.h, pb.v.n, k0, len, pb.d, vec);
  float ak[kPart / 8][4], av[kPart / 8][4];
  clear(ak);
  clear(av);
  // the first query that sees key k0
  const int qfirst = pb.causal ? max(0, k0 - (pb.Nk - pb.Nq)) / COLS * COLS : 0;
  const float sl = pb.scale * kLog2e;
  if (k0 < len) {
#pragma unroll 1
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
      const T* qb = q + b * pb.q.b + h * pb.q.h;
      const T* gb = dout + b * pb.dout.b + h * pb.dout.h;
      const long row0 = ((long)b * pb.H + h) * pb.Nq;
#pragma unroll 1
      for (int q0 = qfirst; q0 < pb.Nq; q0 += COLS) {
        __syncthreads();
        load_tile<T, COLS, DP, kThreads>(sQ, qb, pb.q.n, q0, pb.Nq, pb.d, vec);
        load_tile<T, COLS, DP, kThreads>(sG, gb, pb.dout.n, q0, pb.Nq, pb.d, vec);
        for (int x = threadIdx.x; x < COLS; x += kThreads) {
          // a row outside the tensor or without keys: exp(S - inf) = 0
          const bool live = q0 + x < pb.Nq && dense_visible(pb, len, q0 + x) > 0;
          row_l2[x] = live ? dense_lse2(__ldg(lse + row0 + q0 + x)) : INFINITY;
          row_dl[x] = live ? __ldg(delta + row0 + q0 + x) : 0.f;
        }
        tiles_arrived();
        float s[N][4], dp[N][4];
        scores<kOwn, DP>(sK + wr * (DP + 4), sQ + wc * (DP + 4), s);
        scores<kOwn, DP>(sV + wr * (DP + 4), sG + wc * (DP + 4), dp);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int c = wc + n * 8 + lane % 4 * 2 + (x & 1);
            const int key = k0 + wr + lane / 4 + (x >> 1) * 8;
            const bool see = key < dense_visible(pb, len, q0 + c);
            const float p = see ? exp2f(fmaf(s[n][x], sl, -row_l2[c])) : 0.f;
            s[n][x] = p;
            dp[n][x] = see ? p * (dp[n][x] - row_dl[c]) : 0.f;
          }
        accumulate<kOwn, DP>(s, sG + wc * (DP + 4) + part, av);
        accumulate<kOwn, DP>(dp, sQ + wc * (DP + 4) + part, ak);
      }
    }
  }
  tiles_arrived();
  if constexpr (!CHANNELS) {  // the other warps' queries, over K and V
    join_ways<WAYS, DP>(way, sK + wr * (DP + 4), ak);
    join_ways<WAYS, DP>(way, sV + wr * (DP + 4), av);
    if (way > 0) return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = k0 + wr + lane / 4 + 8 * i;
    if (row >= pb.Nk) continue;
    T* kr = dk + b * pb.dk.b + hk * pb.dk.h + (long)row * pb.dk.n;
    T* vr = dv + b * pb.dv.b + hk * pb.dv.h + (long)row * pb.dv.n;
#pragma unroll
    for (int n = 0; n < kPart / 8; ++n) {
      const int c = part + n * 8 + lane % 4 * 2;
      store_pair(kr, ak[n][2 * i] * pb.scale, ak[n][2 * i + 1] * pb.scale, c, pb.d, vec);
      store_pair(vr, av[n][2 * i], av[n][2 * i + 1], c, pb.d, vec);
    }
  }
}

// dQ of a tile of queries: dQ = scale dS K over the tiles of visible keys.
template <typename T, int DP, int ROWS, int COLS, int WAYS>
__global__ void __launch_bounds__(2 * ROWS * WAYS)
    dense_dq_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                    const float* __restrict__ lse, const float* __restrict__ delta,
                    const T* __restrict__ dout, T* __restrict__ dq, DenseProblem pb, bool vec) {
  constexpr int kThreads = 2 * ROWS * WAYS, kOwn = COLS / WAYS, N = kOwn / 8;
  extern __shared__ __align__(16) float smf[];
  float* sQ = smf;
  float* sG = sQ + ROWS * (DP + 4);
  float* sK = sG + ROWS * (DP + 4);
  float* sV = sK + COLS * (DP + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // first row and column
  const int wr = warp / WAYS * 16, way = warp % WAYS, wc = way * kOwn;
  const int tiles = (pb.Nq + ROWS - 1) / ROWS, bh = blockIdx.x / tiles;
  const int q0 = (int)(blockIdx.x % tiles) * ROWS, h = bh % pb.H, b = bh / pb.H;
  const int hk = h / (pb.H / pb.Hkv);
  const int len = dense_len(pb, b);
  const T* kb = k + b * pb.k.b + hk * pb.k.h;
  const T* vb = v + b * pb.v.b + hk * pb.v.h;
  load_tile<T, ROWS, DP, kThreads>(sQ, q + b * pb.q.b + h * pb.q.h, pb.q.n, q0, pb.Nq, pb.d, vec);
  load_tile<T, ROWS, DP, kThreads>(sG, dout + b * pb.dout.b + h * pb.dout.h, pb.dout.n, q0, pb.Nq,
                                   pb.d, vec);
  int vis[2];
  float l2[2], dl[2], acc[DP / 8][4];
  clear(acc);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = q0 + wr + lane / 4 + 8 * i;
    const bool ok = row < pb.Nq;
    const long at = ((long)b * pb.H + h) * pb.Nq + row;
    vis[i] = ok ? dense_visible(pb, len, row) : 0;
    l2[i] = ok ? dense_lse2(__ldg(lse + at)) : 0.f;
    dl[i] = ok ? __ldg(delta + at) : 0.f;
  }
  const int end = dense_visible(pb, len, min(q0 + ROWS, pb.Nq) - 1);
  const float sl = pb.scale * kLog2e;
#pragma unroll 1
  for (int k0 = 0; k0 < end; k0 += COLS) {
    __syncthreads();
    load_tile<T, COLS, DP, kThreads>(sK, kb, pb.k.n, k0, len, pb.d, vec);
    load_tile<T, COLS, DP, kThreads>(sV, vb, pb.v.n, k0, len, pb.d, vec);
    tiles_arrived();
    float s[N][4], dp[N][4];
    scores<kOwn, DP>(sQ + wr * (DP + 4), sK + wc * (DP + 4), s);
    scores<kOwn, DP>(sG + wr * (DP + 4), sV + wc * (DP + 4), dp);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool see = k0 + wc + n * 8 + lane % 4 * 2 + (x & 1) < vis[x >> 1];
        const float p = exp2f(fmaf(s[n][x], sl, -l2[x >> 1]));
        s[n][x] = see ? p * (dp[n][x] - dl[x >> 1]) : 0.f;
      }
    accumulate<kOwn, DP>(s, sK + wc * (DP + 4), acc);
  }
  tiles_arrived();
  join_ways<WAYS, DP>(way, sQ + wr * (DP + 4), acc);  // over the queries
  if (way > 0) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = q0 + wr + lane / 4 + 8 * i;
    if (row >= pb.Nq) continue;
    T* qr = dq + b * pb.dq.b + h * pb.dq.h + (long)row * pb.dq.n;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
      store_pair(qr, acc[n][2 * i] * pb.scale, acc[n][2 * i + 1] * pb.scale,
                 n * 8 + lane % 4 * 2, pb.d, vec);
  }
}

bool rows_allow_four(const void* p, const HeadStrides& s, size_t elt) {
  return (reinterpret_cast<uintptr_t>(p) % (4 * elt)) == 0 && s.b % 4 == 0 && s.h % 4 == 0 &&
         s.n % 4 == 0;
}

// Rows of a CTA: 64 read each streamed tile half as often, 32 where 64 would
// leave the SMs fewer than four CTAs each.
inline bool few(long rows, long heads) { return (rows + 63) / 64 * heads < 4L * num_sms(); }

// Keys of a tile of the forward pass.
constexpr int fwd_cols(int d) { return d <= 128 ? 64 : 32; }

// Ranges of at least two tiles, up to four CTAs of 32 queries per SM.
KeySplit split_keys(const DenseProblem& pb) {
  const int cols = fwd_cols(pb.d);
  const long ctas = (long)((pb.Nq + 31) / 32) * pb.H * pb.B;
  return split_of(pb, (pb.Nk + cols - 1) / cols, ctas, 4L * num_sms(), 2);
}

template <typename T, int DP, int ROWS>
cudaError_t forward_rows(const T* q, const T* k, const T* v, T* out, float* lse,
                         const DenseProblem& pb, const KeySplit& split, bool vec,
                         cudaStream_t stream, int* launches) {
  constexpr int COLS = fwd_cols(DP);
  constexpr int smem = (ROWS + 2 * COLS) * (DP + 4) * (int)sizeof(float);
  constexpr auto kernel = dense_fwd_kernel<T, DP, ROWS, COLS>;
  cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((pb.Nq + ROWS - 1) / ROWS) * pb.H * pb.B * split.splits;
  e = timed_launch("dense_fwd_f32", stream, launches, [&] {
    kernel<<<grid, 4 * ROWS, smem, stream>>>(q, k, v, out, lse, pb, split, vec);
  });
  if (e != cudaSuccess || split.splits == 1) return e;
  return dense_join<T>(out, lse, pb, split, stream, launches);
}

template <typename T, int DP>
cudaError_t forward_dp(const T* q, const T* k, const T* v, T* out, float* lse,
                       const DenseProblem& pb, const KeySplit& split, bool vec,
                       cudaStream_t stream, int* launches) {
  return few(pb.Nq, (long)pb.H * pb.B)
             ? forward_rows<T, DP, 32>(q, k, v, out, lse, pb, split, vec, stream, launches)
             : forward_rows<T, DP, 64>(q, k, v, out, lse, pb, split, vec, stream, launches);
}

template <typename T, int DP, int ROWS, int COLS, int WAYS>
cudaError_t dkv_rows(const T* q, const T* k, const T* v, const float* lse, const float* delta,
                     const T* dout, T* dk, T* dv, const DenseProblem& pb, bool vec,
                     cudaStream_t stream, int* launches) {
  constexpr int smem = 2 * (ROWS + COLS) * (DP + 4) * (int)sizeof(float);
  constexpr auto kernel = dense_dkv_kernel<T, DP, ROWS, COLS, WAYS, (DP == 256)>;
  cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((pb.Nk + ROWS - 1) / ROWS) * pb.Hkv * pb.B;
  return timed_launch("dense_dkv_f32", stream, launches, [&] {
    kernel<<<grid, 2 * ROWS * WAYS, smem, stream>>>(q, k, v, lse, delta, dout, dk, dv, pb, vec);
  });
}

template <typename T, int DP, int ROWS, int COLS, int WAYS>
cudaError_t dq_rows(const T* q, const T* k, const T* v, const float* lse, const float* delta,
                    const T* dout, T* dq, const DenseProblem& pb, bool vec, cudaStream_t stream,
                    int* launches) {
  constexpr int smem = 2 * (ROWS + COLS) * (DP + 4) * (int)sizeof(float);
  constexpr auto kernel = dense_dq_kernel<T, DP, ROWS, COLS, WAYS>;
  cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((pb.Nq + ROWS - 1) / ROWS) * pb.H * pb.B;
  return timed_launch("dense_dq_f32", stream, launches, [&] {
    kernel<<<grid, 2 * ROWS * WAYS, smem, stream>>>(q, k, v, lse, delta, dout, dq, pb, vec);
  });
}

// Fewer than one and a half CTAs of 32 rows per SM: four warps a row block.
inline bool scarce(long rows, long heads) {
  return 2 * ((rows + 31) / 32 * heads) < 3L * num_sms();
}

template <typename T, int DP>
cudaError_t backward_dp(const T* q, const T* k, const T* v, const float* lse, const float* delta,
                        const T* dout, T* dq, T* dk, T* dv, const DenseProblem& pb, bool vec,
                        cudaStream_t stream, int* launches) {
  // (registers of the two sums of 128 channels; four tiles of 64 rows of 256
  // channels exceed shared memory)
  constexpr int kKeyCols = DP == 64 ? 64 : 32, kCols = DP == 256 ? 32 : 64;
  constexpr int kTall = DP == 256 ? 32 : 64, kMany = DP == 256 ? 2 : 4;
  cudaError_t e = cudaSuccess;
  if (pb.Nk > 0) {
    const long heads = (long)pb.Hkv * pb.B;
    const auto run = scarce(pb.Nk, heads) ? dkv_rows<T, DP, 32, kCols, kMany>
                     : few(pb.Nk, heads)  ? dkv_rows<T, DP, 32, kKeyCols, 2>
                                          : dkv_rows<T, DP, kTall, kKeyCols, 2>;
    e = run(q, k, v, lse, delta, dout, dk, dv, pb, vec, stream, launches);
  }
  if (e == cudaSuccess && pb.Nq > 0) {
    const long heads = (long)pb.H * pb.B;
    const auto run = scarce(pb.Nq, heads) ? dq_rows<T, DP, 32, kCols, kMany>
                     : few(pb.Nq, heads)  ? dq_rows<T, DP, 32, kCols, 2>
                                          : dq_rows<T, DP, kTall, kCols, 2>;
    e = run(q, k, v, lse, delta, dout, dq, pb, vec, stream, launches);
  }
  return e;
}

}  // namespace

size_t dense_f32_workspace_bytes(const DenseProblem& pb) {
  return pb.Nq == 0 ? 0 : split_bytes(pb, split_keys(pb));
}

template <typename T>
cudaError_t dense_f32_forward(const T* q, const T* k, const T* v, T* out, float* lse,
                              const DenseProblem& pb, float* workspace, cudaStream_t stream,
                              int* launches) {
  if (pb.Nq == 0) return cudaSuccess;
  const bool vec = pb.d % 4 == 0 && rows_allow_four(q, pb.q, sizeof(T)) &&
                   rows_allow_four(k, pb.k, sizeof(T)) && rows_allow_four(v, pb.v, sizeof(T)) &&
                   rows_allow_four(out, pb.out, sizeof(T));
  KeySplit split = split_keys(pb);
  place_split(pb, workspace, &split);
  const auto forward = pb.d <= 64    ? forward_dp<T, 64>
                       : pb.d <= 128 ? forward_dp<T, 128>
                                     : forward_dp<T, 256>;
  return forward(q, k, v, out, lse, pb, split, vec, stream, launches);
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
cudaError_t dense_f32_backward(const T* q, const T* k, const T* v, const T* out,
                                const float* lse, const T* dout, T* dq, T* dk, T* dv,
                                float* delta, const DenseProblem& pb, cudaStream_t stream,
                                int* launches) {
  bool vec = pb.d % 4 == 0;
  const void* p[7] = {q, k, v, dout, dq, dk, dv};
  const HeadStrides s[7] = {pb.q, pb.k, pb.v, pb.dout, pb.dq, pb.dk, pb.dv};
  for (int x = 0; x < 7; ++x) vec = vec && rows_allow_four(p[x], s[x], sizeof(T));
  cudaError_t e = dense_delta<T>(out, dout, delta, pb, stream, launches);
  if (e != cudaSuccess) return e;
  const auto backward = pb.d <= 64    ? backward_dp<T, 64>
                        : pb.d <= 128 ? backward_dp<T, 128>
                                      : backward_dp<T, 256>;
  return backward(q, k, v, lse, delta, dout, dq, dk, dv, pb, vec, stream, launches);
}

template cudaError_t dense_f32_forward<float>(const float*, const float*, const float*, float*, float*,
                                              const DenseProblem&, float*, cudaStream_t, int*);
template cudaError_t dense_f32_forward<bf16>(const bf16*, const bf16*, const bf16*, bf16*, float*,
                                              const DenseProblem&, float*, cudaStream_t, int*);
template cudaError_t dense_f32_backward<float>(const float*, const float*, const float*,
                                                const float*, const float*, const float*, float*,
                                                float*, float*, float*, const DenseProblem&,
                                                cudaStream_t, int*);
template cudaError_t dense_f32_backward<bf16>(const bf16*, const bf16*, const bf16*, const bf16*,
                                               const float*, const bf16*, bf16*, bf16*, bf16*,
                                               float*, const DenseProblem&, cudaStream_t, int*);
template cudaError_t dense_delta<float>(const float*, const float*, float*, const DenseProblem&,
                                        cudaStream_t, int*);
template cudaError_t dense_delta<bf16>(const bf16*, const bf16*, float*, const DenseProblem&,
                                       cudaStream_t, int*);

}  // namespace monarch
