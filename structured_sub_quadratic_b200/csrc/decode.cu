// Exact softmax attention of one new token per sequence over a paged cache.
//
// The cache of a sequence is a list of pages; key j sits in row j % page_size
// of page table[b][j / page_size].  The keys are cut into chunks that CTAs
// take independently, each for all query heads that share its key/value head
// (so the cache is read once); a chunk gives its own maximum, sum and
// unnormalised output, and a second launch joins the chunks in order (no
// atomics).  Bound: the bytes of the cache.
#include "dense.cuh"

#include <math.h>

#include <algorithm>

#include "launch.cuh"
#include "timing.cuh"

namespace monarch {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 128;
constexpr int kTile = 32;       // keys per tile
constexpr int kHeads = 8;       // query heads per CTA
constexpr int kBadIndex = MONARCH_DEVICE_BAD_INDEX_FLAG;

struct Split {
  int chunk;   // keys per chunk
  int chunks;  // chunks of the longest sequence that the table allows
  int hg;      // groups of kHeads query heads per key/value head
};

Split make_split(const DecodeProblem& pb) {
  Split s;
  const long top = (long)pb.max_pages * pb.page_size;
  s.hg = (pb.H / pb.Hkv + kHeads - 1) / kHeads;
  const long units = (long)pb.B * pb.Hkv * s.hg;
  // about eight CTAs per SM in all, at least 128 keys each
  long n = std::max(1L, std::min((top + 127) / 128, 8L * num_sms() / std::max(1L, units)));
  s.chunk = (int)(((top + n - 1) / n + kTile - 1) / kTile * kTile);
  s.chunk = std::max(s.chunk, kTile);
  s.chunks = (int)std::max(1L, (top + s.chunk - 1) / s.chunk);
  return s;
}

__device__ __forceinline__ int seq_len(const DecodeProblem& pb, int b, int* status) {
  const int n = __ldg(pb.lens + b);
  const int top = pb.max_pages * pb.page_size;
  if (n < 0 || n > top) {
    atomicCAS(status, 0, kBadIndex);
    return min(max(n, 0), top);
  }
  return n;
}

// Partial results: [chunk][b][h] of (maximum in log2 units, sum), then
// [chunk][b][h][d] of unnormalised outputs.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads)
    decode_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc,
                  float2* __restrict__ part_ml, float* __restrict__ part_o, DecodeProblem pb,
                  Split sp, int* status) {
  constexpr int kPitch = DP + 4, kCols = (DP + kThreads - 1) / kThreads;
  extern __shared__ __align__(16) float smf[];
  float* sQ = smf;                     // [kHeads][DP]
  float* sK = sQ + kHeads * DP;        // [kTile][kPitch]
  float* sV = sK + kTile * kPitch;
  float* sP = sV + kTile * kPitch;     // [kHeads][kTile]
  __shared__ float sM[kHeads], sZ[kHeads], sC[kHeads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int x = blockIdx.x;
  const int c = x % sp.chunks;
  x /= sp.chunks;
  const int hg = x % sp.hg;
  x /= sp.hg;
  const int hk = x % pb.Hkv, b = x / pb.Hkv;
  const int group = pb.H / pb.Hkv;
  const int h0 = hk * group + hg * kHeads;
  const int nh = min(kHeads, (hk + 1) * group - h0);
  const int len = seq_len(pb, b, status);
  const int j0 = c * sp.chunk, j1 = min(len, j0 + sp.chunk);
  if (j0 >= j1) return;  // the join reads no chunk from the length on
  for (int i = tid; i < kHeads * DP; i += kThreads) {
    const int h = i / DP, e = i % DP;
    sQ[i] = h < nh && e < pb.d ? to_f32(q[b * pb.q_b + (h0 + h) * pb.q_h + e]) : 0.f;
  }
  if (tid < kHeads) {
    sM[tid] = -INFINITY;
    sZ[tid] = 0.f;
  }
  float o[kCols][kHeads];
#pragma unroll
  for (int i = 0; i < kCols; ++i)
#pragma unroll
    for (int h = 0; h < kHeads; ++h) o[i][h] = 0.f;
  const float sl = pb.scale * kLog2e;
  for (int t0 = j0; t0 < j1; t0 += kTile) {
    __syncthreads();
    for (int i = tid; i < kTile * DP; i += kThreads) {
      const int r = i / DP, e = i % DP, j = t0 + r;
      float kv = 0.f, vv = 0.f;
      if (j < j1 && e < pb.d) {
        const int page = __ldg(pb.table + (long)b * pb.max_pages + j / pb.page_size);
        if (page >= 0 && page < pb.n_pages) {
          kv = to_f32(kc[page * pb.k_page + hk * pb.k_h + (j % pb.page_size) * pb.k_n + e]);
          vv = to_f32(vc[page * pb.v_page + hk * pb.v_h + (j % pb.page_size) * pb.v_n + e]);
        } else {
          atomicCAS(status, 0, kBadIndex);
        }
      }
      sK[r * kPitch + e] = kv;
      sV[r * kPitch + e] = vv;
    }
    __syncthreads();
    for (int h = warp; h < kHeads; h += kThreads / 32) {  // lane = key
      float s = 0.f;
#pragma unroll 4
      for (int e = 0; e < DP; e += 4) {
        const float4 a = *reinterpret_cast<const float4*>(sQ + h * DP + e);
        const float4 w = *reinterpret_cast<const float4*>(sK + lane * kPitch + e);
        s = fmaf(a.x, w.x, s);
        s = fmaf(a.y, w.y, s);
        s = fmaf(a.z, w.z, s);
        s = fmaf(a.w, w.w, s);
      }
      s = t0 + lane < j1 ? s * sl : -INFINITY;
      const float m0 = sM[h], mn = fmaxf(m0, warp_max(s));
      const float base = mn == -INFINITY ? 0.f : mn;
      const float p = exp2f(s - base);
      sP[h * kTile + lane] = p;
      const float z = warp_sum(p), corr = exp2f(m0 - base);
      __syncwarp();
      if (lane == 0) {
        sM[h] = mn;
        sZ[h] = sZ[h] * corr + z;
        sC[h] = corr;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int e = tid + i * kThreads;
      if (e >= DP) break;
#pragma unroll
      for (int h = 0; h < kHeads; ++h) o[i][h] *= sC[h];
      for (int r = 0; r < kTile; ++r) {
        const float w = sV[r * kPitch + e];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) o[i][h] = fmaf(sP[h * kTile + r], w, o[i][h]);
      }
    }
  }
  __syncthreads();
  const long at = ((long)c * pb.B + b) * pb.H + h0;
  if (tid < nh) part_ml[at + tid] = make_float2(sM[tid], sZ[tid]);
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    const int e = tid + i * kThreads;
    if (e < pb.d)
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h < nh) part_o[(at + h) * pb.d + e] = o[i][h];
  }
}

// One warp per (b, h): the chunks' results weighted by exp(m - max) and summed.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    decode_join_kernel(T* __restrict__ out, float* __restrict__ lse,
                       const float2* __restrict__ part_ml, const float* __restrict__ part_o,
                       DecodeProblem pb, Split sp) {
  const int row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= pb.B * pb.H) return;
  const int b = row / pb.H, h = row % pb.H;
  const int len = min(max(__ldg(pb.lens + b), 0), pb.max_pages * pb.page_size);
  const int n = (len + sp.chunk - 1) / sp.chunk;
  const long step = (long)pb.B * pb.H;
  float m = -INFINITY;
  for (int c = lane; c < n; c += 32) m = fmaxf(m, part_ml[c * step + row].x);
  m = warp_max(m);
  const float base = m == -INFINITY ? 0.f : m;
  float z = 0.f;
  for (int c = lane; c < n; c += 32) {
    const float2 ml = part_ml[c * step + row];
    z += ml.y * exp2f(ml.x - base);
  }
  z = warp_sum(z);
  for (int e = lane; e < pb.d; e += 32) {
    float acc = 0.f;
    for (int c = 0; c < n; ++c)
      acc = fmaf(part_o[(c * step + row) * pb.d + e], exp2f(part_ml[c * step + row].x - base), acc);
    out[b * pb.out_b + h * pb.out_h + e] = from_f32<T>(n > 0 ? acc / z : 0.f);
  }
  if (lane == 0) lse[row] = n > 0 ? (m + log2f(z)) * kLn2 : -INFINITY;
}

template <typename T, int DP>
cudaError_t forward_dp(const T* q, const T* k, const T* v, T* out, float* lse,
                       const DecodeProblem& pb, float* ws, int* status, cudaStream_t stream,
                       int* launches) {
  const Split sp = make_split(pb);
  const long rows = (long)sp.chunks * pb.B * pb.H;
  float2* ml = reinterpret_cast<float2*>(ws);
  float* po = ws + 2 * rows;
  const size_t smem = (kHeads * DP + 2 * kTile * (DP + 4) + kHeads * kTile) * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<T, DP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((long)sp.chunks * sp.hg * pb.Hkv * pb.B);
  e = timed_launch("decode_simt", stream, launches, [&] {
    decode_kernel<T, DP><<<grid, kThreads, smem, stream>>>(q, k, v, ml, po, pb, sp, status);
  });
  if (e != cudaSuccess) return e;
  const unsigned joins = (unsigned)((pb.B * pb.H + kThreads / 32 - 1) / (kThreads / 32));
  return timed_launch("decode_join", stream, launches, [&] {
    decode_join_kernel<T><<<joins, kThreads, 0, stream>>>(out, lse, ml, po, pb, sp);
  });
}

}  // namespace

size_t decode_workspace_bytes(const DecodeProblem& pb) {
  const Split sp = make_split(pb);
  return (size_t)sp.chunks * pb.B * pb.H * (pb.d + 2) * sizeof(float);
}

template <typename T>
cudaError_t decode_forward(const T* q, const T* k, const T* v, T* out, float* lse,
                           const DecodeProblem& pb, float* ws, int* status, cudaStream_t stream,
                           int* launches) {
  if (pb.d <= 64) return forward_dp<T, 64>(q, k, v, out, lse, pb, ws, status, stream, launches);
  if (pb.d <= 128) return forward_dp<T, 128>(q, k, v, out, lse, pb, ws, status, stream, launches);
  return forward_dp<T, 256>(q, k, v, out, lse, pb, ws, status, stream, launches);
}

template cudaError_t decode_forward<float>(const float*, const float*, const float*, float*,
                                           float*, const DecodeProblem&, float*, int*,
                                           cudaStream_t, int*);
template cudaError_t decode_forward<bf16>(const bf16*, const bf16*, const bf16*, bf16*, float*,
                                          const DecodeProblem&, float*, int*, cudaStream_t, int*);

}  // namespace monarch
