// The join of a forward pass whose keys were split over CTAs.
#include "dense.cuh"

#include <math.h>

#include <algorithm>

#include "launch.cuh"
#include "tc_ptx.cuh"
#include "timing.cuh"

namespace monarch {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256;

// A warp per row: the ranges weighted by exp2(m - max) and summed in order.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    dense_join_kernel(T* __restrict__ out, float* __restrict__ lse, DenseProblem pb, KeySplit s) {
  tc::pdl_wait();
  const long rows = (long)pb.B * pb.H * pb.Nq;
  const long row = (long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  // lane = range
  const float2 mz = lane < s.splits ? s.mz[lane * rows + row] : make_float2(-INFINITY, 0.f);
  const float m = warp_max(mz.y > 0.f ? mz.x : -INFINITY);
  const bool counts = !(mz.y == 0.f);  // (a sum that is NaN stays)
  const float w = counts ? exp2f(mz.x - (m == -INFINITY ? 0.f : m)) : 0.f;
  const float z = warp_sum(counts ? w * mz.y : 0.f);
  const bool any = __any_sync(0xffffffffu, counts);
  const long bh = row / pb.Nq;
  T* o = out + bh / pb.H * pb.out.b + bh % pb.H * pb.out.h + row % pb.Nq * pb.out.n;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int r = 0; r < s.splits; ++r) {
    const float f = __shfl_sync(0xffffffffu, w, r);
    const bool written = __shfl_sync(0xffffffffu, (int)counts, r);
    const float* p = s.o + (r * rows + row) * pb.d;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = written && i * 32 + lane < pb.d ? p[i * 32 + lane] : 0.f;
      acc[i] = fmaf(x, f, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i * 32 + lane < pb.d) o[i * 32 + lane] = from_f32<T>(any ? acc[i] / z : 0.f);
  if (lane == 0) lse[row] = any ? (m + log2f(z)) * kLn2 : -INFINITY;
}

}  // namespace

KeySplit split_of(const DenseProblem& pb, int n, long have, long ctas, int least) {
  KeySplit s;
  const long want = std::min({ctas / std::max(1L, have), (long)(n / least), (long)kMaxSplits});
  const int ranges = (int)std::max(1L, want);
  s.per = (n + ranges - 1) / ranges;
  s.splits = s.per > 0 ? (n + s.per - 1) / s.per : 1;
  return s;
}

size_t split_bytes(const DenseProblem& pb, const KeySplit& s) {
  return s.splits == 1
             ? 0
             : ((size_t)s.splits * pb.B * pb.H * pb.Nq * (pb.d + 2) + 1) * sizeof(float);
}

// Rows of d floats first (16-byte aligned for a d that is a multiple of 4), then
// pairs, on an even float.
void place_split(const DenseProblem& pb, float* workspace, KeySplit* s) {
  if (s->splits == 1) return;
  const size_t rows = (size_t)s->splits * pb.B * pb.H * pb.Nq;
  s->o = workspace;
  s->mz = reinterpret_cast<float2*>(workspace + rows * pb.d + (rows * pb.d & 1));
}

template <typename T>
cudaError_t dense_join(T* out, float* lse, const DenseProblem& pb, const KeySplit& s,
                       cudaStream_t stream, int* launches) {
  const long rows = (long)pb.B * pb.H * pb.Nq, each = kThreads / 32;
  return timed_launch("dense_join", stream, launches, [&] {
    return launch_pdl(dense_join_kernel<T>, dim3((unsigned)((rows + each - 1) / each)),
                      dim3(kThreads), 0, stream, out, lse, pb, s);
  });
}

template cudaError_t dense_join<float>(float*, float*, const DenseProblem&, const KeySplit&,
                                       cudaStream_t, int*);
template cudaError_t dense_join<bf16>(bf16*, float*, const DenseProblem&, const KeySplit&,
                                      cudaStream_t, int*);

}  // namespace monarch
