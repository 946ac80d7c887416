// Rotary positions of q and k: each pair (a, b) of a token's channels turns
// by the angle t = position * frequency of the pair,
//   a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t)
// (inverse: by -t, which is the gradient with respect to the input).
// The rotated channels are the first `rot` of a token, cut into one section
// per position axis; a pair is two neighbours of a section (interleaved) or
// the same place of its two halves.  The other channels are copied.
//
// Angles are far too large for 32 bits (a position of 10^6 leaves 2^-4 rad):
// position * (frequency / 2 pi) is formed and reduced to a fraction of a turn
// in 64 bits, then sincospi runs in 32 on a value in [-1, 1] (error 1e-7).
// Each CTA forms the cosines and sines of its token once, in shared memory,
// for every head of q and k.
#include "dense.cuh"

#include <math.h>

#include "timing.cuh"

namespace monarch {
namespace {

constexpr int kThreads = 256;

// First and second channel of pair r, its axis.
__device__ __forceinline__ void pair_channels(const RotaryProblem& pb, int r, int* first,
                                              int* second, int* axis) {
  int a = 0, start = 0;
  while (a + 1 < pb.axes && r >= pb.dims[a] / 2) {
    r -= pb.dims[a] / 2;
    start += pb.dims[a];
    ++a;
  }
  *axis = a;
  *first = pb.interleaved ? start + 2 * r : start + r;
  *second = pb.interleaved ? *first + 1 : *first + pb.dims[a] / 2;
}

__device__ __forceinline__ int token_position(const RotaryProblem& pb, int b, int n, int axis) {
  if (pb.positions) return __ldg(pb.positions + b * pb.pos_b + (long)axis * pb.N + n);
  int inner = 1;
  for (int a = pb.axes - 1; a > axis; --a) inner *= pb.grid[a];
  return n / inner % pb.grid[axis];
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(const T* q, const T* k, T* qo, T* ko,
                  const __grid_constant__ RotaryProblem pb) {
  __shared__ float2 cs[kRotaryPairs];
  __shared__ int2 ch[kRotaryPairs];
  const int n = blockIdx.x % pb.N, b = blockIdx.x / pb.N;
  const int pairs = pb.rot / 2;
  for (int r = threadIdx.x; r < pairs; r += kThreads) {
    int first, second, axis;
    pair_channels(pb, r, &first, &second, &axis);
    double t = token_position(pb, b, n, axis) * pb.turns[r];
    t -= rint(t);
    float s, c;
    sincospif(2.f * (float)t, &s, &c);
    if (pb.inverse) s = -s;
    cs[r] = make_float2(c * pb.magnitude, s * pb.magnitude);
    ch[r] = make_int2(first, second);
  }
  __syncthreads();
  // a unit is a pair, or a channel that is copied
  const int units = pairs + pb.d - pb.rot;
  const int total = (pb.H[0] + pb.H[1]) * units;
  for (int x = threadIdx.x; x < total; x += kThreads) {
    int h = x / units;
    const int u = x % units, t = h >= pb.H[0];
    if (t) h -= pb.H[0];
    const T* src = (t ? k : q) + b * pb.in[t].b + h * pb.in[t].h + n * pb.in[t].n;
    T* dst = (t ? ko : qo) + b * pb.out[t].b + h * pb.out[t].h + n * pb.out[t].n;
    if (u < pairs) {
      const float2 w = cs[u];
      const int2 c = ch[u];
      const float a = to_f32(src[c.x]), e = to_f32(src[c.y]);
      dst[c.x] = from_f32<T>(a * w.x - e * w.y);
      dst[c.y] = from_f32<T>(e * w.x + a * w.y);
    } else {
      dst[u + pairs] = src[u + pairs];
    }
  }
}

}  // namespace

template <typename T>
cudaError_t rotary_forward(const T* const in[2], T* const out[2], const RotaryProblem& pb,
                           cudaStream_t stream, int* launches) {
  return timed_launch("rotary", stream, launches, [&] {
    rotary_kernel<T><<<(unsigned)pb.B * pb.N, kThreads, 0, stream>>>(in[0], in[1], out[0], out[1],
                                                                    pb);
  });
}

template cudaError_t rotary_forward<float>(const float* const[2], float* const[2],
                                           const RotaryProblem&, cudaStream_t, int*);
template cudaError_t rotary_forward<bf16>(const bf16* const[2], bf16* const[2],
                                          const RotaryProblem&, cudaStream_t, int*);

}  // namespace monarch
