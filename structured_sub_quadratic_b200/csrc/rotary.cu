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
//
// A thread keeps one place of one token (a unit: a pair, or 16-byte chunks of
// pairs) and its cosines and sines in registers, and walks the heads of q and
// k, so each angle is formed once.  Bound: reading and writing every element
// once.
#include "dense.cuh"

#include <math.h>

#include <algorithm>

#include "launch.cuh"
#include "timing.cuh"

namespace monarch {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads whose loads are in flight together

// What a unit holds.  Chunks are read and written as 16 bytes:
//   kPairs        one pair of any layout and alignment (element accesses)
//   kInterleaved  a chunk of neighbouring pairs
//   kHalves       a chunk of first members and the chunk of their partners
enum class Unit { kPairs, kInterleaved, kHalves };

// Cosine and sine of pair r of an axis at `position`.
__device__ __forceinline__ float2 turn(const RotaryProblem& pb, int r, int position) {
  double t = position * pb.turns[r];
  t -= rint(t);
  float s, c;
  sincospif(2.f * (float)t, &s, &c);
  if (pb.inverse) s = -s;
  return make_float2(c * pb.magnitude, s * pb.magnitude);
}

__device__ __forceinline__ int token_position(const RotaryProblem& pb, int b, int n, int axis) {
  if (pb.positions) return __ldg(pb.positions + b * pb.pos_b + (long)axis * pb.N + n);
  int inner = 1;
  for (int a = pb.axes - 1; a > axis; --a) inner *= pb.grid[a];
  return n / inner % pb.grid[axis];
}

template <typename T, int E>
struct alignas(E == 1 ? sizeof(T) : 16) Chunk {  // 16 bytes, or one element
  T x[E];
};

template <typename T, int E>
__device__ __forceinline__ void read(Chunk<T, E>& c, const T* p) {
  if constexpr (E == 1)
    c.x[0] = *p;
  else
    *reinterpret_cast<uint4*>(c.x) = *reinterpret_cast<const uint4*>(p);
}

template <typename T, int E>
__device__ __forceinline__ void write(const Chunk<T, E>& c, T* p) {
  if constexpr (E == 1)
    *p = c.x[0];
  else
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(c.x);
}

// Units of a token, tokens of a CTA, heads of a CTA (blockIdx.y).
struct Shape {
  int units, tokens, heads;
};

template <typename T, Unit U>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(const T* q, const T* k, T* qo, T* ko, const __grid_constant__ RotaryProblem pb,
                  Shape sh) {
  constexpr int E = U == Unit::kPairs ? 1 : 16 / (int)sizeof(T);
  constexpr int kTurns = U == Unit::kInterleaved ? E / 2 : E;
  const int u = threadIdx.x % sh.units;
  const long token = (long)blockIdx.x * sh.tokens + threadIdx.x / sh.units;
  if ((int)threadIdx.x >= sh.units * sh.tokens || token >= (long)pb.B * pb.N) return;
  const int n = (int)(token % pb.N), b = (int)(token / pb.N);

  // The unit's first channels (`first`, and `second` of its partners, -1 for
  // none) and turns.  Pairs are counted axis after axis, then what is copied.
  int first, second = -1, rotated = 0;  // rotated: pairs of an interleaved chunk
  float2 w[kTurns];
  if constexpr (U == Unit::kInterleaved) {
    first = u * E;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int c = first + 2 * i;  // a section starts at an even channel
      if (c < pb.rot) {
        int axis = 0, start = 0;
        while (c >= start + pb.dims[axis]) start += pb.dims[axis++];
        w[i] = turn(pb, c / 2, token_position(pb, b, n, axis));
        rotated = i + 1;
      }
    }
  } else {
    int axis = 0, start = 0, r = u * E;
    while (axis < pb.axes && r >= pb.dims[axis] / 2) {
      r -= pb.dims[axis] / 2;
      start += pb.dims[axis++];
    }
    if (axis < pb.axes) {
      first = pb.interleaved ? start + 2 * r : start + r;
      second = pb.interleaved ? first + 1 : first + pb.dims[axis] / 2;
      const int position = token_position(pb, b, n, axis);
#pragma unroll
      for (int i = 0; i < kTurns; ++i) w[i] = turn(pb, start / 2 + r + i, position);
    } else {
      first = start + r;
    }
  }

  auto rotate = [&](Chunk<T, E>& x, Chunk<T, E>& y) {
    if constexpr (U == Unit::kInterleaved) {
#pragma unroll
      for (int i = 0; i < kTurns; ++i)
        if (i < rotated) {
          const float a = to_f32(x.x[2 * i]), e = to_f32(x.x[2 * i + 1]);
          x.x[2 * i] = from_f32<T>(a * w[i].x - e * w[i].y);
          x.x[2 * i + 1] = from_f32<T>(e * w[i].x + a * w[i].y);
        }
    } else if (second >= 0) {
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const float a = to_f32(x.x[i]), e = to_f32(y.x[i]);
        x.x[i] = from_f32<T>(a * w[i].x - e * w[i].y);
        y.x[i] = from_f32<T>(e * w[i].x + a * w[i].y);
      }
    }
  };

  const int h0 = blockIdx.y * sh.heads, h1 = min(h0 + sh.heads, pb.H[0] + pb.H[1]);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int lo = max(h0 - (t ? pb.H[0] : 0), 0), hi = min(h1 - (t ? pb.H[0] : 0), pb.H[t]);
    const T* src = (t ? k : q) + b * pb.in[t].b + n * pb.in[t].n;
    T* dst = (t ? ko : qo) + b * pb.out[t].b + n * pb.out[t].n;
    for (int h = lo; h < hi; h += kBatch) {
      Chunk<T, E> x[kBatch], y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < hi) {
          const T* p = src + (h + i) * pb.in[t].h;
          read(x[i], p + first);
          if (second >= 0) read(y[i], p + second);
        }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < hi) {
          rotate(x[i], y[i]);
          T* p = dst + (h + i) * pb.out[t].h;
          write(x[i], p + first);
          if (second >= 0) write(y[i], p + second);
        }
    }
  }
}

// Halves whose size is no whole chunk (three axes of a 128-channel head, say):
// a warp takes the rows of a few tokens that fill 32 chunks, reads and writes
// them as chunks, and turns the pairs in shared memory in between.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    rotary_staged_kernel(const T* q, const T* k, T* qo, T* ko,
                         const __grid_constant__ RotaryProblem pb, Shape sh) {
  constexpr int E = 16 / (int)sizeof(T);
  constexpr int kChunks = 64, kPairs = 4;  // of a warp; of a lane (32 chunks hold 128 pairs)
  __shared__ Chunk<T, E> buf[kThreads / 32][kBatch][kChunks];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_chunks = pb.d / E, row_pairs = pb.rot / 2;
  const long t0 = ((long)blockIdx.x * (kThreads / 32) + warp) * sh.tokens;
  const int rows = (int)min((long)sh.tokens, (long)pb.B * pb.N - t0);
  if (rows <= 0) return;
  auto place = [&](int row, int* b) {  // token of a row, and its batch
    *b = (int)((t0 + row) / pb.N);
    return (int)((t0 + row) % pb.N);
  };
  // this lane's chunks and pairs
  int at[kPairs], to[kPairs];
  float2 w[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int x = i * 32 + lane, row = x / row_pairs;
    at[i] = -1;
    if (row >= rows) continue;
    int axis = 0, start = 0, r = x % row_pairs;
    while (r >= pb.dims[axis] / 2) {
      r -= pb.dims[axis] / 2;
      start += pb.dims[axis++];
    }
    int b;
    const int n = place(row, &b);
    at[i] = row * pb.d + start + r;
    to[i] = at[i] + pb.dims[axis] / 2;
    w[i] = turn(pb, start / 2 + r, token_position(pb, b, n, axis));
  }
  long src[2][2], dst[2][2];  // element offsets of the chunks in q and k (-1: none)
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int x = c * 32 + lane, row = x / row_chunks;
    int b;
    const int n = place(min(row, rows - 1), &b);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      src[t][c] = row < rows ? b * pb.in[t].b + n * pb.in[t].n + x % row_chunks * E : -1;
      dst[t][c] = b * pb.out[t].b + n * pb.out[t].n + x % row_chunks * E;
    }
  }
  const bool two = rows * row_chunks > 32;  // uniform: rows of more than 32 chunks
  const int h0 = blockIdx.y * sh.heads, h1 = min(h0 + sh.heads, pb.H[0] + pb.H[1]);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int lo = max(h0 - (t ? pb.H[0] : 0), 0), hi = min(h1 - (t ? pb.H[0] : 0), pb.H[t]);
    const T* in = t ? k : q;
    T* out = t ? ko : qo;
    for (int h = lo; h < hi; h += kBatch) {
      Chunk<T, E> x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < hi && src[t][0] >= 0) read(x[i], in + src[t][0] + (h + i) * pb.in[t].h);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < hi) {
          if (src[t][0] >= 0) buf[warp][i][lane] = x[i];
          if (two && src[t][1] >= 0) {
            read(x[i], in + src[t][1] + (h + i) * pb.in[t].h);
            buf[warp][i][32 + lane] = x[i];
          }
        }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < hi) {
          T* row = buf[warp][i][0].x;
#pragma unroll
          for (int p = 0; p < kPairs; ++p)
            if (at[p] >= 0) {
              const float a = to_f32(row[at[p]]), e = to_f32(row[to[p]]);
              row[at[p]] = from_f32<T>(a * w[p].x - e * w[p].y);
              row[to[p]] = from_f32<T>(e * w[p].x + a * w[p].y);
            }
        }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < hi) {
          if (src[t][0] >= 0)
            write(buf[warp][i][lane], out + dst[t][0] + (h + i) * pb.out[t].h);
          if (two && src[t][1] >= 0)
            write(buf[warp][i][32 + lane], out + dst[t][1] + (h + i) * pb.out[t].h);
        }
      __syncwarp();
    }
  }
}

// CTAs along the tokens, and the heads of a CTA: with few tokens, the heads
// are spread until there are four CTAs per SM.
inline dim3 grid_of(const RotaryProblem& pb, long tokens, Shape* sh) {
  const long blocks = ((long)pb.B * pb.N + tokens - 1) / tokens;
  const int heads = pb.H[0] + pb.H[1];
  const int groups =
      (int)std::min<long>(std::min(heads, 65535), std::max(1L, 4L * num_sms() / blocks));
  sh->heads = (heads + groups - 1) / groups;
  return dim3((unsigned)blocks, (heads + sh->heads - 1) / sh->heads);
}

template <typename T, Unit U>
cudaError_t launch(const T* const in[2], T* const out[2], const RotaryProblem& pb, int units,
                   cudaStream_t stream, int* launches) {
  Shape sh;
  sh.units = units;
  sh.tokens = kThreads / units;
  const dim3 grid = grid_of(pb, sh.tokens, &sh);
  return timed_launch("rotary", stream, launches, [&] {
    rotary_kernel<T, U><<<grid, kThreads, 0, stream>>>(in[0], in[1], out[0], out[1], pb, sh);
  });
}

template <typename T>
cudaError_t launch_staged(const T* const in[2], T* const out[2], const RotaryProblem& pb,
                          cudaStream_t stream, int* launches) {
  Shape sh = {};
  sh.tokens = std::max(1, 32 / (pb.d / (16 / (int)sizeof(T))));  // of a warp
  const dim3 grid = grid_of(pb, sh.tokens * (kThreads / 32), &sh);
  return timed_launch("rotary_staged", stream, launches, [&] {
    rotary_staged_kernel<T><<<grid, kThreads, 0, stream>>>(in[0], in[1], out[0], out[1], pb, sh);
  });
}

}  // namespace

template <typename T>
cudaError_t rotary_forward(const T* const in[2], T* const out[2], const RotaryProblem& pb,
                           cudaStream_t stream, int* launches) {
  constexpr int E = 16 / sizeof(T);
  bool chunks = pb.d % E == 0, halves = true;
  for (int t = 0; t < 2; ++t) {
    if (pb.H[t] == 0) continue;
    for (const HeadStrides& s : {pb.in[t], pb.out[t]})
      chunks = chunks && s.b % E == 0 && s.h % E == 0 && s.n % E == 0;
    for (const void* p : {(const void*)in[t], (const void*)out[t]})
      chunks = chunks && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
  }
  for (int a = 0; a < pb.axes; ++a) halves = halves && pb.dims[a] % (2 * E) == 0;
  if (chunks && pb.interleaved)
    return launch<T, Unit::kInterleaved>(in, out, pb, pb.d / E, stream, launches);
  if (chunks && halves)
    return launch<T, Unit::kHalves>(in, out, pb, pb.rot / (2 * E) + (pb.d - pb.rot) / E, stream,
                                    launches);
  if (chunks) return launch_staged<T>(in, out, pb, stream, launches);
  return launch<T, Unit::kPairs>(in, out, pb, pb.rot / 2 + pb.d - pb.rot, stream, launches);
}

template cudaError_t rotary_forward<float>(const float* const[2], float* const[2],
                                           const RotaryProblem&, cudaStream_t, int*);
template cudaError_t rotary_forward<bf16>(const bf16* const[2], bf16* const[2],
                                          const RotaryProblem&, cudaStream_t, int*);

}  // namespace monarch
