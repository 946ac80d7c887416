// Rotary positions of q and k: each pair (a, b) of a token's channels turns
// by the angle t = position * frequency of the pair,
//   a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t)
// (inverse: by -t, which is the gradient with respect to the input).
// The rotated channels are the first `rot` of a token, cut into one section
// per position axis; a pair is two neighbours of a section (interleaved) or
// the same place of its two halves.  The other channels are copied.
//
// Angles are far too large for 32 bits (a position of 10^6 leaves 2^-4 rad).
// A frequency is held as a fraction of a turn in units of 2^-64, so that
// position * frequency modulo 2^64 is the angle reduced to one turn, off by less
// than 2^-32 turns for any 32-bit position (the fraction is cut, 2^-64, and its
// division rounded, 2^-66, for frequencies up to 1); its top 32 bits are the
// angle.
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

// Cosine and sine of pair r at `position`.  For bf16 rows the special function
// unit's (off by 2^-21 on [-pi, pi], a thousandth of bf16's step): with few
// heads to share them, the angles cost more than the rows.
template <typename T>
__device__ __forceinline__ float2 turn(const RotaryProblem& pb, const unsigned long long* turns,
                                       int r, int position) {
  const unsigned long long t = (unsigned long long)(long long)position * turns[r];
  const float half_turns = (float)(int)(t >> 32) * 0x1p-31f;  // in [-1, 1]
  float s, c;
  if constexpr (sizeof(T) == 2)
    __sincosf(half_turns * 3.14159265f, &s, &c);
  else
    sincospif(half_turns, &s, &c);
  if (pb.inverse) s = -s;
  return make_float2(c * pb.magnitude, s * pb.magnitude);
}

// The frequencies in shared memory: lanes that read different entries of a
// kernel argument wait for one another.
__device__ __forceinline__ void copy_turns(unsigned long long* turns, const RotaryProblem& pb) {
  for (int r = threadIdx.x; r < pb.rot / 2; r += blockDim.x) turns[r] = pb.turns[r];
  __syncthreads();
}

// The positions of one token.
struct Place {
  int p[kRotaryAxes];

  __device__ __forceinline__ Place(const RotaryProblem& pb, int b, int n) {
#pragma unroll
    for (int a = kRotaryAxes - 1; a >= 0; --a) {
      p[a] = 0;
      if (a >= pb.axes) continue;
      if (pb.positions) {
        p[a] = __ldg(pb.positions + b * pb.pos_b + (long)a * pb.N + n);
      } else {
        const int outer = n / pb.grid[a];
        p[a] = n - outer * pb.grid[a];
        n = outer;
      }
    }
  }
};

// Where channel c < rot lies: its section's start and half, and its position.
struct Section {
  int start, half, position;

  __device__ __forceinline__ Section(const RotaryProblem& pb, const Place& at, int c) {
    start = 0;
    half = pb.dims[0] / 2;
    position = at.p[0];
    int end = pb.dims[0];
#pragma unroll
    for (int a = 1; a < kRotaryAxes; ++a)
      if (a < pb.axes && c >= end) {
        start = end;
        half = pb.dims[a] / 2;
        position = at.p[a];
        end += pb.dims[a];
      }
  }
};

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

// Units of a token, tokens that a CTA takes at a time, heads of a CTA
// (blockIdx.y), and groups of tokens, which the CTAs take in turn.
struct Shape {
  int units, tokens, heads;
  unsigned blocks;
};

template <typename T, Unit U>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(const T* q, const T* k, T* qo, T* ko, const __grid_constant__ RotaryProblem pb,
                  Shape sh) {
  constexpr int E = U == Unit::kPairs ? 1 : 16 / (int)sizeof(T);
  constexpr int kTurns = U == Unit::kInterleaved ? E / 2 : E;
  __shared__ unsigned long long turns[kRotaryPairs];
  copy_turns(turns, pb);
  const int u = threadIdx.x % sh.units;
  for (unsigned block = blockIdx.x; block < sh.blocks; block += gridDim.x) {
    // (tokens fit 31 bits, and a division of 64 costs more than a row)
    const unsigned token = block * sh.tokens + threadIdx.x / sh.units;
    if ((int)threadIdx.x >= sh.units * sh.tokens || token >= (unsigned)pb.B * pb.N) return;
    const int b = (int)(token / pb.N), n = (int)(token - (unsigned)b * pb.N);
    const Place place(pb, b, n);

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
          w[i] = turn<T>(pb, turns, c / 2, Section(pb, place, c).position);
          rotated = i + 1;
        }
      }
    } else {
      const int r = u * E;
      if (2 * r < pb.rot) {
        const Section s(pb, place, 2 * r);  // pair r has channel 2 r of its section, interleaved
        first = pb.interleaved ? 2 * r : s.start / 2 + r;
        second = pb.interleaved ? first + 1 : first + s.half;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) w[i] = turn<T>(pb, turns, r + i, s.position);
      } else {
        first = pb.rot / 2 + r;
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
}

// Halves whose size is no whole chunk (three axes of a 128-channel head, say):
// a warp takes the rows of a few tokens that fill up to 32 chunks, one a lane.
// Each lane turns the channels of its own chunk, x cos t -+ partner sin t, and
// reads the partners, wherever they lie, from the warp's chunks in shared
// memory.  Word w of lane i's chunk sits at 32 w + i, so that lanes reading
// the same place of their chunks touch different banks.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    rotary_staged_kernel(const T* q, const T* k, T* qo, T* ko,
                         const __grid_constant__ RotaryProblem pb, Shape sh) {
  constexpr int E = 16 / (int)sizeof(T), kPerWord = 4 / (int)sizeof(T);
  __shared__ uint32_t buf[kThreads / 32][kBatch][4][32];
  __shared__ unsigned long long turns[kRotaryPairs];
  copy_turns(turns, pb);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (unsigned block = blockIdx.x; block < sh.blocks; block += gridDim.x) {
    const unsigned t0 = (block * (kThreads / 32) + warp) * sh.tokens;
    if (t0 >= (unsigned)pb.B * pb.N) return;  // (whole warps)
    const int rows = (int)min((unsigned)sh.tokens, (unsigned)pb.B * pb.N - t0);
    const int row = lane / sh.units, first = lane % sh.units * E;
    const bool mine = row < rows;
    const unsigned token = t0 + (mine ? row : 0);
    const int b = (int)(token / pb.N), n = (int)(token - (unsigned)b * pb.N);
    const Place place(pb, b, n);
    float2 w[E];   // cosine; sine, negative for the first member of a pair
    int other[E];  // byte offset of the partner in a buffer
    int turned = 0;  // channels of the chunk that turn (the first ones)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = first + i;
      other[i] = 0;
      w[i] = make_float2(1.f, 0.f);
      if (c >= pb.rot) continue;
      turned = i + 1;
      const Section s(pb, place, c);
      const int r = c - s.start;
      const bool lead = r < s.half;
      const int at = row * pb.d + (lead ? c + s.half : c - s.half), chunk = at / E, in = at % E;
      other[i] = ((in / kPerWord) * 32 + chunk) * 4 + in % kPerWord * (int)sizeof(T);
      w[i] = turn<T>(pb, turns, s.start / 2 + (lead ? r : r - s.half), s.position);
      if (lead) w[i].y = -w[i].y;
    }
    auto turn_chunk = [&](Chunk<T, E>& x, const uint32_t (*stage)[32]) {
      const char* base = reinterpret_cast<const char*>(stage);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float a = to_f32(x.x[i]), e = to_f32(*reinterpret_cast<const T*>(base + other[i]));
        if (i < turned) x.x[i] = from_f32<T>(fmaf(e, w[i].y, a * w[i].x));
      }
    };
    const int h0 = blockIdx.y * sh.heads, h1 = min(h0 + sh.heads, pb.H[0] + pb.H[1]);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int lo = max(h0 - (t ? pb.H[0] : 0), 0), hi = min(h1 - (t ? pb.H[0] : 0), pb.H[t]);
      const T* src = (t ? k : q) + b * pb.in[t].b + n * pb.in[t].n + lo * pb.in[t].h + first;
      T* dst = (t ? ko : qo) + b * pb.out[t].b + n * pb.out[t].n + lo * pb.out[t].h + first;
      for (int h = lo; h < hi; h += kBatch) {
        Chunk<T, E> x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (mine && h + i < hi) read(x[i], src + i * pb.in[t].h);
        __syncwarp();  // the batch before is read
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (mine && h + i < hi) {
            const uint32_t* word = reinterpret_cast<const uint32_t*>(x[i].x);
#pragma unroll
            for (int y = 0; y < 4; ++y) buf[warp][i][y][lane] = word[y];
          }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (mine && h + i < hi) {
            turn_chunk(x[i], buf[warp][i]);
            write(x[i], dst + i * pb.out[t].h);
          }
        src += kBatch * pb.in[t].h;
        dst += kBatch * pb.out[t].h;
      }
    }
  }
}

// CTAs along the tokens, and the heads of a CTA: with few tokens, the heads
// are spread until there are four CTAs per SM; with many, a CTA takes several
// groups (its copy of the frequencies costs as much as a row of a few heads).
inline dim3 grid_of(const RotaryProblem& pb, long tokens, Shape* sh) {
  const long blocks = ((long)pb.B * pb.N + tokens - 1) / tokens;
  const int heads = pb.H[0] + pb.H[1];
  const int groups =
      (int)std::min<long>(std::min(heads, 65535), std::max(1L, 4L * num_sms() / blocks));
  sh->heads = (heads + groups - 1) / groups;
  sh->blocks = (unsigned)blocks;
  return dim3((unsigned)std::min(blocks, 16L * num_sms()), (heads + sh->heads - 1) / sh->heads);
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
  sh.units = pb.d / (16 / (int)sizeof(T));  // chunks of a token, at most 32
  sh.tokens = 32 / sh.units;                // of a warp
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
  if (chunks && pb.d <= 32 * E) return launch_staged<T>(in, out, pb, stream, launches);
  return launch<T, Unit::kPairs>(in, out, pb, pb.rot / 2 + pb.d - pb.rot, stream, launches);
}

template cudaError_t rotary_forward<float>(const float* const[2], float* const[2],
                                           const RotaryProblem&, cudaStream_t, int*);
template cudaError_t rotary_forward<bf16>(const bf16* const[2], bf16* const[2],
                                          const RotaryProblem&, cudaStream_t, int*);

}  // namespace monarch
