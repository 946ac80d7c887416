// Exact (dense) softmax attention: problem description and launchers shared
// by its entry points (dense_api.cu), the CUDA-core kernels (dense_f32.cu)
// and the paged decode kernels (decode.cu).
//
//   S = scale q k^T,  P = softmax of S over the visible keys,  O = P V,
//   lse = log of the sum of exp(S) over them.
// Key j is visible to query i of batch b when j < k_lens[b] and, for causal
// calls, j <= i + Nk - Nq (the last query sees every key).  A row without a
// visible key, or whose visible keys all score -inf, has O = 0, lse = -inf and
// no gradient.  Query head h reads key/value head h / (H / Hkv).
#pragma once

#include <limits.h>
#include <math.h>

#include "common.cuh"

namespace monarch {

// Element strides of a (B, H, N, d) tensor; the d elements of a token are
// contiguous.
struct HeadStrides {
  long b, h, n;
};

struct DenseProblem {
  int B, H, Hkv, Nq, Nk, d;
  int causal;
  const int* k_lens;  // device, or null: every key
  float scale;        // > 0
  HeadStrides q, k, v, out, dout, dq, dk, dv;
};

// Number of keys of batch b (lengths outside [0, Nk] are taken as the nearer end).
__device__ __forceinline__ int dense_len(const DenseProblem& pb, int b) {
  return pb.k_lens ? min(max(__ldg(pb.k_lens + b), 0), pb.Nk) : pb.Nk;
}

// Keys [0, n) visible to query i of a batch with `len` keys.
__device__ __forceinline__ int dense_visible(const DenseProblem& pb, int len, int i) {
  return pb.causal ? max(0, min(len, i + pb.Nk - pb.Nq + 1)) : len;
}

// A row's lse in log2 units, for P = exp2(S - lse): P = 0 in a row without weights.
__device__ __forceinline__ float dense_lse2(float lse) {
  return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
}

// A forward pass of few CTAs cuts the keys into `splits` ranges of `per` key
// tiles; their unnormalised results [split][b][h][i] are joined in order by a
// second launch (dense_join.cu).
struct KeySplit {
  int splits = 1, per = 0;
  float* o = nullptr;    // [d]
  float2* mz = nullptr;  // maximum in log2 units, sum (0: no key seen, o not written)
};
constexpr int kMaxSplits = 32;  // a lane each in the join

// n tiles of keys in ranges of at least `least` tiles, about `ctas` in all.
KeySplit split_of(const DenseProblem& pb, int n, long have, long ctas, int least);
size_t split_bytes(const DenseProblem& pb, const KeySplit& s);
void place_split(const DenseProblem& pb, float* workspace, KeySplit* s);
template <typename T>
cudaError_t dense_join(T* out, float* lse, const DenseProblem& pb, const KeySplit& s,
                       cudaStream_t stream, int* launches);

// fp32 kernels (dense_f32.cu): every shape, stride and alignment.
size_t dense_f32_workspace_bytes(const DenseProblem& pb);
template <typename T>
cudaError_t dense_f32_forward(const T* q, const T* k, const T* v, T* out, float* lse,
                              const DenseProblem& pb, float* workspace, cudaStream_t stream,
                              int* launches);
template <typename T>
cudaError_t dense_f32_backward(const T* q, const T* k, const T* v, const T* out,
                                const float* lse, const T* dout, T* dq, T* dk, T* dv,
                                float* delta, const DenseProblem& pb, cudaStream_t stream,
                                int* launches);

// Tensor-core kernels (dense_tc.cu): bf16, d a multiple of 8 up to 128, rows
// of 16-byte alignment.
bool dense_tc_rows(const void* p, const HeadStrides& s, int N, int d);
// Bytes of workspace that the forward pass needs (0: none).
size_t dense_tc_workspace_bytes(const DenseProblem& pb);
cudaError_t dense_tc_forward(const bf16* q, const bf16* k, const bf16* v, bf16* out, float* lse,
                             const DenseProblem& pb, float* workspace, int* status,
                             cudaStream_t stream, int* launches);
cudaError_t dense_tc_backward(const bf16* q, const bf16* k, const bf16* v, const bf16* out,
                              const float* lse, const bf16* dout, bf16* dq, bf16* dk, bf16* dv,
                              float* delta, const DenseProblem& pb, int* status,
                              cudaStream_t stream, int* launches);

// delta[b, h, i] = sum_x dout out, (B, H, Nq) contiguous.
template <typename T>
cudaError_t dense_delta(const T* out, const T* dout, float* delta, const DenseProblem& pb,
                        cudaStream_t stream, int* launches);

// One query per sequence and head over a paged cache.
struct DecodeProblem {
  int B, H, Hkv, d;
  int n_pages, page_size, max_pages;
  float scale;                // > 0
  long q_b, q_h, out_b, out_h;  // element strides
  long k_page, k_h, k_n;
  long v_page, v_h, v_n;
  const int* table;  // (B, max_pages)
  const int* lens;   // (B)
};

// Bytes of workspace that a decode call needs (0: none).
size_t decode_workspace_bytes(const DecodeProblem& pb);

template <typename T>
cudaError_t decode_forward(const T* q, const T* k, const T* v, T* out, float* lse,
                           const DecodeProblem& pb, float* workspace, int* status,
                           cudaStream_t stream, int* launches);

// Rotary positions (rotary.cu).
constexpr int kRotaryAxes = 4, kRotaryPairs = 128;

struct RotaryProblem {
  int B, N, d;
  int H[2];            // heads of q and k (0: no such tensor)
  HeadStrides in[2], out[2];
  int axes, rot;       // axes; rotated channels (the first `rot` of each token)
  int dims[kRotaryAxes];
  int grid[kRotaryAxes];  // raster grid of the tokens (positions == null)
  const int* positions;   // device, (axes, N) per batch
  long pos_b;             // elements between batches (0: shared)
  int interleaved, inverse;
  float magnitude;
  // turns per position of each pair, axis after axis, modulo 1, in units of 2^-64
  unsigned long long turns[kRotaryPairs];
};

template <typename T>
cudaError_t rotary_forward(const T* const in[2], T* const out[2], const RotaryProblem& pb,
                           cudaStream_t stream, int* launches);

}  // namespace monarch
