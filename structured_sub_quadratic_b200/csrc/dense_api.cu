// C ABI of the exact-attention operators (declared in include/monarch_attn.h):
// argument checks, the choice of kernels, and nothing kept between calls (the
// caller passes the workspace, so calls on different streams and captured
// graphs share no state).
#include "monarch_attn.h"

#include <math.h>

#include <initializer_list>

#include "dense.cuh"
#include "entry.cuh"

namespace {

using monarch::bf16;
using monarch::DecodeProblem;
using monarch::DenseProblem;
using monarch::HeadStrides;
using monarch::RotaryProblem;

size_t elt_size(int dtype) { return dtype == MONARCH_DTYPE_BF16 ? 2 : 4; }

// One strided (B, H, N, d) argument.
struct View {
  const void* ptr;
  long B, H, N, d;
  HeadStrides s;
  bool empty() const { return B == 0 || H == 0 || N == 0; }
  // elements from the first to behind the last
  long extent() const { return (B - 1) * s.b + (H - 1) * s.h + (N - 1) * s.n + d; }
};

// Strides are non-negative, offsets stay within 2^40 elements, and the
// pointer is aligned to an element.
bool view_ok(const View& v, size_t elt) {
  if (v.empty()) return true;
  if (!v.ptr || reinterpret_cast<uintptr_t>(v.ptr) % elt) return false;
  const long size[3] = {v.B, v.H, v.N}, step[3] = {v.s.b, v.s.h, v.s.n};
  for (int x = 0; x < 3; ++x)
    if (size[x] > 1 && (step[x] < 0 || step[x] > (1L << 40) / (size[x] - 1))) return false;
  return v.extent() <= (1L << 40);
}

// No two elements of an output share an address: sorted by stride, each
// dimension steps over everything inside it.
bool distinct(const View& v) {
  if (v.empty()) return true;
  long size[3] = {v.B, v.H, v.N}, step[3] = {v.s.b, v.s.h, v.s.n};
  for (int x = 0; x < 3; ++x)
    for (int y = x + 1; y < 3; ++y)
      if (step[y] < step[x]) {
        long t = step[x]; step[x] = step[y]; step[y] = t;
        t = size[x]; size[x] = size[y]; size[y] = t;
      }
  long inner = v.d;
  for (int x = 0; x < 3; ++x) {
    if (size[x] == 1) continue;
    if (step[x] < inner) return false;
    inner = step[x] * (size[x] - 1) + inner;
  }
  return true;
}

bool ranges_meet(const void* a, size_t na, const void* b, size_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return na && nb && x < y + nb && y < x + na;
}

// The lengths of a dense call: aligned, and apart from what it writes.
bool lens_ok(const int* k_lens, int B, std::initializer_list<View> outputs, size_t elt,
             const void* lse, size_t lse_bytes, const void* workspace, size_t workspace_bytes) {
  if (!k_lens) return true;
  if (reinterpret_cast<uintptr_t>(k_lens) % sizeof(int)) return false;
  const size_t n = B * sizeof(int);
  for (const View& o : outputs)
    if (!o.empty() && ranges_meet(o.ptr, o.extent() * elt, k_lens, n)) return false;
  return !ranges_meet(lse, lse_bytes, k_lens, n) &&
         !ranges_meet(workspace, workspace_bytes, k_lens, n);
}

bool views_meet(const View& a, const View& b, size_t elt) {
  if (a.empty() || b.empty()) return false;
  return ranges_meet(a.ptr, a.extent() * elt, b.ptr, b.extent() * elt);
}

// Strides of dimensions of one element never enter an address: zero, so that
// an odd value in them cannot steer the choice of kernels.
HeadStrides strides_of(const long long* s, int which, long B, long H, long N, long d) {
  HeadStrides r = {H * N * d, N * d, d};
  if (s) r = {s[3 * which], s[3 * which + 1], s[3 * which + 2]};
  if (B <= 1) r.b = 0;
  if (H <= 1) r.h = 0;
  if (N <= 1) r.n = 0;
  return r;
}

// The current device's status word.
int status_word(int** out) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? monarch::device_status_word(dev, out) : monarch::cuda_failure(e);
}

bool dtype_ok(int dtype) { return dtype == MONARCH_DTYPE_BF16 || dtype == MONARCH_DTYPE_F32; }

// Sizes of a dense call; tiles of 32 rows of every head must fit a grid.
int dense_sizes(int B, int H, int Hkv, int Nq, int Nk, int d, int causal, float scale) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || Nq < 0 || Nk < 0) return MONARCH_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return MONARCH_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return MONARCH_ERR_INVALID_ARG;
  if (d < 1 || d > 256) return MONARCH_ERR_UNSUPPORTED;
  if (Nq > (1 << 30) || Nk > (1 << 30) || (long long)B * H > (1LL << 30))
    return MONARCH_ERR_INVALID_ARG;
  const long long tiles = (long long)((Nq > Nk ? Nq : Nk) + 31) / 32;
  if (tiles * B * H > INT_MAX) return MONARCH_ERR_INVALID_ARG;
  return MONARCH_OK;
}

DenseProblem dense_problem(int B, int H, int Hkv, int Nq, int Nk, int d, int causal,
                           const int* k_lens, float scale) {
  DenseProblem pb = {};
  pb.B = B;
  pb.H = H;
  pb.Hkv = Hkv;
  pb.Nq = Nq;
  pb.Nk = Nk;
  pb.d = d;
  pb.causal = causal;
  pb.k_lens = k_lens;
  pb.scale = scale;
  return pb;
}

}  // namespace

extern "C" {

size_t monarch_attn_dense_bwd_workspace_bytes(int B, int H, int Nq) {
  if (B < 1 || H < 1 || Nq < 0) return 0;
  return (size_t)B * H * Nq * sizeof(float);
}

size_t monarch_attn_dense_fwd_workspace_bytes(int dtype, int B, int H, int Nq, int Nk, int d) {
  if (!dtype_ok(dtype) || dense_sizes(B, H, H, Nq, Nk, d, 0, 1.f) != MONARCH_OK) return 0;
  const DenseProblem pb = dense_problem(B, H, H, Nq, Nk, d, 0, nullptr, 1.f);
  // (which kernels take bf16 tensors depends on their alignment, too)
  const size_t f32 = monarch::dense_f32_workspace_bytes(pb);
  const size_t tc = dtype == MONARCH_DTYPE_BF16 ? monarch::dense_tc_workspace_bytes(pb) : 0;
  return f32 > tc ? f32 : tc;
}

int monarch_attn_dense_fwd(int dtype, const void* q, const void* k, const void* v, void* out,
                           float* lse, int B, int H, int Hkv, int Nq, int Nk, int d,
                           const long long* strides, int causal, const int* k_lens, float scale,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  int* launches = monarch::launch_counter();
  *launches = 0;
  if (!dtype_ok(dtype)) return MONARCH_ERR_INVALID_ARG;
  int st = dense_sizes(B, H, Hkv, Nq, Nk, d, causal, scale);
  if (st != MONARCH_OK) return st;
  const size_t elt = elt_size(dtype);
  DenseProblem pb = dense_problem(B, H, Hkv, Nq, Nk, d, causal, k_lens, scale);
  pb.q = strides_of(strides, 0, B, H, Nq, d);
  pb.k = strides_of(strides, 1, B, Hkv, Nk, d);
  pb.v = strides_of(strides, 2, B, Hkv, Nk, d);
  pb.out = strides_of(strides, 3, B, H, Nq, d);
  const View in[3] = {{q, B, H, Nq, d, pb.q}, {k, B, Hkv, Nk, d, pb.k}, {v, B, Hkv, Nk, d, pb.v}};
  const View o = {out, B, H, Nq, d, pb.out};
  const size_t lse_bytes = (size_t)B * H * Nq * sizeof(float);
  const size_t need = monarch_attn_dense_fwd_workspace_bytes(dtype, B, H, Nq, Nk, d);
  if (need && (!workspace || reinterpret_cast<uintptr_t>(workspace) & 15u ||
               workspace_bytes < need || ranges_meet(workspace, need, lse, lse_bytes)))
    return MONARCH_ERR_INVALID_ARG;
  for (const View& x : in) {
    if (!view_ok(x, elt) || views_meet(x, o, elt)) return MONARCH_ERR_INVALID_ARG;
    if (!x.empty() && (ranges_meet(x.ptr, x.extent() * elt, lse, lse_bytes) ||
                       ranges_meet(x.ptr, x.extent() * elt, workspace, need)))
      return MONARCH_ERR_INVALID_ARG;
  }
  if (!view_ok(o, elt) || !distinct(o)) return MONARCH_ERR_INVALID_ARG;
  if (Nq > 0 && (!lse || reinterpret_cast<uintptr_t>(lse) % sizeof(float) ||
                 ranges_meet(out, o.extent() * elt, lse, lse_bytes) ||
                 ranges_meet(out, o.extent() * elt, workspace, need)))
    return MONARCH_ERR_INVALID_ARG;
  if (!lens_ok(k_lens, B, {o}, elt, lse, lse_bytes, workspace, need))
    return MONARCH_ERR_INVALID_ARG;
  cudaError_t e;
  if (dtype == MONARCH_DTYPE_F32) {
    e = monarch::dense_f32_forward<float>(
        static_cast<const float*>(q), static_cast<const float*>(k), static_cast<const float*>(v),
        static_cast<float*>(out), lse, pb, static_cast<float*>(workspace), stream, launches);
  } else if (Nq > 0 && Nk > 0 && monarch::dense_tc_rows(q, pb.q, Nq, d) &&
             monarch::dense_tc_rows(k, pb.k, Nk, d) && monarch::dense_tc_rows(v, pb.v, Nk, d) &&
             monarch::dense_tc_rows(out, pb.out, Nq, d)) {
    int* status = nullptr;
    if ((st = status_word(&status)) != MONARCH_OK) return st;
    e = monarch::dense_tc_forward(static_cast<const bf16*>(q), static_cast<const bf16*>(k),
                                  static_cast<const bf16*>(v), static_cast<bf16*>(out), lse, pb,
                                  static_cast<float*>(workspace), status, stream, launches);
  } else {
    e = monarch::dense_f32_forward<bf16>(
        static_cast<const bf16*>(q), static_cast<const bf16*>(k), static_cast<const bf16*>(v),
        static_cast<bf16*>(out), lse, pb, static_cast<float*>(workspace), stream, launches);
  }
  return e == cudaSuccess ? MONARCH_OK : monarch::cuda_failure(e);
}

int monarch_attn_dense_bwd(int dtype, const void* q, const void* k, const void* v,
                           const void* out, const float* lse, const void* dout, void* dq,
                           void* dk, void* dv, int B, int H, int Hkv, int Nq, int Nk, int d,
                           const long long* strides, int causal, const int* k_lens, float scale,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  int* launches = monarch::launch_counter();
  *launches = 0;
  if (!dtype_ok(dtype)) return MONARCH_ERR_INVALID_ARG;
  int st = dense_sizes(B, H, Hkv, Nq, Nk, d, causal, scale);
  if (st != MONARCH_OK) return st;
  const size_t elt = elt_size(dtype);
  DenseProblem pb = dense_problem(B, H, Hkv, Nq, Nk, d, causal, k_lens, scale);
  pb.q = strides_of(strides, 0, B, H, Nq, d);
  pb.k = strides_of(strides, 1, B, Hkv, Nk, d);
  pb.v = strides_of(strides, 2, B, Hkv, Nk, d);
  pb.out = strides_of(strides, 3, B, H, Nq, d);
  pb.dout = strides_of(strides, 4, B, H, Nq, d);
  pb.dq = strides_of(strides, 5, B, H, Nq, d);
  pb.dk = strides_of(strides, 6, B, Hkv, Nk, d);
  pb.dv = strides_of(strides, 7, B, Hkv, Nk, d);
  const View in[5] = {{q, B, H, Nq, d, pb.q},
                      {k, B, Hkv, Nk, d, pb.k},
                      {v, B, Hkv, Nk, d, pb.v},
                      {out, B, H, Nq, d, pb.out},
                      {dout, B, H, Nq, d, pb.dout}};
  const View o[3] = {{dq, B, H, Nq, d, pb.dq}, {dk, B, Hkv, Nk, d, pb.dk}, {dv, B, Hkv, Nk, d, pb.dv}};
  const size_t lse_bytes = (size_t)B * H * Nq * sizeof(float);
  const size_t need = monarch_attn_dense_bwd_workspace_bytes(B, H, Nq);
  if (Nq > 0 && (!lse || reinterpret_cast<uintptr_t>(lse) % sizeof(float)))
    return MONARCH_ERR_INVALID_ARG;
  if (need && (!workspace || reinterpret_cast<uintptr_t>(workspace) & 15u ||
               workspace_bytes < need || ranges_meet(workspace, need, lse, lse_bytes)))
    return MONARCH_ERR_INVALID_ARG;
  for (const View& x : in) {
    if (!view_ok(x, elt)) return MONARCH_ERR_INVALID_ARG;
    if (!x.empty() && ranges_meet(workspace, need, x.ptr, x.extent() * elt))
      return MONARCH_ERR_INVALID_ARG;
  }
  for (int a = 0; a < 3; ++a) {
    if (!view_ok(o[a], elt) || !distinct(o[a])) return MONARCH_ERR_INVALID_ARG;
    for (const View& x : in)
      if (views_meet(x, o[a], elt)) return MONARCH_ERR_INVALID_ARG;
    for (int b = a + 1; b < 3; ++b)
      if (views_meet(o[a], o[b], elt)) return MONARCH_ERR_INVALID_ARG;
    if (!o[a].empty() && (ranges_meet(workspace, need, o[a].ptr, o[a].extent() * elt) ||
                          ranges_meet(lse, lse_bytes, o[a].ptr, o[a].extent() * elt)))
      return MONARCH_ERR_INVALID_ARG;
  }
  if (!lens_ok(k_lens, B, {o[0], o[1], o[2]}, elt, nullptr, 0, workspace, need))
    return MONARCH_ERR_INVALID_ARG;
  float* delta = static_cast<float*>(workspace);
  cudaError_t e;
  if (dtype == MONARCH_DTYPE_F32) {
    e = monarch::dense_f32_backward<float>(
        static_cast<const float*>(q), static_cast<const float*>(k), static_cast<const float*>(v),
        static_cast<const float*>(out), lse, static_cast<const float*>(dout),
        static_cast<float*>(dq), static_cast<float*>(dk), static_cast<float*>(dv), delta, pb,
        stream, launches);
    return e == cudaSuccess ? MONARCH_OK : monarch::cuda_failure(e);
  }
  const bf16 *bq = static_cast<const bf16*>(q), *bk = static_cast<const bf16*>(k),
             *bv = static_cast<const bf16*>(v), *bo = static_cast<const bf16*>(out),
             *bg = static_cast<const bf16*>(dout);
  bf16 *gq = static_cast<bf16*>(dq), *gk = static_cast<bf16*>(dk), *gv = static_cast<bf16*>(dv);
  if (Nq > 0 && Nk > 0 && monarch::dense_tc_rows(q, pb.q, Nq, d) &&
      monarch::dense_tc_rows(k, pb.k, Nk, d) && monarch::dense_tc_rows(v, pb.v, Nk, d) &&
      monarch::dense_tc_rows(dout, pb.dout, Nq, d) && monarch::dense_tc_rows(dq, pb.dq, Nq, d) &&
      monarch::dense_tc_rows(dk, pb.dk, Nk, d) && monarch::dense_tc_rows(dv, pb.dv, Nk, d)) {
    int* status = nullptr;
    if ((st = status_word(&status)) != MONARCH_OK) return st;
    e = monarch::dense_tc_backward(bq, bk, bv, bo, lse, bg, gq, gk, gv, delta, pb, status, stream,
                                   launches);
  } else {
    e = monarch::dense_f32_backward<bf16>(bq, bk, bv, bo, lse, bg, gq, gk, gv, delta, pb, stream,
                                           launches);
  }
  return e == cudaSuccess ? MONARCH_OK : monarch::cuda_failure(e);
}

namespace {

int decode_problem(int dtype, int B, int H, int Hkv, int d, int n_pages, int page_size,
                   int max_pages, float scale, DecodeProblem* pb) {
  if (!dtype_ok(dtype)) return MONARCH_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || n_pages < 0 || page_size < 1 || max_pages < 0)
    return MONARCH_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return MONARCH_ERR_INVALID_ARG;
  if (d < 1 || d > 256) return MONARCH_ERR_UNSUPPORTED;
  if ((long long)max_pages * page_size > (1LL << 30) || (long long)B * H > (1LL << 24))
    return MONARCH_ERR_INVALID_ARG;
  *pb = DecodeProblem{};
  pb->B = B;
  pb->H = H;
  pb->Hkv = Hkv;
  pb->d = d;
  pb->n_pages = n_pages;
  pb->page_size = page_size;
  pb->max_pages = max_pages;
  pb->scale = scale;
  return MONARCH_OK;
}

}  // namespace

size_t monarch_attn_dense_decode_workspace_bytes(int dtype, int B, int H, int Hkv, int d,
                                                 int page_size, int max_pages) {
  DecodeProblem pb;
  if (decode_problem(dtype, B, H, Hkv, d, 0, page_size, max_pages, 1.f, &pb) != MONARCH_OK)
    return 0;
  return monarch::decode_workspace_bytes(pb);
}

int monarch_attn_dense_decode(int dtype, const void* q, const void* k_cache, const void* v_cache,
                              const int* page_table, const int* lens, void* out, float* lse,
                              int B, int H, int Hkv, int d, int n_pages, int page_size,
                              int max_pages, const long long* strides, float scale,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  int* launches = monarch::launch_counter();
  *launches = 0;
  DecodeProblem pb;
  int st = decode_problem(dtype, B, H, Hkv, d, n_pages, page_size, max_pages, scale, &pb);
  if (st != MONARCH_OK) return st;
  const size_t elt = elt_size(dtype);
  // q and out as (B, H, 1, d); the caches as (pages, Hkv, page_size, d)
  const HeadStrides sq = strides_of(strides, 0, B, H, 1, d);
  const HeadStrides sk = strides_of(strides, 1, n_pages, Hkv, page_size, d);
  const HeadStrides sv = strides_of(strides, 2, n_pages, Hkv, page_size, d);
  const HeadStrides so = strides_of(strides, 3, B, H, 1, d);
  const View in[3] = {{q, B, H, 1, d, sq},
                      {k_cache, n_pages, Hkv, page_size, d, sk},
                      {v_cache, n_pages, Hkv, page_size, d, sv}};
  const View o = {out, B, H, 1, d, so};
  if (!view_ok(o, elt) || !distinct(o)) return MONARCH_ERR_INVALID_ARG;
  const size_t rows = (size_t)B * H, out_bytes = o.extent() * elt;
  const size_t need = monarch::decode_workspace_bytes(pb);
  struct Range {
    const void* p;
    size_t n;
  };
  const Range writes[3] = {{out, out_bytes}, {lse, rows * sizeof(float)}, {workspace, need}};
  const Range reads[2] = {{page_table, (size_t)B * max_pages * sizeof(int)},
                          {lens, B * sizeof(int)}};
  if (!lse || !lens || (max_pages > 0 && !page_table)) return MONARCH_ERR_INVALID_ARG;
  for (const void* p : {(const void*)lse, (const void*)lens, (const void*)page_table})
    if (reinterpret_cast<uintptr_t>(p) % 4) return MONARCH_ERR_INVALID_ARG;
  if (need && (!workspace || reinterpret_cast<uintptr_t>(workspace) & 15u ||
               workspace_bytes < need))
    return MONARCH_ERR_INVALID_ARG;
  for (const View& x : in) {
    if (!view_ok(x, elt)) return MONARCH_ERR_INVALID_ARG;
    for (const Range& w : writes)
      if (!x.empty() && ranges_meet(x.ptr, x.extent() * elt, w.p, w.n))
        return MONARCH_ERR_INVALID_ARG;
  }
  for (int a = 0; a < 3; ++a) {
    for (int b = a + 1; b < 3; ++b)
      if (ranges_meet(writes[a].p, writes[a].n, writes[b].p, writes[b].n))
        return MONARCH_ERR_INVALID_ARG;
    for (const Range& r : reads)
      if (ranges_meet(writes[a].p, writes[a].n, r.p, r.n)) return MONARCH_ERR_INVALID_ARG;
  }
  pb.q_b = sq.b;
  pb.q_h = sq.h;
  pb.out_b = so.b;
  pb.out_h = so.h;
  pb.k_page = sk.b;
  pb.k_h = sk.h;
  pb.k_n = sk.n;
  pb.v_page = sv.b;
  pb.v_h = sv.h;
  pb.v_n = sv.n;
  pb.table = page_table;
  pb.lens = lens;
  int* status = nullptr;
  if ((st = status_word(&status)) != MONARCH_OK) return st;
  const cudaError_t e =
      dtype == MONARCH_DTYPE_BF16
          ? monarch::decode_forward<bf16>(static_cast<const bf16*>(q),
                                          static_cast<const bf16*>(k_cache),
                                          static_cast<const bf16*>(v_cache),
                                          static_cast<bf16*>(out), lse, pb,
                                          static_cast<float*>(workspace), status, stream, launches)
          : monarch::decode_forward<float>(static_cast<const float*>(q),
                                           static_cast<const float*>(k_cache),
                                           static_cast<const float*>(v_cache),
                                           static_cast<float*>(out), lse, pb,
                                           static_cast<float*>(workspace), status, stream,
                                           launches);
  return e == cudaSuccess ? MONARCH_OK : monarch::cuda_failure(e);
}

int monarch_attn_rotary(int dtype, const void* q, const void* k, void* q_out, void* k_out, int B,
                        int H, int Hkv, int N, int d, const long long* strides, int n_axes,
                        const int* axis_dims, const int* grid, const int* positions,
                        long long positions_batch_stride, const double* freqs, double magnitude,
                        int interleaved, int inverse, cudaStream_t stream) {
  int* launches = monarch::launch_counter();
  *launches = 0;
  if (!dtype_ok(dtype)) return MONARCH_ERR_INVALID_ARG;
  if (B < 1 || H < 0 || Hkv < 0 || H + (long long)Hkv < 1 || N < 0 || !axis_dims || !freqs)
    return MONARCH_ERR_INVALID_ARG;
  if (d < 1 || d > 256) return MONARCH_ERR_UNSUPPORTED;
  if (n_axes < 1 || n_axes > monarch::kRotaryAxes) return MONARCH_ERR_UNSUPPORTED;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1) ||
      !isfinite(magnitude))
    return MONARCH_ERR_INVALID_ARG;
  if (N > (1 << 30) || (long long)B * N > INT_MAX || ((long long)H + Hkv) * d > (1 << 24))
    return MONARCH_ERR_INVALID_ARG;
  if ((grid == nullptr) == (positions == nullptr)) return MONARCH_ERR_INVALID_ARG;
  RotaryProblem pb = {};
  pb.B = B;
  pb.N = N;
  pb.d = d;
  pb.H[0] = H;
  pb.H[1] = Hkv;
  pb.axes = n_axes;
  long long tokens = 1;
  for (int a = 0; a < n_axes; ++a) {
    if (axis_dims[a] < 2 || axis_dims[a] % 2 || axis_dims[a] > d) return MONARCH_ERR_INVALID_ARG;
    pb.dims[a] = axis_dims[a];
    pb.rot += axis_dims[a];
    if (grid) {
      if (grid[a] < 1 || (tokens *= grid[a]) > N) return MONARCH_ERR_INVALID_ARG;
      pb.grid[a] = grid[a];
    }
  }
  if (pb.rot > d || (grid && tokens != N)) return MONARCH_ERR_INVALID_ARG;
  for (int r = 0; r < pb.rot / 2; ++r) {
    if (!isfinite(freqs[r])) return MONARCH_ERR_INVALID_ARG;
    // whole turns per position leave the angle as it is
    const long double t = freqs[r] / (2 * 3.14159265358979323846264338328L);
    const long double part = t - floorl(t);
    pb.turns[r] = part < 1 ? (unsigned long long)ldexpl(part, 64) : 0;
  }
  pb.positions = positions;
  pb.pos_b = positions_batch_stride;
  if (positions && (reinterpret_cast<uintptr_t>(positions) % sizeof(int) ||
                    (pb.pos_b != 0 && (pb.pos_b < (long)n_axes * N || pb.pos_b > (1L << 40)))))
    return MONARCH_ERR_INVALID_ARG;
  pb.interleaved = interleaved;
  pb.inverse = inverse;
  pb.magnitude = (float)magnitude;
  const size_t elt = elt_size(dtype);
  const void* in_ptr[2] = {q, k};
  void* out_ptr[2] = {q_out, k_out};
  View in[2], out[2];
  for (int t = 0; t < 2; ++t) {
    pb.in[t] = strides_of(strides, 2 * t, B, pb.H[t], N, d);
    pb.out[t] = strides_of(strides, 2 * t + 1, B, pb.H[t], N, d);
    in[t] = {in_ptr[t], B, pb.H[t], N, d, pb.in[t]};
    out[t] = {out_ptr[t], B, pb.H[t], N, d, pb.out[t]};
    if (!view_ok(in[t], elt) || !view_ok(out[t], elt) || !distinct(out[t]))
      return MONARCH_ERR_INVALID_ARG;
  }
  if (N == 0) return MONARCH_OK;
  const size_t pos_bytes =
      positions ? (size_t)((B - 1) * pb.pos_b + (long)n_axes * N) * sizeof(int) : 0;
  // An output is its own input (rotated in place), or apart from both inputs.
  // Two tensors that interleave in memory are apart when each token holds
  // the heads of one behind the heads of the other.
  auto apart = [&](const View& a, const View& b) {
    if (!views_meet(a, b, elt)) return true;
    if (a.s.b != b.s.b || a.s.n != b.s.n) return false;
    const View &lo = a.ptr < b.ptr ? a : b, &hi = a.ptr < b.ptr ? b : a;
    const long gap = (static_cast<const char*>(hi.ptr) - static_cast<const char*>(lo.ptr));
    const long lo_span = (lo.H - 1) * lo.s.h + lo.d, hi_span = (hi.H - 1) * hi.s.h + hi.d;
    if (gap % (long)elt) return false;
    const long end = gap / (long)elt + hi_span;
    return lo_span <= gap / (long)elt && (N == 1 || end <= a.s.n) &&
           (B == 1 || (N - 1) * a.s.n + end <= a.s.b);
  };
  auto same = [](const View& a, const View& b) {
    return a.ptr == b.ptr && a.s.b == b.s.b && a.s.h == b.s.h && a.s.n == b.s.n;
  };
  if (!apart(out[0], out[1])) return MONARCH_ERR_INVALID_ARG;
  for (int t = 0; t < 2; ++t) {
    if (!same(in[t], out[t]) && !apart(in[t], out[t])) return MONARCH_ERR_INVALID_ARG;
    if (!apart(in[t], out[1 - t])) return MONARCH_ERR_INVALID_ARG;
    if (!out[t].empty() && ranges_meet(out[t].ptr, out[t].extent() * elt, positions, pos_bytes))
      return MONARCH_ERR_INVALID_ARG;
  }
  cudaError_t e;
  if (dtype == MONARCH_DTYPE_BF16) {
    const bf16* src[2] = {static_cast<const bf16*>(q), static_cast<const bf16*>(k)};
    bf16* dst[2] = {static_cast<bf16*>(q_out), static_cast<bf16*>(k_out)};
    e = monarch::rotary_forward<bf16>(src, dst, pb, stream, launches);
  } else {
    const float* src[2] = {static_cast<const float*>(q), static_cast<const float*>(k)};
    float* dst[2] = {static_cast<float*>(q_out), static_cast<float*>(k_out)};
    e = monarch::rotary_forward<float>(src, dst, pb, stream, launches);
  }
  return e == cudaSuccess ? MONARCH_OK : monarch::cuda_failure(e);
}

}  // extern "C"
