// abi_attention.cu -- the extern "C" entry points of the attention sublayer's
// operators (declared in include/attnres.h): argument checks, then dispatch.
// Nothing here allocates device memory, synchronises, prints or aborts.
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "launch.h"

namespace attnres {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 40;
constexpr int64_t kMaxStride = (int64_t)1 << 31;
constexpr int kMaxHeads = 1 << 16;
constexpr int kMaxGroup = 16;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int vec_elems(int dtype) { return dtype == ATTNRES_BF16 ? 8 : 4; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? ATTNRES_OK : ATTNRES_ERR_CUDA; }
bool good_eps(float eps) { return std::isfinite(eps) && eps >= 0.f; }
// Finite and no zero, and 1 / scale is finite too.
bool good_scale(float s) { return std::isfinite(s) && s != 0.f && std::isfinite(1.f / s); }

// A row stride: a multiple of the vector width; `apart`: no less than the row's width.
int check_stride(int64_t stride, int64_t width, int dtype, bool apart) {
  if (stride % vec_elems(dtype)) return ATTNRES_ERR_ALIGNMENT;
  return stride < 0 || stride > kMaxStride || (apart && stride < width) ? ATTNRES_ERR_SHAPE : ATTNRES_OK;
}

int check_batch(int64_t B, int64_t T, int dtype, int64_t &rows) {
  if (dtype != ATTNRES_F32 && dtype != ATTNRES_BF16) return ATTNRES_ERR_DTYPE;
  if (B < 0 || T < 0 || B > kMaxRows || T > INT32_MAX || (T && B > kMaxRows / T)) return ATTNRES_ERR_SHAPE;
  rows = B * T;
  return ATTNRES_OK;
}

// What the head norm's entry points check of their common arguments.
int check_heads(int64_t B, int64_t T, int Hq, int Hk, int64_t d, int dtype, int64_t q_stride, int64_t k_stride, int rot,
                int interleaved, float eps, int64_t &rows) {
  int st = check_batch(B, T, dtype, rows);
  if (st) return st;
  const int pair = 2 * vec_elems(dtype);
  if (Hq < 1 || Hk < 1 || Hq > kMaxHeads || Hk > kMaxHeads || d < 1) return ATTNRES_ERR_SHAPE;
  if (d % pair || rot % pair) return ATTNRES_ERR_ALIGNMENT;
  if (!head_norm_supported(d, dtype) || rot < 0 || rot > d) return ATTNRES_ERR_SHAPE;
  if (interleaved != 0 && interleaved != 1) return ATTNRES_ERR_VALUE;
  if (!good_eps(eps)) return ATTNRES_ERR_VALUE;
  if ((st = check_stride(q_stride, Hq * d, dtype, false))) return st;
  return check_stride(k_stride, Hk * d, dtype, false);
}

bool misaligned(const void *p, int to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Token indices, and the loops that step past their ends, stay within 32 bits.
int check_pages(int64_t num_pages, int page_size, int max_pages) {
  return num_pages < 0 || page_size < 1 || max_pages < 0 || (int64_t)page_size * max_pages > (int64_t)1 << 30
             ? ATTNRES_ERR_SHAPE : ATTNRES_OK;
}

// An output that is one of the inputs: CTAs would read what others have written.
bool among(const void *out, const void *x, const void *y, const void *z, const void *w = nullptr) {
  return out && (out == x || out == y || out == z || out == w);
}

// An output may lie on its own input, row on row (a work item reads a head
// before it writes it); on other rows some would read what others have written.
bool shifted(const void *out, int64_t out_stride, const void *in, int64_t in_stride, int64_t rows) {
  return out == in && rows > 1 && out_stride != in_stride;
}

int check_linear(int64_t B, int64_t T, int H, int64_t dk, int64_t dv, int dtype, int64_t &rows) {
  int st = check_batch(B, T, dtype, rows);
  if (st) return st;
  if (H < 1 || H > kMaxHeads || dk < 1 || dv < 1) return ATTNRES_ERR_SHAPE;
  if (B > (int64_t)INT32_MAX / 4096 / H) return ATTNRES_ERR_SHAPE;     // the grid's x extent
  if (dk % vec_elems(dtype) || dv % vec_elems(dtype)) return ATTNRES_ERR_ALIGNMENT;
  return linear_supported(dk, dv, dtype) ? ATTNRES_OK : ATTNRES_ERR_SHAPE;
}

int64_t forward_bytes(int64_t B, int64_t T, int H, int64_t dk, int64_t dv, int dtype) {
  return 4 * linear_workspace_floats(B, T, H, (int)dk, (int)dv, dtype);
}
int64_t backward_bytes(int64_t B, int64_t T, int H, int64_t dk, int64_t dv, int dtype) {
  const int64_t a = forward_bytes(B, T, H, dk, dv, dtype), b = forward_bytes(B, T, H, dv, dk, dtype);
  return a > b ? a : b;
}

}  // namespace
}  // namespace attnres

using namespace attnres;

extern "C" {

int attnres_head_norm_rotate(const void *q, const void *k, int64_t B, int64_t T, int Hq, int Hk, int64_t d, int dtype,
                             int64_t q_stride, int64_t k_stride, const float *q_weight, const float *k_weight,
                             const int32_t *positions, const double *inv_freq, int rot, int interleaved, float eps,
                             void *q_out, void *k_out, int64_t q_out_stride, int64_t k_out_stride, void *stream) {
  int64_t rows = 0;
  int st = check_heads(B, T, Hq, Hk, d, dtype, q_stride, k_stride, rot, interleaved, eps, rows);
  if (st) return st;
  if ((st = check_stride(q_out_stride, Hq * d, dtype, true))) return st;
  if ((st = check_stride(k_out_stride, Hk * d, dtype, true))) return st;
  if (rows == 0) return ATTNRES_OK;
  if (!q || !k || !q_out || !k_out || (rot && !inv_freq)) return ATTNRES_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || misaligned(q_weight) ||
      misaligned(k_weight) || misaligned(positions, 4) || misaligned(inv_freq, 8))
    return ATTNRES_ERR_ALIGNMENT;
  if (q_out == k || k_out == q || q_out == k_out || shifted(q_out, q_out_stride, q, q_stride, rows) ||
      shifted(k_out, k_out_stride, k, k_stride, rows))
    return ATTNRES_ERR_VALUE;
  HeadNormArgs a{};
  a.q = q; a.k = k; a.q_stride = q_stride; a.k_stride = k_stride; a.rows = rows; a.T = T;
  a.Hq = Hq; a.Hk = Hk; a.d = (int)d; a.dtype = dtype; a.q_weight = q_weight; a.k_weight = k_weight;
  a.positions = positions; a.inv_freq = inv_freq; a.rot = rot; a.interleaved = interleaved; a.eps = eps;
  a.q_out = q_out; a.k_out = k_out; a.q_out_stride = q_out_stride; a.k_out_stride = k_out_stride;
  a.stream = static_cast<cudaStream_t>(stream);
  return cuda_status(launch_head_norm(a));
}

int attnres_head_norm_rotate_append(const void *q, const void *k, const void *v, int64_t B, int64_t T, int Hq, int Hk,
                                    int64_t d, int dtype, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                    const float *q_weight, const float *k_weight, const int32_t *positions,
                                    const double *inv_freq, int rot, int interleaved, float eps, void *q_out,
                                    int64_t q_out_stride, void *k_cache, void *v_cache, int64_t num_pages,
                                    int page_size, const int32_t *page_table, int max_pages, void *stream) {
  int64_t rows = 0;
  int st = check_heads(B, T, Hq, Hk, d, dtype, q_stride, k_stride, rot, interleaved, eps, rows);
  if (st) return st;
  if ((st = check_stride(v_stride, Hk * d, dtype, false))) return st;
  if ((st = check_stride(q_out_stride, Hq * d, dtype, true))) return st;
  if ((st = check_pages(num_pages, page_size, max_pages))) return st;
  if (rows == 0) return ATTNRES_OK;
  const bool store = num_pages > 0 && max_pages > 0;
  if (!q || !k || !v || !q_out || (rot && !inv_freq)) return ATTNRES_ERR_NULL;
  if (store && (!k_cache || !v_cache || !page_table)) return ATTNRES_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || misaligned(k_cache) ||
      misaligned(v_cache) || misaligned(q_weight) || misaligned(k_weight) || misaligned(positions, 4) ||
      misaligned(inv_freq, 8) || misaligned(page_table, 4))
    return ATTNRES_ERR_ALIGNMENT;
  if (q_out == k || q_out == v || shifted(q_out, q_out_stride, q, q_stride, rows)) return ATTNRES_ERR_VALUE;
  if (store && (k_cache == v_cache || among(k_cache, q, k, v, q_out) || among(v_cache, q, k, v, q_out)))
    return ATTNRES_ERR_VALUE;
  HeadNormArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.rows = rows; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = (int)d; a.dtype = dtype;
  a.q_weight = q_weight; a.k_weight = k_weight; a.positions = positions; a.inv_freq = inv_freq; a.rot = rot;
  a.interleaved = interleaved; a.eps = eps; a.q_out = q_out; a.q_out_stride = q_out_stride;
  a.k_out = k_cache; a.v_cache = v_cache; a.page_table = page_table; a.num_pages = num_pages;
  a.page_size = page_size; a.max_pages = store ? max_pages : 0;
  a.stream = static_cast<cudaStream_t>(stream);
  return cuda_status(launch_head_norm(a));
}

int64_t attnres_head_norm_rotate_backward_workspace_rows(void) { return 2 * (int64_t)head_norm_backward_ctas(); }

int attnres_head_norm_rotate_backward(const void *q, const void *k, int64_t B, int64_t T, int Hq, int Hk, int64_t d,
                                      int dtype, int64_t q_stride, int64_t k_stride, const float *q_weight,
                                      const float *k_weight, const int32_t *positions, const double *inv_freq, int rot,
                                      int interleaved, float eps, const void *grad_q, const void *grad_k,
                                      int64_t grad_q_stride, int64_t grad_k_stride, void *dq, void *dk,
                                      float *grad_q_weight, float *grad_k_weight, float *workspace,
                                      int64_t workspace_rows, void *stream) {
  int64_t rows = 0;
  int st = check_heads(B, T, Hq, Hk, d, dtype, q_stride, k_stride, rot, interleaved, eps, rows);
  if (st) return st;
  if ((st = check_stride(grad_q_stride, Hq * d, dtype, false))) return st;
  if ((st = check_stride(grad_k_stride, Hk * d, dtype, false))) return st;
  if (misaligned(grad_q_weight) || misaligned(grad_k_weight) || misaligned(workspace)) return ATTNRES_ERR_ALIGNMENT;
  const bool weights = grad_q_weight || grad_k_weight;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    cudaError_t e = cudaSuccess;
    if (grad_q_weight) e = cudaMemsetAsync(grad_q_weight, 0, (size_t)d * sizeof(float), s);
    if (e == cudaSuccess && grad_k_weight) e = cudaMemsetAsync(grad_k_weight, 0, (size_t)d * sizeof(float), s);
    return cuda_status(e);
  }
  if (!q || !k || !grad_q || !grad_k || !dq || !dk || (rot && !inv_freq) || (weights && !workspace))
    return ATTNRES_ERR_NULL;
  if (weights && workspace_rows < 2) return ATTNRES_ERR_CAPACITY;
  if (!aligned16(q) || !aligned16(k) || !aligned16(grad_q) || !aligned16(grad_k) || !aligned16(dq) || !aligned16(dk) ||
      misaligned(q_weight) || misaligned(k_weight) || misaligned(positions, 4) || misaligned(inv_freq, 8))
    return ATTNRES_ERR_ALIGNMENT;
  if (dq == dk || among(dq, k, grad_k, nullptr) || among(dk, q, grad_q, nullptr) ||
      shifted(dq, Hq * d, q, q_stride, rows) || shifted(dq, Hq * d, grad_q, grad_q_stride, rows) ||
      shifted(dk, Hk * d, k, k_stride, rows) || shifted(dk, Hk * d, grad_k, grad_k_stride, rows))
    return ATTNRES_ERR_VALUE;
  HeadNormBackwardArgs a{};
  a.q = q; a.k = k; a.grad_q = grad_q; a.grad_k = grad_k;
  a.q_stride = q_stride; a.k_stride = k_stride; a.gq_stride = grad_q_stride; a.gk_stride = grad_k_stride;
  a.rows = rows; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = (int)d; a.dtype = dtype;
  a.q_weight = q_weight; a.k_weight = k_weight; a.positions = positions; a.inv_freq = inv_freq; a.rot = rot;
  a.interleaved = interleaved; a.eps = eps; a.dq = dq; a.dk = dk;
  a.grad_q_weight = grad_q_weight; a.grad_k_weight = grad_k_weight;
  a.workspace = weights ? workspace : nullptr; a.workspace_rows = workspace_rows; a.stream = s;
  return cuda_status(launch_head_norm_backward(a));
}

int64_t attnres_paged_attention_workspace_bytes(int Hq, int Hk, int64_t d, int dtype) {
  if (dtype != ATTNRES_F32 && dtype != ATTNRES_BF16) return ATTNRES_ERR_DTYPE;
  if (Hk < 1 || Hq < Hk || Hq > kMaxHeads || Hq % Hk || Hq / Hk > kMaxGroup || d < 1) return ATTNRES_ERR_SHAPE;
  if (d % vec_elems(dtype)) return ATTNRES_ERR_ALIGNMENT;
  if (!paged_supported(d, dtype)) return ATTNRES_ERR_SHAPE;
  return paged_workspace_bytes(Hq / Hk, d, dtype);
}

int attnres_paged_attention(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                            int64_t num_pages, int page_size, const int32_t *page_table, int max_pages,
                            const int32_t *lengths, int64_t B, int Hq, int Hk, int64_t d, int dtype, float scale,
                            void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
  const int64_t need = attnres_paged_attention_workspace_bytes(Hq, Hk, d, dtype);
  if (need < 0) return (int)need;
  if (B < 0 || B > INT32_MAX / Hk) return ATTNRES_ERR_SHAPE;           // the join's grid
  int st = check_stride(q_stride, Hq * d, dtype, false);
  if (st) return st;
  if ((st = check_pages(num_pages, page_size, max_pages))) return st;
  if (!std::isfinite(scale)) return ATTNRES_ERR_VALUE;
  if (B == 0) return ATTNRES_OK;
  if (!q || !lengths || !out || !workspace) return ATTNRES_ERR_NULL;
  if (num_pages > 0 && max_pages > 0 && (!k_cache || !v_cache || !page_table)) return ATTNRES_ERR_NULL;
  if (workspace_bytes < need) return ATTNRES_ERR_CAPACITY;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || misaligned(k_cache) || misaligned(v_cache) ||
      misaligned(page_table, 4) || misaligned(lengths, 4) || misaligned(lse, 4))
    return ATTNRES_ERR_ALIGNMENT;
  PagedArgs a{};
  a.q = q; a.q_stride = q_stride; a.k_cache = k_cache; a.v_cache = v_cache; a.num_pages = num_pages;
  a.page_size = page_size; a.max_pages = num_pages > 0 ? max_pages : 0; a.page_table = page_table; a.lengths = lengths;
  a.B = B; a.Hq = Hq; a.Hk = Hk; a.d = (int)d; a.dtype = dtype; a.scale = scale; a.out = out; a.lse = lse;
  a.workspace = workspace; a.stream = static_cast<cudaStream_t>(stream);
  return cuda_status(launch_paged(a));
}

int64_t attnres_linear_attention_workspace_bytes(int64_t B, int64_t T, int H, int64_t dk, int64_t dv, int dtype) {
  int64_t rows = 0;
  const int st = check_linear(B, T, H, dk, dv, dtype, rows);
  return st ? st : forward_bytes(B, T, H, dk, dv, dtype);
}
int64_t attnres_linear_attention_backward_workspace_bytes(int64_t B, int64_t T, int H, int64_t dk, int64_t dv,
                                                          int dtype) {
  int64_t rows = 0;
  const int st = check_linear(B, T, H, dk, dv, dtype, rows);
  return st ? st : backward_bytes(B, T, H, dk, dv, dtype);
}

int attnres_linear_attention(const void *q, const void *k, const void *v, int64_t B, int64_t T, int H, int64_t dk,
                             int64_t dv, int dtype, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                             const float *log_decay, float scale, const int32_t *lengths, const float *state,
                             void *out, float *state_out, void *workspace, int64_t workspace_bytes, void *stream) {
  int64_t rows = 0;
  int st = check_linear(B, T, H, dk, dv, dtype, rows);
  if (st) return st;
  if (!good_scale(scale)) return ATTNRES_ERR_VALUE;
  if ((st = check_stride(q_stride, H * dk, dtype, true)) || (st = check_stride(k_stride, H * dk, dtype, true)) ||
      (st = check_stride(v_stride, H * dv, dtype, true)))
    return st;
  if (B == 0 || (rows == 0 && !state_out)) return ATTNRES_OK;
  if (!log_decay || (rows && (!q || !k || !v || !out))) return ATTNRES_ERR_NULL;
  const int64_t need = forward_bytes(B, T, H, dk, dv, dtype);
  if (need && !workspace) return ATTNRES_ERR_NULL;
  if (workspace_bytes < need) return ATTNRES_ERR_CAPACITY;
  if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(out) || misaligned(log_decay, 4) ||
      misaligned(lengths, 4) || misaligned(state) || misaligned(state_out) || misaligned(workspace))
    return ATTNRES_ERR_ALIGNMENT;
  if (rows && among(out, q, k, v)) return ATTNRES_ERR_VALUE;
  LinearArgs a{};
  a.a = q; a.b = k; a.c = v; a.a_stride = q_stride; a.b_stride = k_stride; a.c_stride = v_stride;
  a.out = out; a.B = B; a.T = T; a.H = H; a.da = (int)dk; a.dc = (int)dv; a.dtype = dtype;
  a.log_decay = log_decay; a.lengths = lengths; a.alpha = scale;
  a.carry = scale; a.gain = 1.f; a.first = state; a.first_pow = 1; a.last = state_out;
  a.workspace = static_cast<float *>(workspace); a.stream = static_cast<cudaStream_t>(stream);
  return cuda_status(launch_linear(a));
}

int attnres_linear_attention_backward(const void *q, const void *k, const void *v, int64_t B, int64_t T, int H,
                                      int64_t dk, int64_t dv, int dtype, int64_t q_stride, int64_t k_stride,
                                      int64_t v_stride, const float *log_decay, float scale, const int32_t *lengths,
                                      const float *state, const void *grad_out, int64_t grad_out_stride,
                                      const float *grad_state, void *dq, void *dk_out, void *dv_out,
                                      float *grad_initial, void *workspace, int64_t workspace_bytes, void *stream) {
  int64_t rows = 0;
  int st = check_linear(B, T, H, dk, dv, dtype, rows);
  if (st) return st;
  if (!good_scale(scale)) return ATTNRES_ERR_VALUE;
  if ((st = check_stride(q_stride, H * dk, dtype, true)) || (st = check_stride(k_stride, H * dk, dtype, true)) ||
      (st = check_stride(v_stride, H * dv, dtype, true)) ||
      (st = check_stride(grad_out_stride, H * dv, dtype, true)))
    return st;
  if (grad_initial && grad_initial == grad_state) return ATTNRES_ERR_VALUE;
  if (B == 0 || (rows == 0 && !grad_initial)) return ATTNRES_OK;
  if (!log_decay || (rows && (!q || !k || !v || !grad_out || !dq || !dk_out || !dv_out))) return ATTNRES_ERR_NULL;
  const int64_t need = backward_bytes(B, T, H, dk, dv, dtype);
  if (need && !workspace) return ATTNRES_ERR_NULL;
  if (workspace_bytes < need) return ATTNRES_ERR_CAPACITY;
  if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(grad_out) || misaligned(dq) ||
      misaligned(dk_out) || misaligned(dv_out) || misaligned(log_decay, 4) || misaligned(lengths, 4) || misaligned(state) ||
      misaligned(grad_state) || misaligned(grad_initial) || misaligned(workspace))
    return ATTNRES_ERR_ALIGNMENT;
  if (rows && (among(dq, q, k, v, grad_out) || among(dk_out, q, k, v, grad_out) || among(dv_out, q, k, v, grad_out)))
    return ATTNRES_ERR_VALUE;
  LinearArgs a{};
  a.B = B; a.T = T; a.H = H; a.dtype = dtype; a.log_decay = log_decay; a.lengths = lengths; a.alpha = scale;
  a.workspace = static_cast<float *>(workspace); a.stream = static_cast<cudaStream_t>(stream);
  // dq = scale F(grad_out, v, k; S_0^T)
  a.a = grad_out; a.a_stride = grad_out_stride; a.b = v; a.b_stride = v_stride; a.c = k; a.c_stride = k_stride;
  a.da = (int)dv; a.dc = (int)dk; a.out = dq;
  a.carry = scale; a.gain = 1.f; a.first = state; a.first_t = true; a.first_pow = 1;
  cudaError_t e = cudaSuccess;
  if (rows) e = launch_linear(a);
  // dv, backwards: scale F(k, q, grad_out) + grad_state's part, which scale
  // does not multiply: the state is the gradient itself, scale enters with
  // the tokens.  Its last state is the initial one's gradient
  a.reverse = true;
  a.carry = 1.f; a.gain = scale; a.first = grad_state; a.first_t = false; a.first_pow = 0;
  a.a = k; a.a_stride = k_stride; a.b = q; a.b_stride = q_stride; a.c = grad_out; a.c_stride = grad_out_stride;
  a.da = (int)dk; a.dc = (int)dv; a.out = dv_out;
  a.last = grad_initial; a.last_pow = 1;
  if (e == cudaSuccess) e = launch_linear(a);
  // dk, backwards: scale F(v, grad_out, q) + grad_state^T's part; its states are dv's, transposed
  a.a = v; a.a_stride = v_stride; a.b = grad_out; a.b_stride = grad_out_stride; a.c = q; a.c_stride = q_stride;
  a.da = (int)dv; a.dc = (int)dk; a.first_t = true; a.out = dk_out; a.last = nullptr;
  a.states_ready = a.states_t = true;
  if (rows && e == cudaSuccess) e = launch_linear(a);
  return cuda_status(e);
}

int attnres_linear_attention_step(const void *q, const void *k, const void *v, int64_t B, int H, int64_t dk,
                                  int64_t dv, int dtype, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                  const float *log_decay, float scale, const float *state, float *state_out, void *out,
                                  void *stream) {
  int64_t rows = 0;
  int st = check_linear(B, 1, H, dk, dv, dtype, rows);
  if (st) return st;
  if (!good_scale(scale)) return ATTNRES_ERR_VALUE;
  if ((st = check_stride(q_stride, H * dk, dtype, true)) || (st = check_stride(k_stride, H * dk, dtype, true)) ||
      (st = check_stride(v_stride, H * dv, dtype, true)))
    return st;
  if (B == 0) return ATTNRES_OK;
  if (!q || !k || !v || !log_decay || !state || !state_out || !out) return ATTNRES_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || misaligned(log_decay, 4) || !aligned16(state) ||
      !aligned16(state_out) || !aligned16(out))
    return ATTNRES_ERR_ALIGNMENT;
  if (among(out, q, k, v)) return ATTNRES_ERR_VALUE;
  LinearStepArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.B = B; a.H = H; a.dk = (int)dk; a.dv = (int)dv; a.dtype = dtype; a.log_decay = log_decay; a.scale = scale;
  a.state = state; a.state_out = state_out; a.out = out; a.stream = static_cast<cudaStream_t>(stream);
  return cuda_status(launch_linear_step(a));
}

}  // extern "C"
