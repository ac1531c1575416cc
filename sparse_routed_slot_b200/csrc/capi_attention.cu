// capi_attention.cu -- the extern "C" entry points of the operators beside the mixer: window and paged
// attention and the block norms (declared in include/rsm.h). Arguments are checked on the host before
// anything is launched, as for the mixer's calls.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "common.cuh"
#include "kernels.h"

namespace {

rsm_status fail(rsm_status s, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return rsm::report_error(s, msg);
}

rsm_status finish(cudaError_t e, const char* where) {
  return e == cudaSuccess ? RSM_OK : fail(RSM_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

#define NEED_PTR(p, name)                                                                    \
  do {                                                                                       \
    if (!(p)) return fail(RSM_ERR_INVALID_ARG, "%s must not be NULL", name);                  \
    if (!aligned(p, 16)) return fail(RSM_ERR_INVALID_ARG, "%s must be 16-byte aligned", name); \
  } while (0)
#define MAY_PTR(p, name)                                                                          \
  do {                                                                                            \
    if ((p) && !aligned(p, 16)) return fail(RSM_ERR_INVALID_ARG, "%s must be 16-byte aligned", name); \
  } while (0)

bool known_dtype(rsm_dtype d) { return d == RSM_F32 || d == RSM_BF16; }

// Head counts and sizes every attention call shares.
rsm_status check_heads(int H, int Hkv, int D, rsm_dtype dtype) {
  if (!known_dtype(dtype)) return fail(RSM_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (H < 0 || Hkv < 0 || D < 1) return fail(RSM_ERR_INVALID_ARG, "H and Hkv must be >= 0 and D >= 1");
  if (H > 0 && (Hkv < 1 || H % Hkv != 0))
    return fail(RSM_ERR_INVALID_ARG, "Hkv (%d) must divide H (%d)", Hkv, H);
  if (H > 0 && H / Hkv > 64) return fail(RSM_ERR_UNSUPPORTED, "H / Hkv must not exceed 64 (got %d)", H / Hkv);
  if (D > 256 || D % 8 != 0) return fail(RSM_ERR_UNSUPPORTED, "D must be a multiple of 8 in [8, 256] (got %d)", D);
  return RSM_OK;
}

rsm_status check_scale(float scale) {
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(RSM_ERR_INVALID_ARG, "scale must be positive and finite");
  return RSM_OK;
}

rsm_status check_window(int B, int T, int H, int Hkv, int D, int window, int sinks, rsm_dtype dtype, float scale) {
  if (B < 0 || T < 0) return fail(RSM_ERR_INVALID_ARG, "B and T must be >= 0");
  rsm_status s = check_heads(H, Hkv, D, dtype);
  if (s != RSM_OK) return s;
  if (window < 1) return fail(RSM_ERR_INVALID_ARG, "window must be >= 1 (got %d)", window);
  if (sinks < 0) return fail(RSM_ERR_INVALID_ARG, "sinks must be >= 0 (got %d)", sinks);
  if ((s = check_scale(scale)) != RSM_OK) return s;
  if ((int64_t)T * H > 0x7fffff00 || (int64_t)B * H > 0x7fffffff) return fail(RSM_ERR_UNSUPPORTED, "B*H or T*H too large");
  return RSM_OK;
}

rsm_status check_low(const void* o_low, rsm_dtype dtype) {
  MAY_PTR(o_low, "o_low");
  if (o_low && dtype != RSM_BF16) return fail(RSM_ERR_INVALID_ARG, "o_low goes with bf16 only");
  return RSM_OK;
}

// Launches of 2^31 blocks and more are refused (8 rows per block in the row kernels).
rsm_status check_rows(int64_t rows) {
  if (rows / 8 > 0x7fffff00) return fail(RSM_ERR_UNSUPPORTED, "too many rows");
  return RSM_OK;
}

rsm_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return RSM_OK;
  if (!ws || have < need)
    return fail(RSM_ERR_WORKSPACE, "workspace of %zu bytes required (got %zu)", need, ws ? have : (size_t)0);
  if (!aligned(ws, 256)) return fail(RSM_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return RSM_OK;
}

template <class A> rsm::AttnParams window_params(const A& a) {
  rsm::AttnParams p{};
  p.B = a.B; p.T = a.T; p.H = a.H; p.Hkv = a.Hkv; p.G = a.H / a.Hkv; p.D = a.D;
  p.window = a.window; p.sinks = a.sinks; p.scale = a.scale;
  p.q = a.q; p.k = a.k; p.v = a.v;
  p.splits = 1;
  return p;
}

// bf16: up to 16 query rows per key/value head and sequence over a paged cache are bound by its read and take the
// streaming kernel; else head dimensions to 128, over pages of 8, 16, 32 or multiples of 64 (or dense), run on the
// tensor cores in tiles. Everything else runs in fp32 on CUDA cores. One kernel takes the whole call: the rows are
// those of max_q, and a single token beside a chunk is walked as a chunk's tile (63 of them over 8192 keys and a
// chunk of 512, 16/4 heads of 128: 283 us in one call, 175 and 59 in two).
cudaError_t launch_forward(const rsm::AttnParams& p, rsm_dtype dtype, cudaStream_t st) {
  if (rsm::attn_decode_supported(p, dtype)) return rsm::launch_attn_decode(p, st);
  return rsm::attn_tc_supported(p, dtype) ? rsm::launch_attn_tc(p, st) : rsm::launch_attn_simt(p, dtype, st);
}
int forward_splits(const rsm::AttnParams& p, rsm_dtype dtype) {
  if (rsm::attn_decode_supported(p, dtype)) return rsm::attn_decode_splits(p);
  return rsm::attn_tc_supported(p, dtype) ? rsm::attn_tc_splits(p) : rsm::attn_simt_splits(p);
}

template <class A> cudaError_t validate_qkv(const A& a, cudaStream_t st) {
  const int64_t nq = (int64_t)a.B * a.T * a.H * a.D, nk = (int64_t)a.B * a.T * a.Hkv * a.D;
  cudaError_t e = rsm::launch_check_finite(a.q, nq, a.dtype, st);
  if (e == cudaSuccess) e = rsm::launch_check_finite(a.k, nk, a.dtype, st);
  if (e == cudaSuccess) e = rsm::launch_check_finite(a.v, nk, a.dtype, st);
  return e;
}

rsm_status check_window_backward(const rsm_window_backward_args* a) {
  if (!a) return fail(RSM_ERR_INVALID_ARG, "args must not be NULL");
  rsm_status s = check_window(a->B, a->T, a->H, a->Hkv, a->D, a->window, a->sinks, a->dtype, a->scale);
  if (s != RSM_OK) return s;
  if ((s = check_rows((int64_t)a->B * a->T * a->H)) != RSM_OK) return s;
  if ((int64_t)a->B * a->T * a->H == 0) return RSM_OK;
  NEED_PTR(a->q, "q"); NEED_PTR(a->k, "k"); NEED_PTR(a->v, "v");
  NEED_PTR(a->o, "o"); NEED_PTR(a->lse, "lse"); NEED_PTR(a->dO, "dO");
  if ((s = check_low(a->o_low, a->dtype)) != RSM_OK) return s;
  MAY_PTR(a->dq, "dq"); MAY_PTR(a->dk, "dk"); MAY_PTR(a->dv, "dv");
  return RSM_OK;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t delta_bytes(const rsm_window_backward_args& a) { return up256((size_t)a.B * a.T * a.H * sizeof(float)); }

size_t window_backward_bytes(const rsm_window_backward_args& a) {
  const rsm::AttnParams p = window_params(a);
  return rsm::attn_tc_supported(p, a.dtype) ? rsm::attn_tc_backward_bytes(p)
                                             : delta_bytes(a) + rsm::attn_simt_backward_bytes(p);
}

rsm_status check_cache(int B, int N, int Hkv, int D, int num_pages, int page_size, int table_width) {
  if (B < 0 || N < 0) return fail(RSM_ERR_INVALID_ARG, "B and N must be >= 0");
  if (num_pages < 0 || table_width < 0) return fail(RSM_ERR_INVALID_ARG, "num_pages and table_width must be >= 0");
  if (page_size < 1) return fail(RSM_ERR_INVALID_ARG, "page_size must be >= 1 (got %d)", page_size);
  // (the kernels add up to a tile to a place)
  if ((int64_t)table_width * page_size > 0x7fffff00)
    return fail(RSM_ERR_UNSUPPORTED, "table_width * page_size must not exceed 2^31 - 256");
  return RSM_OK;
}

rsm_status check_paged(const rsm_paged_args* a) {
  if (!a) return fail(RSM_ERR_INVALID_ARG, "args must not be NULL");
  rsm_status s = check_heads(a->H, a->Hkv, a->D, a->dtype);
  if (s != RSM_OK) return s;
  s = check_cache(a->B, a->N, a->Hkv, a->D, a->num_pages, a->page_size, a->table_width);
  if (s != RSM_OK) return s;
  if (a->max_q < 0) return fail(RSM_ERR_INVALID_ARG, "max_q must be >= 0");
  if (a->window < 0 || a->sinks < 0) return fail(RSM_ERR_INVALID_ARG, "window and sinks must be >= 0");
  if ((s = check_scale(a->scale)) != RSM_OK) return s;
  if ((int64_t)a->N * a->H > 0x7fffff00 || (int64_t)a->max_q * a->H > 0x7fffff00 || (int64_t)a->B * a->H > 0x7fffffff)
    return fail(RSM_ERR_UNSUPPORTED, "N*H, max_q*H or B*H too large");
  if ((int64_t)a->N * a->H == 0 || a->B == 0 || a->max_q == 0) return RSM_OK;
  NEED_PTR(a->q, "q"); NEED_PTR(a->o, "o");
  if (a->num_pages > 0) { NEED_PTR(a->k_cache, "k_cache"); NEED_PTR(a->v_cache, "v_cache"); }
  if (a->table_width > 0) NEED_PTR(a->page_table, "page_table");
  NEED_PTR(a->cu_q, "cu_q"); NEED_PTR(a->kv_len, "kv_len");
  MAY_PTR(a->lse, "lse");
  return RSM_OK;
}

rsm::AttnParams paged_params(const rsm_paged_args& a) {
  rsm::AttnParams p{};
  p.B = a.B; p.T = a.N; p.H = a.H; p.Hkv = a.Hkv; p.G = a.H / a.Hkv; p.D = a.D;
  p.window = a.window; p.sinks = a.window > 0 ? a.sinks : 0; p.scale = a.scale;
  p.q = a.q; p.k = a.k_cache; p.v = a.v_cache; p.o = a.o; p.lse = a.lse;
  // with an empty table no entry is ever read; the pointer only has to tell paged from dense
  p.table = a.page_table ? a.page_table : a.cu_q;
  p.cu_q = a.cu_q; p.kv_len = a.kv_len;
  p.num_pages = a.num_pages; p.page = a.page_size; p.table_width = a.table_width;
  p.max_q = std::min(a.max_q, a.N);
  p.splits = forward_splits(p, a.dtype);
  return p;
}

// Whether the blocks that share a row's keys leave partial results to a second kernel.
bool has_parts(const rsm::AttnParams& p, rsm_dtype dtype) {
  return p.splits > 1 && !(rsm::attn_decode_supported(p, dtype) && rsm::attn_decode_joins(p));
}

size_t paged_bytes(const rsm::AttnParams& p, rsm_dtype dtype) {
  if (!has_parts(p, dtype)) return 0;
  const size_t rows = (size_t)p.T * p.H;
  return up256((size_t)p.splits * rows * p.D * sizeof(float)) + up256((size_t)p.splits * rows * sizeof(float));
}

rsm_status check_norm_sizes(int64_t rows, int d, rsm_dtype y_dtype, rsm_dtype dtype, rsm_act act, float scale,
                            float eps) {
  if (rows < 0 || d < 1) return fail(RSM_ERR_INVALID_ARG, "rows must be >= 0 and d >= 1");
  if (!known_dtype(dtype) || !known_dtype(y_dtype)) return fail(RSM_ERR_INVALID_ARG, "unknown dtype");
  if (y_dtype != dtype && y_dtype != RSM_F32) return fail(RSM_ERR_UNSUPPORTED, "y_dtype must be dtype or fp32");
  if (act != RSM_ACT_SILU && act != RSM_ACT_SIGMOID) return fail(RSM_ERR_INVALID_ARG, "unknown act %d", (int)act);
  if (!std::isfinite(scale)) return fail(RSM_ERR_INVALID_ARG, "scale must be finite");
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(RSM_ERR_INVALID_ARG, "eps must be positive and finite");
  if (d > 8192 || d % 4 != 0) return fail(RSM_ERR_UNSUPPORTED, "d must be a multiple of 4 in [4, 8192] (got %d)", d);
  if (rows > 0x7fffffff) return fail(RSM_ERR_UNSUPPORTED, "too many rows");
  return RSM_OK;
}

rsm_status check_norm_backward(const rsm_block_norm_backward_args* a) {
  if (!a) return fail(RSM_ERR_INVALID_ARG, "args must not be NULL");
  rsm_status s = check_norm_sizes(a->rows, a->d, a->y_dtype, a->dtype, a->act, a->scale, a->eps);
  if (s != RSM_OK) return s;
  if (a->rows > 0) {
    NEED_PTR(a->y, "y"); NEED_PTR(a->residual, "residual"); NEED_PTR(a->w_post, "w_post");
  }
  MAY_PTR(a->gate, "gate"); MAY_PTR(a->w_pre, "w_pre"); MAY_PTR(a->dh, "dh"); MAY_PTR(a->dx, "dx");
  if (a->dx && !a->w_pre) return fail(RSM_ERR_INVALID_ARG, "dx needs w_pre");
  if (a->dgate && !a->gate) return fail(RSM_ERR_INVALID_ARG, "dgate needs gate");
  if (a->dw_pre && !a->w_pre) return fail(RSM_ERR_INVALID_ARG, "dw_pre needs w_pre");
  MAY_PTR(a->dy, "dy"); MAY_PTR(a->dgate, "dgate"); MAY_PTR(a->dresidual, "dresidual");
  MAY_PTR(a->dw_post, "dw_post"); MAY_PTR(a->dw_pre, "dw_pre");
  return RSM_OK;
}

}  // namespace

extern "C" {

rsm_status rsm_window_forward(const rsm_window_args* a, void* stream) {
  rsm::report_error(RSM_OK, "");
  if (!a) return fail(RSM_ERR_INVALID_ARG, "args must not be NULL");
  rsm_status s = check_window(a->B, a->T, a->H, a->Hkv, a->D, a->window, a->sinks, a->dtype, a->scale);
  if (s != RSM_OK) return s;
  if ((s = check_rows((int64_t)a->B * a->T * a->H)) != RSM_OK) return s;
  if ((int64_t)a->B * a->T * a->H == 0) return RSM_OK;
  NEED_PTR(a->q, "q"); NEED_PTR(a->k, "k"); NEED_PTR(a->v, "v"); NEED_PTR(a->o, "o");
  MAY_PTR(a->lse, "lse");
  if ((s = check_low(a->o_low, a->dtype)) != RSM_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = a->flags & RSM_FLAG_VALIDATE ? validate_qkv(*a, st) : cudaSuccess;
  if (e == cudaSuccess) {
    rsm::AttnParams p = window_params(*a);
    p.o = a->o;
    p.lse = a->lse;
    p.o_low = a->o_low;
    e = launch_forward(p, a->dtype, st);
  }
  return finish(e, "rsm_window_forward");
}

size_t rsm_window_backward_workspace_size(const rsm_window_backward_args* a) {
  if (check_window_backward(a) != RSM_OK) return (size_t)-1;
  return (int64_t)a->B * a->T * a->H == 0 ? 0 : window_backward_bytes(*a);
}

rsm_status rsm_window_backward(const rsm_window_backward_args* a, void* stream) {
  rsm::report_error(RSM_OK, "");
  rsm_status s = check_window_backward(a);
  if (s != RSM_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if ((int64_t)a->B * a->T * a->H == 0) {  // no query heads: the keys' gradients are empty sums
    const size_t bytes = (size_t)a->B * a->T * a->Hkv * a->D * (a->dtype == RSM_F32 ? 4 : 2);
    if (a->dk && bytes) e = cudaMemsetAsync(a->dk, 0, bytes, st);
    if (a->dv && bytes && e == cudaSuccess) e = cudaMemsetAsync(a->dv, 0, bytes, st);
    return finish(e, "rsm_window_backward (no query heads)");
  }
  if ((s = check_workspace(a->workspace, a->workspace_bytes, window_backward_bytes(*a))) != RSM_OK) return s;
  if (a->flags & RSM_FLAG_VALIDATE) {
    e = validate_qkv(*a, st);
    if (e == cudaSuccess) e = rsm::launch_check_finite(a->dO, (int64_t)a->B * a->T * a->H * a->D, a->dtype, st);
  }
  rsm::AttnParams p = window_params(*a);
  p.o = const_cast<void*>(a->o);
  p.lse = const_cast<float*>(a->lse);
  p.o_low = const_cast<void*>(a->o_low);
  p.dO = a->dO;
  p.dq = a->dq; p.dk = a->dk; p.dv = a->dv;
  if (e == cudaSuccess && rsm::attn_tc_supported(p, a->dtype)) {
    e = rsm::launch_attn_tc_backward(p, a->workspace, st);
  } else if (e == cudaSuccess) {
    p.delta = static_cast<float*>(a->workspace);
    e = rsm::launch_attn_delta(p, a->dtype, st);
    float* parts = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + delta_bytes(*a));
    if (e == cudaSuccess) e = rsm::launch_attn_simt_backward(p, a->dtype, parts, st);
  }
  return finish(e, "rsm_window_backward");
}

rsm_status rsm_paged_append(const rsm_paged_append_args* a, void* stream) {
  rsm::report_error(RSM_OK, "");
  if (!a) return fail(RSM_ERR_INVALID_ARG, "args must not be NULL");
  rsm_status s = check_heads(a->Hkv, a->Hkv, a->D, a->dtype);
  if (s != RSM_OK) return s;
  s = check_cache(a->B, a->N, a->Hkv, a->D, a->num_pages, a->page_size, a->table_width);
  if (s != RSM_OK) return s;
  if ((int64_t)a->N * a->Hkv == 0 || a->B == 0) return RSM_OK;
  NEED_PTR(a->k, "k"); NEED_PTR(a->v, "v");
  if (a->num_pages > 0) { NEED_PTR(a->k_cache, "k_cache"); NEED_PTR(a->v_cache, "v_cache"); }
  if (a->table_width > 0) NEED_PTR(a->page_table, "page_table");
  NEED_PTR(a->cu_q, "cu_q"); NEED_PTR(a->kv_len, "kv_len");
  return finish(rsm::launch_paged_append(*a, static_cast<cudaStream_t>(stream)), "rsm_paged_append");
}

size_t rsm_paged_workspace_size(const rsm_paged_args* a) {
  if (check_paged(a) != RSM_OK) return (size_t)-1;
  if ((int64_t)a->N * a->H == 0 || a->B == 0 || a->max_q == 0) return 0;
  return paged_bytes(paged_params(*a), a->dtype);
}

rsm_status rsm_paged_forward(const rsm_paged_args* a, void* stream) {
  rsm::report_error(RSM_OK, "");
  rsm_status s = check_paged(a);
  if (s != RSM_OK) return s;
  if ((int64_t)a->N * a->H == 0 || a->B == 0 || a->max_q == 0) return RSM_OK;
  rsm::AttnParams p = paged_params(*a);
  if ((s = check_workspace(a->workspace, a->workspace_bytes, paged_bytes(p, a->dtype))) != RSM_OK) return s;
  const bool parts = has_parts(p, a->dtype);
  if (parts) {
    p.part_o = static_cast<float*>(a->workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<char*>(a->workspace) +
                                          up256((size_t)p.splits * p.T * p.H * p.D * sizeof(float)));
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = a->flags & RSM_FLAG_VALIDATE
                      ? rsm::launch_check_finite(a->q, (int64_t)a->N * a->H * a->D, a->dtype, st)
                      : cudaSuccess;
  if (e == cudaSuccess) e = launch_forward(p, a->dtype, st);
  if (e == cudaSuccess && parts) e = rsm::launch_attn_combine(p, a->dtype, st);
  return finish(e, "rsm_paged_forward");
}

rsm_status rsm_block_norm_forward(const rsm_block_norm_args* a, void* stream) {
  rsm::report_error(RSM_OK, "");
  if (!a) return fail(RSM_ERR_INVALID_ARG, "args must not be NULL");
  rsm_status s = check_norm_sizes(a->rows, a->d, a->y_dtype, a->dtype, a->act, a->scale, a->eps);
  if (s != RSM_OK) return s;
  if (a->rows == 0) return RSM_OK;
  NEED_PTR(a->y, "y"); NEED_PTR(a->residual, "residual"); NEED_PTR(a->w_post, "w_post"); NEED_PTR(a->h, "h");
  MAY_PTR(a->gate, "gate"); MAY_PTR(a->w_pre, "w_pre"); MAY_PTR(a->x, "x");
  if (!a->x != !a->w_pre) return fail(RSM_ERR_INVALID_ARG, "x and w_pre go together");
  return finish(rsm::launch_block_norm(*a, static_cast<cudaStream_t>(stream)), "rsm_block_norm_forward");
}

size_t rsm_block_norm_backward_workspace_size(const rsm_block_norm_backward_args* a) {
  if (check_norm_backward(a) != RSM_OK) return (size_t)-1;
  return a->rows == 0 ? 0 : rsm::block_norm_backward_workspace_bytes(*a);
}

rsm_status rsm_block_norm_backward(const rsm_block_norm_backward_args* a, void* stream) {
  rsm::report_error(RSM_OK, "");
  rsm_status s = check_norm_backward(a);
  if (s != RSM_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) {  // no rows: the weights' gradients are empty sums
    cudaError_t e = a->dw_post ? cudaMemsetAsync(a->dw_post, 0, (size_t)a->d * 4, st) : cudaSuccess;
    if (e == cudaSuccess && a->dw_pre) e = cudaMemsetAsync(a->dw_pre, 0, (size_t)a->d * 4, st);
    return finish(e, "rsm_block_norm_backward (no rows)");
  }
  s = check_workspace(a->workspace, a->workspace_bytes, rsm::block_norm_backward_workspace_bytes(*a));
  if (s != RSM_OK) return s;
  return finish(rsm::launch_block_norm_backward(*a, st), "rsm_block_norm_backward");
}

}  // extern "C"
