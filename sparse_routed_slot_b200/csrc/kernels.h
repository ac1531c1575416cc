// kernels.h -- launch functions of the librsm kernels (internal; the public ABI is rsm.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rsm.h"

namespace rsm {

cudaError_t launch_route(const float* logits, int64_t rows, int M, int K, int32_t* idx_out,
                         float* score_out, int router, int validate, cudaStream_t stream);

// Routing records for the tensor prefill (route_rec.cu, M = 128, K <= 32) over rows given as
// [B, T, H]: route_record_bytes(K) bytes per row, rows in [B, H, T] order; also the ranked
// indices and scores in the input row order when idx_out / score_out are not null.
bool route_records_supported(int M, int K);
int route_record_bytes(int K);
cudaError_t launch_route_records(const float* logits, const float* f, const void* k, int64_t B, int64_t T,
                                 int64_t H, int M, int K, int decay_slot, int router, int validate,
                                 unsigned char* rec, int32_t* idx_out, float* score_out, int32_t* counts,
                                 cudaStream_t stream);

// Adds the per-slot selection counts of routing records ([pairs, T] rows) to counts[pairs][128].
cudaError_t launch_record_counts(const unsigned char* rec, int64_t pairs, int64_t T, int K, int32_t* counts,
                                 cudaStream_t stream);

cudaError_t launch_decode(const rsm_decode_args& a, cudaStream_t stream);

// Gradients on CUDA cores (backward.cu).
size_t backward_smem_bytes(int M, int K, int Dv);
size_t backward_workspace_bytes(const rsm_backward_args& a);
cudaError_t launch_backward(const rsm_backward_args& a, cudaStream_t stream);

// CUDA-core fp32 chunked prefill (any supported size).
cudaError_t launch_prefill_simt(const rsm_forward_args& a, cudaStream_t stream);
size_t prefill_simt_smem_bytes(int M, int Dv);

// tcgen05 tensor-core chunked prefill. `supported` tells whether the shape/dtype can run there.
bool prefill_tc_supported(const rsm_forward_args& a);
size_t prefill_tc_workspace_bytes(const rsm_forward_args& a);
int prefill_tc_launches(const rsm_forward_args& a);  // kernel launches of one call
cudaError_t launch_prefill_tc(const rsm_forward_args& a, cudaStream_t stream);

// Attention (window and paged). One parameter block serves every attention kernel: `table` is null
// for dense [B,T,...] tensors (T = tokens of a sequence) and set for a paged cache (T = N, all new
// tokens; k and v are the caches).
struct AttnParams {
  int B, T, H, Hkv, G, D;
  int window, sinks;  // window <= 0: no limit
  float scale;
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  void* o_low;        // what rounding left of o, or null
  const int32_t* table;
  const int32_t* cu_q;
  const int32_t* kv_len;
  int num_pages, page, table_width;
  int max_q;
  int splits;         // blocks that share a row's keys; > 1: partial results below
  float* part_o;      // [splits][rows][D], normalised
  float* part_lse;    // [splits][rows]
  // backward
  const void* dO;
  void* dq;
  void* dk;
  void* dv;
  float* delta;       // [rows]: dO . o
};

// CUDA-core kernels in fp32 (any dtype, head dimension and page size).
int attn_simt_splits(const AttnParams& p);
cudaError_t launch_attn_simt(const AttnParams& p, rsm_dtype dtype, cudaStream_t stream);
size_t attn_simt_backward_bytes(const AttnParams& p);  // of `part`
cudaError_t launch_attn_simt_backward(const AttnParams& p, rsm_dtype dtype, float* part, cudaStream_t stream);
// Tensor-core forward (attn_tc.cu): bf16, head dimensions to 128, page sizes that fit its tiles.
bool attn_tc_supported(const AttnParams& p, rsm_dtype dtype);
int attn_tc_splits(const AttnParams& p);
cudaError_t launch_attn_tc(const AttnParams& p, cudaStream_t stream);
// Few query rows per key/value head (attn_decode.cu): bf16, paged, single tokens above all.
bool attn_decode_supported(const AttnParams& p, rsm_dtype dtype);
int attn_decode_splits(const AttnParams& p);
// Whether p.splits blocks join in the kernel (no partial results, no second kernel).
bool attn_decode_joins(const AttnParams& p);
cudaError_t launch_attn_decode(const AttnParams& p, cudaStream_t stream);
// Its gradients (attn_tc_backward.cu), dense only; the workspace holds attn_tc_backward_bytes(p) bytes.
size_t attn_tc_backward_bytes(const AttnParams& p);
cudaError_t launch_attn_tc_backward(const AttnParams& p, void* workspace, cudaStream_t stream);
// delta = dO . o for every row (the first step of the fp32 backward).
cudaError_t launch_attn_delta(const AttnParams& p, rsm_dtype dtype, cudaStream_t stream);
// Joins the partial results of p.splits blocks into o and lse.
cudaError_t launch_attn_combine(const AttnParams& p, rsm_dtype dtype, cudaStream_t stream);
cudaError_t launch_paged_append(const rsm_paged_append_args& a, cudaStream_t stream);
// Raises RSM_ERR_NONFINITE when one of n values is not finite.
cudaError_t launch_check_finite(const void* x, int64_t n, rsm_dtype dtype, cudaStream_t stream);

// Norms around a block (block_norm.cu).
cudaError_t launch_block_norm(const rsm_block_norm_args& a, cudaStream_t stream);
size_t block_norm_backward_workspace_bytes(const rsm_block_norm_backward_args& a);
cudaError_t launch_block_norm_backward(const rsm_block_norm_backward_args& a, cudaStream_t stream);

// Profiling events of the calling host thread (rsm_forward_set_profile_events): when set, launch
// functions record event i after their i-th kernel (event 0 before the first).
struct ProfileEvents {
  void* const* events = nullptr;
  int n = 0;
  int next = 0;
};
ProfileEvents& profile_events();
// Records the next profiling event on `stream` (no-op when none are set).
cudaError_t profile_mark(cudaStream_t stream);

// Sets the message rsm_last_error() returns on this host thread; returns `s`.
rsm_status report_error(rsm_status s, const char* msg);

}  // namespace rsm
