/*
 * rsm.h -- C ABI of librsm, a B200 (sm_100a) implementation of the routing-state-model (RSM)
 * sequence mixer of Raven ("Raven: High-Recall Sequence Modeling with Sparse Memory Routing").
 *
 * The mixer, per batch b, head h and token t (Raven README, github.com/xiaol/SelectingMemory,
 * "How Raven Works"):
 *   S_t      = the K of M slots with the largest router logits (ties: lower slot index first)
 *   s_i      = sigmoid(logit_i)                         for i in S_t, 0 otherwise
 *   a_i      = exp(s_i * f)                             f = per-head or per-slot log-decay, f <= 0
 *   H[i,:]   = a_i * H[i,:] + (1 - a_i) * k_i * v       for i in S_t; other rows keep their bits
 *   o_t      = sum_i q_i * H[i,:]                       (read after the write)
 * with a state H of M slot rows by Dv columns per (b,h). "Model Structure" of the same README
 * names the two decay families (Mamba2: one log-decay per head and token; GLA: one per slot) and
 * the two kernels (chunked for training/prefill, fused recurrent for generation).
 *
 * Conventions for every entry point:
 *   - The caller owns all memory. Pointers are DEVICE pointers unless stated otherwise, 16-byte
 *     aligned, row-major and contiguous in the layouts given below. The library never allocates.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream). Work is
 *     enqueued asynchronously; argument errors are returned synchronously before any launch,
 *     and a failed launch returns RSM_ERR_CUDA. rsm_last_error() describes the last failure of
 *     the calling host thread.
 *   - Logits and f must be finite and f <= 0 (a very negative finite f stands for "forget").
 *     These are preconditions; they are checked only when RSM_FLAG_VALIDATE is set.
 *   - Slots not selected at a step (decode) or in the whole call (prefill) are left bit-identical
 *     in the state.
 *   - Supported sizes: 32 <= M <= 256 with M a power of two, 1 <= K <= M, 1 <= Dv <= 256 with
 *     Dv % 4 == 0. Other sizes return RSM_ERR_UNSUPPORTED.
 *
 * Beside the mixer stand the other operators of a hybrid stack, in which attention layers alternate
 * with mixer layers (Raven README "Model Structure": optional standard attention layers at specified
 * indices; paperlayer.ai summary section A.6: full or sliding-window attention interleaved,
 * norms, output gating and skip connections around every block): rsm_window_* (prompts and training),
 * rsm_paged_* (serving) and rsm_block_norm_*.
 */
#ifndef RSM_H_
#define RSM_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define RSM_API __attribute__((visibility("default")))
#else
#define RSM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rsm_status {
  RSM_OK = 0,
  RSM_ERR_INVALID_ARG = 1,  /* null pointer where one is required, bad size, misalignment */
  RSM_ERR_UNSUPPORTED = 2,  /* valid arguments outside the sizes this build implements */
  RSM_ERR_CUDA = 3,         /* a CUDA call or launch failed; see rsm_last_error() */
  RSM_ERR_NONFINITE = 4,    /* RSM_FLAG_VALIDATE found a non-finite input, or f > 0 */
  RSM_ERR_WORKSPACE = 5,    /* workspace missing or smaller than the call's ..._workspace_size() */
  RSM_ERR_TIMEOUT = 6,      /* a bounded device wait gave up (reported by rsm_get_device_status) */
  RSM_ERR_BAD_PAGE = 7      /* a page table or length outside the cache (reported by rsm_get_device_status) */
} rsm_status;

typedef enum rsm_dtype { RSM_F32 = 0, RSM_BF16 = 1 } rsm_dtype;

typedef enum rsm_decay {
  RSM_DECAY_HEAD = 0,  /* f has one value per (b,t,h): Mamba2-style scalar log-decay            */
  RSM_DECAY_SLOT = 1   /* f has one value per (b,t,h,slot): GLA-style per-slot log-decay         */
} rsm_decay;

typedef enum rsm_path {
  RSM_PATH_AUTO = 0,    /* tensor-core path when the shape allows it, else the CUDA-core path    */
  RSM_PATH_SIMT = 1,    /* CUDA-core fp32 chunked path (any supported size, any input dtype)     */
  RSM_PATH_TENSOR = 2   /* tcgen05/TMEM tensor-core path; RSM_ERR_UNSUPPORTED when not available */
} rsm_path;

/* Router score of a selected slot (the selected set is the same for every variant: both scores
 * are monotone in the logit). Raven README "Model Structure" (top-k sigmoid/softmax router) and
 * "Usage" (router_score 'sigmoid' or 'softmax'); paperlayer.ai summary section 6.2.1 (sigmoid vs
 * softmax scores) and section 4.1 (the selected weights are normalised to sum to one). */
typedef enum rsm_router {
  RSM_ROUTER_SIGMOID = 0,       /* s_i = sigmoid(l_i) (default; the README pseudocode)                 */
  RSM_ROUTER_SOFTMAX = 1,       /* s_i = e^{l_i} / sum over all M slots of e^{l_j}                    */
  RSM_ROUTER_SIGMOID_NORM = 2,  /* sigmoid scores divided by their sum over the K selected slots      */
  RSM_ROUTER_SOFTMAX_NORM = 3   /* softmax scores divided by their sum over the K selected slots      */
} rsm_router;

enum {
  /* Device-side check of the preconditions: a non-finite logit, a non-finite or positive f, or (in the
   * attention calls) a non-finite q, k, v or dO is
   * reported as RSM_ERR_NONFINITE by rsm_get_device_status (results are then undefined). */
  RSM_FLAG_VALIDATE = 1,
  /* Testing aid for the bounded-wait error paths (no counterpart on the pages; never set in normal
   * use): in rsm_decode_step the routing warps hand over no routing slot and the warps waiting for
   * one give up after a short bound, so every CTA takes its timeout exit, the call writes neither o
   * nor the state, and rsm_get_device_status reports RSM_ERR_TIMEOUT. In rsm_backward the first token's
   * copy is withheld and the sweeps' waits get a bound of one poll, so the first wait expires with
   * the next tokens' copies in flight: the kernel stops, drains those copies (with the normal
   * bound) and reports RSM_ERR_TIMEOUT; the gradients are then undefined. Other calls ignore it. */
  RSM_FLAG_TEST_STALL_ROUTING = 256
};

/* ---------------------------------------------------------------------------------------------
 * rsm_route -- TopK routing of router logits.
 *   Raven README "How Raven Works" (route_scores = TopK(sigmoid(r_proj(x)))); paperlayer.ai summary
 *   section 4.1 (keep the top-K scores, set the rest to zero). Ranking is on the fp32 logits
 *   (sigmoid is monotone and saturates in fp32); exact ties go to the lower slot index, and
 *   -0.0 ties +0.0.
 *   logits    [rows, M] fp32 (device)
 *   idx_out   [rows, K] int32 (device): selected slots in rank order (logit desc, index asc)
 *   score_out [rows, K] fp32 (device, may be NULL): sigmoid(logit) of each selected slot
 *   rows may be 0 (nothing is launched).
 * ------------------------------------------------------------------------------------------- */
RSM_API rsm_status rsm_route(const float* logits, int64_t rows, int M, int K, int32_t* idx_out,
                     float* score_out, void* stream);

/* rsm_route with a router variant (score_out holds that variant's scores) and RSM_FLAG_* flags
 * (RSM_FLAG_VALIDATE reports non-finite logits through rsm_get_device_status). */
RSM_API rsm_status rsm_route_ex(const float* logits, int64_t rows, int M, int K, rsm_router router,
                                int flags, int32_t* idx_out, float* score_out, void* stream);

/* ---------------------------------------------------------------------------------------------
 * rsm_forward -- chunked prefill over T tokens.
 *   The recurrence above, evaluated chunk by chunk (paperlayer.ai summary, section A.5: the
 *   sequence is split into n chunks of length C, T = n*C, for stability and parallelism; a
 *   ragged last chunk is allowed here). The result does not depend on the chunk length beyond
 *   rounding.
 *   q, k    [B,T,H,M] in qkv_dtype (fp32 or bf16)
 *   v       [B,T,H,Dv] in qkv_dtype
 *   logits  [B,T,H,M] fp32
 *   f       [B,T,H] fp32 (RSM_DECAY_HEAD) or [B,T,H,M] fp32 (RSM_DECAY_SLOT)
 *   H0      [B,H,M,Dv] fp32 initial state, or NULL for zeros. May alias HT.
 *   o       [B,T,H,Dv] fp32 output (required)
 *   HT      [B,H,M,Dv] fp32 final state, or NULL to skip
 *   idx_out, score_out  [B,T,H,K] (int32, fp32), or NULL to skip: the routing of every token
 *   workspace / workspace_bytes: device scratch of at least rsm_forward_workspace_size(args)
 *     bytes (256-byte aligned); may be NULL when that size is 0. Its contents are not preserved.
 *   path: which implementation to run (RSM_PATH_AUTO normally).
 * ------------------------------------------------------------------------------------------- */
typedef struct rsm_forward_args {
  int B, T, H, M, K, Dv;
  rsm_dtype qkv_dtype;
  rsm_decay decay;
  const void* q;
  const void* k;
  const void* v;
  const float* logits;
  const float* f;
  const float* H0;
  float* o;
  float* HT;
  int32_t* idx_out;
  float* score_out;
  void* workspace;
  size_t workspace_bytes;
  rsm_path path;
  int flags; /* RSM_FLAG_* */
  rsm_router router;     /* score of the selected slots (RSM_ROUTER_SIGMOID = 0 by default)        */
  int32_t* slot_counts;  /* [B,H,M] int32 or NULL: the number of tokens of the call that selected
                            each slot is ADDED to it (the per-slot counts behind the paper's
                            "effective sequence length" analysis, paperlayer.ai summary 7.1) */
} rsm_forward_args;

/* Bytes of device workspace rsm_forward needs for these arguments (0 when none). Depends only on
 * the sizes, dtype, decay and path fields. Returns (size_t)-1 for arguments rsm_forward rejects. */
RSM_API size_t rsm_forward_workspace_size(const rsm_forward_args* args);
RSM_API rsm_status rsm_forward(const rsm_forward_args* args, void* stream);

/* The implementation rsm_forward would run for these arguments: RSM_PATH_SIMT or RSM_PATH_TENSOR
 * (RSM_PATH_AUTO resolved), or -1 for arguments rsm_forward rejects. Host-only. */
RSM_API int rsm_forward_selected_path(const rsm_forward_args* args);

/* Number of kernel launches one rsm_forward call makes for these arguments (for accounting and
 * profiling: tensor path = routing records + [segment summary + segment scan +] chunk scan; SIMT
 * path = 1; 0 when B*H == 0 or T == 0), or -1 for arguments rsm_forward rejects. Host-only. */
RSM_API int rsm_forward_kernel_launches(const rsm_forward_args* args);

/* Profiling aid (no counterpart on the pages): while set, every rsm_forward call made on the
 * calling host thread records `events[0]` on its stream before its first kernel and `events[i]`
 * after its i-th kernel (i = 1 .. rsm_forward_kernel_launches(args)), so that the caller can time
 * each kernel with cudaEventElapsedTime. `events` are cudaEvent_t handles passed as void*, owned
 * by the caller; `n_events` must be at least the launches of the calls that follow plus one (a
 * call that needs more returns RSM_ERR_INVALID_ARG before any launch). NULL / 0 stops recording.
 * The events are only recorded, never waited on or destroyed, by the library. Host-only. */
RSM_API rsm_status rsm_forward_set_profile_events(void* const* events, int n_events);

/* ---------------------------------------------------------------------------------------------
 * rsm_forward_noalloc -- rsm_forward for callers that cannot allocate device memory.
 *   The pages have no counterpart to this call; it exists for callers with no way to allocate:
 *   work recorded into a CUDA graph capture (an allocation would break the capture), programs
 *   whose allocator owns every byte of the device, or runtimes with a fixed memory plan. Where
 *   rsm_forward needs a caller-supplied workspace (the tensor-core path: routing records of every
 *   token, 144 bytes per token and head for K <= 16 and 288 for K <= 32, plus the segment states
 *   when a long sequence is split), this call uses a scratch array built into the library instead;
 *   the caller passes only the inputs and outputs (args->workspace and args->workspace_bytes are
 *   ignored). Results are bit-identical to those of rsm_forward.
 *   Limit: the scratch holds rsm_forward_noalloc_max_scratch() bytes (16 MiB), about 116,000
 *   token-heads (B*T*H) at K <= 16 before segment states; sizes whose workspace would exceed it
 *   return RSM_ERR_WORKSPACE with the sizes in rsm_last_error(), before anything is launched.
 *   The array occupies device memory on every GPU that loads the library, until exit. The first
 *   call on each device (and the first after a device reset) looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call before any stream
 *   capture. All calls share the array and it keeps the last call's contents (nothing in it needs
 *   to start at zero): calls whose GPU work overlaps in time, on any streams or host threads of
 *   one device, race and must not be issued. No CUDA allocation routine is called.
 * ------------------------------------------------------------------------------------------- */
RSM_API rsm_status rsm_forward_noalloc(const rsm_forward_args* args, void* stream);
RSM_API size_t rsm_forward_noalloc_max_scratch(void);

/* ---------------------------------------------------------------------------------------------
 * rsm_decode_step -- one generation token per (b,h): fused routing, sparse decay/write of the K
 *   selected rows of the carried state in place, and the read o = q.H over all M rows.
 *   Raven README "Model Structure" (fused recurrent computation for inference).
 *   q, k    [B,H,M] in qkv_dtype;  v [B,H,Dv] in qkv_dtype
 *   logits  [B,H,M] fp32;          f [B,H] or [B,H,M] fp32
 *   state   [B,H,M,Dv] fp32, read and updated in place (only the K selected rows are written)
 *   o       [B,H,Dv] fp32 output
 *   idx_out, score_out [B,H,K] or NULL
 * ------------------------------------------------------------------------------------------- */
typedef struct rsm_decode_args {
  int B, H, M, K, Dv;
  rsm_dtype qkv_dtype;
  rsm_decay decay;
  const void* q;
  const void* k;
  const void* v;
  const float* logits;
  const float* f;
  float* state;
  float* o;
  int32_t* idx_out;
  float* score_out;
  int flags; /* RSM_FLAG_* */
  rsm_router router;     /* score of the selected slots (RSM_ROUTER_SIGMOID = 0 by default)        */
  int32_t* slot_counts;  /* [B,H,M] int32 or NULL: 1 is added for every slot selected at the step */
} rsm_decode_args;

RSM_API rsm_status rsm_decode_step(const rsm_decode_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * rsm_backward -- gradients of the prefill (training). Reverse-mode differentiation of the
 *   recurrence above with the sigmoid router: given dO = dL/do and dHT = dL/dH_T, it returns
 *   dL/dq, dL/dk, dL/dv, dL/dlogits, dL/df and dL/dH0. The TopK cut is piecewise constant in the
 *   logits, so unselected slots get no key or logit gradient. Raven README "Model Structure"
 *   (chunked computation for training) and the fork's reverse-scan backward.
 *   Inputs as rsm_forward (q, k, v in qkv_dtype; logits, f, H0 fp32; H0 may be NULL = zeros)
 *   dO    [B,T,H,Dv] fp32, or NULL for zero
 *   dHT   [B,H,M,Dv] fp32, or NULL for zero
 *   dq, dk, dlogits [B,T,H,M] fp32; dv [B,T,H,Dv] fp32; df [B,T,H] or [B,T,H,M] fp32;
 *   dH0 [B,H,M,Dv] fp32 (each output may be NULL to skip it)
 *   workspace: at least rsm_backward_workspace_size(args) bytes (256-byte aligned): the routing
 *     of every token, its K entries (slot, decay, write weight, score, rate, key; 32 bytes each)
 *     and a tape of the K state rows each token overwrites (T*K*Dv*4 bytes per (b,h) stream).
 *   Supported: the sizes of rsm_forward with M*Dv <= 24576 (the state and its gradient stay in
 *   shared memory), router RSM_ROUTER_SIGMOID. The arithmetic is fp32 on CUDA cores.
 * ------------------------------------------------------------------------------------------- */
typedef struct rsm_backward_args {
  int B, T, H, M, K, Dv;
  rsm_dtype qkv_dtype;
  rsm_decay decay;
  const void* q;
  const void* k;
  const void* v;
  const float* logits;
  const float* f;
  const float* H0;
  const float* dO;
  const float* dHT;
  float* dq;
  float* dk;
  float* dv;
  float* dlogits;
  float* df;
  float* dH0;
  void* workspace;
  size_t workspace_bytes;
  rsm_router router;
  int flags; /* RSM_FLAG_* */
} rsm_backward_args;

/* Bytes of workspace rsm_backward needs, or (size_t)-1 for arguments it rejects. Host-only. */
RSM_API size_t rsm_backward_workspace_size(const rsm_backward_args* args);
RSM_API rsm_status rsm_backward(const rsm_backward_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * rsm_window_forward -- causal attention over a sliding window whose first tokens stay visible.
 *   Query i sees key j when j <= i and (i - j < window or j < sinks); a window of at least T is
 *   plain causal attention. With G = H / Hkv, query head h reads key/value head h / G.
 *     s_ij = scale q_i.k_j over the keys seen, lse_i = log sum_j e^{s_ij},
 *     o_i = sum_j e^{s_ij - lse_i} v_j
 *   q       [B,T,H,D] in dtype;  k, v [B,T,Hkv,D] in dtype
 *   o       [B,T,H,D] in dtype (required)
 *   lse     [B,T,H] fp32, or NULL to skip: natural logarithm of the row's sum (the backward reads it)
 *   o_low   [B,T,H,D] bf16, or NULL to skip (bf16 inputs only): what rounding left of o, that is the
 *           unrounded result minus o, for the backward
 *   Scores, softmax statistics and sums are fp32. With bf16 inputs the softmax weights are rounded
 *   to bf16 for the product with v; with fp32 inputs everything is fp32.
 *   q, k and v must be finite (checked when RSM_FLAG_VALIDATE is set): a weight of zero does not
 *   hide an infinity in v.
 *   Supported: 8 <= D <= 256 with D % 8 == 0, Hkv dividing H with H / Hkv <= 64, window >= 1,
 *   sinks >= 0, scale > 0 and finite, T*H < 2^31. B, T or H may be 0 (nothing is launched). Outputs
 *   must not alias inputs or one another.
 *   bf16 with D <= 128 runs on the tensor cores; a larger D, and fp32, on CUDA cores in fp32, at about a
 *   seventeenth of that rate (8 x 2048 tokens, window 512: 4 heads of 256 take 1493 us, 8 of 128 take 88).
 * ------------------------------------------------------------------------------------------- */
typedef struct rsm_window_args {
  int B, T, H, Hkv, D;
  int window, sinks;
  rsm_dtype dtype;
  float scale;
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  void* o_low;
  int flags; /* RSM_FLAG_* */
} rsm_window_args;

RSM_API rsm_status rsm_window_forward(const rsm_window_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * rsm_window_backward -- gradients of rsm_window_forward. With delta_i = dO_i.o_i,
 * p_ij = e^{s_ij - lse_i} and ds_ij = p_ij (dO_i.v_j - delta_i):
 *   dq_i = scale sum_j ds_ij k_j;  dk_j = scale sum_i ds_ij q_i;  dv_j = sum_i p_ij dO_i
 * the sums of dk and dv running over the query heads that share the key/value head, too.
 *   q, k, v, o, lse, o_low: the forward's inputs and outputs;  dO [B,T,H,D] in dtype. o_low may be NULL:
 *     delta is then formed with the rounded o, which rows of few keys show in dq and dk (windows of 3 to
 *     9 keys: off by about 3.6e-3 of their norm instead of 2.6e-3, what rounding ds and the results costs).
 *   dq [B,T,H,D], dk, dv [B,T,Hkv,D] in dtype (each may be NULL to skip it)
 *   workspace: at least rsm_window_backward_workspace_size(args) bytes (256-byte aligned); its
 *     contents are not preserved.
 *   The gradients are the same, bit for bit, from call to call: no sum is left to the order in
 *   which blocks finish. Sizes as rsm_window_forward; with H = 0, dk and dv are zeros. Outputs must
 *   not alias inputs or one another.
 * ------------------------------------------------------------------------------------------- */
typedef struct rsm_window_backward_args {
  int B, T, H, Hkv, D;
  int window, sinks;
  rsm_dtype dtype;
  float scale;
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const float* lse;
  const void* o_low;
  const void* dO;
  void* dq;
  void* dk;
  void* dv;
  void* workspace;
  size_t workspace_bytes;
  int flags; /* RSM_FLAG_* */
} rsm_window_backward_args;

/* Bytes of workspace rsm_window_backward needs, or (size_t)-1 for arguments it rejects. Host-only. */
RSM_API size_t rsm_window_backward_workspace_size(const rsm_window_backward_args* args);
RSM_API rsm_status rsm_window_backward(const rsm_window_backward_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * The paged cache. Keys and values of place p of sequence b stand in page
 * page_table[b][p / page_size], row p % page_size. Sequence b brings n_b = cu_q[b+1] - cu_q[b] new
 * tokens, which are rows cu_q[b] .. cu_q[b+1]-1 of q, k and v and stand at places
 * kv_len[b] - n_b .. kv_len[b] - 1: kv_len counts the new tokens. n_b may be 0.
 *   k_cache, v_cache  [num_pages, page_size, Hkv, D] in dtype
 *   page_table        [B, table_width] int32
 *   cu_q              [B + 1] int32, starting at 0 and not falling;  kv_len [B] int32
 * These three are read on the device and never trusted with an address: an offset outside [0, N] is
 * clamped; a page outside the cache and places past the table's end are left out (not written, not
 * seen) and reported as RSM_ERR_BAD_PAGE by rsm_get_device_status. Pages of which no place is written
 * (or, in rsm_paged_forward, seen) are not looked up: behind a window their entries may be anything. Places
 * below zero are not written, and a new token at one sees nothing. Rows of o (and lse) behind cu_q[B] keep
 * their bits.
 *
 * rsm_paged_append -- writes the new tokens' k and v [N,Hkv,D] to their places. Two tokens must
 * not share a place (a page in two sequences' tables is fine while neither writes to it).
 * ------------------------------------------------------------------------------------------- */
typedef struct rsm_paged_append_args {
  int B, N, Hkv, D;
  int num_pages, page_size, table_width;
  rsm_dtype dtype;
  const void* k;
  const void* v;
  void* k_cache;
  void* v_cache;
  const int32_t* page_table;
  const int32_t* cu_q;
  const int32_t* kv_len;
  int flags; /* RSM_FLAG_* (none applies) */
} rsm_paged_append_args;

RSM_API rsm_status rsm_paged_append(const rsm_paged_append_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * rsm_paged_forward -- attention of the new tokens over the cache, which already holds their own
 * keys and values (rsm_paged_append on the same stream). The token at place p sees places j <= p,
 * and with window > 0 of those only p - j < window or j < sinks (window = 0: no limit, sinks unused).
 *   q    [N,H,D] in dtype;  o [N,H,D] in dtype;  lse [N,H] fp32 or NULL
 *   max_q  no sequence has more new tokens than this (tokens past it are not computed: their rows
 *          keep their bits). With max_q = 1 this is the single-token generation step.
 *   A row that sees nothing gets o = 0 and lse = -infinity. What the cache holds at places that no
 *   computed token of the sequence sees (behind kv_len[b], or hidden by the window) does not matter (it
 *   may be NaN); what it holds at the others must be finite.
 *   workspace: at least rsm_paged_workspace_size(args) bytes (256-byte aligned; may be NULL when
 *     that is 0): partial results of long caches that several blocks share.
 *   Sizes as rsm_window_forward; page_size >= 1, N*H and max_q*H < 2^31, table_width*page_size <=
 *   2^31 - 256.
 *   Fast in bf16: any D and page_size while max_q * H / Hkv <= 16; more rows with D <= 128 and a
 *   page_size of 8, 16, 32 or a multiple of 64. Chunks over other pages or heads, and fp32, run on CUDA
 *   cores (4 x 512 tokens over 8192 keys, 16/4 heads of 128: 147 us with pages of 64, 7.7 ms with 24).
 *   Outputs must not alias inputs or one another.
 * ------------------------------------------------------------------------------------------- */
typedef struct rsm_paged_args {
  int B, N, max_q, H, Hkv, D;
  int num_pages, page_size, table_width;
  int window, sinks;
  rsm_dtype dtype;
  float scale;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* page_table;
  const int32_t* cu_q;
  const int32_t* kv_len;
  void* o;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  int flags; /* RSM_FLAG_VALIDATE checks q */
} rsm_paged_args;

/* Bytes of workspace rsm_paged_forward needs (0 when none), or (size_t)-1 for arguments it rejects.
 * Host-only. */
RSM_API size_t rsm_paged_workspace_size(const rsm_paged_args* args);
RSM_API rsm_status rsm_paged_forward(const rsm_paged_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * rsm_block_norm_forward -- the norms around a block, with its output gate and residual scale:
 *   n = y rsqrt(mean(y^2) + eps) w_post         norm of the block's output y
 *   h = residual + scale n act(gate)            gated, scaled and added to the residual stream
 *   x = h rsqrt(mean(h^2) + eps) w_pre          norm before the next block (of h before rounding)
 *   act(g) = g sigmoid(g) (SILU) or sigmoid(g).
 *   y        [rows,d] in y_dtype (fp32, such as the mixer's o, or dtype)
 *   gate     [rows,d] in dtype, or NULL for no gate (act is then ignored)
 *   residual [rows,d] in dtype;  w_post, w_pre [d] fp32 (w_pre NULL: x is not computed)
 *   h, x     [rows,d] in dtype (x NULL exactly when w_pre is). h may alias residual or, with
 *            y_dtype = dtype, y.
 *   Supported: d % 4 == 0, 4 <= d <= 8192, y_dtype = dtype or fp32. rows may be 0.
 * ------------------------------------------------------------------------------------------- */
typedef enum rsm_act { RSM_ACT_SILU = 0, RSM_ACT_SIGMOID = 1 } rsm_act;

typedef struct rsm_block_norm_args {
  int64_t rows;
  int d;
  rsm_dtype y_dtype, dtype;
  rsm_act act;
  float scale, eps;
  const void* y;
  const void* gate;
  const void* residual;
  const float* w_post;
  const float* w_pre;
  void* h;
  void* x;
  int flags; /* RSM_FLAG_* (none applies) */
} rsm_block_norm_args;

RSM_API rsm_status rsm_block_norm_forward(const rsm_block_norm_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * rsm_block_norm_backward -- gradients of rsm_block_norm_forward.
 *   y, gate, residual, w_post, w_pre: the forward's inputs (everything else is recomputed)
 *   dh, dx   [rows,d] in dtype: gradients of h and x (dh NULL = zero; dx NULL = zero, and needs w_pre
 *            otherwise)
 *   dy [rows,d] in y_dtype; dgate (NULL without a gate), dresidual [rows,d] in dtype;
 *   dw_post, dw_pre [d] fp32 (each output may be NULL to skip it). Outputs must not alias inputs.
 *   workspace: at least rsm_block_norm_backward_workspace_size(args) bytes (256-byte aligned): the
 *     blocks' partial sums of dw_post and dw_pre, added up in a fixed order.
 * ------------------------------------------------------------------------------------------- */
typedef struct rsm_block_norm_backward_args {
  int64_t rows;
  int d;
  rsm_dtype y_dtype, dtype;
  rsm_act act;
  float scale, eps;
  const void* y;
  const void* gate;
  const void* residual;
  const float* w_post;
  const float* w_pre;
  const void* dh;
  const void* dx;
  void* dy;
  void* dgate;
  void* dresidual;
  float* dw_post;
  float* dw_pre;
  void* workspace;
  size_t workspace_bytes;
  int flags; /* RSM_FLAG_* (none applies) */
} rsm_block_norm_backward_args;

/* Bytes of workspace rsm_block_norm_backward needs, or (size_t)-1 for arguments it rejects. Host-only. */
RSM_API size_t rsm_block_norm_backward_workspace_size(const rsm_block_norm_backward_args* args);
RSM_API rsm_status rsm_block_norm_backward(const rsm_block_norm_backward_args* args, void* stream);

/* Human-readable name of a status code (static storage). */
RSM_API const char* rsm_status_string(rsm_status status);

/* Detail of the last failure on the calling host thread ("" if none). */
RSM_API const char* rsm_last_error(void);

/* Synchronizes `stream`, then reads and clears the library's device status word for the current
 * device: RSM_OK, RSM_ERR_NONFINITE (validation found bad inputs), RSM_ERR_BAD_PAGE (a paged call met a
 * page or a length outside the cache) or RSM_ERR_TIMEOUT (a bounded device wait expired). Errors of the synchronization itself return RSM_ERR_CUDA. */
RSM_API rsm_status rsm_get_device_status(void* stream);

/* Library version as major*10000 + minor*100 + patch. */
RSM_API int rsm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RSM_H_ */
