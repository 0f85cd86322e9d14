/*
 * gg.h -- C ABI of the GB300 (sm_103a) Mixture-of-Experts grouped GEMM library.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - T = num_tokens, topk = experts per token, R = T * topk routed rows,
 *    E = experts.  A "flat slot" f = t * topk + j names slot j of token t.
 *    An "expert-order row" i lies in [offsets[e], offsets[e+1]) for its expert.
 *  - bf16 tensors are passed as `gg_bf16*` (raw IEEE bfloat16 bits), row-major,
 *    rows contiguous.  Weights W are (E, N, K) with K contiguous.
 *  - Every pointer argument is a DEVICE pointer owned by the caller, unless it
 *    is documented otherwise.  The library allocates no device memory.
 *  - Calls are asynchronous on `stream` (a cudaStream_t passed as void*; NULL
 *    = the legacy default stream).  Inputs must stay valid until the stream
 *    reaches the call.
 *  - Return value: GG_OK (0), or a negative GG_ERR_* code for an error found
 *    synchronously on the host (bad arguments, unsupported shape, launch
 *    failure).  Nothing is launched when an error is returned.
 *  - `status` (optional, may be NULL): a device int32 the kernels set, with an
 *    atomic compare-and-swap from 0, to a GG_DEV_* code when they find bad
 *    input data (an expert id out of range, a row index out of range) or a
 *    bounded wait ran out.  The offending access is skipped, never performed.
 *    The caller zeroes it and reads it after synchronising, or lets
 *    gg_read_status do both (it maps the word to GG_ERR_DEVICE_CHECK or
 *    GG_ERR_TIMEOUT).
 *  - `workspace` (the entry points that take one): caller-owned device
 *    scratch of at least gg_workspace_size() bytes for that call, 16-byte
 *    aligned; no initialisation needed, contents garbage afterwards.  Too
 *    small -> GG_ERR_WORKSPACE with nothing launched.
 *  - Size rules (else GG_ERR_UNSUPPORTED): row widths K and N multiples of 8
 *    (16-byte rows), every tensor pointer 16-byte aligned, E <= GG_MAX_EXPERTS,
 *    topk <= GG_MAX_TOPK, R < 2^31.
 *  - An empty problem (no rows or no output columns) returns GG_OK without a
 *    launch; an empty reduction writes zeros, and then the inputs that have
 *    no elements (the reduced-over operands) may be NULL.
 *
 * Sources cited below (page title, then section):
 *  [U] unslothai--unsloth unsloth/kernels/moe/grouped_gemm/interface.py
 *  [V] vllm third_party/triton_kernels/matmul_ogs.py
 *  [W] VLA/wall_x/fusions/backend.py
 */
#ifndef GG_H
#define GG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t gg_bf16;

/* host-side return codes */
#define GG_OK 0
#define GG_ERR_INVALID_ARG (-1)
#define GG_ERR_UNSUPPORTED (-2)
#define GG_ERR_CUDA (-3)
#define GG_ERR_DEVICE_CHECK (-4) /* from gg_read_status: a kernel found bad input data */
#define GG_ERR_TIMEOUT (-5)      /* from gg_read_status: a bounded wait in a kernel ran out */
#define GG_ERR_WORKSPACE (-6)

/* device status word codes */
#define GG_DEV_OK 0
#define GG_DEV_BAD_EXPERT_ID 1
#define GG_DEV_BAD_ROW_INDEX 2
#define GG_DEV_SIZES_MISMATCH 3
#define GG_DEV_TIMEOUT 4
#define GG_DEV_BAD_ADAPTER_ID 5

#define GG_MAX_EXPERTS 2048
#define GG_MAX_TOPK 64
#define GG_ROUTE_NOALLOC_SCRATCH_BYTES (1u << 20)
/* gg_forward_combine without a workspace (bf16 accumulation) takes topk up to this */
#define GG_COMBINE_BF16_MAX_TOPK 16
/* low-rank adapters: largest rank (a multiple of 8) */
#define GG_LORA_MAX_RANK 256
/* rotary positions: position axes a pair can take its angle from, heads of q and k together */
#define GG_ROPE_MAX_AXES 4
#define GG_ROPE_MAX_HEADS 65536

/* element types of gg_rope, gg_act8_* and the residual stream of gg_block_norm */
#define GG_DTYPE_BF16 0
#define GG_DTYPE_F16 1
#define GG_DTYPE_F32 2

/* 8-bit forms of kept activations */
#define GG_ACT8_INT8 0
#define GG_ACT8_E4M3 1
/* widest row of gg_block_norm */
#define GG_NORM_MAX_K 16384

/* operations for gg_workspace_size */
#define GG_OP_ROUTE 1            /* gg_route_hist_offsets */
#define GG_OP_BACKWARD_DW 2      /* gg_backward_dW with a gathered operand */
#define GG_OP_FORWARD_COMBINE 3  /* gg_forward_combine, fp32 accumulation */
/* flags for gg_workspace_size */
#define GG_PERMUTE_X 1
#define GG_PERMUTE_Y 2

/* Human-readable text for a GG_* return code (static storage). */
const char* gg_status_string(int code);
/* Human-readable text for a GG_DEV_* device status code (static storage). */
const char* gg_device_status_string(int code);
/* Text of the last CUDA error seen by a host call on this thread. */
const char* gg_last_cuda_error(void);

/* Bytes of workspace an entry point needs for this problem (0: it takes none,
 * or needs none for these flags).  Same size arguments as the call (for a
 * call without N or K pass 0); flags: GG_PERMUTE_X | GG_PERMUTE_Y as the
 * call's permute flags.  No counterpart on the pages: the library allocates
 * nothing, so every scratch buffer comes from the caller through this size. */
size_t gg_workspace_size(int op, int64_t T, int topk, int E, int64_t N, int64_t K, int flags);

/* Synchronises `stream`, reads the device status word `status` (device int32)
 * and returns GG_OK when it is GG_DEV_OK, GG_ERR_TIMEOUT for GG_DEV_TIMEOUT,
 * GG_ERR_DEVICE_CHECK for any other device code, GG_ERR_CUDA if the read
 * fails.  *code (host int32, may be NULL) receives the GG_DEV_* code.  The
 * word is left as it is.  No counterpart on the pages. */
int gg_read_status(const int32_t* status, int32_t* code, void* stream);

/* Tile schedule of the grouped-GEMM launches (process-wide; returns the
 * previous mode, or GG_ERR_INVALID_ARG for an unknown one).
 *   GG_SCHEDULE_AUTO (default): 2-CTA launches over experts whose tiles are
 *     long (at least 48 reduction blocks of 64 a tile; dW: a mean expert of
 *     at least 32 blocks) hand tiles out dynamically, from a device counter
 *     in tile order, so the pairs that read one operand tile read it at about
 *     the same time and DRAM sees it once; shorter tiles keep the static
 *     round-robin (pair p takes tiles p, p + P, ...).
 *   GG_SCHEDULE_STATIC, GG_SCHEDULE_DYNAMIC: always that schedule (dynamic
 *     only where the launch supports it; the dual GEMM is always static).
 * Results are identical bit for bit under either schedule: a tile's sums
 * do not depend on which pair computes it.  The dynamic schedule uses one of
 * 1024 device counter pairs per launch, in turn, reset by the launch itself
 * as it ends: more than 1023 dynamic launches in flight at once on one
 * device (streams that run concurrently, or replays of one captured graph
 * running concurrently with themselves) is not supported.  Launches of more
 * than 2^30 tiles keep the static schedule.  No counterpart on the pages. */
#define GG_SCHEDULE_AUTO 0
#define GG_SCHEDULE_STATIC 1
#define GG_SCHEDULE_DYNAMIC 2
int gg_set_gemm_schedule(int mode);

/* Diagnostic: runs, in one CTA, the bounded mbarrier wait that every
 * pipelined kernel of this library uses, on a barrier phase nothing ever
 * completes, with a limit of limit_ns (0 < limit_ns <= 2 s).  The wait gives
 * up, sets *status to GG_DEV_TIMEOUT (if it was 0) and writes *result = 0
 * (1 would mean the phase completed).  status and result are device int32s.
 * Lets a caller check that a stuck wait ends with an error status instead of
 * a hang, leaving the context usable.  No counterpart on the pages. */
int gg_selftest_bounded_wait(int32_t* status, int32_t* result, uint64_t limit_ns, void* stream);

/* Diagnostic: gg_block_norm (bf16 stream, topk > 3 rows a token in token-slot order with
 * weights 1, w_post = w_pre = w, eps 1e-6) and gg_block_norm_bwd (bf16 stream and y, dh = dx,
 * the same w, no vectors' gradients), except that of token `withheld` (< T) the copies of one
 * stage are left out (of a row that two CTAs share, the first half's): the wait for them runs
 * out after 20 ms, the CTAs that have the row leave early and status is GG_DEV_TIMEOUT.
 *  record [CTAs, 3] int32, CTAs <= 2432, those behind the launch's left as they were: whether a
 *  CTA left early; stages that it filled and left without waiting for them (0, or its shared
 *  memory would be written behind it); stages that it filled again before they were full (0).
 * Tokens of other CTAs come out as they would; those of the CTAs that left are as they
 * were from the withheld one on.  No counterpart on the pages. */
int gg_selftest_block_norm_wait(const gg_bf16* h, const gg_bf16* Y, int topk, const float* w, int64_t T,
                                int64_t K, int64_t withheld, gg_bf16* out_h, gg_bf16* out_x,
                                int32_t* record, int32_t* status, void* stream);
int gg_selftest_block_norm_bwd_wait(const gg_bf16* dx, const gg_bf16* h, const gg_bf16* y, const float* w,
                                    int64_t T, int64_t K, int64_t withheld, gg_bf16* out_dh, gg_bf16* dy,
                                    int32_t* record, int32_t* status, void* stream);

/* ------------------------------------------------------------------ route --
 * Routing metadata from the router's choices ([U] grouped_gemm_forward
 * docstring: m_sizes = tokens per expert, gather_indices sliced by
 * cumsum(m_sizes) gives each expert's token slots; [V] RoutingData.expt_hist,
 * GatherIndx / ScatterIndx; [V] ragged-dw comment for the padded layout;
 * [W] permute).
 *
 *  topk_ids       [T, topk] int32 expert id of each slot (must be in [0, E)).
 *  pad_block      > 0: also write padded_offsets; <= 0: padded_offsets unused.
 *  m_sizes        [E]   out: rows per expert.
 *  offsets        [E+1] out: exclusive prefix of m_sizes, offsets[E] = R.
 *  padded_offsets [E+1] out (or NULL): prefix of ceil(m_e/pad_block)*pad_block.
 *  gather_idx     [R]   out: flat slot f held by expert-order row i; within an
 *                       expert, slots ascend (stable order).
 *  row_id_map     [R]   out (or NULL): inverse, row_id_map[gather_idx[i]] = i.
 *  workspace      device scratch of at least gg_route_workspace_size() bytes,
 *                 owned by the caller; contents need no initialisation and are
 *                 garbage afterwards.  Too small -> GG_ERR_WORKSPACE.
 * An id outside [0, E) sets GG_DEV_BAD_EXPERT_ID; that slot is not counted and
 * gets no row (the outputs are then incomplete). */
size_t gg_route_workspace_size(int64_t T, int topk, int E);
int gg_route_hist_offsets(const int32_t* topk_ids, int64_t T, int topk, int E, int pad_block,
                          int32_t* m_sizes, int32_t* offsets, int32_t* padded_offsets,
                          int32_t* gather_idx, int32_t* row_id_map, void* workspace,
                          size_t workspace_bytes, int32_t* status, void* stream);

/* ------------------------------------------------ route, allocation-free --
 * No counterpart on the pages.  Same outputs as gg_route_hist_offsets, for
 * callers that cannot allocate device memory or pass a workspace: a runtime
 * that owns all device memory in its own arena and hands this code only its
 * input and output buffers, or a latency-critical path that must not pay for
 * an allocation.  There is no workspace argument: the counting sort's scratch
 * is a static device array of GG_ROUTE_NOALLOC_SCRATCH_BYTES (1 MiB) that
 * every GPU loading the library holds until the process exits.
 *  - The first call on each device looks up that array's device address
 *    (once per device, with that device current); make that first call
 *    before any stream capture.
 *  - Each device holds its own copy of the array, shared by every call on
 *    that device: calls that overlap on the same device (concurrent streams)
 *    race on it, so the caller must serialise them; calls on different
 *    devices do not interfere.  No state carries over between calls.
 *  - A problem whose scratch, ceil(T*topk/256) * E * 4 bytes, exceeds the
 *    array returns GG_ERR_WORKSPACE without launching.  A device numbered 64
 *    or higher returns GG_ERR_UNSUPPORTED.
 * Allocates nothing. */
int gg_route_hist_offsets_noalloc(const int32_t* topk_ids, int64_t T, int topk, int E,
                                  int pad_block, int32_t* m_sizes, int32_t* offsets,
                                  int32_t* padded_offsets, int32_t* gather_idx,
                                  int32_t* row_id_map, int32_t* status, void* stream);

/* ---------------------------------------------------------------- permute --
 * Token rows into expert order ([W] permute; [U] permute_x): for every slot f
 * of token t, Xp[row_id_map[f], :] = X[t, :].  Equivalently
 * Xp[i, :] = X[gather_idx[i] / topk, :].  Bit-exact copy.
 *  X [T, K] bf16, row_id_map [R] int32 (from gg_route_hist_offsets),
 *  Xp [R, K] bf16 out.  A map entry outside [0, R) sets GG_DEV_BAD_ROW_INDEX. */
int gg_permute(const gg_bf16* X, const int32_t* row_id_map, int64_t T, int topk, int64_t K,
               gg_bf16* Xp, int32_t* status, void* stream);

/* ------------------------------------------------------ unpermute-combine --
 * Expert outputs back to token order, weighted combine over a token's slots
 * ([W] unpermute: combine with routing probabilities; [V] matmul_ogs_torch:
 * accumulate every slot of a token in fp32):
 *   out[t, :] = bf16( sum_{j<topk} w[t*topk+j] * Y[row(t*topk+j), :] )
 * summed in fp32 in j order.
 *  Y [R, N] bf16; row_id_map [R] int32, or NULL when Y is already in
 *  token-slot order (row(f) = f, e.g. after a forward with permute_y);
 *  topk_w [T, topk] fp32, or NULL for unit weights; out [T, N] bf16.
 * With row_id_map = NULL and topk_w = NULL this is the top-k sum of a
 * token-slot-ordered tensor ([U] GroupedGemm.backward, the sum over topk). */
int gg_unpermute_combine(const gg_bf16* Y, const int32_t* row_id_map, const float* topk_w,
                         int64_t T, int topk, int64_t N, gg_bf16* out, int32_t* status,
                         void* stream);

/* ----------------------------------------------- unpermute-combine, bwd --
 * Gradient of gg_unpermute_combine ([W] unpermute_bwd: gradients of the
 * unpermute forward, taking the forward's input for the probabilities'
 * gradient; no probabilities means unit weights).  With G = dL/d out:
 *   dY[row(f), :] = bf16( w[f] * G[t, :] )            for every slot f = t*topk + j
 *   dw[f]         = sum_n G[t, n] * Y[row(f), n]      (fp32)
 *  G [T, N] bf16; Y [R, N] bf16, the forward's input (needed only for dw);
 *  row_id_map [R] int32 or NULL (identity); topk_w [T, topk] fp32 or NULL (1);
 *  dY [R, N] bf16 out (every row written once); dw [T, topk] fp32 out or NULL.
 *  dw without Y -> GG_ERR_INVALID_ARG.  Deterministic (fixed reduction order).
 *  A map entry outside [0, R) sets GG_DEV_BAD_ROW_INDEX; that slot gets dw 0. */
int gg_unpermute_combine_bwd(const gg_bf16* G, const gg_bf16* Y, const int32_t* row_id_map,
                             const float* topk_w, int64_t T, int topk, int64_t N, gg_bf16* dY,
                             float* dw, int32_t* status, void* stream);

/* ---------------------------------------------------------------- forward --
 * Grouped GEMM forward ([U] grouped_gemm_forward; [V] matmul_ogs docstring:
 * Y[idx_y(e)] = X[idx_x(e)] @ W[e]^T):
 *   for every expert-order row i of expert e:
 *     a   = X[gather_idx[i] / topk]  if permute_x  (X is [T, K])
 *           X[i]                      otherwise    (X is [R, K], expert order)
 *     y   = a @ W[e]^T                (fp32 accumulate)
 *     y  *= topk_w[gather_idx[i]]     if fuse_mul_post (needs permute_y)
 *     Y[gather_idx[i]] = bf16(y)      if permute_y (token-slot order)
 *     Y[i]             = bf16(y)      otherwise
 *  W [E, N, K] bf16; m_sizes [E] int32 with sum R; gather_idx [R] (needed when
 *  a permute flag is set); topk_w [T, topk] fp32 (needed for fuse_mul_post);
 *  Y [R, N] bf16 out.  permute_x and permute_y may be combined (gather on
 *  load and scatter on store in one pass). */
int gg_forward(const gg_bf16* X, const gg_bf16* W, const int32_t* m_sizes,
               const int32_t* gather_idx, const float* topk_w, int64_t T, int topk, int E,
               int64_t N, int64_t K, int permute_x, int permute_y, int fuse_mul_post,
               gg_bf16* Y, int32_t* status, void* stream);

/* ---------------------------------------------- forward + fused combine --
 * The forward grouped GEMM with the weighted top-k combine of
 * gg_unpermute_combine fused into its epilogue as atomic adds ([V] the
 * scatter path: with several active experts per token each token row is a
 * sum over its slots; the output starts zeroed):
 *   out[t] = sum over the slots f = t*topk + j of  w[f] * (a_f @ W[e(f)]^T)
 *   a_f, W[e] as gg_forward (permute_x selects X [T, K] with the gather, else
 *   X [R, K] in expert order); w = topk_w [T, topk] fp32, or 1 when NULL.
 *  out [T, N] bf16 out.  Two accumulations:
 *   - with a workspace of gg_workspace_size(GG_OP_FORWARD_COMBINE, T, topk,
 *     E, N, K, 0) bytes (T*N fp32): the call zeroes it, every slot's scaled
 *     fp32 row is added there with fp32 atomic adds, and one pass rounds the
 *     sums to bf16 into out (any topk);
 *   - workspace NULL: out is zeroed and every slot's row, rounded to bf16, is
 *     added with bf16 atomic adds (each add rounds); topk above
 *     GG_COMBINE_BF16_MAX_TOPK returns GG_ERR_WORKSPACE, since the summed
 *     roundings of more slots approach the 1e-2 relative error bound.
 *  NOT deterministic: the order of a token's topk adds depends on scheduling,
 *  so the last bits can differ from run to run; gg_forward with permute_y and
 *  gg_unpermute_combine give the deterministic result (one fp32 sum, rounded
 *  once).  The per-slot rows are not stored, so training that needs them
 *  (the routing-weight gradient of gg_unpermute_combine_bwd) uses that path. */
int gg_forward_combine(const gg_bf16* X, const gg_bf16* W, const int32_t* m_sizes,
                       const int32_t* gather_idx, const float* topk_w, int64_t T, int topk, int E,
                       int64_t N, int64_t K, int permute_x, gg_bf16* out, void* workspace,
                       size_t workspace_bytes, int32_t* status, void* stream);

/* ------------------------------------------------------ forward + SwiGLU --
 * The forward grouped GEMM with the gated activation fused into its epilogue
 * ([V] FusedActivation with reduction_n = 2: each pair of adjacent output
 * columns reduces to one).  Output columns are interleaved gate/up:
 *   y   = as gg_forward (no scatter, no scale)          [R, N]
 *   A[i, c] = bf16( silu(y[2c]) * y[2c+1] )             [R, N/2], from the fp32 y
 *   silu(g) = g / (1 + exp(-g))
 *  Y [R, N] bf16 out, or NULL to store only the activation (inference);
 *  training keeps Y for gg_swiglu_bwd.  N must be a multiple of 16. */
int gg_forward_swiglu(const gg_bf16* X, const gg_bf16* W, const int32_t* m_sizes,
                      const int32_t* gather_idx, int64_t T, int topk, int E, int64_t N, int64_t K,
                      int permute_x, gg_bf16* Y, gg_bf16* A, int32_t* status, void* stream);

/* Gradient of that activation: from the stored H = y [rows, 2I] and
 * dA = dL/dA [rows, I] (bf16), with s = 1 / (1 + exp(-g)):
 *   dH[r, 2c]   = dA * u * s * (1 + g * (1 - s))      (gate)
 *   dH[r, 2c+1] = dA * g * s                            (up)
 * dH [rows, 2I] bf16 out.  I must be a multiple of 8. */
int gg_swiglu_bwd(const gg_bf16* H, const gg_bf16* dA, int64_t rows, int64_t I, gg_bf16* dH,
                  void* stream);

/* ------------------------------------------------------------ backward dX --
 * Gradient of the forward's input ([U] grouped_gemm_dX; GroupedGemm.backward):
 *   for every expert-order row i of expert e:
 *     g  = dY[gather_idx[i]] if permute_y else dY[i]     (dY is [R, N])
 *     dx = g @ W[e]                                      (reduce over N)
 *     dX[gather_idx[i]] = bf16(dx) if permute_x (token-slot order) else dX[i]
 *  dX [R, K] bf16 out.  dX_tok [T, K] bf16 out or NULL: with permute_x, the
 *  per-token sum over its topk slots of the stored bf16 dX rows (fp32 sum in
 *  slot order).  dX_tok without permute_x -> GG_ERR_INVALID_ARG.  The flags
 *  are those of the forward call being differentiated. */
int gg_backward_dX(const gg_bf16* dY, const gg_bf16* W, const int32_t* m_sizes,
                   const int32_t* gather_idx, int64_t T, int topk, int E, int64_t N, int64_t K,
                   int permute_x, int permute_y, gg_bf16* dX, gg_bf16* dX_tok, int32_t* status,
                   void* stream);

/* ---------------------------------------------- backward dX + SwiGLU bwd --
 * The backward dX of a grouped GEMM whose input was the SwiGLU activation of
 * gg_forward_swiglu, with the activation's backward fused into the epilogue
 * (the two steps of gg_backward_dX and gg_swiglu_bwd in one pass; the
 * activation gradient never goes to memory and is not rounded to bf16):
 *   for every expert-order row i of expert e:
 *     da = dY[i] @ W[e]                                  (fp32, [K])
 *     g = H[i, 2c], u = H[i, 2c+1], s = 1 / (1 + exp(-g))
 *     dH[i, 2c]   = bf16( da[c] * u * s * (1 + g * (1 - s)) )
 *     dH[i, 2c+1] = bf16( da[c] * g * s )
 *  dY [R, N] bf16 in expert order (gg_permute a token-slot-order gradient
 *  first); W [E, N, K]; H [R, 2K] bf16, the stored forward output of
 *  gg_forward_swiglu (expert order); dH [R, 2K] bf16 out. */
int gg_backward_dX_swiglu(const gg_bf16* dY, const gg_bf16* W, const int32_t* m_sizes, int64_t T,
                          int topk, int E, int64_t N, int64_t K, const gg_bf16* H, gg_bf16* dH,
                          int32_t* status, void* stream);

/* ------------------------------------------------------------ backward dW --
 * Gradient of the expert weights ([U] grouped_gemm_dW; [V] ragged-dw comment:
 * the reduction dimension is each expert's own rows):
 *   dW[e] = sum over expert-order rows i of e of  outer(g_i, a_i)   -> (N, K)
 *     a_i = X[gather_idx[i] / topk] if permute_x else X[i]
 *     g_i = dY[gather_idx[i]]       if permute_y else dY[i]
 *  fp32 accumulate, bf16 out; an expert with no rows gets dW[e] = 0.
 *  X [T, K] if permute_x else [R, K]; dY [R, N]; dW [E, N, K] bf16 out.
 *  workspace (may be NULL): with a permute flag and at least
 *  gg_workspace_size(GG_OP_BACKWARD_DW, T, topk, E, N, K, flags) bytes, the
 *  gathered operands are first copied into expert order there (X rows
 *  R*K*2 bytes, dY rows R*N*2 bytes) and the reduction reads dense tiles;
 *  with NULL the row gathers are fused into the reduction's operand loads,
 *  which is 2.5-4x slower on sm_103a (each reduction block needs 64 newly
 *  gathered rows, fetched in 16-byte pieces).  Both give the same products. */
int gg_backward_dW(const gg_bf16* X, const gg_bf16* dY, const int32_t* m_sizes,
                   const int32_t* gather_idx, int64_t T, int topk, int E, int64_t N, int64_t K,
                   int permute_x, int permute_y, gg_bf16* dW, void* workspace,
                   size_t workspace_bytes, int32_t* status, void* stream);

/* --------------------------------------------------------- dual asymmetric --
 * Two experts' GEMMs with different row counts and output widths in one
 * launch ([W] asym_dual_gmm_separated):  Y0 = op(X0) @ op(W0),
 * Y1 = op(X1) @ op(W1), shared reduction length k.
 *  trans_a = 0: X0 [m0, k], X1 [m1, k];  trans_a = 1: X0 [k, m0], X1 [k, m1].
 *  trans_b = 0: W0 [k, n0], W1 [k, n1];  trans_b = 1: W0 [n0, k], W1 [n1, k].
 *  Y0 [m0, n0], Y1 [m1, n1] bf16 out, fp32 accumulate.
 *  m0, m1, n0, n1 and k must be multiples of 8 (16-byte rows either way). */
int gg_dual_asym(const gg_bf16* X0, const gg_bf16* X1, const gg_bf16* W0, const gg_bf16* W1,
                 gg_bf16* Y0, gg_bf16* Y1, int64_t m0, int64_t m1, int64_t k, int64_t n0,
                 int64_t n1, int trans_a, int trans_b, int32_t* status, void* stream);

/* ------------------------------------------------------- expert parallel --
 * Rows routed to experts held by other ranks ([V] FusedComm and
 * post_matmul_comm_torch: routed rows exchanged between the ranks that hold
 * different experts).  G ranks; rank r holds experts [r*E_loc, (r+1)*E_loc),
 * E = G * E_loc <= GG_MAX_EXPERTS.  After gg_route_hist_offsets and
 * gg_permute over all E experts, rank r's rows for rank d's experts are the
 * contiguous block d of its expert-order rows.  The caller exchanges, with
 * its own collectives (e.g. NCCL all-to-all), first the counts
 * (recv_m[s][e] = rank s's m_sizes[r*E_loc + e]), then the rows: rank r
 * receives from each source s, in source order, s's rows for r's experts,
 * expert after expert.  The local GEMMs want expert-contiguous rows:
 *   received row j of block (s, e), q-th in it, becomes local row
 *   row_map[j] = local_off[e] + sum_{s'<s} recv_m[s'][e] + q,
 * local_off = exclusive prefix of local_m_sizes[e] = sum_s recv_m[s][e]; so
 * gg_permute(X_recv, row_map, topk = 1) gives them, and after the local
 * GEMMs gg_unpermute_combine(Y_loc, row_map, NULL, R_loc, 1) puts the results
 * back in received order for the return exchange.  Within an expert, rows
 * stay in (source rank, source row) order: the order of one routing of every
 * rank's tokens numbered rank after rank. */

/* Host-side plan (no GPU work; all arrays host memory).  m_sizes [G*E_loc]:
 * this rank's histogram over all experts; recv_m [G][E_loc]: received counts.
 * Out: send_counts [G] rows for each rank, recv_counts [G] rows from each
 * rank, local_m_sizes [E_loc]; row_map [R_loc] (or NULL) as above, row_map_len
 * must be R_loc = sum of recv_m.  Negative counts -> GG_ERR_INVALID_ARG. */
int gg_ep_plan(const int32_t* m_sizes, const int32_t* recv_m, int G, int E_loc, int64_t* send_counts,
               int64_t* recv_counts, int32_t* local_m_sizes, int32_t* row_map, int64_t row_map_len);

/* The same row_map computed on the device from the device copy of recv_m
 * [G][E_loc] (int32), for R_loc received rows; row_map [R_loc] int32 out.
 * R_loc not equal to the sum of recv_m (or a negative count) sets
 * GG_DEV_SIZES_MISMATCH; rows past the counted ones get -1. */
int gg_ep_recv_map(const int32_t* recv_m, int G, int E_loc, int64_t R_loc, int32_t* row_map,
                   int32_t* status, void* stream);

/* ------------------------------------------------------ low-rank adapters --
 * One shared projection W with the low-rank adapters of many requests beside
 * it: each token's row takes its own adapter a = ids[t] (-1: none).
 *   U[t] = bf16( scale[a] * (X[t] @ A[a]^T) )            (0 without an adapter)
 *   Y[t] = bf16( X[t] @ W^T + U[t] @ B[a]^T )            (fp32 accumulate)
 * Rows stay in the caller's order; ids may come in runs (sequences) or mixed.
 *  X [T, K], W [N, K], A [L, r, K], B [L, N, r], Y [T, N], U [T, r] bf16, rows
 *  contiguous; scale [L] fp32, or NULL for 1.  r a multiple of 8, at most
 *  GG_LORA_MAX_RANK (a smaller rank is zero-padded by the caller); N, K
 *  multiples of 8; L <= GG_MAX_EXPERTS.  A row is computed from its own adapter
 *  alone: infinities or NaN in one adapter or row reach no other row.
 *  U is kept for the backward (needed by it alone).  Outputs (here and in the
 *  backward) overlap neither inputs nor one another: kernels of a call run side
 *  by side.  No counterpart on the pages.
 *
 * gg_lora_plan reads a batch's ids once: the adapters that occur in each 256
 * rows, as row masks, and the rows sorted by adapter, into a buffer of
 * gg_lora_plan_size(T, L) bytes (16-byte aligned; 0 bytes: T or L out of
 * range).  One plan serves every projection and layer of the batch, forward and
 * backward.  An id outside [-1, L) sets GG_DEV_BAD_ADAPTER_ID and counts as -1. */
size_t gg_lora_plan_size(int64_t T, int L);
int gg_lora_plan(const int32_t* ids, int64_t T, int L, void* plan, size_t plan_bytes, int32_t* status,
                 void* stream);
int gg_lora_forward(const gg_bf16* X, const gg_bf16* W, const gg_bf16* A, const gg_bf16* B,
                    const float* scale, const void* plan, int64_t T, int L, int r, int64_t N,
                    int64_t K, gg_bf16* Y, gg_bf16* U, int32_t* status, void* stream);

/* Gradient of gg_lora_forward (W is frozen; gg_backward_dW gives its gradient):
 *   V[t]  = scale[a] * (dY[t] @ B[a])                     (kept in the workspace)
 *   dX[t] = bf16( dY[t] @ W + bf16(V[t]) @ A[a] )         (fp32 accumulate)
 *   dA[a] = bf16( sum over tokens t of adapter a of outer(V[t], X[t]) )
 *   dB[a] = bf16( sum over tokens t of adapter a of outer(dY[t], U[t]) )
 *  dY [T, N], U [T, r] the forward's; dX [T, K], dA [L, r, K], dB [L, N, r] out,
 *  each may be NULL (not computed; its operands may then be NULL too: X for dA,
 *  U for dB, W and A for dX).  An adapter without tokens gets zeros.
 *  dX takes V rounded to bf16, as the forward takes U (the tensor cores' operand);
 *  dA, which sums V over tokens, takes it as two bf16 of its sign (2^-16 of V), so
 *  an infinity in X or V stays one.
 *  workspace: gg_lora_backward_workspace_size(T, r) bytes, 16-byte aligned
 *  (whichever gradients are wanted; 327680 r bytes of it are partial sums, whatever
 *  T).  Deterministic (fixed reduction orders). */
size_t gg_lora_backward_workspace_size(int64_t T, int r);
int gg_lora_backward(const gg_bf16* dY, const gg_bf16* X, const gg_bf16* W, const gg_bf16* A,
                     const gg_bf16* B, const float* scale, const void* plan, const gg_bf16* U,
                     int64_t T, int L, int r, int64_t N, int64_t K, gg_bf16* dX, gg_bf16* dA,
                     gg_bf16* dB, void* workspace, size_t workspace_bytes, int32_t* status,
                     void* stream);

/* -------------------------------------------------------- rotary positions --
 * Rotary positions on the heads of q and k ([W] rope, rope_bwd), in one launch:
 * pair i of a head (0 <= i < rot / 2) turns by th = positions[t] * f_i,
 *   x1' = attention_scale * (x1 cos th - x2 sin th)
 *   x2' = attention_scale * (x2 cos th + x1 sin th)
 * (x1, x2) = elements (i, i + rot/2), or (2i, 2i + 1) when interleaved; the
 * elements from rot on are copied.  backward != 0: the gradient, th negated.
 * fp32 arithmetic, one rounding; the angle is exact to fp32 at any position.
 *  q, out_q: n_q heads of T tokens, element (t, h, c) at t * tok + h * head + c
 *  (strides in elements, as given per tensor); k, out_k likewise with n_k heads
 *  (n_q or n_k may be 0).  An output may be its input (same strides: in place,
 *  the elements from rot on untouched) or must not overlap it, and its heads must
 *  not overlap one another (token or head strides below the width written, 0
 *  included, are refused).
 *  positions [axes, T] int32 (any value); axes > 1: sections (HOST array, axes
 *  entries, sum rot / 2) gives each axis its consecutive pairs, so tokens can
 *  carry a time, a height and a width.
 *  steps [rot / 2] int64: f_i / (2 pi) turns in units of 2^-64 (rounded; scaled
 *  frequencies for long contexts are just other steps).
 *  dtype GG_DTYPE_*; D head width, rot even, 0 <= rot <= D, rot <= 1024. */
int gg_rope(const void* q, int64_t q_tok, int64_t q_head, int n_q, const void* k, int64_t k_tok,
            int64_t k_head, int n_k, void* out_q, int64_t oq_tok, int64_t oq_head, void* out_k,
            int64_t ok_tok, int64_t ok_head, const int32_t* positions, int axes,
            const int32_t* sections, const int64_t* steps, float attention_scale, int64_t T, int D,
            int rot, int interleaved, int dtype, int backward, void* stream);

/* --------------------------------------------- activations kept in 8 bits --
 * What a training step keeps from its forward for its backward, in 8.25 bits an
 * element.  Blocks of 32 consecutive columns of a row share a scale, a power of two:
 *   amax = max |x| of the block;  e = the least integer >= -117 with amax <= M 2^e
 *          (M = 127: GG_ACT8_INT8, 448: GG_ACT8_E4M3);  scale byte s = e + 127
 *   code = x 2^-e rounded half to even to an 8-bit integer, or to e4m3
 *   the code stands for code 2^e
 * The scaling is exact, so the rounding to 8 bits is the only one: an int8 value is
 * off by at most 2^(e-1) (amax / 127 at most), an e4m3 one by 2^-4 of itself (2^(e-10)
 * where it is below 2^(e-6)).  A block that holds an infinity, a NaN or an |x| of
 * 2^127 or more has s = 255 and stands for NaN throughout (its codes say nothing).
 *  Rows of C columns (a multiple of 8), nb = ceil(C / 32) blocks:
 *   codes  [rows, 32 nb] bytes, 16-byte aligned; the columns past C hold 0
 *   scales [rows, 4 ceil(nb / 4)] bytes, 4-byte aligned; what lies past nb says nothing
 * No counterpart on the pages.
 *
 * gg_act8_pack: X [rows, C] of dtype GG_DTYPE_*.
 * gg_act8_unpack: out [rows, C] of dtype (one rounding where it has fewer bits, none in
 *  bf16 and fp32), row i from source row i, or from gather_idx[i] / div ([rows] int32:
 *  with div = topk the layer's input in expert order, as gg_permute gives it, for
 *  gg_backward_dW); an index outside [0, src_rows * div) sets GG_DEV_BAD_ROW_INDEX and
 *  its row is zeroed.  Without gather_idx rows must be src_rows. */
int gg_act8_pack(const void* X, int dtype, int64_t rows, int64_t C, int fmt, uint8_t* codes,
                 uint8_t* scales, void* stream);
int gg_act8_unpack(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t src_rows,
                   int64_t C, const int32_t* gather_idx, int div, int64_t rows, void* out,
                   int dtype, int32_t* status, void* stream);

/* gg_forward_swiglu with its pre-activation kept in 8 bits: y [R, N] goes from the
 * fp32 accumulators to codes [R, 32 ceil(N / 32)] and scales in the epilogue (it is
 * never stored in bf16); A [R, N/2] as there, from the fp32 y (its quotient is within two
 * fp32 steps, and 0 for gates under -87.3, where silu is under 2^-119).  The other
 * arguments as there.  Codes, scales and A overlap neither inputs (m_sizes and gather_idx
 * among them) nor one another (GG_ERR_INVALID_ARG). */
int gg_forward_swiglu_act8(const gg_bf16* X, const gg_bf16* W, const int32_t* m_sizes,
                           const int32_t* gather_idx, int64_t T, int topk, int E, int64_t N,
                           int64_t K, int permute_x, int fmt, uint8_t* codes, uint8_t* scales,
                           gg_bf16* A, int32_t* status, void* stream);

/* gg_swiglu_bwd from the kept pre-activation (codes and scales of [rows, 2I]):
 *   dH [rows, 2I] bf16 out as there, with (g, u) the values that the codes stand for;
 *   A [rows, I] bf16 out, or NULL: silu(g) u again, so that a step need not keep the
 *   activation for the next weight's gradient.  I a multiple of 8. */
int gg_swiglu_bwd_act8(const uint8_t* codes, const uint8_t* scales, int fmt, const gg_bf16* dA,
                       int64_t rows, int64_t I, gg_bf16* dH, gg_bf16* A, void* stream);

/* -------------------------------------------------- norms around a block --
 * From the rows that a block leaves to the input of the next, in one pass:
 *   y[t]  = sum_{j<topk} topk_w[t, j] Y[row(t*topk + j)]      (as gg_unpermute_combine)
 *   n[t]  = y[t] w_post / sqrt(mean(y[t]^2) + eps)            (y[t] when w_post is NULL)
 *   h'[t] = res_scale h[t] + gate token_gate[t] n[t]
 *   x[t]  = h'[t] w_pre / sqrt(mean(h'[t]^2) + eps)
 * in fp32, each output rounded once (x from the fp32 h').
 *  h, out_h [T, K] of h_dtype (GG_DTYPE_BF16 or GG_DTYPE_F32): the residual stream;
 *  out_h may be h (in place).
 *  Y [T*topk, K] bf16, row_id_map [T*topk] or NULL (token-slot order), topk_w [T, topk]
 *  fp32 or NULL (1); with topk = 1 and neither, Y is the block's output as it is.  A map
 *  entry outside [0, T*topk) sets GG_DEV_BAD_ROW_INDEX and adds nothing.
 *  w_post, w_pre, gate [K] fp32, token_gate [T] fp32; w_post, gate and token_gate may be
 *  NULL (no norm, 1, 1).
 *  out_x [T, K] bf16, needs w_pre; NULL: no second norm.
 *  Y NULL: the norm of h alone (h' is h: res_scale is not used, out_h is not written and
 *  may be NULL).
 *  out_y [T, K] bf16, or y_codes and y_scales in the 8-bit form fmt (at most one of the
 *  two): y, rounded, for the backward; both may be NULL.
 *  K a multiple of 8, at most GG_NORM_MAX_K; eps > 0 (a row of zeros is normed to zeros).
 *  Squares are summed in fp32: a row whose sum of squares passes its range is normed to
 *  zeros.  Rows are copied behind bounded waits (status: GG_DEV_TIMEOUT).
 *  Outputs may not overlap inputs or one another (GG_ERR_INVALID_ARG), but out_h may be h:
 *  the whole of it, and then no other input's memory, but for a Y of the same address and
 *  bf16 rows with topk = 1 and no map.  No counterpart on the pages. */
int gg_block_norm(const void* h, int h_dtype, const gg_bf16* Y, const int32_t* row_id_map,
                  const float* topk_w, int topk, const float* w_post, const float* gate,
                  const float* token_gate, float res_scale, const float* w_pre, float eps,
                  int64_t T, int64_t K, void* out_h, gg_bf16* out_x, gg_bf16* out_y,
                  uint8_t* y_codes, uint8_t* y_scales, int fmt, int32_t* status, void* stream);

/* Its gradients, at the stored h' and y (the norms' statistics are taken from them again):
 *   G[t]    = dh'[t] + r (w_pre dx[t] - h'[t] r^2 mean(w_pre dx[t] h'[t])),
 *             r = 1 / sqrt(mean(h'[t]^2) + eps)
 *   dh[t]   = res_scale G[t]
 *   dy[t]   = q (m - y[t] q^2 mean(m y[t])),  m = w_post gate token_gate[t] G[t],
 *             q = 1 / sqrt(mean(y[t]^2) + eps)                (m when w_post is NULL)
 *   dw_pre  = sum_t dx[t] h'[t] r         dw_post = sum_t gate token_gate[t] G[t] y[t] q
 *   dgate   = sum_t token_gate[t] G[t] n[t]        dtoken_gate[t] = sum_c G[t] gate n[t]
 * dy feeds gg_unpermute_combine_bwd where the forward combined expert rows.
 *  dh, out_dh [T, K] of h_dtype; dh NULL: 0; out_dh may be dh (in place), or NULL.
 *  dx [T, K] bf16, NULL without the second norm (w_pre is then NULL too).
 *  h [T, K] of h_dtype: the forward's out_h (without a block: its h).
 *  y [T, K] bf16, or y_codes and y_scales in fmt; none of them: no block (dy, dw_post,
 *  dgate and dtoken_gate NULL; dh[t] = G[t], for h' is h).
 *  dy [T, K] bf16; dw_post, dw_pre, dgate [K], dtoken_gate [T] fp32, each may be NULL.
 *  workspace: gg_block_norm_bwd_workspace_size(T, K) bytes, 16-byte aligned: partial sums
 *  over tokens (may be NULL when none of dw_post, dw_pre and dgate is wanted).
 *  Outputs, the workspace among them, overlap neither inputs nor one another
 *  (GG_ERR_INVALID_ARG), but out_dh may be dh: the whole of it, and then no other input's
 *  memory, but for dx, h or y of the same address and as long rows.
 *  A row whose squares' sum passes fp32's range (which the forward norms to zeros) gets the
 *  zero gradient through that norm; where products of its elements with the gradients pass
 *  it too, NaN, and so do the vectors'.
 *  Deterministic (fixed summation orders). */
size_t gg_block_norm_bwd_workspace_size(int64_t T, int64_t K);
int gg_block_norm_bwd(const void* dh, const gg_bf16* dx, const void* h, int h_dtype,
                      const gg_bf16* y, const uint8_t* y_codes, const uint8_t* y_scales, int fmt,
                      const float* w_post, const float* gate, const float* token_gate,
                      float res_scale, const float* w_pre, float eps, int64_t T, int64_t K,
                      void* out_dh, gg_bf16* dy, float* dw_post, float* dw_pre, float* dgate,
                      float* dtoken_gate, void* workspace, size_t workspace_bytes, int32_t* status,
                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GG_H */
