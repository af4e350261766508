/*
 * mok.h — C ABI of the GB300 (sm_103a) DeepSeek-V3-style mixture-of-experts layer.
 *
 * The layer (page "Mixture-of-Kittens: Nhân kernel MoE nguồn mở tối ưu cho hệ thống NVL72",
 * section "Chồng lấp tính toán và truyền tải trong MoE"): a router projection picks the top-k
 * routed experts of every token and gives each a router weight; every selected expert runs a
 * SwiGLU FFN (gate and up projections, SiLU(gate) * up, down projection); the output is the
 * always-on shared expert plus the router-weighted sum of the routed experts:
 *
 *     logits = x W_router + b                     (fp32)
 *     topk   = the k largest logits, ties to the lower expert index
 *     w_j    = softmax(logits)[e_j] / sum_{i<k} softmax(logits)[e_i]
 *     y      = FFN_shared(x) + sum_j w_j FFN_{e_j}(x),   FFN(x) = (SiLU(x Wg) * (x Wu)) Wd
 *
 * Dispatch follows the pull schedule of the same page, section "Lập lịch" (each expert's
 * destination rows list its source tokens; one GPU, so the source rank is always 0) and the
 * pull example of the page "Метод и эксперименты" (tokens ascend inside an expert's region).
 * Results are bit-identical from run to run (page "Mixture-of-Kittens; MoE megakernel", key
 * points): every reduction runs in a fixed order and no floating-point atomics are used.
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller unless stated otherwise.
 *    The library never allocates, frees or synchronises (except mok_read_device_status and the
 *    host-buffer entry point, which say so).  Work is enqueued on `stream` and runs
 *    asynchronously.
 *  - Layouts are row-major and dense: x[T,d], W_router[d,E], W_gate/W_up[E,d,F],
 *    W_down[E,F,d], Ws_gate/Ws_up[d,Fs], Ws_down[Fs,d]; bf16 unless noted.
 *  - Preconditions (checked on the host; violations return MOK_ERR_UNSUPPORTED or
 *    MOK_ERR_INVALID_ARG and enqueue nothing): T >= 0; d % 128 == 0; F % 128 == 0;
 *    Fs % 128 == 0 when n_shared == 1; n_shared in {0,1}; 1 <= k <= 8; k <= E <= 512;
 *    E % 8 == 0; every pointer 16-byte aligned; workspace at least mok_workspace_size().
 *  - Device-side failures (a bounded wait that ran out, an out-of-range expert index) are
 *    recorded as a nonzero status word inside the workspace; nothing traps.  Read it with
 *    mok_read_device_status().  The word is sticky: clear it with mok_clear_device_status()
 *    (or allocate the workspace zeroed).
 *  - Return value: MOK_OK or a negative mok_status.  No entry point exits or aborts.
 */
#ifndef MOK_H
#define MOK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *mok_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
  MOK_OK = 0,
  MOK_ERR_INVALID_ARG = -1, /* null pointer, negative size, bad enum */
  MOK_ERR_UNSUPPORTED = -2, /* shape or alignment outside the preconditions */
  MOK_ERR_WORKSPACE = -3,   /* workspace too small */
  MOK_ERR_CUDA = -4,        /* a CUDA runtime / driver call failed */
  MOK_ERR_TIMEOUT = -5,     /* (device status) a bounded wait inside a kernel ran out */
  MOK_ERR_DEVICE_CHECK = -6 /* (device status) an index failed a device-side range check */
} mok_status;

typedef enum { MOK_BF16 = 0, MOK_MXFP8 = 1, MOK_NVFP4 = 2 } mok_dtype;

typedef enum { MOK_PASS_FORWARD = 0, MOK_PASS_BACKWARD = 1 } mok_pass;

/* Sizes of one layer call.  T tokens, d model dim, E routed experts, k experts per token,
 * F routed-expert intermediate, F_shared shared-expert intermediate, n_shared in {0,1},
 * dtype = arithmetic of the expert GEMMs (MOK_MXFP8: E4M3 values with one UE8M0 scale per
 * 32 elements along the reduction dimension; MOK_NVFP4: E2M1 values with one E4M3 scale per
 * 16 elements along the reduction dimension and one fp32 scale per tensor, forward only; the
 * router and combine stay fp32/bf16). */
typedef struct {
  int64_t T;
  int32_t d, E, k, F, F_shared, n_shared;
  int32_t dtype;
} mok_dims;

/* Layer weights (device, caller-owned). `prepared` is the output of mok_prepare_weights and is
 * required when dtype is MOK_MXFP8 or MOK_NVFP4 (ignored for MOK_BF16); `prepared_bwd`, the output of
 * mok_prepare_weights_bwd, is required by mok_moe_backward when dtype == MOK_MXFP8. */
typedef struct {
  const void *W_router;     /* [d,E] bf16 */
  const float *router_bias; /* [E] fp32, or NULL */
  const void *W_gate;       /* [E,d,F] bf16 */
  const void *W_up;         /* [E,d,F] bf16 */
  const void *W_down;       /* [E,F,d] bf16 */
  const void *Ws_gate;      /* [d,Fs] bf16 (NULL when n_shared == 0) */
  const void *Ws_up;        /* [d,Fs] bf16 */
  const void *Ws_down;      /* [Fs,d] bf16 */
  const void *prepared;     /* mok_prepared_size() bytes, or NULL */
  const void *prepared_bwd; /* mok_prepared_bwd_size() bytes, or NULL */
} mok_weights;

/* Bytes of device workspace needed by the entry points of `pass` (MOK_PASS_FORWARD covers
 * mok_route, mok_dispatch_index and mok_moe_forward; MOK_PASS_BACKWARD covers
 * mok_moe_backward).  Returns 0 for invalid dims. */
size_t mok_workspace_size(const mok_dims *dims, int pass);

/* Bytes of the activations mok_moe_forward saves for mok_moe_backward: G and U for the routed
 * rows and the shared expert (bf16 for MOK_BF16, fp32 for MOK_MXFP8, whose backward quantises
 * dG, dU and w*h derived from them), and with MOK_BF16 also x in expert order. */
size_t mok_saved_size(const mok_dims *dims);

/* Bytes of the prepared-weights buffer for dims->dtype (0 for MOK_BF16). */
size_t mok_prepared_size(const mok_dims *dims);

/* MXFP8: quantise the routed and shared expert weights once into `prepared` (E4M3 values and
 * UE8M0 scales, blocks of 32 along each weight's reduction dimension, same rule as
 * mok_mx_quantize_rows), transposed to K-major, in this order (each region 1 KB aligned):
 * W_gate codes [E][F][d] and scales; W_up likewise; W_down codes [E][d][F] and scales; then the
 * shared expert's three the same way.  The scales of a K-major matrix [N][K] (N rows, K/32 scale
 * bytes per row) are stored in 512-byte atoms [N/128][K/128]: the atom of row tile a and K block
 * b holds row n = 128a + 32 r1 + r0 (r0 < 32, r1 < 4), block 4b + j at byte 16 r0 + 4 r1 + j,
 * the shared-memory image the block-scaled MMA's scale copy reads.  No-op for MOK_BF16.
 * MXFP8 needs d % 256 == 0. */
int mok_prepare_weights(const mok_dims *dims, const mok_weights *w, void *prepared,
                        mok_stream_t stream);
/* NVFP4 (MOK_NVFP4; the first page, "Mixture-of-Kittens: Nhân kernel MoE ...", names NVFP4 as
 * the format of its authors' earlier kernels and defines neither format nor recipe; the format
 * is NVIDIA's NVFP4 and the recipe the plain two-level one): mok_prepare_weights quantises every
 * expert weight along its reduction dimension (K = d for gate and up, F for down), each matrix
 * with its own tensor scale: A = the matrix's amax, S = 2688 / A in fp32 (1 when A is 0); a block
 * of 16 with amax a takes the E4M3 scale s = rn((a / 6) * S) (saturating); an element v the E2M1
 * code rn(v * (S / s)) (ties to the even code, saturating at 6; sign bit when the product is
 * negative; 0 when s is 0); every step an fp32 operation rounded to nearest even.  Layout, in
 * this order, each region 1 KB aligned: W_gate codes, W_gate scales, W_up codes, W_up scales,
 * W_down codes, W_down scales, the shared expert's six likewise (E = 1), then g[3E + 3] fp32
 * (1 / S of gate e, up e, down e for e < E, then the shared gate, up, down), amax[3E + 3]
 * (scratch), act[2] fp32 (the calibrated activation amaxes, below).  Codes of a matrix with K
 * rows and N columns: for each 64-element K block kb and column n, 32 bytes at
 * ((m * K/64 + kb) * N + n) * 32 (m = the expert), byte j holding elements 2j (low nibble) and
 * 2j + 1 (high nibble) of the block; its 4 scale bytes (one per 16 elements) at
 * ((m * K/64 + kb) * N + n) * 4.  The activation amaxes are reset to 0 (tensor scale 1).
 * NVFP4 needs d % 256 == 0. */

/* NVFP4: sets the calibrated tensor amaxes of the forward's two quantised activations, x (the
 * layer input, quantised along d) and h (SiLU(G) * U, quantised along F from its fp32 value),
 * in `prepared` (the static form of the per-tensor scale: values beyond them saturate).  Both
 * must be finite and >= 0 (0 gives the tensor scale 1).  Returns MOK_ERR_INVALID_ARG for another
 * dtype, a NULL or unaligned buffer, or a negative or non-finite amax. */
int mok_nvfp4_set_activation_amax(const mok_dims *dims, void *prepared, float amax_x,
                                  float amax_h, mok_stream_t stream);

/* MXFP8 backward: the expert weights quantised once more, along the reduction dimension of the
 * backward GEMM that reads each (same rule and atom layout as mok_prepare_weights), in this order
 * (each region 1 KB aligned): W_down codes [E][F][d] (blocks along d, for dY W_down^T) and
 * scales; W_gate codes [E][d][F] (blocks along F, for dG W_gate^T) and scales; W_up likewise;
 * then the shared expert's Ws_down [Fs][d], Ws_gate [d][Fs], Ws_up [d][Fs] the same way.  No
 * transposes: each weight's rows are already along that K.  mok_prepared_bwd_size() bytes
 * (0 for MOK_BF16, where this call is a no-op).  The MXFP8 backward needs F % 256 == 0 and
 * Fs % 256 == 0 besides d % 256 == 0. */
size_t mok_prepared_bwd_size(const mok_dims *dims);
int mok_prepare_weights_bwd(const mok_dims *dims, const mok_weights *w, void *prepared_bwd,
                            mok_stream_t stream);

/* MXFP8 quantiser of activations: src[rows,K] bf16 -> q[rows,K] E4M3 codes and
 * scales[rows,K/32] UE8M0 bytes, one block per 32 consecutive elements of a row: scale 2^s with
 * s the smallest integer such that amax <= 448 * 2^s (amax / 448 rounded up to a power of two),
 * s in [-127,127] (an all-zero block gets 0x00), codes = round-to-nearest-even E4M3 of v * 2^-s
 * with saturation to +-448.  K % 128 == 0.  The MXFP8 format of the layer (page
 * "Mixture-of-Kittens; MoE megakernel", key points); the scale rule as read for the MXFP8
 * workload of the layer. */
int mok_mx_quantize_rows(int64_t rows, int K, const void *src, void *q, void *scales,
                         mok_stream_t stream);

/* Router: logits = x W_router + bias in fp32 (bf16 tensor-core products, fp32 accumulation),
 * top-k by (logit descending, index ascending), weights = softmax over all experts
 * renormalised over the selected ones.  Page "Mixture-of-Kittens: Nhân kernel MoE ...",
 * section "Chồng lấp tính toán và truyền tải trong MoE".
 *   x[T,d] bf16, W_router[d,E] bf16, bias[E] fp32 or NULL
 *   -> topk_idx[T,k] int32 (slot order = descending logit), topk_w[T,k] fp32,
 *      logits[T,E] fp32 (optional, NULL to skip).
 * topk_idx and topk_w may both be NULL: logits alone, for mok_select_experts. */
int mok_route(const mok_dims *dims, const void *x, const void *W_router, const float *bias,
              int32_t *topk_idx, float *topk_w, float *logits, void *ws, size_t ws_bytes,
              mok_stream_t stream);

/* Pull schedule (page "Mixture-of-Kittens: Nhân kernel MoE ...", section "Lập lịch"): a
 * deterministic counting sort of the T*k routes by expert, built from per-chunk histograms and
 * a prefix scan, with no atomics.  Within an expert, routes are ordered by token id.
 *   topk_idx[T,k] int32 (each value in [0,E)), topk_w[T,k] fp32
 *   -> counts[E], offsets[E+1] (offsets[0]=0, offsets[E]=T*k), sorted_tok[T*k] (token of each
 *      destination row), sorted_w[T*k] (its router weight), inv_pos[T,k] (destination row of
 *      route (t,j)).  An index outside [0,E) sets MOK_ERR_DEVICE_CHECK in the status word and
 *      that route is dropped. */
int mok_dispatch_index(const mok_dims *dims, const int32_t *topk_idx, const float *topk_w,
                       int32_t *counts, int32_t *offsets, int32_t *sorted_tok, float *sorted_w,
                       int32_t *inv_pos, void *ws, size_t ws_bytes, mok_stream_t stream);

/* Forward of the expert part given a routing (the output of mok_dispatch_index):
 * pull-gathers each expert's rows, runs the gate/up GEMM with SiLU(gate)*up fused in its
 * epilogue and the down GEMM with the router weight fused in its epilogue (routed experts and
 * the shared expert in one persistent launch per phase), then combines every token's rows in
 * ascending expert order on top of the shared-expert row (fp32 accumulation, one bf16
 * rounding).
 *   -> y[T,d] bf16.  `saved` (mok_saved_size bytes or NULL) receives what the backward needs:
 *   G and U (bf16; for MOK_MXFP8 the block-scaled products in fp32), and for MOK_BF16 x in
 *   expert order.  MOK_NVFP4: x is quantised with its calibrated amax, the gate/up GEMM's
 *   epilogue quantises h along F, both GEMMs multiply f16 NVFP4 values decoded from the
 *   prepared weights and apply the tensor scales in their epilogues; forward only (`saved` must
 *   be NULL, else MOK_ERR_UNSUPPORTED). */
int mok_moe_forward(const mok_dims *dims, const mok_weights *w, const void *x,
                    const int32_t *topk_idx, const int32_t *offsets, const int32_t *sorted_tok,
                    const float *sorted_w, const int32_t *inv_pos, void *y, void *saved,
                    void *ws, size_t ws_bytes, mok_stream_t stream);

/* Backward of the layer for upstream gradient dY[T,d] bf16, with the top-k selection held
 * constant (unselected experts get no gradient).  Uses `saved` from mok_moe_forward with the
 * same routing.  Outputs (bf16 unless noted; fp32 accumulation, fixed summation order):
 *   dX[T,d] (including the router path dlogits W_router^T), dW_gate/dW_up[E,d,F],
 *   dW_down[E,F,d] (experts with no token get zeros), dWs_gate/dWs_up[d,Fs], dWs_down[Fs,d]
 *   (NULL when n_shared == 0), dlogits[T,E] fp32 (zero off the selection),
 *   dW_router[d,E] (NULL to skip).
 * MOK_MXFP8 (the MXFP8 reading of the training step): every expert GEMM multiplies E4M3
 * operands with UE8M0 scales per 32 along its own reduction dimension — dY and W_down along d,
 * dG, dU, W_gate, W_up along F, and for the weight gradients x, dG, dU, w*h and dY along each
 * expert's tokens (blocks of 32 from its first token, in token order) — with fp32 accumulation;
 * the router terms dlogits W_router^T and x^T dlogits stay bf16.  Needs w->prepared_bwd and a
 * `saved` from an MXFP8 forward; F % 256 == 0, Fs % 256 == 0 and
 * 2 (ceil(T k / 128) + E) d / 64 < 2^31 (T below about 150M tokens at d = 7168, k = 8), else
 * MOK_ERR_UNSUPPORTED.  MOK_NVFP4 has no backward: MOK_ERR_UNSUPPORTED. */
int mok_moe_backward(const mok_dims *dims, const mok_weights *w, const void *x, const void *dY,
                     const void *saved, const int32_t *topk_idx, const float *topk_w,
                     const int32_t *offsets, const int32_t *sorted_tok, const float *sorted_w,
                     const int32_t *inv_pos, void *dX, void *dW_gate, void *dW_up, void *dW_down,
                     void *dWs_gate, void *dWs_up, void *dWs_down, float *dlogits,
                     void *dW_router, void *ws, size_t ws_bytes, mok_stream_t stream);

/* The whole layer forward (route, dispatch, expert forward) with x and y in HOST memory:
 * copies x_host[T,d] (bf16) to the workspace, runs the layer and copies y back to
 * y_host[T,d].  Pinned host memory makes the copies asynchronous; the call returns without
 * waiting (synchronise the stream before reading y_host, or writing x_host again).  Routing
 * tensors live inside the workspace (mok_workspace_size(dims, MOK_PASS_FORWARD) +
 * mok_layer_host_extra_size(dims)).  The copy of x runs on a library-owned copy stream into one
 * of two device buffers of the workspace, alternating per call, so that a call's copy overlaps
 * the kernels of the previous call on the same workspace; `stream` waits for it before the
 * layer runs, so synchronising `stream` still covers the whole call.  The library keeps one
 * copy stream per device and two events per workspace (for the 16 most recent workspaces).
 * When y_host is pinned (mapped) host memory, the final combine writes y straight into it;
 * otherwise y is combined in the workspace and copied back on `stream`. */
size_t mok_layer_host_extra_size(const mok_dims *dims);
int mok_layer_forward_host(const mok_dims *dims, const mok_weights *w, const void *x_host,
                           void *y_host, void *ws, size_t ws_bytes, mok_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Around the layer: the norm in front of it, the router's auxiliary losses, gradient clipping and
 * the optimiser.  The pages describe only the layer; these entry points carry a pre-norm residual
 * block built on it through a training step (and its norm through a serving step).  Same
 * conventions as above: caller-owned device memory, work enqueued on `stream`, nothing allocated,
 * bit-identical reruns.
 * ------------------------------------------------------------------------------------------- */

/* Element type of a tensor that may come in 16 or 32 bits. */
typedef enum { MOK_T_BF16 = 0, MOK_T_F32 = 1 } mok_elem;
/* Layout of MXFP8 scale bytes: [rows, K/32] row-major, or the 512-byte atoms
 * [ceil(rows/128)][K/128] that the layer's block-scaled GEMMs read (mok_prepare_weights). */
typedef enum { MOK_SCALES_ROWS = 0, MOK_SCALES_ATOMS = 1 } mok_scale_layout;

/* RMS norm with the residual's addition: h = x + residual (x when residual is NULL),
 * v = h / sqrt(mean(h^2) + eps) * weight per row of d elements, everything in fp32.
 *   x[T,d] bf16, residual[T,d] of res_type (or NULL), weight[d] of weight_type
 *   -> y[T,d] = v in bf16 (NULL to skip), residual_out[T,d] = h in res_type (required with a
 *      residual, NULL without), and with codes != NULL the MXFP8 form of v: codes[T,d] E4M3 and
 *      scales in scale_layout, by the rule of mok_mx_quantize_rows applied to v itself (not to
 *      its bf16 rounding).  The atoms' padding rows (T to the next multiple of 128) are zero.
 * At least one of y and codes.  residual_out may be residual and y may be x (in place).
 * T >= 0, 0 < d <= 32768, d % 8 == 0 (d % 128 == 0 with codes), eps > 0; 16-byte aligned
 * pointers.  One launch. */
int mok_rms_norm(int64_t T, int d, float eps, const void *x, const void *residual, int res_type,
                 const void *weight, int weight_type, void *y, void *residual_out, void *codes,
                 void *scales, int scale_layout, mok_stream_t stream);

/* Bytes of workspace of mok_rms_norm_backward (0 for invalid sizes). */
size_t mok_rms_norm_workspace_size(int64_t T, int d);

/* Gradients of mok_rms_norm.  With s[T,d] (res_type) the rows that were normalised (residual_out
 * of the forward, or x in bf16 when there was no residual), rho = 1 / sqrt(mean(s^2) + eps)
 * (recomputed), xhat = s rho and g = dy weight:
 *   ds = rho (g - xhat mean(g xhat)) + dres,   dweight = sum over rows of dy xhat.
 *   dy[T,d] bf16, dres[T,d] of res_type (the gradient that arrives through residual_out) or NULL
 *   -> ds in bf16 in dx[T,d] (NULL to skip) and in res_type in dresidual[T,d] (NULL to skip; at
 *      least one of the two), dweight[d] fp32 (rows summed in a fixed order).
 * ds is the gradient of x and of the residual alike.  dx may be dy, dresidual may be dres or s.
 * Sizes and alignment as in mok_rms_norm.  Two launches, the second begins under the first. */
int mok_rms_norm_backward(int64_t T, int d, float eps, const void *dy, const void *s, int res_type,
                          const void *weight, int weight_type, const void *dres, void *dx,
                          void *dresidual, float *dweight, void *ws, size_t ws_bytes,
                          mok_stream_t stream);

/* Bytes of workspace of mok_balance_loss for n_seqs sequences (0 for invalid sizes). */
size_t mok_balance_loss_workspace_size(const mok_dims *dims, int64_t n_seqs);

/* Balance loss and z loss of the router, per-expert counts and the gradient of the logits.
 * Tokens seq_offsets[s] <= t < seq_offsets[s+1] form sequence s; a token whose token_mask byte is
 * 0, or that is in no sequence, is left out of everything.  With p_t = softmax(logits_t),
 * n the number of valid tokens, n_s those of sequence s and c[s,e] how many of them chose e:
 *   balance = alpha sum_s (n_s / n) sum_e f[s,e] P[s,e],  f[s,e] = E c[s,e] / (k n_s),
 *             P[s,e] = the mean of p_t[e] over the sequence's valid tokens;
 *   z       = z_coef / n sum_t (log sum_e exp(logits_t[e]))^2;
 *   dlogits = grad d(balance + z)/d logits, the selection (and so c) held constant.
 *   logits[T,E] fp32, topk_idx[T,k] int32 (both from mok_route), seq_offsets[n_seqs+1] int32
 *   ascending on the device (NULL: one sequence of all tokens, n_seqs == 1), token_mask[T] bytes
 *   or NULL, grad a device scalar or NULL (1)
 *   -> counts[n_seqs,E] int32, loss[2] fp32 = {balance, z}, dlogits[T,E] fp32 (NULL to skip; rows
 *      of left-out tokens are zero, whatever their logits hold).
 * Experts masked with -inf logits get probability and gradient 0; a token all of whose logits are
 * -inf gives no loss and no gradient (finite logits are logits, however low: a row of the type's lowest
 * value is a uniform one with a huge z loss, unless token_mask leaves it out).  An index outside [0,E) sets MOK_ERR_DEVICE_CHECK in the
 * status word of ws and its route is not counted.  dims->T, E, k are used; n_seqs >= 1,
 * n_seqs * E < 2^31; logits, counts, dlogits and ws are 16-byte aligned.  The gradient goes into mok_moe_backward_aux. */
int mok_balance_loss(const mok_dims *dims, const float *logits, const int32_t *topk_idx,
                     const int32_t *seq_offsets, int64_t n_seqs, const uint8_t *token_mask,
                     float alpha, float z_coef, const float *grad, int32_t *counts, float *loss,
                     float *dlogits, void *ws, size_t ws_bytes, mok_stream_t stream);

/* Bytes of workspace of mok_grad_norm for tensors of these element counts (0 when invalid). */
size_t mok_grad_norm_workspace_size(int n_tensors, const int64_t *numel);

/* Norm of all gradients together: out[2] fp32 on the device = {norm, factor} with norm the root
 * of the sum of squares over every tensor (fp32 partial sums in a fixed order, joined in 64 bits)
 * and factor = min(1, max_norm / norm) (1 when max_norm <= 0, NaN when the norm is not finite or
 * its square overflows fp32).
 * grads, numel and types (mok_elem) are HOST arrays of n_tensors entries; they may be reused as
 * soon as the call returns.  Tensors are 16-byte aligned; empty ones are fine. */
int mok_grad_norm(int n_tensors, const void *const *grads, const int64_t *numel,
                  const int32_t *types, float max_norm, float *out, void *ws, size_t ws_bytes,
                  mok_stream_t stream);

/* Format of the AdamW states.  MOK_STATE_MXFP8: E4M3 codes [numel] and one UE8M0 byte per 32
 * consecutive elements [ceil(numel/32)], scale rule of mok_mx_quantize_rows, dithered rounding:
 * element i goes to the upper of its two neighbouring codes when its place between them plus
 * (r + 1/2) / 2^16 reaches 1.  With x = 0x85EBCA6B i + 0x9E3779B9 step, x ^= x >> 15,
 * x *= 0x2C1B3C6D, x ^= x >> 12, x *= 0x297A2D39, x ^= x >> 15 (all mod 2^32), r is x's high half
 * for exp_avg and its low half for exp_avg_sq.  The mean over steps is the value, so averages
 * that move by less than half a code per step still move.  exp_avg_sq > 0 never takes code 0 (its
 * step would be exp_avg / eps), so it has a lower limit, 2^-9 of the block's scale: where an
 * element's gradients are below 1/479 to 1/339 of the largest of its 32 (which of them depends on
 * where that one lies between two scales), exp_avg_sq is held at the limit and the step is too small
 * by the ratio of the roots: at 1/1000 it is 0.34 to 0.48 of the exact one, at 1/3000 0.11 to 0.16.
 * Weights whose blocks span such ratios want MOK_STATE_F32. */
typedef enum { MOK_STATE_F32 = 0, MOK_STATE_MXFP8 = 1 } mok_state_format;

/* One tensor of mok_adamw_step (device pointers, 16-byte aligned; the scales need not be).  No two
 * buffers of a call share memory, except that gradients may. */
typedef struct {
  void *param;               /* [numel] of param_type, updated */
  const void *grad;          /* [numel] of grad_type */
  float *master;             /* [numel] fp32 copy of a bf16 param, updated; NULL for an fp32 one */
  void *exp_avg;             /* [numel] fp32 or E4M3 codes, updated */
  void *exp_avg_sq;          /* [numel] likewise */
  uint8_t *exp_avg_scale;    /* [ceil(numel/32)], NULL for MOK_STATE_F32 */
  uint8_t *exp_avg_sq_scale;
  int64_t numel;
  double weight_decay;
  int32_t param_type;        /* mok_elem */
  int32_t grad_type;
} mok_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps;
  int64_t step;              /* 1 for the first step */
  int32_t state_format;      /* mok_state_format */
} mok_adamw_args;

/* One AdamW step over all tensors: with g = factor grad (factor = clip[1], or 1 when clip is
 * NULL), m = beta1 m + (1 - beta1) g, v = beta2 v + (1 - beta2) g^2,
 *   w = w - lr (m / (1 - beta1^step) / (sqrt(v / (1 - beta2^step)) + eps) + weight_decay w),
 * all in fp32 on the master (or the fp32 param); a bf16 param is the rounded master.  `tensors`
 * is a HOST array, free for reuse when the call returns; clip is the device output of
 * mok_grad_norm: when its factor is NaN (a norm that is not finite) the step leaves everything
 * unchanged.  0 <= beta < 1, eps >= 1e-15, step >= 1. */
int mok_adamw_step(const mok_adamw_args *args, const mok_adamw_tensor *tensors, int n_tensors,
                   const float *clip, mok_stream_t stream);

/* mok_moe_forward for MOK_MXFP8 with x already quantised: x_codes[T,d] and x_scales (atoms,
 * T rows x d) as mok_rms_norm or the layer's own quantiser write them; skips the layer's pass
 * over x.  Same outputs as mok_moe_forward on the same codes.  MOK_ERR_UNSUPPORTED for another
 * dtype. */
int mok_moe_forward_mx(const mok_dims *dims, const mok_weights *w, const void *x_codes,
                       const void *x_scales, const int32_t *topk_idx, const int32_t *offsets,
                       const int32_t *sorted_tok, const float *sorted_w, const int32_t *inv_pos,
                       void *y, void *saved, void *ws, size_t ws_bytes, mok_stream_t stream);

/* mok_moe_backward with a further gradient of the logits (dlogits_aux[T,E] fp32, from
 * mok_balance_loss; NULL: exactly mok_moe_backward), added in fp32 before dlogits is used: dX and
 * dW_router include it and the output dlogits is the sum. */
int mok_moe_backward_aux(const mok_dims *dims, const mok_weights *w, const void *x, const void *dY,
                         const void *saved, const int32_t *topk_idx, const float *topk_w,
                         const int32_t *offsets, const int32_t *sorted_tok, const float *sorted_w,
                         const int32_t *inv_pos, const float *dlogits_aux, void *dX, void *dW_gate,
                         void *dW_up, void *dW_down, void *dWs_gate, void *dWs_up, void *dWs_down,
                         float *dlogits, void *dW_router, void *ws, size_t ws_bytes,
                         mok_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Other routers, norms on both sides of a block and activations kept in 8 bits.  Same conventions.
 * ------------------------------------------------------------------------------------------- */

typedef enum { MOK_SCORE_SOFTMAX = 0, MOK_SCORE_SIGMOID = 1 } mok_score;
typedef enum { MOK_GROUP_MAX = 0, MOK_GROUP_TOP2 = 1 } mok_group_score;

/* How a router chooses experts from its logits (mok_select_experts). */
typedef struct {
  int32_t score;       /* mok_score */
  int32_t n_groups;    /* groups of E / n_groups neighbouring experts; 1: none */
  int32_t topk_groups; /* groups that stay */
  int32_t group_score; /* mok_group_score: a group's largest key, or the sum of its two largest */
  int32_t renormalise; /* weights over the chosen scores' sum */
  float scale;         /* factor of the weights */
} mok_selection;

/* Choice of the experts from logits[T,E] fp32 (of mok_route): with s = softmax(logits) or
 * sigmoid(logits) of a token and keys c = s + sel_bias (sel_bias[E] fp32 or NULL: it ranks, the
 * weights do not see it),
 *  - a group's score is its largest key or the sum of its two largest (its one, where it has one);
 *    the topk_groups best groups stay;
 *  - topk_idx[T,k] are the k largest keys of the groups that stay, in descending order (without
 *    sel_bias the order is that of the logits);
 *  - topk_w[T,k] = scale s_j / sum_i s_i over the chosen (0 when the sum is), or scale s_j.
 * Where fp32 cannot tell two keys apart they are computed in 64 bits; of keys that are equal there the
 * one of the larger logit comes first, of equal logits that of the lower index.  Experts of one bias
 * (or none) are so ranked as in exact arithmetic, whatever the logits; where biases differ, 64 bits
 * decide.  Groups likewise by their largest keys; sums of two are compared in 64 bits, and where these
 * are equal the lower group comes first.  Experts whose logit is at or below -1e30
 * (-inf, a type's lowest value) are shut off: s = 0, no key, chosen (lower index first) only where
 * the groups that stay have fewer than k others; a token without open experts gets weights 0.  A
 * bias at or below -1e30 makes its expert the last choice likewise, with its score.  A logit that is
 * NaN, and a bias that is NaN or at or above 1e30, count as -inf and set MOK_ERR_DEVICE_CHECK in the
 * status word of ws (256 bytes at least: any workspace of the library, zeroed once).
 * dims->T, E, k are used; 1 <= n_groups <= 32, E % n_groups == 0, 1 <= topk_groups <= n_groups,
 * k <= topk_groups E / n_groups, scale finite; logits, sel_bias and ws are 16-byte aligned.  One
 * launch.  The results go into mok_dispatch_index. */
int mok_select_experts(const mok_dims *dims, const mok_selection *sel, const float *logits,
                       const float *sel_bias, int32_t *topk_idx, float *topk_w, void *ws,
                       size_t ws_bytes, mok_stream_t stream);

/* Gradient of the logits for dtopk_w[T,k], the gradient of mok_select_experts' weights, with the
 * choice held constant; dlogits_aux[T,E] (of mok_balance_loss, or NULL) is added.  With p_j =
 * s_j / sum_i s_i:
 *   renormalised: dlogits_{e_j} = scale p_j (dw_j - sum_i p_i dw_i), times 1 - s_j for sigmoid
 *   scores; sigmoid: scale s_j (1 - s_j) dw_j; softmax: scale s_e (dw_e - sum_i s_i dw_i) for every
 *   expert (dw_e = 0 where e was not chosen); 0 elsewhere.
 * An index outside [0,E) sets MOK_ERR_DEVICE_CHECK in the status word of ws and is left out; routes
 * that name one expert twice add up.  Experts that are shut off get dlogits_aux alone (0 without it):
 * mok_balance_loss leaves out -inf, but a token all of whose logits are finite is one of its tokens
 * whatever they are, and at a type's lowest value its z loss is huge or infinite; such tokens are left
 * out by its token_mask.  sel's groups are not used but checked.  logits, dlogits_aux, dlogits and ws are 16-byte aligned; dlogits may be
 * dlogits_aux.  One launch. */
int mok_select_experts_backward(const mok_dims *dims, const mok_selection *sel, const float *logits,
                                const int32_t *topk_idx, const float *dtopk_w,
                                const float *dlogits_aux, float *dlogits, void *ws, size_t ws_bytes,
                                mok_stream_t stream);

/* mok_moe_backward_aux for a routing of mok_select_experts with this sel and logits (sel NULL:
 * exactly mok_moe_backward_aux, logits unused). */
int mok_moe_backward_select(const mok_dims *dims, const mok_weights *w, const void *x,
                            const void *dY, const void *saved, const mok_selection *sel,
                            const float *logits, const int32_t *topk_idx, const float *topk_w,
                            const int32_t *offsets, const int32_t *sorted_tok,
                            const float *sorted_w, const int32_t *inv_pos,
                            const float *dlogits_aux, void *dX, void *dW_gate, void *dW_up,
                            void *dW_down, void *dWs_gate, void *dWs_up, void *dWs_down,
                            float *dlogits, void *dW_router, void *ws, size_t ws_bytes,
                            mok_stream_t stream);

/* The parameters of mok_sandwich_norm and of its backward pass. */
typedef struct {
  float eps;               /* of both norms, > 0 */
  float res_scale;         /* factor of the residual */
  int32_t res_type;        /* mok_elem of residual, residual_out, h, dres and dresidual */
  int32_t post_type, gate_type, weight_type; /* mok_elem */
  const void *post_weight; /* [d]: the norm after the branch */
  const void *gate;        /* [d], by channel, or NULL (1) */
  const float *token_gate; /* [T], by token, or NULL (1) */
  const void *weight;      /* [d]: the next norm, or NULL (none) */
} mok_sandwich;

/* The norm after a branch, its gate, the scaled residual and the next norm, in one pass per row of
 * d elements, everything in fp32:
 *   h = res_scale residual + token_gate gate post_weight x / sqrt(mean(x^2) + eps),
 *   v = h / sqrt(mean(h^2) + eps) weight.
 *   x[T,d] bf16, residual[T,d] of res_type
 *   -> residual_out[T,d] = h in res_type; with weight: y[T,d] = v in bf16 (NULL to skip) and, with
 *      codes, the MXFP8 form of v as in mok_rms_norm (at least one of the two); with x_codes,
 *      x_scales, h_codes, h_scales (all or none) what the backward pass reads in 8 bits: the MXFP8
 *      forms of x and of h (before its rounding to res_type), codes[T,d] and scales[T,d/32].
 * residual_out may be residual, y may be x.  T >= 0, 0 < d <= 32768, d % 8 == 0 (d % 128 == 0 with
 * codes of any kind); 16-byte aligned pointers (token_gate 4).  There is no status word: a row whose
 * copy does not arrive within the library's limit on waits is NaN in every output, and so may be the
 * rows that its block takes after it.  One launch. */
int mok_sandwich_norm(const mok_sandwich *args, int64_t T, int d, const void *x,
                      const void *residual, void *residual_out, void *y, void *codes, void *scales,
                      int scale_layout, void *x_codes, void *x_scales, void *h_codes,
                      void *h_scales, mok_stream_t stream);

/* Bytes of workspace of mok_sandwich_norm_backward (0 for invalid sizes). */
size_t mok_sandwich_norm_workspace_size(int64_t T, int d);

/* Gradients of mok_sandwich_norm.  With rho1, rho2 the reciprocal roots, xhat = x rho1, hhat = h rho2
 * (recomputed), W = post_weight gate and g = dy weight:
 *   ds = rho2 (g - hhat mean(g hhat)) + dres,  dresidual = res_scale ds,
 *   dx = rho1 token_gate (ds W - xhat mean(ds W xhat)),  dtoken_gate[t] = sum ds W xhat,
 *   dpost_weight = gate A, dgate = post_weight A with A = sum over rows of token_gate ds xhat,
 *   dweight = sum over rows of dy hhat (rows in a fixed order).
 *   dy[T,d] bf16 (with weight, else NULL), dres[T,d] of res_type (the gradient that arrives through
 *   residual_out) or NULL: at least one.  x[T,d] bf16 and h[T,d] of res_type (residual_out; NULL
 *   without weight), or with x_scales and h_scales [T,d/32] their MXFP8 forms as the forward pass
 *   wrote them: the gradients are then those at the values that these hold.
 *   -> dx[T,d] bf16, dresidual[T,d] of res_type, dpost_weight[d], dgate[d] (with gate),
 *      dtoken_gate[T] (with token_gate), dweight[d] (with weight) fp32.
 * dx may be dy, dresidual may be dres.  Sizes and alignment as in mok_sandwich_norm.  Where a wait runs
 * out, the status word of ws (zeroed once) becomes MOK_ERR_TIMEOUT, the row in question and those that
 * its block takes after it are NaN in dx, dresidual and dtoken_gate, and so are the gradients of the
 * weights.  Two launches, the second begins under the first. */
int mok_sandwich_norm_backward(const mok_sandwich *args, int64_t T, int d, const void *dy,
                               const void *dres, const void *x, const void *x_scales, const void *h,
                               const void *h_scales, void *dx, void *dresidual, float *dpost_weight,
                               float *dgate, float *dtoken_gate, float *dweight, void *ws,
                               size_t ws_bytes, mok_stream_t stream);

/* Activations in 8 bits and back, for what a training step keeps between its passes: src[rows,K] of
 * type (mok_elem) -> codes[rows,K] E4M3 and scales[rows,K/32] UE8M0 by the rule of
 * mok_mx_quantize_rows (NaN stays NaN, its block's scale is that of the others), and codes times scales
 * -> dst[rows,K] of type, exact but where it leaves the type's range (a scale byte 255 is NaN);
 * scale_layout: that of the scales read.  rows >= 0, K % 32 == 0 (K % 128 == 0 with scale atoms),
 * rows * K <= 2^40; 16-byte aligned pointers.  One launch each. */
int mok_activation_pack(int64_t rows, int K, const void *src, int type, void *codes, void *scales,
                        mok_stream_t stream);
int mok_activation_unpack(int64_t rows, int K, const void *codes, const void *scales,
                          int scale_layout, void *dst, int type, mok_stream_t stream);

/* What mok_moe_forward saved for the backward pass, in 8 bits: `packed` (mok_packed_saved_size bytes;
 * 0 for dims without a backward pass) receives G and U of the routed rows and of the shared expert as
 * mok_activation_pack gives them; x in expert order, which `saved` also holds for MOK_BF16, is left
 * out.  mok_saved_unpack fills `saved` again, from `packed` and (MOK_BF16) from x[T,d] by inv_pos, for
 * mok_moe_backward with the same routing: `saved` may serve many layers in turn.  At the
 * DeepSeek-V3 training shape (T = 8192, d = 7168, k = 8, F = Fs = 2048) 0.31 GB are kept per layer in
 * place of 1.54 GB (bf16) or 1.21 GB (MXFP8).  One launch; mok_saved_unpack two for MOK_BF16. */
size_t mok_packed_saved_size(const mok_dims *dims);
int mok_saved_pack(const mok_dims *dims, const void *saved, void *packed, mok_stream_t stream);
int mok_saved_unpack(const mok_dims *dims, const void *packed, const void *x,
                     const int32_t *inv_pos, void *saved, mok_stream_t stream);

/* Schedule of the bf16 expert GEMMs of mok_moe_forward (process-wide; default
 * MOK_SCHEDULE_TWO_LAUNCHES):
 *  - MOK_SCHEDULE_TWO_LAUNCHES: gate/up + SwiGLU, then down + router weight, each one persistent
 *    launch whose CTAs take the tiles c, c + grid, c + 2 grid, ...
 *  - MOK_SCHEDULE_FUSED: both phases in one persistent launch.  CTAs claim tiles in order from a
 *    device work counter (every gate/up tile before any down tile) and a down tile first waits,
 *    bounded, until every gate/up tile of its M tile has written its h rows (a readiness counter
 *    per M tile).  This is the fused, device-scheduled form of the layer's kernel (page
 *    "Mixture-of-Kittens: Nhân kernel MoE ...", intro and section "Lập lịch"; page
 *    "Mixture-of-Kittens; MoE megakernel", key points); on one GPU it measured about 1% slower
 *    than two launches at the DeepSeek-V3 shape, hence not the default.
 * Results are bit-identical under both.  Shapes run in CTA pairs (at least 320 routed rows per
 * expert) or with d % 256 != 0 always use two launches.  Returns MOK_OK, or MOK_ERR_INVALID_ARG
 * for another value; *previous (NULL to skip) receives the schedule before the call. */
typedef enum { MOK_SCHEDULE_TWO_LAUNCHES = 0, MOK_SCHEDULE_FUSED = 1 } mok_schedule;
int mok_set_forward_schedule(int schedule, int *previous);

/* Human-readable name of a status code (static string). */
const char *mok_status_string(int status);

/* Synchronises `stream`, copies the device status word of `ws` into *status_out (MOK_OK or a
 * negative code).  The one entry point that waits on the GPU. */
int mok_read_device_status(const void *ws, int *status_out, mok_stream_t stream);

/* Enqueues a reset of the device status word of `ws` to MOK_OK. */
int mok_clear_device_status(void *ws, mok_stream_t stream);

/* Number of kernel launches the last successful call of each entry point enqueued on this
 * host thread (for launch accounting in benchmarks). */
int mok_last_launch_count(void);

/* Pull schedule without a workspace: same inputs as mok_dispatch_index and, for valid inputs,
 * the same outputs, but the scratch it needs (a status word and the per-chunk expert histogram)
 * lives in a device array owned by the library (a 256-byte header plus a 1 MiB histogram), so
 * the call allocates nothing and takes no `ws`.  The pages describe no such variant; it exists
 * for callers that may not allocate device memory when they build the routing (a runtime that
 * reserves all memory at start-up, or code that must not trigger the device-wide
 * synchronisation of cudaMalloc/cudaFree).
 *  - Limit: E * ceil(T / 64) <= 262144 (T <= 65536 tokens at E = 256, T <= 32768 at E = 512);
 *    larger sizes return MOK_ERR_WORKSPACE and enqueue nothing.
 *  - The first call on each device looks up the array's device address (with that device
 *    current) and caches it; make that first call before any stream capture.
 *  - Every device holds the array until the process exits.  All calls on a device share it
 *    and it keeps the last call's contents, so calls whose GPU work overlaps (different
 *    streams, no ordering between them) race; order them on one stream.
 *  - Invalid routing is not reported: an expert index outside [0,E) drops that route
 *    (inv_pos = -1, offsets[E] < T*k), where mok_dispatch_index would also set
 *    MOK_ERR_DEVICE_CHECK in its workspace status word.  Callers that cannot vouch for their
 *    indices can compare offsets[E] with T*k. */
int mok_dispatch_index_noalloc(const mok_dims *dims, const int32_t *topk_idx, const float *topk_w,
                               int32_t *counts, int32_t *offsets, int32_t *sorted_tok,
                               float *sorted_w, int32_t *inv_pos, mok_stream_t stream);

/* Failure-detection self-test: launches one block that waits, with the library's bounded-wait
 * code and a budget of budget_ns (at most 2 s), on a barrier nothing arrives on.  The wait runs
 * out, MOK_ERR_TIMEOUT is recorded in the status word of `ws` and the kernel returns normally,
 * so the context stays usable.  It exercises the error path of the kernels' waits without
 * faulting or hanging the GPU. */
int mok_selftest_bounded_wait(void *ws, int64_t budget_ns, mok_stream_t stream);

/* Failure-detection self-test of the norms on both sides: the next launch of mok_sandwich_norm or of
 * mok_sandwich_norm_backward by the calling host thread leaves out the copies of rows `first` and above
 * and gives every wait for a row budget_ns (at most 2 s), so that the waits for these rows run out, as
 * for copies that do not arrive.  (No effect on rows so wide that they are read without such copies.)
 * first -1 withdraws it. */
int mok_selftest_lost_rows(int64_t first, int64_t budget_ns);

/* Kernel timing for benchmarks.  While enabled on the calling host thread, every entry point
 * records a CUDA event pair around each kernel it launches, on the launch stream (the events do
 * not change what the GPU executes).  enable = 0 stops recording. */
int mok_timing_enable(int enable);

/* Waits for the recorded events, then returns per kernel name (up to max_kernels entries,
 * `names` holds max_kernels * 32 bytes, NUL-terminated) the number of launches and their summed
 * device time in milliseconds; *n_out = entries written.  Clears the record. */
int mok_timing_collect(char *names, int *launches, double *ms, int max_kernels, int *n_out);

#ifdef __cplusplus
}
#endif

#endif /* MOK_H */
