/*
 * la_token.h -- C ABI of the token-wise operators that stand next to the
 * frame-wise scan of la_scan.h on NVIDIA B200 (sm_100a): the gated delta rule
 * with one update per token (chunked, its backward pass, and one token at a
 * time) and the residual addition with RMSNorm and an 8-bit output (and its
 * backward pass).
 *
 * The conventions of la_scan.h hold (device pointers of the current device,
 * 16-byte aligned, caller-owned buffers, work enqueued on `stream`, argument
 * errors returned before anything is enqueued, no allocation, no
 * synchronisation), except where a paragraph below says otherwise.  No call
 * here uses streams of the library's own, and no result depends on the order of
 * atomics: equal inputs give equal bits, and calls can be captured into CUDA
 * graphs.  Calls that may run at the same time need workspaces of their own.
 *
 * Gated delta rule, per batch item b and value head h, t = 1..T, the state S
 * key-major [D, D] as in la_scan.h:
 *     alpha_t = exp(log_alpha_t),  kh_t = k_scale k_t,  qh_t = q_scale q_t
 *     S_t = alpha_t (I - beta_t kh_t kh_t^T) S_{t-1} + beta_t kh_t v_t^T
 *     o_t = qh_t S_t
 * which is la_scan_gdn's recurrence with frames of one token.  Consecutive
 * value heads share a key head when Hv > Hk: value head h reads q and k of
 * head h / (Hv / Hk).
 *
 * log_alpha = -inf forgets the state (as does any value of -104 or less, whose
 * exponential is 0 in float32).  Positive log_alpha is computed as written and may
 * overflow, in the chunked kernels where the sum of neighbouring ones passes 88.  NaN and infinities spread to later tokens as the recurrence
 * carries them, and in the chunked kernels also to the earlier tokens of the
 * same 64; rows behind a sequence's length never matter.  Forgetting is a product
 * with 0: a state that holds NaN or infinity stays NaN in the value columns that hold
 * it (and in no others), on every path.  To start anew from one, pass zeros or
 * state_in = NULL.
 */
#ifndef LA_TOKEN_H
#define LA_TOKEN_H

#include "la_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Inputs of the gated delta rule.  Strides are in elements, in the order
 * batch, head, token; the D values of a row are contiguous.  Each stride is a
 * multiple of 16 bytes and not negative; strides of 0 (a broadcast input) are
 * allowed.  log_alpha, beta [B, Hv, T] and the states [B, Hv, D, D] are
 * contiguous float32.
 */
typedef struct la_delta {
    const void* q;             /* [B, Hk, T, D] of dtype dt */
    const void* k;             /* [B, Hk, T, D]             */
    const void* v;             /* [B, Hv, T, D]             */
    long long q_stride[3], k_stride[3], v_stride[3];
    const float* log_alpha;    /* [B, Hv, T] */
    const float* beta;         /* [B, Hv, T] */
    const float* state_in;     /* [B, Hv, D, D] or NULL (zeros) */
    const int* lengths;        /* [B] or NULL: sequence b has lengths[b] tokens (taken into
                                  [0, T]); rows behind them are not read                   */
    float k_scale, q_scale;    /* finite */
    int dt;                    /* la_dtype of q, k, v and of o and the gradients */
    int B, Hk, Hv, T, D;       /* Hk divides Hv; D a multiple of 16 in [16, 256] */
} la_delta;

/*
 * Forward pass over T tokens.
 * o         out: [B, Hv, T, D] of dtype dt with strides o_stride.  Rows must not
 *                overlap each other, nor may what lies from o's first to its last
 *                element overlap what lies from an input's first to its last (o between
 *                an input's rows is refused).  Rows behind a sequence's length are left
 *                as they were.
 * state_out out: [B, Hv, D, D] f32, the state after the sequence's last token,
 *                or NULL.  state_out == in->state_in is allowed.
 * T == 0 writes the initial state to state_out and nothing else.
 * workspace: la_delta_workspace_size(0, ...) bytes, 256-byte aligned.
 *
 * Heads up to 128 wide run chunked on tensor cores (chunks of 64 tokens) from about
 * 16 to 40 tokens on, by type and number of heads; shorter calls and wider heads run
 * token by token in float32 (la_delta_plan tells).  With few heads a long sequence is
 * cut into segments that run side by side.
 * The chunked kernels bound every wait on the device; la_query_device_status(workspace,
 * stream) tells whether one ran out (LA_ERR_TIMEOUT), as it does for the scans.
 */
LA_API la_status la_gated_delta_rule(const la_delta* in, void* o, const long long o_stride[3],
                                     float* state_out, void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream);

/*
 * Backward pass: the gradients of a loss whose gradient by o is d_o and by
 * the final state is dstate_out.  The forward pass is computed again from the
 * inputs; nothing of it needs to be kept.
 * d_o        in : [B, Hv, T, D] of dtype dt with strides do_stride (0 allowed);
 *                 rows behind a sequence's length are not read.
 * dstate_out in : [B, Hv, D, D] f32 or NULL (zeros).
 * dq, dk     out: [B, Hk, T, D] of dtype dt, contiguous: summed over the value
 *                 heads that share the key head, in their order.
 * dv         out: [B, Hv, T, D] of dtype dt, contiguous.
 * dlog_alpha, dbeta out: [B, Hv, T] f32.  dlog_alpha is exactly 0 where there is no
 *                 state to scale: at a token that forgets it, and at the first one
 *                 without in->state_in.
 * dstate_in  out: [B, Hv, D, D] f32 or NULL; may be dstate_out.
 * Gradients of rows behind a sequence's length are 0.
 * D <= 128, else LA_ERR_UNSUPPORTED.
 * workspace: la_delta_workspace_size(1, ...) bytes, 256-byte aligned.
 */
LA_API la_status la_gated_delta_rule_backward(const la_delta* in, const void* d_o,
                                              const long long do_stride[3],
                                              const float* dstate_out, void* dq, void* dk,
                                              void* dv, float* dlog_alpha, float* dbeta,
                                              float* dstate_in, void* workspace,
                                              size_t workspace_bytes, cudaStream_t stream);

/*
 * One token for every sequence (decoding): in->T is 1, the token strides are
 * not used, state_out is required and may be in->state_in (in place).  A
 * sequence of length 0 keeps its state and its row of o.  No workspace.
 */
LA_API la_status la_gated_delta_step(const la_delta* in, void* o, const long long o_stride[3],
                                     float* state_out, cudaStream_t stream);

/* Workspace bytes of la_gated_delta_rule (backward == 0) or of its backward
 * pass (backward != 0); 0 for an unsupported shape. */
LA_API size_t la_delta_workspace_size(int backward, la_dtype dt, int B, int Hk, int Hv, int T,
                                      int D);

/* Name of the kernels that a call of this shape runs ("delta_chunked",
 * "delta_recurrent") and their number, or NULL for an unsupported shape. */
LA_API const char* la_delta_plan(int backward, la_dtype dt, int B, int Hk, int Hv, int T, int D,
                                 int* kernels);

/*
 * Residual addition, RMSNorm and an output in e4m3 with scales, per row of N:
 *     h = round_dt(x + residual)                   (h = x without a residual)
 *     y = h / sqrt(mean(h^2) + eps) * weight
 *     scale = max |y| / 448 over each group of columns (1 where that is 0 in float32)
 *     y8 = e4m3(y / scale)
 * h is normalised as it is stored, so that the backward pass sees the same h.  The
 * quotient is y times the float32 reciprocal of scale (off by 1.5 roundings of float32
 * in place of half of one) and is rounded to nearest even, so that a value within those
 * of the middle between two e4m3 numbers may go to the other one.
 * group = 128: a scale for each 128 columns (the last group may be shorter);
 * group = 0: one scale for the row.  A row that holds NaN or infinity gives
 * NaN in what it reaches.  The squares are summed in float32: a row whose sum of
 * squares is above 3.4e38 gives zeros, and eps = 0 needs one of at least 1e-37.
 * x, residual in : [rows, N] of dtype dt; residual may be NULL.
 * weight      in : [N] f32.
 * h           out: [rows, N] of dtype dt or NULL; may be x or residual.
 * y8          out: [rows, N] e4m3.   scale out: [rows, ceil(N / group)] f32.
 * rows >= 0; N a multiple of 16 in [16, 16384], else LA_ERR_UNSUPPORTED.
 */
LA_API la_status la_add_rms_norm_fp8(const void* x, const void* residual, const float* weight,
                                     void* h, void* y8, float* scale, la_dtype dt,
                                     long long rows, int N, int group, float eps,
                                     cudaStream_t stream);

/*
 * Backward pass of the norm and the addition, the 8-bit rounding passed
 * straight through: with r = 1 / sqrt(mean(h^2) + eps), t = dy * weight,
 *     dx = r t - h r^3 mean(t h) + dh          (the gradient of x and of residual)
 *     dweight = sum over rows of dy h r        (in a fixed order)
 * dy, h  in : [rows, N] of dtype dt (h as the forward pass stored it).
 * dh     in : [rows, N] of dtype dt or NULL: the gradient that h gets from elsewhere.
 * dx     out: [rows, N] of dtype dt; may be dy or dh.    dweight out: [N] f32 or NULL.
 * workspace: la_norm_workspace_size(rows, N) bytes, 256-byte aligned; not
 * used when dweight is NULL.
 */
LA_API la_status la_add_rms_norm_backward(const void* dy, const void* h, const float* weight,
                                          const void* dh, void* dx, float* dweight, la_dtype dt,
                                          long long rows, int N, float eps, void* workspace,
                                          size_t workspace_bytes, cudaStream_t stream);
LA_API size_t la_norm_workspace_size(long long rows, int N);

#ifdef __cplusplus
}
#endif
#endif /* LA_TOKEN_H */
