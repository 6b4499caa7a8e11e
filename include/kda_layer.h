/*
 * kda_layer.h -- C ABI of the operators around the KDA recurrence on GB300
 * (sm_103a): the short causal convolution, the selective state-space scan and
 * the norms before and after a block with its gate and residual scale.
 *
 * The conventions are those of kda.h: the caller owns every buffer, nothing is
 * allocated, tensors are device pointers with the innermost dimension
 * contiguous, calls are asynchronous on `stream`, and errors that the host can
 * see return before anything is launched.  What differs:
 *   - Activations may be column slices of a wider tensor: a token stride (in
 *     elements, 0 = dense) is part of the shape.  Any stride and any base that
 *     is a multiple of the element size is accepted; 16-byte alignment of both
 *     selects the wide loads.
 *   - Parameters (taps, biases, norm weights, decay rates) are float32.
 *   - Where `workspace` is optional (documented per entry point), a NULL skips
 *     the report of errors found on the device.  Otherwise its first word
 *     holds the call's device status after the call (see
 *     kda_read_device_status); its contents on entry do not matter.
 *   - Outputs alias no input unless an entry point says so.
 */
#ifndef KDA_LAYER_H_
#define KDA_LAYER_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Short causal convolution: each channel d of each sequence on its own,
 *
 *     u[t, d] = bias[d] + sum_{j < W} weight[d, j] x[t - (W - 1) + j, d]
 *     y[t, d] = silu(u) or u
 *
 * where x before the sequence's first token is the start state (zeros when
 * NULL).  The state of a sequence is its last W - 1 inputs, oldest first:
 * [N, W-1, D] in `dtype`; a sequence shorter than W - 1 keeps the newest rows
 * of its start state in front.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t B;          /* fixed length: batch size.  Packed: must be 1. */
  int32_t T;          /* tokens per sequence (fixed) or in total (packed), >= 0 */
  int32_t D;          /* channels, 1 .. 2^31 - 1024 */
  int32_t W;          /* taps: 2, 3 or 4 */
  int32_t num_seqs;   /* packed: number of sequences; ignored when cu_seqlens is NULL */
  kda_dtype dtype;    /* x, y and the states (and dy, dx, dinit, dfinal) */
  int32_t silu;       /* nonzero: y = silu(u) */
  int64_t ldx;        /* elements between tokens of x (and dx is dense); 0 = D */
} kda_conv_shape;

/* Prompts.  x [B,T,D] (token stride ldx), weight f32 [D,W], bias f32 [D] or
 * NULL, cu_seqlens device int32 [num_seqs+1] or NULL, init_state [N,W-1,D] or
 * NULL, y [B,T,D] dense, final_state [N,W-1,D] or NULL.  final_state must not
 * alias init_state.  workspace: optional, >= 256 bytes, 256-byte aligned;
 * malformed cu_seqlens are reported there (KDA_ERR_BAD_SEQLENS; every access
 * stays inside the buffers). */
kda_status kda_conv_fwd(const kda_conv_shape* s, const void* x, const float* weight,
                        const float* bias, const int32_t* cu_seqlens, const void* init_state,
                        void* y, void* final_state, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Single tokens: T = 1..8 tokens of each of B sequences, `state` [B,W-1,D]
 * updated in place.  num_commit: device int32 [B] or NULL; as in
 * kda_decode_commit, sequence n keeps the state after its first num_commit[n]
 * tokens (a count outside 0..T is reported as KDA_ERR_INVALID_ARG and leaves
 * its state unchanged).  y [B,T,D], or NULL with num_commit (a pure replay). */
kda_status kda_conv_step(const kda_conv_shape* s, const void* x, const float* weight,
                         const float* bias, const int32_t* num_commit, void* state, void* y,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of sum(y dy) + sum(final_state dfinal) for kda_conv_fwd's inputs.
 * dy [B,T,D] dense, dfinal [N,W-1,D] or NULL; dx [B,T,D] dense, dweight f32
 * [D,W], dbias f32 [D] or NULL, dinit [N,W-1,D] or NULL.  The pre-activations
 * are recomputed.  Sums over tokens are taken in a fixed order (repeatable bit
 * for bit).  workspace: required, kda_conv_bwd_workspace_size(s) bytes. */
size_t kda_conv_bwd_workspace_size(const kda_conv_shape* s);
kda_status kda_conv_bwd(const kda_conv_shape* s, const void* x, const float* weight,
                        const float* bias, const int32_t* cu_seqlens, const void* init_state,
                        const void* dy, const void* dfinal, void* dx, float* dweight,
                        float* dbias, void* dinit, void* workspace, size_t workspace_bytes,
                        void* stream);

/* ------------------------------------------------------------------------
 * Selective state-space scan, one decay per token and head.  Per sequence and
 * head h, whose group is h / (H / G):
 *
 *     delta_t = dt_t, or softplus(dt_t + dt_bias[h]) with dt_softplus
 *     S  <- exp(delta_t A[h]) S + delta_t B_t x_t^T        (ds x dx)
 *     y_t = S^T C_t + D[h] x_t
 *
 * States are float32 [N,H,ds,dx], dx fastest; h0, hT and state are 16-byte aligned.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t B;           /* as kda_conv_shape */
  int32_t T;
  int32_t H;           /* heads, a multiple of G */
  int32_t G;           /* groups that share B_t and C_t */
  int32_t ds, dx;      /* state and head sizes, each 64 or 128 */
  int32_t num_seqs;
  kda_dtype in_dtype;  /* x, dt, B, C */
  kda_dtype out_dtype; /* y */
  int32_t dt_softplus; /* nonzero: delta = softplus(dt + dt_bias) */
  int64_t ldx, lddt, ldb, ldc; /* elements between tokens; 0 = dense (H dx, H, G ds, G ds) */
} kda_scan_shape;

/* Prompts.  x [B,T,H,dx], dt [B,T,H], A f32 [H] (<= 0), Bm and Cm [B,T,G,ds],
 * D f32 [H] or NULL (0), dt_bias f32 [H] or NULL (0; only with dt_softplus),
 * h0 f32 [N,H,ds,dx] or NULL (zeros), y [B,T,H,dx] dense, hT f32 [N,H,ds,dx] or
 * NULL (may alias h0).  workspace: kda_scan_workspace_size(s) bytes, 256-byte
 * aligned.  delta >= 0 is expected; a token whose delta is 0 leaves the state
 * as it is.  Decays of any strength are exact to float32's rounding.  float32
 * inputs are worked on in float32 throughout; with bf16 inputs the tensor-core
 * path rounds one operand of the output's products to 16 bits (2.4e-6 of the
 * outputs' rms; the states keep float32's 24).  That path takes x, Bm, Cm and y on
 * 16-byte boundaries with token strides of x, Bm, Cm that are multiples of 8;
 * others are worked on token by token.  An x, dt,
 * Bm or Cm that is not finite reaches no earlier token and no other sequence; an
 * x makes its own channel's outputs from its token on and final state unspecified
 * (in general NaN, also where the sum would be an infinity).  Zero-length sequences write hT = h0 (or 0).
 * kda_scan_workspace_size: with B = 1 and num_seqs > 0 enough for a packed call
 * and for a fixed-length one; otherwise for a fixed-length one. */
size_t kda_scan_workspace_size(const kda_scan_shape* s);
kda_status kda_scan_fwd(const kda_scan_shape* s, const void* x, const void* dt, const float* A,
                        const void* Bm, const void* Cm, const float* D, const float* dt_bias,
                        const int32_t* cu_seqlens, const float* h0, void* y, float* hT,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Single tokens: T = 1..8 tokens of each of B sequences, `state` f32
 * [B,H,ds,dx] updated in place; num_commit and y as in kda_conv_step.
 * workspace: optional, as in kda_conv_fwd. */
kda_status kda_scan_step(const kda_scan_shape* s, const void* x, const void* dt, const float* A,
                         const void* Bm, const void* Cm, const float* D, const float* dt_bias,
                         const int32_t* num_commit, float* state, void* y, void* workspace,
                         size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Norms before and after a block, its gate and its residual scale.  Per row of
 * d channels (rms(v) = v / sqrt(mean(v^2) + eps)):
 *
 *     z = act(gate)                              (1 without a gate)
 *     m = rms(x) weight z, or with gate_first rms(x z) weight
 *                                                (no norm when weight is NULL)
 *     r = residual + scale res_scale m           (0 and 1 when NULL)
 *     y = rms(r) out_weight                      (only when out_weight is given)
 *
 * Everything is evaluated in float32 and each output rounded once (y comes from
 * the unrounded r).
 * ---------------------------------------------------------------------- */
typedef enum { KDA_GATE_NONE = 0, KDA_GATE_SIGMOID = 1, KDA_GATE_SILU = 2 } kda_gate;

typedef struct {
  int64_t tokens;       /* >= 0 */
  int32_t heads;        /* rows per token, >= 1 */
  int32_t d;            /* channels per row, 1 .. 8192 */
  kda_dtype dtype;      /* x, gate, y, dx, dgate, dy */
  kda_dtype res_dtype;  /* residual, r and their gradients: dtype or KDA_F32 */
  kda_gate gate;
  int32_t gate_first;   /* nonzero: the gate multiplies x before the norm */
  float scale, eps;
  int64_t ldx, ldgate;  /* elements between tokens of x and gate; 0 = heads d */
} kda_norm_shape;

/* x, gate [tokens,heads,d]; weight, res_scale, out_weight f32 [d] or NULL;
 * residual [tokens,heads,d] dense or NULL; r dense or NULL (may alias residual);
 * y dense, given exactly when out_weight is. */
kda_status kda_norm_fwd(const kda_norm_shape* s, const void* x, const float* weight,
                        const void* gate, const void* residual, const float* res_scale,
                        const float* out_weight, void* r, void* y, void* stream);

/* Gradients of sum(r dr) + sum(y dy).  dr may be NULL (0); dy is given exactly
 * when out_weight is, unless dr is given (then a NULL dy is 0).  dx dense;
 * dgate, dresidual dense, dweight, dres_scale, dout_weight f32 [d], each NULL
 * when its operand is absent or its gradient is not wanted.  Sums over rows are
 * taken in a fixed order.  workspace: kda_norm_bwd_workspace_size(s) bytes,
 * 256-byte aligned. */
size_t kda_norm_bwd_workspace_size(const kda_norm_shape* s);
kda_status kda_norm_bwd(const kda_norm_shape* s, const void* x, const float* weight,
                        const void* gate, const void* residual, const float* res_scale,
                        const float* out_weight, const void* dr, const void* dy, void* dx,
                        void* dgate, void* dresidual, float* dweight, float* dres_scale,
                        float* dout_weight, void* workspace, size_t workspace_bytes,
                        void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KDA_LAYER_H_ */
