/*
 * moe_block.h - C ABI of libmoe's operators around the MoE layer (moe.h):
 * the layer norm in front of it, the dense gated feed-forward block that
 * stands in for it in a model's dense layers, matrix products with weights
 * held in 8-bit integers, dense or grouped by the layer's routing, dense
 * products with bias, activation and residual, the norms, gate and residual
 * between two blocks, and the balance loss of the layer's router.
 *
 * Conventions as in moe.h: device pointers unless stated otherwise, memory
 * and workspaces owned by the caller, nothing allocated or retained, work
 * enqueued on `stream` without synchronising, every check on the host
 * before anything is enqueued, moe_status codes, deterministic results (no
 * floating-point atomics), no state between calls: calls may run
 * concurrently when their workspaces and outputs differ. Tensors have to be
 * on the current device. Matrices are dense row-major and 16-byte aligned
 * except where a row stride is given; workspaces are 256-byte aligned.
 * Outputs may not overlap inputs unless an entry says so.
 */
#ifndef MOE_BLOCK_H_
#define MOE_BLOCK_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ layer norm */

/*
 * y[t] = (x[t] - mean[t]) * rstd[t] * weight + bias,  with
 * mean[t] = sum_j x[t,j] / width, rstd[t] = 1 / sqrt(var[t] + eps) and
 * var[t] = sum_j (x[t,j] - mean[t])^2 / width.
 *
 * dtype is the storage type of x, y, grad_out and grad_x; weight, bias,
 * mean, rstd and the gradients of weight and bias are fp32 in both modes.
 * Sums are fp32. Rows may lie apart: ld_* is the number of elements between
 * rows (0: width), and these four arrays need only the alignment of their
 * elements. y may be x, and grad_x may be grad_out or x, with equal strides.
 *
 * Supported (else MOE_ERR_UNSUPPORTED): width <= 16384, rows < 2^31.
 */
typedef struct {
  int64_t rows;
  int32_t width;
  int32_t dtype; /* moe_dtype */
  float eps;     /* finite, >= 0 */
  int64_t ld_x, ld_y, ld_grad_out, ld_grad_x;
} moe_norm;

/*
 * Forward. weight and bias may be NULL (ones, zeros). mean and rstd
 * [rows], both or neither NULL, are what moe_layer_norm_bwd reads.
 * rows == 0 is a successful no-op.
 */
int moe_layer_norm(const moe_norm* n, const void* x, const float* weight, const float* bias,
                   void* y, float* mean, float* rstd, void* stream);

/* Workspace bytes (host) of moe_layer_norm_bwd; 0 for an invalid problem. */
size_t moe_layer_norm_workspace_bytes(const moe_norm* n);

/*
 * Backward of L = sum(y * grad_out), with g = grad_out * weight and
 * xh = (x - mean) rstd:
 *   grad_x      = rstd (g - mean_j(g) - xh mean_j(g xh))
 *   grad_weight = sum_t grad_out xh,  grad_bias = sum_t grad_out
 * grad_weight and grad_bias (each may be NULL: not wanted) are fully
 * overwritten; the sums over rows run in one fixed order. With rows == 0
 * they are zeroed. weight may be NULL (ones); eps is not read.
 */
int moe_layer_norm_bwd(const moe_norm* n, const void* x, const float* weight, const float* mean,
                       const float* rstd, const void* grad_out, void* grad_x, float* grad_weight,
                       float* grad_bias, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------- gated feed-forward block */

/* Activation of the gate branch. */
typedef enum {
  MOE_ACT_SILU = 0,      /* a / (1 + exp(-a)) */
  MOE_ACT_GELU = 1,      /* a Phi(a), Phi the normal distribution function */
  MOE_ACT_GELU_TANH = 2, /* a (1 + tanh(sqrt(2/pi) (a + 0.044715 a^3))) / 2 */
  MOE_ACT_RELU = 3,      /* max(a, 0); slope 0 at 0 */
  MOE_ACT_NONE = 4       /* a; moe_linear only */
} moe_act;

/*
 *   out = (act(x W_gate) * (x W_up)) W_down
 * the expert FFN of moe.h (FFN_e) as a block of its own: x [tokens, d_model],
 * W_gate and W_up [d_model, d_hidden], W_down [d_hidden, d_model], out
 * [tokens, d_model], all in dtype; accumulation is fp32. The hidden values
 * act(x W_gate) * (x W_up) are rounded to dtype for the second product (as
 * the routed experts' are), and in the backward pass so are the gradients of
 * the two pre-activations. In bf16 and up to 16 tokens the second product
 * takes the hidden values as a sum of two bf16 numbers instead (2^-17); the
 * backward's h is rounded there too.
 *
 * Supported (else MOE_ERR_UNSUPPORTED): d_model and d_hidden up to 32768
 * (any value), tokens * max(d_model, 2 * d_hidden) < 2^36.
 */
typedef struct {
  int64_t tokens;
  int32_t d_model;
  int32_t d_hidden;
  int32_t dtype;      /* moe_dtype */
  int32_t act;        /* moe_act */
  int32_t grad_dtype; /* moe_dtype of the three weight gradients: MOE_FP32, or
                         dtype (rounded once from fp32 sums) */
} moe_ffn;

/* Workspace bytes (host) of moe_gated_ffn without `saved` (training = 0), or
 * of that, moe_gated_ffn with `saved` and moe_gated_ffn_bwd (training = 1); 0
 * for an invalid problem. */
size_t moe_gated_ffn_workspace_bytes(const moe_ffn* f, int training);

/* Bytes (host) of the buffer that moe_gated_ffn fills for
 * moe_gated_ffn_bwd: h in dtype, and act(a) and b act'(a), in fp32 or, in
 * bf16, rounded to 20 bits (2^-12). */
size_t moe_gated_ffn_saved_bytes(const moe_ffn* f);

/* Forward. saved: NULL for inference, or moe_gated_ffn_saved_bytes(f) bytes
 * (256-byte aligned). tokens == 0 is a successful no-op. */
int moe_gated_ffn(const moe_ffn* f, const void* x, const void* w_gate, const void* w_up,
                  const void* w_down, void* saved, void* out, void* workspace,
                  size_t workspace_bytes, void* stream);

/*
 * Backward of L = sum(out * grad_out), with a = x W_gate, b = x W_up and
 * h = act(a) b:
 *   dh = grad_out W_down^T, da = dh b act'(a), db = dh act(a)
 *   grad_x = da W_gate^T + db W_up^T
 *   grad_gate = x^T da, grad_up = x^T db, grad_down = h^T grad_out
 * Everything is fully overwritten; with tokens == 0 the weight gradients are
 * zeroed. saved is read only.
 */
int moe_gated_ffn_bwd(const moe_ffn* f, const void* x, const void* w_gate, const void* w_up,
                      const void* w_down, const void* saved, const void* grad_out, void* grad_x,
                      void* grad_gate, void* grad_up, void* grad_down, void* workspace,
                      size_t workspace_bytes, void* stream);

/* ------------------------------------------- products in 8-bit integers */

/* Type of a linear_i8 input that is already quantised. */
enum { MOE_I8 = 2 };

/* Bytes between rows of 8-bit matrices (host): width rounded up to a
 * multiple of 128; the bytes past width are zero. 0 for width < 1. */
int64_t moe_i8_pitch(int32_t width);

/*
 * Rows of x [rows, width] (dtype fp32 or bf16; ld_x elements between rows, 0:
 * width) in 8 bits with a scale each:
 *   scale[t] = max_j |x[t,j]| * (1 / 127),  q[t,j] = rint(x[t,j] / scale[t])
 * in fp32, 1 / 127 a number of fp32 and the division rounded to nearest, rint
 * to nearest even, clamped to [-127, 127]: what torch makes on this device of
 * scale = x.abs().amax(1) / 127, q = round(x / scale). A zero row has scale 0
 * and q 0; a row with an infinity or a NaN has scale NaN and q 0, so that
 * whatever is made of it is NaN. q is [rows, moe_i8_pitch(width)], its padding
 * zeroed. It is the layout of activations and, with a row for each output
 * channel, of weights.
 * Supported: rows < 2^31, width <= 65536.
 */
int moe_quantize_rows(int64_t rows, int32_t width, int32_t dtype, const void* x, int64_t ld_x,
                      int8_t* q, float* scale, void* stream);

/*
 * Weights in the layer's layout, w [groups, width, outputs] (dtype), to
 * 8-bit rows: q [groups, outputs, moe_i8_pitch(width)], scale [groups,
 * outputs], each output channel a row quantised as above. For gated
 * weights, quantise gate and up into one array by calling it once for each
 * with q_rows, the number of rows between groups in q and scale (0:
 * outputs), set to 2 * d_hidden. Supported: width <= 65536, outputs <= 65536.
 */
int moe_quantize_weight(int32_t groups, int32_t width, int32_t outputs, int32_t dtype,
                        const void* w, int64_t q_rows, int8_t* q, float* scale, void* stream);

/*
 * y[r, n] = x_scale[i] * w_scale[g, n] * sum_k xq[i, k] wq[g, n, k] (+ bias[n])
 * over the integers (the sum is exact), y in dtype.
 *
 * Dense (groups == 1, no routing): r = i = 0 .. tokens-1.
 * Routed (a moe_routing): r = sorted row j of expert g's segment
 *   [expert_offsets[g], expert_offsets[g+1]), input row i = perm[j] / top_k
 *   when gather is set (the layer's tokens), else i = j (rows already in
 *   expert order, tokens * top_k of them). With capacity > 0 an expert's
 *   rows past its first `capacity` are left as they are in y.
 * gated: the `outputs` weight rows of a group are d gate rows and d up rows
 *   (outputs = 2 d), and y[r, n] = SiLU(gate) * up has d columns; bias is
 *   not supported with it.
 *
 * x_dtype MOE_I8: x is xq [rows, moe_i8_pitch(inputs)] with x_scale [rows];
 * MOE_FP32 or MOE_BF16: x is [rows, inputs], quantised within the call as
 * moe_quantize_rows does, and x_scale is ignored.
 *
 * Supported (else MOE_ERR_UNSUPPORTED): inputs and outputs up to 65536 (any
 * value; outputs even when gated), groups <= 64, tokens * top_k < 2^31 and
 * fewer than 2^24 output tiles of 64 x 64.
 */
typedef struct {
  int64_t tokens;
  int32_t inputs;
  int32_t outputs;
  int32_t x_dtype;
  int32_t dtype; /* moe_dtype of y */
  int32_t groups;
  int32_t top_k;    /* routed: token-slots per token; 1 when dense */
  int32_t gather;   /* routed: 1 = x rows are tokens, 0 = x rows are sorted */
  int32_t gated;
  int32_t capacity; /* routed: as moe_problem.capacity */
} moe_i8_linear;

/* Workspace bytes (host); 0 for an invalid problem. */
size_t moe_linear_i8_workspace_bytes(const moe_i8_linear* l);

/* bias: NULL or fp32 [outputs]. r: NULL when dense; of a routing only
 * expert_offsets and (gather) perm are read. tokens == 0 is a no-op. */
int moe_linear_i8(const moe_i8_linear* l, const void* x, const float* x_scale, const int8_t* wq,
                  const float* w_scale, const float* bias, const moe_routing* r, void* y,
                  void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------- product with bias, activation and residual */

/*
 *   y = act(x W + bias) + residual
 * x [tokens, inputs], W [inputs, outputs], residual and y [tokens, outputs] in
 * dtype, bias fp32 [outputs]; sums are fp32 and y is rounded once. In bf16 the
 * slopes act'(a) are kept in 20 bits for the backward pass (off by at most
 * 6.4e-7), where from 17 tokens on da is rounded to bf16 for its two products.
 *
 * Supported (else MOE_ERR_UNSUPPORTED): inputs and outputs up to 65536 (any
 * value), tokens < 2^31, tokens * max(inputs, outputs) < 2^36.
 */
typedef struct {
  int64_t tokens;
  int32_t inputs;
  int32_t outputs;
  int32_t dtype;      /* moe_dtype */
  int32_t act;        /* moe_act */
  int32_t grad_dtype; /* moe_dtype of the weights' gradient: MOE_FP32, or dtype
                         (rounded once from fp32 sums) */
} moe_linear;

/* Workspace bytes (host) of moe_linear_fwd (training = 0), or of it and
 * moe_linear_bwd (training = 1); 0 for an invalid problem. */
size_t moe_linear_workspace_bytes(const moe_linear* l, int training);

/* Bytes (host) of the buffer that moe_linear_fwd fills for moe_linear_bwd: the
 * slopes act'(a). 0 with MOE_ACT_NONE, which keeps nothing, and for an
 * invalid problem. */
size_t moe_linear_saved_bytes(const moe_linear* l);

/* Forward. bias and residual may be NULL. saved: NULL for inference (or with
 * MOE_ACT_NONE, where it is not touched), else moe_linear_saved_bytes(l) bytes
 * (256-byte aligned). tokens == 0 is a successful no-op. A y that shares memory
 * with x, W or the residual is refused (MOE_ERR_INVALID), as are gradients that
 * share it with each other or with an input of moe_linear_bwd. */
int moe_linear_fwd(const moe_linear* l, const void* x, const void* w, const float* bias,
                   const void* residual, void* saved, void* y, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * Backward of L = sum(y * grad_out), with a = x W + bias and
 * da = grad_out act'(a):
 *   grad_x = da W^T, grad_w = x^T da, grad_bias = sum_t da (fp32; NULL: not
 *   wanted); the residual's gradient is grad_out itself.
 * Everything is fully overwritten; with tokens == 0 the gradients of the
 * parameters are zeroed. saved is read only, and not at all with MOE_ACT_NONE.
 */
int moe_linear_bwd(const moe_linear* l, const void* x, const void* w, const void* saved,
                   const void* grad_out, void* grad_x, void* grad_w, float* grad_bias,
                   void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------- between two blocks */

typedef enum {
  MOE_NORM_LAYER = 0, /* (x - mean) / sqrt(var + eps), as moe_layer_norm */
  MOE_NORM_RMS = 1    /* x / sqrt(mean_j(x^2) + eps) */
} moe_norm_kind;

/*
 * What lies between two blocks of a residual stream: the norm after the block
 * whose output is z, a gate, the residual, and the norm before the next block:
 *   u = norm(z) post_weight + post_bias   (post = 0: u = z)
 *   out = scale res + gate u
 *   y = norm(out) pre_weight + pre_bias   (pre = 0: not computed)
 * Everything between z, res and out, y is fp32 and rounded once; y is made of
 * the out that is not rounded. dtype is the storage type of the matrices,
 * parameters and their gradients are fp32 in both modes.
 *
 * Rows may lie apart: ld_* is the number of elements between rows (0: width),
 * and the matrices need only the alignment of their elements. out and y may be
 * z or res, and grad_z and grad_res may be z, res, grad_out or grad_y, each
 * another one and with equal strides (MOE_ERR_INVALID where these differ).
 *
 * Supported (else MOE_ERR_UNSUPPORTED): width <= 16384, rows < 2^31.
 */
typedef struct {
  int64_t rows;
  int32_t width;
  int32_t dtype; /* moe_dtype */
  int32_t kind;  /* moe_norm_kind, of both norms */
  int32_t post;  /* 1: the norm after the block is there */
  int32_t pre;   /* 1: the norm before the next block is there */
  float eps;     /* finite, >= 0 */
  float scale;   /* of the residual; finite */
  int64_t ld_z, ld_res, ld_out, ld_y, ld_grad_out, ld_grad_y, ld_grad_z, ld_grad_res;
} moe_residual_norm;

/* Parameters [width] (device, fp32, read only); each may be NULL (weights and
 * gate: ones, biases: zeros). */
typedef struct {
  const float* post_weight;
  const float* post_bias;
  const float* gate;
  const float* pre_weight;
  const float* pre_bias;
} moe_norm_params;

/* Their gradients [width] (device, fp32, fully overwritten); each may be NULL
 * (not wanted). */
typedef struct {
  float* post_weight;
  float* post_bias;
  float* gate;
  float* pre_weight;
  float* pre_bias;
} moe_norm_grads;

/*
 * Forward. y is NULL exactly where pre is 0. stats: NULL, or [4, rows] fp32
 * (mean and 1 / deviation of z, then of out) for moe_residual_norm_bwd.
 * rows == 0 is a successful no-op.
 */
int moe_residual_norm_fwd(const moe_residual_norm* n, const void* z, const void* res,
                          const moe_norm_params* params, void* out, void* y, float* stats,
                          void* stream);

/* Workspace bytes (host) of moe_residual_norm_bwd; 0 for an invalid problem. */
size_t moe_residual_norm_workspace_bytes(const moe_residual_norm* n);

/*
 * Backward of L = sum(out * grad_out) + sum(y * grad_y); grad_out may be NULL
 * (no such term), grad_y is NULL exactly where pre is 0. z and res are the
 * forward's, unchanged. The sums over rows run in one fixed order. Gradients of
 * a norm that is not there are zeros. With rows == 0 the parameters' gradients
 * are zeroed. eps is not read.
 */
int moe_residual_norm_bwd(const moe_residual_norm* n, const void* z, const void* res,
                          const moe_norm_params* params, const float* stats, const void* grad_out,
                          const void* grad_y, void* grad_z, void* grad_res,
                          const moe_norm_grads* grads, void* workspace, size_t workspace_bytes,
                          void* stream);

/* ------------------------------------------------- balance of the router */

/*
 * Load-balance loss and z loss of the layer's router over a batch, with the
 * loads of the experts. With l = x w_router (fp32 as the layer's router, but
 * not in its order of additions), p = softmax(l) over all experts, n the
 * number of tokens that the mask keeps and sums over those tokens:
 *   counts[e]    = number of their token-slots that topk_idx gives to expert e
 *   mean_prob[e] = sum_t p[t,e] / n
 *   loss[1] = experts sum_e counts[e] / (n top_k) mean_prob[e]
 *   loss[2] = sum_t logsumexp_e(l[t])^2 / n
 *   loss[0] = balance loss[1] + z loss[2]
 * With n == 0 all of them are zeros. Tokens that the mask leaves out may hold
 * anything, NaN included. x, grad_x and saved are aligned as usual, the other
 * arrays need only the alignment of their elements.
 *
 * Supported (else MOE_ERR_UNSUPPORTED): what moe_problem supports of tokens,
 * experts (<= 64), top_k and d_model (a multiple of 128, at most 8192).
 */
typedef struct {
  int64_t tokens;
  int32_t experts;
  int32_t top_k;
  int32_t d_model;
  int32_t dtype;  /* moe_dtype of x and grad_x */
  float balance;  /* coefficients of the two losses; finite */
  float z;
} moe_balance;

/* Workspace bytes (host) of moe_balance_loss and moe_balance_loss_bwd; 0 for an
 * invalid problem. */
size_t moe_balance_workspace_bytes(const moe_balance* b);

/* Bytes (host) of the buffer that moe_balance_loss fills for
 * moe_balance_loss_bwd: the gradient of loss[0] by the logits in fp32, and the
 * router's matrix, in bf16 as sums of two bf16 numbers (2^-17; grad_x, with the
 * logits' gradient in two as well, is 2^-16 off before it is rounded). 0 for an invalid
 * problem. */
size_t moe_balance_saved_bytes(const moe_balance* b);

/*
 * Forward. topk_idx [tokens, top_k] as moe_route leaves it (entries that are
 * no expert are not counted); mask: NULL (all tokens) or a byte a token, 0:
 * left out. counts [experts] int32, mean_prob [experts] and loss [3] fp32 are
 * fully overwritten. saved: NULL, or moe_balance_saved_bytes(b) bytes
 * (256-byte aligned).
 */
int moe_balance_loss(const moe_balance* b, const void* x, const float* w_router,
                     const int32_t* topk_idx, const uint8_t* mask, int32_t* counts,
                     float* mean_prob, float* loss, void* saved, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * Backward of grad_loss[0] loss[0] with the counts held fixed (grad_loss: one
 * fp32 number on the device, or NULL: 1), for the x and mask of the forward call
 * that filled saved, which holds the w_router of that call:
 *   dl[t,e] = p[t,e] (balance experts (f_e - sum_j f_j p[t,j]) + 2 z logsumexp_t) / n,
 *   f = counts / (n top_k), 0 for tokens that the mask leaves out
 *   grad_x = dl w_router^T, grad_router = x^T dl
 * add = 0: both are fully overwritten (with tokens == 0 grad_router is
 * zeroed); add = 1: both are added to what is there, the layer's own
 * gradients for instance (moe_bwd), rounded once.
 */
int moe_balance_loss_bwd(const moe_balance* b, const void* x, const uint8_t* mask,
                         const void* saved, const float* grad_loss, int add, void* grad_x,
                         float* grad_router, void* workspace, size_t workspace_bytes,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H_ */
