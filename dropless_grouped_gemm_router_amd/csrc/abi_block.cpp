// C ABI of the operators around the layer (moe_block.h): argument checks,
// all on the host before anything is enqueued, workspace sizes and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "block.h"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool ok_ptr(const void* p, size_t a = 16) { return p != nullptr && aligned(p, a); }
bool is_float(int t) { return t == MOE_FP32 || t == MOE_BF16; }
size_t bytes_of(int t) { return t == MOE_BF16 ? 2 : 4; }
// Whether two arrays of na and nb bytes share any (a null one shares none).
bool share(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return a && b && p < q + nb && q < p + na;
}
int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

constexpr int64_t kRowLimit = int64_t{1} << 31;

int check_norm(const moe_norm* n) {
  if (!n || n->rows < 0 || n->width < 1 || !is_float(n->dtype)) return MOE_ERR_INVALID;
  if (!std::isfinite(n->eps) || n->eps < 0.0f) return MOE_ERR_INVALID;
  for (int64_t ld : {n->ld_x, n->ld_y, n->ld_grad_out, n->ld_grad_x})
    if (ld != 0 && ld < n->width) return MOE_ERR_INVALID;
  if (n->width > 16384 || n->rows >= kRowLimit) return MOE_ERR_UNSUPPORTED;
  for (int64_t ld : {n->ld_x, n->ld_y, n->ld_grad_out, n->ld_grad_x})
    if (ld >= kRowLimit) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_ffn(const moe_ffn* f) {
  if (!f || f->tokens < 0 || f->d_model < 1 || f->d_hidden < 1 || !is_float(f->dtype))
    return MOE_ERR_INVALID;
  if (f->act < MOE_ACT_SILU || f->act > MOE_ACT_RELU) return MOE_ERR_INVALID;
  if (f->grad_dtype != MOE_FP32 && f->grad_dtype != f->dtype) return MOE_ERR_INVALID;
  if (f->d_model > 32768 || f->d_hidden > 32768 || f->tokens >= kRowLimit) return MOE_ERR_UNSUPPORTED;
  const int64_t wide = f->d_model > 2 * f->d_hidden ? f->d_model : 2 * f->d_hidden;
  // a launch stays under 2^32 threads: 256 for 64 x 64 outputs
  if (f->tokens >= (int64_t{1} << 36) / wide) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_i8(const moe_i8_linear* l) {
  if (!l || l->tokens < 0 || l->inputs < 1 || l->outputs < 1 || l->groups < 1 || l->top_k < 1 ||
      l->capacity < 0)
    return MOE_ERR_INVALID;
  if (!is_float(l->dtype) || (!is_float(l->x_dtype) && l->x_dtype != MOE_I8)) return MOE_ERR_INVALID;
  if ((l->gather != 0 && l->gather != 1) || (l->gated != 0 && l->gated != 1)) return MOE_ERR_INVALID;
  if (l->gated && l->outputs % 2) return MOE_ERR_INVALID;
  if (l->top_k > l->groups) return MOE_ERR_INVALID;
  if (l->groups > 64 || l->inputs > 65536 || l->outputs > 65536) return MOE_ERR_UNSUPPORTED;
  // token-slots, and the threads of a launch (256 for 64 x 64 outputs)
  if (l->tokens > (kRowLimit - 1) / l->top_k) return MOE_ERR_UNSUPPORTED;
  const int64_t tiles = (l->tokens * l->top_k + 63) / 64 + l->groups;
  if (tiles >= (int64_t{1} << 24) / ((l->outputs + 63) / 64)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_linear(const moe_linear* l) {
  if (!l || l->tokens < 0 || l->inputs < 1 || l->outputs < 1 || !is_float(l->dtype)) return MOE_ERR_INVALID;
  if (l->act < MOE_ACT_SILU || l->act > MOE_ACT_NONE) return MOE_ERR_INVALID;
  if (l->grad_dtype != MOE_FP32 && l->grad_dtype != l->dtype) return MOE_ERR_INVALID;
  if (l->inputs > 65536 || l->outputs > 65536 || l->tokens >= kRowLimit) return MOE_ERR_UNSUPPORTED;
  const int64_t wide = l->inputs > l->outputs ? l->inputs : l->outputs;
  // a launch stays under 2^32 threads: 256 for 64 x 64 outputs
  if (l->tokens >= (int64_t{1} << 36) / wide) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_residual_norm(const moe_residual_norm* n) {
  if (!n || n->rows < 0 || n->width < 1 || !is_float(n->dtype)) return MOE_ERR_INVALID;
  if (n->kind != MOE_NORM_LAYER && n->kind != MOE_NORM_RMS) return MOE_ERR_INVALID;
  if ((n->post != 0 && n->post != 1) || (n->pre != 0 && n->pre != 1)) return MOE_ERR_INVALID;
  if (!std::isfinite(n->eps) || n->eps < 0.0f || !std::isfinite(n->scale)) return MOE_ERR_INVALID;
  if (n->width > 16384 || n->rows >= kRowLimit) return MOE_ERR_UNSUPPORTED;
  for (int64_t ld : {n->ld_z, n->ld_res, n->ld_out, n->ld_y, n->ld_grad_out, n->ld_grad_y, n->ld_grad_z,
                     n->ld_grad_res}) {
    if (ld != 0 && ld < n->width) return MOE_ERR_INVALID;
    if (ld >= kRowLimit) return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

// Whether an output lies over an input with other rows than the input's: a row
// would be stored over one that is still to be read.
struct Rows {
  const void* p;
  int64_t ld;
};
bool askew(const moe_residual_norm& n, std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
  auto ld = [&](int64_t v) { return v ? v : static_cast<int64_t>(n.width); };
  for (const Rows& o : outs)
    for (const Rows& i : ins)
      if (o.p && o.p == i.p && n.rows > 1 && ld(o.ld) != ld(i.ld)) return true;
  return false;
}

bool ok_params(const moe_norm_params* p) {
  return p && aligned(p->post_weight, 4) && aligned(p->post_bias, 4) && aligned(p->gate, 4) &&
         aligned(p->pre_weight, 4) && aligned(p->pre_bias, 4);
}

int check_balance(const moe_balance* b) {
  if (!b || b->tokens < 0 || b->experts < 1 || b->top_k < 1 || b->top_k > b->experts || b->d_model < 1 ||
      !is_float(b->dtype) || !std::isfinite(b->balance) || !std::isfinite(b->z))
    return MOE_ERR_INVALID;
  if (b->experts > 64 || b->d_model % 128 || b->d_model > 8192) return MOE_ERR_UNSUPPORTED;
  if (b->tokens > (kRowLimit - 1) / b->top_k) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

MOE_EXPORT int moe_layer_norm(const moe_norm* n, const void* x, const float* weight,
                              const float* bias, void* y, float* mean, float* rstd, void* stream) {
  const int st = check_norm(n);
  if (st != MOE_OK) return st;
  if (n->rows == 0) return MOE_OK;
  const size_t e = bytes_of(n->dtype);
  if (!ok_ptr(x, e) || !ok_ptr(y, e) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || (mean == nullptr) != (rstd == nullptr))
    return MOE_ERR_INVALID;
  return hip_status(moe::launch_norm(*n, x, weight, bias, y, mean, rstd, as_stream(stream)));
}

MOE_EXPORT size_t moe_layer_norm_workspace_bytes(const moe_norm* n) {
  return check_norm(n) == MOE_OK ? moe::norm_ws_bytes(*n) : 0;
}

MOE_EXPORT int moe_layer_norm_bwd(const moe_norm* n, const void* x, const float* weight,
                                  const float* mean, const float* rstd, const void* grad_out,
                                  void* grad_x, float* grad_weight, float* grad_bias,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_norm(n);
  if (st != MOE_OK) return st;
  if (!aligned(grad_weight, 4) || !aligned(grad_bias, 4)) return MOE_ERR_INVALID;
  if (n->rows > 0) {
    const size_t e = bytes_of(n->dtype);
    if (!ok_ptr(x, e) || !aligned(weight, 4) || !ok_ptr(mean, 4) || !ok_ptr(rstd, 4) ||
        !ok_ptr(grad_out, e) || !ok_ptr(grad_x, e))
      return MOE_ERR_INVALID;
    if (grad_weight || grad_bias) {
      if (!ok_ptr(workspace, 256)) return MOE_ERR_INVALID;
      if (workspace_bytes < moe::norm_ws_bytes(*n)) return MOE_ERR_WORKSPACE;
    }
  }
  return hip_status(moe::launch_norm_bwd(*n, x, weight, mean, rstd, grad_out, grad_x, grad_weight,
                                         grad_bias, workspace, as_stream(stream)));
}

MOE_EXPORT size_t moe_gated_ffn_workspace_bytes(const moe_ffn* f, int training) {
  return check_ffn(f) == MOE_OK ? moe::ffn_block_ws_bytes(*f, training != 0) : 0;
}

MOE_EXPORT size_t moe_gated_ffn_saved_bytes(const moe_ffn* f) {
  return check_ffn(f) == MOE_OK ? moe::ffn_block_saved_bytes(*f) : 0;
}

MOE_EXPORT int moe_gated_ffn(const moe_ffn* f, const void* x, const void* w_gate, const void* w_up,
                             const void* w_down, void* saved, void* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const int st = check_ffn(f);
  if (st != MOE_OK) return st;
  if (f->tokens == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(w_gate) || !ok_ptr(w_up) || !ok_ptr(w_down) || !ok_ptr(out) ||
      !aligned(saved, 256) || !ok_ptr(workspace, 256))
    return MOE_ERR_INVALID;
  if (workspace_bytes < moe::ffn_block_ws_bytes(*f, saved != nullptr)) return MOE_ERR_WORKSPACE;
  return hip_status(moe::launch_ffn_block(*f, x, w_gate, w_up, w_down, saved, out, workspace,
                                          as_stream(stream)));
}

MOE_EXPORT int moe_gated_ffn_bwd(const moe_ffn* f, const void* x, const void* w_gate,
                                 const void* w_up, const void* w_down, const void* saved,
                                 const void* grad_out, void* grad_x, void* grad_gate,
                                 void* grad_up, void* grad_down, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const int st = check_ffn(f);
  if (st != MOE_OK) return st;
  if (!ok_ptr(grad_gate) || !ok_ptr(grad_up) || !ok_ptr(grad_down)) return MOE_ERR_INVALID;
  if (f->tokens > 0) {
    if (!ok_ptr(x) || !ok_ptr(w_gate) || !ok_ptr(w_up) || !ok_ptr(w_down) || !ok_ptr(saved, 256) ||
        !ok_ptr(grad_out) || !ok_ptr(grad_x) || !ok_ptr(workspace, 256))
      return MOE_ERR_INVALID;
    if (workspace_bytes < moe::ffn_block_ws_bytes(*f, true)) return MOE_ERR_WORKSPACE;
  }
  return hip_status(moe::launch_ffn_block_bwd(*f, x, w_gate, w_up, w_down, saved, grad_out, grad_x,
                                              grad_gate, grad_up, grad_down, workspace,
                                              as_stream(stream)));
}

MOE_EXPORT int64_t moe_i8_pitch(int32_t width) { return width < 1 ? 0 : moe::i8_pitch(width); }

MOE_EXPORT int moe_quantize_rows(int64_t rows, int32_t width, int32_t dtype, const void* x,
                                 int64_t ld_x, int8_t* q, float* scale, void* stream) {
  if (rows < 0 || width < 1 || !is_float(dtype) || (ld_x != 0 && ld_x < width)) return MOE_ERR_INVALID;
  if (rows >= kRowLimit || width > 65536 || ld_x >= kRowLimit) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(x, bytes_of(dtype)) || !ok_ptr(q) || !ok_ptr(scale, 4)) return MOE_ERR_INVALID;
  return hip_status(moe::launch_quantize_rows(rows, width, dtype, x, ld_x, q, scale, as_stream(stream)));
}

MOE_EXPORT int moe_quantize_weight(int32_t groups, int32_t width, int32_t outputs, int32_t dtype,
                                   const void* w, int64_t q_rows, int8_t* q, float* scale,
                                   void* stream) {
  if (groups < 1 || width < 1 || outputs < 1 || !is_float(dtype) ||
      (q_rows != 0 && q_rows < outputs))
    return MOE_ERR_INVALID;
  if (groups > 64 || width > 65536 || outputs > 65536 || q_rows > 2 * 65536) return MOE_ERR_UNSUPPORTED;
  if (!ok_ptr(w) || !ok_ptr(q) || !ok_ptr(scale, 4)) return MOE_ERR_INVALID;
  return hip_status(moe::launch_quantize_weight(groups, width, outputs, dtype, w, q_rows, q, scale,
                                                as_stream(stream)));
}

MOE_EXPORT size_t moe_linear_i8_workspace_bytes(const moe_i8_linear* l) {
  return check_i8(l) == MOE_OK ? moe::linear_i8_ws_bytes(*l) : 0;
}

MOE_EXPORT int moe_linear_i8(const moe_i8_linear* l, const void* x, const float* x_scale,
                             const int8_t* wq, const float* w_scale, const float* bias,
                             const moe_routing* r, void* y, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const int st = check_i8(l);
  if (st != MOE_OK) return st;
  if (l->gated && bias) return MOE_ERR_UNSUPPORTED;
  if (!r && (l->groups > 1 || l->gather || l->capacity)) return MOE_ERR_INVALID;
  if (l->tokens == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(wq) || !ok_ptr(w_scale, 4) || !aligned(bias, 4) || !ok_ptr(y))
    return MOE_ERR_INVALID;
  if (l->x_dtype == MOE_I8 && !ok_ptr(x_scale, 4)) return MOE_ERR_INVALID;
  if (r && (!ok_ptr(r->expert_offsets, 4) || (l->gather && !ok_ptr(r->perm, 4)))) return MOE_ERR_INVALID;
  if (l->x_dtype != MOE_I8) {
    if (!ok_ptr(workspace, 256)) return MOE_ERR_INVALID;
    if (workspace_bytes < moe::linear_i8_ws_bytes(*l)) return MOE_ERR_WORKSPACE;
  }
  return hip_status(moe::launch_linear_i8(*l, x, x_scale, wq, w_scale, bias, r, y, workspace,
                                          as_stream(stream)));
}

MOE_EXPORT size_t moe_linear_workspace_bytes(const moe_linear* l, int training) {
  return check_linear(l) == MOE_OK ? moe::linear_ws_bytes(*l, training != 0) : 0;
}

MOE_EXPORT size_t moe_linear_saved_bytes(const moe_linear* l) {
  return check_linear(l) == MOE_OK ? moe::linear_saved_bytes(*l) : 0;
}

MOE_EXPORT int moe_linear_fwd(const moe_linear* l, const void* x, const void* w, const float* bias,
                              const void* residual, void* saved, void* y, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const int st = check_linear(l);
  if (st != MOE_OK) return st;
  if (l->tokens == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(w) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(saved, 256) ||
      !ok_ptr(y) || !ok_ptr(workspace, 256))
    return MOE_ERR_INVALID;
  if (workspace_bytes < moe::linear_ws_bytes(*l, false)) return MOE_ERR_WORKSPACE;
  // y is stored tile by tile while others still read
  const size_t e = bytes_of(l->dtype), nx = l->tokens * l->inputs * e, ny = l->tokens * l->outputs * e;
  const size_t nw = static_cast<size_t>(l->inputs) * l->outputs * e;
  if (share(y, ny, residual, ny) || share(y, ny, x, nx) || share(y, ny, w, nw)) return MOE_ERR_INVALID;
  return hip_status(moe::launch_linear(*l, x, w, bias, residual, saved, y, workspace, as_stream(stream)));
}

MOE_EXPORT int moe_linear_bwd(const moe_linear* l, const void* x, const void* w, const void* saved,
                              const void* grad_out, void* grad_x, void* grad_w, float* grad_bias,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_linear(l);
  if (st != MOE_OK) return st;
  if (!ok_ptr(grad_w) || !aligned(grad_bias, 16)) return MOE_ERR_INVALID;
  if (l->tokens > 0) {
    if (!ok_ptr(x) || !ok_ptr(w) || !ok_ptr(grad_out) || !ok_ptr(grad_x) || !ok_ptr(workspace, 256))
      return MOE_ERR_INVALID;
    if (l->act != MOE_ACT_NONE && !ok_ptr(saved, 256)) return MOE_ERR_INVALID;
    if (workspace_bytes < moe::linear_ws_bytes(*l, true)) return MOE_ERR_WORKSPACE;
    const size_t e = bytes_of(l->dtype), nx = l->tokens * l->inputs * e, ny = l->tokens * l->outputs * e;
    const size_t cells = static_cast<size_t>(l->inputs) * l->outputs, nw = cells * e, ng = cells * bytes_of(l->grad_dtype);
    if (share(grad_x, nx, x, nx) || share(grad_x, nx, w, nw) || share(grad_x, nx, grad_out, ny) ||
        share(grad_w, ng, x, nx) || share(grad_w, ng, w, nw) || share(grad_w, ng, grad_out, ny) ||
        share(grad_x, nx, grad_w, ng))
      return MOE_ERR_INVALID;
  }
  return hip_status(moe::launch_linear_bwd(*l, x, w, saved, grad_out, grad_x, grad_w, grad_bias, workspace,
                                           as_stream(stream)));
}

MOE_EXPORT int moe_residual_norm_fwd(const moe_residual_norm* n, const void* z, const void* res,
                                     const moe_norm_params* params, void* out, void* y, float* stats,
                                     void* stream) {
  const int st = check_residual_norm(n);
  if (st != MOE_OK) return st;
  if (!ok_params(params)) return MOE_ERR_INVALID;
  if (n->rows == 0) return MOE_OK;
  const size_t e = bytes_of(n->dtype);
  if (!ok_ptr(z, e) || !ok_ptr(res, e) || !ok_ptr(out, e) || !aligned(y, e) || !aligned(stats, 4) ||
      (y != nullptr) != (n->pre == 1) || out == y)
    return MOE_ERR_INVALID;
  if (askew(*n, {{out, n->ld_out}, {y, n->ld_y}}, {{z, n->ld_z}, {res, n->ld_res}})) return MOE_ERR_INVALID;
  return hip_status(moe::launch_residual_norm(*n, z, res, *params, out, y, stats, as_stream(stream)));
}

MOE_EXPORT size_t moe_residual_norm_workspace_bytes(const moe_residual_norm* n) {
  return check_residual_norm(n) == MOE_OK ? moe::residual_norm_ws_bytes(*n) : 0;
}

MOE_EXPORT int moe_residual_norm_bwd(const moe_residual_norm* n, const void* z, const void* res,
                                     const moe_norm_params* params, const float* stats, const void* grad_out,
                                     const void* grad_y, void* grad_z, void* grad_res,
                                     const moe_norm_grads* grads, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  const int st = check_residual_norm(n);
  if (st != MOE_OK) return st;
  if (!ok_params(params) || !grads) return MOE_ERR_INVALID;
  bool any = false;
  for (const float* g : {grads->post_weight, grads->post_bias, grads->gate, grads->pre_weight, grads->pre_bias}) {
    if (!aligned(g, 4)) return MOE_ERR_INVALID;
    any = any || g;
  }
  if (n->rows > 0) {
    const size_t e = bytes_of(n->dtype);
    if (!ok_ptr(z, e) || !ok_ptr(res, e) || !ok_ptr(stats, 4) || !aligned(grad_out, e) || !aligned(grad_y, e) ||
        !ok_ptr(grad_z, e) || !ok_ptr(grad_res, e) || grad_z == grad_res)
      return MOE_ERR_INVALID;
    if ((grad_y != nullptr) != (n->pre == 1)) return MOE_ERR_INVALID;
    if (askew(*n, {{grad_z, n->ld_grad_z}, {grad_res, n->ld_grad_res}},
              {{z, n->ld_z}, {res, n->ld_res}, {grad_out, n->ld_grad_out}, {grad_y, n->ld_grad_y}}))
      return MOE_ERR_INVALID;
    if (any) {
      if (!ok_ptr(workspace, 256)) return MOE_ERR_INVALID;
      if (workspace_bytes < moe::residual_norm_ws_bytes(*n)) return MOE_ERR_WORKSPACE;
    }
  }
  return hip_status(moe::launch_residual_norm_bwd(*n, z, res, *params, stats, grad_out, grad_y, grad_z, grad_res,
                                                  *grads, workspace, as_stream(stream)));
}

MOE_EXPORT size_t moe_balance_workspace_bytes(const moe_balance* b) {
  return check_balance(b) == MOE_OK ? moe::balance_ws_bytes(*b) : 0;
}

MOE_EXPORT size_t moe_balance_saved_bytes(const moe_balance* b) {
  return check_balance(b) == MOE_OK ? moe::balance_saved_bytes(*b) : 0;
}

MOE_EXPORT int moe_balance_loss(const moe_balance* b, const void* x, const float* w_router,
                                const int32_t* topk_idx, const uint8_t* mask, int32_t* counts,
                                float* mean_prob, float* loss, void* saved, void* workspace,
                                size_t workspace_bytes, void* stream) {
  const int st = check_balance(b);
  if (st != MOE_OK) return st;
  if (!ok_ptr(counts, 4) || !ok_ptr(mean_prob, 4) || !ok_ptr(loss, 4) || !aligned(saved, 256) || !ok_ptr(workspace, 256) ||
      !ok_ptr(w_router, 4))
    return MOE_ERR_INVALID;
  if (b->tokens > 0 && (!ok_ptr(x) || !ok_ptr(topk_idx, 4))) return MOE_ERR_INVALID;
  if (workspace_bytes < moe::balance_ws_bytes(*b)) return MOE_ERR_WORKSPACE;
  return hip_status(moe::launch_balance(*b, x, w_router, topk_idx, mask, counts, mean_prob, loss, saved, workspace,
                                        as_stream(stream)));
}

MOE_EXPORT int moe_balance_loss_bwd(const moe_balance* b, const void* x, const uint8_t* mask,
                                    const void* saved, const float* grad_loss, int add, void* grad_x,
                                    float* grad_router, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  const int st = check_balance(b);
  if (st != MOE_OK) return st;
  if (add != 0 && add != 1) return MOE_ERR_INVALID;
  if (!ok_ptr(grad_router, 4) || !aligned(grad_loss, 4)) return MOE_ERR_INVALID;
  if (b->tokens > 0) {
    if (!ok_ptr(x) || !ok_ptr(saved, 256) || !ok_ptr(grad_x) || !ok_ptr(workspace, 256))
      return MOE_ERR_INVALID;
    if (workspace_bytes < moe::balance_ws_bytes(*b)) return MOE_ERR_WORKSPACE;
  }
  return hip_status(moe::launch_balance_bwd(*b, x, mask, saved, grad_loss, add != 0, grad_x, grad_router,
                                            workspace, as_stream(stream)));
}
