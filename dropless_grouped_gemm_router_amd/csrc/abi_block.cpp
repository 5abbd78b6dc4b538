// C ABI of the operators around the layer (moe_block.h): argument checks,
// all on the host before anything is enqueued, workspace sizes and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "block.h"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool ok_ptr(const void* p, size_t a = 16) { return p != nullptr && aligned(p, a); }
bool is_float(int t) { return t == MOE_FP32 || t == MOE_BF16; }
size_t bytes_of(int t) { return t == MOE_BF16 ? 2 : 4; }
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
