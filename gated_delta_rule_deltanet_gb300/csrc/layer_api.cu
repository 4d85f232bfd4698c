// layer_api.cu -- the C ABI of the layer around the recurrence: argument validation and dispatch.
// Everything here runs on the host before any launch.
#include <math.h>

#include "layer_common.cuh"

namespace kda {
size_t linear_workspace_bytes(const kda_linear_params_t& p, bool bwd);
cudaError_t launch_linear_fwd(const kda_linear_params_t& p, const void* x, const void* w, const float* bias,
                              const void* res, void* y, void* z, void* workspace, int32_t* err,
                              cudaStream_t st);
cudaError_t launch_linear_bwd(const kda_linear_params_t& p, const void* x, const void* w, const void* z,
                              const void* dy, void* dx, void* dw, float* dbias, void* workspace,
                              int32_t* err, cudaStream_t st);
cudaError_t launch_residual_norm(const kda_norm_params_t& p, const void* x, const void* res,
                                 const void* gate, const float* post_w, const float* w, void* h,
                                 void* y, int32_t* err, cudaStream_t st);
size_t residual_norm_bwd_workspace(const kda_norm_params_t& p);
cudaError_t launch_residual_norm_bwd(const kda_norm_params_t& p, const void* x, const void* h,
                                     const void* gate, const float* post_w, const float* w,
                                     const void* dy, const void* dh, void* dx, void* dres,
                                     void* dgate, float* dpost_w, float* dw, void* workspace,
                                     int32_t* err, cudaStream_t st);
cudaError_t launch_gated_norm(const kda_norm_params_t& p, const void* o, const void* gate,
                              const float* w, void* y, cudaStream_t st);
size_t gated_norm_bwd_workspace(const kda_norm_params_t& p);
cudaError_t launch_gated_norm_bwd(const kda_norm_params_t& p, const void* o, const void* gate,
                                  const float* w, const void* dy, void* d_o, void* dgate, float* dw,
                                  void* workspace, cudaStream_t st);
}  // namespace kda

static_assert(sizeof(kda_linear_params_t) == 80, "kda_linear_params_t layout is part of the ABI");
static_assert(sizeof(kda_norm_params_t) == 56, "kda_norm_params_t layout is part of the ABI");

namespace {

bool is_dtype(int32_t d) { return d == KDA_DTYPE_F32 || d == KDA_DTYPE_BF16; }

// aligned to its elements
bool elem_aligned(const void* p, int32_t dt) {
  return reinterpret_cast<uintptr_t>(p) % kda::dtype_bytes(dt) == 0;
}
bool f32_aligned(const void* p) { return elem_aligned(p, KDA_DTYPE_F32); }

kda_status_t to_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// row strides are 0 (dense) or at least the row; strides stay below what a tensor map can say
bool stride_ok(int64_t stride, int64_t cols, int64_t rows) {
  const int64_t s = stride ? stride : cols;
  return s >= cols && s <= (int64_t{1} << 36) && rows <= (int64_t{1} << 60) / s;
}

constexpr uint32_t kLinearFlags =
    KDA_FLAG_CUDA_CORES | KDA_FLAG_UNALIGNED_X | KDA_FLAG_UNALIGNED_W | KDA_FLAG_UNALIGNED_DY;

// A bf16 operand that the tensor cores read: 16-byte aligned unless its flag announces a copy
// (rows that are not a multiple of 8 elements apart are copied anyway).
bool operand_ok(const kda_linear_params_t* p, const void* base, int64_t stride, uint32_t flag) {
  if (!elem_aligned(base, p->dtype)) return false;
  if (p->dtype != KDA_DTYPE_BF16 || (p->flags & (KDA_FLAG_CUDA_CORES | flag)) || stride % 8) return true;
  return reinterpret_cast<uintptr_t>(base) % 16 == 0;
}

kda_status_t check_linear(const kda_linear_params_t* p) {
  if (!p) return KDA_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->in_features < 1 || p->out_features < 1) return KDA_ERR_INVALID_ARG;
  if (!is_dtype(p->dtype) || !is_dtype(p->y_dtype) || !is_dtype(p->residual_dtype) || !is_dtype(p->dw_dtype))
    return KDA_ERR_INVALID_ARG;
  if (p->activation < KDA_ACT_NONE || p->activation > KDA_ACT_SIGMOID) return KDA_ERR_INVALID_ARG;
  if (!isfinite(p->scale) || (p->flags & ~kLinearFlags)) return KDA_ERR_INVALID_ARG;
  const int64_t T = p->tokens, K = p->in_features, N = p->out_features;
  if (!stride_ok(p->x_row_stride, K, T) || !stride_ok(p->w_row_stride, K, N) ||
      !stride_ok(p->y_row_stride, N, T) || !stride_ok(p->residual_row_stride, N, T))
    return KDA_ERR_INVALID_ARG;
  if (T > 0x7fffffffLL || K > (1 << 24) || N > (1 << 24)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws && bytes >= need && reinterpret_cast<uintptr_t>(ws) % 256 == 0);
}

constexpr int kMaxFeatures = 16384, kMaxHead = 1024;

kda_status_t check_norm(const kda_norm_params_t* p, bool gated) {
  if (!p) return KDA_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->features < 1 || (gated && p->num_heads < 1)) return KDA_ERR_INVALID_ARG;
  if (!is_dtype(p->x_dtype) || !is_dtype(p->y_dtype)) return KDA_ERR_INVALID_ARG;
  if (!is_dtype(gated ? p->gate_dtype : p->h_dtype)) return KDA_ERR_INVALID_ARG;
  if (!(p->eps > 0.f) || !isfinite(p->eps)) return KDA_ERR_INVALID_ARG;
  if (gated) {
    if (p->activation != KDA_ACT_SIGMOID && p->activation != KDA_ACT_SILU && p->activation != KDA_ACT_NONE)
      return KDA_ERR_INVALID_ARG;
    if (p->features > kMaxHead) return KDA_ERR_UNSUPPORTED;
    if (p->tokens > 0x7fffffffLL / p->num_heads) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(p->gate_row_stride, static_cast<int64_t>(p->num_heads) * p->features, p->tokens))
      return KDA_ERR_INVALID_ARG;
  } else {
    if (!isfinite(p->scale) || p->y_dtype != p->x_dtype) return KDA_ERR_INVALID_ARG;
    if (p->features > kMaxFeatures || p->tokens > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(p->gate_row_stride, p->features, p->tokens)) return KDA_ERR_INVALID_ARG;
  }
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_linear_workspace_size(const kda_linear_params_t* p, int32_t backward, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const kda_status_t s = check_linear(p);
  if (s != KDA_OK) return s;
  *bytes = kda::linear_workspace_bytes(*p, backward != 0);
  return KDA_OK;
}

kda_status_t kda_linear_fwd(const kda_linear_params_t* p, const void* x, const void* w, const float* bias,
                            const void* residual, void* y, void* pre_act, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const kda_status_t s = check_linear(p);
  if (s != KDA_OK) return s;
  if (p->tokens == 0) return KDA_OK;
  if (!x || !w || !y) return KDA_ERR_INVALID_ARG;
  const int64_t K = p->in_features;
  if (!operand_ok(p, x, p->x_row_stride ? p->x_row_stride : K, KDA_FLAG_UNALIGNED_X) ||
      !operand_ok(p, w, p->w_row_stride ? p->w_row_stride : K, KDA_FLAG_UNALIGNED_W) ||
      !elem_aligned(pre_act, p->dtype) || !elem_aligned(y, p->y_dtype) ||
      !elem_aligned(residual, p->residual_dtype) || !f32_aligned(bias))
    return KDA_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, kda::linear_workspace_bytes(*p, false))) return KDA_ERR_WORKSPACE;
  int32_t* err = kda::layer_error_word();
  if (!err) return KDA_ERR_CUDA;
  return to_status(kda::launch_linear_fwd(*p, x, w, bias, residual, y, pre_act, workspace, err,
                                          static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_linear_bwd(const kda_linear_params_t* p, const void* x, const void* w, const void* pre_act,
                            const void* d_y, void* dx, void* dw, float* dbias, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const kda_status_t s = check_linear(p);
  if (s != KDA_OK) return s;
  if (p->tokens > 0 && (!d_y || (dx && !w) || (dw && !x))) return KDA_ERR_INVALID_ARG;
  if (p->tokens > 0 && p->activation != KDA_ACT_NONE && !pre_act) return KDA_ERR_INVALID_ARG;
  const int64_t K = p->in_features, N = p->out_features;
  if (!operand_ok(p, x, p->x_row_stride ? p->x_row_stride : K, KDA_FLAG_UNALIGNED_X) ||
      !operand_ok(p, w, p->w_row_stride ? p->w_row_stride : K, KDA_FLAG_UNALIGNED_W) ||
      !elem_aligned(pre_act, p->dtype) || !elem_aligned(d_y, p->y_dtype) ||
      (p->activation == KDA_ACT_NONE && p->y_dtype == p->dtype &&
       !operand_ok(p, d_y, p->y_row_stride ? p->y_row_stride : N, KDA_FLAG_UNALIGNED_DY)) ||
      !elem_aligned(dx, p->dtype) || !elem_aligned(dw, p->dw_dtype) ||
      !f32_aligned(dbias))
    return KDA_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, kda::linear_workspace_bytes(*p, true))) return KDA_ERR_WORKSPACE;
  int32_t* err = kda::layer_error_word();
  if (!err) return KDA_ERR_CUDA;
  return to_status(kda::launch_linear_bwd(*p, x, w, pre_act, d_y, dx, dw, dbias, workspace, err,
                                          static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_norm_workspace_size(const kda_norm_params_t* p, int32_t gated, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const kda_status_t s = check_norm(p, gated != 0);
  if (s != KDA_OK) return s;
  *bytes = gated ? kda::gated_norm_bwd_workspace(*p) : kda::residual_norm_bwd_workspace(*p);
  return KDA_OK;
}

kda_status_t kda_residual_norm_fwd(const kda_norm_params_t* p, const void* x, const void* residual,
                                   const void* gate, const float* post_weight, const float* weight,
                                   void* h, void* y, void* stream) {
  const kda_status_t s = check_norm(p, false);
  if (s != KDA_OK) return s;
  if (p->tokens == 0) return KDA_OK;
  if ((weight == nullptr) != (y == nullptr) || (!h && !y) || !x) return KDA_ERR_INVALID_ARG;
  if (!f32_aligned(post_weight) || !f32_aligned(weight) || !elem_aligned(x, p->x_dtype) ||
      !elem_aligned(y, p->x_dtype) || !elem_aligned(residual, p->h_dtype) || !elem_aligned(h, p->h_dtype) ||
      !elem_aligned(gate, p->gate_per_token ? p->x_dtype : KDA_DTYPE_F32))
    return KDA_ERR_INVALID_ARG;
  int32_t* err = kda::layer_error_word();
  if (!err) return KDA_ERR_CUDA;
  return to_status(kda::launch_residual_norm(*p, x, residual, gate, post_weight, weight, h, y, err,
                                             static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_residual_norm_bwd(const kda_norm_params_t* p, const void* x, const void* h,
                                   const void* gate, const float* post_weight, const float* weight,
                                   const void* d_y, const void* d_h, void* dx, void* d_residual,
                                   void* d_gate, float* d_post_weight, float* d_weight,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const kda_status_t s = check_norm(p, false);
  if (s != KDA_OK) return s;
  const bool rows = p->tokens > 0;
  if (rows && ((weight == nullptr) != (d_y == nullptr) || (!d_y && !d_h) || !dx)) return KDA_ERR_INVALID_ARG;
  if (rows && ((d_y && !h) || ((gate || post_weight) && !x))) return KDA_ERR_INVALID_ARG;
  if ((weight && !d_weight) || (post_weight && !d_post_weight) || (gate && !d_gate)) return KDA_ERR_INVALID_ARG;
  const int32_t gdt = p->gate_per_token ? p->x_dtype : KDA_DTYPE_F32;
  if (!f32_aligned(post_weight) || !f32_aligned(weight) || !f32_aligned(d_post_weight) || !f32_aligned(d_weight) ||
      !elem_aligned(x, p->x_dtype) || !elem_aligned(d_y, p->x_dtype) || !elem_aligned(dx, p->x_dtype) ||
      !elem_aligned(h, p->h_dtype) || !elem_aligned(d_h, p->h_dtype) || !elem_aligned(d_residual, p->h_dtype) ||
      !elem_aligned(gate, gdt) || !elem_aligned(d_gate, gdt))
    return KDA_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, kda::residual_norm_bwd_workspace(*p))) return KDA_ERR_WORKSPACE;
  int32_t* err = kda::layer_error_word();
  if (!err) return KDA_ERR_CUDA;
  return to_status(kda::launch_residual_norm_bwd(*p, x, h, gate, post_weight, weight, d_y, d_h, dx,
                                                 d_residual, d_gate, d_post_weight, d_weight, workspace, err,
                                                 static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_gated_norm_fwd(const kda_norm_params_t* p, const void* o, const void* gate,
                                const float* weight, void* y, void* stream) {
  const kda_status_t s = check_norm(p, true);
  if (s != KDA_OK) return s;
  if (!weight || !f32_aligned(weight) || !elem_aligned(o, p->x_dtype) || !elem_aligned(gate, p->gate_dtype) ||
      !elem_aligned(y, p->y_dtype))
    return KDA_ERR_INVALID_ARG;
  if (p->tokens == 0) return KDA_OK;
  if (!o || !gate || !y) return KDA_ERR_INVALID_ARG;
  return to_status(kda::launch_gated_norm(*p, o, gate, weight, y, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_gated_norm_bwd(const kda_norm_params_t* p, const void* o, const void* gate,
                                const float* weight, const void* d_y, void* d_o, void* d_gate,
                                float* d_weight, void* workspace, size_t workspace_bytes, void* stream) {
  const kda_status_t s = check_norm(p, true);
  if (s != KDA_OK) return s;
  if (!weight || !d_weight) return KDA_ERR_INVALID_ARG;
  if (p->tokens > 0 && (!o || !gate || !d_y || !d_o || !d_gate)) return KDA_ERR_INVALID_ARG;
  if (!f32_aligned(weight) || !f32_aligned(d_weight) || !elem_aligned(o, p->x_dtype) ||
      !elem_aligned(d_o, p->x_dtype) || !elem_aligned(gate, p->gate_dtype) ||
      !elem_aligned(d_gate, p->gate_dtype) || !elem_aligned(d_y, p->y_dtype))
    return KDA_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, kda::gated_norm_bwd_workspace(*p))) return KDA_ERR_WORKSPACE;
  return to_status(kda::launch_gated_norm_bwd(*p, o, gate, weight, d_y, d_o, d_gate, d_weight, workspace,
                                              static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
