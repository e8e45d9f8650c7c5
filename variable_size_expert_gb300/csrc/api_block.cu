// C ABI of the layers around the experts (declared in include/mgg.h):
// argument checks and launches for layer norm, the expert choice and the
// dense products.
#include <math.h>

#include "../../include/mgg.h"
#include "common.cuh"
#include "internal.h"

using namespace mgg;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool float_type(mgg_dtype d) { return d == MGG_BF16 || d == MGG_F32; }
size_t size_of(mgg_dtype d) { return d == MGG_F32 ? 4 : 2; }
mgg_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MGG_OK : MGG_ERR_CUDA; }
mgg_status zero(void* p, size_t bytes, cudaStream_t st) {
  return p ? from_cuda(cudaMemsetAsync(p, 0, bytes, st)) : MGG_OK;
}

}  // namespace

extern "C" {

mgg_status mgg_layer_norm_forward(const void* x, mgg_dtype x_dtype, int64_t ldx, const void* weight,
                                  const void* bias, mgg_dtype w_dtype, int T, int K, float eps,
                                  void* y, mgg_dtype y_dtype, float* mean, float* rstd,
                                  void* stream) {
  const NvtxRange nvtx("mgg_layer_norm_forward");
  if (T < 0 || K < 1 || ldx < K || !(eps >= 0.f) || !isfinite(eps)) return MGG_ERR_INVALID_ARG;
  if (!float_type(x_dtype) || !float_type(w_dtype) || !float_type(y_dtype)) return MGG_ERR_DTYPE;
  if (T == 0) return MGG_OK;
  if (!x || !weight || !y || !mean || !rstd) return MGG_ERR_INVALID_ARG;
  if (!aligned(x, size_of(x_dtype)) || !aligned(weight, size_of(w_dtype)) ||
      !aligned(bias, size_of(w_dtype)) || !aligned(y, size_of(y_dtype)) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return MGG_ERR_ALIGNMENT;
  const mgg_status s = check_arch();
  if (s != MGG_OK) return s;
  return from_cuda(launch_norm_fwd(x, x_dtype == MGG_F32, ldx, weight, bias, w_dtype == MGG_F32, T,
                                   K, eps, y, y_dtype == MGG_F32, mean, rstd,
                                   static_cast<cudaStream_t>(stream)));
}

mgg_status mgg_layer_norm_backward(const void* dy, mgg_dtype y_dtype, const void* x,
                                   mgg_dtype x_dtype, int64_t ldx, const void* weight,
                                   mgg_dtype w_dtype, const float* mean, const float* rstd, int T,
                                   int K, void* dx, void* dweight, void* dbias, void* ws,
                                   size_t ws_bytes, void* stream) {
  const NvtxRange nvtx("mgg_layer_norm_backward");
  if (T < 0 || K < 1 || ldx < K || !dweight) return MGG_ERR_INVALID_ARG;
  if (!float_type(x_dtype) || !float_type(w_dtype) || !float_type(y_dtype)) return MGG_ERR_DTYPE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t wb = size_of(w_dtype);
  if (!aligned(dweight, wb) || !aligned(dbias, wb)) return MGG_ERR_ALIGNMENT;
  if (T == 0) {
    const mgg_status s = check_arch();
    if (s != MGG_OK) return s;
    const mgg_status z = zero(dweight, K * wb, st);
    return z != MGG_OK ? z : zero(dbias, K * wb, st);
  }
  if (!dy || !x || !weight || !mean || !rstd || !dx) return MGG_ERR_INVALID_ARG;
  if (!aligned(dy, size_of(y_dtype)) || !aligned(x, size_of(x_dtype)) || !aligned(weight, wb) ||
      !aligned(dx, size_of(x_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4))
    return MGG_ERR_ALIGNMENT;
  mgg_status s = check_arch();
  if (s != MGG_OK) return s;
  if (!ws || !aligned(ws, 256) ||
      ws_bytes < mgg_workspace_bytes(MGG_OP_LAYER_NORM_BACKWARD, T, 0, 0, 0, K, x_dtype))
    return MGG_ERR_WORKSPACE;
  return from_cuda(launch_norm_bwd(dy, y_dtype == MGG_F32, x, x_dtype == MGG_F32, ldx, weight,
                                   w_dtype == MGG_F32, mean, rstd, T, K, dx, dweight, dbias,
                                   static_cast<float*>(ws), st));
}

static mgg_status check_select(mgg_dtype dtype, int64_t ldl, int T, int E, int k,
                               mgg_scoring scoring, float scale) {
  if (T < 0 || E < 1 || E > kMaxExperts || k < 1 || k > MGG_MAX_TOPK || k > E || ldl < E)
    return MGG_ERR_INVALID_ARG;
  if (scoring != MGG_SCORE_SOFTMAX && scoring != MGG_SCORE_SIGMOID) return MGG_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return MGG_ERR_INVALID_ARG;
  if (!float_type(dtype)) return MGG_ERR_DTYPE;
  return MGG_OK;
}

mgg_status mgg_select_experts(const void* logits, mgg_dtype dtype, int64_t ldl, int T, int E, int k,
                              mgg_scoring scoring, const float* bias, int groups, int topk_groups,
                              int renormalize, float scale, int32_t* expert_ids,
                              float* topk_weights, void* stream) {
  const NvtxRange nvtx("mgg_select_experts");
  const int group_score = scoring & (MGG_GROUP_BEST | MGG_GROUP_TWO_BEST);
  scoring = static_cast<mgg_scoring>(scoring & ~(MGG_GROUP_BEST | MGG_GROUP_TWO_BEST));
  mgg_status s = check_select(dtype, ldl, T, E, k, scoring, scale);
  if (s != MGG_OK) return s;
  if (group_score == (MGG_GROUP_BEST | MGG_GROUP_TWO_BEST)) return MGG_ERR_INVALID_ARG;
  const bool two_best =
      groups > 1 && (group_score ? group_score == MGG_GROUP_TWO_BEST : scoring == MGG_SCORE_SIGMOID);
  if (groups < 1 || groups > 32 || E % groups != 0 || topk_groups < 1 || topk_groups > groups ||
      k > topk_groups * (E / groups))
    return MGG_ERR_INVALID_ARG;
  if (T == 0) return MGG_OK;
  if (!logits || !expert_ids || !topk_weights) return MGG_ERR_INVALID_ARG;
  if (!aligned(logits, size_of(dtype)) || !aligned(bias, 4) || !aligned(expert_ids, 4) ||
      !aligned(topk_weights, 4))
    return MGG_ERR_ALIGNMENT;
  s = check_arch();
  if (s != MGG_OK) return s;
  return from_cuda(launch_select(logits, dtype == MGG_F32, ldl, T, E, k,
                                 scoring == MGG_SCORE_SOFTMAX, bias, groups, topk_groups, two_best,
                                 renormalize != 0, scale, expert_ids, topk_weights,
                                 static_cast<cudaStream_t>(stream)));
}

mgg_status mgg_select_experts_backward(const float* dtopk, const void* logits, mgg_dtype dtype,
                                       int64_t ldl, const int32_t* expert_ids,
                                       const float* topk_weights, int T, int E, int k,
                                       mgg_scoring scoring, int renormalize, float scale,
                                       void* dlogits, int32_t* dev_status, void* stream) {
  const NvtxRange nvtx("mgg_select_experts_backward");
  mgg_status s = check_select(dtype, ldl, T, E, k, scoring, scale);
  if (s != MGG_OK) return s;
  if (T == 0) return MGG_OK;
  if (!dtopk || !logits || !expert_ids || !topk_weights || !dlogits || !dev_status)
    return MGG_ERR_INVALID_ARG;
  if (!aligned(logits, size_of(dtype)) || !aligned(dlogits, size_of(dtype)) || !aligned(dtopk, 4) ||
      !aligned(expert_ids, 4) || !aligned(topk_weights, 4))
    return MGG_ERR_ALIGNMENT;
  s = check_arch();
  if (s != MGG_OK) return s;
  return from_cuda(launch_select_bwd(dtopk, logits, dtype == MGG_F32, ldl, expert_ids,
                                     topk_weights, T, E, k, scoring == MGG_SCORE_SOFTMAX,
                                     renormalize != 0, scale, dlogits, dev_status,
                                     static_cast<cudaStream_t>(stream)));
}

static bool known_act(mgg_activation a) {
  return a == MGG_ACT_NONE || a == MGG_ACT_RELU || a == MGG_ACT_SILU || a == MGG_ACT_GELU;
}

mgg_status mgg_linear_forward(const void* x, int64_t ldx, const void* W, const void* bias,
                              mgg_dtype bias_dtype, const void* residual, mgg_dtype residual_dtype,
                              int64_t ldr, int T, int K, int N, mgg_activation activation,
                              void* out, mgg_dtype out_dtype, void* pre, int32_t* dev_status,
                              void* stream) {
  const NvtxRange nvtx("mgg_linear_forward");
  if (T < 0 || K < 1 || N < 1 || ldx < K || (residual && ldr < N) || !known_act(activation))
    return MGG_ERR_INVALID_ARG;
  if (!float_type(out_dtype) || (bias && !float_type(bias_dtype)) ||
      (residual && !float_type(residual_dtype)))
    return MGG_ERR_DTYPE;
  if (K % 8 != 0 || ldx % 8 != 0) return MGG_ERR_ALIGNMENT;
  if (T == 0) return MGG_OK;
  if (!x || !W || !out || !dev_status) return MGG_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(out, size_of(out_dtype)) ||
      !aligned(bias, size_of(bias_dtype)) || !aligned(residual, size_of(residual_dtype)) ||
      !aligned(pre, 2))
    return MGG_ERR_ALIGNMENT;
  const mgg_status s = check_arch();
  if (s != MGG_OK) return s;
  DenseParams p{};
  DenseProduct& d = p.pr[0];
  d.M = T;
  d.N = N;
  d.Kc = K;
  d.out = out;
  d.out_f32 = out_dtype == MGG_F32;
  d.epilogue = bias || residual || pre || activation != MGG_ACT_NONE;
  p.bias = bias;
  p.bias_f32 = bias_dtype == MGG_F32;
  p.bias_vec = bias && aligned(bias, 16);
  p.act = activation;
  p.residual = residual;
  p.res_f32 = residual_dtype == MGG_F32;
  p.ldr = ldr;
  p.res_vec = residual && aligned(residual, 16) && ldr % (p.res_f32 ? 4 : 8) == 0;
  p.pre = pre;
  p.dev_status = dev_status;
  p.wait_limit = wait_limit();
  return from_cuda(launch_dense_forward(p, DenseOperand{x, T, K, ldx}, DenseOperand{W, N, K, K},
                                        static_cast<cudaStream_t>(stream)));
}

mgg_status mgg_linear_backward(const void* dy, mgg_dtype dy_dtype, int64_t lddy, const void* x,
                               int64_t ldx, const void* W, const void* pre,
                               mgg_activation activation, int T, int K, int N, void* dx, void* dW,
                               void* dbias, mgg_dtype bias_dtype, int32_t* dev_status, void* ws,
                               size_t ws_bytes, void* stream) {
  const NvtxRange nvtx("mgg_linear_backward");
  if (T < 0 || K < 1 || N < 1 || ldx < K || lddy < N || !known_act(activation))
    return MGG_ERR_INVALID_ARG;
  if (!float_type(dy_dtype) || (dbias && !float_type(bias_dtype))) return MGG_ERR_DTYPE;
  if (K % 8 != 0 || ldx % 8 != 0) return MGG_ERR_ALIGNMENT;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!aligned(dW, 16) || !aligned(dbias, size_of(bias_dtype))) return MGG_ERR_ALIGNMENT;
  if (T == 0) {
    const mgg_status s = check_arch();
    if (s != MGG_OK) return s;
    const mgg_status z = zero(dW, static_cast<size_t>(N) * K * 2, st);
    return z != MGG_OK ? z : zero(dbias, static_cast<size_t>(N) * size_of(bias_dtype), st);
  }
  if (!dy || !x || !W || !dev_status || (activation != MGG_ACT_NONE && !pre))
    return MGG_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(dx, 16) || !aligned(dy, size_of(dy_dtype)) ||
      !aligned(pre, 2))
    return MGG_ERR_ALIGNMENT;
  mgg_status s = check_arch();
  if (s != MGG_OK) return s;
  if (!ws || !aligned(ws, 256) || ws_bytes < dense_bwd_ws_bytes(T, N)) return MGG_ERR_WORKSPACE;
  DenseBackward a{};
  a.dy = dy;
  a.dy_f32 = dy_dtype == MGG_F32;
  a.lddy = lddy;
  a.x = x;
  a.ldx = ldx;
  a.W = W;
  a.pre = pre;
  a.act = activation;
  a.T = T;
  a.K = K;
  a.N = N;
  a.dx = dx;
  a.dW = dW;
  a.db = dbias;
  a.db_f32 = bias_dtype == MGG_F32;
  a.dev_status = dev_status;
  a.wait_limit = wait_limit();
  return from_cuda(launch_dense_backward(a, ws, st));
}

}  // extern "C"
