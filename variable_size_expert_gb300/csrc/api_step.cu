// C ABI of what a training step needs around the blocks (declared in
// include/mgg.h): argument checks and launches for the balance loss, the cross
// entropy over a vocabulary and the AdamW step.
#include <math.h>

#include <algorithm>

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
  return p && bytes ? from_cuda(cudaMemsetAsync(p, 0, bytes, st)) : MGG_OK;
}

mgg_status check_balance(mgg_dtype dtype, int64_t ldl, int T, int E, int sequences,
                         mgg_scoring scoring) {
  if (T < 0 || T > kMostRows || E < 1 || E > kMaxExperts || ldl < E || sequences < 1 || T % sequences != 0)
    return MGG_ERR_INVALID_ARG;
  if (scoring != MGG_SCORE_SOFTMAX && scoring != MGG_SCORE_SIGMOID) return MGG_ERR_INVALID_ARG;
  return float_type(dtype) ? MGG_OK : MGG_ERR_DTYPE;
}

mgg_status check_vocab(int64_t ldx, int T, int K, int V, float z_loss) {
  if (T < 0 || K < 1 || V < 1 || ldx < K || !(z_loss >= 0.f) || !isfinite(z_loss) ||
      std::max({T, K, V}) > kMostRows)
    return MGG_ERR_INVALID_ARG;
  return K % 8 == 0 && ldx % 8 == 0 ? MGG_OK : MGG_ERR_ALIGNMENT;
}

}  // namespace

extern "C" {

mgg_status mgg_balance_loss(const void* logits, mgg_dtype dtype, int64_t ldl,
                            const int32_t* expert_ids, const uint8_t* mask, int T, int E, int k,
                            int sequences, mgg_scoring scoring, float* loss, int32_t* counts,
                            float* slope, int32_t* dev_status, void* ws, size_t ws_bytes,
                            void* stream) {
  const NvtxRange nvtx("mgg_balance_loss");
  mgg_status s = check_balance(dtype, ldl, T, E, sequences, scoring);
  if (s != MGG_OK) return s;
  if (k < 1 || k > MGG_MAX_TOPK || !loss || !counts || !slope) return MGG_ERR_INVALID_ARG;
  if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(slope, 4)) return MGG_ERR_ALIGNMENT;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    s = check_arch();
    const size_t all = static_cast<size_t>(sequences) * E * 4;
    if (s == MGG_OK) s = zero(loss, 4, st);
    if (s == MGG_OK) s = zero(counts, all, st);
    return s == MGG_OK ? zero(slope, all, st) : s;
  }
  if (!logits || !expert_ids || !dev_status) return MGG_ERR_INVALID_ARG;
  if (!aligned(logits, size_of(dtype)) || !aligned(expert_ids, 4)) return MGG_ERR_ALIGNMENT;
  s = check_arch();
  if (s != MGG_OK) return s;
  const size_t need = balance_ws_bytes(T, E, sequences);
  if (need && (!ws || !aligned(ws, 256) || ws_bytes < need)) return MGG_ERR_WORKSPACE;
  BalanceArgs a{};
  a.logits = logits, a.f32 = dtype == MGG_F32, a.ldl = ldl, a.ids = expert_ids, a.mask = mask;
  a.T = T, a.E = E, a.k = k, a.sequences = sequences, a.softmax = scoring == MGG_SCORE_SOFTMAX;
  a.loss = loss, a.counts = counts, a.slope = slope, a.dev_status = dev_status;
  return from_cuda(launch_balance(a, ws, st));
}

mgg_status mgg_balance_loss_backward(const float* dloss, const void* logits, mgg_dtype dtype,
                                     int64_t ldl, const float* slope, const uint8_t* mask, int T,
                                     int E, int sequences, mgg_scoring scoring, void* dlogits,
                                     void* stream) {
  const NvtxRange nvtx("mgg_balance_loss_backward");
  mgg_status s = check_balance(dtype, ldl, T, E, sequences, scoring);
  if (s != MGG_OK) return s;
  if (T == 0) return MGG_OK;
  if (!dloss || !logits || !slope || !dlogits) return MGG_ERR_INVALID_ARG;
  if (!aligned(logits, size_of(dtype)) || !aligned(dlogits, size_of(dtype)) || !aligned(slope, 4) ||
      !aligned(dloss, 4))
    return MGG_ERR_ALIGNMENT;
  s = check_arch();
  if (s != MGG_OK) return s;
  BalanceArgs a{};
  a.logits = logits, a.f32 = dtype == MGG_F32, a.ldl = ldl, a.mask = mask;
  a.T = T, a.E = E, a.k = 1, a.sequences = sequences, a.softmax = scoring == MGG_SCORE_SOFTMAX;
  a.slope = const_cast<float*>(slope), a.dloss = dloss, a.dlogits = dlogits;
  return from_cuda(launch_balance_bwd(a, static_cast<cudaStream_t>(stream)));
}

mgg_status mgg_linear_cross_entropy(const void* x, int64_t ldx, const void* W, const void* targets,
                                    int targets_i64, int64_t ignore_index, int T, int K, int V,
                                    mgg_reduction reduction, float z_loss, float* loss, float* lse,
                                    float* weight, int32_t* dev_status, void* ws, size_t ws_bytes,
                                    void* stream) {
  const NvtxRange nvtx("mgg_linear_cross_entropy");
  mgg_status s = check_vocab(ldx, T, K, V, z_loss);
  if (s != MGG_OK) return s;
  if (reduction != MGG_REDUCE_NONE && reduction != MGG_REDUCE_SUM && reduction != MGG_REDUCE_MEAN)
    return MGG_ERR_INVALID_ARG;
  if (!weight || (!loss && (T > 0 || reduction != MGG_REDUCE_NONE))) return MGG_ERR_INVALID_ARG;
  if (!aligned(weight, 4) || !aligned(loss, 4)) return MGG_ERR_ALIGNMENT;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T > 0) {
    if (!x || !W || !targets || !lse || !dev_status) return MGG_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(lse, 4) || !aligned(targets, targets_i64 ? 8 : 4))
      return MGG_ERR_ALIGNMENT;
  }
  s = check_arch();
  if (s != MGG_OK) return s;
  if (T > 0 && (!ws || !aligned(ws, 256) || ws_bytes < vocab_fwd_ws_bytes(T, K, V))) return MGG_ERR_WORKSPACE;
  VocabForward a{};
  a.x = x, a.ldx = ldx, a.W = W, a.targets = targets, a.i64 = targets_i64 != 0, a.ignore = ignore_index;
  a.T = T, a.K = K, a.V = V, a.reduction = reduction, a.z_loss = z_loss;
  a.loss = loss, a.lse = lse, a.weight = weight, a.dev_status = dev_status, a.wait_limit = wait_limit();
  return from_cuda(launch_vocab_forward(a, ws, st));
}

mgg_status mgg_linear_cross_entropy_backward(const float* dloss, int per_token, const float* weight,
                                             const void* x, int64_t ldx, const void* W,
                                             const void* targets, int targets_i64,
                                             int64_t ignore_index, const float* lse, int T, int K,
                                             int V, float z_loss, void* dx, void* dW,
                                             int32_t* dev_status, void* ws, size_t ws_bytes,
                                             void* stream) {
  const NvtxRange nvtx("mgg_linear_cross_entropy_backward");
  mgg_status s = check_vocab(ldx, T, K, V, z_loss);
  if (s != MGG_OK) return s;
  if (!aligned(dx, 16) || !aligned(dW, 16)) return MGG_ERR_ALIGNMENT;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    s = check_arch();
    return s == MGG_OK ? zero(dW, static_cast<size_t>(V) * K * 2, st) : s;
  }
  if (!dloss || !weight || !x || !W || !targets || !lse || !dev_status) return MGG_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(lse, 4) || !aligned(dloss, 4) || !aligned(weight, 4) ||
      !aligned(targets, targets_i64 ? 8 : 4))
    return MGG_ERR_ALIGNMENT;
  s = check_arch();
  if (s != MGG_OK) return s;
  if (!ws || !aligned(ws, 256) || ws_bytes < vocab_bwd_ws_bytes(T, K, V)) return MGG_ERR_WORKSPACE;
  if (!dx && !dW) return MGG_OK;
  VocabBackward a{};
  a.dloss = dloss, a.per_token = per_token != 0, a.weight = weight, a.x = x, a.ldx = ldx, a.W = W;
  a.targets = targets, a.i64 = targets_i64 != 0, a.ignore = ignore_index, a.lse = lse;
  a.T = T, a.K = K, a.V = V, a.z_loss = z_loss, a.dx = dx, a.dW = dW;
  a.dev_status = dev_status, a.wait_limit = wait_limit();
  return from_cuda(launch_vocab_backward(a, ws, st));
}

mgg_status mgg_adamw_step(const mgg_adamw_tensor* tensors, int count, mgg_dtype p_dtype,
                          mgg_dtype g_dtype, int bits, double lr, const float* lr_dev, double beta1,
                          double beta2, double eps, double decay, int64_t step,
                          const int32_t* step_dev, const float* grad_scale, void* stream) {
  const NvtxRange nvtx("mgg_adamw_step");
  auto rate = [](double v) { return v >= 0.0 && isfinite(v); };
  if (count < 0 || (count > 0 && !tensors) || (bits != 8 && bits != 32)) return MGG_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !rate(eps) || !rate(decay) ||
      (!lr_dev && !rate(lr)) || (!step_dev && step < 1))
    return MGG_ERR_INVALID_ARG;
  if (!float_type(p_dtype) || !float_type(g_dtype)) return MGG_ERR_DTYPE;
  if (!aligned(lr_dev, 4) || !aligned(step_dev, 4) || !aligned(grad_scale, 4)) return MGG_ERR_ALIGNMENT;
  bool master = false, any = false;
  for (int i = 0; i < count; ++i) {
    const mgg_adamw_tensor& t = tensors[i];
    if (t.n < 0) return MGG_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!any) master = t.master != nullptr;
    any = true;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || (t.master != nullptr) != master ||
        (bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
      return MGG_ERR_INVALID_ARG;
    const size_t sb = bits == 8 ? 1 : 4;
    if (!aligned(t.param, size_of(p_dtype)) || !aligned(t.grad, size_of(g_dtype)) || !aligned(t.master, 4) ||
        !aligned(t.exp_avg, sb) || !aligned(t.exp_avg_sq, sb) || !aligned(t.exp_avg_scale, 4) ||
        !aligned(t.exp_avg_sq_scale, 4))
      return MGG_ERR_ALIGNMENT;
  }
  if (master && p_dtype == MGG_F32) return MGG_ERR_INVALID_ARG;
  if (!any) return MGG_OK;
  const mgg_status s = check_arch();
  if (s != MGG_OK) return s;
  AdamwArgs a{};
  a.tensors = tensors, a.count = count, a.p_f32 = p_dtype == MGG_F32, a.g_f32 = g_dtype == MGG_F32;
  a.master = master, a.bits8 = bits == 8;
  a.lr = lr, a.beta1 = beta1, a.beta2 = beta2, a.eps = eps, a.decay = decay, a.step = step;
  a.lr_dev = lr_dev, a.step_dev = step_dev, a.grad_scale = grad_scale;
  return from_cuda(launch_adamw(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
