// The choice of the experts from the gate's logits, and its gradient.
//
// Per token (one warp): scores p_e, selection keys, the best topk_groups
// groups, the k best keys, the weights of the chosen.
//   softmax: p = softmax over the unmasked logits; key = logit, or p + bias
//            with a bias (the logit orders as p does, without p's rounding)
//   sigmoid: p = 1 / (1 + exp(-logit)); key = p (+ bias)
// A logit that is NaN, -inf or its type's lowest value masks the expert; +inf
// counts as the largest finite value.  Keys are compared as order-preserving
// 32-bit integers (monotone map of the f32 bits), so a round of the top-k is
// two integer warp reductions: the largest key, then the lowest expert that
// holds it.  0 marks a chosen expert, 1 an expert that cannot be chosen on
// its merits (masked, or outside the kept groups): such experts are taken
// only when nothing else is left, lowest index first, with weight 0, so that
// the k ids are always valid and distinct.
//
// Each lane holds V consecutive experts in registers.  The kernel is bound by
// instruction issue, not by its bytes (a few KB per token).
#include "common.cuh"
#include "internal.h"

namespace mgg {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t order_key(float f) {
  if (!(f > -INFINITY)) return 1u;  // -inf, NaN
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// The masked logit of the type's lowest value, -inf or NaN reads as -inf,
// +inf as the largest finite f32.
template <typename T>
__device__ __forceinline__ float open_logit(T v);
template <>
__device__ __forceinline__ float open_logit<float>(float v) {
  return v > -3.402823466e38f ? fminf(v, 3.402823466e38f) : -INFINITY;
}
template <>
__device__ __forceinline__ float open_logit<__nv_bfloat16>(__nv_bfloat16 b) {
  const float v = __bfloat162float(b);
  return v > __uint_as_float(0xff7f0000u) ? fminf(v, 3.402823466e38f) : -INFINITY;
}

// V consecutive logits from expert e0 (out of range: masked).
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int e0, int E, bool vec, float (&l)[V]) {
  constexpr int PER = 16 / sizeof(T);
  if constexpr (V % PER == 0) {
    if (vec) {  // E a multiple of V's 16-byte pieces, rows 16-byte aligned
#pragma unroll
      for (int i = 0; i < V; i += PER) {
        if (e0 + i < E) {
          const uint4 q = *reinterpret_cast<const uint4*>(row + e0 + i);
          const uint32_t u[4] = {q.x, q.y, q.z, q.w};
          if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) l[i + j] = open_logit<float>(__uint_as_float(u[j]));
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              l[i + j] = open_logit<__nv_bfloat16>(__ushort_as_bfloat16(
                  static_cast<unsigned short>(u[j / 2] >> (16 * (j & 1)))));
          }
        } else {
#pragma unroll
          for (int j = 0; j < PER; ++j) l[i + j] = -INFINITY;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = e0 + i < E ? open_logit<T>(row[e0 + i]) : -INFINITY;
}

struct SelectArgs {
  const void* logits;
  long long ldl;
  const float* bias;
  int T, E, k;
  bool softmax;
  int groups, topk_groups;
  bool renorm;
  float scale;
  int32_t* ids;
  float* weights;
  bool vec;
};

template <typename T, int V>
__global__ void __launch_bounds__(kWarps * 32) select_kernel(const SelectArgs a) {
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  if (t >= a.T) return;
  const int E = a.E, e0 = lane * V;
  float p[V];
  uint32_t key[V];
  load_logits<T, V>(static_cast<const T*>(a.logits) + t * a.ldl, e0, E, a.vec, p);
  if (a.softmax) {
    float top = p[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, p[i]);
    top = warp_max(top);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = order_key(p[i]);
      p[i] = p[i] > -INFINITY ? expf(p[i] - top) : 0.f;
      sum += p[i];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] *= inv;
      if (a.bias && key[i] > 1u) key[i] = order_key(p[i] + a.bias[e0 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool open = p[i] > -INFINITY;
      // below -87 exp(-logit) nears f32's end, and 1 + exp(-logit) has long
      // been exp(-logit): exp(logit) itself, down to the denormals, so that a
      // row of very low logits keeps its proportions; 0 where masked
      p[i] = p[i] < -87.f ? expf(p[i]) : 1.f / (1.f + expf(-p[i]));
      key[i] = open ? order_key(a.bias ? p[i] + a.bias[e0 + i] : p[i]) : 1u;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (e0 + i >= E) key[i] = 0u;  // no expert here

  if (a.groups > 1) {
    // lane g keeps the score of group g
    const int gs = E / a.groups;
    uint32_t mine = 0u;
    for (int g = 0; g < a.groups; ++g) {
      uint32_t x = 0u, y = 0u;  // the lane's best two keys in the group
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = e0 + i;
        const uint32_t u = e >= g * gs && e < (g + 1) * gs ? key[i] : 0u;
        y = max(y, min(x, u));
        x = max(x, u);
      }
      const uint32_t b1 = __reduce_max_sync(kFull, x);
      uint32_t score = b1;
      if (!a.softmax) {
        const int owner = __ffs(__ballot_sync(kFull, x == b1)) - 1;
        const uint32_t b2 = __reduce_max_sync(kFull, lane == owner ? y : x);
        if (b1 > 1u && b2 > 1u) score = order_key(key_value(b1) + key_value(b2));
      }
      if (lane == g) mine = score;
    }
    uint32_t kept = 0u;
    for (int r = 0; r < a.topk_groups; ++r) {
      const uint32_t b = __reduce_max_sync(kFull, mine);
      const int g = __ffs(__ballot_sync(kFull, mine == b)) - 1;
      kept |= 1u << g;
      if (lane == g) mine = 0u;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < E && !((kept >> ((e0 + i) / gs)) & 1u)) key[i] = 1u;
  }

  // k rounds: the largest key, the lowest expert among equals
  int id_mine = 0;
  float w_mine = 0.f;
  uint32_t best = 0u;
  int slot = 0;
  auto rescan = [&]() {
    best = key[0];
    slot = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > best) best = key[i], slot = i;
  };
  rescan();
  for (int r = 0; r < a.k; ++r) {
    const uint32_t b = __reduce_max_sync(kFull, best);
    const int owner = __ffs(__ballot_sync(kFull, best == b)) - 1;
    float w = 0.f;
    const int id = __shfl_sync(kFull, e0 + slot, owner);
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == slot) {
          w = b > 1u ? p[i] : 0.f;
          key[i] = 0u;
        }
      rescan();
    }
    w = __shfl_sync(kFull, w, owner);
    if (lane == r) {
      id_mine = id;
      w_mine = w;
    }
  }
  if (a.renorm) {
    const float tot = warp_sum(w_mine);
    w_mine = tot > 0.f ? w_mine / tot : 0.f;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id_mine;
    a.weights[t * a.k + lane] = w_mine * a.scale;
  }
}

// ---------------------------------------------------------------- backward
// The choice is held fixed; with dot = sum_i g_i w_i over the chosen:
//   softmax, renormalised: dl_j = w_j (g_j - dot / scale)
//   softmax:               dl_e = [e chosen] w_j g_j - p_e dot
//   sigmoid, renormalised: dl_j = w_j (1 - p_j) (g_j - dot / scale)
//   sigmoid:               dl_j = w_j (1 - p_j) g_j
// The weights carry p already, so only the dense case reads whole logits and
// only sigmoid the chosen ones.  Each warp scatters its token's k values into
// a zeroed row in shared memory and writes the row out whole (equal ids, which
// the choice never gives, add up in order).
struct SelectBwdArgs {
  const float* g;
  const void* logits;
  long long ldl;
  const int32_t* ids;
  const float* w;
  int T, E, k;
  bool softmax, renorm;
  float scale;
  void* out;
  int32_t* dev_status;
  bool vec;
};

template <typename T>
__device__ __forceinline__ void put(T* p, float v);
template <>
__device__ __forceinline__ void put<float>(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void put<__nv_bfloat16>(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}

template <typename T, int V>
__global__ void __launch_bounds__(kWarps * 32) select_bwd_kernel(const SelectBwdArgs a) {
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int E = a.E;
  float* row = rows + warp * (32 * V);
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < V; ++i) row[i * 32 + lane] = 0.f;
  pdl_wait();
  if (t >= a.T) return;
  const T* lr = static_cast<const T*>(a.logits) + t * a.ldl;
  float p[V];
  const bool dense = a.softmax && !a.renorm;
  if (dense) {
    load_logits<T, V>(lr, lane * V, E, a.vec, p);
    float top = p[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, p[i]);
    top = warp_max(top);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = p[i] > -INFINITY ? expf(p[i] - top) : 0.f;
      sum += p[i];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= inv;
  }
  int id = -1 - lane;  // lanes without a choice: all different, none an expert
  float w = 0.f, g = 0.f;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    w = a.w[t * a.k + lane];
    g = a.g[t * a.k + lane];
    if (id < 0 || id >= E) {
      atomicOr(a.dev_status, kDevBadExpertId);
      id = -1 - lane;
      w = 0.f;
    }
    if (w == 0.f) g = 0.f;  // a void choice takes no part, whatever its gradient holds
  }
  const float dot = warp_sum(g * w);
  float d = w * g;
  if (a.renorm) d = w * (g - dot / a.scale);
  if (!a.softmax && id >= 0) {
    const float l = open_logit<T>(lr[id]);
    d *= 1.f - 1.f / (1.f + expf(-l));
  }
  __syncwarp();
  const unsigned same = __match_any_sync(kFull, id);
  if (__all_sync(kFull, same == (1u << lane))) {
    if (id >= 0) row[id] = d;
  } else {
    for (int r = 0; r < a.k; ++r) {
      if (lane == r && id >= 0) row[id] += d;
      __syncwarp();
    }
  }
  __syncwarp();
  T* out = static_cast<T*>(a.out) + t * E;
  if (dense) {
#pragma unroll
    for (int i = 0; i < V; ++i) row[lane * V + i] -= p[i] * dot;
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    if (e < E) put<T>(out + e, row[e]);
  }
}

template <typename T>
cudaError_t select_t(const SelectArgs& a, cudaStream_t st) {
  const dim3 grid(cdiv(a.T, kWarps)), block(kWarps * 32);
  if (a.E <= 32) return launch_pdl(select_kernel<T, 1>, grid, block, 0, st, a);
  if (a.E <= 64) return launch_pdl(select_kernel<T, 2>, grid, block, 0, st, a);
  if (a.E <= 128) return launch_pdl(select_kernel<T, 4>, grid, block, 0, st, a);
  if (a.E <= 256) return launch_pdl(select_kernel<T, 8>, grid, block, 0, st, a);
  if (a.E <= 512) return launch_pdl(select_kernel<T, 16>, grid, block, 0, st, a);
  return launch_pdl(select_kernel<T, 32>, grid, block, 0, st, a);
}
template <typename T>
cudaError_t select_bwd_t(const SelectBwdArgs& a, cudaStream_t st) {
  const dim3 grid(cdiv(a.T, kWarps)), block(kWarps * 32);
  auto smem = [](int v) { return static_cast<size_t>(kWarps) * 32 * v * 4; };
  if (a.E <= 32) return launch_pdl(select_bwd_kernel<T, 1>, grid, block, smem(1), st, a);
  if (a.E <= 64) return launch_pdl(select_bwd_kernel<T, 2>, grid, block, smem(2), st, a);
  if (a.E <= 128) return launch_pdl(select_bwd_kernel<T, 4>, grid, block, smem(4), st, a);
  if (a.E <= 256) return launch_pdl(select_bwd_kernel<T, 8>, grid, block, smem(8), st, a);
  if (a.E <= 512) return launch_pdl(select_bwd_kernel<T, 16>, grid, block, smem(16), st, a);
  return launch_pdl(select_bwd_kernel<T, 32>, grid, block, smem(32), st, a);
}

// 16-byte loads of the logits: rows on 16-byte boundaries and whole pieces.
bool vec_logits(const void* p, long long ldl, int E, bool f32) {
  const int per = f32 ? 4 : 8;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ldl % per == 0 && E % per == 0;
}

}  // namespace

cudaError_t launch_select(const void* logits, bool f32, long long ldl, int T, int E, int k,
                          bool softmax, const float* bias, int groups, int topk_groups,
                          bool renorm, float scale, int32_t* ids, float* weights,
                          cudaStream_t st) {
  const SelectArgs a{logits, ldl,         bias,   T,     E,   k,       softmax,
                     groups, topk_groups, renorm, scale, ids, weights, vec_logits(logits, ldl, E, f32)};
  return f32 ? select_t<float>(a, st) : select_t<__nv_bfloat16>(a, st);
}

cudaError_t launch_select_bwd(const float* g, const void* logits, bool f32, long long ldl,
                              const int32_t* ids, const float* w, int T, int E, int k,
                              bool softmax, bool renorm, float scale, void* out,
                              int32_t* dev_status, cudaStream_t st) {
  const SelectBwdArgs a{g,       logits, ldl,   ids, w,          T, E, k,
                        softmax, renorm, scale, out, dev_status, vec_logits(logits, ldl, E, f32)};
  return f32 ? select_bwd_t<float>(a, st) : select_bwd_t<__nv_bfloat16>(a, st);
}

}  // namespace mgg
