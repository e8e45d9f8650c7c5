// The choice of the experts from the gate's logits, and its gradient.
//
// Per token (one warp): scores p_e, selection keys, the best topk_groups
// groups, the k best keys, the weights of the chosen.
//   softmax: p = softmax over the unmasked logits; key = logit, or p + bias
//            with a bias (the logit orders as p does, without p's rounding) or
//            where two keys are added up
//   sigmoid: p = 1 / (1 + exp(-logit)); key = p (+ bias)
// A logit that is NaN, -inf or its type's lowest value masks the expert; +inf
// counts as the largest finite value.  Keys are compared as order-preserving
// 32-bit integers (monotone map of the f32 bits), so a round of the top-k is an
// integer warp reduction for the largest key and a ballot (lanes in expert order)
// or a second reduction (beyond 256 experts) for the lowest expert that holds
// it.  0 marks a chosen expert, 1 an expert that cannot be chosen on
// its merits (masked, or outside the kept groups): such experts are taken
// only when nothing else is left, lowest index first, with weight 0, so that
// the k ids are always valid and distinct.
//
// Up to 256 experts each lane holds V consecutive ones in registers.  The kernel is bound by
// instruction issue, not by its bytes (1 KB per token at E = 256), so the work
// per round of the top-k is what counts: up to V = 8 a lane sorts its keys once
// and a round pops the winner's list.
// Measured: 64 x 128 bf16, k = 8 5 to 6 us (latency); 16384 x 256 f32 sigmoid with
// bias, 4 of 8 groups 16.4 us (1.1 TB/s); gradient, dense, 16384 x 256 10.3 us
// (3.4 TB/s).
#include "common.cuh"
#include "internal.h"

namespace mgg {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t order_key(float f) {
  const int u = __float_as_int(f + 0.f);  // -0 -> +0
  const uint32_t k = static_cast<uint32_t>(u ^ ((u >> 31) | 0x80000000));
  return f > -INFINITY ? k : 1u;  // -inf, NaN
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
  if constexpr (V == 4 && PER == 8) {
    if (vec) {  // 8 bytes a lane
      uint2 q = make_uint2(0xff80ff80u, 0xff80ff80u);  // -inf
      if (e0 < E) q = *reinterpret_cast<const uint2*>(row + e0);
      const uint32_t u[2] = {q.x, q.y};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        l[j] = open_logit<T>(__ushort_as_bfloat16(static_cast<unsigned short>(u[j / 2] >> (16 * (j & 1)))));
      return;
    }
  } else if constexpr (V % PER == 0) {
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
  bool two_best;  // a group's score: the sum of its two best keys, else its best
  bool renorm;
  float scale;
  int32_t* ids;
  float* weights;
  bool vec, vec_bias;  // 16-byte loads
};

// Keys of the experts outside the topk_groups best groups become 1.  Returns
// the lanes whose experts stay, or 0 where the groups share lanes.
template <int V>
__device__ __forceinline__ uint32_t keep_groups(const SelectArgs& a, int e0, int lane,
                                                uint32_t (&key)[V]) {
  const int gs = a.E / a.groups;
  const int L = gs / V;  // lanes per group, where that divides evenly
  auto score = [&](uint32_t b1, uint32_t b2) {
    return a.two_best && b1 > 1u && b2 > 1u ? order_key(key_value(b1) + key_value(b2)) : b1;
  };
  if (gs % V == 0 && (L & (L - 1)) == 0) {
    // a lane's experts are of one group and the group's lanes an aligned
    // power of two: two best keys per lane, then over the group's lanes
    uint32_t x = 0u, y = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      y = max(y, min(x, key[i]));
      x = max(x, key[i]);
    }
    for (int o = 1; o < L; o <<= 1) {
      const uint32_t x2 = __shfl_xor_sync(kFull, x, o), y2 = __shfl_xor_sync(kFull, y, o);
      y = max(min(x, x2), max(y, y2));
      x = max(x, x2);
    }
    const int lg = __ffs(L) - 1, mine_g = lane >> lg;
    uint32_t mine = e0 < a.E ? score(x, y) : 0u;
    bool kept = false;
    for (int r = 0; r < a.topk_groups; ++r) {
      const uint32_t b = __reduce_max_sync(kFull, mine);
      const int g = (__ffs(__ballot_sync(kFull, mine == b)) - 1) >> lg;
      if (g == mine_g) mine = 0u, kept = true;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!kept && e0 + i < a.E) key[i] = 1u;
    return __ballot_sync(kFull, kept);
  }
  // any other size: group by group, lane g keeps the score of group g
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
    const int owner = __ffs(__ballot_sync(kFull, x == b1)) - 1;
    const uint32_t b2 = __reduce_max_sync(kFull, lane == owner ? y : x);
    if (lane == g) mine = score(b1, b2);
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
    if (e0 + i < a.E && !((kept >> ((e0 + i) / gs)) & 1u)) key[i] = 1u;
  return 0u;
}

// k rounds: the largest key, the lowest expert among equals; lane r keeps round
// r's expert and key.  Returns the last round's key (the same in every lane).
// e0: the lane's first expert, lanes in expert order.
template <int V>
__device__ __forceinline__ uint32_t top_k(uint32_t (&key)[V], int e0, int k, int lane, int& id_mine,
                                          uint32_t& key_mine) {
  static_assert(V <= 8, "4-bit places");
  uint32_t b = 0u;
  // Each lane's keys in descending order (odd-even transposition with strict
  // comparisons: equal keys keep their order), their places as 4-bit digits.
  uint32_t place[V];
#pragma unroll
  for (int i = 0; i < V; ++i) place[i] = i;
#pragma unroll
  for (int r = 0; r < V; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < V; i += 2) {
      const bool swap = key[i + 1] > key[i];
      const uint32_t hi = max(key[i], key[i + 1]), lo = min(key[i], key[i + 1]);
      const uint32_t ph = swap ? place[i + 1] : place[i], pl = swap ? place[i] : place[i + 1];
      key[i] = hi, key[i + 1] = lo;
      place[i] = ph, place[i + 1] = pl;
    }
  uint32_t places = 0u;
#pragma unroll
  for (int i = 0; i < V; ++i) places |= place[i] << (4 * i);
  for (int r = 0; r < k; ++r) {
    b = __reduce_max_sync(kFull, key[0]);
    const int owner = __ffs(__ballot_sync(kFull, key[0] == b)) - 1;
    const int id = __shfl_sync(kFull, e0 + static_cast<int>(places & 15u), owner);
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
      key[V - 1] = 0u;
      places >>= 4;
    }
    if (lane == r) id_mine = id, key_mine = b;
  }
  return b;
}

// Per warp: 32 V scores, and room to spread half of the keys.
template <int V>
constexpr bool kSpread = V >= 4;
template <int V>
constexpr int kRowFloats = 32 * V + (kSpread<V> ? 16 * V + 16 : 0);

template <typename T, int V>
__global__ void __launch_bounds__(kWarps * 32) select_kernel(const SelectArgs a) {
  extern __shared__ float scores[];  // [kWarps][kRowFloats]
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  if (t >= a.T) return;
  const int E = a.E, e0 = lane * V;
  float p[V];
  uint32_t key[V];
  load_logits<T, V>(static_cast<const T*>(a.logits) + t * a.ldl, e0, E, a.vec, p);
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = 0.f;
  if (a.bias) {
    bool done = false;
    if constexpr (V % 4 == 0) {
      if (a.vec_bias) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
          if (e0 + i < E) {
            const float4 v = *reinterpret_cast<const float4*>(a.bias + e0 + i);
            bias[i] = v.x, bias[i + 1] = v.y, bias[i + 2] = v.z, bias[i + 3] = v.w;
          }
        done = true;
      }
    }
    if (!done) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < E) bias[i] = a.bias[e0 + i];
    }
  }
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
      if ((a.bias || a.two_best) && key[i] > 1u) key[i] = order_key(p[i] + bias[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float l = p[i];
      p[i] = __frcp_rn(1.f + expf(-l));  // (correctly rounded, as the division)
      // below -87 exp(-logit) nears f32's end, and 1 + exp(-logit) has long
      // been exp(-logit): exp(logit) itself, down to the denormals, so that a
      // row of very low logits keeps its proportions; 0 where masked
      if (l < -87.f) p[i] = expf(l);
      key[i] = order_key(l > -INFINITY ? p[i] + bias[i] : l);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (e0 + i >= E) key[i] = 0u;  // no expert here

  const uint32_t kept = a.groups > 1 ? keep_groups<V>(a, e0, lane, key) : 0u;

  // the scores where every lane can read them
  float* row = scores + (threadIdx.x >> 5) * kRowFloats<V>;
#pragma unroll
  for (int i = 0; i < V; ++i) row[e0 + i] = p[i];

  int id_mine = 0;
  uint32_t key_mine = 0u;
  bool done = false;
  if constexpr (kSpread<V>) {
    if (kept && __popc(kept) <= 16) {
      // At most half of the lanes hold experts that stay: spread those over all
      // of them, half as many keys each.
      constexpr int VC = V / 2;
      uint32_t* keys = reinterpret_cast<uint32_t*>(row + 32 * V);
      int* first = reinterpret_cast<int*>(keys + 16 * V);
      const int rank = __popc(kept & ((1u << lane) - 1u)), n = __popc(kept);
      if ((kept >> lane) & 1u) {
#pragma unroll
        for (int i = 0; i < V; ++i) keys[rank * V + i] = key[i];
        first[rank] = e0;
      }
      __syncwarp();
      uint32_t half[VC];
      const bool has = lane / 2 < n;
#pragma unroll
      for (int i = 0; i < VC; ++i) half[i] = has ? keys[lane * VC + i] : 0u;
      const int h0 = has ? first[lane / 2] + (lane & 1) * VC : 0;
      // (fewer than k that can be chosen on their merits: over all experts below)
      done = top_k<VC>(half, h0, a.k, lane, id_mine, key_mine) > 1u;
    }
  }
  if (!done) top_k<V>(key, e0, a.k, lane, id_mine, key_mine);
  __syncwarp();
  float w_mine = lane < a.k && key_mine > 1u ? row[id_mine] : 0.f;
  if (a.renorm) {
    const float tot = warp_sum(w_mine);
    w_mine = tot > 0.f ? w_mine / tot : 0.f;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id_mine;
    a.weights[t * a.k + lane] = w_mine * a.scale;
  }
}

// More than 256 experts: the scores and keys of a token in shared memory, lane l
// with experts l, l + 32, ...  Loops instead of unrolled registers: the code of
// 32 experts per lane did not fit the instruction cache (13 us for 32 tokens).
constexpr int kWideWarps = 4;
template <typename T>
__global__ void __launch_bounds__(kWideWarps * 32) select_wide_kernel(const SelectArgs a) {
  extern __shared__ float wide[];  // [kWideWarps][2][E]
  const int lane = threadIdx.x & 31, E = a.E;
  const long long t = static_cast<long long>(blockIdx.x) * kWideWarps + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  if (t >= a.T) return;
  float* p = wide + (threadIdx.x >> 5) * 2 * E;
  uint32_t* key = reinterpret_cast<uint32_t*>(p + E);
  const T* lr = static_cast<const T*>(a.logits) + t * a.ldl;
  float top = -INFINITY;
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const float l = open_logit<T>(lr[e]);
    p[e] = l;
    top = fmaxf(top, l);
  }
  float inv = 1.f;
  const bool by_logit = a.softmax && !a.bias && !a.two_best;
  if (a.softmax) {
    top = warp_max(top);
    float sum = 0.f;
#pragma unroll 4
    for (int e = lane; e < E; e += 32) sum += p[e] > -INFINITY ? expf(p[e] - top) : 0.f;
    sum = warp_sum(sum);
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const float l = p[e], bias = a.bias ? a.bias[e] : 0.f;
    float s;
    if (a.softmax) {
      s = l > -INFINITY ? expf(l - top) * inv : 0.f;
    } else {
      s = __frcp_rn(1.f + expf(-l));
      if (l < -87.f) s = expf(l);  // (as above)
    }
    p[e] = s;
    key[e] = order_key(l > -INFINITY ? (by_logit ? l : s + bias) : l);
  }
  __syncwarp();
  if (a.groups > 1) {
    // group by group, lane g keeps the score of group g
    const int gs = E / a.groups;
    uint32_t mine = 0u;
    for (int g = 0; g < a.groups; ++g) {
      uint32_t x = 0u, y = 0u;
      for (int i = lane; i < gs; i += 32) {
        const uint32_t u = key[g * gs + i];
        y = max(y, min(x, u));
        x = max(x, u);
      }
      const uint32_t b1 = __reduce_max_sync(kFull, x);
      const int owner = __ffs(__ballot_sync(kFull, x == b1)) - 1;
      const uint32_t b2 = __reduce_max_sync(kFull, lane == owner ? y : x);
      if (lane == g)
        mine = a.two_best && b1 > 1u && b2 > 1u ? order_key(key_value(b1) + key_value(b2)) : b1;
    }
    uint32_t kept = 0u;
    for (int r = 0; r < a.topk_groups; ++r) {
      const uint32_t b = __reduce_max_sync(kFull, mine);
      const int g = __ffs(__ballot_sync(kFull, mine == b)) - 1;
      kept |= 1u << g;
      if (lane == g) mine = 0u;
    }
    for (int g = 0; g < a.groups; ++g)
      if (!((kept >> g) & 1u))
        for (int i = lane; i < gs; i += 32) key[g * gs + i] = 1u;
    __syncwarp();
  }
  // k rounds; a lane's best: its largest key, the lowest expert among equals
  uint32_t best = 0u;
  int at = 0;
  auto rescan = [&]() {
    best = 0u;
#pragma unroll 8
    for (int e = lane; e < E; e += 32) {
      const uint32_t u = key[e];
      if (u > best) best = u, at = e;
    }
  };
  rescan();
  int id_mine = 0;
  uint32_t key_mine = 0u;
  for (int r = 0; r < a.k; ++r) {
    const uint32_t b = __reduce_max_sync(kFull, best);
    const int id = static_cast<int>(__reduce_min_sync(kFull, best == b ? static_cast<unsigned>(at) : ~0u));
    if (lane == (id & 31)) {
      key[id] = 0u;
      rescan();
    }
    if (lane == r) id_mine = id, key_mine = b;
  }
  float w = lane < a.k && key_mine > 1u ? p[id_mine] : 0.f;
  if (a.renorm) {
    const float tot = warp_sum(w);
    w = tot > 0.f ? w / tot : 0.f;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id_mine;
    a.weights[t * a.k + lane] = w * a.scale;
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
  bool vec, vec_out;
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
  if (dense) load_logits<T, V>(lr, lane * V, E, a.vec, p);
  // (loaded beside the logits: one latency for all)
  int id = -1 - lane;  // lanes without a choice: all different, none an expert
  float w = 0.f, g = 0.f;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    w = a.w[t * a.k + lane];
    g = a.g[t * a.k + lane];
  }
  if (dense) {
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
  if (lane < a.k) {
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
    // 1 - p = 1 / (1 + exp(l)): from a rounded p it has three digits left at a
    // logit of 10 and none from 17 on
    d *= 1.f / (1.f + expf(l));
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
  if constexpr (V % 4 == 0) {
    // four consecutive experts per access, lane after lane
    if (a.vec_out) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const int e = dense ? lane * V + i : (i / 4) * 128 + lane * 4;
        if (e >= E) continue;
        float4 v = *reinterpret_cast<const float4*>(row + e);
        if (dense) {
          v.x -= p[i] * dot, v.y -= p[i + 1] * dot;
          v.z -= p[i + 2] * dot, v.w -= p[i + 3] * dot;
        }
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(out + e) = v;
        else
          *reinterpret_cast<uint2*>(out + e) = make_uint2(cvt_bf16x2(v.x, v.y), cvt_bf16x2(v.z, v.w));
      }
      return;
    }
  }
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

size_t row_smem(int v) { return static_cast<size_t>(kWarps) * 32 * v * 4; }
template <typename T, int V>
cudaError_t select_tv(const SelectArgs& a, cudaStream_t st) {
  return launch_pdl(select_kernel<T, V>, dim3(cdiv(a.T, kWarps)), dim3(kWarps * 32),
                    kWarps * kRowFloats<V> * sizeof(float), st, a);
}
template <typename T>
cudaError_t select_t(const SelectArgs& a, cudaStream_t st) {
  if (a.E <= 32) return select_tv<T, 1>(a, st);
  if (a.E <= 64) return select_tv<T, 2>(a, st);
  if (a.E <= 128) return select_tv<T, 4>(a, st);
  if (a.E <= 256) return select_tv<T, 8>(a, st);
  return launch_pdl(select_wide_kernel<T>, dim3(cdiv(a.T, kWideWarps)), dim3(kWideWarps * 32),
                    static_cast<size_t>(kWideWarps) * 2 * a.E * sizeof(float), st, a);
}
template <typename T>
cudaError_t select_bwd_t(const SelectBwdArgs& a, cudaStream_t st) {
  const dim3 grid(cdiv(a.T, kWarps)), block(kWarps * 32);
  if (a.E <= 32) return launch_pdl(select_bwd_kernel<T, 1>, grid, block, row_smem(1), st, a);
  if (a.E <= 64) return launch_pdl(select_bwd_kernel<T, 2>, grid, block, row_smem(2), st, a);
  if (a.E <= 128) return launch_pdl(select_bwd_kernel<T, 4>, grid, block, row_smem(4), st, a);
  if (a.E <= 256) return launch_pdl(select_bwd_kernel<T, 8>, grid, block, row_smem(8), st, a);
  if (a.E <= 512) return launch_pdl(select_bwd_kernel<T, 16>, grid, block, row_smem(16), st, a);
  return launch_pdl(select_bwd_kernel<T, 32>, grid, block, row_smem(32), st, a);
}

// 16-byte loads of the logits: rows on 16-byte boundaries and whole pieces.
bool vec_logits(const void* p, long long ldl, int E, bool f32) {
  const int per = f32 ? 4 : 8;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ldl % per == 0 && E % per == 0;
}

}  // namespace

cudaError_t launch_select(const void* logits, bool f32, long long ldl, int T, int E, int k,
                          bool softmax, const float* bias, int groups, int topk_groups,
                          bool two_best, bool renorm, float scale, int32_t* ids, float* weights,
                          cudaStream_t st) {
  const SelectArgs a{logits,   ldl,    bias,  T,   E,       k, softmax, groups, topk_groups,
                     two_best, renorm, scale, ids, weights, vec_logits(logits, ldl, E, f32),
                     reinterpret_cast<uintptr_t>(bias) % 16 == 0 && E % 4 == 0};
  return f32 ? select_t<float>(a, st) : select_t<__nv_bfloat16>(a, st);
}

cudaError_t launch_select_bwd(const float* g, const void* logits, bool f32, long long ldl,
                              const int32_t* ids, const float* w, int T, int E, int k,
                              bool softmax, bool renorm, float scale, void* out,
                              int32_t* dev_status, cudaStream_t st) {
  const SelectBwdArgs a{g,       logits, ldl,   ids, w,          T, E, k,
                        softmax, renorm, scale, out, dev_status, vec_logits(logits, ldl, E, f32),
                        reinterpret_cast<uintptr_t>(out) % 16 == 0 && E % 4 == 0};
  return f32 ? select_bwd_t<float>(a, st) : select_bwd_t<__nv_bfloat16>(a, st);
}

}  // namespace mgg
