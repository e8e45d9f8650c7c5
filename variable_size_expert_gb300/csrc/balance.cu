// Balance loss of the gate, with the experts' counts:
//   p_te  = softmax_e(z_t), or sigmoid(z_te) / sum_j sigmoid(z_tj)
//   n_b   = tokens of sequence b that count; count_be = their choices of expert e
//   loss  = 1/B' sum_b sum_e (E count_be / (k n_b)) (1/n_b sum_t p_te),  B' the
//           sequences with tokens
//         = sum_be slope_be sum_t p_te,  slope_be = E count_be / (k n_b^2 B')
//   dz_te = dloss p_te (slope_be - sum_j p_tj slope_bj)   (sigmoid: times 1 - a_te)
//
// Bound by the logits' bytes, and below some megabytes by the launches.  Forward:
// blocks over runs of a sequence's tokens leave their column sums of p and their
// counts; a second kernel adds these up in the blocks' order (the same bits every
// time), forms the slopes and the loss.  A token's logits lie in the registers of
// `lanes` lanes (a power of two, 32 from 128 experts on), so that a softmax is
// log2(lanes) shuffles and small gates fill their warps with tokens.  A call that one
// cluster of blocks gets through is one launch without a workspace: the blocks read one
// another's sums from shared memory.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mgg {
namespace {

constexpr int kFwdThreads = 512, kBwdThreads = 256;

struct BalanceParams {
  const void* logits;
  long long ldl;
  const int32_t* ids;
  const uint8_t* mask;
  int T, E, k, len, sequences;  // len: tokens of a sequence
  int lanes;
  int chunks, rows;             // of a sequence: blocks, and tokens of one
  bool joined;                  // the blocks are one cluster, which finishes by itself
  float* sums;                  // [sequences * chunks][E]
  int32_t* hits;                // [sequences * chunks][E]
  int32_t* tokens;              // [sequences * chunks]
  int* ticket;
  float* loss;
  int32_t* counts;
  float* slope;
  float* parts;                 // the joining blocks' shares of the loss
  const float* dloss;
  void* dlogits;
  int32_t* dev_status;
};

// VEC elements at p, as floats; 16-byte aligned where VEC > 1
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  if constexpr (VEC == 1) {
    v[0] = static_cast<float>(*p);
  } else if constexpr (sizeof(T) == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
  if constexpr (VEC == 1) {
    *p = static_cast<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                                              cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
  }
}

// One instruction each, within 2 ulp (a probability is as good as its logit's f32
// rounding; with expf and a division the sigmoids took 35 instructions an element,
// 14 us of 16384 x 256).
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// v joined over a token's lanes (WARP: all 32, as with more than one piece a lane; a
// loop over their number cost a third of the instructions).
template <bool WARP, typename F>
__device__ __forceinline__ float over_lanes(float v, int lanes, F join) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2)
    if (WARP || o < lanes) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A token's logits (NV pieces of VEC in each of its lanes) to scores s and the
// inverse of their sum over the token: p = s r.  rest[]: of sigmoid scores 1 - a_te,
// else left.  As in the choice of the experts NaN, -inf and the type's lowest value
// mask an expert (s = 0) and +inf is the largest finite number.  Sigmoids are taken
// relative to the token's largest where that is below a half (c = min(0, top)):
// a e^-c = 1 / (e^c + e^(c - z)), so that a token whose scores all vanish in f32
// keeps its distribution.
template <typename T, bool SOFTMAX, bool WARP, int N>
__device__ __forceinline__ float scores(float (&z)[N], float (&rest)[SOFTMAX ? 1 : N], int lanes) {
  constexpr float kLow = sizeof(T) == 4 ? -3.402823466e38f : -3.389531390e38f;
  constexpr float kMost = 3.402823466e38f;
  constexpr float kLog2e = 1.4426950408889634f;
  float top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    z[i] = z[i] > kLow ? SOFTMAX ? fminf(z[i], kMost) : z[i] : -INFINITY;
    top = fmaxf(top, z[i]);
  }
  top = over_lanes<WARP>(top, lanes, [](float a, float b) { return fmaxf(a, b); });
  if constexpr (SOFTMAX) {
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      z[i] = ex2((z[i] - ref) * kLog2e);
      sum += z[i];
    }
  } else {
    const float c = top == -INFINITY ? 0.f : fminf(top, 0.f), ec = ex2(c * kLog2e);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool open = z[i] != -INFINITY;
      // (2^126 stands for all that is larger: its reciprocal is still a number)
      const float e = ex2(fminf((c - z[i]) * kLog2e, 126.f));
      const float r = rcp(ec + e);
      rest[i] = e * r;  // 1 - a without its cancellation
      z[i] = open ? r : 0.f;
      sum += z[i];
    }
  }
  sum = over_lanes<WARP>(sum, lanes, [](float a, float b) { return a + b; });
  return sum > 0.f ? __fdividef(1.f, sum) : 0.f;
}

// NV pieces of a row, `stride` elements apart, those from `width` on as `fill`.
template <typename T, int VEC, int NV>
__device__ __forceinline__ void load_row(const T* row, float fill, int width, int stride, float* v) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (j * stride < width) {
      load_vec<T, VEC>(row + j * stride, v + j * VEC);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j * VEC + i] = fill;
    }
  }
}

// E hits / (k n^2 live), 0 of a sequence without tokens
__device__ __forceinline__ float slope_of(int hits, int E, int k, int n, int live) {
  if (n == 0) return 0.f;
  return static_cast<float>(hits) * (static_cast<float>(E) / static_cast<float>(k)) /
         (static_cast<float>(n) * static_cast<float>(n)) / static_cast<float>(live);
}

constexpr int kCluster = 8;  // blocks of the one launch, at most

// tokens that a lane has in flight
template <int N>
constexpr int kUnroll = N >= 32 ? 1 : N >= 16 ? 2 : 4;

template <typename T, bool SOFTMAX, int VEC, int NV>
__global__ void __launch_bounds__(kFwdThreads) balance_sums_kernel(const BalanceParams p) {
  constexpr int N = VEC * NV, U = kUnroll<N>;
  constexpr int kWarps = kFwdThreads / 32;
  __shared__ float sums[kWarps / 2 * 1024];
  __shared__ int hits[1024];
  __shared__ int tokens;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seq = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const int t0 = seq * p.len + chunk * p.rows, t1 = min(t0 + p.rows, (seq + 1) * p.len);
  if (blockIdx.x == 0 && threadIdx.x == 0 && !p.joined) *p.ticket = 0;
  for (int e = threadIdx.x; e < p.E; e += kFwdThreads) hits[e] = 0;
  if (threadIdx.x == 0) tokens = 0;
  // the choices of the block's tokens, those that count; each thread's first one is read
  // ahead of the logits
  const int choices = (t1 - t0) * p.k;
  auto choice = [&](int i, int* e) {
    *e = p.ids[static_cast<long long>(t0) * p.k + i];
    return !p.mask || p.mask[t0 + i / p.k] != 0;
  };
  int first = 0;
  const bool any = static_cast<int>(threadIdx.x) < choices && choice(threadIdx.x, &first);
  const int sub = lane & (p.lanes - 1), place = lane / p.lanes;  // in the token, of the token in the warp
  const int per = 32 / p.lanes, step = kWarps * per;
  const int width = p.E - sub * VEC;  // columns from this lane's first on
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  int mine = 0;
  for (int tb = t0 + warp * per; tb < t1; tb += U * step) {  // (the same in every lane of a warp)
    float z[U][N];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(tb + u * step + place, t1 - 1);  // (past the end: a token that is not used)
      on[u] = tb + u * step + place < t1 && (!p.mask || p.mask[t]);
      load_row<T, VEC, NV>(static_cast<const T*>(p.logits) + t * p.ldl + sub * VEC, -INFINITY, width, VEC * p.lanes,
                           z[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float rest[SOFTMAX ? 1 : N];
      const float r = scores<T, SOFTMAX, (NV > 1), N>(z[u], rest, p.lanes);
      const float w = on[u] ? r : 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(z[u][i], w, acc[i]);
      mine += on[u] && sub == 0;
    }
  }
  for (int o = p.lanes; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  __syncthreads();  // (hits, tokens are zero)
  if (lane == 0 && mine) atomicAdd(&tokens, mine);
  auto count = [&](bool on, int e) {
    if (!on) return;
    if (e < 0 || e >= p.E)
      atomicOr(p.dev_status, kDevBadExpertId);
    else
      atomicAdd(&hits[e], 1);
  };
  // (four on their way at a time: 16384 choices a block 11.8 to 9.4 us)
  count(any, first);
  for (int i = threadIdx.x + kFwdThreads; i < choices; i += 4 * kFwdThreads) {
    int e[4];
    bool on[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) on[u] = i + u * kFwdThreads < choices && choice(i + u * kFwdThreads, &e[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u) count(on[u], e[u]);
  }
  // the warps' sums meet in two steps, in the warps' order
  auto put = [&](int w) {
    if (lane < p.lanes)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = ((i / VEC) * p.lanes + sub) * VEC + i % VEC;
        if (e < p.E) sums[w * p.E + e] = acc[i];
      }
  };
  if (warp >= kWarps / 2) put(warp - kWarps / 2);
  __syncthreads();
  if (warp < kWarps / 2 && lane < p.lanes) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = ((i / VEC) * p.lanes + sub) * VEC + i % VEC;
      if (e < p.E) acc[i] += sums[warp * p.E + e];
    }
  }
  __syncthreads();
  if (warp < kWarps / 2) put(warp);
  __syncthreads();
  const long long out = static_cast<long long>(blockIdx.x) * p.E;
  for (int e = threadIdx.x; e < p.E; e += kFwdThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps / 2; ++w) s += sums[w * p.E + e];
    if (p.joined) {
      sums[e] = s;  // (which no other thread reads before the barrier)
    } else {
      p.sums[out + e] = s;
      p.hits[out + e] = hits[e];
    }
  }
  if (!p.joined) {
    if (threadIdx.x == 0) p.tokens[blockIdx.x] = tokens;
    return;
  }
  // the cluster's blocks share the columns out and read one another's sums
  __shared__ float shares[kWarps], total[kCluster];
  __shared__ int s_n[kCluster], s_live;
  const int rank = blockIdx.x, blocks = gridDim.x;
  cluster_sync_all();
  if (warp == 0) {
    const int mine = lane < blocks ? ld_cluster_s32(mapa_shared(smem_u32(&tokens), lane)) : 0;
    int n = 0;
    for (int c = 0; c < p.chunks; ++c) n += __shfl_sync(0xffffffffu, mine, (lane * p.chunks + c) & 31);
    if (lane < p.sequences) s_n[lane] = n;
    const uint32_t live = __ballot_sync(0xffffffffu, lane < p.sequences && n != 0);
    if (lane == 0) s_live = __popc(live);
  }
  __syncthreads();
  float share = 0.f;
  for (int i = rank * kFwdThreads + threadIdx.x; i < p.sequences * p.E; i += blocks * kFwdThreads) {
    const int b = i / p.E, e = i - b * p.E;
    float f[kCluster];
    int h[kCluster];
#pragma unroll
    for (int c = 0; c < kCluster; ++c)
      if (c < p.chunks) {
        f[c] = ld_cluster_f32(mapa_shared(smem_u32(&sums[e]), b * p.chunks + c));
        h[c] = ld_cluster_s32(mapa_shared(smem_u32(&hits[e]), b * p.chunks + c));
      }
    float sum = 0.f;
    int hit = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c)
      if (c < p.chunks) sum += f[c], hit += h[c];
    const float slope = slope_of(hit, p.E, p.k, s_n[b], s_live);
    p.counts[i] = hit;
    p.slope[i] = slope;
    share += slope * sum;
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) share += __shfl_xor_sync(0xffffffffu, share, o);
  if (lane == 0) shares[warp] = share;
  __syncthreads();
  if (threadIdx.x == 0) {
    share = 0.f;
    for (int w = 0; w < kWarps; ++w) share += shares[w];
    st_cluster_s32(mapa_shared(smem_u32(&total[rank]), 0), __float_as_int(share));
  }
  cluster_sync_all();  // (no block leaves before the others have read its sums)
  if (rank == 0 && threadIdx.x == 0) {
    share = 0.f;
    for (int r = 0; r < blocks; ++r) share += total[r];
    *p.loss = share;
  }
}

// An item is 32 experts of one sequence: a lane each, the chunks dealt out to the
// warps, which read theirs at once: 8 warps up to 80 chunks, 32 beyond (38 chunks of 8
// sequences x 256 10.3 us with 8, 11.1 with 32; 304 of 16384 x 8 10.3 and 6.9).
constexpr int kJoinFew = 8, kJoinMany = 32, kJoinAhead = 10;
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32) balance_join_kernel(const BalanceParams p) {
  constexpr int kThreads = WARPS * 32;
  __shared__ float s_sum[WARPS][32];
  __shared__ int s_hit[WARPS][32];
  __shared__ int s_n[WARPS], s_live[WARPS];
  __shared__ bool last;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cols = cdiv(p.E, 32), items = cols * p.sequences;
  int live = 0;  // sequences with tokens
  if (p.chunks == 1) {
    for (int b = threadIdx.x; b < p.sequences; b += kThreads) live += p.tokens[b] != 0;
  } else if (p.sequences > 1) {  // (few: a warp each)
    for (int b = warp; b < p.sequences; b += WARPS) {
      bool any = false;
      for (int c = lane; c < p.chunks; c += 32) any |= p.tokens[b * p.chunks + c] != 0;
      live += __any_sync(0xffffffffu, any) && lane == 0;
    }
  }
  live = __reduce_add_sync(0xffffffffu, live);
  if (lane == 0) s_live[warp] = live;
  float share = 0.f;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int b = it / cols, e = (it % cols) * 32 + lane;
    float sum = 0.f;
    int hit = 0, n = 0;
    for (int c = threadIdx.x; c < p.chunks; c += kThreads) n += p.tokens[b * p.chunks + c];
    for (int c = warp; c < p.chunks; c += kJoinAhead * WARPS) {
      float f[kJoinAhead];
      int h[kJoinAhead];
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) {
        const bool any = c + WARPS * u < p.chunks && e < p.E;
        const long long at = (static_cast<long long>(b) * p.chunks + c + WARPS * u) * p.E + e;
        f[u] = any ? p.sums[at] : 0.f;
        h[u] = any ? p.hits[at] : 0;
      }
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) sum += f[u], hit += h[u];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    s_sum[warp][lane] = sum;
    s_hit[warp][lane] = hit;
    if (lane == 0) s_n[warp] = n;
    __syncthreads();
    if (warp == 0) {
      live = __reduce_add_sync(0xffffffffu, lane < WARPS ? s_live[lane] : 0);
      n = __reduce_add_sync(0xffffffffu, lane < WARPS ? s_n[lane] : 0);
      if (p.sequences == 1) live = n != 0;
      sum = 0.f, hit = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) sum += s_sum[w][lane], hit += s_hit[w][lane];
      const float slope = slope_of(hit, p.E, p.k, n, live);
      if (e < p.E) {
        p.counts[static_cast<long long>(b) * p.E + e] = hit;
        p.slope[static_cast<long long>(b) * p.E + e] = slope;
        share += slope * sum;
      }
    }
    __syncthreads();
  }
  if (warp == 0) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) share += __shfl_xor_sync(0xffffffffu, share, o);
    if (gridDim.x == 1) {
      if (lane == 0) *p.loss = share;
      last = false;
    } else if (lane == 0) {
      p.parts[blockIdx.x] = share;
      __threadfence();
      last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
  }
  __syncthreads();
  if (!last || warp) return;
  __threadfence();
  float sum = 0.f;
  for (int i = lane; i < static_cast<int>(gridDim.x); i += 32) sum += __ldcg(p.parts + i);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) *p.loss = sum;
}

template <typename T, bool SOFTMAX, int VEC, int NV>
__global__ void __launch_bounds__(kBwdThreads, VEC* NV <= 8 ? 4 : 1) balance_grad_kernel(const BalanceParams p) {
  constexpr int N = VEC * NV, U = N >= 16 ? 1 : 2;
  constexpr int SV = VEC > 1 ? 4 : 1;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane & (p.lanes - 1), place = lane / p.lanes, per = 32 / p.lanes;
  const int warps = gridDim.x * (kBwdThreads / 32), step = warps * per;
  const int width = p.E - sub * VEC, stride = VEC * p.lanes;
  const float g = *p.dloss;
  for (int tb = (blockIdx.x * (kBwdThreads / 32) + warp) * per; tb < p.T; tb += U * step) {
    float z[U][N];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(tb + u * step + place, p.T - 1);  // (past the end: a token that is not stored)
      on[u] = !p.mask || p.mask[t];
      load_row<T, VEC, NV>(static_cast<const T*>(p.logits) + t * p.ldl + sub * VEC, -INFINITY, width, stride, z[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u * step + place;
      // (the same rows again and again: they lie in L1)
      const float* slope = p.slope + sub * VEC;
      if (p.sequences > 1) slope += static_cast<long long>(min(t, p.T - 1) / p.len) * p.E;
      float s[N];
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; i += SV) {
          if (j * stride < width) {
            load_vec<float, SV>(slope + j * stride + i, &s[j * VEC + i]);
          } else {
#pragma unroll
            for (int q = 0; q < SV; ++q) s[j * VEC + i + q] = 0.f;
          }
        }
      float rest[SOFTMAX ? 1 : N];
      const float r = scores<T, SOFTMAX, (NV > 1), N>(z[u], rest, p.lanes);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) dot = fmaf(z[u][i], s[i], dot);
      dot = over_lanes<(NV > 1)>(dot, p.lanes, [](float a, float b) { return a + b; });
      dot *= r;
      const float w = on[u] ? r * g : 0.f;
      if (t >= p.T) continue;
      T* out = static_cast<T*>(p.dlogits) + static_cast<long long>(t) * p.E + sub * VEC;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float d = (z[u][i] * w) * (s[i] - dot);
        if constexpr (!SOFTMAX) d *= rest[i];
        z[u][i] = d;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j * stride < width) store_vec<T, VEC>(out + j * stride, &z[u][j * VEC]);
    }
  }
}

// ---------------------------------------------------------------- host
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Blocks of a sequence's sums: one cluster of eight in all up to 131072 logits
// (*joined), else two an SM, of at least 32 tokens each.  In a graph and called one
// after the other, us:
//   logits        one block   one cluster   two launches
//   512 x 8       4.4, 5.3    4.5, 5.2      5.9, 8.4
//   1024 x 64    18.4, 18.8   5.5, 5.7      9.0, 9.0
//   16384 x 8    33.5, 34.0   7.0, 7.2      6.8, 8.4
//   2048 x 64    33.8, 34.2   7.2, 7.6      9.1, 9.1
//   4096 x 64    64.6, 65.0  11.5, 11.7     9.2, 9.9
int plan_chunks(int T, int E, int sequences, bool* joined) {
  const int len = T / sequences;
  const long long n = static_cast<long long>(T) * E;
  *joined = n <= 131072 && sequences <= kCluster && (sequences & (sequences - 1)) == 0;
  if (*joined) return kCluster / sequences;
  return std::max(1, std::min(cdiv(2 * num_sms(), sequences), cdiv(len, 32)));
}

// The widest pieces that every row starts on; then the lanes of a token.
template <typename F>
cudaError_t by_layout(const BalanceArgs& a, bool grads, int* lanes, F&& f) {
  const int wide = a.f32 ? 4 : 8;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) |
                       (grads ? reinterpret_cast<uintptr_t>(a.dlogits) | reinterpret_cast<uintptr_t>(a.slope) : 0);
  const int vec = at % 16 == 0 && a.ldl % wide == 0 && a.E % wide == 0 ? wide : 1;
  *lanes = 1;
  while (*lanes < 32 && *lanes * vec < a.E) *lanes *= 2;
  const int nv = cdiv(a.E, *lanes * vec);
  if (vec == 1) {
    if (nv <= 1) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 1>());
    if (nv <= 2) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 2>());
    if (nv <= 4) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
    if (nv <= 8) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
    if (nv <= 16) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 1>(), std::integral_constant<int, 32>());
  }
  if (nv <= 1) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 1>());
  if (nv <= 2) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 2>());
  if (nv <= 4) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 2>(), std::integral_constant<int, 8>());
}

// f(type, scoring) for the logits' type and the scoring
template <typename F>
cudaError_t by_type(const BalanceArgs& a, F&& f) {
  if (a.f32) return a.softmax ? f(float(), std::true_type()) : f(float(), std::false_type());
  return a.softmax ? f(__nv_bfloat16(), std::true_type()) : f(__nv_bfloat16(), std::false_type());
}

BalanceParams params(const BalanceArgs& a) {
  BalanceParams p{};
  p.logits = a.logits, p.ldl = a.ldl, p.ids = a.ids, p.mask = a.mask;
  p.T = a.T, p.E = a.E, p.k = a.k, p.sequences = a.sequences, p.len = a.T / a.sequences;
  p.loss = a.loss, p.counts = a.counts, p.slope = a.slope;
  p.dloss = a.dloss, p.dlogits = a.dlogits, p.dev_status = a.dev_status;
  return p;
}

}  // namespace

constexpr int kJoinBlocks = 1024;  // at most

size_t balance_ws_bytes(int T, int E, int sequences) {
  bool joined;
  const size_t blocks = static_cast<size_t>(sequences) * plan_chunks(T, E, sequences, &joined);
  if (joined) return 0;
  return 2 * round256(blocks * E * 4) + round256(blocks * 4) + round256(kJoinBlocks * 4) + 256;
}

cudaError_t launch_balance(const BalanceArgs& a, void* ws, cudaStream_t st) {
  BalanceParams p = params(a);
  p.chunks = plan_chunks(a.T, a.E, a.sequences, &p.joined);
  p.rows = cdiv(p.len, p.chunks);
  const size_t blocks = static_cast<size_t>(a.sequences) * p.chunks;
  char* at = static_cast<char*>(ws);
  p.sums = reinterpret_cast<float*>(at), at += round256(blocks * a.E * 4);
  p.hits = reinterpret_cast<int32_t*>(at), at += round256(blocks * a.E * 4);
  p.tokens = reinterpret_cast<int32_t*>(at), at += round256(blocks * 4);
  p.parts = reinterpret_cast<float*>(at), at += round256(kJoinBlocks * 4);
  p.ticket = reinterpret_cast<int*>(at);
  cudaError_t e = by_type(a, [&](auto type, auto softmax) {
    using T = decltype(type);
    return by_layout(a, false, &p.lanes, [&](auto wide, auto nv) {
      constexpr int VEC = wide() == 1 ? 1 : 16 / sizeof(T), NV = VEC == 8 && nv() > 4 ? 4 : nv();
      const dim3 grid(static_cast<unsigned>(blocks)), block(kFwdThreads);
      if (p.joined)
        return launch_pdl_clusters(balance_sums_kernel<T, softmax(), VEC, NV>, grid, block, 0, static_cast<int>(blocks),
                                   st, p);
      return launch_pdl(balance_sums_kernel<T, softmax(), VEC, NV>, grid, block, 0, st, p);
    });
  });
  if (e != cudaSuccess || p.joined) return e;
  const long long items = static_cast<long long>(cdiv(a.E, 32)) * a.sequences;
  const dim3 grid(static_cast<unsigned>(std::min<long long>(items, kJoinBlocks)));
  return p.chunks <= kJoinFew * kJoinAhead ? launch_pdl(balance_join_kernel<kJoinFew>, grid, dim3(kJoinFew * 32), 0, st, p)
                                           : launch_pdl(balance_join_kernel<kJoinMany>, grid, dim3(kJoinMany * 32), 0, st, p);
}

cudaError_t launch_balance_bwd(const BalanceArgs& a, cudaStream_t st) {
  BalanceParams p = params(a);
  return by_type(a, [&](auto type, auto softmax) {
    using T = decltype(type);
    return by_layout(a, true, &p.lanes, [&](auto wide, auto nv) {
      constexpr int VEC = wide() == 1 ? 1 : 16 / sizeof(T), NV = VEC == 8 && nv() > 4 ? 4 : nv();
      const int per = kBwdThreads / p.lanes;  // tokens of a block and step
      const int blocks = std::max(1, std::min(cdiv(a.T, per), 8 * num_sms()));
      return launch_pdl(balance_grad_kernel<T, softmax(), VEC, NV>, dim3(blocks), dim3(kBwdThreads), 0, st, p);
    });
  });
}

}  // namespace mgg
