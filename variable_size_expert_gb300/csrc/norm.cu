// Layer norm over the last dimension, forward and backward.
//
//   mean = sum_k x / K,  rstd = (sum_k (x - mean)^2 / K + eps)^-1/2,
//   y = (x - mean) rstd w + b
//   with g = dy w and xh = (x - mean) rstd:
//   dx = rstd (g - sum_k g / K - xh sum_k (g xh) / K)
//   dw = sum_t dy xh,  db = sum_t dy
//
// Both directions are bound by HBM: the row is read once and kept in
// registers (the variance is a second pass over the registers, so no
// cancellation of large means), the result written once.  All sums are f32.
//
// Backward: dw and db run down the columns while dx runs along the rows.  A
// group of TPR threads owns a row, each thread the same columns of every row
// its group visits, so the column sums stay in registers for the whole
// kernel; the next row's values are requested before the current row's
// reduction, whose barrier would otherwise drain the loads in flight.  At
// the end the groups of a block add up in shared memory in group order and
// the block writes one partial row; a second kernel adds the partial rows in
// block order.  No atomics: equal inputs give equal bits.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mgg {
namespace {

constexpr int kRegRow = 16384;  // longest row kept in registers

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// VEC consecutive elements as they lie in memory: 8 where both sides are bf16
// and 4 where one is f32 (16 bytes of the wider), single elements for VEC = 1.
template <typename T, int VEC>
struct Raw {
  T v[VEC];
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 q;
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 q;
};
template <>
struct Raw<float, 4> {
  float4 q;
};
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
  Raw<T, VEC> r;
  if constexpr (VEC == 1)
    r.v[0] = *p;
  else
    r = *reinterpret_cast<const Raw<T, VEC>*>(p);
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Raw<T, VEC>& r, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_f<T>(r.v[0]);
  } else if constexpr (sizeof(T) == 4) {
    f[0] = r.q.x, f[1] = r.q.y, f[2] = r.q.z, f[3] = r.q.w;
  } else {
    uint32_t u[VEC / 2];
    u[0] = r.q.x, u[1] = r.q.y;
    if constexpr (VEC == 8) u[2] = r.q.z, u[3] = r.q.w;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_f(T* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(f[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint2*>(p) =
        make_uint2(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]));
  } else {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]),
                   pack_bf16x2_rn(f[4], f[5]), pack_bf16x2_rn(f[6], f[7]));
  }
}
// the weight or bias (f32 or bf16), VEC elements from column c
template <int VEC>
__device__ __forceinline__ void load_param(const void* w, bool w_f32, int c, float (&f)[VEC]) {
  if (!w_f32) {
    unpack<__nv_bfloat16, VEC>(
        load_raw<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w) + c), f);
  } else if constexpr (VEC == 8) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
    const float4 a = q[0], b = q[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack<float, VEC>(load_raw<float, VEC>(static_cast<const float*>(w) + c), f);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the TPR threads of a row group (TPR a multiple of 32); the result
// in every thread.  `slots` holds TPR/32 values per call site and parity.
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float* slots, int group, int tig) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    if ((tig & 31) == 0) slots[tig >> 5] = v;
    bar_named(1 + group, TPR);
    v = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) v += slots[w];
  }
  return v;
}

// ---------------------------------------------------------------- forward
template <typename XT, typename YT, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    norm_fwd_kernel(const XT* x, long long ldx, const void* w, const void* b, bool w_f32, int T,
                    int K, float eps, YT* y, float* mean_out, float* rstd_out) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kGroups = kThreads / TPR;
  __shared__ float slots[2][kGroups][TPR / 32];
  const int group = threadIdx.x / TPR, tig = threadIdx.x % TPR;
  pdl_trigger();
  pdl_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kGroups + group;
  if (t >= T) return;  // whole groups leave: their barriers are their own
  const XT* xr = x + t * ldx;
  float f[NV][VEC];
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tig) * VEC;
    if (c < K) {
      unpack<XT, VEC>(load_raw<XT, VEC>(xr + c), f[j]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[j][i] = 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s += f[j][i];
  const float mean = group_sum<TPR>(s, slots[0][group], group, tig) / K;
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = (j * TPR + tig) * VEC < K;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      f[j][i] -= mean;
      if (in) q = fmaf(f[j][i], f[j][i], q);
    }
  }
  const float rstd = 1.f / sqrtf(group_sum<TPR>(q, slots[1][group], group, tig) / K + eps);
  if (tig == 0) {
    mean_out[t] = mean;
    rstd_out[t] = rstd;
  }
  YT* yr = y + t * K;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tig) * VEC;
    if (c < K) {
      float wv[VEC], o[VEC];
      load_param<VEC>(w, w_f32, c, wv);
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = f[j][i] * rstd * wv[i];
      if (b) {
        load_param<VEC>(b, w_f32, c, wv);
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] += wv[i];
      }
      store_f<YT, VEC>(yr + c, o);
    }
  }
}

// Rows longer than the registers hold: the row is read three times (the
// later reads come from L2).
template <typename XT, typename YT>
__global__ void __launch_bounds__(512)
    norm_fwd_long_kernel(const XT* x, long long ldx, const void* w, const void* b, bool w_f32,
                         int T, int K, float eps, YT* y, float* mean_out, float* rstd_out) {
  __shared__ float slots[2][16];
  pdl_trigger();
  pdl_wait();
  const long long t = blockIdx.x;
  const XT* xr = x + t * ldx;
  float s = 0.f;
  for (int c = threadIdx.x; c < K; c += 512) s += to_f<XT>(xr[c]);
  const float mean = group_sum<512>(s, slots[0], 0, threadIdx.x) / K;
  float q = 0.f;
  for (int c = threadIdx.x; c < K; c += 512) {
    const float d = to_f<XT>(xr[c]) - mean;
    q = fmaf(d, d, q);
  }
  const float rstd = 1.f / sqrtf(group_sum<512>(q, slots[1], 0, threadIdx.x) / K + eps);
  if (threadIdx.x == 0) {
    mean_out[t] = mean;
    rstd_out[t] = rstd;
  }
  for (int c = threadIdx.x; c < K; c += 512) {
    float wv[1], bv[1] = {0.f};
    load_param<1>(w, w_f32, c, wv);
    if (b) load_param<1>(b, w_f32, c, bv);
    y[t * K + c] = from_f<YT>((to_f<XT>(xr[c]) - mean) * rstd * wv[0] + bv[0]);
  }
}

// ---------------------------------------------------------------- backward
constexpr int kBwdThreads = 512;

template <typename XT, typename YT, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(TPR > kBwdThreads ? TPR : kBwdThreads)
    norm_bwd_kernel(const YT* dy, const XT* x, long long ldx, const void* w, bool w_f32,
                    const float* mean, const float* rstd, int T, int K, XT* dx, float* part) {
  constexpr int kThreads = TPR > kBwdThreads ? TPR : kBwdThreads;
  constexpr int kGroups = kThreads / TPR;
  __shared__ float slots[2][2][kGroups][TPR / 32];
  const int group = threadIdx.x / TPR, tig = threadIdx.x % TPR;
  pdl_trigger();
  pdl_wait();
  const int step = gridDim.x * kGroups;
  float wv[NV][VEC], aw[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tig) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) wv[j][i] = aw[j][i] = ab[j][i] = 0.f;
    if (c < K) load_param<VEC>(w, w_f32, c, wv[j]);
  }
  Raw<XT, VEC> rx[NV];
  Raw<YT, VEC> rg[NV];
  float m = 0.f, r = 0.f;
  auto fetch = [&](long long t) {
    m = mean[t];
    r = rstd[t];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tig) * VEC;
      if (c < K) {
        rx[j] = load_raw<XT, VEC>(x + t * ldx + c);
        rg[j] = load_raw<YT, VEC>(dy + t * K + c);
      }
    }
  };
  long long t = static_cast<long long>(blockIdx.x) * kGroups + group;
  if (t < T) fetch(t);
  for (int par = 0; t < T; t += step, par ^= 1) {
    const float rs = r;
    float xh[NV][VEC], g[NV][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = (j * TPR + tig) * VEC < K;
      if (in) {
        unpack<XT, VEC>(rx[j], xh[j]);
        unpack<YT, VEC>(rg[j], g[j]);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (!in) xh[j][i] = g[j][i] = 0.f;
        else xh[j][i] = (xh[j][i] - m) * rs;
        aw[j][i] = fmaf(g[j][i], xh[j][i], aw[j][i]);
        ab[j][i] += g[j][i];
        g[j][i] *= wv[j][i];
        s1 += g[j][i];
        s2 = fmaf(g[j][i], xh[j][i], s2);
      }
    }
    if (t + step < T) fetch(t + step);
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (TPR > 32) {
      // two sums, one barrier: the slots alternate, so the next row's writes
      // cannot meet this row's reads
      if ((tig & 31) == 0) {
        slots[par][0][group][tig >> 5] = s1;
        slots[par][1][group][tig >> 5] = s2;
      }
      bar_named(1 + group, TPR);
      s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < TPR / 32; ++i) {
        s1 += slots[par][0][group][i];
        s2 += slots[par][1][group][i];
      }
    }
    s1 /= K;
    s2 /= K;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tig) * VEC;
      if (c < K) {
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = rs * (g[j][i] - s1 - xh[j][i] * s2);
        store_f<XT, VEC>(dx + t * K + c, o);
      }
    }
  }
  // the block's partial row: groups added in order
  extern __shared__ float acc[];  // [2][K] when the block has several groups
  float* pw = part + static_cast<long long>(blockIdx.x) * K;
  float* pb = part + static_cast<long long>(gridDim.x + blockIdx.x) * K;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tig) * VEC;
      if (c < K) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          pw[c + i] = aw[j][i];
          pb[c + i] = ab[j][i];
        }
      }
    }
  } else {
    for (int gi = 0; gi < kGroups; ++gi) {
      if (group == gi) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (j * TPR + tig) * VEC;
          if (c < K) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              acc[c + i] = gi ? acc[c + i] + aw[j][i] : aw[j][i];
              acc[K + c + i] = gi ? acc[K + c + i] + ab[j][i] : ab[j][i];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < K; c += kThreads) {
      pw[c] = acc[c];
      pb[c] = acc[K + c];
    }
  }
}

// The same with the rows to come on their way through shared memory: each
// thread copies its own pieces of the next rows (cp.async, D rows ahead) into
// slots that only it reads, so the copies need no barrier and the loads of D
// rows are in flight whatever the reduction waits for.  The register version
// above keeps one row in flight: 135 us instead of 68 for 8191 x 7163 bf16.
//
// SHIFT: rows that do not start on VEC-element boundaries (odd widths).  Where
// x, dy and dx share each row's residue m (row t starts m = t K mod VEC
// elements past a boundary), a thread reads the aligned pieces that cover the
// row, whose columns start at -m; pieces at the row's ends overlap the rows
// beside it (never another 16-byte word than the row's own) and their foreign
// elements are left out.  The residue repeats every VEC / gcd(K, VEC) rows, a
// divisor of 8: each group takes rows of one residue, so that its threads keep
// their columns and the column sums stay in registers.
// Row slots: three of two f32 rows fill the shared memory, four of less.
template <typename XT, typename YT>
__host__ __device__ constexpr int pipe_depth() {
  return sizeof(XT) + sizeof(YT) == 8 ? 3 : 4;
}
template <typename XT, typename YT, int VEC, int TPR, int NV, bool SHIFT>
__global__ void __launch_bounds__(TPR > kBwdThreads ? TPR : kBwdThreads)
    norm_bwd_pipe_kernel(const YT* dy, const XT* x, long long ldx, const void* w, bool w_f32,
                         const float* mean, const float* rstd, int T, int K, XT* dx, float* part,
                         int period) {
  constexpr int kThreads = TPR > kBwdThreads ? TPR : kBwdThreads;
  constexpr int kGroups = kThreads / TPR;
  constexpr int XB = VEC * sizeof(XT), YB = VEC * sizeof(YT);
  __shared__ float slots[2][2][kGroups][TPR / 32];
  extern __shared__ __align__(16) uint8_t ring[];  // [depth][NV]([threads] x, [threads] dy)
  const int group = threadIdx.x / TPR, tig = threadIdx.x % TPR;
  constexpr int kRow = kThreads * (XB + YB);  // bytes of one j of one row slot
  const uint32_t mine_x = smem_u32(ring) + threadIdx.x * XB;
  const uint32_t mine_y = smem_u32(ring) + kThreads * XB + threadIdx.x * YB;
  pdl_trigger();
  pdl_wait();
  const int gid = blockIdx.x * kGroups + group, gn = gridDim.x * kGroups;
  // this group's rows: gid mod period, then every gn-th (gn is a multiple of period)
  const int first = SHIFT ? gid % period + period * (gid / period) : gid;
  const int step = gn;
  const int m = SHIFT ? static_cast<int>((static_cast<long long>(first) * K) % VEC) : 0;
  float wv[NV][VEC], aw[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tig) * VEC - m;
#pragma unroll
    for (int i = 0; i < VEC; ++i) wv[j][i] = aw[j][i] = ab[j][i] = 0.f;
    if constexpr (!SHIFT) {
      if (c < K) load_param<VEC>(w, w_f32, c, wv[j]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (c + i >= 0 && c + i < K) {
          float one[1];
          load_param<1>(w, w_f32, c + i, one);
          wv[j][i] = one[0];
        }
    }
  }
  auto copy = [&](long long t, int slot) {
    if (t < T) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + tig) * VEC - m;
        if (c >= K) continue;
        const uint32_t o = (slot * NV + j) * kRow;
        const XT* xs = x + t * ldx + c;
        const YT* ys = dy + t * K + c;
        if constexpr (XB == 16)
          cp_async_16_full(mine_x + o, xs);
        else
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(mine_x + o), "l"(xs) : "memory");
        if constexpr (YB == 16)
          cp_async_16_full(mine_y + o, ys);
        else
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(mine_y + o), "l"(ys) : "memory");
      }
    }
    cp_async_commit();  // (an empty group past the last row keeps the count)
  };
  constexpr int depth = pipe_depth<XT, YT>(), D = depth - 1;  // slots, rows ahead
  long long t = first;
#pragma unroll
  for (int i = 0; i < D; ++i) copy(t + static_cast<long long>(i) * step, i);
  int slot = 0;
  for (int par = 0; t < T; t += step, par ^= 1) {
    copy(t + static_cast<long long>(D) * step, slot + D >= depth ? slot + D - depth : slot + D);
    const float mu = mean[t], rs = rstd[t];
    cp_async_wait<D>();
    float xh[NV][VEC], g[NV][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tig) * VEC - m;
      const uint8_t* at = ring + (slot * NV + j) * kRow;
      if (c < K) {
        unpack<XT, VEC>(*reinterpret_cast<const Raw<XT, VEC>*>(at + threadIdx.x * XB), xh[j]);
        unpack<YT, VEC>(*reinterpret_cast<const Raw<YT, VEC>*>(at + kThreads * XB + threadIdx.x * YB), g[j]);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (c >= K || (SHIFT && (c + i < 0 || c + i >= K))) xh[j][i] = g[j][i] = 0.f;
        else xh[j][i] = (xh[j][i] - mu) * rs;
        aw[j][i] = fmaf(g[j][i], xh[j][i], aw[j][i]);
        ab[j][i] += g[j][i];
        g[j][i] *= wv[j][i];
        s1 += g[j][i];
        s2 = fmaf(g[j][i], xh[j][i], s2);
      }
    }
    if (++slot == depth) slot = 0;
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (TPR > 32) {
      // two sums, one barrier: the slots alternate, so the next row's writes
      // cannot meet this row's reads
      if ((tig & 31) == 0) {
        slots[par][0][group][tig >> 5] = s1;
        slots[par][1][group][tig >> 5] = s2;
      }
      bar_named(1 + group, TPR);
      s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < TPR / 32; ++i) {
        s1 += slots[par][0][group][i];
        s2 += slots[par][1][group][i];
      }
    }
    s1 /= K;
    s2 /= K;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tig) * VEC - m;
      if (c >= K) continue;
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = rs * (g[j][i] - s1 - xh[j][i] * s2);
      if (!SHIFT || (c >= 0 && c + VEC <= K)) {
        store_f<XT, VEC>(dx + t * K + c, o);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (c + i >= 0 && c + i < K) dx[t * K + c + i] = from_f<XT>(o[i]);
      }
    }
  }
  // the block's partial row: groups added in order, over the ring
  cp_async_wait<0>();
  __syncthreads();
  float* acc = reinterpret_cast<float*>(ring);  // [2][K]
  float* pw = part + static_cast<long long>(blockIdx.x) * K;
  float* pb = part + static_cast<long long>(gridDim.x + blockIdx.x) * K;
  for (int gi = 0; gi < kGroups; ++gi) {
    if (group == gi) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + tig) * VEC - m;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if (c + i < 0 || c + i >= K) continue;
          acc[c + i] = gi ? acc[c + i] + aw[j][i] : aw[j][i];
          acc[K + c + i] = gi ? acc[K + c + i] + ab[j][i] : ab[j][i];
        }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < K; c += kThreads) {
    pw[c] = acc[c];
    pb[c] = acc[K + c];
  }
}

// Rows longer than the registers hold: dx row by row (two passes), and the
// column sums by blocks of 32 columns over a range of rows each.
template <typename XT, typename YT>
__global__ void __launch_bounds__(512)
    norm_bwd_long_dx_kernel(const YT* dy, const XT* x, long long ldx, const void* w, bool w_f32,
                            const float* mean, const float* rstd, int T, int K, XT* dx) {
  __shared__ float slots[2][16];
  pdl_trigger();
  pdl_wait();
  const long long t = blockIdx.x;
  const float m = mean[t], r = rstd[t];
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < K; c += 512) {
    float wv[1];
    load_param<1>(w, w_f32, c, wv);
    const float g = to_f<YT>(dy[t * K + c]) * wv[0];
    s1 += g;
    s2 = fmaf(g, (to_f<XT>(x[t * ldx + c]) - m) * r, s2);
  }
  s1 = group_sum<512>(s1, slots[0], 0, threadIdx.x) / K;
  s2 = group_sum<512>(s2, slots[1], 0, threadIdx.x) / K;
  for (int c = threadIdx.x; c < K; c += 512) {
    float wv[1];
    load_param<1>(w, w_f32, c, wv);
    const float xh = (to_f<XT>(x[t * ldx + c]) - m) * r;
    dx[t * K + c] = from_f<XT>(r * (to_f<YT>(dy[t * K + c]) * wv[0] - s1 - xh * s2));
  }
}
template <typename XT, typename YT>
__global__ void __launch_bounds__(256)
    norm_bwd_long_cols_kernel(const YT* dy, const XT* x, long long ldx, const float* mean,
                              const float* rstd, int T, int K, float* part) {
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= K) return;
  float aw = 0.f, ab = 0.f;
  for (long long t = blockIdx.y; t < T; t += gridDim.y) {
    const float g = to_f<YT>(dy[t * K + c]);
    aw = fmaf(g, (to_f<XT>(x[t * ldx + c]) - mean[t]) * rstd[t], aw);
    ab += g;
  }
  part[static_cast<long long>(blockIdx.y) * K + c] = aw;
  part[static_cast<long long>(gridDim.y + blockIdx.y) * K + c] = ab;
}

// Partial rows part[2][nb][K] -> dw, db, added in block order: 32 columns
// per block, 32 row lanes each summing every 32nd partial, then a tree.
__global__ void __launch_bounds__(1024)
    column_sums_kernel(const float* part, int nb, int K, void* dw, void* db, bool w_f32) {
  __shared__ float s[32][33];
  pdl_trigger();
  pdl_wait();
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  const float* p = part + static_cast<long long>(blockIdx.y) * nb * K;
  float v = 0.f;
  if (c < K)
    for (int i = ry; i < nb; i += 32) v += p[static_cast<long long>(i) * K + c];
  s[ry][cx] = v;
  __syncthreads();
  v = warp_sum(s[cx][ry]);  // warp ry: the 32 row lanes of column ry
  const int co = blockIdx.x * 32 + ry;
  void* out = blockIdx.y ? db : dw;
  if (cx == 0 && co < K && out) {
    if (w_f32)
      static_cast<float*>(out)[co] = v;
    else
      static_cast<__nv_bfloat16*>(out)[co] = __float2bfloat16_rn(v);
  }
}

}  // namespace

cudaError_t launch_column_sums(const float* part, int nb, int K, void* out0, void* out1,
                               bool out_f32, cudaStream_t st) {
  return launch_pdl(column_sums_kernel, dim3(cdiv(K, 32), out1 ? 2 : 1), dim3(1024), 0, st, part,
                    nb, K, out0, out1, out_f32);
}

namespace {

struct FwdArgs {
  const void* x;
  long long ldx;
  const void *w, *b;
  bool w_f32;
  int T, K;
  float eps;
  void* y;
  float *mean, *rstd;
};

template <typename XT, typename YT, int VEC, int TPR, int NV>
cudaError_t fwd_t(const FwdArgs& a, cudaStream_t st) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  return launch_pdl(norm_fwd_kernel<XT, YT, VEC, TPR, NV>, dim3(cdiv(a.T, kThreads / TPR)),
                    dim3(kThreads), 0, st, static_cast<const XT*>(a.x), a.ldx, a.w, a.b, a.w_f32,
                    a.T, a.K, a.eps, static_cast<YT*>(a.y), a.mean, a.rstd);
}

template <typename XT, typename YT>
cudaError_t fwd(const FwdArgs& a, bool vec, cudaStream_t st) {
  const int K = a.K;
  if (K > kRegRow)
    return launch_pdl(norm_fwd_long_kernel<XT, YT>, dim3(a.T), dim3(512), 0, st,
                      static_cast<const XT*>(a.x), a.ldx, a.w, a.b, a.w_f32, a.T, K, a.eps,
                      static_cast<YT*>(a.y), a.mean, a.rstd);
  if (vec) {
    // a warp per row up to 2048 columns (64 values a lane, no barrier), then
    // 16 values a thread
    constexpr int V = sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 : 4;
    if (K <= 512) return fwd_t<XT, YT, V, 32, 16 / V>(a, st);
    if (K <= 1024) return fwd_t<XT, YT, V, 32, 32 / V>(a, st);
    if (K <= 2048 && a.T >= 4 * num_sms()) return fwd_t<XT, YT, V, 32, 64 / V>(a, st);
    if (K <= 2048) return fwd_t<XT, YT, V, 128, 16 / V>(a, st);
    if (K <= 4096) return fwd_t<XT, YT, V, 256, 16 / V>(a, st);
    if (K <= 8192) return fwd_t<XT, YT, V, 512, 16 / V>(a, st);
    return fwd_t<XT, YT, V, 1024, 16 / V>(a, st);
  }
  if (K <= 512) return fwd_t<XT, YT, 1, 32, 16>(a, st);
  if (K <= 4096) return fwd_t<XT, YT, 1, 256, 16>(a, st);
  if (K <= 8192) return fwd_t<XT, YT, 1, 512, 16>(a, st);
  return fwd_t<XT, YT, 1, 1024, 16>(a, st);
}

struct BwdArgs {
  const void *dy, *x;
  long long ldx;
  const void* w;
  bool w_f32;
  const float *mean, *rstd;
  int T, K;
  void *dx, *dw, *db;
  float* part;
};

template <typename XT, typename YT, int TPR>
cudaError_t bwd_t(const BwdArgs& a, int* nb, cudaStream_t st) {
  constexpr int VEC = 1, NV = 16;
  constexpr int kThreads = TPR > kBwdThreads ? TPR : kBwdThreads;
  constexpr int kGroups = kThreads / TPR;
  *nb = std::min(norm_bwd_blocks(), cdiv(a.T, kGroups));
  const size_t smem = kGroups > 1 ? static_cast<size_t>(2) * a.K * 4 : 0;
  return launch_pdl(norm_bwd_kernel<XT, YT, VEC, TPR, NV>, dim3(*nb), dim3(kThreads), smem, st,
                    static_cast<const YT*>(a.dy), static_cast<const XT*>(a.x), a.ldx, a.w, a.w_f32,
                    a.mean, a.rstd, a.T, a.K, static_cast<XT*>(a.dx), a.part);
}

template <typename XT, typename YT, int TPR, bool SHIFT>
cudaError_t bwd_pipe_t(const BwdArgs& a, int* nb, cudaStream_t st) {
  constexpr int VEC = sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 : 4;
  constexpr int NV = 16 / VEC;
  constexpr int kThreads = TPR > kBwdThreads ? TPR : kBwdThreads;
  constexpr int kGroups = kThreads / TPR;
  constexpr size_t kRing = static_cast<size_t>(pipe_depth<XT, YT>()) * NV * kThreads * VEC * (sizeof(XT) + sizeof(YT));
  int period = 1;
  if (SHIFT)
    for (period = VEC; period > 1 && (static_cast<long long>(a.K) * (period / 2)) % VEC == 0;) period /= 2;
  // a multiple of eight blocks, so that the groups divide by any period
  *nb = std::max(8, std::min(norm_bwd_blocks(), cdiv(cdiv(a.T, kGroups), 8) * 8));
  const size_t smem = std::max(kRing, static_cast<size_t>(2) * a.K * 4);
  static bool done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  auto kern = norm_bwd_pipe_kernel<XT, YT, VEC, TPR, NV, SHIFT>;
  if (dev >= 64 || !done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = true;
  }
  return launch_pdl(kern, dim3(*nb), dim3(kThreads), smem, st, static_cast<const YT*>(a.dy),
                    static_cast<const XT*>(a.x), a.ldx, a.w, a.w_f32, a.mean, a.rstd, a.T, a.K,
                    static_cast<XT*>(a.dx), a.part, period);
}
// K: the row's columns, with SHIFT those of the pieces that cover it
template <typename XT, typename YT, bool SHIFT>
cudaError_t bwd_pipe(const BwdArgs& a, int* nb, cudaStream_t st) {
  constexpr int VEC = sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 : 4;
  const int K = a.K + (SHIFT ? VEC - 1 : 0);
  if (K <= 512) return bwd_pipe_t<XT, YT, 32, SHIFT>(a, nb, st);
  if (K <= 1024) return bwd_pipe_t<XT, YT, 64, SHIFT>(a, nb, st);
  if (K <= 2048) return bwd_pipe_t<XT, YT, 128, SHIFT>(a, nb, st);
  if (K <= 4096) return bwd_pipe_t<XT, YT, 256, SHIFT>(a, nb, st);
  return bwd_pipe_t<XT, YT, 512, SHIFT>(a, nb, st);
}

enum BwdPath { kByElement, kAligned, kShifted };

template <typename XT, typename YT>
cudaError_t bwd(const BwdArgs& a, BwdPath path, cudaStream_t st) {
  const int K = a.K;
  int nb = 0;
  cudaError_t e;
  if (K > kRegRow) {
    e = launch_pdl(norm_bwd_long_dx_kernel<XT, YT>, dim3(a.T), dim3(512), 0, st,
                   static_cast<const YT*>(a.dy), static_cast<const XT*>(a.x), a.ldx, a.w, a.w_f32,
                   a.mean, a.rstd, a.T, K, static_cast<XT*>(a.dx));
    if (e != cudaSuccess) return e;
    nb = std::min(norm_bwd_blocks(), a.T);
    e = launch_pdl(norm_bwd_long_cols_kernel<XT, YT>, dim3(cdiv(K, 256), nb), dim3(256), 0, st,
                   static_cast<const YT*>(a.dy), static_cast<const XT*>(a.x), a.ldx, a.mean,
                   a.rstd, a.T, K, a.part);
  } else if (path == kAligned && K <= 8192) {
    e = bwd_pipe<XT, YT, false>(a, &nb, st);
  } else if (path == kShifted && K <= 8192 - 7) {
    e = bwd_pipe<XT, YT, true>(a, &nb, st);
  } else {
    if (K <= 512) e = bwd_t<XT, YT, 32>(a, &nb, st);
    else if (K <= 2048) e = bwd_t<XT, YT, 128>(a, &nb, st);
    else if (K <= 8192) e = bwd_t<XT, YT, 512>(a, &nb, st);
    else e = bwd_t<XT, YT, 1024>(a, &nb, st);
  }
  if (e != cudaSuccess) return e;
  return launch_column_sums(a.part, nb, K, a.dw, a.db, a.w_f32, st);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace


int norm_bwd_blocks() { return std::max(8, num_sms() / 8 * 8); }

// 16-byte accesses where every row of every operand starts on a 16-byte
// boundary, else element by element.
cudaError_t launch_norm_fwd(const void* x, bool x_f32, long long ldx, const void* w, const void* b,
                            bool w_f32, int T, int K, float eps, void* y, bool y_f32, float* mean,
                            float* rstd, cudaStream_t st) {
  const bool vec = K % 8 == 0 && ldx % 8 == 0 && aligned16(x) && aligned16(w) &&
                   (!b || aligned16(b)) && aligned16(y);
  const FwdArgs a{x, ldx, w, b, w_f32, T, K, eps, y, mean, rstd};
  using B = __nv_bfloat16;
  if (x_f32) return y_f32 ? fwd<float, float>(a, vec, st) : fwd<float, B>(a, vec, st);
  return y_f32 ? fwd<B, float>(a, vec, st) : fwd<B, B>(a, vec, st);
}

cudaError_t launch_norm_bwd(const void* dy, bool y_f32, const void* x, bool x_f32, long long ldx,
                            const void* w, bool w_f32, const float* mean, const float* rstd, int T,
                            int K, void* dx, void* dw, void* db, float* part, cudaStream_t st) {
  const int vec = x_f32 || y_f32 ? 4 : 8;
  BwdPath path = kByElement;
  if (aligned16(x) && aligned16(dy) && aligned16(dx)) {
    if (K % vec == 0 && ldx % vec == 0 && aligned16(w)) path = kAligned;
    else if (ldx % vec == K % vec) path = kShifted;
  }
  const BwdArgs a{dy, x, ldx, w, w_f32, mean, rstd, T, K, dx, dw, db, part};
  using B = __nv_bfloat16;
  if (x_f32) return y_f32 ? bwd<float, float>(a, path, st) : bwd<float, B>(a, path, st);
  return y_f32 ? bwd<B, float>(a, path, st) : bwd<B, B>(a, path, st);
}

}  // namespace mgg
