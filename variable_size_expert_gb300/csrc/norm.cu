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

// VEC consecutive elements as they lie in memory: 16-byte accesses for
// VEC = 8, single elements for VEC = 1 (odd widths, unaligned rows).
template <typename T, int VEC>
struct Raw {
  T v[VEC];
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 q;
};
template <>
struct Raw<float, 8> {
  float4 q[2];
};
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
  Raw<T, VEC> r;
  if constexpr (VEC == 1) {
    r.v[0] = *p;
  } else if constexpr (sizeof(T) == 2) {
    r.q = *reinterpret_cast<const uint4*>(p);
  } else {
    r.q[0] = reinterpret_cast<const float4*>(p)[0];
    r.q[1] = reinterpret_cast<const float4*>(p)[1];
  }
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Raw<T, VEC>& r, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_f<T>(r.v[0]);
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t u[4] = {r.q.x, r.q.y, r.q.z, r.q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    f[0] = r.q[0].x, f[1] = r.q[0].y, f[2] = r.q[0].z, f[3] = r.q[0].w;
    f[4] = r.q[1].x, f[5] = r.q[1].y, f[6] = r.q[1].z, f[7] = r.q[1].w;
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_f(T* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(f[0]);
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]),
                   pack_bf16x2_rn(f[4], f[5]), pack_bf16x2_rn(f[6], f[7]));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}
// the weight or bias (f32 or bf16), VEC elements from column c
template <int VEC>
__device__ __forceinline__ void load_param(const void* w, bool w_f32, int c, float (&f)[VEC]) {
  if (w_f32)
    unpack<float, VEC>(load_raw<float, VEC>(static_cast<const float*>(w) + c), f);
  else
    unpack<__nv_bfloat16, VEC>(
        load_raw<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w) + c), f);
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
    if (K <= 512) return fwd_t<XT, YT, 8, 32, 2>(a, st);
    if (K <= 1024) return fwd_t<XT, YT, 8, 32, 4>(a, st);
    if (K <= 2048) return fwd_t<XT, YT, 8, 128, 2>(a, st);
    if (K <= 4096) return fwd_t<XT, YT, 8, 256, 2>(a, st);
    if (K <= 8192) return fwd_t<XT, YT, 8, 512, 2>(a, st);
    return fwd_t<XT, YT, 8, 1024, 2>(a, st);
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

template <typename XT, typename YT, int VEC, int TPR, int NV>
cudaError_t bwd_t(const BwdArgs& a, int* nb, cudaStream_t st) {
  constexpr int kThreads = TPR > kBwdThreads ? TPR : kBwdThreads;
  constexpr int kGroups = kThreads / TPR;
  *nb = std::min(norm_bwd_blocks(), cdiv(a.T, kGroups));
  const size_t smem = kGroups > 1 ? static_cast<size_t>(2) * a.K * 4 : 0;
  return launch_pdl(norm_bwd_kernel<XT, YT, VEC, TPR, NV>, dim3(*nb), dim3(kThreads), smem, st,
                    static_cast<const YT*>(a.dy), static_cast<const XT*>(a.x), a.ldx, a.w, a.w_f32,
                    a.mean, a.rstd, a.T, a.K, static_cast<XT*>(a.dx), a.part);
}

template <typename XT, typename YT>
cudaError_t bwd(const BwdArgs& a, bool vec, cudaStream_t st) {
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
  } else if (vec) {
    if (K <= 512) e = bwd_t<XT, YT, 8, 32, 2>(a, &nb, st);
    else if (K <= 1024) e = bwd_t<XT, YT, 8, 64, 2>(a, &nb, st);
    else if (K <= 2048) e = bwd_t<XT, YT, 8, 128, 2>(a, &nb, st);
    else if (K <= 4096) e = bwd_t<XT, YT, 8, 256, 2>(a, &nb, st);
    else if (K <= 8192) e = bwd_t<XT, YT, 8, 512, 2>(a, &nb, st);
    else e = bwd_t<XT, YT, 8, 1024, 2>(a, &nb, st);
  } else {
    if (K <= 512) e = bwd_t<XT, YT, 1, 32, 16>(a, &nb, st);
    else if (K <= 2048) e = bwd_t<XT, YT, 1, 128, 16>(a, &nb, st);
    else if (K <= 8192) e = bwd_t<XT, YT, 1, 512, 16>(a, &nb, st);
    else e = bwd_t<XT, YT, 1, 1024, 16>(a, &nb, st);
  }
  if (e != cudaSuccess) return e;
  return launch_column_sums(a.part, nb, K, a.dw, a.db, a.w_f32, st);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

cudaError_t launch_column_sums(const float* part, int nb, int K, void* out0, void* out1,
                               bool out_f32, cudaStream_t st) {
  return launch_pdl(column_sums_kernel, dim3(cdiv(K, 32), out1 ? 2 : 1), dim3(1024), 0, st, part,
                    nb, K, out0, out1, out_f32);
}

int norm_bwd_blocks() { return num_sms(); }

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
  const bool vec = K % 8 == 0 && ldx % 8 == 0 && aligned16(x) && aligned16(w) && aligned16(dy) &&
                   aligned16(dx);
  const BwdArgs a{dy, x, ldx, w, w_f32, mean, rstd, T, K, dx, dw, db, part};
  using B = __nv_bfloat16;
  if (x_f32) return y_f32 ? bwd<float, float>(a, vec, st) : bwd<float, B>(a, vec, st);
  return y_f32 ? bwd<B, float>(a, vec, st) : bwd<B, B>(a, vec, st);
}

}  // namespace mgg
