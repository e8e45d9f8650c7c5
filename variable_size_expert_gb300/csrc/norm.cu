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
//
// Which kernel: few rows take a block per row (or rows) in the forward; many, and
// all in the backward, the rings of the second half where rows are aligned or
// shifted alike; rows of differing alignment or of more than 8192 elements the
// kernels that keep a row in registers, of more than 16384 those that read a row
// again.
// Measured (inputs from HBM): forward 16384 x 2048 f32 to bf16 35.4 us (5.7 TB/s,
// 84% of the measured copy rate), 16 x 7168 5.2 us (latency); backward 4096 x
// 2048 20.6 us, 4.4 of it the column sums, 8191 x 7163 bf16 74.7 us (4.7 TB/s).
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
        make_uint2(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]));
  } else {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]),
                   cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
  }
}
// the same as packed pairs
template <typename T, int VEC>
__device__ __forceinline__ void unpack2v(const Raw<T, VEC>& r, F2 (&f)[VEC / 2]) {
  float v[VEC];
  unpack<T, VEC>(r, v);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) f[i] = pack2(v[2 * i], v[2 * i + 1]);
}
// keeps the elements i of a piece with lo <= i < hi, zeroes the others
template <typename T, int VEC>
__device__ __forceinline__ void keep_range(Raw<T, VEC>& r, int lo, int hi) {
  if constexpr (sizeof(T) == 4) {
    r.q.x = 0 >= lo && 0 < hi ? r.q.x : 0.f;
    r.q.y = 1 >= lo && 1 < hi ? r.q.y : 0.f;
    r.q.z = 2 >= lo && 2 < hi ? r.q.z : 0.f;
    r.q.w = 3 >= lo && 3 < hi ? r.q.w : 0.f;
  } else {
    auto word = [&](int i) {
      return (i >= lo && i < hi ? 0x0000ffffu : 0u) | (i + 1 >= lo && i + 1 < hi ? 0xffff0000u : 0u);
    };
    r.q.x &= word(0);
    r.q.y &= word(2);
    if constexpr (VEC == 8) {
      r.q.z &= word(4);
      r.q.w &= word(6);
    }
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

// Sum over the TPR threads of a row group (TPR a power of two); the result in
// every thread.  `slots` holds TPR/32 values per call site and parity; every
// warp adds them up with one read per lane.
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float* slots, int group, int tig) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    constexpr int NW = TPR / 32;
    if ((tig & 31) == 0) slots[tig >> 5] = v;
    bar_named(1 + group, TPR);
    v = slots[tig & (NW - 1)];
#pragma unroll
    for (int o = NW / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}
// Two sums over a warp in five shuffles: lanes 0-15 get a's, 16-31 b's.
__device__ __forceinline__ float warp_sum2(float a, float b) {
  const bool hi = threadIdx.x & 16;
  float v = hi ? b : a;
  v += __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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
  // the parameters are on their way while the sums are formed
  float wv[NV][VEC], bv[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tig) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) bv[j][i] = 0.f;
    if (c < K) {
      load_param<VEC>(w, w_f32, c, wv[j]);
      if (b) load_param<VEC>(b, w_f32, c, bv[j]);
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
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = fmaf(f[j][i] * rstd, wv[j][i], bv[j][i]);
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

// By element, in registers: rows of differing alignment, and rows of more than
// 8192 elements (8191 x 7163 bf16 with rows padded to 7170 133 us; shifted alike,
// through the ring below, 75).
template <typename XT, typename YT, int TPR, int NV>
__global__ void __launch_bounds__(TPR > kBwdThreads ? TPR : kBwdThreads)
    norm_bwd_kernel(const YT* dy, const XT* x, long long ldx, const void* w, bool w_f32,
                    const float* mean, const float* rstd, int T, int K, XT* dx, float* part) {
  constexpr int VEC = 1;
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

// ---------------------------------------------------------------- rows through shared memory
// The persistent kernels below keep the next rows on their way through shared
// memory: each thread copies its own pieces (cp.async) into slots that only it
// reads, so the copies need no barrier and several rows are in flight whatever
// the reductions wait for.
//
// SHIFT: rows that do not start on VEC-element boundaries (odd widths).  Where
// all matrices share each row's residue m (row t starts m = t K mod VEC
// elements past a boundary), a thread takes the aligned pieces that cover the
// row, whose columns start at -m; pieces at the row's ends overlap the rows
// beside it (never another 16-byte word than the row's own) and their foreign
// elements are zeroed on reading.  The groups of all blocks take the rows in
// turn and blocks come in eights (ring_blocks), so a group's rows lie a multiple
// of 8 apart, hence of VEC: they share one residue, and its threads keep their
// columns, the weights of them in registers.
template <int BYTES>
__device__ __forceinline__ void cp_async_piece(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    cp_async_16_full(dst, src);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// weights (or biases) of this thread's columns, zero outside the row
template <int VEC, int TPR, int NV, bool SHIFT>
__device__ __forceinline__ void load_columns(const void* w, bool w_f32, int tig, int m, int K,
                                             F2 (&out)[NV][VEC / 2]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tig) * VEC - m;
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.f;
    if (!SHIFT) {
      if (c < K) load_param<VEC>(w, w_f32, c, v);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (c + i >= 0 && c + i < K) {
          float one[1];
          load_param<1>(w, w_f32, c + i, one);
          v[i] = one[0];
        }
    }
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) out[j][i] = pack2(v[2 * i], v[2 * i + 1]);
  }
}

// store a piece of a row, whole or (at the ends of a shifted row) by element
template <typename T, int VEC, bool SHIFT>
__device__ __forceinline__ void store_piece(T* at, int c, int K, const F2 (&v)[VEC / 2]) {
  float o[VEC];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) unpack2(v[i], o[2 * i], o[2 * i + 1]);
  if (!SHIFT || (c >= 0 && c + VEC <= K)) {
    store_f<T, VEC>(at, o);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i >= 0 && c + i < K) at[i] = from_f<T>(o[i]);
  }
}

// Backward: one barrier per row (the sums' slots alternate); a row's xh and
// g w stay in registers between its sums and its gradient.  Packed f32
// arithmetic.
// Row slots: three of two f32 rows fill the shared memory, four of less.
template <typename XT, typename YT>
__host__ __device__ constexpr int pipe_depth() {
  return sizeof(XT) + sizeof(YT) == 8 ? 3 : 4;
}
template <typename XT, typename YT, int VEC, int TPR, int NV, bool SHIFT>
__global__ void __launch_bounds__(kBwdThreads)
    norm_bwd_pipe_kernel(const YT* dy, const XT* x, long long ldx, const void* w, bool w_f32,
                         const float* mean, const float* rstd, int T, int K, XT* dx, float* part) {
  constexpr int kThreads = kBwdThreads;
  constexpr int kGroups = kThreads / TPR;
  constexpr int XB = VEC * sizeof(XT), YB = VEC * sizeof(YT), H = VEC / 2;
  constexpr int NW = TPR / 32;
  __shared__ float slots[2][kGroups][2][NW];
  extern __shared__ __align__(16) uint8_t ring[];  // [depth][NV]([threads] x, [threads] dy)
  const int group = threadIdx.x / TPR, tig = threadIdx.x % TPR;
  constexpr int kRow = kThreads * (XB + YB);  // bytes of one j of one row slot
  uint8_t* mine_x = ring + threadIdx.x * XB;
  uint8_t* mine_y = ring + kThreads * XB + threadIdx.x * YB;
  pdl_trigger();
  pdl_wait();
  // this group's rows: first, then every step-th
  const int first = blockIdx.x * kGroups + group, step = gridDim.x * kGroups;
  const int m = SHIFT ? static_cast<int>((static_cast<long long>(first) * K) % VEC) : 0;
  const int rows = first < T ? (T - 1 - first) / step + 1 : 0;
  const int c0 = tig * VEC - m;      // column of the first piece; piece j: + j * kStride
  constexpr int kStride = TPR * VEC;
  // pointers that advance by a row of this group
  const XT* xs = x + first * ldx + c0;
  const YT* ys = dy + static_cast<long long>(first) * K + c0;
  XT* out = dx + static_cast<long long>(first) * K + c0;
  const long long sx = step * ldx, sk = static_cast<long long>(step) * K;
  auto copy = [&](int i, int slot) {  // row i of this group, the rows in order
    if (i < rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (c0 + j * kStride >= K) continue;
        const int o = slot * (NV * kRow) + j * kRow;
        cp_async_piece<XB>(smem_u32(mine_x + o), xs + j * kStride);
        cp_async_piece<YB>(smem_u32(mine_y + o), ys + j * kStride);
      }
      xs += sx;
      ys += sk;
    }
    cp_async_commit();  // (an empty group past the last row keeps the count)
  };
  constexpr int depth = pipe_depth<XT, YT>(), D = depth - 1;  // slots, rows ahead
#pragma unroll
  for (int i = 0; i < D; ++i) copy(i, i);
  F2 wv[NV][H], aw[NV][H], ab[NV][H];
  load_columns<VEC, TPR, NV, SHIFT>(w, w_f32, tig, m, K, wv);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < H; ++i) aw[j][i] = ab[j][i] = both(0.f);
  // xh and g w of a landed row, and its sums: into slots[par], or (a warp per
  // row) returned
  const float inv_k = 1.f / K;
  F2 xh[NV][H], g[NV][H];
  auto sums = [&](int slot, float mu, float rs, int par) -> float {
    F2 s1 = both(0.f), s2 = both(0.f);
    const F2 nmu = both(-mu), rs2 = both(rs);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + j * kStride;
      if (c >= K) continue;
      const int o = slot * (NV * kRow) + j * kRow;
      Raw<XT, VEC> rx = *reinterpret_cast<const Raw<XT, VEC>*>(mine_x + o);
      Raw<YT, VEC> ry = *reinterpret_cast<const Raw<YT, VEC>*>(mine_y + o);
      if (SHIFT && (c < 0 || c + VEC > K)) {
        keep_range<XT, VEC>(rx, -c, K - c);
        keep_range<YT, VEC>(ry, -c, K - c);
      }
      unpack2v<XT, VEC>(rx, xh[j]);
      unpack2v<YT, VEC>(ry, g[j]);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        xh[j][i] = mul2(add2(xh[j][i], nmu), rs2);
        aw[j][i] = fma2(g[j][i], xh[j][i], aw[j][i]);
        ab[j][i] = add2(ab[j][i], g[j][i]);
        g[j][i] = mul2(g[j][i], wv[j][i]);
        s1 = add2(s1, g[j][i]);
        s2 = fma2(g[j][i], xh[j][i], s2);
      }
    }
    float a, b, c, d;
    unpack2(s1, a, b);
    unpack2(s2, c, d);
    a = warp_sum2(a + b, c + d);
    if (TPR > 32 && (tig & 15) == 0) slots[par][group][(tig >> 4) & 1][tig >> 5] = a;
    return a;
  };
  const float *pm = mean + first, *pr = rstd + first;
  float rs = 0.f, held = 0.f;
  int slot = 0, ahead = D, par = 0;
  if (rows > 0) {
    rs = *pr;
    cp_async_wait<D - 1>();
    held = sums(0, *pm, rs, 0);
  }
#pragma unroll 1
  for (int r = 0; r < rows; ++r, par ^= 1) {
    const bool more = r + 1 < rows;
    pm += step, pr += step;
    const float mu1 = more ? *pm : 0.f, rs1 = more ? *pr : 0.f;
    float v = held;
    if constexpr (TPR > 32) {
      bar_named(1 + group, TPR);  // the parts of this row's sums are there
      v = slots[par][group][(tig >> 4) & 1][tig & (NW - 1)];
#pragma unroll
      for (int o = NW / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    const float s1 = __shfl_sync(0xffffffffu, v, 0), s2 = __shfl_sync(0xffffffffu, v, 16);
    const F2 n1 = both(-s1 * inv_k), n2 = both(-s2 * inv_k), rs2 = both(rs);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + j * kStride;
      if (c >= K) continue;
      F2 o[H];
#pragma unroll
      for (int i = 0; i < H; ++i) o[i] = mul2(rs2, fma2(xh[j][i], n2, add2(g[j][i], n1)));
      store_piece<XT, VEC, SHIFT>(out + j * kStride, c, K, o);
    }
    out += sk;
    copy(r + D, ahead);
    if (++ahead == depth) ahead = 0;
    if (++slot == depth) slot = 0;
    cp_async_wait<D - 1>();  // the next row has landed
    if (more) held = sums(slot, mu1, rs1, par ^ 1);
    rs = rs1;
  }
  // the block's partial row: every group's sums over the ring (64 KB at most),
  // then added in group order
  cp_async_wait<0>();
  __syncthreads();
  float* acc = reinterpret_cast<float*>(ring);  // [groups][2][K]
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = c0 + j * kStride;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      float w0, w1, b0, b1;
      unpack2(aw[j][i], w0, w1);
      unpack2(ab[j][i], b0, b1);
      const int k = c + 2 * i;
      float* at = acc + group * 2 * K + k;
      if (k >= 0 && k < K) at[0] = w0, at[K] = b0;
      if (k + 1 >= 0 && k + 1 < K) at[1] = w1, at[K + 1] = b1;
    }
  }
  __syncthreads();
  float* pw = part + static_cast<long long>(blockIdx.x) * K;
  float* pb = part + static_cast<long long>(gridDim.x + blockIdx.x) * K;
  for (int c = threadIdx.x; c < K; c += kThreads) {
    float vw = 0.f, vb = 0.f;
#pragma unroll 4
    for (int gi = 0; gi < kGroups; ++gi) {
      vw += acc[gi * 2 * K + c];
      vb += acc[gi * 2 * K + K + c];
    }
    pw[c] = vw;
    pb[c] = vb;
  }
}

// Forward, for many rows: six row slots (32 KB each in f32), weights and
// biases of a thread's 16 columns in registers.  A group takes its rows in
// pairs with one barrier a pair: what bounds a group is the chain from a row's
// copy to its store.  So that one exchange is enough, each warp finds mean and
// squares of its own columns around its own mean, and the warps' are joined,
//   M2 = sum_w M2_w + n_w (mean_w - mean)^2,
// which loses nothing to a large mean either.
constexpr int kFwdDepth = 6;
template <typename XT, typename YT, int VEC, int TPR, int NV, bool SHIFT>
__global__ void __launch_bounds__(kBwdThreads)
    norm_fwd_pipe_kernel(const XT* x, long long ldx, const void* w, const void* b, bool w_f32,
                         int T, int K, float eps, YT* y, float* mean_out, float* rstd_out) {
  constexpr int kThreads = kBwdThreads;
  constexpr int kGroups = kThreads / TPR;
  constexpr int XB = VEC * sizeof(XT), H = VEC / 2;
  constexpr int NW = TPR / 32, R = 2;  // rows at a time
  __shared__ float2 slots[2][kGroups][NW][R];
  __shared__ float counts[kGroups][NW];
  extern __shared__ __align__(16) uint8_t ring[];  // [depth][NV][threads]
  const int group = threadIdx.x / TPR, tig = threadIdx.x % TPR;
  uint8_t* mine = ring + threadIdx.x * XB;
  pdl_trigger();
  pdl_wait();
  const int first = blockIdx.x * kGroups + group, step = gridDim.x * kGroups;
  const int m = SHIFT ? static_cast<int>((static_cast<long long>(first) * K) % VEC) : 0;
  const float inv_k = 1.f / K;
  const int rows = first < T ? (T - 1 - first) / step + 1 : 0;
  const int c0 = tig * VEC - m;
  constexpr int kStride = TPR * VEC, kPiece = kThreads * XB;
  const XT* xs = x + first * ldx + c0;
  YT* out = y + static_cast<long long>(first) * K + c0;
  const long long sx = step * ldx, sk = static_cast<long long>(step) * K;
  int next = 0;  // row to copy, its slot
  int to = 0;
  auto copy = [&]() {
#pragma unroll
    for (int i = 0; i < R; ++i, ++next) {
      if (next < rows) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (c0 + j * kStride < K)
            cp_async_piece<XB>(smem_u32(mine + to * (NV * kPiece) + j * kPiece), xs + j * kStride);
        xs += sx;
      }
      if (++to == kFwdDepth) to = 0;
    }
    cp_async_commit();
  };
  constexpr int D = kFwdDepth / R - 1;  // pairs ahead
#pragma unroll
  for (int i = 0; i < D; ++i) copy();
  F2 wv[NV][H], bv[NV][H];
  load_columns<VEC, TPR, NV, SHIFT>(w, w_f32, tig, m, K, wv);
  if (b) {
    load_columns<VEC, TPR, NV, SHIFT>(b, w_f32, tig, m, K, bv);
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < H; ++i) bv[j][i] = both(0.f);
  }
  // columns of this warp, and of warp (lane mod NW), whose sums the lane joins
  float own = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    own += static_cast<float>(max(0, min(c0 + j * kStride + VEC, K) - max(c0 + j * kStride, 0)));
  own = warp_sum(own);
  const float inv_own = own > 0.f ? 1.f / own : 0.f;
  float n = own, inv_n = inv_own;
  if constexpr (NW > 1) {
    if ((tig & 31) == 0) counts[group][tig >> 5] = own;
    bar_named(1 + group, TPR);
    n = counts[group][tig & (NW - 1)];
    inv_n = n > 0.f ? 1.f / n : 0.f;
  }
  float *pm = mean_out + first, *pr = rstd_out + first;
  int slot = 0;
#pragma unroll 1
  for (int row = 0, par = 0; row < rows; row += R, par ^= 1) {
    copy();
    cp_async_wait<D>();
    F2 f[R][NV][H];
    float mine_mean[R], sq[R], sums[R], mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 s = both(0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * kStride;
        if (c >= K) continue;
        Raw<XT, VEC> q = *reinterpret_cast<const Raw<XT, VEC>*>(mine + slot * (NV * kPiece) + j * kPiece);
        if (SHIFT && (c < 0 || c + VEC > K)) keep_range<XT, VEC>(q, -c, K - c);
        unpack2v<XT, VEC>(q, f[r][j]);
#pragma unroll
        for (int i = 0; i < H; ++i) s = add2(s, f[r][j][i]);
      }
      if (++slot == kFwdDepth) slot = 0;
      float lo, hi;
      unpack2(s, lo, hi);
      sums[r] = lo + hi;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) sums[r] += __shfl_xor_sync(0xffffffffu, sums[r], o);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mine_mean[r] = sums[r] * inv_own;
      const F2 nm = both(-mine_mean[r]);
      F2 q = both(0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * kStride;
        if (c >= K) continue;
        const bool edge = SHIFT && (c < 0 || c + VEC > K);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          f[r][j][i] = add2(f[r][j][i], nm);
          F2 v = f[r][j][i];
          if (edge) {  // outside the row: no part in the variance
            float a, d;
            unpack2(v, a, d);
            v = pack2(c + 2 * i >= 0 && c + 2 * i < K ? a : 0.f,
                      c + 2 * i + 1 >= 0 && c + 2 * i + 1 < K ? d : 0.f);
          }
          q = fma2(v, v, q);
        }
      }
      float lo, hi;
      unpack2(q, lo, hi);
      sq[r] = lo + hi;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) sq[r] += __shfl_xor_sync(0xffffffffu, sq[r], o);
    if constexpr (NW > 1) {
      // (the slots of even and odd pairs alternate: a pair's writes cannot meet
      // the reads of the pair before)
      if ((tig & 31) == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) slots[par][group][tig >> 5][r] = make_float2(sums[r], sq[r]);
      bar_named(1 + group, TPR);
      float all[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 v = slots[par][group][tig & (NW - 1)][r];
        all[r] = sums[r] = v.x;
        sq[r] = v.y;
      }
#pragma unroll
      for (int o = NW / 2; o; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) all[r] += __shfl_xor_sync(0xffffffffu, all[r], o);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        mean[r] = all[r] * inv_k;
        const float d = sums[r] * inv_n - mean[r];
        sq[r] = fmaf(n * d, d, sq[r]);
      }
#pragma unroll
      for (int o = NW / 2; o; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) sq[r] += __shfl_xor_sync(0xffffffffu, sq[r], o);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) mean[r] = mine_mean[r];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row + r >= rows) break;
      rstd[r] = 1.f / sqrtf(sq[r] * inv_k + eps);
      if (tig == 0) {
        *pm = mean[r];
        *pr = rstd[r];
      }
      pm += step, pr += step;
      const F2 shift = both(mine_mean[r] - mean[r]), rs = both(rstd[r]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * kStride;
        if (c >= K) continue;
        F2 o[H];
#pragma unroll
        for (int i = 0; i < H; ++i)
          o[i] = fma2(mul2(add2(f[r][j][i], shift), rs), wv[j][i], bv[j][i]);
        store_piece<YT, VEC, SHIFT>(out + j * kStride, c, K, o);
      }
      out += sk;
    }
  }
  cp_async_wait<0>();
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

// How the rows lie: element by element, all on piece boundaries, or all with
// the same residue per row.
enum RowPath { kByElement, kAligned, kShifted };

// Blocks of the rings: a multiple of eight (see SHIFT above), one an SM at most,
// no more than the rows need.
int ring_blocks(int T, int groups) {
  return std::min(norm_bwd_blocks(), cdiv(cdiv(T, groups), 8) * 8);
}

template <typename K>
cudaError_t allow_ring(K kern, bool* done) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && done[dev]) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024);
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

template <typename XT, typename YT, int TPR, bool SHIFT>
cudaError_t fwd_pipe_t(const FwdArgs& a, cudaStream_t st) {
  constexpr int VEC = sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 : 4, NV = 16 / VEC;
  constexpr int kGroups = kBwdThreads / TPR;
  constexpr size_t smem = static_cast<size_t>(kFwdDepth) * NV * kBwdThreads * VEC * sizeof(XT);
  auto kern = norm_fwd_pipe_kernel<XT, YT, VEC, TPR, NV, SHIFT>;
  static bool done[64] = {};
  const cudaError_t e = allow_ring(kern, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ring_blocks(a.T, kGroups)), dim3(kBwdThreads), smem, st,
                    static_cast<const XT*>(a.x), a.ldx, a.w, a.b, a.w_f32, a.T, a.K, a.eps,
                    static_cast<YT*>(a.y), a.mean, a.rstd);
}
template <typename XT, typename YT, bool SHIFT>
cudaError_t fwd_pipe(const FwdArgs& a, cudaStream_t st) {
  const int K = a.K + (SHIFT ? 7 : 0);
  if (K <= 512) return fwd_pipe_t<XT, YT, 32, SHIFT>(a, st);
  if (K <= 1024) return fwd_pipe_t<XT, YT, 64, SHIFT>(a, st);
  if (K <= 2048) return fwd_pipe_t<XT, YT, 128, SHIFT>(a, st);
  if (K <= 4096) return fwd_pipe_t<XT, YT, 256, SHIFT>(a, st);
  return fwd_pipe_t<XT, YT, 512, SHIFT>(a, st);
}

template <typename XT, typename YT>
cudaError_t fwd(const FwdArgs& a, RowPath path, cudaStream_t st) {
  const int K = a.K;
  if (K > kRegRow)
    return launch_pdl(norm_fwd_long_kernel<XT, YT>, dim3(a.T), dim3(512), 0, st,
                      static_cast<const XT*>(a.x), a.ldx, a.w, a.b, a.w_f32, a.T, K, a.eps,
                      static_cast<YT*>(a.y), a.mean, a.rstd);
  // The ring pays once it has turned over, counted in elements per thread and 16
  // columns: after two rounds of rows, eight at the widths where a block takes
  // two rows and hides one behind the other, one for shifted rows, which are
  // read by element else.  Measured, block per row against ring, inputs in L2:
  // 512 x 7168 bf16 7.5 and 6.1 us, 4096 x 7168 58 and 28; 4096 x 2048 f32 9.3
  // and 11.2, 8192 x 2048 20.7 and 19.3; 8192 x 512 bf16 5.7 and 5.2; 1024 x 2047
  // 7.3 and 6.9.
  const int turns = path == kShifted ? 1 : K > 512 && K <= 2048 ? 8 : 2;
  const bool many = static_cast<long long>(a.T) * K > static_cast<long long>(turns) * num_sms() * kBwdThreads * 16;
  if (many && path == kAligned && K <= 8192) return fwd_pipe<XT, YT, false>(a, st);
  if (many && path == kShifted && K <= 8192 - 7) return fwd_pipe<XT, YT, true>(a, st);
  if (path == kAligned) {
    constexpr int V = sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 : 4;  // 16 values a thread
    if (K <= 512) return fwd_t<XT, YT, V, 32, 16 / V>(a, st);
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
  constexpr int NV = 16;
  constexpr int kThreads = TPR > kBwdThreads ? TPR : kBwdThreads;
  constexpr int kGroups = kThreads / TPR;
  *nb = std::min(norm_bwd_blocks(), cdiv(a.T, kGroups));
  const size_t smem = kGroups > 1 ? static_cast<size_t>(2) * a.K * 4 : 0;
  return launch_pdl(norm_bwd_kernel<XT, YT, TPR, NV>, dim3(*nb), dim3(kThreads), smem, st,
                    static_cast<const YT*>(a.dy), static_cast<const XT*>(a.x), a.ldx, a.w, a.w_f32,
                    a.mean, a.rstd, a.T, a.K, static_cast<XT*>(a.dx), a.part);
}

template <typename XT, typename YT, int TPR, bool SHIFT>
cudaError_t bwd_pipe_t(const BwdArgs& a, int* nb, cudaStream_t st) {
  constexpr int VEC = sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 : 4;
  constexpr int NV = 16 / VEC;
  constexpr int kThreads = kBwdThreads;
  constexpr int kGroups = kThreads / TPR;
  constexpr size_t kRing = static_cast<size_t>(pipe_depth<XT, YT>()) * NV * kThreads * VEC * (sizeof(XT) + sizeof(YT));
  *nb = ring_blocks(a.T, kGroups);
  const size_t smem = std::max(kRing, static_cast<size_t>(2) * kGroups * a.K * 4);
  auto kern = norm_bwd_pipe_kernel<XT, YT, VEC, TPR, NV, SHIFT>;
  static bool done[64] = {};
  const cudaError_t e = allow_ring(kern, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(*nb), dim3(kThreads), smem, st, static_cast<const YT*>(a.dy),
                    static_cast<const XT*>(a.x), a.ldx, a.w, a.w_f32, a.mean, a.rstd, a.T, a.K,
                    static_cast<XT*>(a.dx), a.part);
}
// K: the row's columns, with SHIFT those of the pieces that cover it
template <typename XT, typename YT, bool SHIFT>
cudaError_t bwd_pipe(const BwdArgs& a, int* nb, cudaStream_t st) {
  const int K = a.K + (SHIFT ? 7 : 0);
  if (K <= 512) return bwd_pipe_t<XT, YT, 32, SHIFT>(a, nb, st);
  if (K <= 1024) return bwd_pipe_t<XT, YT, 64, SHIFT>(a, nb, st);
  if (K <= 2048) return bwd_pipe_t<XT, YT, 128, SHIFT>(a, nb, st);
  if (K <= 4096) return bwd_pipe_t<XT, YT, 256, SHIFT>(a, nb, st);
  return bwd_pipe_t<XT, YT, 512, SHIFT>(a, nb, st);
}

template <typename XT, typename YT>
cudaError_t bwd(const BwdArgs& a, RowPath path, cudaStream_t st) {
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

// Pieces (16 bytes of the wider type) where the bases are aligned and either
// every row starts on a piece boundary or all matrices share the rows'
// residues; else element by element.
static RowPath row_path(bool any_f32, int K, long long ldx, bool bases, bool params) {
  const int vec = any_f32 ? 4 : 8;
  if (!bases) return kByElement;
  if (K % vec == 0 && ldx % vec == 0 && params) return kAligned;
  return ldx % vec == K % vec ? kShifted : kByElement;
}

cudaError_t launch_norm_fwd(const void* x, bool x_f32, long long ldx, const void* w, const void* b,
                            bool w_f32, int T, int K, float eps, void* y, bool y_f32, float* mean,
                            float* rstd, cudaStream_t st) {
  const RowPath path = row_path(x_f32 || y_f32, K, ldx, aligned16(x) && aligned16(y),
                                aligned16(w) && aligned16(b));
  const FwdArgs a{x, ldx, w, b, w_f32, T, K, eps, y, mean, rstd};
  using B = __nv_bfloat16;
  if (x_f32) return y_f32 ? fwd<float, float>(a, path, st) : fwd<float, B>(a, path, st);
  return y_f32 ? fwd<B, float>(a, path, st) : fwd<B, B>(a, path, st);
}

cudaError_t launch_norm_bwd(const void* dy, bool y_f32, const void* x, bool x_f32, long long ldx,
                            const void* w, bool w_f32, const float* mean, const float* rstd, int T,
                            int K, void* dx, void* dw, void* db, float* part, cudaStream_t st) {
  const RowPath path = row_path(x_f32 || y_f32, K, ldx,
                                aligned16(x) && aligned16(dy) && aligned16(dx), aligned16(w));
  const BwdArgs a{dy, x, ldx, w, w_f32, mean, rstd, T, K, dx, dw, db, part};
  using B = __nv_bfloat16;
  if (x_f32) return y_f32 ? bwd<float, float>(a, path, st) : bwd<float, B>(a, path, st);
  return y_f32 ? bwd<B, float>(a, path, st) : bwd<B, B>(a, path, st);
}

}  // namespace mgg
