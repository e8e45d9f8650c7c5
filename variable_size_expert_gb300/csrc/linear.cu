// Dense products on the tensor cores (tcgen05, bf16 operands, f32
// accumulation in tensor memory) for the layers around the experts:
//   forward   z = x W^T + b;  out = act(z) + residual
//   backward  dz = dy act'(z) (bf16);  dx = dz W;  dW = dz^T x;  db = sum_t dz
//
// Every product is D[M, N] = sum_k A[m, k] B[n, k] over operands that lie in
// memory either with k contiguous ("K-major": x and W in the forward, dz in
// dx) or with m / n contiguous ("MN-major": W in dx, dz and x in dW); TMA
// loads both kinds as 128-byte-swizzled blocks of 64 and the matrix
// descriptors say which it is.  No operand is transposed in memory.
//
// Two kernels:
//  dense_pair_kernel  persistent, one cluster of two CTAs per SM pair, tiles
//    of 256 x 256 (MMA M = 256, N = 256, cta_group::2: each SM holds 128 rows
//    of A and of B, so a tile costs each SM half the bytes of a single-CTA
//    tile).  Two accumulators in tensor memory, so the epilogue of a tile
//    runs under the next tile's MMAs.  A launch takes the tiles of up to two
//    products: the backward runs dx and dW as one tile space, whose last
//    round is the only partly filled one.
//    Bound by the matrix units at the power limit: 8192 x 2048 x 8192 171 us
//    (1610 TFLOP/s sustained), with bias, GELU and kept z 196; dx and dW 338;
//    with little to contract by its stores (8192 x 64 x 8192 40 us, 3.4 TB/s).
//    A product's operands are bf16, so dz is rounded to it, as in the library's
//    other backward products: dx and dW are off by 2.35e-3 (relative, root mean
//    square) where the rounding of the result alone gives 1.66e-3.  A second
//    product with the rest of dz would remove that and double the operations of
//    kernels that the matrix units bound.  dbias sums dz before it is rounded.
//  dense_cta_kernel  one tile of 128 x BN (BN 16..256) per cluster of S CTAs,
//    which split the contraction and add their partial accumulators through
//    distributed shared memory in rank order (the same bits every time).  For
//    products with too few 256 x 256 tiles to fill the GPU: a decode step's
//    few tokens, the gate's few columns.  The longer of the two output sides
//    lies on the MMA's 128 rows, so that the shorter costs only its own width.
//    Two warps load and two multiply: 1024 x 8192 x 1024 21 us, 35 with one of
//    each.  A decode step's 16 x 7168 x 2048 7.0 us (30 MB, 63% of the measured
//    copy rate): start-up, the first loads and the join take 2.6 us.
#include "pair.cuh"

namespace mgg {
namespace {

// ---------------------------------------------------------------- epilogue math
// The activations run once per output element on the few warps that empty the
// accumulators, so their instruction count matters (CUDA's erff and expf with
// IEEE divisions took the GELU epilogue past the MMAs it should hide under:
// 246 us against 197 for 8192 x 2048 x 8192).  The approximate exponential
// and reciprocal are each one instruction, within 2 ulp, denormals flushed
// (values under 1e-38); exp(-z) = inf gives a sigmoid of 0.
__device__ __forceinline__ float sigmoid_f(float z) {
  return rcp_f(1.f + exp2_f(z * -1.4426950408889634f));
}
// Phi(z) = (1 + erf(z / sqrt 2)) / 2 with Abramowitz & Stegun 7.1.26,
//   erf(x) = 1 - (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + p x), x >= 0,
// absolute error at most 1.5e-7; here x = |z| / sqrt 2, with the 1 / sqrt 2
// in p and the half in the a's.  The error falls with exp(-z^2 / 2) but slower
// than Phi: z Phi(z) is right to 3e-7 |z| everywhere, which a bf16 output does not
// show; of its own value to 4e-6 at z = -2, 5e-4 at -4, 4e-3 at -6.  *e receives exp(-z^2 / 2), which is the
// exp(-x^2) of the formula and the density's exponential in the gradient.
__device__ __forceinline__ F2 normal_cdf2(float z0, float z1, F2* e) {
  const F2 z = pack2(z0, z1);
  float x0, x1;
  unpack2(mul2(mul2(z, z), both(-0.72134752044448170f)), x0, x1);  // log2(e) / 2
  *e = pack2(exp2_f(x0), exp2_f(x1));
  const F2 t = pack2(rcp_f(fmaf(0.23164189f, fabsf(z0), 1.f)), rcp_f(fmaf(0.23164189f, fabsf(z1), 1.f)));
  F2 q = fma2(both(0.5307027145f), t, both(-0.7265760135f));
  q = fma2(q, t, both(0.7107068705f));
  q = fma2(q, t, both(-0.142248368f));
  q = fma2(q, t, both(0.127414796f));
  q = mul2(q, mul2(t, *e));  // Phi(-|z|)
  float q0, q1;
  unpack2(q, q0, q1);
  return pack2(z0 < 0.f ? q0 : 1.f - q0, z1 < 0.f ? q1 : 1.f - q1);
}

// v = act(v)
template <int ACT, int N>
__device__ __forceinline__ void act_n(float (&v)[N]) {
  static_assert(N % 2 == 0, "");
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if constexpr (ACT == kActRelu) {
      v[i] = v[i] < 0.f ? 0.f : v[i];  // (fmaxf would turn NaN into 0)
      v[i + 1] = v[i + 1] < 0.f ? 0.f : v[i + 1];
    } else if constexpr (ACT == kActSilu) {
      v[i] *= sigmoid_f(v[i]);
      v[i + 1] *= sigmoid_f(v[i + 1]);
    } else if constexpr (ACT == kActGelu) {
      F2 e;
      unpack2(mul2(pack2(v[i], v[i + 1]), normal_cdf2(v[i], v[i + 1], &e)), v[i], v[i + 1]);
    }
  }
}
// g = g act'(z); of ReLU a choice, not a product: a closed unit passes nothing on,
// whatever its g holds
template <int ACT, int N>
__device__ __forceinline__ void slope_n(float (&g)[N], const float (&z)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float z0 = z[i], z1 = N > 1 ? z[i + (N > 1)] : 0.f;
    if constexpr (ACT == kActRelu) {
      g[i] = z0 > 0.f ? g[i] : 0.f;
      if constexpr (N > 1) g[i + 1] = z1 > 0.f ? g[i + 1] : 0.f;
      continue;
    }
    float s0, s1;
    if constexpr (ACT == kActSilu) {
      const float a = sigmoid_f(z0), b = sigmoid_f(z1);
      s0 = a * fmaf(z0, 1.f - a, 1.f), s1 = b * fmaf(z1, 1.f - b, 1.f);
    } else if constexpr (ACT == kActGelu) {
      F2 e;
      const F2 c = normal_cdf2(z0, z1, &e);
      unpack2(fma2(mul2(pack2(z0, z1), both(0.39894228040143268f)), e, c), s0, s1);
    } else {
      s0 = s1 = 1.f;
    }
    g[i] *= s0;
    if constexpr (N > 1) g[i + 1] *= s1;
  }
}

template <int N>
__device__ __forceinline__ void act_all(int act, float (&v)[N]) {
  if (act == kActRelu) act_n<kActRelu>(v);
  else if (act == kActSilu) act_n<kActSilu>(v);
  else if (act == kActGelu) act_n<kActGelu>(v);
}

template <int N>
__device__ __forceinline__ void scale_all(float scale, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= scale;
}

__device__ __forceinline__ float load_any(const void* p, bool f32, long long i) {
  return f32 ? static_cast<const float*>(p)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// v += bias[c0 .. c0 + 31]: the same addresses in every lane, so a 16-byte
// load serves the warp with one L1 access (32 shuffles of a lane's own column
// took longer than the addition hides).
__device__ __forceinline__ void add_bias(const DenseParams& p, int c0, int N, float (&v)[32]) {
  if (p.bias_vec && c0 + 32 <= N) {
    if (p.bias_f32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + c0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = q[i];
        v[4 * i] += x.x, v[4 * i + 1] += x.y, v[4 * i + 2] += x.z, v[4 * i + 3] += x.w;
      }
    } else {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bias) + c0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = q[i];
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] += __uint_as_float(u[j] << 16);
          v[8 * i + 2 * j + 1] += __uint_as_float(u[j] & 0xffff0000u);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c0 + i < N) v[i] += load_any(p.bias, p.bias_f32, c0 + i);
  }
}

// v += residual, rows row0.. (of M), columns c0 .. c0 + 31 (below N): read with
// consecutive lanes on consecutive elements into the staging area as f32, then
// each lane takes its own row.
__device__ __forceinline__ void add_residual(const DenseParams& p, uint32_t stg, int lane, int row0,
                                             int M, int c0, int N, float (&v)[32]) {
  if (p.res_vec && N % 4 == 0) {
    // four columns a lane, four rows per instruction
    const int kq = lane & 7, c = c0 + 4 * kq, rq = lane >> 3;
    const long long o = static_cast<long long>(row0 + rq) * p.ldr + c;
    float4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row0 + rq + 4 * j < M && c < N) {
        if (p.res_f32) {
          x[j] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) + o + 4 * j * p.ldr);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(
              static_cast<const __nv_bfloat16*>(p.residual) + o + 4 * j * p.ldr);
          x[j] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                             __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      st_shared_v4(stg + sw128_offset(rq + 4 * j, kq), x[j].x, x[j].y, x[j].z, x[j].w);
  } else {
    const int c = c0 + lane;
    const long long o = static_cast<long long>(row0) * p.ldr + c;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 16) {
      float x[16];  // (loaded together: a shared store holds the next load back)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        x[r] = row0 + r0 + r < M && c < N ? load_any(p.residual, p.res_f32, o + (r0 + r) * p.ldr) : 0.f;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        st_shared_f32(stg + sw128_offset(r0 + r, lane >> 2) + (lane & 3) * 4, x[r]);
    }
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float4 x = ld_shared_v4(stg + sw128_offset(lane, c));
    v[4 * c] += x.x, v[4 * c + 1] += x.y, v[4 * c + 2] += x.z, v[4 * c + 3] += x.w;
  }
  __syncwarp();  // the staging area is free again
}

// ---------------------------------------------------------------- pair kernel
struct PairMaps {
  CUtensorMap a[2], b[2], res;
};

// The tiles' order and the options of a launch of the pair kernel.
struct PairExtra {
  int slices[2];
  int longer, deal_pairs, deal;  // see tile_of
  const float *scale0, *scale1;  // of kActScale
};
struct PTile {
  int q;           // product
  int m0, n0;      // first row and column
  int slice;       // of the contraction
  int kb0, nkb;    // its blocks
};
template <bool EXTRA>
__device__ __forceinline__ PTile decode_pair(const DenseParams& p, const PairExtra& x, int tau) {
  PTile t;
  t.q = EXTRA && tau >= p.pr[0].tiles ? 1 : 0;
  const DenseProduct& d = p.pr[t.q];
  int local = tau - (t.q ? p.pr[0].tiles : 0);
  const int blocks = cdiv(d.Kc, BK), slices = EXTRA ? x.slices[t.q] : 1;
  t.slice = 0, t.kb0 = 0, t.nkb = blocks;
  if (slices > 1) {
    const int per = d.tiles / slices;
    t.slice = local / per;
    local -= t.slice * per;
    t.kb0 = static_cast<int>(static_cast<long long>(t.slice) * blocks / slices);
    t.nkb = static_cast<int>(static_cast<long long>(t.slice + 1) * blocks / slices) - t.kb0;
  }
  band_tile(local, d.M, d.N, t.m0, t.n0);
  return t;
}
// The i-th tile of a pair, -1 after its last; `mine` of them are of the product with
// the longer contraction.  Its tiles are dealt out one after the other; the pairs left
// with one fewer of them (from x.deal_pairs on) then take x.deal tiles of the other
// product, about as long as that one, before those are dealt out in turn too.  (Dealt
// out by their number alone, 128 tiles of 128 blocks and 256 of 64 gave four pairs 512
// blocks of 431 on average; so none has more than 448.)
__device__ __forceinline__ int tile_of(const DenseParams& p, const PairExtra& x, int pair, int npairs, int mine,
                                       int i) {
  const int f = x.longer, tail = p.pr[1 - f].tiles;
  if (i < mine) return (f ? p.pr[0].tiles : 0) + pair + i * npairs;
  i -= mine;
  int t;
  const int few = npairs - x.deal_pairs;  // pairs with one fewer
  if (pair >= x.deal_pairs && i < x.deal) {
    t = i * few + pair - x.deal_pairs;
  } else {
    if (pair >= x.deal_pairs) i -= x.deal;
    t = x.deal * few + i * npairs + pair;
  }
  return t < tail ? (f ? t : p.pr[0].tiles + t) : -1;
}

// ACT is a template argument and the column loop is not unrolled: with the
// activations as runtime branches of an unrolled loop the epilogue's code
// outgrew the instruction cache, which the lone producer and MMA threads share.
// EXTRA: two products, slices or a factor; a single product's tiles go by their number
// (the order by length costs 4% where a tile is two blocks, 8192 x 128 x 8192).
template <int ACT, bool EXTRA>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    dense_pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ DenseParams p,
                      const __grid_constant__ PairExtra x) {
  extern __shared__ uint8_t smem_raw[];
  const PSmem m = carve_pair(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (warp == 5 && lane == 0) {
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
  }
  if (threadIdx.x == 0) {
    init_pair(m);
  }
  if (warp == 4) {
    tmem_alloc_cg2(smem_u32(m.tmem_slot), 512);
    tmem_relinquish_cg2();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *m.tmem_slot;
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{m.abort_flag, p.dev_status, p.wait_limit};
  const int total = p.pr[0].tiles;
  // this pair's tiles of the product with the longer contraction
  const int head = EXTRA ? p.pr[x.longer].tiles : 0;
  const int mine = pair < head ? (head - 1 - pair) / npairs + 1 : 0;
  // the i-th tile of this pair after `tau`
  auto next = [&](int i, int& tau) {
    if constexpr (EXTRA) {
      tau = tile_of(p, x, pair, npairs, mine, i);
      return tau >= 0;
    } else {
      tau = i ? tau + npairs : pair;
      return tau < total;
    }
  };
  const uint32_t full_l = mapa_shared(m.full, 0);
  const uint32_t acc_empty_l = mapa_shared(m.acc_empty, 0);

  if (warp == 5) {
    // ------------------------------------------------ TMA
    Ring r{0, 0, 0};
    bool ok = true;
    for (int i = 0, tau = 0; ok && next(i, tau); ++i) {
      const PTile t = decode_pair<EXTRA>(p, x, tau);
      const DenseProduct& d = p.pr[t.q];
      const int ar = t.m0 + static_cast<int>(rank) * kHalf;
      const int br = t.n0 + static_cast<int>(rank) * kHalf;
      const CUtensorMap *ma = &maps.a[t.q], *mb = &maps.b[t.q];
      // (the three layouts of the forward, dx and dW)
      if (d.a_mn)
        ok = produce<true, true>(m, ma, mb, full_l, leader, ar, br, t.kb0, t.nkb, r, wc);
      else if (d.b_mn)
        ok = produce<false, true>(m, ma, mb, full_l, leader, ar, br, t.kb0, t.nkb, r, wc);
      else
        ok = produce<false, false>(m, ma, mb, full_l, leader, ar, br, t.kb0, t.nkb, r, wc);
    }
    if (lane == 0) drain_copies(m, r.it, leader);
    __syncwarp();
  } else if (warp == 4) {
    // ------------------------------------------------ MMA issue
    if (leader) {
      int tcount = 0;
      Ring r{0, 0, 0};
      bool ok = true;
      for (int i = 0, tau = 0; ok && next(i, tau); ++i) {
        // (of the tile only its product and length: this warp is what tiles wait for)
        const int q = EXTRA && tau >= p.pr[0].tiles ? 1 : 0;
        const DenseProduct& d = p.pr[q];
        const int nkb = EXTRA && x.slices[q] > 1 ? decode_pair<EXTRA>(p, x, tau).nkb : cdiv(d.Kc, BK);
        const int acc = tcount & 1;
        if (!__all_sync(0xffffffffu, wait_bar(m.acc_empty + 8 * acc, ((tcount >> 1) & 1) ^ 1, wc)))
          break;
        tc_fence_after();
        const uint32_t dt = tmem_base + acc * 256;
        if (d.a_mn)
          ok = multiply<true, true>(m, dt, nkb, r, wc);
        else if (d.b_mn)
          ok = multiply<false, true>(m, dt, nkb, r, wc);
        else
          ok = multiply<false, false>(m, dt, nkb, r, wc);
        if (!ok) break;
        if (elect_one()) tc_commit_cg2_mc(m.acc_full + 8 * acc, 0x3);
        ++tcount;
      }
      if (elect_one()) {
        tc_commit_cg2(m.drain);
        wait_bar_drain(m.drain, 0, DRAIN_LIMIT);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------ epilogue
    // Four warps per 64 columns of the tile; a warp holds rows 32 (w % 4) ..
    // +31 of this CTA's 128 (the quarter of tensor memory that it can read),
    // lane i row i.  The results leave through staged blocks by plain stores
    // (TMA stores waited for the staging area to be read, 96 against 82 us for
    // bias + GELU + z of 8192 x 64 x 8192; no difference at K = 2048).
    const int quad = warp & 3, group = warp < 4 ? 0 : (warp - 2) >> 2;
    const int ew = group * 4 + quad;
    const uint32_t stg = m.sEpi + ew * EPI_WARP;
    const uint32_t res_bar = m.res_full + 8 * ew;
    const int row_w = static_cast<int>(rank) * kHalf + quad * 32;
    int tcount = 0, res_n = 0;
    bool res_open = false;  // a residual block is on its way
    const float scale = ACT == kActScale ? *x.scale0 * *x.scale1 : 1.f;
    for (int i = 0, tau = 0; next(i, tau); ++i) {
      const PTile t = decode_pair<EXTRA>(p, x, tau);
      const DenseProduct& d = p.pr[t.q];
      const int row0 = t.m0 + row_w;
      const int acc = tcount & 1;
      const int col_w = t.n0 + group * 64;  // first column of this warp
      const int nblk = std::max(0, std::min(2, cdiv(d.N - col_w, 32)));  // 32-column blocks
      const bool epi = d.epilogue;
      // To an f32 output the residual's 32 x 32 block comes by TMA into the
      // staging area that the result then takes: the first one while the tile
      // is multiplied, unless z passes through the staging area before.  A
      // bf16 output with a residual leaves 32 columns at a time (the residual's
      // block takes the whole staging area).
      const bool res_tma = epi && p.res_tma && row0 < d.M;
      auto fetch_res = [&](int c0) {
        // Every lane's reads and writes of the staging area come before the
        // copy that overwrites it: they are ordinary accesses, the copy is of
        // the async proxy, so the warp's barrier alone does not order them.
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(res_bar, p.res_f32 ? 4096 : 2048);
          tma_load_2d(stg, &maps.res, res_bar, c0, t.slice * d.M + row0);
        }
        res_open = true;
      };
      if (res_tma && nblk > 0 && !p.pre) fetch_res(col_w);
      if (!__all_sync(0xffffffffu, wait_bar(m.acc_full + 8 * acc, (tcount >> 1) & 1, wc))) break;
      tc_fence_after();
      const uint32_t taddr =
          tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256 + group * 64;
      // The accumulator has been read (into registers, by loads that are done:
      // no other memory is handed over, and a release at cluster scope would
      // wait 0.5 us for this warp's stores in flight).
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_l + 8 * acc);
      };
      if (nblk == 0) release();  // nothing of the tile here
      // columns 32 b .. of the tile with the bias, v
      auto load = [&](int b, float(&v)[32]) {
        tmem_ld32(taddr + b * 32, v);
        tmem_ld_wait();
        if constexpr (ACT == kActScale) scale_all<32>(scale, v);
        if (epi && p.bias) add_bias(p, col_w + b * 32, d.N, v);
      };
      auto act_res = [&](int b, float(&v)[32]) {
        act_n<ACT>(v);
        const int c0 = col_w + b * 32;
        if (res_tma) {
          if (b > 0 || p.pre) fetch_res(c0);
          const bool ok = __all_sync(0xffffffffu, wait_bar(res_bar, res_n & 1, wc));
          res_open = !ok;
          ++res_n;
          if (p.res_f32) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 x = ld_shared_v4(stg + sw128_offset(lane, c));
              v[4 * c] += x.x, v[4 * c + 1] += x.y, v[4 * c + 2] += x.z, v[4 * c + 3] += x.w;
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float4 x = ld_shared_v4(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
              const uint32_t u[4] = {__float_as_uint(x.x), __float_as_uint(x.y),
                                     __float_as_uint(x.z), __float_as_uint(x.w)};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                v[8 * c + 2 * j] += __uint_as_float(u[j] << 16);
                v[8 * c + 2 * j + 1] += __uint_as_float(u[j] & 0xffff0000u);
              }
            }
          }
        } else if (epi && p.residual) {
          add_residual(p, stg, lane, row0, d.M, c0, d.N, v);
        }
      };
      if (epi && p.pre && nblk > 0) {
#pragma unroll 1
        for (int b = 0; b < nblk; ++b) {
          float v[32];
          load(b, v);
          stage_bf16(stg, lane, b, v);
        }
        stage_flush(stg, lane, p.pre_vec, p.pre, false, row0, d.M, d.N, col_w, d.N);
      }
      if (d.out_f32) {
#pragma unroll 1
        for (int b = 0; b < nblk; ++b) {
          float v[32];
          load(b, v);
          if (b == nblk - 1) release();
          act_res(b, v);
          __syncwarp();  // every lane has read its residual row
          stage_f32(stg, lane, v);
          stage_flush(stg, lane, d.out_vec, static_cast<float*>(d.out) + static_cast<long long>(t.slice) * d.M * d.N,
                      true, row0, d.M, d.N, col_w + b * 32, d.N);
        }
      } else if (nblk > 0) {
        const bool by_half = epi && p.residual;
#pragma unroll 1
        for (int b = 0; b < nblk; ++b) {
          float v[32];
          load(b, v);
          if (b == nblk - 1) release();
          act_res(b, v);
          stage_bf16(stg, lane, by_half ? 0 : b, v);
          if (by_half)
            stage_flush(stg, lane, d.out_vec, d.out, false, row0, d.M, d.N, col_w + 32 * b,
                        std::min(d.N, col_w + 32 * b + 32));
        }
        if (!by_half)
          stage_flush(stg, lane, d.out_vec, d.out, false, row0, d.M, d.N, col_w, d.N);
      }
      ++tcount;
    }
    if (lane == 0 && res_open) wait_bar_drain(res_bar, res_n & 1, DRAIN_LIMIT);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 4) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_cg2(tmem_base, 512);
  }
}

// ---------------------------------------------------------------- single-CTA tiles, split contraction
struct CtaMaps {
  CUtensorMap a, b;
};
struct CtaParams {
  DenseProduct d;
  int swap;        // the tile's 128 rows run along the output's columns
  int Mr, Nc;      // extents along the tile's rows and columns
  int BN;          // tile columns (16..256, a multiple of 16)
  int splits;      // CTAs per cluster: pieces of the contraction
  int per;         // columns that each CTA of a cluster finishes (a multiple of 4, or of 8
                   // along the output's rows)
  int slots;       // of the ring, an even number
  int b_bytes;     // B bytes per block
  int nacc;        // accumulators (2 or 4), see the MMA loop
  int tmem_cols;
  int vec_out, vec_pre;  // stores in 16-byte pieces
};
constexpr int kCtaThreads = 256;  // warps 4 and 6 multiply, 5 and 7 load; 0-3 or all finish
constexpr int kCtaMeta = 256 + 1024;  // barriers, the tile's biases
constexpr int kMaxSlots = 12;
static_assert(8 * (2 * kMaxSlots + 2) + 8 <= 256, "barrier area");
size_t cta_smem(const CtaParams& c) {
  return 1024 + static_cast<size_t>(c.slots) * (OPER + c.b_bytes) +
         (c.splits > 1 ? static_cast<size_t>(c.splits) * c.per * 512 : 0) + kCtaMeta;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Sixteen columns of one row of a swapped tile, which are output[col, row]:
// consecutive lanes read and write consecutive elements.
__device__ __forceinline__ void residual16(const CtaParams& c, const DenseParams& p, int row, int col0,
                                           int end, float (&r)[16]) {
  const bool any = c.d.epilogue && p.residual && row < c.Mr;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    r[i] = any && col0 + i < end
               ? load_any(p.residual, p.res_f32, static_cast<long long>(col0 + i) * p.ldr + row)
               : 0.f;
}
__device__ __forceinline__ void finish16(const CtaParams& c, const DenseParams& p, float bias, int row,
                                         int col0, int end, float (&v)[16], const float (&r)[16]) {
  if (row >= c.Mr) return;
  const DenseProduct& d = c.d;
  const long long o = static_cast<long long>(col0) * d.N + row;
  const int nv = end - col0;
  auto store = [&](void* out, bool f32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i >= nv) continue;
      if (f32)
        static_cast<float*>(out)[o + static_cast<long long>(i) * d.N] = v[i];
      else
        static_cast<__nv_bfloat16*>(out)[o + static_cast<long long>(i) * d.N] = __float2bfloat16_rn(v[i]);
    }
  };
  if (d.epilogue) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += bias;
    if (p.pre) store(p.pre, false);
    act_all<16>(p.act, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += r[i];
  }
  store(d.out, d.out_f32);
}

template <bool A_MN, bool B_MN, bool SPLIT>
__global__ void __launch_bounds__(kCtaThreads, 2)
    dense_cta_kernel(const __grid_constant__ CtaMaps maps, const __grid_constant__ CtaParams c,
                     const __grid_constant__ DenseParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw_addr);
  const int b_bytes = c.b_bytes, slots = c.slots;
  const uint32_t stage_bytes = OPER + b_bytes;
  const int S = SPLIT ? c.splits : 1;
  const uint32_t recv = base + slots * stage_bytes;  // partial sums from the cluster
  const uint32_t meta = recv + (S > 1 ? S * c.per * 512 : 0);
  const uint32_t full = meta, empty = meta + 8 * kMaxSlots, acc_full = empty + 8 * kMaxSlots,
                 got = acc_full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (got + 8 - base));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / S;
  const int tr = cdiv(c.Mr, 128);
  const int m0 = (tile % tr) * 128, n0 = (tile / tr) * c.BN;
  const int nkb = cdiv(c.d.Kc, BK);
  const int kb0 = static_cast<int>(static_cast<long long>(rank) * nkb / S);
  const int kb1 = static_cast<int>(static_cast<long long>(rank + 1) * nkb / S);
  const int own0 = rank * c.per, own1 = std::min(c.BN, own0 + c.per);  // columns finished here

  if (warp == 5 && lane == 0) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (threadIdx.x < slots) {
    mbar_init(full + 8 * threadIdx.x, 1);
    mbar_init(empty + 8 * threadIdx.x, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    mbar_init(acc_full, 2);
    mbar_init(got, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (S > 1 && own1 > own0) mbar_arrive_expect_tx(got, S * (own1 - own0) * 512);
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(tmem_slot), c.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_arrive();  // this CTA's barriers exist
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{abort_flag, p.dev_status, p.wait_limit};

  // Warps 5 and 7 load, and warps 4 and 6 multiply, the even and the odd blocks:
  // waiting, issuing and committing take one warp 250 ns a block, a tile of 128
  // columns' MMAs 130 (1024 x 8192 x 1024 in whole tiles 35 us with one warp
  // of each kind, 22 with two).  The number of slots is even, so that a slot
  // has one warp on either side.  As above, the warps stay converged and
  // elected lanes issue.
  if (warp >= 4) {
    const int first = (warp - 4) >> 1;
    int s = first, it = first;
    uint32_t ph = 0;
    auto next = [&]() {
      it += 2;
      if ((s += 2) >= slots) s -= slots, ph ^= 1;
    };
    if (warp & 1) {
#pragma unroll 1
      for (int k = (kb0 + first) * BK; k < kb1 * BK; k += 2 * BK) {
        if (it >= slots && !__all_sync(0xffffffffu, wait_bar(empty + 8 * s, ph ^ 1, wc))) break;
        if (elect_one()) {
          const uint32_t fb = full + 8 * s;
          const uint32_t a = base + s * stage_bytes, b = a + OPER;
          mbar_arrive_expect_tx(fb, stage_bytes);
          if constexpr (A_MN) {
            tma_load_2d(a, &maps.a, fb, m0, k);
            tma_load_2d(a + CHUNK, &maps.a, fb, m0 + 64, k);
          } else {
            tma_load_2d(a, &maps.a, fb, k, m0);
          }
          if constexpr (B_MN) {
            for (int j = 0; j * CHUNK < b_bytes; ++j)
              tma_load_2d(b + j * CHUNK, &maps.b, fb, n0 + 64 * j, k);
          } else {
            tma_load_2d(b, &maps.b, fb, k, n0);
          }
        }
        next();
      }
      // the copies land before the block may exit
      for (int j = it - 2; j >= first && j > it - 2 - slots; j -= 2)
        wait_bar_drain(full + 8 * (j % slots), (j / slots) & 1, DRAIN_LIMIT);
    } else {
      const uint32_t idesc = idesc_bf16_f32(128, c.BN, A_MN, B_MN);
      constexpr uint64_t kA = (A_MN ? 16 * 128 : 32) >> 4, kB = (B_MN ? 16 * 128 : 32) >> 4;
      const uint64_t a0 = sw128_desc(base, A_MN ? CHUNK : 16, 1024);
      const uint64_t b0 = sw128_desc(base + OPER, B_MN ? CHUNK : 16, 1024);
      const uint32_t adv = stage_bytes >> 4;
      // Each warp has an accumulator of its own, or two where the tile is
      // narrow (an MMA that adds onto the accumulator of the one before waits
      // for it); the epilogue adds them up.
      const int own = c.nacc / 2;
      uint32_t dt[BK / 16];
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk) dt[kk] = tmem_base + (first + (kk & (own - 1)) * 2) * c.BN;
#pragma unroll 1
      for (int kb = kb0 + first; kb < kb1; kb += 2) {
        if (!__all_sync(0xffffffffu, wait_bar(full + 8 * s, ph, wc))) break;
        tc_fence_after();
        const uint64_t ad = a0 + s * adv, bd = b0 + s * adv;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            tc_mma_bf16(dt[kk], ad + kk * kA, bd + kk * kB, idesc, it > first || kk >= own);
          tc_commit(empty + 8 * s);
        }
        next();
      }
      if (elect_one()) {
        tc_commit(acc_full);
        wait_bar_drain(acc_full, 0, DRAIN_LIMIT);
      }
    }
    __syncwarp();
  }

  // ------------------------------------------------ epilogue
  // Thread = tile row (tensor memory lane).  Warps w and w + 4 can read the same
  // quarter of tensor memory: for wide tiles they share its columns (2048 x 2048 x
  // 2048 with a residual 22.7 to 19.0 us); of narrow ones, or with the tile's
  // rows along the output's columns, warps 0-3 finish alone, without waiting for
  // the others (16 x 7168 x 2048 8.0 to 7.1).
  const int quad = warp & 3, half = warp >> 2;
  const bool both = !c.swap && c.BN >= 128, epi_warp = both || warp < 4;
  auto sync_epi = [&]() {
    if (both)
      __syncthreads();
    else
      bar_named(1, 128);
  };
  const int tl = quad * 32 + lane;
  const int row = m0 + tl;
  const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
  // 16 columns from j, the accumulators added up (of a single block only the
  // first warp's are written)
  auto load16 = [&](int j, float(&v)[16]) {
    const int step = kb1 - kb0 > 1 ? 1 : 2;
    const bool two = step < c.nacc;
    float x[16];
    tmem_ld16(taddr + j, v);
    if (two) tmem_ld16(taddr + step * c.BN + j, x);
    tmem_ld_wait();
    if (two)
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] += x[i];
    for (int a = 2 * step; a < c.nacc; a += step) {
      tmem_ld16(taddr + a * c.BN + j, x);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] += x[i];
    }
  };
  // the same over the cluster's pieces, in rank order (the same bits every time)
  auto sum16 = [&](int j, float(&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    const uint32_t src = recv + (((j - own0) >> 2) * 128 + tl) * 16;
    for (int q = 0; q < S; ++q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (j + 4 * i >= own1) continue;
        const float4 x = ld_shared_v4(src + q * c.per * 512 + i * 2048);
        v[4 * i] += x.x, v[4 * i + 1] += x.y, v[4 * i + 2] += x.z, v[4 * i + 3] += x.w;
      }
    }
  };
  // the biases, and a swapped tile's first residuals, while the tile is
  // multiplied (each is an L2 latency that would follow the accumulators)
  const uint32_t biases = meta + 256;
  float bias_row = 0.f, res[16];
  const int cend = std::min(c.Nc, n0 + own1);
  if (epi_warp && c.d.epilogue && p.bias) {
    if (c.swap) {
      if (row < c.Mr) bias_row = load_any(p.bias, p.bias_f32, row);
    } else {
      for (int j = threadIdx.x; j < c.BN && warp < 4; j += 128)
        st_shared_f32(biases + 4 * j, n0 + j < c.Nc ? load_any(p.bias, p.bias_f32, n0 + j) : 0.f);
      sync_epi();
    }
  }
  if (c.swap && epi_warp) residual16(c, p, row, n0 + own0, cend, res);
  if (S > 1) cluster_wait();  // every CTA's barriers exist
  bool ok = false;
  if (epi_warp) {
    ok = __all_sync(0xffffffffu, wait_bar(acc_full, 0, wc));
    tc_fence_after();
  }
  if (S > 1 && epi_warp) {
    // Each CTA finishes `per` of the tile's columns: every CTA lays its partial
    // sums down over the ring (every MMA that read it is done) and sends each
    // its columns in one copy, counted on its barrier.  (Sixteen bytes at a
    // time from registers the receiver's count takes longer than the copy.)
#pragma unroll 1
    for (int j = 16 * half; j < c.BN; j += both ? 32 : 16) {
      float v[16];
      load16(j, v);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_shared_v4(base + (((j >> 2) + i) * 128 + tl) * 16, v[4 * i], v[4 * i + 1], v[4 * i + 2],
                     v[4 * i + 3]);
    }
    fence_proxy_async_smem();
    sync_epi();
    const int cols = min(c.per, c.BN - lane * c.per);  // of the CTA of rank `lane`
    if (warp == 0 && lane < S && cols > 0)
      dsmem_copy(mapa_shared(recv + rank * c.per * 512, lane), base + lane * c.per * 512, cols * 512,
                 mapa_shared(got, lane));
    __syncwarp();
    if (own1 > own0) ok = __all_sync(0xffffffffu, wait_bar(got, 0, wc)) && ok;
  }
  // After this barrier what the CTA sent has arrived (every CTA has waited for
  // all that was sent to it): its ring is free, and it may leave.
  if (S > 1) cluster_arrive();
  if (S > 1 && !c.swap) cluster_wait();
  if (ok && c.swap) {
#pragma unroll 1
    for (int j = own0; j < own1 && n0 + j < c.Nc; j += 16) {
      float v[16];
      if (S > 1)
        sum16(j, v);
      else
        load16(j, v);
      if (j > own0) residual16(c, p, row, n0 + j, cend, res);
      finish16(c, p, bias_row, row, n0 + j, cend, v, res);
    }
  } else if (ok) {
    // rows of the output: through staged blocks, over the pipeline's buffers;
    // the residual's blocks beside them
    const DenseProduct& d = c.d;
    const uint32_t stg = base + warp * 4096, stg_res = stg + (both ? 32768 : 16384);
    const int row0 = m0 + quad * 32;
    auto load32 = [&](int j, float(&v)[32]) {  // columns n0 + j .. with the bias
      float h[16];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (j + 16 * k >= own1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[16 * k + i] = 0.f;
          continue;
        }
        if (S > 1)
          sum16(j + 16 * k, h);
        else
          load16(j + 16 * k, h);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[16 * k + i] = h[i];
      }
      if (d.epilogue && p.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // (past BN: columns that are not stored)
          const float4 bv = ld_shared_v4(biases + 4 * j + 16 * i);
          v[4 * i] += bv.x, v[4 * i + 1] += bv.y, v[4 * i + 2] += bv.z, v[4 * i + 3] += bv.w;
        }
      }
    };
    const int per = d.out_f32 ? 32 : 64;
#pragma unroll 1
    for (int j0 = own0 + half * per; j0 < own1 && n0 + j0 < d.N; j0 += both ? 2 * per : per) {
      const int halves = std::min(per / 32, cdiv(own1 - j0, 32));
      if (d.epilogue && p.pre) {
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
          float v[32];
          load32(j0 + 32 * h, v);
          stage_bf16(stg, lane, h, v);
        }
        stage_flush(stg, lane, c.vec_pre, p.pre, false, row0, d.M, d.N, n0 + j0,
                    std::min(cend, n0 + j0 + per));
      }
#pragma unroll 1
      for (int h = 0; h < halves; ++h) {
        float v[32];
        load32(j0 + 32 * h, v);
        if (d.epilogue) {
          act_all<32>(p.act, v);
          if (p.residual)
            add_residual(p, stg_res, lane, row0, d.M, n0 + j0 + 32 * h, d.N, v);
        }
        if (d.out_f32)
          stage_f32(stg, lane, v);
        else
          stage_bf16(stg, lane, h, v);
      }
      stage_flush(stg, lane, c.vec_out, d.out, d.out_f32, row0, d.M, d.N, n0 + j0, cend);
    }
  }
  if (S > 1 && c.swap) cluster_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, c.tmem_cols);
  }
}

// ---------------------------------------------------------------- backward prep
// dz = bf16(dy act'(pre)) [T, ldz] in one pass, and the column sums of the
// unrounded dz over each block's rows: part[blockIdx.y][N].  Bound by its
// bytes: pieces of eight columns per thread (VEC = 8) where rows start on their
// boundaries, else of four, two or one.  A block is `lanes` threads along the columns
// and 256 / lanes rows; its partial sums add up in shared memory in row order.
struct DzArgs {
  const void* dy;
  long long lddy;
  const __nv_bfloat16* pre;
  int T, N, rows, lanes;
  __nv_bfloat16* dz;  // null: sums only
  int ldz;
  float* part;        // null: no sums
};
// VEC consecutive elements as they lie in memory
template <typename T, int VEC>
struct Piece {
  T v;
};
template <>
struct Piece<__nv_bfloat16, 2> {
  uint32_t q;
};
template <>
struct Piece<float, 2> {
  float2 q;
};
template <>
struct Piece<__nv_bfloat16, 4> {
  uint2 q;
};
template <>
struct Piece<float, 4> {
  float4 q;
};
template <>
struct Piece<__nv_bfloat16, 8> {
  uint4 q;
};
template <>
struct Piece<float, 8> {
  float4 q[2];
};
template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> load_piece(const T* p) {
  Piece<T, VEC> r;
  if constexpr (VEC == 8 && sizeof(T) == 4) {
    r.q[0] = reinterpret_cast<const float4*>(p)[0];
    r.q[1] = reinterpret_cast<const float4*>(p)[1];
  } else {
    r = *reinterpret_cast<const Piece<T, VEC>*>(p);
  }
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void floats(const Piece<T, VEC>& r, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = static_cast<float>(r.v);
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  } else {
    const float* f = reinterpret_cast<const float*>(&r);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = f[j];
  }
}
template <int VEC>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* o, const float (&v)[VEC]) {
  if constexpr (VEC == 1)
    *o = __float2bfloat16_rn(v[0]);
  else if constexpr (VEC == 2)
    *reinterpret_cast<uint32_t*>(o) = cvt_bf16x2(v[0], v[1]);
  else if constexpr (VEC == 4)
    *reinterpret_cast<uint2*>(o) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
  else
    *reinterpret_cast<uint4*>(o) = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                                              cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
}
template <int ACT, typename DT, int VEC>
__global__ void __launch_bounds__(256, 4) dense_dz_kernel(const DzArgs a) {
  __shared__ float acc[256 * VEC];
  pdl_trigger();
  pdl_wait();
  const int cx = threadIdx.x % a.lanes, ry = threadIdx.x / a.lanes, nr = 256 / a.lanes;
  const int n = (blockIdx.x * a.lanes + cx) * VEC;
  const int t0 = blockIdx.y * a.rows, t1 = min(a.T, t0 + a.rows);
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
  if (n < a.N) {
    // rows in batches whose loads are all issued before the first is used
    // (the stores to dz keep the compiler from moving later loads up)
    constexpr int U = VEC == 1 ? 8 : sizeof(DT) == 4 && VEC == 8 ? 2 : 4;
    for (int tb = t0 + ry; tb < t1; tb += U * nr) {
      Piece<DT, VEC> dy[U];
      Piece<__nv_bfloat16, VEC> pre[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = min(tb + u * nr, t1 - 1);  // (past the end: a row that is not used)
        dy[u] = load_piece<DT, VEC>(static_cast<const DT*>(a.dy) + t * a.lddy + n);
        if constexpr (ACT != kActNone)
          pre[u] = load_piece<__nv_bfloat16, VEC>(a.pre + static_cast<long long>(t) * a.N + n);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u * nr;
        if (t >= t1) break;
        float v[VEC];
        floats<DT, VEC>(dy[u], v);
        if constexpr (ACT != kActNone) {
          float z[VEC];
          floats<__nv_bfloat16, VEC>(pre[u], z);
          slope_n<ACT>(v, z);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += v[i];
        if (a.dz) store_bf16<VEC>(a.dz + static_cast<long long>(t) * a.ldz + n, v);
      }
    }
  }
  if (!a.part) return;
  const int width = a.lanes * VEC;
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[ry * width + cx * VEC + i] = sum[i];
  __syncthreads();
  const int c = threadIdx.x;
  if (c < width && blockIdx.x * width + c < a.N) {
    float v = 0.f;
    for (int r = 0; r < nr; ++r) v += acc[r * width + c];
    a.part[static_cast<long long>(blockIdx.y) * a.N + blockIdx.x * width + c] = v;
  }
}

// ---------------------------------------------------------------- host
}  // namespace

// Co-resident clusters of two (persistent grid).
int dense_pair_count() {  // (one block per SM, whatever the activation)
  static int cache[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && cache[dev]) return cache[dev];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms() & ~1);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, dense_pair_kernel<kActNone, false>, &cfg) != cudaSuccess || n < 1)
    n = num_sms() / 2;
  n = std::min(n, num_sms() / 2);
  if (dev < 64) cache[dev] = n;
  return n;
}

namespace {

template <int ACT, bool EXTRA>
cudaError_t launch_pairs_act(const PairMaps& maps, const DenseParams& p, const PairExtra& x, int total,
                             cudaStream_t st) {
  static bool done[64] = {};
  cudaError_t e = allow_smem(dense_pair_kernel<ACT, EXTRA>, kPairSmem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(dense_pair_kernel<ACT, EXTRA>, dim3(2 * std::min(dense_pair_count(), total)),
                    dim3(kPairThreads), kPairSmem, st, maps, p, x);
}

cudaError_t launch_pairs(DenseParams p, const PairOptions& opt, const DenseOperand* a, const DenseOperand* b,
                         int n, cudaStream_t st) {
  PairExtra x{};
  x.scale0 = opt.scale0, x.scale1 = opt.scale1;
  PairMaps maps;
  memset(&maps, 0, sizeof(maps));
  int total = 0;
  for (int q = 0; q < 2; ++q) {
    DenseProduct& d = p.pr[q];
    if (q >= n) {
      d.tiles = 0;
      continue;
    }
    x.slices[q] = std::max(1, opt.slices[q]);
    d.tiles = cdiv(d.M, 256) * cdiv(d.N, 256) * x.slices[q];
    total += d.tiles;
    d.out_vec = vec_rows(d.out, d.N, d.out_f32);
    if (!tmap_operand(&maps.a[q], a[q], d.a_mn, kHalf) ||
        !tmap_operand(&maps.b[q], b[q], d.b_mn, kHalf))
      return cudaErrorInvalidValue;
  }
  p.pre_vec = p.pre && vec_rows(p.pre, p.pr[0].N, false);
  const int pairs = std::min(dense_pair_count(), total);
  // a tile's time in blocks of the contraction: its own and storing it (see use_pairs)
  auto cost = [&](int q) {
    return q < n ? std::max(cdiv(cdiv(p.pr[q].Kc, BK), x.slices[q]) + 4, 9) : 0;
  };
  x.longer = cost(1) > cost(0);
  x.deal_pairs = p.pr[x.longer].tiles % pairs;
  x.deal = n > 1 && x.deal_pairs ? (2 * cost(x.longer) + cost(1 - x.longer)) / (2 * cost(1 - x.longer)) : 0;
  p.res_tma = p.residual && p.res_vec && p.pr[0].out_f32;
  if (p.res_tma && !encode_tmap_residual(&maps.res, p.residual, p.res_f32, x.slices[0] * p.pr[0].M, p.pr[0].N, p.ldr))
    return cudaErrorInvalidValue;
  if (p.act == kActScale) return launch_pairs_act<kActScale, true>(maps, p, x, total, st);
  if (n > 1 || x.slices[0] > 1) {  // (gradients: no activation)
    if (p.act != kActNone) return cudaErrorInvalidValue;
    return launch_pairs_act<kActNone, true>(maps, p, x, total, st);
  }
  if (p.act == kActRelu) return launch_pairs_act<kActRelu, false>(maps, p, x, total, st);
  if (p.act == kActSilu) return launch_pairs_act<kActSilu, false>(maps, p, x, total, st);
  if (p.act == kActGelu) return launch_pairs_act<kActGelu, false>(maps, p, x, total, st);
  return launch_pairs_act<kActNone, false>(maps, p, x, total, st);
}

// The kernel for a product, by estimated time in us, fitted to sweeps of 16 to
// 8192 rows, 64 to 2048 columns and contractions of 512 to 8192 over every tile
// width and split (within 10% of most).  A tile of 128 x BN takes 0.125 us a
// block of the contraction up to 32 columns (the handshakes), 0.19 at 128, 0.28
// at 256 (its MMAs and operands); two CTAs on an SM share that rate.  Storing
// it takes 0.4 us + 17 ns a column (14 a column of whole 128 where eight warps
// store it; 45 and 90 with its rows along the output's columns; 70 and 56 where
// rows do not start on 16-byte boundaries), joining S pieces 0.5 us a piece, 12
// ns a column of the tile and 55 of a CTA's own; a further round of CTAs that have
// an SM each starts 1.5 us late.  A 256 x 256 tile on a pair takes 0.275 us a
// block and 1.2 us to store (4.6), 2.5 at least.  Measured on both sides: 4096 x
// 2048 x 64 in tiles of 32 columns 6.9 us, of 128 8.3; 64 x 4096 x 2048 in four
// pieces of 32 columns 7.0, in eight 7.9, whole 11; 4096 x 4096 x 1024 in tiles
// of 256 24.7, of 128 30.2, on pairs 25.4; 13314 x 456 x 456 in tiles of 64 15.0,
// of 128 20.4; 5135 x 1928 x 626 on pairs 18.9, in tiles of 256 28.5; 16 x 7168 x
// 2048 in four pieces 7.0, in six 7.35, in eight 7.3.
// Clusters of eight CTAs that fill an SM each find too few places; tiles wider
// than 64 split at most four ways, wider than 128 not at all (their partial
// sums would not fit over the ring).
struct CtaPlan {
  bool swap;
  int BN, splits;
  double us;
};
bool whole_rows(const DenseProduct& d) { return vec_rows(d.out, d.N, d.out_f32); }
CtaPlan plan_cta(const DenseProduct& d) {
  CtaPlan best{false, 16, 1, 1e30};
  const int nkb = cdiv(d.Kc, BK);
  const int sms = num_sms();
  for (int swap = 0; swap < 2; ++swap) {
    const int mr = swap ? d.N : d.M, nc = swap ? d.M : d.N;
    // (a few rows on the 128-row side would be read by every tile at once:
    // 6 x 216 x 4248 9 us against 5)
    if (mr < 128 && nc > mr) continue;
    int last = 0;
    for (int bn : {16, 32, 64, 96, 128, 192, 256}) {
      if (bn > 16 && nc <= last) break;
      last = bn;
      const long long tiles = static_cast<long long>(cdiv(mr, 128)) * cdiv(nc, bn);
      for (int s : {1, 2, 3, 4, 8}) {
        if (s > nkb || s > (bn <= 64 ? 8 : bn <= 128 ? 4 : 1)) break;
        const int blocks = cdiv(nkb, s);
        const double column = swap ? (bn <= 64 ? 0.045 : 0.09) : whole_rows(d) ? 0.017 : 0.07;
        const double store = swap || bn < 128 ? column * bn : 0.8 * column * (128 * cdiv(bn, 128));
        const bool two = bn <= 64 || (bn <= 128 && (blocks + 1) * (OPER + 128 * bn) <= 110 * 1024);
        const long long ctas = tiles * s, slots = two ? 2LL * sms : sms;
        const double rounds = static_cast<double>((ctas + slots - 1) / slots);
        const double block = std::max(0.125, 0.1 + 0.0007 * bn) * (ctas > sms && two ? 2.05 : 1.0);
        const double join = s > 1 ? 0.5 * s + 0.012 * bn + 0.055 * cdiv(bn, s) : 0.0;
        const double us = 2.0 + rounds * (blocks * block + 0.4 + store + join) +
                          (two ? 0.0 : 1.5 * (rounds - 1));
        if (us < best.us) best = CtaPlan{swap != 0, bn, s, us};
      }
    }
  }
  return best;
}
bool use_pairs(const DenseProduct& d, const CtaPlan& cta) {
  const long long tiles = static_cast<long long>(cdiv(d.M, 256)) * cdiv(d.N, 256);
  const long long pairs = num_sms() / 2;
  const double tile = std::max(cdiv(d.Kc, BK) * 0.275 + (whole_rows(d) ? 1.2 : 4.6), 2.5);
  const double us = 6.4 + static_cast<double>((tiles + pairs - 1) / pairs) * tile;
  return us <= cta.us;
}

template <bool A_MN, bool B_MN, bool SPLIT>
cudaError_t launch_cta_s(const CtaMaps& maps, const CtaParams& c, const DenseParams& p,
                         cudaStream_t st) {
  static bool done[64] = {};
  auto kern = dense_cta_kernel<A_MN, B_MN, SPLIT>;
  cudaError_t e = allow_smem(kern, 232448, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cdiv(c.Mr, 128) * cdiv(c.Nc, c.BN) * c.splits);
  cfg.blockDim = dim3(kCtaThreads);
  cfg.dynamicSmemBytes = cta_smem(c);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, c, p);
}
template <bool A_MN, bool B_MN>
cudaError_t launch_cta_t(const CtaMaps& maps, const CtaParams& c, const DenseParams& p,
                         cudaStream_t st) {
  return c.splits > 1 ? launch_cta_s<A_MN, B_MN, true>(maps, c, p, st)
                      : launch_cta_s<A_MN, B_MN, false>(maps, c, p, st);
}

cudaError_t launch_cta(const DenseParams& p, int q, const CtaPlan& plan, const DenseOperand& a,
                       const DenseOperand& b, cudaStream_t st) {
  CtaParams c{};
  c.d = p.pr[q];
  c.swap = plan.swap;
  c.Mr = plan.swap ? c.d.N : c.d.M;
  c.Nc = plan.swap ? c.d.M : c.d.N;
  const DenseOperand& ra = plan.swap ? b : a;
  const DenseOperand& rb = plan.swap ? a : b;
  if (plan.swap) std::swap(c.d.a_mn, c.d.b_mn);
  c.BN = plan.BN;
  c.splits = plan.splits;
  c.per = c.swap ? (cdiv(c.BN, c.splits) + 3) & ~3 : (cdiv(c.BN, c.splits) + 7) & ~7;
  c.b_bytes = c.d.b_mn ? cdiv(c.BN, 64) * CHUNK : c.BN * 128;
  // The ring has an SM's room where every CTA has an SM of its own (512 x 2048 x
  // 2048 in tiles of 64 columns 7.8 us against 8.9), else half of it for narrow
  // tiles.  Clusters of eight leave the other half free: they find too few
  // places else (16 x 7168 x 2048 in eight pieces 10 us against 7).
  const long long ctas = static_cast<long long>(cdiv(c.Mr, 128)) * cdiv(c.Nc, c.BN) * c.splits;
  const bool alone = c.BN > 64 || (ctas <= num_sms() && c.splits <= 4);
  const int room = (alone ? 225 : 112) * 1024 - 1024 - kCtaMeta - (c.splits > 1 ? c.splits * c.per * 512 : 0);
  const int fit = std::min({kMaxSlots, room / (OPER + c.b_bytes), cdiv(cdiv(c.d.Kc, BK), c.splits) + 1});
  c.slots = std::max(2, fit & ~1);
  c.nacc = c.BN <= 64 ? 4 : 2;
  c.tmem_cols = 32;
  while (c.tmem_cols < c.nacc * c.BN) c.tmem_cols *= 2;
  c.vec_out = vec_rows(c.d.out, c.d.N, c.d.out_f32);
  c.vec_pre = p.pre && vec_rows(p.pre, c.d.N, false);
  CtaMaps maps;
  if (!tmap_operand(&maps.a, ra, c.d.a_mn, 128) || !tmap_operand(&maps.b, rb, c.d.b_mn, c.BN))
    return cudaErrorInvalidValue;
  if (c.d.a_mn)
    return c.d.b_mn ? launch_cta_t<true, true>(maps, c, p, st) : launch_cta_t<true, false>(maps, c, p, st);
  return c.d.b_mn ? launch_cta_t<false, true>(maps, c, p, st) : launch_cta_t<false, false>(maps, c, p, st);
}

// Blocks of the dz pass: columns first, then enough row ranges for two blocks
// per SM.
struct DzPlan {
  int vec, lanes, bx, by, rows;
};
DzPlan plan_dz(int T, int N, int vec) {
  DzPlan p;
  p.vec = vec;
  p.lanes = 32;
  while (p.lanes > 1 && (p.lanes / 2) * p.vec >= N) p.lanes /= 2;
  p.bx = cdiv(N, p.lanes * p.vec);
  const int per = 256 / p.lanes;  // rows of one step of a block
  p.by = std::max(1, std::min(cdiv(T, per), cdiv(4 * num_sms(), p.bx)));
  p.rows = cdiv(cdiv(T, p.by), per) * per;
  p.by = cdiv(T, p.rows);
  return p;
}
int max_partials(int T, int N) {
  int n = 1;
  for (int vec : {1, 2, 4, 8}) n = std::max(n, plan_dz(T, N, vec).by);
  return n;
}

template <int ACT, int VEC>
cudaError_t launch_dz_v(const DzPlan& pl, const DzArgs& a, bool dy_f32, cudaStream_t st) {
  const dim3 grid(pl.bx, pl.by), block(256);
  return dy_f32 ? launch_pdl(dense_dz_kernel<ACT, float, VEC>, grid, block, 0, st, a)
                : launch_pdl(dense_dz_kernel<ACT, __nv_bfloat16, VEC>, grid, block, 0, st, a);
}
template <int ACT>
cudaError_t launch_dz(const DzPlan& pl, const DzArgs& a, bool dy_f32, cudaStream_t st) {
  if (pl.vec == 8) return launch_dz_v<ACT, 8>(pl, a, dy_f32, st);
  if (pl.vec == 4) return launch_dz_v<ACT, 4>(pl, a, dy_f32, st);
  if (pl.vec == 2) return launch_dz_v<ACT, 2>(pl, a, dy_f32, st);
  return launch_dz_v<ACT, 1>(pl, a, dy_f32, st);
}

bool dy_is_operand(const DenseBackward& a) {
  return a.act == kActNone && !a.dy_f32 && a.lddy % 8 == 0 && aligned16(a.dy);
}
size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int dz_ld(int N) { return (N + 7) / 8 * 8; }

}  // namespace

size_t dense_bwd_ws_bytes(int T, int N) {
  return round256(static_cast<size_t>(T) * dz_ld(N) * 2) +
         round256(static_cast<size_t>(max_partials(T, N)) * N * 4);
}

cudaError_t launch_dense_forward(const DenseParams& p, const DenseOperand& x,
                                 const DenseOperand& W, cudaStream_t st) {
  const CtaPlan plan = plan_cta(p.pr[0]);
  return use_pairs(p.pr[0], plan) ? launch_pairs(p, PairOptions{}, &x, &W, 1, st)
                                  : launch_cta(p, 0, plan, x, W, st);
}

// Up to two products (those with an output): one launch where both take 256 x
// 256 tiles.  The epilogue's operands in p are the first one's.
cudaError_t launch_dense_products(const DenseParams& q, const PairOptions& opt, const DenseProduct* pr,
                                  const DenseOperand* a, const DenseOperand* b, cudaStream_t st) {
  DenseParams p = q;
  PairOptions o = opt;
  DenseOperand pa[2], pb[2];
  int n = 0;
  for (int i = 0; i < 2; ++i) {
    if (!pr[i].out) continue;
    p.pr[n] = pr[i];
    o.slices[n] = opt.slices[i];
    const CtaPlan plan = opt.always ? CtaPlan{} : plan_cta(pr[i]);
    if (opt.always || use_pairs(pr[i], plan)) {
      pa[n] = a[i], pb[n] = b[i];
      ++n;
      continue;
    }
    const cudaError_t e = launch_cta(p, n, plan, a[i], b[i], st);
    if (e != cudaSuccess) return e;
  }
  return n ? launch_pairs(p, o, pa, pb, n, st) : cudaSuccess;
}

// Up to four launches: dz, then dx and dW (one launch where both take 256 x
// 256 tiles), then the bias gradient's sums.  Each waits for the one before:
// dx, dW and the sums depend on dz alone, but only a grid's own wait makes an
// earlier grid's writes visible to it.
cudaError_t launch_dense_backward(const DenseBackward& a, void* ws, cudaStream_t st) {
  const bool direct = dy_is_operand(a);
  const int ldz = dz_ld(a.N);
  __nv_bfloat16* dz = static_cast<__nv_bfloat16*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                         round256(static_cast<size_t>(a.T) * ldz * 2));
  const bool gemm = a.dx || a.dW;
  __nv_bfloat16* dz_out = direct || !gemm ? nullptr : dz;
  float* part_out = a.db ? part : nullptr;
  cudaError_t e = cudaSuccess;
  int parts = 0;
  if (dz_out || part_out) {
    // the widest pieces that every row of dy and z starts on
    int vec = 8;
    while (vec > 1 && (a.N % vec || a.lddy % vec || !aligned16(a.dy) || !aligned16(a.pre))) vec /= 2;
    const DzPlan pl = plan_dz(a.T, a.N, vec);
    parts = pl.by;
    const DzArgs z{a.dy, a.lddy,  static_cast<const __nv_bfloat16*>(a.pre), a.T, a.N, pl.rows,
                   pl.lanes, dz_out, ldz, part_out};
    if (a.act == kActRelu) e = launch_dz<kActRelu>(pl, z, a.dy_f32, st);
    else if (a.act == kActSilu) e = launch_dz<kActSilu>(pl, z, a.dy_f32, st);
    else if (a.act == kActGelu) e = launch_dz<kActGelu>(pl, z, a.dy_f32, st);
    else e = launch_dz<kActNone>(pl, z, a.dy_f32, st);
    if (e != cudaSuccess) return e;
  }
  const DenseOperand z = direct ? DenseOperand{a.dy, a.T, a.N, a.lddy} : DenseOperand{dz, a.T, a.N, ldz};
  const DenseOperand x{a.x, a.T, a.K, a.ldx}, W{a.W, a.N, a.K, a.K};
  DenseParams p{};
  p.dev_status = a.dev_status;
  p.wait_limit = a.wait_limit;
  DenseProduct dx{}, dW{};
  dx.M = a.T, dx.N = a.K, dx.Kc = a.N, dx.b_mn = true, dx.out = a.dx;
  dW.M = a.N, dW.N = a.K, dW.Kc = a.T, dW.a_mn = dW.b_mn = true, dW.out = a.dW;
  const DenseProduct pr[2] = {dx, dW};
  const DenseOperand oa[2] = {z, z}, ob[2] = {W, x};
  if (e == cudaSuccess) e = launch_dense_products(p, PairOptions{}, pr, oa, ob, st);
  if (e == cudaSuccess && part_out)
    e = launch_column_sums(part, parts, a.N, a.db, nullptr, a.db_f32, st);
  return e;
}

}  // namespace mgg
