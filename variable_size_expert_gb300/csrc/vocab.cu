// Cross entropy over a vocabulary straight from the hidden states, the logits
// z = x W^T never kept:
//   forward   lse_t = log sum_v exp z_tv;  loss_t = lse_t - z_t,target + c lse_t^2
//   backward  d_tv = exp(z_tv - lse_t) (1 + 2 c lse_t) - [v = target_t]
//             dx = g d W,  dW = g d^T x
//
// Both directions run the 256 x 256 tiles of linear.cu's pair kernel (tcgen05,
// operands by TMA, two accumulators in tensor memory); what differs is the
// epilogue.  A thread holds one row (token) of the accumulator, so a tile's
// maximum and sum need no other lane.
//   forward   each tile leaves one pair (reference c, sum of 2^(z log2(e) - c)) a
//             row, 8 bytes for 256 logits, and the target's logit; a second
//             kernel joins the tiles' pairs and adds the losses up.
//   backward  the vocabulary in pieces: the logits again, d in bfloat16 into the
//             workspace (the operand of both products), then dx += d W and dW =
//             d^T x as one launch of the dense products, dx summed in f32 over
//             the pieces.  d is kept without the loss's gradient g, which
//             multiplies the accumulators: (p - 1) rounds to bfloat16 better
//             than any multiple of it, and a small g does not leave the type's
//             range.  (g of each token its own multiplies d before.)
//             Up to 128 tokens d is kept in two bfloat16 parts, as further rows of
//             both products: a tile of 256 rows has room for them, and with few
//             tokens there are no many roundings for one token's to vanish among
//             (one token: dW off by up to 2^-8 in its target's row, now by the
//             rounding of the result alone).
#include "pair.cuh"

namespace mgg {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct VocabMaps {
  CUtensorMap a, b;
};
struct VocabParams {
  int T, V, K;          // V: columns of this launch
  int v0, vocab;        // the first one's index, of how many in all
  const void* targets;  // [T] int64 or int32
  bool i64;
  long long ignore;
  // forward
  float2* part;         // [cdiv(V, 256)][T]: (c, sum)
  float* target_z;      // [T]
  int* ticket;          // zeroed for the joining kernel
  // backward
  const float* lse;
  float z2;             // 2 c
  const float* gtok;    // [T] or null; times *weight
  const float* weight;
  __nv_bfloat16* d;     // [T][ldd], 16-byte rows
  int ldd;
  bool split;           // d in two parts, rows t and T + t
  int32_t* dev_status;
  long long wait_limit;
};

// Token t's target: its index, -1 where it does not count, -2 where it is no index.
__device__ __forceinline__ int target_of(const void* targets, bool i64, long long ignore, int vocab,
                                         int t) {
  const long long y = i64 ? static_cast<const long long*>(targets)[t]
                          : static_cast<long long>(static_cast<const int32_t*>(targets)[t]);
  if (y == ignore) return -1;
  return y >= 0 && y < vocab ? static_cast<int>(y) : -2;
}

// Joins (c, s) and (c2, s2), sums relative to 2^c.
__device__ __forceinline__ void join(float& c, float& s, float c2, float s2) {
  const float m = fmaxf(c, c2);
  const float r = m == -INFINITY ? 0.f : m;
  s = s * exp2_f(c - r) + s2 * exp2_f(c2 - r);
  c = m;
}

template <bool BACK>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    vocab_pair_kernel(const __grid_constant__ VocabMaps maps, const __grid_constant__ VocabParams p) {
  extern __shared__ uint8_t smem_raw[];
  const PSmem m = carve_pair(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (warp == 5 && lane == 0) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (threadIdx.x == 0) init_pair(m);
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
  const int total = cdiv(p.T, 256) * cdiv(p.V, 256), nkb = cdiv(p.K, BK);
  const uint32_t full_l = mapa_shared(m.full, 0);
  const uint32_t acc_empty_l = mapa_shared(m.acc_empty, 0);
  if (!BACK && blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;

  if (warp == 5) {
    // ------------------------------------------------ TMA
    Ring r{0, 0, 0};
    bool ok = true;
    for (int tau = pair; ok && tau < total; tau += npairs) {
      int m0, n0;
      band_tile(tau, p.T, p.V, m0, n0);
      const int half = static_cast<int>(rank) * kHalf;
      ok = produce<false, false>(m, &maps.a, &maps.b, full_l, leader, m0 + half, n0 + half, nkb, r, wc);
    }
    if (lane == 0) drain_copies(m, r.it, leader);
    __syncwarp();
  } else if (warp == 4) {
    // ------------------------------------------------ MMA issue
    if (leader) {
      int tcount = 0;
      Ring r{0, 0, 0};
      for (int tau = pair; tau < total; tau += npairs) {
        const int acc = tcount & 1;
        if (!__all_sync(0xffffffffu, wait_bar(m.acc_empty + 8 * acc, ((tcount >> 1) & 1) ^ 1, wc)))
          break;
        tc_fence_after();
        if (!multiply<false, false>(m, tmem_base + acc * 256, nkb, r, wc)) break;
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
    // Four warps per 64 columns of the tile, a warp 32 rows, a lane one.
    const int quad = warp & 3, group = warp < 4 ? 0 : (warp - 2) >> 2;
    const int ew = group * 4 + quad;
    const uint32_t stg = m.sEpi + ew * EPI_WARP;
    // (forward) the groups' statistics, two tiles' in turn: [tile][group][row]
    const uint32_t stat = m.sEpi + quad * 2048 + lane * 8;
    int tcount = 0;
    for (int tau = pair; tau < total; tau += npairs) {
      int m0, n0;
      band_tile(tau, p.T, p.V, m0, n0);
      const int row0 = m0 + static_cast<int>(rank) * kHalf + quad * 32, row = row0 + lane;
      const int acc = tcount & 1;
      const int col_w = n0 + group * 64;
      const int nv = p.V - col_w;  // columns from col_w on (may be none)
      // while the tile is multiplied: the row's target, of this warp's columns
      const int y = row < p.T ? target_of(p.targets, p.i64, p.ignore, p.vocab, row) : -1;
      const int at = y >= 0 ? y - p.v0 - col_w : -1;
      float ref = 0.f, f = 0.f, one = 0.f;
      if (BACK && row < p.T) {
        const float lse = p.lse[row];
        const float g = y < 0 ? 0.f : p.gtok ? p.gtok[row] * *p.weight : 1.f;
        ref = lse * kLog2e;
        f = (1.f + p.z2 * lse) * g;
        one = g;
        if (y == -2 && p.v0 + col_w == 0) atomicOr(p.dev_status, kDevBadTarget);
      }
      bool ok = __all_sync(0xffffffffu, wait_bar(m.acc_full + 8 * acc, (tcount >> 1) & 1, wc));
      // the four groups of a quarter meet below: they leave together
      if (!BACK) ok = bar_and(1 + quad, 128, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr =
          tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256 + group * 64;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_l + 8 * acc);
      };
      if constexpr (BACK) {
        if (nv <= 0) release();
        // (few tokens) d in two parts: rounded, and what the rounding left
        const int parts = nv <= 0 ? 0 : p.split ? 2 : 1;
#pragma unroll 1
        for (int part = 0; part < parts; ++part) {
#pragma unroll 1
          for (int b = 0; b < 2 && 32 * b < nv; ++b) {
            float v[32];
            tmem_ld32(taddr + b * 32, v);
            tmem_ld_wait();
            if (part + 1 == parts && (b == 1 || nv <= 32)) release();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = exp2_f(fmaf(v[i], kLog2e, -ref)) * f;
            const int i1 = at - 32 * b;
            if (__any_sync(0xffffffffu, i1 >= 0 && i1 < 32)) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i == i1) v[i] -= one;
            }
            if (y < 0) {  // (also where the row's logits are not finite)
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0.f;
            }
            if (part) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] -= __bfloat162float(__float2bfloat16_rn(v[i]));
            }
            stage_bf16(stg, lane, b, v);
          }
          stage_flush(stg, lane, true, p.d + static_cast<long long>(part) * p.T * p.ldd, false, row0, p.T,
                      p.ldd, col_w, p.V);
        }
      } else {
        float v[64];
        {
          float(&lo)[32] = *reinterpret_cast<float(*)[32]>(v);
          float(&hi)[32] = *reinterpret_cast<float(*)[32]>(v + 32);
          tmem_ld32(taddr, lo);
          tmem_ld32(taddr + 32, hi);
          tmem_ld_wait();
        }
        release();
        if (nv < 64) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= nv) v[i] = -INFINITY;
        }
        if (at >= 0 && at < 64) {
          float z = 0.f;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i == at) z = v[i];
          p.target_z[row] = z;
        }
        float top[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) top[i] = v[i];
#pragma unroll
        for (int i = 8; i < 64; ++i) top[i & 7] = fmaxf(top[i & 7], v[i]);
#pragma unroll
        for (int w = 4; w > 0; w /= 2)
#pragma unroll
          for (int i = 0; i < w; ++i) top[i] = fmaxf(top[i], top[i + w]);
        // c as it is rounded is what the sum refers to: no error of it is left
        const float c = top[0] * kLog2e;
        const F2 mc = both(c == -INFINITY ? 0.f : -c), l2 = both(kLog2e);
        F2 sum[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float e0, e1;
          unpack2(fma2(pack2(v[i], v[i + 1]), l2, mc), e0, e1);
          sum[(i >> 1) & 3] = add2(sum[(i >> 1) & 3], pack2(exp2_f(e0), exp2_f(e1)));
        }
        float s0, s1;
        unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
        float s = s0 + s1, cc = c;
        // the four groups of a quarter meet in shared memory: one barrier a tile,
        // as the first group reads this tile's half while the others write the
        // next tile's
        const uint32_t mine = stat + (tcount & 1) * 1024;
        if (group) {
          st_shared_f32(mine + group * 256, cc);
          st_shared_f32(mine + group * 256 + 4, s);
        }
        bar_named(1 + quad, 128);
        if (group == 0 && row < p.T) {
#pragma unroll
          for (int g = 1; g < 4; ++g)
            join(cc, s, ld_shared_f32(mine + g * 256), ld_shared_f32(mine + g * 256 + 4));
          p.part[static_cast<long long>(n0 >> 8) * p.T + row] = make_float2(cc, s);
        }
      }
      ++tcount;
    }
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

// ---------------------------------------------------------------- joining the tiles
// A block joins the pairs of 32 tokens (a lane each, the tiles dealt out to its
// eight warps), and the block that ends last adds up the blocks' losses in their
// order: the same bits every time.
struct JoinParams {
  const float2* part;
  int tiles, T, vocab;
  const float* target_z;
  const void* targets;
  bool i64;
  long long ignore;
  float zc;
  int reduction;  // MGG_REDUCE_*
  float* lse;
  float* losses;  // [T] with MGG_REDUCE_NONE
  float* total;   // [1] otherwise
  float* weight;  // [1]
  float2* blocks;
  int* ticket;
  int32_t* dev_status;
};
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) vocab_join_kernel(const JoinParams p) {
  __shared__ float2 sh[8][32];
  __shared__ bool last;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * 32 + lane;
  float c = -INFINITY, s = 0.f;
  if (t < p.T) {
    for (int i = warp; i < p.tiles; i += 32) {
      float2 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        q[u] = i + 8 * u < p.tiles ? p.part[static_cast<long long>(i + 8 * u) * p.T + t]
                                   : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int u = 0; u < 4; ++u) join(c, s, q[u].x, q[u].y);
    }
  }
  sh[warp][lane] = make_float2(c, s);
  __syncthreads();
  if (warp == 0) {
    float loss = 0.f, n = 0.f;
    if (t < p.T) {
#pragma unroll
      for (int w = 1; w < 8; ++w) join(c, s, sh[w][lane].x, sh[w][lane].y);
      const float lse = kLn2 * (c + log2f(s));
      p.lse[t] = lse;
      const int y = target_of(p.targets, p.i64, p.ignore, p.vocab, t);
      if (y >= 0) {
        loss = lse - p.target_z[t] + p.zc * lse * lse;
        n = 1.f;
      } else if (y == -2) {
        atomicOr(p.dev_status, kDevBadTarget);
      }
      if (p.reduction == MGG_REDUCE_NONE) p.losses[t] = loss;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
      loss += __shfl_xor_sync(0xffffffffu, loss, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (lane == 0) {
      p.blocks[blockIdx.x] = make_float2(loss, n);
      __threadfence();
      last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float loss = 0.f, n = 0.f;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kJoinThreads) {
    const float2 q = __ldcg(p.blocks + i);
    loss += q.x, n += q.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    loss += __shfl_xor_sync(0xffffffffu, loss, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if (lane == 0) sh[0][warp] = make_float2(loss, n);
  __syncthreads();
  if (threadIdx.x == 0) {
    loss = 0.f, n = 0.f;
    for (int w = 0; w < 8; ++w) loss += sh[0][w].x, n += sh[0][w].y;
    const float w = p.reduction == MGG_REDUCE_MEAN ? 1.f / fmaxf(n, 1.f) : 1.f;
    if (p.reduction != MGG_REDUCE_NONE) *p.total = loss * w;
    *p.weight = w;
  }
}

__global__ void vocab_empty_kernel(float* total, float* weight) {
  if (total) *total = 0.f;
  *weight = 1.f;
}

template <bool BACK>
cudaError_t launch_tiles(const DenseOperand& x, const DenseOperand& W, const VocabParams& p,
                         cudaStream_t st) {
  static bool done[64] = {};
  cudaError_t e = allow_smem(vocab_pair_kernel<BACK>, kPairSmem, done);
  if (e != cudaSuccess) return e;
  VocabMaps maps;
  if (!tmap_operand(&maps.a, x, false, kHalf) || !tmap_operand(&maps.b, W, false, kHalf))
    return cudaErrorInvalidValue;
  const long long tiles = static_cast<long long>(cdiv(p.T, 256)) * cdiv(p.V, 256);
  return launch_pdl(vocab_pair_kernel<BACK>,
                    dim3(2 * static_cast<int>(std::min<long long>(dense_pair_count(), tiles))),
                    dim3(kPairThreads), kPairSmem, st, maps, p);
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Tokens up to which d is kept in two parts.
constexpr int kSplitTokens = 128;

// [x; x], rows dense: the other operand of d's two parts in dW.
__global__ void __launch_bounds__(256) vocab_twice_kernel(const uint4* x, long long ldx, int T, int K8, uint4* out) {
  pdl_trigger();
  pdl_wait();
  for (int i = blockIdx.x * 256 + threadIdx.x; i < T * K8; i += gridDim.x * 256) {
    const int t = i / K8, k = i - t * K8;
    const uint4 v = x[t * ldx + k];
    out[i] = v;
    out[T * K8 + i] = v;
  }
}
// dx = scale (rows t + rows T + t of sum)
__global__ void __launch_bounds__(256) vocab_join_dx_kernel(const float4* sum, const float* scale0,
                                                            const float* scale1, int n4, uint2* dx) {
  pdl_trigger();
  pdl_wait();
  const float g = scale0 ? *scale0 * *scale1 : 1.f;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n4; i += gridDim.x * 256) {
    const float4 a = sum[i], b = sum[n4 + i];
    dx[i] = make_uint2(cvt_bf16x2((a.x + b.x) * g, (a.y + b.y) * g), cvt_bf16x2((a.z + b.z) * g, (a.w + b.w) * g));
  }
}

// Columns of a piece of the backward: d takes rows x that many bfloat16 values.
int piece_columns(int T, int V) {
  const long long most = 64LL << 20;  // bytes of d
  const int rows = T <= kSplitTokens ? 2 * T : T;
  const long long cols = std::max<long long>(2048, most / (2LL * rows) / 256 * 256);
  return static_cast<int>(std::min<long long>(cols, (V + 7) / 8 * 8));
}
// What the backward keeps: d; the f32 sum of dx (over pieces or parts); [x; x].
struct BackLayout {
  int cols;
  bool split;
  size_t sum, twice, total;  // offsets of the second and third
};
BackLayout back_layout(int T, int K, int V) {
  BackLayout l;
  l.cols = piece_columns(T, V);
  l.split = T <= kSplitTokens;
  const size_t rows = l.split ? 2 * static_cast<size_t>(T) : T;
  l.sum = round256(rows * l.cols * 2);
  l.twice = l.sum + (l.split || l.cols < V ? round256(rows * K * 4) : 0);
  l.total = l.twice + (l.split ? round256(rows * K * 2) : 0);
  return l;
}

}  // namespace

// forward: the tiles' pairs, the targets' logits, the joining blocks' sums, their ticket
size_t vocab_fwd_ws_bytes(int T, int V) {
  return round256(static_cast<size_t>(cdiv(V, 256)) * T * 8) + round256(static_cast<size_t>(T) * 4) +
         round256(static_cast<size_t>(cdiv(T, 32)) * 8) + 256;
}
size_t vocab_bwd_ws_bytes(int T, int K, int V) { return back_layout(T, K, V).total; }

cudaError_t launch_vocab_forward(const VocabForward& a, void* ws, cudaStream_t st) {
  if (a.T == 0) {
    vocab_empty_kernel<<<1, 1, 0, st>>>(a.reduction == MGG_REDUCE_NONE ? nullptr : a.loss, a.weight);
    return cudaGetLastError();
  }
  char* at = static_cast<char*>(ws);
  auto take = [&](size_t bytes) {
    char* r = at;
    at += round256(bytes);
    return r;
  };
  const int tn = cdiv(a.V, 256);
  VocabParams p{};
  p.T = a.T, p.V = a.V, p.K = a.K, p.vocab = a.V;
  p.targets = a.targets, p.i64 = a.i64, p.ignore = a.ignore;
  p.part = reinterpret_cast<float2*>(take(static_cast<size_t>(tn) * a.T * 8));
  p.target_z = reinterpret_cast<float*>(take(static_cast<size_t>(a.T) * 4));
  JoinParams j{};
  j.blocks = reinterpret_cast<float2*>(take(static_cast<size_t>(cdiv(a.T, 32)) * 8));
  p.ticket = reinterpret_cast<int*>(take(4));
  p.dev_status = a.dev_status, p.wait_limit = a.wait_limit;
  cudaError_t e = launch_tiles<false>(DenseOperand{a.x, a.T, a.K, a.ldx}, DenseOperand{a.W, a.V, a.K, a.K}, p, st);
  if (e != cudaSuccess) return e;
  j.part = p.part, j.tiles = tn, j.T = a.T, j.vocab = a.V, j.target_z = p.target_z;
  j.targets = a.targets, j.i64 = a.i64, j.ignore = a.ignore, j.zc = a.z_loss, j.reduction = a.reduction;
  j.lse = a.lse, j.losses = a.loss, j.total = a.loss, j.weight = a.weight;
  j.ticket = p.ticket, j.dev_status = a.dev_status;
  return launch_pdl(vocab_join_kernel, dim3(cdiv(a.T, 32)), dim3(kJoinThreads), 0, st, j);
}

cudaError_t launch_vocab_backward(const VocabBackward& a, void* ws, cudaStream_t st) {
  const BackLayout l = back_layout(a.T, a.K, a.V);
  char* const base = static_cast<char*>(ws);
  __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(base);
  float* sum = reinterpret_cast<float*>(base + l.sum);
  const int rows = l.split ? 2 * a.T : a.T;
  const DenseOperand x{a.x, a.T, a.K, a.ldx};
  DenseOperand xd = x;  // beside d's rows
  const float* const scale = a.per_token ? nullptr : a.dloss;
  cudaError_t e = cudaSuccess;
  if (l.split && a.dW) {
    void* twice = base + l.twice;
    const int K8 = a.K / 8;
    e = launch_pdl(vocab_twice_kernel, dim3(cdiv(a.T * K8, 256)), dim3(256), 0, st,
                   static_cast<const uint4*>(a.x), a.ldx / 8, a.T, K8, static_cast<uint4*>(twice));
    xd = DenseOperand{twice, rows, a.K, a.K};
  }
  for (int v0 = 0; e == cudaSuccess && v0 < a.V; v0 += l.cols) {
    const int n = std::min(l.cols, a.V - v0);
    const char* W = static_cast<const char*>(a.W) + static_cast<size_t>(v0) * a.K * 2;
    VocabParams p{};
    p.T = a.T, p.V = n, p.K = a.K, p.v0 = v0, p.vocab = a.V;
    p.targets = a.targets, p.i64 = a.i64, p.ignore = a.ignore;
    p.lse = a.lse, p.z2 = 2.f * a.z_loss, p.gtok = a.per_token ? a.dloss : nullptr, p.weight = a.weight;
    p.d = d, p.ldd = l.cols, p.split = l.split;
    p.dev_status = a.dev_status, p.wait_limit = a.wait_limit;
    const DenseOperand Wp{W, n, a.K, a.K}, dp{d, rows, n, l.cols};
    e = launch_tiles<true>(x, Wp, p, st);
    if (e != cudaSuccess) return e;
    const bool first = v0 == 0, direct = v0 + n == a.V && !l.split;  // dx in place
    // Every product is multiplied by the loss's gradient as it leaves, but dx's
    // parts, which meet first.
    DenseParams q{};
    q.scale0 = scale, q.scale1 = a.weight;
    q.dev_status = a.dev_status, q.wait_limit = a.wait_limit;
    DenseProduct dx{}, dW{};
    dx.M = rows, dx.N = a.K, dx.Kc = n, dx.b_mn = true;
    dx.out = !a.dx ? nullptr : direct ? a.dx : sum;
    dx.out_f32 = !direct, dx.epilogue = !first;
    dW.M = n, dW.N = a.K, dW.Kc = rows, dW.a_mn = dW.b_mn = true;
    dW.out = a.dW ? static_cast<char*>(a.dW) + static_cast<size_t>(v0) * a.K * 2 : nullptr;
    if (!first) {
      q.residual = sum;
      q.res_f32 = q.res_vec = true;
      q.ldr = a.K;
    }
    q.act = scale ? kActScale : kActNone;
    const DenseOperand oa[2] = {dp, dp}, ob[2] = {Wp, xd};
    if (l.split && scale) {
      const DenseProduct none{}, only_dx[2] = {dx, none}, only_dW[2] = {none, dW};
      DenseParams plain = q;
      plain.act = kActNone;
      e = launch_dense_products(plain, only_dx, oa, ob, st);
      if (e == cudaSuccess) {
        q.residual = nullptr;
        e = launch_dense_products(q, only_dW, oa, ob, st);
      }
    } else {
      const DenseProduct pr[2] = {dx, dW};
      e = launch_dense_products(q, pr, oa, ob, st);
    }
  }
  if (e == cudaSuccess && l.split && a.dx)
    e = launch_pdl(vocab_join_dx_kernel, dim3(cdiv(a.T * a.K / 4, 256)), dim3(256), 0, st,
                   reinterpret_cast<const float4*>(sum), scale, a.weight, a.T * a.K / 4,
                   static_cast<uint2*>(a.dx));
  return e;
}

}  // namespace mgg
