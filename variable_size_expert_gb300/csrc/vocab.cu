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
//             Up to 4 tokens d is kept in f32 and both gradients leave one pass over
//             W.  Up to 128 d is kept in two bfloat16 parts, as further rows of
//             both products: a tile of 256 rows has room for them, and with few
//             tokens there are no many roundings for one token's to vanish among
//             (one token: dW off by up to 2^-8 in its target's row, now by the
//             rounding of the result alone).  Beyond, d's rounding takes the gradients'
//             relative error from 0.00165 (the result's own) to 0.0019, with a gradient
//             of each token its own to 0.0024; a second part would double the products.
//             Tokens that do not count have d = 0, which is not enough for dW: 0 times
//             a NaN or an infinity in their rows of x would be NaN in all of it.  dW's
//             x is therefore a copy in which their rows are zeros.
//
// Bound by the matrix units at the power limit: loss of 8192 x 2048 x 32768 645 us
// (1705 TFLOP/s), gradients of 4096 x 2048 x 32768 990 us (1666); with few tokens by
// the weights' bytes.
#include <stdlib.h>

#include "pair.cuh"

namespace mgg {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The matrix units cut every sum they add to off: over 2048 terms a logit loses 1.3e-5
// of 6 or so, always towards zero, and a loss, which averages many, keeps that (1.6e-6
// of it, ten times the error of f32 sums).  The forward therefore has them add up a
// run of blocks at a time and adds those sums in f32, in the registers of the epilogue,
// under the next run's products.  Runs of eight blocks (512 terms) leave 3e-7 to 5e-7
// of a mean over many tokens; of 8192 x 2048 x 32768 they take 636 us, of four 670, of
// two 754.  With up to 256 tokens, where W's bytes are the bound and few tokens average
// less away, four (two with up to 32) cost nothing.  (For d a logit need not be as good.)
constexpr int kRunBlocks = 8, kRunFew = 4, kRunFewest = 2;

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
  float2* part;         // [tiles along V][T]: (c, sum)
  float* target_z;      // [T]
  int* ticket;          // zeroed for the joining kernel
  int run;              // see kRunBlocks
  // backward
  const float* lse;
  float z2;             // 2 c
  const float* gtok;    // [T] or null; times *weight
  const float* weight;
  __nv_bfloat16* d;     // [T][ldd], 16-byte rows
  int ldd;
  bool split;           // d in two parts, rows t and T + t
  const uint4* x;       // rows ldx8 16-byte pieces apart, to copy as dW's operand,
  uint4* x_out;         // out_ld8 apart; or null
  long long ldx8, out_ld8;
  float* df;            // or d in f32, [T][ldd] (few tokens)
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

// Thread `at` of `step`: its share of the copy of rows x K8 16-byte pieces, `ld` apart, to
// rows `out_ld` apart; `copies` of all, one behind the other.  With targets the rows of
// tokens that do not count become zeros.  Four pieces are under way a thread.
__device__ __forceinline__ void copy_pieces(const uint4* x, long long ld, int rows, int K8, uint4* out,
                                            long long out_ld, int copies, const void* targets, bool i64,
                                            long long ignore, int vocab, int at, int step) {
  const int dt = step / K8, dk = step % K8;
  int t = at / K8, k = at % K8;
  while (t < rows) {
    uint4 v[4];
    long long to[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      to[u] = t < rows ? t * out_ld + k : -1;
      v[u] = make_uint4(0, 0, 0, 0);
      if (t < rows && (!targets || target_of(targets, i64, ignore, vocab, t) >= 0)) v[u] = x[t * ld + k];
      t += dt, k += dk;
      if (k >= K8) k -= K8, ++t;
    }
    for (int c = 0; c < copies; ++c)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (to[u] >= 0) out[c * rows * out_ld + to[u]] = v[u];
  }
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
  // blocks of the contraction that one accumulator adds up
  const int run = BACK ? nkb : p.run;
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
      ok = produce<false, false>(m, &maps.a, &maps.b, full_l, leader, m0 + half, n0 + half, 0, nkb, r, wc);
    }
    if (lane == 0) drain_copies(m, r.it, leader);
    __syncwarp();
  } else if (warp == 4) {
    // ------------------------------------------------ MMA issue
    if (leader) {
      int tcount = 0;
      Ring r{0, 0, 0};
      bool ok = true;
      for (int tau = pair; ok && tau < total; tau += npairs) {
        for (int kb = 0; ok && kb < nkb; kb += run, ++tcount) {
          const int acc = tcount & 1;
          ok = __all_sync(0xffffffffu, wait_bar(m.acc_empty + 8 * acc, ((tcount >> 1) & 1) ^ 1, wc));
          if (!ok) break;
          tc_fence_after();
          ok = multiply<false, false>(m, tmem_base + acc * 256, min(run, nkb - kb), r, wc);
          if (ok && elect_one()) tc_commit_cg2_mc(m.acc_full + 8 * acc, 0x3);
        }
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
    int tcount = 0, parity = 0;
    // dW's x, while the first tile is multiplied.  (A launch of its own costs 3 us:
    // gradients of 512 x 2048 x 32768 153 us with it, 149 so and without any copy; with few
    // columns, whose products are no longer than the copy, 16384 x 512 x 1024 101 and 95.)
    if (BACK && p.x_out)
      copy_pieces(p.x, p.ldx8, p.T, p.K >> 3, p.x_out, p.out_ld8, 1, p.targets, p.i64, p.ignore, p.vocab,
                  (blockIdx.x * kEpiWarps + ew) * 32 + lane, gridDim.x * kEpiWarps * 32);
    for (int tau = pair; tau < total; tau += npairs, parity ^= 1) {
      int m0, n0;
      band_tile(tau, p.T, p.V, m0, n0);
      const int row0 = m0 + static_cast<int>(rank) * kHalf + quad * 32, row = row0 + lane;
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
      auto arrived = [&]() {
        const bool ok = __all_sync(0xffffffffu, wait_bar(m.acc_full + 8 * (tcount & 1), (tcount >> 1) & 1, wc));
        tc_fence_after();
        return ok;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_l + 8 * (tcount & 1));
      };
      const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + group * 64;
      if constexpr (BACK) {
        if (!arrived()) break;
        const uint32_t taddr = taddr0 + (tcount & 1) * 256;
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
        bool ok = true;
        for (int kb = 0; ok && kb < nkb; kb += run) {
          ok = arrived();
          if (!ok) break;
          const uint32_t taddr = taddr0 + (tcount & 1) * 256;
          // (sixteen columns at a time: 64 sums and 32 more do not fit a thread's 96
          // registers, and with spilled ones 8192 x 2048 x 32768 takes 876 us, not 632)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float x[16];
            tmem_ld16(taddr + 16 * q, x);
            tmem_ld_wait();
            if (q == 3) release();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[16 * q + i] = kb ? v[16 * q + i] + x[i] : x[i];
          }
          ++tcount;
        }
        // the four groups of a quarter meet below: they leave together
        if (!bar_and(1 + quad, 128, ok)) break;
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
        const uint32_t mine = stat + parity * 1024;
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
      if (BACK) ++tcount;
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

// ---------------------------------------------------------------- few tokens
// Up to 32 tokens the weights' bytes are the bound: tiles of 128 rows of W by N
// tokens (16 or 32), W's rows on the rows of the accumulator, two blocks an SM with a
// ring each, so that 190 KB an SM are in flight: the loss of 16 x 2048 x 32768 29 us
// (134 MB, 68% of the measured copy rate; start, last epilogue and the joining kernel
// are 9 of it).  A vocabulary of few tiles leaves SMs idle: the blocks of a cluster then share
// a tile's contraction out, leave their sums in shared memory and finish a share of its
// tokens each.  On pair tiles every SM asks for the same few rows of x at once, 40
// us (of 64 tokens 32 there, 34 here); one block an SM that walks over the tiles with
// two accumulators 31.6.  A lane then holds a vocabulary entry, not a token: the
// forward turns the tile through shared memory and reduces a token with a warp, the
// backward stores d as it lies.  The forward's runs of the contraction have an
// accumulator each and meet in f32 (see kRunBlocks); runs beyond half of the tensor
// memory (contractions over 2048, over 1024 from 17 tokens on) take the accumulators in
// turn, and the epilogue's warps empty one while the next are multiplied (16 x 2048 x
// 32768, where both ways are open, 29.1 us so, 28.2 with all read at the end).  With
// longer runs in place of more of them 32 tokens' lse of 32 x 16384 x 19500 were 7.7e-6
// of 11.9 too low on average (positive terms: 1.5e-4 of 74); so 7e-7 and 1e-6, as at any
// other length.
constexpr int kFewTokens = 32, kFewThreads = 192, kFewSlots = 6, kFewAccs = 16;
constexpr int kFewMeta = 512;
struct FewParams {
  int N;          // tokens of a block, rounded up to 16
  int split;      // blocks of a cluster that share the contraction out
  int slots, run, tmem_cols;
  int accs;       // accumulators, up to kFewAccs
};
size_t few_smem(int N, int slots) {
  return 1024 + std::max(static_cast<size_t>(slots) * (OPER + N * 128), static_cast<size_t>(N) * 132 * 4) + kFewMeta;
}
template <bool BACK, bool SPLIT>
__global__ void __launch_bounds__(kFewThreads, 2)
    vocab_few_kernel(const __grid_constant__ VocabMaps maps, const __grid_constant__ VocabParams p,
                     const __grid_constant__ FewParams f) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw_addr);
  const uint32_t stage = OPER + f.N * 128;
  const uint32_t ring = max(f.slots * stage, f.N * 132u * 4);
  const uint32_t full = base + ring, empty = full + 8 * kFewSlots, done = empty + 8 * kFewSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + ring + 16 * kFewSlots + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t acc_full = done + 16, acc_empty = acc_full + 8 * kFewAccs;  // (forward)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = SPLIT ? f.split : 1, tile = blockIdx.x / split, rank = blockIdx.x % split;
  const int n0 = tile * 128, t0 = SPLIT ? blockIdx.y * kFewTokens : 0;
  const int kb0 = cdiv(p.K, BK) * rank / split, nkb = cdiv(p.K, BK) * (rank + 1) / split - kb0;
  const int runs = cdiv(nkb, f.run);
  const bool in_turn = !BACK && runs > f.accs;  // (the backward has one run)

  if (threadIdx.x == 0) {
    for (int s = 0; s < f.slots; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (in_turn && warp == 1 && lane < f.accs) {
    mbar_init(acc_full + 8 * lane, 1);
    mbar_init(acc_empty + 8 * lane, 4);
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), f.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{abort_flag, p.dev_status, p.wait_limit};
  if (!BACK && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.ticket = 0;
  // the backward's: what token `lane` of the block brings to d, under the products (read
  // for each in the epilogue, gradients of 32 x 256 x 131072 84 us; so 73)
  const int tokens = min(kFewTokens, p.T - t0);
  int own_y = -1;
  float own_lse = 0.f, own_g = 0.f, own_f = 0.f;
  if (BACK && warp < 4 && lane < tokens) {
    const int t = t0 + lane;
    own_y = target_of(p.targets, p.i64, p.ignore, p.vocab, t);
    const float lse = p.lse[t];
    own_lse = -lse * kLog2e;
    own_g = own_y < 0 ? 0.f : p.gtok ? p.gtok[t] * *p.weight : 1.f;
    own_f = (1.f + p.z2 * lse) * own_g;
    if (own_y == -2 && p.v0 + n0 == 0 && rank == 0 && warp == 0) atomicOr(p.dev_status, kDevBadTarget);
  }

  if (warp == 4) {
    Ring r{0, 0, 0};
#pragma unroll 1
    for (int k = kb0 * BK; k < (kb0 + nkb) * BK; k += BK) {
      if (r.it >= f.slots && !__all_sync(0xffffffffu, wait_bar(empty + 8 * r.s, r.ph ^ 1, wc))) break;
      if (elect_one()) {
        const uint32_t a = base + r.s * stage;
        mbar_arrive_expect_tx(full + 8 * r.s, stage);
        tma_load_2d(a, &maps.b, full + 8 * r.s, k, n0);
        tma_load_2d(a + OPER, &maps.a, full + 8 * r.s, k, t0);
      }
      r.next(f.slots);
    }
    // the copies land before the block may exit
    for (int j = max(0, r.it - f.slots); j < r.it; ++j)
      wait_bar_drain(full + 8 * (j % f.slots), (j / f.slots) & 1, DRAIN_LIMIT);
    __syncwarp();
  } else if (warp == 5) {
    const uint32_t idesc = idesc_bf16_f32(128, f.N, false, false);
    const uint64_t a0 = sw128_desc(base, 16, 1024), b0 = sw128_desc(base + OPER, 16, 1024);
    Ring r{0, 0, 0}, a{0, 0, 0};  // the operands' slots, the accumulators
    bool ok = true;
#pragma unroll 1
    for (int kb = 0, in = 0; kb < nkb; ++kb) {
      if (in == 0 && a.it >= f.accs) {
        ok = __all_sync(0xffffffffu, wait_bar(acc_empty + 8 * a.s, a.ph ^ 1, wc));
        if (!ok) break;
        tc_fence_after();
      }
      ok = __all_sync(0xffffffffu, wait_bar(full + 8 * r.s, r.ph, wc));
      if (!ok) break;
      tc_fence_after();
      const uint64_t ad = a0 + r.s * (stage >> 4), bd = b0 + r.s * (stage >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc_mma_bf16(tmem_base + a.s * f.N, ad + kk * 2, bd + kk * 2, idesc, in || kk);
        tc_commit(empty + 8 * r.s);
      }
      r.next(f.slots);
      if (++in == f.run || kb + 1 == nkb) {
        if (in_turn && elect_one()) tc_commit(acc_full + 8 * a.s);
        a.next(f.accs);
        in = 0;
      }
    }
    if (elect_one()) {
      tc_commit(done);
      wait_bar_drain(done, 0, DRAIN_LIMIT);
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  }
  const uint32_t taddr = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
  float sums[BACK ? 1 : kFewTokens];  // of this thread's row of W and each token
  if (!BACK && in_turn && warp < 4) {
    Ring a{0, 0, 0};
#pragma unroll 1
    while (a.it < runs) {
      if (!__all_sync(0xffffffffu, wait_bar(acc_full + 8 * a.s, a.ph, wc))) break;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < kFewTokens; j += 16) {
        if (j >= f.N) break;
        float x[16];
        tmem_ld16(taddr + a.s * f.N + j, x);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[j + i] = a.it ? sums[j + i] + x[i] : x[i];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + 8 * a.s);
      a.next(f.accs);
    }
  }
  // ------------------------------------------------ epilogue
  __syncthreads();  // every MMA is done; all warps, no wait of their own
  tc_fence_after();
  const bool ok = *abort_flag == 0;
  const int tl = warp * 32 + lane, row = n0 + tl;
  // the logit of the block's token i and this thread's row of W to its gradient
  auto store_d = [&](int i, float z) {
    const long long t = t0 + i;
    const int y = __shfl_sync(0xffffffffu, own_y, i);
    const float g = __shfl_sync(0xffffffffu, own_g, i);
    float d = exp2_f(fmaf(z, kLog2e, __shfl_sync(0xffffffffu, own_lse, i))) * __shfl_sync(0xffffffffu, own_f, i);
    if (y == p.v0 + row) d -= g;
    if (y < 0) d = 0.f;
    if (row < p.V && p.df) {
      p.df[t * p.ldd + row] = d;
    } else if (row < p.V) {
      const __nv_bfloat16 hi = __float2bfloat16_rn(d);
      p.d[t * p.ldd + row] = hi;
      if (p.split) p.d[(p.T + t) * p.ldd + row] = __float2bfloat16_rn(d - __bfloat162float(hi));
    }
  };
  auto turn = [&](int i, float z) { st_shared_f32(base + (i * 132 + tl) * 4, row < p.V ? z : -INFINITY); };
  if (in_turn && ok && warp < 4) {
#pragma unroll
    for (int i = 0; i < kFewTokens; ++i)
      if (i < f.N) turn(i, sums[BACK ? 0 : i]);
  } else if (ok && warp < 4) {
#pragma unroll 1
    for (int j = 0; j < f.N; j += 16) {
      float v[16], x[16];
      tmem_ld16(taddr + j, v);
      tmem_ld_wait();
      for (int k = 1; k < runs; ++k) {
        tmem_ld16(taddr + k * f.N + j, x);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += x[i];
      }
      if constexpr (!BACK || SPLIT) {
#pragma unroll
        for (int i = 0; i < 16; ++i) turn(j + i, v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (j + i >= tokens) break;
          store_d(j + i, v[i]);
        }
      }
    }
  }
  // the parts of a sum lie in the cluster's blocks, which share the tokens out
  if (SPLIT) cluster_sync_all();
  else if (!BACK) __syncthreads();
  auto logit = [&](int t, int r) {
    const uint32_t at = base + (t * 132 + r) * 4;
    if (!SPLIT) return ld_shared_f32(at);
    float z = 0.f;
    for (int c = 0; c < split; ++c) z += ld_cluster_f32(mapa_shared(at, c));
    return z;
  };
  if (BACK) {
    if (SPLIT && ok && warp < 4)
      for (int t = rank; t < tokens; t += split) store_d(t, logit(t, tl));
  } else {
    for (int t = rank + warp * split; ok && t < tokens; t += kFewThreads / 32 * split) {
      float v[4], top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = logit(t, 32 * i + lane);
        top = fmaxf(top, v[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float c = top * kLog2e, r = c == -INFINITY ? 0.f : c;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) s += exp2_f(fmaf(v[i], kLog2e, -r));
#pragma unroll
      for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
      const int at = target_of(p.targets, p.i64, p.ignore, p.vocab, t0 + t) - n0;
      if (lane == 0) p.part[static_cast<long long>(tile) * p.T + t0 + t] = make_float2(c, s);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at == 32 * i + lane) p.target_z[t0 + t] = v[i];
    }
  }
  if (SPLIT) cluster_sync_all();  // (no block leaves before the others have read its sums)
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, f.tmem_cols);
  }
}

// ---------------------------------------------------------------- joining the tiles
// A block joins the pairs of 32 tokens (a lane each, the tiles dealt out to its
// warps; then a warp each), and the block that ends last adds up the blocks' losses in their
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
constexpr int kJoinThreads = 1024, kJoinWarps = kJoinThreads / 32;
__global__ void __launch_bounds__(kJoinThreads) vocab_join_kernel(const JoinParams p) {
  __shared__ float2 sh[kJoinWarps][33];
  __shared__ float2 each[kJoinWarps];
  __shared__ bool last;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (the token that this warp finishes: its target is on its way meanwhile)
  const int own = blockIdx.x * 32 + warp;
  const int y = own < p.T ? target_of(p.targets, p.i64, p.ignore, p.vocab, own) : -1;
  const float z = y >= 0 ? p.target_z[own] : 0.f;
  const int t = blockIdx.x * 32 + lane;
  float c = -INFINITY, s = 0.f;
  if (t < p.T) {
    for (int i = warp; i < p.tiles; i += 4 * kJoinWarps) {
      float2 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        q[u] = i + kJoinWarps * u < p.tiles ? p.part[static_cast<long long>(i + kJoinWarps * u) * p.T + t]
                                            : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int u = 0; u < 4; ++u) join(c, s, q[u].x, q[u].y);
    }
  }
  sh[warp][lane] = make_float2(c, s);
  __syncthreads();
  // warp w: the block's token w
  const float2 q = sh[lane][warp];
  c = q.x, s = q.y;
#pragma unroll
  for (int o = 16; o > 0; o /= 2)
    join(c, s, __shfl_xor_sync(0xffffffffu, c, o), __shfl_xor_sync(0xffffffffu, s, o));
  if (lane == 0) {
    float loss = 0.f, n = 0.f;
    if (own < p.T) {
      const float lse = kLn2 * (c + log2f(s));
      p.lse[own] = lse;
      if (y >= 0) {
        loss = lse - z + p.zc * lse * lse;
        n = 1.f;
      } else if (y == -2) {
        atomicOr(p.dev_status, kDevBadTarget);
      }
      if (p.reduction == MGG_REDUCE_NONE) p.losses[own] = loss;
    }
    each[warp] = make_float2(loss, n);
  }
  __syncthreads();
  auto over_warps = [&](float2 e) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
      e.x += __shfl_xor_sync(0xffffffffu, e.x, o);
      e.y += __shfl_xor_sync(0xffffffffu, e.y, o);
    }
    return e;
  };
  auto finish = [&](float2 e) {
    const float w = p.reduction == MGG_REDUCE_MEAN ? 1.f / fmaxf(e.y, 1.f) : 1.f;
    if (p.reduction != MGG_REDUCE_NONE) *p.total = e.x * w;
    *p.weight = w;
  };
  if (warp == 0) {
    const float2 e = over_warps(each[lane]);
    if (lane == 0) {
      last = false;
      if (gridDim.x == 1) {
        finish(e);
      } else {
        p.blocks[blockIdx.x] = e;
        __threadfence();
        last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x) - 1;
      }
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float2 e = make_float2(0.f, 0.f);
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kJoinThreads) {
    const float2 b = __ldcg(p.blocks + i);
    e.x += b.x, e.y += b.y;
  }
  e = over_warps(e);
  if (lane == 0) each[warp] = e;
  __syncthreads();
  if (warp == 0) {
    e = over_warps(each[lane]);
    if (lane == 0) finish(e);
  }
}

__global__ void vocab_empty_kernel(float* total, float* weight) {
  if (total) *total = 0.f;
  *weight = 1.f;
}

// Blocks of a cluster that share a tile's contraction out: as many as find room, with four
// of its steps or more, of contractions of 1024 on (the loss of 16 x 4096 x 2048 23.1 us
// without, 9.0 on clusters of eight; of 16 x 1024 x 2048 9.8 and 7.4; of 16 x 512 x 4096 7.8
// and, of two, 8.4).
int few_split(int T, int K, int V) {
  const long long blocks = static_cast<long long>(cdiv(T, kFewTokens)) * cdiv(V, 128);
  int split = 1;
  while (split < 8 && 2 * split * blocks <= 2 * num_sms() && cdiv(K, BK) >= std::max(16, 8 * split)) split *= 2;
  return split;
}
// More tokens go by groups of 32 where that leaves clusters of four: 256 x 256 tiles would
// leave most SMs idle (loss, gradients of 64 x 4096 x 2048 25 and 43 us on them, 11 and 28
// so; of 128 x 2048 x 2048 17 and 32, 13 and 27; of 128 x 1024 x 4096, clusters of two, 13
// and 27, 14 and 30).
bool by_few(int T, int K, int V) { return T <= kFewTokens || few_split(T, K, V) >= 4; }
// Rows of W that one pair (c, s) of the forward stands for.
int tile_columns(int T, int K, int V) { return by_few(T, K, V) ? 128 : 256; }

template <bool BACK, bool SPLIT>
cudaError_t launch_few_as(const VocabMaps& maps, const VocabParams& p, const FewParams& f, cudaStream_t st) {
  static bool done[64] = {};
  const cudaError_t e = allow_smem(vocab_few_kernel<BACK, SPLIT>, 116 * 1024, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(cdiv(p.V, 128) * f.split, cdiv(p.T, kFewTokens));
  const size_t smem = few_smem(f.N, f.slots);
  if (SPLIT)
    return launch_pdl_clusters(vocab_few_kernel<BACK, SPLIT>, grid, dim3(kFewThreads), smem, f.split, st, maps, p, f);
  return launch_pdl(vocab_few_kernel<BACK, SPLIT>, grid, dim3(kFewThreads), smem, st, maps, p, f);
}
template <bool BACK>
cudaError_t launch_few(const DenseOperand& x, const DenseOperand& W, const VocabParams& p, cudaStream_t st) {
  FewParams f;
  f.N = (std::min(p.T, kFewTokens) + 15) / 16 * 16;
  f.split = few_split(p.T, p.K, p.V);
  const int nkb = cdiv(cdiv(p.K, BK), f.split);
  // half of an SM's shared memory and tensor memory
  f.slots = std::min({kFewSlots, (112 * 1024 - 1024 - kFewMeta) / (OPER + f.N * 128), nkb});
  f.run = BACK ? nkb : p.run;
  f.accs = std::min(256 / f.N, cdiv(nkb, f.run));
  f.tmem_cols = 32;
  while (f.tmem_cols < f.accs * f.N) f.tmem_cols *= 2;
  VocabMaps maps;
  if (!tmap_operand(&maps.a, x, false, f.N) || !tmap_operand(&maps.b, W, false, 128)) return cudaErrorInvalidValue;
  return f.split > 1 ? launch_few_as<BACK, true>(maps, p, f, st) : launch_few_as<BACK, false>(maps, p, f, st);
}

template <bool BACK>
cudaError_t launch_tiles(const DenseOperand& x, const DenseOperand& W, const VocabParams& p,
                         cudaStream_t st) {
  if (by_few(p.T, p.K, p.V)) return launch_few<BACK>(x, W, p, st);
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

// Tokens up to which d, in bfloat16, is kept in two parts.
constexpr int kSplitTokens = 128;

// Rows whose pitch is no multiple of 64 bytes cost: an operand's 128-byte rows then
// lie across three or more 64-byte pieces of the L2, whose way to the SMs is what the
// pair kernel is closest to (loss of 8192 x 2040 x 32768 758 us, with x copied to rows
// on 128-byte boundaries 594; gradients 2117, with both copied 1790).  x is copied
// where there are enough tokens to gain from it, a piece of W where its copy (134 MB
// take 40 us) is a few percent of the products.
constexpr int kCopyTokens = 256, kCopyWTokens = 2048;
bool off_lines(const void* p, long long ld) { return reinterpret_cast<uintptr_t>(p) % 64 || ld % 32; }
int line_ld(int K) { return (K + 63) / 64 * 64; }

// ([x; x], copied twice, is the other operand of d's two parts in dW.)
__global__ void __launch_bounds__(256) vocab_copy_kernel(const uint4* x, long long ld, int rows, int K8,
                                                         int out_ld, int copies, const void* targets, bool i64,
                                                         long long ignore, int vocab, uint4* out) {
  pdl_trigger();
  pdl_wait();
  copy_pieces(x, ld, rows, K8, out, out_ld, copies, targets, i64, ignore, vocab, blockIdx.x * 256 + threadIdx.x,
              gridDim.x * 256);
}
// o's rows to `to`, on 128-byte boundaries; with `a` x's, those that do not count as zeros
cudaError_t copy_rows(DenseOperand* o, void* to, int copies, const VocabBackward* a, cudaStream_t st) {
  const int ld = line_ld(o->cols);
  const long long n = static_cast<long long>(o->rows) * (o->cols / 8);
  const unsigned blocks = static_cast<unsigned>(std::min<long long>((n + 255) / 256, 8 * num_sms()));
  const cudaError_t e = launch_pdl(vocab_copy_kernel, dim3(blocks), dim3(256), 0, st,
                                   static_cast<const uint4*>(o->ptr), o->ld / 8, o->rows, o->cols / 8, ld / 8,
                                   copies, a ? a->targets : nullptr, a && a->i64, a ? a->ignore : 0LL,
                                   a ? a->V : 0, static_cast<uint4*>(to));
  *o = DenseOperand{to, o->rows, o->cols, ld};
  return e;
}

// dx = scale (the sum of its parts, [parts][T K]).  GROUPS groups of threads share the
// parts of a block's values: eight for few values of many parts, which otherwise are as
// many latencies (gradients of 32 x 256 x 131072 95 us with one, 84 with eight; of 512 x
// 4096 x 2048 44 with one, 53 with eight), 32 from 65 parts on.
template <int GROUPS>
constexpr int kJoinDxThreads = GROUPS == 1 ? 256 : GROUPS * 32;
template <int GROUPS>
__global__ void __launch_bounds__(kJoinDxThreads<GROUPS>) vocab_join_dx_kernel(const float4* sum, int parts, long long n4,
                                                            const float* scale0, const float* scale1, uint2* dx) {
  constexpr int kWide = kJoinDxThreads<GROUPS> / GROUPS;
  __shared__ float4 sh[GROUPS > 1 ? GROUPS : 1][GROUPS > 1 ? kWide : 1];
  pdl_trigger();
  pdl_wait();
  const float g = scale0 ? *scale0 * *scale1 : 1.f;
  const int group = threadIdx.x / kWide, lane = threadIdx.x % kWide;
  // (the same number of rounds in every thread of the block)
  for (long long at = static_cast<long long>(blockIdx.x) * kWide; at < n4; at += static_cast<long long>(gridDim.x) * kWide) {
    const long long i = at + lane;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = group; i < n4 && k < parts; k += 8 * GROUPS) {
      float4 b[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        b[u] = k + u * GROUPS < parts ? sum[(k + u * GROUPS) * n4 + i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) a.x += b[u].x, a.y += b[u].y, a.z += b[u].z, a.w += b[u].w;
    }
    if constexpr (GROUPS > 1) {
      sh[group][lane] = a;
      __syncthreads();
      for (int k = 1; group == 0 && k < GROUPS; ++k) {
        const float4 b = sh[k][lane];
        a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
      }
      __syncthreads();
    }
    if (group == 0 && i < n4) dx[i] = make_uint2(cvt_bf16x2(a.x * g, a.y * g), cvt_bf16x2(a.z * g, a.w * g));
  }
}
cudaError_t join_dx(const float* sum, int parts, int T, int K, const float* scale0, const float* scale1, void* dx,
                    cudaStream_t st) {
  const long long n4 = static_cast<long long>(T) * K / 4;
  auto launch = [&](auto kernel, long long blocks, int threads) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, st,
                      reinterpret_cast<const float4*>(sum), parts, n4, scale0, scale1, static_cast<uint2*>(dx));
  };
  if (n4 > 65536 || parts < 8)
    return launch(vocab_join_dx_kernel<1>, std::min<long long>((n4 + 255) / 256, 16 * num_sms()), kJoinDxThreads<1>);
  return parts <= 64 ? launch(vocab_join_dx_kernel<8>, (n4 + 31) / 32, kJoinDxThreads<8>)
                     : launch(vocab_join_dx_kernel<32>, (n4 + 31) / 32, kJoinDxThreads<32>);
}

// ---------------------------------------------------------------- both gradients of very few tokens
// Up to 4 tokens dx and dW are sums of a few products an element, bound by W read and
// dW written once: no tensor cores, d in f32.  A thread holds eight columns of every
// token's x and of its sum of dx, and walks down rows of W: each is read, added to dx
// with d's column, and leaves as dW's.  Its rows wait in a ring of its own in shared
// memory (only the thread that copied them reads them: no barrier), 16 under way.  The
// blocks take chunks of rows from W's end, which d's kernel has read last and L2 still
// holds, and write dW past it.  The blocks' sums of dx meet afterwards.  d, dx and dW of
// 1, 2 and 4 x 2048 x 32768 take 70, 71 and 74 us (on pair tiles, of one contraction
// block each, 97 to 99; with four loads under way a thread 112 to 121), of 2 x 2048 x
// 8192 23 (39), of 2 x 512 x 4096 12.3 (18.6).  From 8 tokens their products bound it: 8 x
// 2048 x 32768 112 us, on pair tiles 99.
constexpr int kThinTokens = 4, kThinRows = 16, kThinStages = 16;  // rows of a chunk; of the ring
struct ThinParams {
  const float* d;            // [T][ldd]
  int ldd;
  const __nv_bfloat16 *x, *W;
  long long ldx;
  int T, K, V;
  const void* targets;       // as in VocabParams
  bool i64;
  long long ignore;
  float* sums;               // [gridDim.y][T][K], or null: no dx
  __nv_bfloat16* dW;         // or null
  const float *scale0, *scale1;  // of dW, or null
};
__device__ __forceinline__ void pairs_of(const uint4& q, F2 (&v)[4]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
template <int TT>
__global__ void __launch_bounds__(128) vocab_thin_kernel(const ThinParams p) {
  __shared__ uint4 ring[kThinStages][128];
  __shared__ float sd[2][kThinRows][TT];
  pdl_trigger();
  pdl_wait();
  const int k0 = (blockIdx.x * blockDim.x + threadIdx.x) * 8;
  const bool in = k0 < p.K;
  const int chunks = (p.V + kThinRows - 1) / kThinRows;
  const int mine = (chunks - static_cast<int>(blockIdx.y) + gridDim.y - 1) / gridDim.y;  // chunks, >= 1
  // the i-th of them, from W's end
  auto first_row = [&](int i) { return (chunks - 1 - (static_cast<int>(blockIdx.y) + i * static_cast<int>(gridDim.y))) * kThinRows; };
  constexpr int S = kThinStages, R = kThinRows, U = 4;
  static_assert(S == R, "the ring holds a chunk");
  const float g = p.scale0 ? *p.scale0 * *p.scale1 : 1.f;
  // rows u .. u+3 of a chunk into the ring (rows behind V stay what they were, unread)
  auto fetch = [&](int i, int u) {
    if (i < mine && in) {
      const int r = first_row(i) + u;
#pragma unroll
      for (int a = 0; a < U; ++a)
        if (r + a < p.V)
          cp_async_16_full(smem_u32(&ring[u + a][threadIdx.x]), p.W + static_cast<long long>(r + a) * p.K + k0);
    }
    cp_async_commit();
  };
  // d of a chunk: up to PER values a thread, through registers to the buffer read next
  constexpr int PER = (R * TT + 31) / 32;
  float dn[PER];
  auto load_d = [&](int i) {
#pragma unroll
    for (int a = 0; a < PER; ++a) {
      const int e = threadIdx.x + a * blockDim.x, t = e / R, r = e % R;
      dn[a] = 0.f;
      if (i < mine && e < R * TT && t < p.T && first_row(i) + r < p.V)
        dn[a] = p.d[static_cast<long long>(t) * p.ldd + first_row(i) + r];
    }
  };
  auto store_d = [&](int b) {
#pragma unroll
    for (int a = 0; a < PER; ++a) {
      const int e = threadIdx.x + a * blockDim.x;
      if (e < R * TT) sd[b][e % R][e / R] = dn[a];
    }
  };
#pragma unroll
  for (int u = 0; u < R; u += U) fetch(0, u);
  load_d(0);
  F2 x[TT][4], acc[TT][4];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    uint4 q = make_uint4(0, 0, 0, 0);
    // (a token that does not count: zeros, whatever its row holds)
    if (in && t < p.T && target_of(p.targets, p.i64, p.ignore, p.V, t) >= 0)
      q = *reinterpret_cast<const uint4*>(p.x + t * p.ldx + k0);
    pairs_of(q, x[t]);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = both(0.f);
  }
  store_d(0);
  __syncthreads();
  for (int c = 0; c < mine; ++c) {
    load_d(c + 1);
    const int rb = first_row(c);
#pragma unroll 1
    for (int u = 0; u < R; u += U) {
      cp_async_wait<R / U - 1>();
      uint4 w[U];
#pragma unroll
      for (int a = 0; a < U; ++a) w[a] = ring[u + a][threadIdx.x];
      fetch(c + 1, u);
#pragma unroll
      for (int a = 0; a < U; ++a) {
        if (rb + u + a >= p.V || !in) break;
        F2 wv[4], out[4];
        pairs_of(w[a], wv);
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = both(0.f);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const F2 d = both(sd[c & 1][u + a][t]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[t][i] = fma2(d, wv[i], acc[t][i]);
            out[i] = fma2(d, x[t][i], out[i]);
          }
        }
        if (p.dW) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float e, f;
            unpack2(out[i], e, f);
            o[i] = cvt_bf16x2(e * g, f * g);
          }
          __stcs(reinterpret_cast<uint4*>(p.dW + static_cast<long long>(rb + u + a) * p.K + k0),
                 make_uint4(o[0], o[1], o[2], o[3]));
        }
      }
    }
    // (the other buffer: its readers are past the barrier before this chunk)
    store_d((c + 1) & 1);
    __syncthreads();
  }
  cp_async_wait<0>();
  if (!in || !p.sums) return;
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    if (t >= p.T) break;
    float* to = p.sums + (static_cast<long long>(blockIdx.y) * p.T + t) * p.K + k0;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(acc[t][i], v[2 * i], v[2 * i + 1]);
    reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
// Threads of a block, blocks along the columns and down the rows: as many as an SM's
// registers hold (of 128 threads six for up to 2 tokens, four for 4: of 4 x 2048 x 32768
// on two 108 us, four 78, six, of which not all fit, 83), with two chunks or more where
// that leaves 64 ranges (2 x 2048 x 8192 29 us, with one 31; 2 x 64 x 512 8.4 and 7.1).
struct ThinPlan {
  int threads, slabs, ranges;
};
ThinPlan plan_thin(int T, int K, int V) {
  ThinPlan l;
  l.threads = std::min(128, cdiv(K / 8, 32) * 32);
  l.slabs = cdiv(K, 8 * l.threads);
  const int blocks = std::max(1, (T <= 2 ? 6 : 4) * num_sms());
  const int chunks = cdiv(V, kThinRows);
  l.ranges = std::max(1, std::min(blocks / l.slabs, std::min(chunks, std::max(64, chunks / 2))));
  return l;
}
template <int TT>
cudaError_t launch_thin_t(const ThinPlan& l, const ThinParams& p, cudaStream_t st) {
  return launch_pdl(vocab_thin_kernel<TT>, dim3(l.slabs, l.ranges), dim3(l.threads), 0, st, p);
}
cudaError_t launch_thin(const ThinPlan& l, const ThinParams& p, cudaStream_t st) {
  return p.T <= 2 ? launch_thin_t<2>(l, p, st) : launch_thin_t<4>(l, p, st);
}

// Columns of a piece of the backward: as many as give d 256 MB (4096 x 2048 x 32768 in
// pieces of 64 MB 1031 us, 128 1013, 256 987), at least 2048; MGG_VOCAB_PIECE sets it.
int piece_columns(int T, int V) {
  const long long most = 256LL << 20;
  const int rows = T <= kSplitTokens ? 2 * T : T;
  long long cols = std::max<long long>(2048, most / (2LL * rows) / 256 * 256);
  if (const char* s = getenv("MGG_VOCAB_PIECE"))
    if (const long long n = atoll(s); n > 0) cols = (std::min(n, 1LL << 30) + 63) / 64 * 64;
  return static_cast<int>(std::min<long long>(cols, (V + 7) / 8 * 8));
}
// What the backward keeps: d; f32 sums of dx (over pieces, of its slices and parts);
// a copy of x or [x; x]; of a piece of W.
struct BackLayout {
  int cols;
  bool split, copy_w;
  int slices;              // of dx's contraction in a piece
  size_t sum, x, w, total; // offsets of the second and on
};
BackLayout back_layout(int T, int K, int V) {
  BackLayout l;
  l.cols = piece_columns(T, V);
  l.split = T <= kSplitTokens;
  const int rows = l.split ? 2 * T : T;
  // dx has few tiles and a long contraction where there are few tokens: cut so that
  // no tile takes longer than half of what a pair has to do (1111 x 1160 over 50257:
  // 25 tiles, 240 us on single-CTA tiles)
  const long long blocks = cdiv(l.cols, BK), tk = cdiv(K, 256);
  const long long work = cdiv(rows, 256) * tk * (blocks + 4) + cdiv(l.cols, 256) * tk * std::max(cdiv(rows, BK) + 4, 9);
  const long long most = std::max<long long>(16, work / std::max(1, num_sms() / 2) / 2);
  l.slices = static_cast<int>(std::min<long long>(32, (blocks + most - 1) / most));
  const size_t sums = static_cast<size_t>(rows) * l.slices;
  l.sum = round256(static_cast<size_t>(rows) * l.cols * 2);
  l.copy_w = T >= kCopyWTokens && K % 32;
  l.x = l.sum + (l.split || l.slices > 1 || l.cols < V ? round256(sums * K * 4) : 0);
  l.w = l.x + round256(static_cast<size_t>(rows) * line_ld(K) * 2);
  l.total = l.w + (l.copy_w ? round256(static_cast<size_t>(l.cols) * line_ld(K) * 2) : 0);
  return l;
}

}  // namespace

// forward: the tiles' pairs, the targets' logits, the joining blocks' sums, their ticket, x
size_t vocab_fwd_ws_bytes(int T, int K, int V) {
  return round256(static_cast<size_t>(cdiv(V, tile_columns(T, K, V))) * T * 8) + round256(static_cast<size_t>(T) * 4) +
         round256(static_cast<size_t>(cdiv(T, 32)) * 8) + 256 +
         (T >= kCopyTokens ? round256(static_cast<size_t>(T) * line_ld(K) * 2) : 0);
}
size_t vocab_bwd_ws_bytes(int T, int K, int V) {
  if (T <= kThinTokens)
    return round256(static_cast<size_t>(T) * ((V + 7) / 8 * 8) * 4) +
           round256(static_cast<size_t>(plan_thin(T, K, V).ranges) * T * K * 4);
  return back_layout(T, K, V).total;
}

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
  const int tn = cdiv(a.V, tile_columns(a.T, a.K, a.V));
  VocabParams p{};
  p.T = a.T, p.V = a.V, p.K = a.K, p.vocab = a.V;
  p.targets = a.targets, p.i64 = a.i64, p.ignore = a.ignore;
  p.part = reinterpret_cast<float2*>(take(static_cast<size_t>(tn) * a.T * 8));
  p.target_z = reinterpret_cast<float*>(take(static_cast<size_t>(a.T) * 4));
  JoinParams j{};
  j.blocks = reinterpret_cast<float2*>(take(static_cast<size_t>(cdiv(a.T, 32)) * 8));
  p.ticket = reinterpret_cast<int*>(take(4));
  p.run = a.T <= kFewTokens ? kRunFewest : a.T <= 256 ? kRunFew : kRunBlocks;
  p.dev_status = a.dev_status, p.wait_limit = a.wait_limit;
  DenseOperand x{a.x, a.T, a.K, a.ldx};
  cudaError_t e = cudaSuccess;
  if (a.T >= kCopyTokens && off_lines(a.x, a.ldx)) e = copy_rows(&x, at, 1, nullptr, st);
  if (e == cudaSuccess) e = launch_tiles<false>(x, DenseOperand{a.W, a.V, a.K, a.K}, p, st);
  if (e != cudaSuccess) return e;
  j.part = p.part, j.tiles = tn, j.T = a.T, j.vocab = a.V, j.target_z = p.target_z;
  j.targets = a.targets, j.i64 = a.i64, j.ignore = a.ignore, j.zc = a.z_loss, j.reduction = a.reduction;
  j.lse = a.lse, j.losses = a.loss, j.total = a.loss, j.weight = a.weight;
  j.ticket = p.ticket, j.dev_status = a.dev_status;
  return launch_pdl(vocab_join_kernel, dim3(cdiv(a.T, 32)), dim3(kJoinThreads), 0, st, j);
}

// Up to 4 tokens: the whole vocabulary at once (d is a few rows), three launches.
static cudaError_t backward_thin(const VocabBackward& a, void* ws, cudaStream_t st) {
  VocabParams p{};
  p.T = a.T, p.V = a.V, p.K = a.K, p.vocab = a.V;
  p.targets = a.targets, p.i64 = a.i64, p.ignore = a.ignore;
  p.lse = a.lse, p.z2 = 2.f * a.z_loss, p.gtok = a.per_token ? a.dloss : nullptr, p.weight = a.weight;
  p.df = static_cast<float*>(ws), p.ldd = (a.V + 7) / 8 * 8;
  p.dev_status = a.dev_status, p.wait_limit = a.wait_limit;
  cudaError_t e = launch_tiles<true>(DenseOperand{a.x, a.T, a.K, a.ldx}, DenseOperand{a.W, a.V, a.K, a.K}, p, st);
  if (e != cudaSuccess) return e;
  const ThinPlan l = plan_thin(a.T, a.K, a.V);
  ThinParams t{};
  t.d = p.df, t.ldd = p.ldd, t.x = static_cast<const __nv_bfloat16*>(a.x);
  t.W = static_cast<const __nv_bfloat16*>(a.W), t.ldx = a.ldx, t.T = a.T, t.K = a.K, t.V = a.V;
  t.targets = a.targets, t.i64 = a.i64, t.ignore = a.ignore;
  float* sums = reinterpret_cast<float*>(static_cast<char*>(ws) + round256(static_cast<size_t>(a.T) * p.ldd * 4));
  t.sums = a.dx ? sums : nullptr, t.dW = static_cast<__nv_bfloat16*>(a.dW);
  t.scale0 = a.per_token ? nullptr : a.dloss, t.scale1 = a.weight;
  e = launch_thin(l, t, st);
  return e == cudaSuccess && a.dx ? join_dx(sums, l.ranges, a.T, a.K, t.scale0, t.scale1, a.dx, st) : e;
}

cudaError_t launch_vocab_backward(const VocabBackward& a, void* ws, cudaStream_t st) {
  if (a.T <= kThinTokens) return backward_thin(a, ws, st);
  const BackLayout l = back_layout(a.T, a.K, a.V);
  char* const base = static_cast<char*>(ws);
  __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(base);
  float* sum = reinterpret_cast<float*>(base + l.sum);
  const int rows = l.split ? 2 * a.T : a.T;
  DenseOperand x{a.x, a.T, a.K, a.ldx};
  const float* const scale = a.per_token ? nullptr : a.dloss;
  cudaError_t e = cudaSuccess;
  // x is copied for its lines, for d's two parts, or for dW alone, which the pair kernel
  // does on its way
  const bool own_copy = l.split ? a.dW != nullptr : a.T >= kCopyTokens && off_lines(a.x, a.ldx);
  const bool on_way = a.dW && !own_copy && !by_few(a.T, a.K, std::min(l.cols, a.V));
  if (own_copy || (a.dW && !on_way)) e = copy_rows(&x, base + l.x, l.split ? 2 : 1, &a, st);
  DenseOperand xd = x;  // beside d's rows
  xd.rows = rows;
  if (on_way) xd.ptr = base + l.x, xd.ld = line_ld(a.K);
  for (int v0 = 0; e == cudaSuccess && v0 < a.V; v0 += l.cols) {
    const int n = std::min(l.cols, a.V - v0);
    const char* W = static_cast<const char*>(a.W) + static_cast<size_t>(v0) * a.K * 2;
    VocabParams p{};
    p.T = a.T, p.V = n, p.K = a.K, p.v0 = v0, p.vocab = a.V;
    p.targets = a.targets, p.i64 = a.i64, p.ignore = a.ignore;
    p.lse = a.lse, p.z2 = 2.f * a.z_loss, p.gtok = a.per_token ? a.dloss : nullptr, p.weight = a.weight;
    p.d = d, p.ldd = l.cols, p.split = l.split;
    if (on_way && v0 == 0) {
      p.x = static_cast<const uint4*>(a.x), p.ldx8 = a.ldx / 8;
      p.x_out = reinterpret_cast<uint4*>(base + l.x), p.out_ld8 = line_ld(a.K) / 8;
    }
    p.dev_status = a.dev_status, p.wait_limit = a.wait_limit;
    DenseOperand Wp{W, n, a.K, a.K};
    const DenseOperand dp{d, rows, n, l.cols};
    if (l.copy_w) e = copy_rows(&Wp, base + l.w, 1, nullptr, st);
    if (e == cudaSuccess) e = launch_tiles<true>(x, Wp, p, st);
    if (e != cudaSuccess) return e;
    const bool parts = l.split || l.slices > 1;
    const bool first = v0 == 0, direct = v0 + n == a.V && !parts;  // dx in place
    // every product is multiplied by the loss's gradient as it leaves
    DenseParams q{};
    q.dev_status = a.dev_status, q.wait_limit = a.wait_limit;
    DenseProduct dx{}, dW{};
    dx.M = rows, dx.N = a.K, dx.Kc = n, dx.b_mn = true;
    dx.out = !a.dx ? nullptr : direct ? a.dx : sum;
    dx.out_f32 = !direct, dx.epilogue = !first;
    dW.M = n, dW.N = a.K, dW.Kc = rows, dW.a_mn = dW.b_mn = true;
    // (on pairs in any case, which know a factor of the product; of 32 rows dW takes 59
    // us on single-CTA tiles, 34 on pairs)
    const PairOptions opt{true, {std::min(l.slices, cdiv(n, BK)), 1}, scale, a.weight};  // (a last piece may be narrow)
    dW.out = a.dW ? static_cast<char*>(a.dW) + static_cast<size_t>(v0) * a.K * 2 : nullptr;
    if (!first) {
      q.residual = sum;
      q.res_f32 = q.res_vec = true;
      q.ldr = a.K;
    }
    q.act = scale ? kActScale : kActNone;
    const DenseOperand oa[2] = {dp, dp}, ob[2] = {Wp, xd};
    const DenseProduct pr[2] = {dx, dW};
    e = launch_dense_products(q, opt, pr, oa, ob, st);
  }
  // (its parts have the factor already)
  if (e == cudaSuccess && (l.split || l.slices > 1) && a.dx)
    e = join_dx(sum, (l.split ? 2 : 1) * l.slices, a.T, a.K, nullptr, nullptr, a.dx, st);
  return e;
}

}  // namespace mgg
