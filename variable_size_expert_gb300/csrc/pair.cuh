// The parts that the kernels of dense products on CTA pairs share (linear.cu,
// vocab.cu): the ring of operand blocks, its producer and MMA loops, the tile
// order, and the staged stores of an epilogue; on the host the operands' tensor
// maps.
#pragma once

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace mgg {
namespace {

constexpr int BK = kBK;                 // contraction step: one 128-byte row of bf16
constexpr int kHalf = 128;              // rows of A, and of B, per CTA and stage of a pair
constexpr int STAGES = 5;
constexpr int OPER = kHalf * BK * 2;    // 16 KB
constexpr int CHUNK = 64 * BK * 2;      // 8 KB: 64 wide MN-major block of one stage
constexpr int EPI_WARP = 32 * 128;      // staging of an epilogue warp: 32 rows x 128 bytes
// pairs: warps 0-3 and 6-17 epilogue, 4 MMA, 5 TMA.  Sixteen epilogue warps
// hide one another's latencies (tensor memory, exponentials, store fences):
// with eight, bias + GELU + kept z took 9.1 us a tile, half of it stalled.
constexpr int kEpiWarps = 16;
constexpr int kPairThreads = 32 * (kEpiWarps + 2);
constexpr int kMeta = 512;
constexpr size_t kPairSmem = 1024 + static_cast<size_t>(STAGES) * 2 * OPER + kEpiWarps * EPI_WARP + kMeta;
static_assert(kPairSmem <= 232448, "shared memory per block");
constexpr long long DRAIN_LIMIT = 200000000LL;

// One instruction each, within 2 ulp, denormals flushed.
__device__ __forceinline__ float exp2_f(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_f(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// ---------------------------------------------------------------- staged stores
// A warp's block of 32 rows x 128 bytes (64 bf16 or 32 f32 columns) in shared
// memory, 16-byte columns XOR-ed by row: written a row per lane, read four rows
// x 128 bytes per store instruction, without bank conflicts both ways.
__device__ __forceinline__ void stage_f32(uint32_t stg, int lane, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    st_shared_v4(stg + sw128_offset(lane, c), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ void stage_bf16(uint32_t stg, int lane, int half, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    st_shared_v4(stg + sw128_offset(lane, 4 * half + c),
                 __uint_as_float(cvt_bf16x2(v[8 * c], v[8 * c + 1])),
                 __uint_as_float(cvt_bf16x2(v[8 * c + 2], v[8 * c + 3])),
                 __uint_as_float(cvt_bf16x2(v[8 * c + 4], v[8 * c + 5])),
                 __uint_as_float(cvt_bf16x2(v[8 * c + 6], v[8 * c + 7])));
}
// The staged block to columns c0 .. cend - 1 of rows row0.. (of M) of base [M, N].
// vec: rows start on 16-byte boundaries.
__device__ __forceinline__ void stage_flush(uint32_t stg, int lane, bool vec, void* base, bool f32,
                                            int row0, int M, int N, int c0, int cend) {
  __syncwarp();
  const int per = f32 ? 32 : 64, size = f32 ? 4 : 2;
  if (vec) {
    const int kq = lane & 7, rq = lane >> 3;  // 16-byte column, first row
    const int c = c0 + kq * (per / 8);
    uint8_t* at = static_cast<uint8_t*>(base) + (static_cast<long long>(row0 + rq) * N + c) * size;
    const long long step = 4LL * N * size;
    float4 q[8];  // (read together: a store holds the next read back)
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = ld_shared_v4(stg + sw128_offset(rq + 4 * j, kq));
#pragma unroll
    for (int j = 0; j < 8; ++j, at += step)
      if (row0 + rq + 4 * j < M && c < cend) *reinterpret_cast<float4*>(at) = q[j];
  } else {
    // a row at a time, four bytes a lane (bf16: two elements, stored together
    // where the rows start on 4-byte boundaries)
    const bool even = !(N & 1) && (reinterpret_cast<uintptr_t>(base) & 3) == 0;
    const int c = c0 + (f32 ? lane : 2 * lane);
    if (c < cend) {
#pragma unroll 1
      for (int r0 = 0; r0 < 32 && row0 + r0 < M; r0 += 8) {
        uint32_t u[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          u[r] = static_cast<uint32_t>(
              ld_shared_s32(stg + sw128_offset(r0 + r, lane >> 2) + (lane & 3) * 4));
        const long long o = static_cast<long long>(row0 + r0) * N + c;
        const int rows = std::min(8, M - row0 - r0);
        if (f32) {
          uint32_t* at = static_cast<uint32_t*>(base) + o;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < rows) at[static_cast<long long>(r) * N] = u[r];
        } else {
          unsigned short* at = static_cast<unsigned short*>(base) + o;
          const bool two = c + 1 < cend;
#pragma unroll
          for (int r = 0; r < 8; ++r, at += N) {
            if (r >= rows) continue;
            if (even && two) {
              *reinterpret_cast<uint32_t*>(at) = u[r];
            } else {
              at[0] = static_cast<unsigned short>(u[r]);
              if (two) at[1] = static_cast<unsigned short>(u[r] >> 16);
            }
          }
        }
      }
    }
  }
  __syncwarp();  // the staging area is free again
}

// ---------------------------------------------------------------- pipeline of a pair
struct PSmem {
  uint32_t sA, sB, sEpi, full, empty, acc_full, acc_empty, drain, pdone, res_full, issued;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
};
__device__ __forceinline__ PSmem carve_pair(uint8_t* raw) {
  PSmem m;
  const uint32_t raw_addr = smem_u32(raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* g = raw + (base - raw_addr);
  m.sA = base;
  m.sB = m.sA + STAGES * OPER;
  m.sEpi = m.sB + STAGES * OPER;
  m.full = m.sEpi + kEpiWarps * EPI_WARP;
  m.empty = m.full + 8 * STAGES;
  m.acc_full = m.empty + 8 * STAGES;
  m.acc_empty = m.acc_full + 16;
  m.drain = m.acc_empty + 16;
  m.pdone = m.drain + 8;
  m.res_full = m.pdone + 8;  // one per epilogue warp
  m.issued = m.res_full + 8 * kEpiWarps;
  m.tmem_slot = reinterpret_cast<uint32_t*>(g + (m.issued + 8 - base));
  m.abort_flag = reinterpret_cast<volatile int*>(m.tmem_slot + 1);
  return m;
}

// Tiles are walked in bands of kBand row blocks, down the band first: the
// tiles in flight at one time then cover about kBand x 9 blocks, the squarest
// set of operand rows for the L2 to hold.
constexpr int kBand = 8;
// First row and column of the local-th 256 x 256 tile of an M x N output.
__device__ __forceinline__ void band_tile(int local, int M, int N, int& m0, int& n0) {
  const int tm = cdiv(M, 256), tn = cdiv(N, 256);
  const int band = local / (kBand * tn);
  const int r = local - band * kBand * tn;
  const int rows = min(kBand, tm - band * kBand);
  n0 = (r / rows) * 256;
  m0 = (band * kBand + r % rows) * 256;
}

// The barriers of a CTA (one thread).
__device__ __forceinline__ void init_pair(const PSmem& m) {
  for (int s = 0; s < STAGES; ++s) {
    mbar_init(m.full + 8 * s, 2);  // both TMA threads announce their own bytes
    mbar_init(m.empty + 8 * s, 1);
  }
  for (int a = 0; a < 2; ++a) {
    mbar_init(m.acc_full + 8 * a, 1);
    mbar_init(m.acc_empty + 8 * a, 2 * kEpiWarps);  // the epilogue warps of both CTAs
  }
  mbar_init(m.drain, 1);
  mbar_init(m.pdone, 1);
  for (int w = 0; w < kEpiWarps; ++w) mbar_init(m.res_full + 8 * w, 1);
  *m.abort_flag = 0;
  fence_mbar_init();
}

// One operand's rows of a stage: 128 rows from r0, contraction from k.
template <bool MN>
__device__ __forceinline__ void load_oper(uint32_t dst, const CUtensorMap* map, uint32_t bar, int r0,
                                          int k) {
  if constexpr (MN) {
    tma_load_2d_cg2(dst, map, bar, r0, k);
    tma_load_2d_cg2(dst + CHUNK, map, bar, r0 + 64, k);
  } else {
    tma_load_2d_cg2(dst, map, bar, k, r0);
  }
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// The producer's and the MMA warp's loops.  Blocks of the contraction pass
// through a ring of slots: full[s] tells that a block has landed, empty[s] that
// its MMAs have read it (slots released by twos, the ring of five runs short:
// gradients of 8192 x 2048 x 8192 1650 instead of 1800 TFLOP/s).  Both loops run
// with the whole warp converged, one elected lane issuing: inside a divergent
// branch every operand of an MMA or a copy costs extra moves into uniform
// registers (15% of a loop of small tiles).
struct Ring {
  int it, s;
  uint32_t ph;
  __device__ __forceinline__ void next(int stages) {
    ++it;
    if (++s == stages) s = 0, ph ^= 1;
  }
};
template <bool A_MN, bool B_MN>
__device__ __forceinline__ bool produce(const PSmem& m, const CUtensorMap* ma,
                                        const CUtensorMap* mb, uint32_t full_l, bool leader, int ar,
                                        int br, int kb0, int nkb, Ring& r, const WaitCtl& wc) {
#pragma unroll 1
  for (int k = kb0 * BK; k < (kb0 + nkb) * BK; k += BK) {
    // (the first round of the slots was never used)
    if (r.it >= STAGES && !__all_sync(0xffffffffu, wait_bar(m.empty + 8 * r.s, r.ph ^ 1, wc)))
      return false;
    if (elect_one()) {
      const uint32_t fb = full_l + 8 * r.s;
      // the leader announces its bytes first; the peer issues its copies first
      // (the phase cannot complete before its arrival)
      if (leader) mbar_arrive_expect_tx(m.full + 8 * r.s, 2 * OPER);
      load_oper<A_MN>(m.sA + r.s * OPER, ma, fb, ar, k);
      load_oper<B_MN>(m.sB + r.s * OPER, mb, fb, br, k);
      if (!leader) mbar_arrive_expect_tx_cluster(fb, 2 * OPER);
    }
    r.next(STAGES);
  }
  return true;
}
template <bool A_MN, bool B_MN>
__device__ __forceinline__ bool multiply(const PSmem& m, uint32_t dt, int nkb, Ring& r,
                                         const WaitCtl& wc) {
  constexpr uint32_t kIdesc = idesc_bf16_f32(256, 256, A_MN, B_MN);
  // per 16 of the contraction: 32 bytes along a K-major row, 16 rows of 128
  // bytes down an MN-major block (descriptors count 16-byte units)
  constexpr uint64_t kA = (A_MN ? 16 * 128 : 32) >> 4, kB = (B_MN ? 16 * 128 : 32) >> 4;
  const uint64_t a0 = sw128_desc(m.sA, A_MN ? CHUNK : 16, 1024);
  const uint64_t b0 = sw128_desc(m.sB, B_MN ? CHUNK : 16, 1024);
#pragma unroll 1
  for (int kb = 0; kb < nkb; ++kb) {
    if (!__all_sync(0xffffffffu, wait_bar(m.full + 8 * r.s, r.ph, wc))) return false;
    tc_fence_after();
    const uint64_t ad = a0 + r.s * (OPER >> 4), bd = b0 + r.s * (OPER >> 4);
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk)
        tc_mma_bf16_cg2(dt, ad + kk * kA, bd + kk * kB, kIdesc, (kb | kk) != 0);
      tc_commit_cg2_mc(m.empty + 8 * r.s, 0x3);
    }
    r.next(STAGES);
  }
  return true;
}

// Every copy lands before either CTA may exit: the peer reports how
// many blocks it issued; for the blocks that one side did not issue
// (only after a timeout) the leader makes that side's arrival and
// waits for the phase, which completes once the issued copies landed.
__device__ __forceinline__ void drain_copies(const PSmem& m, int it, bool leader) {
  if (!leader) {
    st_cluster_s32(mapa_shared(m.issued, 0), it);
    mbar_arrive_cluster(mapa_shared(m.pdone, 0));
  } else {
    const bool rep = wait_bar_cluster_drain(m.pdone, 0, DRAIN_LIMIT);
    const int other = rep ? ld_shared_s32(m.issued) : it;
    const int hi = std::max(it, other);
    for (int j = std::max(0, hi - STAGES); j < hi; ++j) {
      const uint32_t b = m.full + 8 * (j % STAGES);
      if (j >= it) mbar_arrive(b);
      if (j >= other) mbar_arrive(b);
      wait_bar_drain(b, (j / STAGES) & 1, DRAIN_LIMIT);
    }
  }
}

// ---------------------------------------------------------------- host
template <typename K>
cudaError_t allow_smem(K kern, size_t smem, bool* done) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && done[dev]) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// bf16 operand [rows][cols] with row stride ld: K-major boxes of 64 columns x
// `box_rows` rows, MN-major boxes of 64 columns x 64 rows.
bool tmap_operand(CUtensorMap* m, const DenseOperand& o, bool mn, int box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(o.cols), static_cast<uint64_t>(o.rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(o.ld) * 2};
  const uint32_t box[2] = {64, static_cast<uint32_t>(mn ? 64 : box_rows)};
  return encode_tmap(m, o.ptr, 2, dims, strides, box);
}

// Rows of an output start on 16-byte boundaries.
bool vec_rows(const void* out, int N, bool f32) {
  return aligned16(out) && (static_cast<long long>(N) * (f32 ? 4 : 2)) % 16 == 0;
}

}  // namespace
}  // namespace mgg
