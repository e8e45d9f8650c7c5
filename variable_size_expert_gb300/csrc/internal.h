// Host-side interface between the C-ABI layer (api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/mgg.h"

namespace mgg {

// An NVTX range over one C-ABI call, named after the entry point, so that
// profiler timelines group each call's kernels (no cost without a tool).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// Tile shapes of the tensor-core kernels.
constexpr int kPairBM = 256;   // CTA-pair tile rows (MMA M, 128 per CTA)
constexpr int kPairBN = 256;   // CTA-pair tile columns (MMA N, B split 128 per CTA)
constexpr int kBK = 64;        // contraction step: one 128-byte swizzle row of bf16
constexpr int kDwPad = 64;     // expert segments of the scaled dY operand are padded to this
constexpr int kMaskedBM = 128; // decode tile: weight rows (MMA M)
constexpr int kMaskedBI = 64;  // decode tile: activation rows per tile (MMA N <= 64)
constexpr int kSimtBM = 64;    // f32 path tile rows
constexpr int kSimtBN = 64;    // f32 path tile columns
constexpr int kRouteChunk = 256;
constexpr int kMaxExperts = 1024;

// Split of the dW contraction ("Grouped GEMM for MoE", §Backward: in dW a hot
// expert has as many tiles as any other but longer contraction loops; the
// remedy named there is to split the contraction across CTAs and reduce).
// work = the contraction steps (kBK rows) summed over all dW tiles, pairs =
// the CTA pairs the dW GEMM runs on.  The target piece length is the ideal
// per-pair load (at least kDwSplitMin steps); an expert whose tiles are more
// than 1.25x that long is cut into the fewest pieces of at most 1.25x the
// target (at most kDwSplitMax, at most one per step), which add into a
// zeroed dW.
constexpr int kDwSplitMin = 16;  // 1024 rows; 8-step pieces measured no faster than whole tiles
constexpr int kDwSplitMax = 16;

__host__ __device__ inline long long dw_split_target(long long work, int pairs) {
  const long long t = pairs > 0 ? (work + pairs - 1) / pairs : work;
  return t > kDwSplitMin ? t : kDwSplitMin;
}
__host__ __device__ inline int dw_split_pieces(int steps, long long target, int smax) {
  if (smax <= 1 || 4LL * steps <= 5LL * target) return 1;
  long long s = (4LL * steps + 5LL * target - 1) / (5LL * target);
  if (s > smax) s = smax;
  if (s > steps) s = steps;
  return s > 1 ? static_cast<int>(s) : 1;
}

// Default pipeline wait limit in SM clock cycles (about a second).
constexpr long long kDefaultWaitLimit = 2000000000LL;

// Row GEMM modes: A gathered through row_token (fused, fused + dtopk, gate/up)
// or loaded in sorted order (bare, scatter); output stored in sorted order
// (bare), weighted and added into token rows (fused, fused + dtopk,
// scatter), or gated into bf16 h (gate/up).
enum RowsMode {
  kModeBare = 0,
  kModeFused = 1,
  kModeFusedDtopk = 2,
  kModeGateUp = 3,
  kModeScatter = 4,
  kModeGateUpSave = 5,  // gate/up forward that also stores g and u (f32) for the backward
  kModeSwiGluBwd = 6    // gated FFN backward: dh = w (dy Wd), then dg, du from the saved g, u
};

// One launch of the row-gathering grouped GEMM (forward, bare, dX).
struct RowsParams {
  const void* A;               // [*, lda] rows, gathered through row_token (or identity)
  int lda;                     // elements per A row
  int Kc;                      // contraction length
  const int32_t* row_token;    // [S] sorted row -> A row; null = identity (bare)
  const float* row_weight;     // [S] fused: per-row scale
  const int32_t* row_assign;   // [S] dtopk: sorted row -> assignment
  const int32_t* tile_start;   // [E+1]
  const int32_t* start;        // [E+1]
  int E;
  int Nout;                    // output columns
  float* out;                  // bare: [rows, Nout]; fused: [T, Nout] accumulated
  int ldo;
  const void* xdot;            // dtopk: x [T, ldx] (same dtype as A)
  int ldx;
  float* dtopk;                // dtopk: [S] indexed by assignment
  int b_merged;                // MN-major B: tmap_b is the 4-D chunked view, one box per stage
  void* hout;                  // gate/up: h [S, ldh] bf16, sorted rows
  int ldh;
  // e4m3 operands (fused and bare modes): A and B rows are moved as 16-bit
  // units, so lda and Kc count byte pairs; the epilogue multiplies by
  // a_scale (per token in the fused mode, per row in the bare mode) and by
  // b_scale[e * Nout + n] (per expert and output column)
  const float* a_scale;
  const float* b_scale;
  // gated FFN: gate/up saved by the forward, [rows, ldgu] f32, g in columns
  // 0..Nout-1 and u in Nout..2 Nout-1 (written by kModeGateUpSave into guout,
  // read by kModeSwiGluBwd from gu, which writes dg | du the same way into hout)
  float* guout;
  const float* gu;
  int ldgu;
  int max_pairs;               // cap on the persistent grid's CTA pairs (0: all that fit)
  // Row-tile height (fused and bare modes, bf16): kRowTilePair runs the
  // 256-row pair tiles only, kRowTileCta the 128-row single-CTA tiles only,
  // kRowTileAuto launches both kernels and each evaluates choose_rows128 on
  // the device; the one not chosen exits at entry.
  int row_tile;
  int pair_workers, cta_workers;  // the two kernels' grids (kRowTileAuto): 76 pairs, 152 CTAs
  int32_t* dev_status;
  long long wait_limit;
};
enum RowTile { kRowTilePair = 0, kRowTileAuto = 1, kRowTileCta = 2 };
// Measured cost of a round of 128 x 256 single-CTA tiles relative to a
// round of 256 x 256 pair tiles (each SM of a pair moves half the weight
// bytes per FLOP of a single CTA): rnum / rden; 1.15 on the skewed forward
// (E=64, k=8, Zipf 1.2: 15.6 against 13.6 us per round).
constexpr int kRow128CostNum = 6;
constexpr int kRow128CostDen = 5;

struct DwParams {
  const void* x;               // [T, K]
  int K;
  int N;
  const void* dyw;             // [S_pad, N] scaled sorted dY, expert segments padded
  const int32_t* counts;       // [E]
  const int32_t* start;        // [E+1]
  const int32_t* pstart;       // [E+1] padded segment starts
  const int32_t* row_token;    // [S]
  const float* row_weight;     // [S] (f32 path)
  const float* dy;             // [T, N] (f32 path)
  int E;
  float* dW;                   // [E, N, K]
  int b_merged;                // tmap_dyw is the 3-D chunked view, one box per stage
  const int32_t* expert_order;  // [E] experts by decreasing row count (null: index order)
  int32_t* tile_counter;       // zeroed counter: dynamic tile queue (null: static schedule)
  // [E+1] exclusive prefix of the tiles of the experts in visiting order,
  // split pieces included (null: E x tiles per expert, no split)
  const int32_t* tile_prefix;
  int max_pairs;               // cap on the persistent grid's CTA pairs (0: all that fit)
  int32_t* dev_status;
  long long wait_limit;
};

struct MaskedParams {
  const void* x;               // [E, M_max, K]
  const int32_t* masked_m;     // [E]
  int E, M_max, N, K;
  float* y;                    // [E, M_max, N]
  // e4m3 operands: K counts byte pairs (rows move as 16-bit units); the
  // epilogue multiplies by x_scale[e * M_max + i] and w_scale[e * N + n]
  const float* x_scale;
  const float* w_scale;
  int32_t* dev_status;
  long long wait_limit;
};

// Activations of the dense products (the values of mgg_activation; the last one,
// for the library's own calls on CTA pairs, multiplies every product by *scale0 *
// *scale1).
enum DenseAct { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActScale = 4 };

// A bf16 operand [rows][cols], row stride ld elements.
struct DenseOperand {
  const void* ptr;
  int rows, cols;
  long long ld;
};
// D[M, N] = sum_k A[m, k] B[n, k]; a_mn / b_mn: the operand lies [k][m] / [k][n].
struct DenseProduct {
  int M, N, Kc;
  bool a_mn, b_mn;
  void* out;        // [M, N] dense
  bool out_f32;     // else bf16
  bool out_vec;     // rows of out start on 16-byte boundaries (set by the launcher)
  bool epilogue;    // bias, activation, residual, z kept
  int tiles;        // set by the launcher
};
struct DenseParams {
  DenseProduct pr[2];
  const void* bias;      // [N] or null
  bool bias_f32, bias_vec;  // bias_vec: 16-byte loads
  int act;
  const void* residual;  // [M, ldr] or null
  bool res_f32, res_vec; // res_vec: base and rows on 16-byte boundaries
  bool res_tma;          // set by the launcher
  long long ldr;
  void* pre;             // bf16 z [M, N] or null
  bool pre_vec;          // rows on 16-byte boundaries (set by the launcher)
  int32_t* dev_status;
  long long wait_limit;
};
struct DenseBackward {
  const void* dy;
  bool dy_f32;
  long long lddy;
  const void* x;
  long long ldx;
  const void* W;
  const void* pre;
  int act;
  int T, K, N;
  void *dx, *dW, *db;    // any may be null
  bool db_f32;
  int32_t* dev_status;
  long long wait_limit;
};

// device properties
int num_sms();
// null-safe argument checks shared by the C-ABI translation units
mgg_status check_arch();
long long wait_limit();

// tensor maps
bool encode_tmap(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                 const uint64_t* strides_bytes, const uint32_t* box);

// [rows][cols] bf16 or f32, row stride ld elements, for TMA loads of 32 rows x
// 32 columns (bf16: 64-byte swizzle, f32: 128-byte)
bool encode_tmap_residual(CUtensorMap* map, const void* base, bool f32, int rows, int cols,
                          long long ld);

// norm.cu
int norm_bwd_blocks();  // partial rows of the weight and bias gradients
cudaError_t launch_norm_fwd(const void* x, bool x_f32, long long ldx, const void* w, const void* b,
                            bool w_f32, int T, int K, float eps, void* y, bool y_f32, float* mean,
                            float* rstd, cudaStream_t st);
cudaError_t launch_norm_bwd(const void* dy, bool y_f32, const void* x, bool x_f32, long long ldx,
                            const void* w, bool w_f32, const float* mean, const float* rstd, int T,
                            int K, void* dx, void* dw, void* db, float* part, cudaStream_t st);
// out0[K] = column sums of part[0][nb][K], out1 (or null) of part[1][nb][K], in a fixed order
cudaError_t launch_column_sums(const float* part, int nb, int K, void* out0, void* out1,
                               bool out_f32, cudaStream_t st);
// select.cu
cudaError_t launch_select(const void* logits, bool f32, long long ldl, int T, int E, int k,
                          bool softmax, const float* bias, int groups, int topk_groups,
                          bool two_best, bool renorm, float scale, int32_t* ids, float* weights,
                          cudaStream_t st);
cudaError_t launch_select_bwd(const float* g, const void* logits, bool f32, long long ldl,
                              const int32_t* ids, const float* w, int T, int E, int k,
                              bool softmax, bool renorm, float scale, void* out,
                              int32_t* dev_status, cudaStream_t st);
// linear.cu
size_t dense_bwd_ws_bytes(int T, int N);
cudaError_t launch_dense_forward(const DenseParams& p, const DenseOperand& x,
                                 const DenseOperand& W, cudaStream_t st);
// What the library's own products on CTA pairs can have beside.
struct PairOptions {
  bool always;                   // on pairs, whatever the estimate says
  int slices[2];                 // pieces of a product's contraction, each with an f32 output
                                 // [M, N] of its own, one behind the other (0: one)
  const float *scale0, *scale1;  // of kActScale
};
cudaError_t launch_dense_products(const DenseParams& q, const PairOptions& opt, const DenseProduct* pr,
                                  const DenseOperand* a, const DenseOperand* b, cudaStream_t st);
cudaError_t launch_dense_backward(const DenseBackward& a, void* ws, cudaStream_t st);

int dense_pair_count();  // co-resident clusters of two (persistent grid)

// vocab.cu
struct VocabForward {
  const void* x;
  long long ldx;
  const void* W;
  const void* targets;
  bool i64;
  long long ignore;
  int T, K, V, reduction;
  float z_loss;
  float *loss, *lse, *weight;
  int32_t* dev_status;
  long long wait_limit;
};
struct VocabBackward {
  const float* dloss;
  bool per_token;
  const float* weight;
  const void* x;
  long long ldx;
  const void* W;
  const void* targets;
  bool i64;
  long long ignore;
  const float* lse;
  int T, K, V;
  float z_loss;
  void *dx, *dW;  // either may be null
  int32_t* dev_status;
  long long wait_limit;
};
size_t vocab_fwd_ws_bytes(int T, int K, int V);
size_t vocab_bwd_ws_bytes(int T, int K, int V);
cudaError_t launch_vocab_forward(const VocabForward& a, void* ws, cudaStream_t st);
cudaError_t launch_vocab_backward(const VocabBackward& a, void* ws, cudaStream_t st);

// Longest side of the balance loss and the vocabulary's products: the kernels count
// rows in 32 bits and step past a side's end.
constexpr int kMostRows = 1 << 30;

// balance.cu
struct BalanceArgs {
  const void* logits;
  bool f32;
  long long ldl;
  const int32_t* ids;    // [T, k] (forward)
  const uint8_t* mask;   // [T] or null
  int T, E, k, sequences;
  bool softmax;
  float* loss;           // [1]
  int32_t* counts;       // [sequences, E]
  float* slope;          // [sequences, E]
  const float* dloss;    // [1] (backward)
  void* dlogits;         // [T, E]
  int32_t* dev_status;
};
size_t balance_ws_bytes(int T, int E, int sequences);
cudaError_t launch_balance(const BalanceArgs& a, void* ws, cudaStream_t st);
cudaError_t launch_balance_bwd(const BalanceArgs& a, cudaStream_t st);

// adamw.cu
struct AdamwArgs {
  const mgg_adamw_tensor* tensors;  // host memory
  int count;
  bool p_f32, g_f32, master, bits8;
  double lr, beta1, beta2, eps, decay;
  long long step;
  const float* lr_dev;       // or null
  const int32_t* step_dev;   // or null
  const float* grad_scale;   // or null
};
cudaError_t launch_adamw(const AdamwArgs& a, cudaStream_t st);

// router.cu
cudaError_t launch_route(const int32_t* ids, const float* w, int T, int k, int E, int BM,
                         int tiles_n, int32_t* counts, int32_t* end_offs, int32_t* start,
                         int32_t* tile_start, int32_t* row_assign, int32_t* row_token,
                         float* row_weight, int32_t* assign_row, int32_t* dev_status, void* ws,
                         cudaStream_t st, float* zero = nullptr, size_t zero_floats = 0);
size_t route_ws_bytes(int T, int k, int E);
cudaError_t launch_offsets_scan(const int32_t* offs, bool is_sizes, int E, int rows, int BM,
                                int tiles_n, int32_t* start, int32_t* tile_start,
                                int32_t* dev_status, cudaStream_t st);
cudaError_t launch_bwd_scan(const int32_t* counts, int E, int BM, int tiles_n, int pad,
                            int32_t* tile_start_dx, int32_t* pstart, cudaStream_t st);
// What the backward prep needs to plan the dW contraction split: it writes
// `tiles` (the dW tile prefix in visiting order, E+1 ints) and zeroes the
// dW slices of the experts it splits.
struct DwSplitPlan {
  int32_t* tiles;   // [E+1]
  float* dW;        // [E, N, K]
  int tpe;          // dW tiles per expert and piece: ceil(K/256) x ceil(N/256)
  int pairs;        // CTA pairs the dW GEMM runs on
  int smax;         // most pieces per expert (1: no split)
};
cudaError_t launch_bwd_prep(const float* dy, int T, int N, int K, int k, const int32_t* counts,
                            const int32_t* start, int BM, int tiles_n, int pad,
                            int32_t* tile_start_dx, int32_t* pstart, const int32_t* assign_row,
                            const float* row_weight, int E, int S_pad_max, void* dy_b, void* dyw,
                            float* dx, float* dtopk, cudaStream_t st,
                            int32_t* expert_order = nullptr, const DwSplitPlan* split = nullptr);
cudaError_t launch_iota_ones(int32_t* iota, float* ones, int n, cudaStream_t st);
cudaError_t launch_debug_schedule(const int32_t* tile_start, const int32_t* start, int E, int BM,
                                  int max_tiles, int32_t* out, cudaStream_t st);

// gemm_pair.cu (tcgen05, cta_group::2)
// f8: e4m3 operands (kModeFused, kModeBare and kModeFusedDtopk, all K-major)
cudaError_t launch_rows_pair(int mode, bool b_mn_major, const CUtensorMap& tmap_a,
                             const CUtensorMap& tmap_b, const RowsParams& p, cudaStream_t st,
                             bool f8 = false);
// gemm_cta.cu (tcgen05, cta_group::1): 128-row tiles, kModeFused or
// kModeBare; tmap_b is the weights' map with 128-row boxes (two per stage)
cudaError_t launch_rows_cta(int mode, const CUtensorMap& tmap_a, const CUtensorMap& tmap_b,
                            const RowsParams& p, cudaStream_t st);
// writes the device's per-call row-tile choice (1: 128-row tiles) to out[0]
cudaError_t launch_row_tile_choice(const int32_t* start, int E, int N, int32_t* out,
                                   cudaStream_t st);
// tmap_dw: dW [E][N][K] f32 as a 3-D map, box {32, 32, 1}, no swizzle.
cudaError_t launch_dw_pair(const CUtensorMap& tmap_dyw, const CUtensorMap& tmap_dw,
                           const DwParams& p, cudaStream_t st);
// gemm_masked.cu (tcgen05)
cudaError_t launch_masked_gemm(const CUtensorMap& tmap_w, const MaskedParams& p, cudaStream_t st,
                               bool f8 = false);
// quant.cu: per-row e4m3 quantisation of a [rows, cols] bf16 or f32 matrix
cudaError_t launch_quantize_fp8(const void* src, bool src_f32, int rows, int cols, uint8_t* q,
                                float* scale, cudaStream_t st);
// W [E, N, K] bf16 -> codes [E, K, N] and scale [E, K], per (expert, column k)
cudaError_t launch_quantize_fp8_cols(const void* W, int E, int N, int K, uint8_t* q, float* scale,
                                     cudaStream_t st);

// simt_f32.cu (exact f32 path)
cudaError_t launch_rows_f32(int mode, bool w_transposed, const RowsParams& p, const float* W,
                            int Kw, cudaStream_t st);
cudaError_t launch_dw_f32(const DwParams& p, cudaStream_t st);
cudaError_t launch_masked_f32(const MaskedParams& p, const float* W, cudaStream_t st);

}  // namespace mgg
