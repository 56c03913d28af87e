// Block-scaled NVFP4 x NVFP4 GEMM with a dequantizing epilogue, and the fused
// multi-segment projection, for sm_100a.
//
// What it computes [picx.dev summary of "Why Gated DeltaNet Survives 4-Bit
// Quantization", "Background": native 4-bit tensor-core GEMMs on NVFP4
// operands; anthology record LIT-800, "Standing in the anthology", and the
// cctest.ai article, "Main findings": fused projections must apply each
// module's own global scale]:
//   out[m,n] = alpha(n) * sum_b sA[m,b] sW[n,b] sum_{k in b} e2m1(A[m,k]) e2m1(W[n,k])
//   alpha(n) = 1 / (gA * gW[segment of n])
//
// Design (one persistent CTA per SM):
//   warp 0    TMA producer: per 256-wide K step, one 2-D TMA box of each
//             operand's codes (128-byte rows, 128B swizzle) and one or two
//             bulk copies of the pre-swizzled E4M3 scale chunks, all landing
//             on one mbarrier with an expected byte count.
//   warp 1    TMEM allocator and MMA issuer: per step, four tcgen05.mma
//             kind::mxf4nvf4 block_scale (K = 64 each) into the FP32
//             accumulator in TMEM, then tcgen05.commit to release the stage.
//   warps 2-5 epilogue: tcgen05.ld the accumulator (one TMEM lane per
//             output row), scale by alpha, round once to bf16 (or keep
//             f32), free the accumulator, store.  With an in-kernel
//             activation (nvfp4_linear) they first quantize X into shared
//             memory.
//   warps 6+  scale copies: one warp for P's scale chunks and one per
//             128-row block of Q's move each step's scales into TMEM
//             (tcgen05.cp 32x128b.warpx4) and signal the MMA warp.  Each
//             tcgen05 instruction holds its issuing thread for tens of
//             cycles; spread over warps, copies and MMAs overlap.
// Two tile shapes:
//   normal  P = activations (128-row tiles), Q = weight (256-row tiles):
//           prefill and fused projections.
//   swap    P = weight (128-row tiles), Q = all activation rows (<= 128):
//           decode, so the 128-row MMA dimension walks the weight; the
//           K loop is split over the CTAs (stream-K) so every SM streams W.
// Every mbarrier wait is bounded (see ptx.cuh); on timeout the CTA drains
// its in-flight copies and MMAs (bounded again), frees TMEM and exits.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "block_quant.cuh"
#include "common.h"
#include "groups.cuh"
#include "ptx.cuh"

#include <type_traits>

namespace nvfp4 {

constexpr int kBM = 128;          // MMA M: rows of operand P per tile
constexpr int kSfChunk = 512;     // bytes of one 128-row x 4-scale chunk
constexpr int kTmemCols = 512;
constexpr int kGroupP = 64;       // tile raster: 64 P-tiles (8192 rows) share each Q-tile sweep
constexpr int kStageOutBytes = 16384;   // one 128-row x 128-byte output sub-tile
constexpr int kEpiBar = 1;        // named barrier id of the 128 epilogue threads

struct alignas(64) GemmParams {
  CUtensorMap tmap_p;
  CUtensorMap tmap_q;
  CUtensorMap tmap_out;  // output [M, N] in 128-byte-wide boxes (normal tiles, TMA store path)
  const uint8_t* sf_p;
  const uint8_t* sf_q;
  void* out;
  uint64_t* ws;          // swapped tiles: tagged FP32 partial tiles, 2 slots per CTA (all words empty between launches)
  unsigned* err;
  uint64_t timeout_ns;   // bound of every wait for work to arrive
  uint64_t drain_ns;     // bound of the waits for a CTA's own copies and MMAs before it exits (>= 1 s)
  int64_t M, N;          // output [M, N]
  int rows_p, rows_q;    // rows of the P and Q operands
  int rb_q;              // 128-row scale blocks allocated for Q
  int kc;                // scale chunks per row block: ceil(K / 64), MXFP4 ceil(K / 128)
  int kmma;              // ceil(K / 64): MMAs per row of tiles
  int kt;                // ceil(K / (64 * kKB)): pipeline steps per tile
  int tiles_p, tiles_q;
  int tma_store;         // 1: output through shared memory and TMA stores
  int w_static;          // 1: the weight lies in memory declared read-only (nvfp4_declare_static)
  int n_seg;
  int test_stall;        // failure-path test only: the split-tile adder never sees its helpers' partials
  int group_p;           // tile raster: P tiles per Q-tile sweep
  CUtensorMap tmap_sfa;  // CTA pairs: scale chunks of P and Q as [chunks, 128] 32-bit words
  CUtensorMap tmap_sfb;
  int seg_end[NVFP4_MAX_SEGMENTS];
  float seg_alpha[NVFP4_MAX_SEGMENTS];
  // activation quantized in the kernel (swapped tiles only): X [M, K]
  // row-major, its global scale, K
  const void* x;
  float x_gs;
  int64_t K;
  // buffer extents, checked by the debug build's bounds checks
  uint64_t sf_p_bytes, sf_q_bytes;   // scale buffers
  uint64_t out_elems;                // M * N
  uint64_t ws_words;                 // K-split workspace, 64-bit words
  uint64_t x_bytes;                  // in-kernel activation X
};

// Groups of rows, each with a weight of its own (nvfp4_grouped_gemm): the
// activation rows of group g are [off[g], off[g + 1]), its weight rows
// [g N, (g + 1) N) of one [E N, K / 2] operand.
struct GroupedGemmParams : GemmParams {
  CUtensorMap tmap_q_box[4];   // activation codes in boxes of 16, 32, 64 and 128 rows
  const int32_t* offsets;      // device [E + 1]
  const float* ga;             // device [E], activation and weight global scales
  const float* gw;
  int E;
  int w_blocks;                // 128-row scale blocks of one group's weight
};

// QX: 0 = the Q operand (activations) arrives quantized, as codes and scales
// in global memory; 1 / 2 = swapped tiles whose activation X (bf16 / f32) the
// kernel quantizes itself into shared memory, all of the CTA's K-steps at
// once, before the first MMA.
// MX: MXFP4 operands (32-element blocks, E8M0 scales, kind::mxf4 with two
// scales per MMA) instead of NVFP4 (16-element blocks, E4M3 scales).
// PAIR: prefill tiles of 256 x 256 computed by a pair of CTAs (a cluster of
// two): each CTA loads its 128 activation rows and half of the 256 weight
// rows (plus all 256 rows' scales); the even CTA issues the M = 256 MMAs and
// scale copies for both (tcgen05 cta_group::2); each CTA drains its own 128
// accumulator rows.
// GROUPED: the rows are split into groups (experts), each multiplied by a
// weight of its own; group offsets are read on the device.  CTA pairs put the
// weight on P, 128 rows a CTA, and up to BN activation rows of one group on
// Q: the MMA's N is as many columns as the tile has rows (rounded up to 32),
// so a group's last tile costs what its rows cost, and each CTA loads its half
// of them in the smallest of four boxes (16, 32, 64, 128 rows).  With the
// activations on P, whose 256 rows are fixed, 32768 rows in 64 groups against
// weights of 2048 x 5120 took 8 % longer.  BN = 256 for large
// groups; BN = 128 leaves room for more stages, and two whole accumulators.
template <int BN, bool SWAP, int QX = 0, bool MX = false, bool PAIR = false, bool GROUPED = false>
struct Cfg {
  static constexpr bool kQx = QX != 0;
  // K per pipeline step: kKB blocks of 64 (one MMA each), 256 deep, as
  // 128-byte rows with the 128B swizzle.  (128-deep steps with 64-byte rows
  // and the 64B swizzle also work, and fit twice as many stages, but measured
  // 40 % slower on prefill tiles: the per-step barrier and commit work then
  // outweighs the earlier buffer release.)
  static constexpr int kKB = 4;
  static constexpr int kRowBytes = 32 * kKB;                         // code bytes per row per step
  static constexpr uint32_t kSwizzleLayout = kRowBytes == 128 ? 2u : 4u;   // descriptor layout type
  static constexpr uint32_t kSbo = 8 * kRowBytes;                    // bytes between 8-row groups
  static constexpr int kSfbBlocks = (BN + 127) / 128;                // 128-row scale blocks of Q
  static constexpr int kABytes = kBM * kRowBytes;
  static constexpr int kBBytes = kQx ? 0 : (PAIR ? BN / 2 : BN) * kRowBytes;   // Q codes per stage (per CTA)
  // scale chunks (128 rows x 4 scales, 512 bytes) per step: a chunk covers 64
  // K-elements of 16-element blocks (one MMA), or 128 of 32-element blocks
  static constexpr int kChunks = MX ? kKB / 2 : kKB;
  static constexpr int kSfaBytes = kChunks * kSfChunk;
  static constexpr int kSfbBytes = kQx ? 0 : kSfbBlocks * kChunks * kSfChunk;
  static constexpr int kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  // double-buffered; grouped tiles of BN = 128 give the second buffer to a
  // seventh stage (1.5 % less time for 2 rows of each of 64 experts)
  static constexpr int kOutBufs = GROUPED && BN == 128 ? 1 : 2;
  // (Eight epilogue warps for grouped tiles of 256, on alternate tiles or on
  // alternate slots: 10 % less time at K = 512, 3 % more at K >= 2048.)
  static constexpr int kOutBytes = SWAP ? 0 : kOutBufs * kStageOutBytes;    // output sub-tiles
  // in-kernel activation: codes (BN rows x 128 B, 128B swizzle) and one
  // 128-row scale block per K-step, for up to kActSteps steps
  static constexpr int kActSteps = kQx ? (BN <= 16 ? 8 : 16) : 0;
  static constexpr int kActCodeBytes = BN * kRowBytes;
  static constexpr int kActSfBytes = kKB * kSfChunk;
  static constexpr int kActBytes = kActSteps * (kActCodeBytes + kActSfBytes);
  // CTA pairs keep 4 stages although 5 fit: 5 ran 2-7 % slower on every
  // prefill and fused shape measured (the deeper ring lets the copy warps
  // run further ahead of MMAs that are not waiting on data)
  static constexpr int kMaxStages = PAIR && BN == 256 ? 4 : 8;
  // Decode tiles with a small activation side keep to under half of the
  // SM's shared memory (and TMEM, and 128 registers), so two CTAs fit on an
  // SM.  With BN = 16 the grid has 2 x SMs CTAs: each streams half as much
  // weight and each SM keeps twice the stages in flight (decode step 12.4
  // against 13.3 us at 8x12288x5120; four stages measured 2 % faster than
  // five).  The profiler's occupancy limits are two CTAs per SM and it sees
  // about 1.8 resident on average, but the occupancy API reports one.  A
  // split tile's summing CTA waits only for partials that CTAs with higher
  // indices produce as their first work item, so the grid completes whenever
  // CTAs start in index order, resident together or not (bounded waits
  // report a timeout otherwise); the opt-in cooperative launch sizes the
  // grid to what the occupancy API admits instead.  BN = 32, and the MXFP4
  // decode tile (13.5 against 10.9 us), are slower at two per SM and keep
  // one CTA per SM.  The in-kernel activation variant follows the same grid (its
  // BN = 16 form holds 8 K-steps of activation instead of 16, covering the
  // same shapes).
  static constexpr bool kCoRes = SWAP && (kQx ? BN <= 16 : BN <= 32);
  static constexpr int kMinBlocks = kCoRes ? 2 : 1;
  static constexpr int kGridPerSm = SWAP && BN <= 16 && !MX ? 2 : 1;
  static constexpr int kSmemBudget = kCoRes ? 104 * 1024 : 222 * 1024;
  static constexpr int kFit = (kSmemBudget - kOutBytes - kActBytes) / kStageBytes;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kOffA + kStages * kABytes;
  static constexpr int kOffSfa = kOffB + kStages * kBBytes;
  static constexpr int kOffSfb = kOffSfa + kStages * kSfaBytes;
  static constexpr int kOffAct = kOffSfb + kStages * kSfbBytes;      // 1024-aligned
  static constexpr int kOffActSf = kOffAct + kActSteps * kActCodeBytes;
  static constexpr int kOffOut = kOffActSf + kActSteps * kActSfBytes;   // 1024-aligned
  static constexpr int kOffBar = kOffOut + kOutBytes;
  // Extra warps issue the scale copies (warp 6: P's scales, warp 7 + rb: the
  // scales of Q's 128-row block rb) so that the MMA warp issues only MMAs; a
  // tcgen05 instruction holds its issuing thread for tens of cycles, but
  // instructions from different threads proceed in parallel.
  static constexpr int kCopyWarps = 1 + kSfbBlocks;
  static constexpr int kThreads = 192 + 32 * kCopyWarps;
  // full, empty, acc_full, acc_empty, drain, one scales-ready barrier per
  // stage, one drain barrier per copy warp, and (in-kernel activation) one
  // activation-ready barrier per K-step
  static constexpr int kNumBars = 2 * kStages + 3 + kStages + kCopyWarps + kActSteps;
  static constexpr int kOffSeg = kOffBar + kNumBars * 8;             // segment table: ends, alphas
  static constexpr int kOffMisc = kOffSeg + 2 * 4 * NVFP4_MAX_SEGMENTS;
  static constexpr int kOffRtab = kOffMisc + 16;                     // in-kernel activation: g / e4m3(s)
  static constexpr int kOffTab = kOffRtab + (kQx ? 1024 : 0);        // grouped: table of groups
  static constexpr int kSmemBytes = kOffTab + (GROUPED ? (int)sizeof(GroupTable) : 0) + 1024;   // + alignment slack
  // TMEM columns.  Normal 128x256 tiles: the copy warps run ahead of the
  // MMAs, so the scales of successive steps use a ring of regions at the top
  // of TMEM ([320,512) for four 48-column regions); the two accumulator
  // buffers, [0,256) and [kAcc1Col, kAcc1Col + 256), fill the rest and
  // overlap, so tile t+1 can start as soon as the epilogue has drained the
  // shared columns of tile t (it drains those 64-column slots first).
  // Swapped (decode) tiles: one accumulator and one scale region per
  // pipeline stage.
  static constexpr int kAccCols = BN < 32 ? 32 : BN;
  static constexpr bool kOverlapAcc = !SWAP && BN == 256;
  static constexpr int kSfaCols = 4 * kChunks;                       // 4 columns per chunk
  static constexpr int kSfbCols = kSfbBlocks * 4 * kChunks;
  static constexpr int kSfStageCols = kSfaCols + kSfbCols;
  // four regions (192 columns) let the copy warps run up to three steps
  // ahead; the accumulators then share 192 columns (3 slots drained first)
  static constexpr int kSfRegions = kOverlapAcc ? 4 : kStages;
  static constexpr int kSfBase = kOverlapAcc ? kTmemCols - kSfRegions * kSfStageCols : kAccCols * (GROUPED ? 2 : 1);
  // grouped pairs of BN = 128: two accumulators side by side
  static constexpr int kAcc1Col = kOverlapAcc ? kSfBase - 256 : GROUPED ? kAccCols : 0;
  static constexpr int kSharedSlots = kOverlapAcc ? (256 - kAcc1Col + 63) / 64 : 0;   // drained before release
  static constexpr int kTmemAlloc = kCoRes ? 256 : kTmemCols;         // columns this CTA allocates
  static_assert(kAcc1Col % 32 == 0, "accumulator column alignment");
  static_assert(kStages >= 2, "pipeline depth");
  static_assert(kSfBase + kSfRegions * kSfStageCols <= kTmemAlloc, "TMEM budget");
  static_assert(!kCoRes || kSmemBytes <= 113 * 1024, "under half of the SM's shared memory");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(BN % 16 == 0 && BN <= 256, "MMA N");
  static_assert(!kQx || (SWAP && BN <= 32), "in-kernel activation: swapped tiles, M <= 32");
  static_assert(!(kQx && MX), "in-kernel activation: NVFP4 only");
  static_assert(!GROUPED || (PAIR && !MX && (BN == 256 || BN == 128)), "grouped: NVFP4 CTA pairs");
  static_assert(!PAIR || (!SWAP && (BN == 256 || GROUPED) && !kQx), "CTA pairs: normal 256 x 256 tiles");
  static constexpr int kMmaM = PAIR ? 2 * kBM : kBM;                 // MMA M (over the pair)
  static constexpr int kGroupTiles = PAIR ? kGroupP / 2 : kGroupP;   // raster group, in tiles of P
  static_assert(kOffAct % 1024 == 0 && kActCodeBytes % 1024 == 0, "activation tiles on swizzle atoms");
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);   // round to nearest even
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void tile_coords(const GemmParams& p, int tile, int& tp, int& tq) {
  const int per_group = p.group_p * p.tiles_q;
  const int group = tile / per_group;
  const int first = group * p.group_p;
  const int gsize = min(p.tiles_p - first, p.group_p);
  const int local = tile - group * per_group;
  tp = first + local % gsize;
  tq = local / gsize;
}

// Work of one CTA, as a sequence of (tile, k-step range) items.
//   normal tiles: whole tiles t = blockIdx.x, blockIdx.x + gridDim.x, ...
//   swapped tiles (stream-K): the tiles_p * kt (tile, k-step) units are cut
//   into gridDim.x contiguous, balanced ranges; CTA c owns units
//   [floor(c U / G), floor((c+1) U / G)).  An item is the part of that range
//   inside one tile.
//   CTA pairs: whole 256 x 256 tiles t = pair, pair + pairs, ... for the
//   pair index blockIdx.x / 2.
struct WorkIter {
  int64_t u, u_end;   // swapped: unit range; normal: next tile index, tile count
  int kt;
  bool swap, pair;
};

__device__ __forceinline__ int64_t unit_begin(int64_t c, int64_t U, int64_t G) { return c * U / G; }

// CTA whose range holds unit u: the largest c with floor(c U / G) <= u.
__device__ __forceinline__ int64_t cta_of_unit(int64_t u, int64_t U, int64_t G) {
  return ((u + 1) * G + U - 1) / U - 1;
}

__device__ __forceinline__ WorkIter work_begin(const GemmParams& p, bool swap, bool pair = false) {
  WorkIter w;
  w.kt = p.kt;
  w.swap = swap;
  w.pair = pair;
  if (swap) {
    const int64_t U = (int64_t)p.tiles_p * p.kt, G = gridDim.x;
    w.u = unit_begin(blockIdx.x, U, G);
    w.u_end = unit_begin(blockIdx.x + 1, U, G);
  } else {
    w.u = pair ? blockIdx.x / 2 : blockIdx.x;
    w.u_end = (int64_t)p.tiles_p * p.tiles_q;
  }
  return w;
}

__device__ __forceinline__ bool work_next(const GemmParams& p, WorkIter& w, int& tp, int& tq, int& kb, int& ke) {
  if (w.u >= w.u_end) return false;
  if (w.swap) {
    tp = (int)(w.u / w.kt);
    tq = 0;
    kb = (int)(w.u - (int64_t)tp * w.kt);
    const int64_t rest = w.u_end - w.u;
    ke = (int)(kb + rest < w.kt ? kb + rest : w.kt);
    w.u += ke - kb;
  } else {
    tile_coords(p, (int)w.u, tp, tq);
    kb = 0;
    ke = w.kt;
    w.u += w.pair ? gridDim.x / 2 : gridDim.x;
  }
  return true;
}

// Work of a CTA pair of a grouped GEMM: tiles of 256 weight rows by up to BN
// activation rows, numbered (group, weight tile, activation tile) with runs
// of up to group_p activation tiles fastest, so that tiles in flight share
// weights and activations in L2.  The tiles are dealt out in turn, and every
// role of either CTA counts through the same numbers.  That leaves the pairs
// unequal (ragged groups have short tiles), but measured better than what
// balances them: pairs that fetch the next tile when they get free (cluster
// launch control) took 2-15 % longer (32768 rows in 64 groups against 2048 x
// 5120: 218 us instead of 213; 16384 rows against 5120 x 1024: 87 instead of
// 76), odd rounds dealt backwards the same to 9 % longer, and contiguous
// shares of equal cost, which spread the pairs over all groups at once and
// their activations over more than the L2, 325 us.
struct GroupWork {
  const GroupTable* tab;
  int E, tiles_p, group_p;
  int total;                // tiles
  int round;
  int g, row0, rows, blk;   // current tile: group, first activation row, rows, first scale block
};

// Number of the pair's next tile, -1 at the end.
__device__ __forceinline__ int group_next_tile(GroupWork& w) {
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int tile = w.round++ * pairs + pair;
  return tile < w.total ? tile : -1;
}

template <int BN>
__device__ __forceinline__ bool group_work_next(GroupWork& w, int& tp, int& tq) {
  const int tile = group_next_tile(w);
  if (tile < 0) return false;
  const GroupTable& t = *w.tab;
  const int g = find_group(t.tiles, w.E, tile / w.tiles_p);
  const int local = tile - t.tiles[g] * w.tiles_p;
  const int cnt = t.tiles[g + 1] - t.tiles[g];
  const int per = w.group_p * w.tiles_p;
  const int q0 = local / per * w.group_p;
  const int run = min(cnt - q0, w.group_p);
  const int l2 = local - q0 * w.tiles_p;
  tp = l2 / run;
  tq = q0 + l2 - tp * run;
  w.g = g;
  w.row0 = t.off[g] + tq * BN;
  w.rows = min(t.off[g + 1] - w.row0, BN);
  w.blk = t.blk[g] + tq * (BN / 128);
  return true;
}

__device__ __forceinline__ int64_t row0_of(const GroupWork& w) { return w.row0; }
__device__ __forceinline__ int64_t row0_of(const WorkIter&) { return 0; }
__device__ __forceinline__ int rows_of(const GroupWork& w) { return w.rows; }
__device__ __forceinline__ int rows_of(const WorkIter&) { return 0; }

// One tile's operands: first code rows and first 128-row scale blocks of P
// and Q, and (grouped) activation rows that this CTA loads.
struct TileSrc {
  int p0, q0, pb, qb, rows;
};

// Segment of output column n, from the table the CTA copied to shared memory.
__device__ __forceinline__ int seg_index_smem(const int* ends, int n_seg, int64_t n) {
  int i = 0;
  while (i < n_seg - 1 && n >= ends[i]) ++i;
  return i;
}

__device__ __forceinline__ float seg_alpha_smem(const int* ends, const float* alphas, int n_seg, int64_t n) {
  return alphas[seg_index_smem(ends, n_seg, n)];
}

// Tagged partial words: FP32 bits in the low half, kFullTag in the high half
// once written; 0 = empty.  An aligned 64-bit store or load is single-copy
// atomic, so a reader that sees the tag sees the value.
constexpr uint32_t kFullTag = 1u;

__device__ __forceinline__ void st_full_word(uint64_t* p, uint32_t value_bits) {
  const uint64_t w = ((uint64_t)kFullTag << 32) | value_bits;
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(w) : "memory");
}

__device__ __forceinline__ void st_word(uint64_t* p, uint64_t w) {
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(w) : "memory");
}

// No "memory" clobber: the polls of one round are independent and may all be
// in flight together (volatile keeps each round's loads inside its loop).
__device__ __forceinline__ uint64_t ld_word(const uint64_t* p) {
  uint64_t w;
  asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(w) : "l"(p));
  return w;
}

// Byte offset of 16-byte chunk c of row r in a 128-row x 128-byte sub-tile
// stored with the 128B swizzle the output tensor map uses.
__device__ __forceinline__ uint32_t swz128(uint32_t r, uint32_t c) { return r * 128 + ((c ^ (r & 7)) << 4); }

template <bool GROUPED>
using GemmParamsOf = std::conditional_t<GROUPED, GroupedGemmParams, GemmParams>;

template <int BN, bool SWAP, bool OUT_F32, int QX = 0, bool MX = false, bool PAIR = false, bool GROUPED = false>
__global__ void __launch_bounds__(Cfg<BN, SWAP, QX, MX, PAIR, GROUPED>::kThreads,
                                  Cfg<BN, SWAP, QX, MX, PAIR, GROUPED>::kMinBlocks)
    nvfp4_gemm_kernel(const __grid_constant__ GemmParamsOf<GROUPED> p) {
  using C = Cfg<BN, SWAP, QX, MX, PAIR, GROUPED>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + C::kOffBar;
  const uint32_t bar_empty = bar_full + 8 * C::kStages;
  const uint32_t bar_acc_full = bar_empty + 8 * C::kStages;
  const uint32_t bar_acc_empty = bar_acc_full + 8;
  const uint32_t bar_drain = bar_acc_empty + 8;
  const uint32_t bar_sf = bar_drain + 8;                     // [kStages]
  const uint32_t bar_cp_drain = bar_sf + 8 * C::kStages;     // [kCopyWarps]
  const uint32_t bar_act = bar_cp_drain + 8 * C::kCopyWarps;  // [kActSteps] in-kernel activation ready
  int* seg_end_s = reinterpret_cast<int*>(smem + C::kOffSeg);
  float* seg_alpha_s = reinterpret_cast<float*>(smem + C::kOffSeg + 4 * NVFP4_MAX_SEGMENTS);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* epi_stop = abort_flag + 1;       // epilogue: the tile whose wait ran out
  constexpr int kNoTile = 0x7FFFFFFF;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // CTA pairs: rank in the pair; the even CTA (leader) issues the tcgen05 work
  const uint32_t prank = PAIR ? (cluster_ctarank() & 1u) : 0u;
  const bool leader = prank == 0;
  // the next kernel in the stream may launch now; it waits for this grid's
  // completion before touching anything this grid reads or writes
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_acc_full, 1);
    // CTA pairs: one arrival per epilogue warp of either CTA; otherwise one
    // per epilogue thread
    mbar_init(bar_acc_empty, PAIR ? 8 : 128);
    mbar_init(bar_drain, 1);
    for (int s = 0; s < C::kStages; ++s) mbar_init(bar_sf + 8 * s, C::kCopyWarps);
    for (int i = 0; i < C::kCopyWarps; ++i) mbar_init(bar_cp_drain + 8 * i, 1);
    for (int j = 0; j < C::kActSteps; ++j) mbar_init(bar_act + 8 * j, 128);
    *abort_flag = 0;
    *epi_stop = kNoTile;
    fence_barrier_init();
    prefetch_tmap(&p.tmap_p);
    prefetch_tmap(&p.tmap_q);
    if (!SWAP && p.tma_store) prefetch_tmap(&p.tmap_out);
    if (PAIR) {
      prefetch_tmap(&p.tmap_sfa);
      prefetch_tmap(&p.tmap_sfb);
    }
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + NVFP4_MAX_SEGMENTS) {
    seg_end_s[threadIdx.x - 64] = p.seg_end[threadIdx.x - 64];
    seg_alpha_s[threadIdx.x - 64] = p.seg_alpha[threadIdx.x - 64];
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      // both CTAs of the pair allocate together (the same columns in each)
      tmem_alloc_pair(smem_u32(tmem_holder), C::kTmemAlloc);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_holder), C::kTmemAlloc);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the even CTA's barriers are initialised before the odd CTA of its pair
  // can arrive on them
  if constexpr (PAIR) cluster_sync();
  const uint32_t tmem_base = *tmem_holder;
  // grouped: the offsets come from an earlier kernel, and every address
  // depends on them
  const GroupTable* tab = reinterpret_cast<const GroupTable*>(smem + C::kOffTab);
  if constexpr (GROUPED) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    load_groups<BN>(*reinterpret_cast<GroupTable*>(smem + C::kOffTab), p.offsets, p.E, p.M, p.err);
  }
  auto begin_work = [&]() {
    if constexpr (GROUPED) {
      GroupWork w;
      w.tab = tab;
      w.E = p.E;
      w.tiles_p = p.tiles_p;
      w.group_p = p.group_p;
      w.total = tab->tiles[p.E] * p.tiles_p;
      w.round = 0;
      w.g = w.row0 = w.rows = w.blk = 0;
      return w;
    } else {
      return work_begin(p, SWAP, PAIR);
    }
  };
  auto next_work = [&](auto& w, int& tp, int& tq, int& kb, int& ke) {
    if constexpr (GROUPED) {
      kb = 0;
      ke = p.kt;
      return group_work_next<BN>(w, tp, tq);
    } else {
      return work_next(p, w, tp, tq, kb, ke);
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // Programmatic dependent launch: this kernel may start while the
    // preceding kernel in the stream still runs, and that kernel may be
    // writing any of the inputs (the weight included).  Before
    // griddepcontrol.wait the weight tiles of the first kStages steps are
    // only prefetched into L2 (a hint that reads nothing into the CTA); every
    // load into shared memory comes after the wait.
    if (lane == 0) {
      const int kc = p.kc, rb_q = p.rb_q;
      uint32_t issued_mask = 0, last_parity = 0;   // for the drain on abort
      bool ok = true;
      // p0: this CTA's first row of P (CTA pairs: its 128-row half of the
      // 256-row tile); q0: the tile's first row of Q
      auto for_steps = [&](const auto& w0, int first, int count, auto&& fn) {
        int tp, tq, kb, ke, j = 0;
        auto w = w0;
        while (ok && j < first + count && next_work(w, tp, tq, kb, ke)) {
          TileSrc t;
          if constexpr (GROUPED) {
            // each CTA of the pair loads half of the MMA's columns
            t.rows = ((w.rows + 31) & ~31) / 2;
            t.p0 = w.g * (int)p.N + tp * 2 * kBM + (int)prank * kBM;
            t.pb = w.g * p.w_blocks + tp * 2 + (int)prank;
            t.q0 = w.row0 + (int)prank * t.rows;
            t.qb = w.blk;
          } else {
            t.p0 = PAIR ? tp * 2 * kBM + (int)prank * kBM : tp * kBM;
            t.pb = t.p0 >> 7;
            t.q0 = tq * BN;
            t.qb = t.q0 >> 7;
            t.rows = 0;
          }
          for (int k = kb; k < ke && j < first + count; ++k, ++j)
            if (j >= first) fn(j, t, k);
        }
      };
      // grouped: index of the box that holds the rows
      auto box_of = [](int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; };
      // grouped: 128-row scale blocks of the tile's activation rows
      auto sfb_blocks = [](const TileSrc& t) { return t.rows > 64 ? 2u : 1u; };
      auto nsfb_of = [&](const TileSrc& t) {
        int n = 0;
#pragma unroll
        for (int rb = 0; rb < C::kSfbBlocks; ++rb)
          if (t.qb + rb < rb_q) ++n;
        return n;
      };
      auto load_p = [&](int stage, const TileSrc& t, int k) {
        const int p0 = t.p0;
        const uint32_t fb = bar_full + 8 * stage;
        const int nch = min(C::kChunks, kc - C::kChunks * k);
        if constexpr (PAIR) {
          // into this CTA's shared memory, completing on the even CTA's barrier
          tma_load_2d_pair(sbase + C::kOffA + stage * C::kABytes, &p.tmap_p, k * C::kRowBytes, p0, fb);
          tma_load_2d_pair(sbase + C::kOffSfa + stage * C::kSfaBytes, &p.tmap_sfa, 0, t.pb * kc + C::kChunks * k, fb);
          return;
        }
        tma_load_2d(sbase + C::kOffA + stage * C::kABytes, &p.tmap_p, k * C::kRowBytes, p0, fb);
        size_t off = ((size_t)t.pb * kc + C::kChunks * k) * kSfChunk;
        if (!bounds_ok(off + (size_t)nch * kSfChunk <= p.sf_p_bytes, p.err)) off = 0;
        bulk_load(sbase + C::kOffSfa + stage * C::kSfaBytes, p.sf_p + off, (uint32_t)nch * kSfChunk, fb);
      };
      auto load_q = [&](int stage, const TileSrc& t, int k) {
        const int q0 = t.q0;
        const uint32_t fb = bar_full + 8 * stage;
        if constexpr (PAIR) {
          // this CTA's 128-row half of the weight tile (grouped: its half of
          // the activation rows), and the scales of all 256 rows (both CTAs
          // copy them into their own TMEM)
          if constexpr (GROUPED)
            tma_load_2d_pair(sbase + C::kOffB + stage * C::kBBytes, &p.tmap_q_box[box_of(t.rows)], k * C::kRowBytes, q0,
                             fb);
          else
            tma_load_2d_pair(sbase + C::kOffB + stage * C::kBBytes, &p.tmap_q, k * C::kRowBytes,
                             q0 + (int)prank * kBM, fb);
#pragma unroll
          for (int rb = 0; rb < C::kSfbBlocks; ++rb)
            if (!GROUPED || rb < sfb_blocks(t))
              tma_load_2d_pair(sbase + C::kOffSfb + stage * C::kSfbBytes + rb * C::kChunks * kSfChunk, &p.tmap_sfb, 0,
                             (t.qb + rb) * kc + C::kChunks * k, fb);
          return;
        }
        const uint32_t sf_bytes = (uint32_t)min(C::kChunks, kc - C::kChunks * k) * kSfChunk;
        const int nsfb = nsfb_of(t);
        tma_load_2d(sbase + C::kOffB + stage * C::kBBytes, &p.tmap_q, k * C::kRowBytes, q0, fb);
#pragma unroll
        for (int rb = 0; rb < C::kSfbBlocks; ++rb)
          if (rb < nsfb) {
            size_t off = ((size_t)(t.qb + rb) * kc + C::kChunks * k) * kSfChunk;
            if (!bounds_ok(off + sf_bytes <= p.sf_q_bytes, p.err)) off = 0;
            bulk_load(sbase + C::kOffSfb + stage * C::kSfbBytes + rb * C::kChunks * kSfChunk, p.sf_q + off, sf_bytes,
                      fb);
          }
      };
      auto expect = [&](int stage, const TileSrc& t, int k) {
        if constexpr (PAIR) {
          // the even CTA's barrier counts both CTAs' bytes (every box moves
          // its full size; rows past the tensor are zero-filled)
          const uint32_t sfb_bytes = GROUPED ? sfb_blocks(t) * C::kChunks * kSfChunk : C::kSfbBytes;
          const uint32_t q_bytes = GROUPED ? (16u << box_of(t.rows)) * C::kRowBytes : C::kBBytes;
          if (leader)
            mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * (C::kABytes + q_bytes + C::kSfaBytes + sfb_bytes));
          return;
        }
        const int nch = min(C::kChunks, kc - C::kChunks * k);
        const uint32_t sf_bytes = (uint32_t)nch * kSfChunk;
        mbar_arrive_expect_tx(bar_full + 8 * stage,
                              C::kABytes + C::kBBytes + sf_bytes * (1 + (C::kQx ? 0 : nsfb_of(t))));
      };
      if constexpr (GROUPED) {
        int stage = 0;
        uint32_t phase = 0;
        for_steps(begin_work(), 0, 1 << 30, [&](int, const TileSrc& t, int k) {
          if (!ok) return;
          if (!mbar_wait(bar_empty + 8 * stage, phase ^ 1, abort_flag, p.err, p.timeout_ns)) { ok = false; return; }
          expect(stage, t, k);
          load_p(stage, t, k);
          load_q(stage, t, k);
          issued_mask |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        });
      } else {
        const auto w0 = begin_work();
        // prologue: the first kStages stages are free
        int npro = 0;
        const bool w_static = p.w_static != 0;
        for_steps(w0, 0, C::kStages, [&](int j, const TileSrc& t, int k) {
          const int p0 = t.p0, q0 = t.q0;
          if (w_static) {
            // a weight declared read-only cannot be written by the preceding
            // kernel: load its first stages now
            expect(j, t, k);
            if (SWAP) load_p(j, t, k);
            else load_q(j, t, k);
            issued_mask |= 1u << j;
          } else {
            const uint32_t sf_bytes = (uint32_t)min(C::kChunks, kc - C::kChunks * k) * kSfChunk;
            if (SWAP) {
              tma_prefetch_l2_2d(&p.tmap_p, k * C::kRowBytes, p0);
              const size_t off = ((size_t)t.pb * kc + C::kChunks * k) * kSfChunk;
              if (bounds_ok(off + sf_bytes <= p.sf_p_bytes, p.err)) bulk_prefetch_l2(p.sf_p + off, sf_bytes);
            } else {
              tma_prefetch_l2_2d(&p.tmap_q, k * C::kRowBytes, PAIR ? q0 + (int)prank * kBM : q0);
            }
          }
          npro = j + 1;
        });
        if (SWAP) {
          // decode tiles stream each weight byte once: bring the rest of this
          // CTA's weight range into L2 now, so that HBM keeps streaming while
          // the preceding kernel finishes (a hint: it reads nothing into the CTA)
          for_steps(w0, C::kStages, 1 << 30, [&](int, const TileSrc& t, int k) {
            const uint32_t sf_bytes = (uint32_t)min(C::kChunks, kc - C::kChunks * k) * kSfChunk;
            tma_prefetch_l2_2d(&p.tmap_p, k * C::kRowBytes, t.p0);
            const size_t off = ((size_t)t.pb * kc + C::kChunks * k) * kSfChunk;
            if (bounds_ok(off + sf_bytes <= p.sf_p_bytes, p.err)) bulk_prefetch_l2(p.sf_p + off, sf_bytes);
          });
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
        for_steps(w0, 0, npro, [&](int j, const TileSrc& t, int k) {
          if (w_static) {
            if (SWAP) {
              if (!C::kQx) load_q(j, t, k);
            } else {
              load_p(j, t, k);
            }
          } else {
            expect(j, t, k);
            load_p(j, t, k);
            if (!C::kQx) load_q(j, t, k);
            issued_mask |= 1u << j;
          }
        });
        int stage = npro % C::kStages;
        uint32_t phase = npro == C::kStages ? 1u : 0u;
        if (npro == C::kStages) {
          for_steps(w0, npro, 1 << 30, [&](int j, const TileSrc& t, int k) {
            if (!ok) return;
            if (!mbar_wait(bar_empty + 8 * stage, phase ^ 1, abort_flag, p.err, p.timeout_ns)) { ok = false; return; }
            expect(stage, t, k);
            load_p(stage, t, k);
            if (!C::kQx) load_q(stage, t, k);
            last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == C::kStages) { stage = 0; phase ^= 1; }
          });
        }
      }
      // let every issued copy land before the CTA exits, whichever role may
      // have given up (when nothing did, the last load of each stage has
      // already landed and each wait returns at once).  The odd CTA of a
      // pair cannot see its loads complete (they count on the even CTA's
      // barrier): it waits until the MMAs have consumed each stage instead,
      // and the cluster-wide barrier before exit keeps it until the even CTA
      // has drained.
      for (int s = 0; s < C::kStages; ++s)
        if (issued_mask & (1u << s)) {
          volatile int never = 0;
          if (leader) (void)mbar_wait(bar_full + 8 * s, (last_parity >> s) & 1, &never, p.err, p.drain_ns);
          else (void)mbar_wait(bar_empty + 8 * s, (last_parity >> s) & 1, &never, p.err, p.drain_ns);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp follows the pipeline; lane 0 issues every MMA.  The copy
    // warps waited for each stage's data and moved its scales into TMEM.
    constexpr uint32_t idesc_full = MX ? idesc_mxf4(C::kMmaM, BN) : idesc_nvf4(C::kMmaM, BN);
    // Descriptors of stage 0, k-block 0; later stages and k-blocks only move
    // the 14-bit start-address field (address >> 4), which never carries.
    const uint64_t a_desc0 = smem_desc(sbase + C::kOffA, 16, C::kSbo, C::kSwizzleLayout);
    const uint64_t b_desc0 = smem_desc(sbase + (C::kQx ? C::kOffAct : C::kOffB), 16, C::kSbo, C::kSwizzleLayout);
    const uint32_t sf_t0 = tmem_base + C::kSfBase;
    int stage = 0, region = 0, lstep = 0;    // lstep: steps of this CTA so far
    uint32_t phase = 0, acc_phase = 0, acc_buf = 0;
    bool ok = true;
    auto w = begin_work();
    int tp, tq, kb0, ke0;
    // CTA pairs: only the even CTA issues (for both)
    while (ok && leader && next_work(w, tp, tq, kb0, ke0)) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_acc_empty, acc_phase ^ 1, abort_flag, p.err, p.timeout_ns))) break;
      tc_fence_after();
      uint32_t idesc = idesc_full;
      // as many columns as the tile has rows; each CTA of a pair holds half
      // of them, in whole 8-row groups
      if constexpr (GROUPED) idesc = idesc_nvf4(C::kMmaM, (w.rows + 31) & ~31);
      const uint32_t acc = tmem_base + (acc_buf ? C::kAcc1Col : 0);
      for (int k = kb0; k < ke0; ++k) {
        if (C::kQx && lstep >= C::kActSteps) {     // the host sizes the grid so this cannot happen
          atomicCAS(p.err, 0u, kErrBounds);
          *abort_flag = 1;
          ok = false;
          break;
        }
        const bool there = mbar_wait(bar_sf + 8 * stage, phase, abort_flag, p.err, p.timeout_ns);
        tc_fence_after();
        if (lane == 0 && there) {
          const uint32_t sfa_t = sf_t0 + region * C::kSfStageCols;
          const uint32_t sfb_t = sfa_t + C::kSfaCols;
          const uint64_t ad = a_desc0 + (uint64_t)((stage * C::kABytes) >> 4);
          const uint64_t bd = b_desc0 + (uint64_t)(((C::kQx ? lstep * C::kActCodeBytes : stage * C::kBBytes)) >> 4);
          const uint32_t acc_in = k != kb0 ? 1u : 0u;
          // MMA kb reads chunk kb (NVFP4, 4 scales each) or half of chunk
          // kb / 2 (MXFP4: scale bytes 0-1 or 2-3 of each TMEM column,
          // selected by the descriptor's scale-factor ids)
          const int nkb = min(C::kKB, p.kmma - C::kKB * k);
          auto mma = [&](int kb) {
            const int c = MX ? kb >> 1 : kb;
            const uint32_t id = MX ? (uint32_t)(kb & 1) * 2u : 0u;
            if constexpr (PAIR)
              tc_mma_block_scaled_pair<MX>(acc, ad + (uint64_t)(kb * 2), bd + (uint64_t)(kb * 2),
                                           idesc | (id << 29) | (id << 4), sfa_t + c * 4,
                                           sfb_t + c * 4 * C::kSfbBlocks, (acc_in | kb) != 0 ? 1u : 0u);
            else
              tc_mma_block_scaled<MX>(acc, ad + (uint64_t)(kb * 2), bd + (uint64_t)(kb * 2),
                                      idesc | (id << 29) | (id << 4), sfa_t + c * 4, sfb_t + c * 4 * C::kSfbBlocks,
                                      (acc_in | kb) != 0 ? 1u : 0u);
          };
          if (nkb == C::kKB) {
#pragma unroll
            for (int kb = 0; kb < C::kKB; ++kb) mma(kb);
          } else {
            for (int kb = 0; kb < nkb; ++kb) mma(kb);
          }
          // the stage is free in both CTAs of a pair
          if constexpr (PAIR) tc_commit_pair_both(bar_empty + 8 * stage);
          else tc_commit(bar_empty + 8 * stage);
        }
        ok = __all_sync(0xFFFFFFFFu, there);     // the lanes stop together
        if (!ok) break;
        if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        if (++region == C::kSfRegions) region = 0;
        ++lstep;
      }
      if (!ok) break;
      if (lane == 0) {
        if constexpr (PAIR) tc_commit_pair_both(bar_acc_full);
        else tc_commit(bar_acc_full);
      }
      __syncwarp();
      acc_phase ^= 1;
      acc_buf ^= 1;
    }
    if (lane == 0 && leader) {
      // every MMA and scale copy issued by this thread has completed once
      // this commit arrives
      if constexpr (PAIR) tc_commit_pair(bar_drain);
      else tc_commit(bar_drain);
      volatile int never = 0;
      (void)mbar_wait(bar_drain, 0, &never, p.err, p.drain_ns);
    }
    __syncwarp();
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue
    const int sp = warp & 3;                 // TMEM subpartition of this warp
    const int row = sp * 32 + lane;          // accumulator lane = tile row of P
    const int et = threadIdx.x - 64;         // epilogue thread index 0..127
    const uint32_t taddr = tmem_base + ((uint32_t)(sp * 32) << 16);
    const int64_t M = p.M, N = p.N;
    const int n_seg = p.n_seg;
    const bool tma_store = !SWAP && p.tma_store;
    uint32_t acc_phase = 0, acc_buf = 0;
    uint32_t out_buf = 0;                    // next staging buffer (TMA store path)
    int tile_no = 0;                         // tiles of this CTA so far
    auto w = begin_work();
    const int64_t U = (int64_t)p.tiles_p * p.kt, G = gridDim.x;
    int tp, tq, kb0, ke0;
    bool first_item = true;
    if constexpr (C::kQx) {
      // ---------------------------------------------- in-kernel activation
      // Quantize the rows of X for every K-step this CTA computes, with the
      // same per-block arithmetic as the quantize kernel, into the MMA's
      // operand layout: codes of step j at kOffAct + j * BN * 128 (row m at
      // m * 128, 16-byte chunks 128B-swizzled), scales of step j at
      // kOffActSf + j * 2048 (the 512-byte chunk of K-block kb holds row m's
      // four scales at m * 16).  Rows [M, BN) and K past the end stay zero.
      constexpr bool kF32 = QX == 2;
      constexpr int kEsz = kF32 ? 4 : 2;
      // the K-steps of this CTA, in the order every role walks them
      int ks[C::kActSteps];
      int nsteps = 0;
      {
        WorkIter wq = work_begin(p, SWAP, PAIR);
        int a, b2, c0, c1;
        while (work_next(p, wq, a, b2, c0, c1))
          for (int k = c0; k < c1 && nsteps < C::kActSteps; ++k) ks[nsteps++] = k;
      }
      const int64_t K = p.K;
      const uint8_t* xb = reinterpret_cast<const uint8_t*>(p.x);
      // A thread owns (row, block) pairs et, et + 128, ... (one pair when
      // M <= 8) and handles them one after the other.  Per pair, windows of
      // kWin steps: the next window's loads are in flight while the current
      // one is quantized (all its blocks together, for instruction-level
      // parallelism: four warps alone cannot hide latency by switching).  A
      // thread publishes step j (its barrier, 128 arrivals) after its last
      // pair's block of step j is stored, so the MMAs can start early.
      // Two-step windows: the first MMAs wait for less quantizing (decode
      // step 12.7 us against 13.2 with four-step windows, 12.8 with one)
      constexpr int kWin = 2;
      const int npairs = (int)M * 16;
      const int nq = et < npairs ? (npairs - 1 - et) / 128 + 1 : 0;   // pairs of this thread
      asm volatile("griddepcontrol.wait;" ::: "memory");      // X is written by the previous kernel
      auto load_window = [&](int pair, int j0, Block16<kF32> (&B)[kWin]) {
        const int m = pair >> 4, bq = pair & 15;
#pragma unroll
        for (int u = 0; u < kWin; ++u) {
          const int jj = j0 + u;
          const int64_t e = (int64_t)(jj < nsteps ? ks[jj] : 0) * 256 + bq * 16;
          if (jj < nsteps && e < K) {
            if (bounds_ok((uint64_t)((int64_t)m * K + e + 16) * kEsz <= p.x_bytes, p.err))
              load_block_at<kF32>(xb + ((int64_t)m * K + e) * kEsz, B[u]);
            else
              B[u] = Block16<kF32>{};
          }
        }
      };
      Block16<kF32> Bc[kWin], Bn[kWin];
      if (nq > 0) load_window(et, 0, Bc);
      float* rtab = reinterpret_cast<float*>(smem + C::kOffRtab);
      rtab[et] = recip_entry(p.x_gs, (uint32_t)et);
      rtab[et + 128] = recip_entry(p.x_gs, (uint32_t)et + 128);
      for (int i = et; i < C::kActBytes / 16; i += 128)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(sbase + C::kOffAct + 16 * i), "r"(0) : "memory");
      named_bar_sync(kEpiBar, 128);                // zeros and rtab are in place
      if (nq == 0)
        for (int jj = 0; jj < nsteps; ++jj) mbar_arrive(bar_act + 8 * jj);
      for (int q = 0; q < nq; ++q) {
        const int pair = et + 128 * q;
        const int m = pair >> 4, bq = pair & 15;
        const bool last = q == nq - 1;
        for (int j0 = 0; j0 < nsteps; j0 += kWin) {
          // prefetch: the next window of this pair, or the first of the next pair
          if (j0 + kWin < nsteps) load_window(pair, j0 + kWin, Bn);
          else if (!last) load_window(pair + 128, 0, Bn);
#pragma unroll
          for (int u = 0; u < kWin; ++u) {
            const int jj = j0 + u;
            const int64_t e = (int64_t)(jj < nsteps ? ks[jj] : 0) * 256 + bq * 16;
            if (jj < nsteps && e < K) {
              uint32_t lo, hi;
              const uint32_t sc = quantize_block<kF32>(Bc[u], p.x_gs, rtab, lo, hi);
              // byte bq * 8 of row m: 16-byte chunk bq / 2, swizzled with m % 8
              *reinterpret_cast<uint2*>(smem + C::kOffAct + jj * C::kActCodeBytes + m * 128 +
                                        ((((bq >> 1) ^ (m & 7))) << 4) + (bq & 1) * 8) = make_uint2(lo, hi);
              smem[C::kOffActSf + jj * C::kActSfBytes + (bq >> 2) * kSfChunk + m * 16 + (bq & 3)] = (uint8_t)sc;
            }
          }
          if (last) {
            fence_proxy_async_smem();              // generic-proxy writes -> tcgen05 reads
#pragma unroll
            for (int u = 0; u < kWin; ++u)
              if (j0 + u < nsteps) mbar_arrive(bar_act + 8 * (j0 + u));
          }
#pragma unroll
          for (int u = 0; u < kWin; ++u) Bc[u] = Bn[u];
        }
      }
    }
    // hand the accumulator back to the MMA warp (CTA pairs: to the even
    // CTA's MMA warp, one arrival per warp of either CTA)
    auto release_acc = [&]() {
      tc_fence_before();
      if constexpr (PAIR) {
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(bar_acc_empty);
          else mbar_arrive_cluster(map_to_rank(bar_acc_empty, 0));
        }
      } else {
        mbar_arrive(bar_acc_empty);
      }
    };
    while (next_work(w, tp, tq, kb0, ke0)) {
      // CTA pairs: this CTA's rows are its 128-row half of the 256-row tile
      const int64_t p0 = PAIR ? (int64_t)tp * 2 * kBM + (int64_t)prank * kBM : (int64_t)tp * kBM;
      const int64_t q0 = GROUPED ? row0_of(w) : (int64_t)tq * BN;
      float g_alpha = 0.0f;
      if constexpr (GROUPED) {
        g_alpha = (float)(1.0 / ((double)p.ga[w.g] * (double)p.gw[w.g]));
      }
      // A warp goes on as a whole or not at all.  Where the four warps share
      // staging buffers they also stop together, at the end of the first tile
      // for which a wait ran out in any of them: that warp writes the tile's
      // number before the tile's first barrier and goes through its barriers
      // with the others (what the tile stores is then not reliable), and
      // behind the last of them all read that number, or a later one, which
      // is not for this tile.  (Nothing on the way of a tile: agreeing by a
      // barrier before the TMEM loads took 107 instead of 101 us for 16000
      // rows in 64 groups against 5120 x 1024, making each store depend on
      // the number 123 instead of 114 for FP32 against 4096 x 256.)
      const bool there = __all_sync(0xFFFFFFFFu, mbar_wait(bar_acc_full, acc_phase, abort_flag, p.err, p.timeout_ns));
      ++tile_no;
      if (!there) {
        if (!(GROUPED || tma_store)) break;
        *epi_stop = tile_no;
      }
      tc_fence_after();
      if constexpr (GROUPED && PAIR) {
        // Lane = weight row = output column n, accumulator column = activation
        // row: the tile leaves transposed.  64 rows at a time (FP32 output: 32)
        // go through a 16 KB buffer of 128-byte-wide, 128B-swizzled sub-tiles
        // [rows][64 or 32 columns] and out as TMA stores, which clip at N; the
        // rows of a slot that runs past the group are stored one by one
        // instead, so no row of a neighbour is touched.  bf16 is transposed on
        // the way in (fragment loads from TMEM, stmatrix.trans): element
        // stores and loads cost 2900 cycles a slot, more than the MMAs of a
        // tile with K = 1024.
        const uint32_t tacc = taddr + (acc_buf ? C::kAcc1Col : 0);
        auto slot_col = [&](int slot) -> int {
          return C::kOverlapAcc && acc_buf == 0 ? ((slot + 4 - C::kSharedSlots) & 3) * 64 : slot * 64;
        };
        constexpr int kEsz = OUT_F32 ? 4 : 2;
        constexpr int kRows = OUT_F32 ? 32 : 64;      // activation rows of a buffer
        constexpr int kSubCols = 128 / kEsz;          // output columns of a sub-tile
        constexpr int kSubBytes = kRows * 128;
        const bool vec = p.tma_store != 0;            // output rows start on 16-byte boundaries
        // the next buffer, once its last store has read it and every thread
        // is done with it
        auto next_buf = [&]() {
          if (C::kOutBufs == 2) out_buf ^= 1;
          if (et == 0) bulk_wait_group_read<C::kOutBufs - 1>();
          named_bar_sync(kEpiBar, 128);
          return sbase + C::kOffOut + out_buf * kStageOutBytes;
        };
        auto flush = [&](uint32_t buf, int col) {     // a filled buffer, rows col ... of the tile
          const bool whole = vec && col + kRows <= w.rows;
          if (whole) fence_proxy_async_smem();
          named_bar_sync(kEpiBar, 128);
          if (whole) {
            if (et == 0) {
#pragma unroll
              for (int sub = 0; sub < 128 / kSubCols; ++sub)
                if (p0 + sub * kSubCols < N)
                  tma_store_2d(&p.tmap_out, buf + sub * kSubBytes, (int32_t)(p0 + sub * kSubCols), (int32_t)(q0 + col));
              bulk_commit_group();
            }
            return;
          }
          // an empty bulk group: the wait in next_buf counts one a buffer
          if (et == 0) bulk_commit_group();
          // 16-byte pieces of the rows that the group has.  (One at a time: four
          // in flight took registers from the slots that wait, and every tile
          // paid for it, 136 instead of 108 us for 64 ragged groups of 250 rows
          // against 5120 x 1024.)
          constexpr int kPieces = 8 * 128 / kSubCols;           // of a row
          const int n_ids = min(kRows, w.rows - col) * kPieces;
#pragma unroll 1
          for (int id = et; id < n_ids; id += 128) {
            const int r = id / kPieces;
            const int64_t n = p0 + id % kPieces * (16 / kEsz);
            if (n >= N) continue;
            const int64_t o = (q0 + col + r) * N + n;
            uint32_t v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(buf + id / 8 % (kPieces / 8) * kSubBytes + swz128(r, id & 7))
                         : "memory");
            if (vec && n + 16 / kEsz <= N) {
              if (bounds_ok((uint64_t)(o + 16 / kEsz) <= p.out_elems, p.err))
                *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p.out) + o * kEsz) =
                    make_uint4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
              for (int e = 0; e < 16 / kEsz; ++e)
                if (n + e < N && bounds_ok((uint64_t)(o + e) < p.out_elems, p.err)) {
                  if constexpr (OUT_F32) reinterpret_cast<uint32_t*>(p.out)[o + e] = v[e];
                  else reinterpret_cast<uint16_t*>(p.out)[o + e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
                }
            }
          }
        };
        if constexpr (!OUT_F32) {
          // v[16 h + 2 j + i]: lanes 16 h + 8 i ... of the warp, rows 8 j ...
          auto load_slot = [&](int col, uint32_t (&v)[32]) {
            if (col >= w.rows) return;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t r[32];
              tmem_ld_16x256b_x8(tacc + ((uint32_t)(16 * h) << 16) + col, r);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                v[h * 16 + i] = pack_bf16x2(__fmul_rn(__uint_as_float(r[2 * i]), g_alpha),
                                            __fmul_rn(__uint_as_float(r[2 * i + 1]), g_alpha));
            }
          };
          // this lane's stmatrix row: activation row lane % 8, output columns
          // 8 (lane / 8) ... of the warp's 32
          const uint32_t st_off = (uint32_t)(sp >> 1) * kSubBytes + swz128(lane & 7, (sp & 1) * 4 + (lane >> 3));
          auto store_slot = [&](int col, const uint32_t (&v)[32]) {
            if (col >= w.rows) return;
            const uint32_t buf = next_buf();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              stmatrix_x4_trans(buf + st_off + j * 1024, v[2 * j], v[2 * j + 1], v[16 + 2 * j], v[16 + 2 * j + 1]);
            flush(buf, col);
          };
          // slots in drain order: the columns that the next accumulator shares
          // go to registers, TMEM goes back, and only then does anything wait
          // for a staging buffer
          static_assert(C::kSharedSlots == (BN == 256 ? 3 : 0), "slots drained before the accumulator goes back");
          uint32_t v0[32], v1[32];
          if constexpr (BN == 256) {
            uint32_t v2[32];
            load_slot(slot_col(0), v0);
            load_slot(slot_col(1), v1);
            load_slot(slot_col(2), v2);
            release_acc();
            store_slot(slot_col(0), v0);
            load_slot(slot_col(3), v0);
            store_slot(slot_col(1), v1);
            store_slot(slot_col(2), v2);
            store_slot(slot_col(3), v0);
          } else {
            release_acc();                            // two accumulators side by side: the next tile's is free
            load_slot(0, v0);
            load_slot(64, v1);
            store_slot(0, v0);
            store_slot(64, v1);
          }
        } else {
          if (!C::kOverlapAcc) release_acc();
#pragma unroll 1
          for (int cc = 0; cc < BN / 32; ++cc) {
            const int col = slot_col(cc / 2) + (cc & 1) * 32;
            const bool has = col < w.rows;
            uint32_t r[32];
            __syncwarp();
            if (has) {
              tmem_ld_32x32b_x32(tacc + col, r);
              tmem_ld_wait();
            }
            if (C::kOverlapAcc && cc == 2 * C::kSharedSlots - 1) release_acc();
            if (!has) continue;
            const uint32_t buf = next_buf();
#pragma unroll
            for (int i = 0; i < 32; ++i)              // the warp's 32 columns are sub-tile sp
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(buf + sp * kSubBytes + swz128(i, lane >> 2) + (lane & 3) * 4),
                           "f"(__fmul_rn(__uint_as_float(r[i]), g_alpha))
                           : "memory");
            flush(buf, col);
          }
        }
      } else if constexpr (!SWAP) {
        const int64_t m = p0 + row;
        // 64-column slots are drained starting with the columns this buffer
        // shares with the other one; TMEM is handed back right after them.
        const uint32_t tacc = taddr + (acc_buf ? C::kAcc1Col : 0);
        auto slot_col = [&](int slot) -> int {
          return C::kOverlapAcc && acc_buf == 0 ? ((slot + 4 - C::kSharedSlots) & 3) * 64 : slot * 64;
        };
        if constexpr (!OUT_F32) {
          // drain the whole accumulator row into registers (bf16 pairs)
          uint32_t packed[BN / 2];
#pragma unroll
          for (int slot = 0; slot < BN / 64; ++slot) {
            const int col = slot_col(slot);
            uint32_t r0[32], r1[32];
            tmem_ld_32x32b_x32(tacc + col, r0);
            tmem_ld_32x32b_x32(tacc + col + 32, r1);
            tmem_ld_wait();
            if (slot == C::kSharedSlots - 1 && C::kOverlapAcc) release_acc();
            const int64_t n0 = q0 + col;
            // one scale for the whole 64-column slot unless a segment
            // boundary falls inside it
            int seg_lo = 0, seg_hi = 0;
            if (n_seg > 1) {
              seg_lo = seg_index_smem(seg_end_s, n_seg, n0);
              seg_hi = seg_index_smem(seg_end_s, n_seg, n0 + 63 < N ? n0 + 63 : N - 1);
            }
            if (seg_lo == seg_hi) {
              const float a = seg_alpha_s[seg_lo];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                packed[slot * 32 + i] = pack_bf16x2(__fmul_rn(__uint_as_float(r0[2 * i]), a),
                                                    __fmul_rn(__uint_as_float(r0[2 * i + 1]), a));
                packed[slot * 32 + 16 + i] = pack_bf16x2(__fmul_rn(__uint_as_float(r1[2 * i]), a),
                                                         __fmul_rn(__uint_as_float(r1[2 * i + 1]), a));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                packed[slot * 32 + i] =
                    pack_bf16x2(__fmul_rn(__uint_as_float(r0[2 * i]),
                                          seg_alpha_smem(seg_end_s, seg_alpha_s, n_seg, n0 + 2 * i)),
                                __fmul_rn(__uint_as_float(r0[2 * i + 1]),
                                          seg_alpha_smem(seg_end_s, seg_alpha_s, n_seg, n0 + 2 * i + 1)));
                packed[slot * 32 + 16 + i] =
                    pack_bf16x2(__fmul_rn(__uint_as_float(r1[2 * i]),
                                          seg_alpha_smem(seg_end_s, seg_alpha_s, n_seg, n0 + 32 + 2 * i)),
                                __fmul_rn(__uint_as_float(r1[2 * i + 1]),
                                          seg_alpha_smem(seg_end_s, seg_alpha_s, n_seg, n0 + 33 + 2 * i)));
              }
            }
          }
          if (!C::kOverlapAcc) release_acc();
          if (tma_store) {
            // 64-column sub-tiles through two 16 KB swizzled staging buffers
#pragma unroll
            for (int sub = 0; sub < BN / 64; ++sub) {
              // sub-tiles wholly past N are skipped outright (uniform across
              // the epilogue), so every buffer written is one whose last
              // store has been committed and waited for
              const int col = slot_col(sub);
              if (q0 + col >= N) continue;
              const uint32_t buf = sbase + C::kOffOut + out_buf * kStageOutBytes;
              if (et == 0) bulk_wait_group_read<1>();          // the store that used buf has read it
              named_bar_sync(kEpiBar, 128);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint32_t* v = &packed[sub * 32 + c * 4];
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + swz128(row, c)), "r"(v[0]),
                             "r"(v[1]), "r"(v[2]), "r"(v[3])
                             : "memory");
              }
              fence_proxy_async_smem();
              named_bar_sync(kEpiBar, 128);
              if (et == 0) {
                tma_store_2d(&p.tmap_out, buf, (int32_t)(q0 + col), (int32_t)p0);
                bulk_commit_group();
              }
              out_buf ^= 1;
            }
          } else if (m < M) {
            __nv_bfloat16* orow = reinterpret_cast<__nv_bfloat16*>(p.out) + m * N;
#pragma unroll
            for (int c = 0; c < BN / 8; ++c) {
              const int64_t n = q0 + slot_col(c / 8) + (c % 8) * 8;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (n + e < N && bounds_ok((uint64_t)(m * N + n + e) < p.out_elems, p.err))
                  reinterpret_cast<uint16_t*>(orow)[n + e] = (uint16_t)(packed[4 * c + e / 2] >> (16 * (e & 1)));
            }
          }
        } else {
          // FP32 output: 32-column chunks in slot order; TMEM is released once
          // the shared columns (the first slot) are out
#pragma unroll 1
          for (int cc = 0; cc < BN / 32; ++cc) {
            const int c = slot_col(cc / 2) / 32 + (cc & 1);
            uint32_t r[32];
            __syncwarp();
            tmem_ld_32x32b_x32(tacc + c * 32, r);
            tmem_ld_wait();
            if (cc == 2 * C::kSharedSlots - 1 && C::kOverlapAcc) release_acc();
            const int64_t n0 = q0 + c * 32;
            int seg_lo = 0, seg_hi = 0;
            if (n_seg > 1) {
              seg_lo = seg_index_smem(seg_end_s, n_seg, n0);
              seg_hi = seg_index_smem(seg_end_s, n_seg, n0 + 31 < N ? n0 + 31 : N - 1);
            }
            if (seg_lo == seg_hi) {
              const float a = seg_alpha_s[seg_lo];
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__fmul_rn(__uint_as_float(r[i]), a));
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                r[i] = __float_as_uint(
                    __fmul_rn(__uint_as_float(r[i]), seg_alpha_smem(seg_end_s, seg_alpha_s, n_seg, n0 + i)));
            }
            if (tma_store && q0 + c * 32 < N) {
              const uint32_t buf = sbase + C::kOffOut + out_buf * kStageOutBytes;
              if (et == 0) bulk_wait_group_read<1>();
              named_bar_sync(kEpiBar, 128);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + swz128(row, j)),
                             "r"(r[4 * j]), "r"(r[4 * j + 1]), "r"(r[4 * j + 2]), "r"(r[4 * j + 3])
                             : "memory");
              fence_proxy_async_smem();
              named_bar_sync(kEpiBar, 128);
              if (et == 0) {
                tma_store_2d(&p.tmap_out, buf, (int32_t)(q0 + c * 32), (int32_t)p0);
                bulk_commit_group();
              }
              out_buf ^= 1;
            } else if (!tma_store && m < M) {
              float* orow = reinterpret_cast<float*>(p.out) + m * N;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int64_t n = q0 + c * 32 + i;
                if (n < N && bounds_ok((uint64_t)(m * N + n) < p.out_elems, p.err)) orow[n] = __uint_as_float(r[i]);
              }
            }
          }
          if (!C::kOverlapAcc) release_acc();
        }
      } else {
        // swap: lane = weight row = output column n; accumulator column =
        // activation row.  The whole accumulator row goes to registers, then
        // TMEM is handed back.
        const int64_t n = p0 + row;
        const float alpha = seg_alpha_smem(seg_end_s, seg_alpha_s, n_seg, n);
        constexpr int kCols = BN < 32 ? BN : 32;
        uint32_t r[(BN + 31) / 32][kCols];
#pragma unroll
        for (int c = 0; c < (BN + 31) / 32; ++c) {
          if constexpr (BN >= 32) {
            tmem_ld_32x32b_x32(taddr + c * 32, r[c]);
          } else {
            uint32_t r8[8];
#pragma unroll
            for (int j = 0; j < BN / 8; ++j) {
              tmem_ld_32x32b_x8(taddr + j * 8, r8);
#pragma unroll
              for (int i = 0; i < 8; ++i) r[0][j * 8 + i] = r8[i];
            }
          }
        }
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(bar_acc_empty);
        auto store_out = [&](int64_t mm, float v) {
          if (!bounds_ok((uint64_t)(mm * N + n) < p.out_elems, p.err)) return;
          if constexpr (OUT_F32) reinterpret_cast<float*>(p.out)[mm * N + n] = v;
          else reinterpret_cast<__nv_bfloat16*>(p.out)[mm * N + n] = __float2bfloat16_rn(v);
        };
        const int64_t tile_u0 = (int64_t)tp * p.kt;
        const int64_t c_first = cta_of_unit(tile_u0, U, G);
        const int64_t c_last = cta_of_unit(tile_u0 + p.kt - 1, U, G);
        if (c_first == c_last) {
          // the whole K range of this tile ran here
          if (n < N) {
#pragma unroll
            for (int c = 0; c < (BN + 31) / 32; ++c)
#pragma unroll
              for (int i = 0; i < kCols; ++i) {
                const int64_t mm = q0 + c * 32 + i;
                if (mm < M) store_out(mm, __fmul_rn(__uint_as_float(r[c][i]), alpha));
              }
          }
        } else {
          // split tile.  The CTA that holds the tile's first K steps (its last
          // work item, so it finishes last) adds the tile up in CTA (= K)
          // order, its own partial from registers.  Every other contributor
          // writes its partial to its slot (2c for CTA c's first item, 2c + 1
          // for its last) as 64-bit words that carry the FP32 value in the low
          // half and a "full" tag in the high half: one single-copy-atomic
          // store per value, so no fence or counter is needed.  The adder
          // polls each word until it is full and clears it for the next
          // launch.
          if ((int64_t)blockIdx.x != c_first) {
            const int64_t part0 = (2 * (int64_t)blockIdx.x + (first_item ? 0 : 1)) * BN * kBM + row;
            uint64_t* part = p.ws + part0;
#pragma unroll
            for (int c = 0; c < (BN + 31) / 32; ++c)
#pragma unroll
              for (int i = 0; i < kCols; ++i) {
                const int mm = c * 32 + i;
                if (q0 + mm < M && bounds_ok((uint64_t)(part0 + (int64_t)mm * kBM) < p.ws_words, p.err))
                  st_full_word(part + (int64_t)mm * kBM, r[c][i]);
              }
          } else {
            float sum[(BN + 31) / 32][kCols];
#pragma unroll
            for (int cb = 0; cb < (BN + 31) / 32; ++cb)
#pragma unroll
              for (int i = 0; i < kCols; ++i) sum[cb][i] = __uint_as_float(r[cb][i]);
            bool ok_all = true;
            for (int64_t c = c_first + 1; c <= c_last && ok_all; ++c) {
              const int64_t slot = 2 * c + (unit_begin(c, U, G) >= tile_u0 ? 0 : 1);
              // the slot's last word is inside the workspace (debug build)
              if (!bounds_ok((uint64_t)((slot + 1) * BN * kBM) <= p.ws_words, p.err)) {
                ok_all = false;
                break;
              }
              uint64_t* src = p.ws + slot * BN * kBM + row;
              // one round polls every word of a 32-column chunk at once
#pragma unroll
              for (int cb = 0; cb < (BN + 31) / 32; ++cb) {
                uint64_t v[kCols];
                const uint64_t t0 = globaltimer_ns();
                while (true) {
#pragma unroll
                  for (int i = 0; i < kCols; ++i) {
                    const int mm = cb * 32 + i;
                    v[i] = q0 + mm < M ? ld_word(src + (int64_t)mm * kBM) : (uint64_t)kFullTag << 32;
                  }
                  uint32_t all = p.test_stall ? 0u : 1u;
#pragma unroll
                  for (int i = 0; i < kCols; ++i) all &= (uint32_t)((v[i] >> 32) == kFullTag);
                  if (all) break;
                  if (globaltimer_ns() - t0 > p.timeout_ns) {
                    atomicCAS(p.err, 0u, kErrTimeout);
                    ok_all = false;
                    break;
                  }
                }
                if (!ok_all) break;
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                  const int mm = cb * 32 + i;
                  sum[cb][i] = __fadd_rn(sum[cb][i], __uint_as_float((uint32_t)v[i]));
                  if (q0 + mm < M) st_word(src + (int64_t)mm * kBM, 0ull);     // empty again
                }
              }
            }
            if (n < N && ok_all) {
#pragma unroll
              for (int cb = 0; cb < (BN + 31) / 32; ++cb)
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                  const int64_t mm = q0 + cb * 32 + i;
                  if (mm < M) store_out(mm, __fmul_rn(sum[cb][i], alpha));
                }
            }
          }
        }
      }
      if ((GROUPED || tma_store) && *epi_stop <= tile_no) break;
      acc_phase ^= 1;
      acc_buf ^= 1;
      first_item = false;
    }
    if (tma_store && et == 0) bulk_wait_group<0>();   // stores done before the CTA's smem goes away
  } else {
    // ------------------------------------------------------------ scale copies
    // warp 6 copies P's scale chunks of each stage into TMEM, warp 7 + rb the
    // chunks of Q's 128-row block rb; each then commits to the stage's
    // scales-ready barrier (kCopyWarps arrivals).  A TMEM scale region is
    // rewritten only once the MMAs that read it last have completed.
    const bool copy_p = warp == 6;
    const int rbq = warp - 7;                   // Q block of this warp
    if (lane == 0 && leader) {                  // CTA pairs: the even CTA copies for both
      const uint64_t desc0 =
          smem_desc(sbase + (copy_p ? C::kOffSfa : (C::kQx ? C::kOffActSf : C::kOffSfb)), 16, 128, 0);
      const uint32_t sf_t0 = tmem_base + C::kSfBase;
      const int kc = p.kc;
      int stage = 0, region = 0;
      int64_t step = 0;                         // pipeline steps issued so far
      uint32_t phase = 0;
      bool ok = true;
      auto w = begin_work();
      int tp, tq, kb0, ke0;
      while (ok && next_work(w, tp, tq, kb0, ke0)) {
        for (int k = kb0; k < ke0; ++k) {
          if (C::kQx && step >= C::kActSteps) { ok = false; break; }
          // in-kernel activation: this step's scales are written by the epilogue warps
          if (C::kQx && !copy_p && !mbar_wait(bar_act + 8 * (int)step, 0, abort_flag, p.err, p.timeout_ns)) {
            ok = false;
            break;
          }
          if (!mbar_wait(bar_full + 8 * stage, phase, abort_flag, p.err, p.timeout_ns)) { ok = false; break; }
          if (C::kSfRegions < C::kStages && step >= C::kSfRegions) {
            // the MMAs of step - kSfRegions read this region: wait for their
            // commit on that step's empty barrier (the full barrier above
            // already covers steps at least kStages back)
            const int64_t s2 = step - C::kSfRegions;
            if (!mbar_wait(bar_empty + 8 * (int)(s2 % C::kStages), (uint32_t)((s2 / C::kStages) & 1), abort_flag, p.err,
                           p.timeout_ns)) { ok = false; break; }
            tc_fence_after();
          }
          const uint32_t sfa_t = sf_t0 + region * C::kSfStageCols;
          const int nch = min(C::kChunks, kc - C::kChunks * k);
          if (copy_p) {
            const uint64_t d = desc0 + (uint64_t)((stage * C::kSfaBytes) >> 4);
            if constexpr (PAIR) {
              for (int c = 0; c < nch; ++c)
                tc_cp_32x128b_warpx4_pair(sfa_t + c * 4, d + (uint64_t)(c * (kSfChunk >> 4)));
            } else if (nch == C::kChunks) {
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
                tc_cp_32x128b_warpx4(sfa_t + c * 4, d + (uint64_t)(c * (kSfChunk >> 4)));
            } else {
              for (int c = 0; c < nch; ++c) tc_cp_32x128b_warpx4(sfa_t + c * 4, d + (uint64_t)(c * (kSfChunk >> 4)));
            }
          } else {
            const uint64_t d = desc0 + (uint64_t)((C::kQx ? step * C::kActSfBytes : stage * C::kSfbBytes) >> 4);
            const uint32_t sfb_t = sfa_t + C::kSfaCols;
            // (grouped: a tile of at most 128 activation rows has one block)
            const int ncp = GROUPED && rbq * 128 >= rows_of(w) ? 0 : nch;
            for (int c = 0; c < ncp; ++c) {
              if constexpr (PAIR)
                tc_cp_32x128b_warpx4_pair(sfb_t + c * 4 * C::kSfbBlocks + rbq * 4,
                                          d + (uint64_t)((rbq * C::kChunks + c) * (kSfChunk >> 4)));
              else
                tc_cp_32x128b_warpx4(sfb_t + c * 4 * C::kSfbBlocks + rbq * 4,
                                     d + (uint64_t)((rbq * C::kChunks + c) * (kSfChunk >> 4)));
            }
          }
          if constexpr (PAIR) tc_commit_pair(bar_sf + 8 * stage);
          else tc_commit(bar_sf + 8 * stage);
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
          if (++region == C::kSfRegions) region = 0;
          ++step;
        }
      }
      // every copy issued by this thread has landed before TMEM is freed
      const uint32_t db = bar_cp_drain + 8 * (warp - 6);
      if constexpr (PAIR) tc_commit_pair(db);
      else tc_commit(db);
      volatile int never = 0;
      (void)mbar_wait(db, 0, &never, p.err, p.drain_ns);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  // no CTA of a cluster leaves while another may still write into, or read
  // from, its shared memory or TMEM (CTA pairs: the even CTA's tensor-core
  // work on both has drained)
  if constexpr (PAIR) cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, C::kTmemAlloc);
    else tmem_dealloc(tmem_base, C::kTmemAlloc);
  }
}

}  // namespace nvfp4
