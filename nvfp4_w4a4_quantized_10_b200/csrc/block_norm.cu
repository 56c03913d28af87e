// Block norm: what lies between two W4A4 linear layers of a transformer block,
// in one pass over the rows.
//
//   b = y_m, or sum_j w_mj y[slot_mj]           (combine of expert rows)
//   b = b * rsqrt(mean_h(b^2) + eps) * post_w   (norm after the block, over
//                                               whole rows or heads of width h)
//   b = b * act(gate_m)
//   v = residual_m + s * b                      (the residual stream)
//   h = v * rsqrt(mean(v^2) + eps) * pre_w      (norm before the next block)
//   out = h, and/or NVFP4(h) for the next GEMM
//
// All steps in FP32 from the inputs' type; v and h are rounded once, where
// they are stored, and the codes come from the unrounded h.
// Memory-bound: every input is read once and every output written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "block_quant.cuh"
#include "common.h"
#include "ptx.cuh"

#include <initializer_list>
#include <mutex>

namespace nvfp4 {

constexpr int kNormMaxK = 32768;
// staged kernel: rows on their way to a CTA, of at least kRingRow bytes each
constexpr int kRingRow = 64 * 1024, kRingBytes = 222 * 1024, kRingSlots = kRingBytes / kRingRow;

struct NormParams {
  const void* y;
  int64_t M, K, y_rows;
  const int32_t* slots;
  const float* slot_weights;
  int top_k;
  const float* post_weight;
  int post_width;          // K, or a power of two from 16 to 512 that divides K
  const void* gate;
  int gate_kind;
  const void* residual;
  float residual_scale;
  void* residual_out;
  const float* pre_weight;
  float eps;
  void* out;
  uint8_t* codes;
  uint8_t* scales;
  float gs;
  int tc_layout;
  int64_t kc;
  uint64_t codes_bytes, scale_bytes, row_elems;
  int ring_slots;          // staged kernel
  int64_t put_rows;        // rows that are copied into the ring: M (fewer in the failure-path test)
  uint64_t timeout_ns, drain_ns;
  int ahead;               // one block a thread: a CTA fetches the rows of the one so far on into L2
  int wide;                // every row and weight starts on a 32-byte boundary
  unsigned* err;
};

template <bool kF32>
__device__ __forceinline__ void store_block(void* p, const float (&f)[16], bool wide) {
  uint4 v[kF32 ? 4 : 2];
  if constexpr (kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                        __float_as_uint(f[4 * i + 3]));
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    v[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
#pragma unroll
  for (int i = 0; i < (kF32 ? 2 : 1); ++i)
    st_32b(reinterpret_cast<uint8_t*>(p) + 32 * i, v[2 * i], v[2 * i + 1], wide);
}

__device__ __forceinline__ void load_weights(const float* w, int at, float (&f)[16], bool wide) {
  Block16<true> B;
  load_block_wide<true>(w + at, B, wide);
  block_floats<true>(B, f);
}

// Sum over the threads of one row: a warp, or the whole CTA.  The order is
// fixed, so results do not depend on timing.  red: one slot a warp, another
// array for each sum of a row, so that one barrier is enough.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* red, int warps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if constexpr (kWarpRow) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float s = lane < warps ? red[lane] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s;
}

// 16 elements from shared memory.  Threads read in turn the 16-byte pieces that
// lie in different banks; selects put them in order.
template <bool kF32>
__device__ __forceinline__ void load_block_shared(uint32_t addr, Block16<kF32>& B) {
  constexpr int kP = kF32 ? 4 : 2;
  const int turn = (threadIdx.x >> (kF32 ? 1 : 2)) & (kP - 1);
#pragma unroll
  for (int i = 0; i < kP; ++i)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(B.v[i].x), "=r"(B.v[i].y), "=r"(B.v[i].z), "=r"(B.v[i].w)
                 : "r"(addr + 16 * (i ^ turn))
                 : "memory");
#pragma unroll
  for (int bit = 1; bit < kP; bit *= 2)
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      if (i & bit) continue;
      const bool swap = turn & bit;
      const uint4 lo = B.v[i], hi = B.v[i + bit];
      B.v[i] = make_uint4(swap ? hi.x : lo.x, swap ? hi.y : lo.y, swap ? hi.z : lo.z, swap ? hi.w : lo.w);
      B.v[i + bit] = make_uint4(swap ? lo.x : hi.x, swap ? lo.y : hi.y, swap ? lo.z : hi.z, swap ? lo.w : hi.w);
    }
}

// Rows on their way through shared memory (staged kernel): a ring of slots of
// one array's row each, filled by bulk copies in the order y, gate, residual,
// next row's y, ...  A slot's barrier counts its copies; what has been read is
// known from the barriers of the row's sums, after which thread 0 refills.
struct RowRing {
  uint32_t base, bars, bytes;
  int slots, arrays;
  int take_slot;
  uint32_t take_phase;
  int64_t put_row;           // next copy: row, array, slot
  int put_array, put_slot, issued;
};

// Shared-memory address of the next array's row, once it is there.
__device__ __forceinline__ uint32_t ring_take(RowRing& r, const NormParams& p, volatile int* abort_flag) {
  // (a wait that runs out sets the error word; the rows are then not reliable)
  (void)mbar_wait(r.bars + 8 * r.take_slot, r.take_phase, abort_flag, p.err, p.timeout_ns);
  const uint32_t at = r.base + r.take_slot * r.bytes;
  if (++r.take_slot == r.slots) {
    r.take_slot = 0;
    r.take_phase ^= 1;
  }
  return at;
}

__device__ __forceinline__ void ring_put(RowRing& r, const NormParams& p, volatile int* abort_flag) {
  if (r.put_row >= p.put_rows || *abort_flag) return;
  const void* src = r.put_array == 0 ? p.y : r.put_array == 1 && p.gate ? p.gate : p.residual;
  const uint32_t bar = r.bars + 8 * r.put_slot;
  mbar_arrive_expect_tx(bar, r.bytes);
  bulk_load(r.base + r.put_slot * r.bytes, reinterpret_cast<const uint8_t*>(src) + r.put_row * r.bytes, r.bytes, bar);
  ++r.issued;
  if (++r.put_slot == r.slots) r.put_slot = 0;
  if (++r.put_array == r.arrays) {
    r.put_array = 0;
    r.put_row += gridDim.x;
  }
}

// NB: 16-element blocks of a thread; kWarpRow: a warp owns a row (K <= 512
// NB), else a CTA does.  One row and done: the block scheduler then keeps
// every SM's loads coming while other rows wait in their reductions (16384 x
// 5120 bf16, residual and norm, with 16-byte accesses: 121 us; a persistent
// grid of 2, 3, 4 or 6 CTAs an SM that walks the rows: 143, 168, 129, 148; 98 us
// with 32-byte accesses, one barrier a sum and the register caps below).
// kStaged: that persistent grid for the longest rows, one CTA an SM, with rows
// on their way by bulk copies while others are computed (RowRing).
// kThreads, kCtas: the CTA's most threads, and CTAs that are to fit on an SM
// (which caps the registers; 48 of them instead of 56 are 4 CTAs instead of 3
// and 99 instead of 108 us in that case).  The caps were measured without
// slots.  Two CTAs of 576 threads (NB = 2) have 56 registers, and spill 44 to
// 112 bytes a thread in bf16 and 64 to 520 in FP32 (most with slots and gate);
// of 512 threads (NB = 1) only with slots, 64 to 216.  Combines of 8 rows of
// 9216 into 2048: 80 us in bf16 (79 % of the copy bandwidth), 162 in FP32 (78 %),
// 187 with a gate (74 %).
template <bool kF32, int NB, bool kWarpRow, bool kSlots, bool kGate, int kThreads, int kCtas, bool kStaged = false>
__global__ void __launch_bounds__(kThreads, kCtas) block_norm_kernel(const NormParams p) {
  __shared__ float red_s[kStaged ? 4 : 2][32];
  __shared__ float quot[8];
  __shared__ uint64_t ring_bars[kStaged ? kRingSlots : 1];
  __shared__ int abort_s;
  extern __shared__ uint8_t ring_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.codes) {                         // (uniform) seen by all after this barrier
    if (threadIdx.x < 8) quot[threadIdx.x] = scale_quotient(p.gs, threadIdx.x);
    __syncthreads();
  }
  const int warps = blockDim.x >> 5;
  const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x;       // thread of the row
  const int nthr = kWarpRow ? 32 : blockDim.x;
  const int nblk = (int)(p.K / 16);
  constexpr int kB = kF32 ? 64 : 32;                             // bytes of a block
  // more than one block a thread: gate and residual are read where they are
  // used, instead of being held in registers through the first norm
  constexpr bool kHold = NB == 1;
  const float inv_k = 1.0f / (float)p.K;
  const bool wide = p.wide != 0;
  volatile int* abort_flag = &abort_s;
  RowRing ring = {};
  if constexpr (kStaged) {
    ring.base = (smem_u32(ring_raw) + 127) & ~127u;
    ring.bars = smem_u32(ring_bars);
    ring.bytes = (uint32_t)nblk * kB;
    ring.slots = p.ring_slots;
    ring.arrays = 1 + (kGate ? 1 : 0) + (p.residual ? 1 : 0);
    ring.put_row = blockIdx.x;
    if (threadIdx.x == 0) {
      abort_s = 0;
      for (int i = 0; i < ring.slots; ++i) mbar_init(ring.bars + 8 * i, 1);
      fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0)
      for (int i = 0; i < ring.slots; ++i) ring_put(ring, p, abort_flag);
  }
  auto block_at = [&](const void* base, int64_t row, int j) {
    return reinterpret_cast<const uint8_t*>(base) + (row * nblk + j) * kB;
  };
  auto do_row = [&](const int64_t m, float (*red)[32]) {
    float f[NB][16];
    int unread = kStaged ? ring.arrays : 0;              // arrays of this row that have not been given back
    uint32_t ring_gate = 0, ring_res = 0;
    // ------------------------------------------------ branch
    Block16<kF32> R[kHold ? NB : 1], G[kHold && kGate ? NB : 1];
    auto load_rest = [&](int b, Block16<kF32>& r, Block16<kF32>& g) {
      const int j = t + b * nthr;
      if constexpr (kStaged) {
        r = g = Block16<kF32>{};
        if (j < nblk && p.residual) load_block_shared<kF32>(ring_res + j * kB, r);
        if (kGate && j < nblk) load_block_shared<kF32>(ring_gate + j * kB, g);
        return;
      }
      r = Block16<kF32>{};
      if (j < nblk && p.residual) load_block_wide<kF32>(block_at(p.residual, m, j), r, wide);
      if constexpr (kGate) {
        g = Block16<kF32>{};
        if (j < nblk) load_block_wide<kF32>(block_at(p.gate, m, j), g, wide);
      }
    };
    if constexpr (kHold) load_rest(0, R[0], G[0]);
    if constexpr (!kWarpRow && !kStaged) {
      // whole rows, asked for by one thread, are in L2 sooner than by the
      // loads of many: those of a later CTA, or, where the rows in flight and
      // as many to come are more than L2 holds, this one's (4096 x 8192 bf16,
      // residual and norm: 46.7 to 41.3 us; 2048 x 17408, gate and two norms:
      // 84.0 to 79.7, and 99 with a later CTA's)
      const int64_t at = kHold ? m + p.ahead : m;
      if (threadIdx.x == 0 && at < p.M) {
        const uint32_t bytes = (uint32_t)nblk * kB;
        if (!kSlots) bulk_prefetch_l2(block_at(p.y, at, 0), bytes);
        if (p.residual) bulk_prefetch_l2(block_at(p.residual, at, 0), bytes);
        if constexpr (kGate) bulk_prefetch_l2(block_at(p.gate, at, 0), bytes);
      }
    }
    if constexpr (!kSlots) {
      Block16<kF32> B[NB];
      uint32_t ring_y = 0;
      if constexpr (kStaged) ring_y = ring_take(ring, p, abort_flag);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int j = t + b * nthr;
        B[b] = Block16<kF32>{};
        if (kStaged && j < nblk) load_block_shared<kF32>(ring_y + j * kB, B[b]);
        if (!kStaged && j < nblk) load_block_wide<kF32>(block_at(p.y, m, j), B[b], wide);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) block_floats<kF32>(B[b], f[b]);
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) f[b][i] = 0.0f;
      // kCh slots at a time, so that their rows' loads overlap
      constexpr int kCh = NB > 1 ? 1 : kF32 ? 2 : 4;
      for (int q0 = 0; q0 < p.top_k; q0 += kCh) {
        int64_t src[kCh];
        float w[kCh];
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          const int64_t at = m * p.top_k + q0 + c;
          src[c] = q0 + c < p.top_k ? p.slots[at] : -1;
          w[c] = q0 + c < p.top_k ? p.slot_weights[at] : 0.0f;
        }
        Block16<kF32> B[kCh][NB];
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          if (src[c] >= p.y_rows || src[c] < -1) {
            atomicCAS(p.err, 0u, kErrBounds);                    // a row y does not have: skipped
            src[c] = -1;
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int j = t + b * nthr;
            B[c][b] = Block16<kF32>{};
            if (src[c] >= 0 && j < nblk)                         // -1: a slot the router left empty
              load_block_wide<kF32>(block_at(p.y, src[c], j), B[c][b], wide);
          }
        }
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          if (src[c] < 0) continue;                              // its weight is not read into the sum
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float x[16];
            block_floats<kF32>(B[c][b], x);
#pragma unroll
            for (int i = 0; i < 16; ++i) f[b][i] = fmaf(w[c], x[i], f[b][i]);
          }
        }
      }
    }
    // ------------------------------------------------ norm after the block
    if (p.post_weight) {
      float ss[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        ss[b] = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss[b] = fmaf(f[b][i], f[b][i], ss[b]);
      }
      if (p.post_width == (int)p.K) {
        float s = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) s += ss[b];
        s = row_sum<kWarpRow>(s, red[0], warps);
        if (kStaged) {                                   // every thread has read y
          if (threadIdx.x == 0) ring_put(ring, p, abort_flag);
          --unread;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) ss[b] = s;
      } else {
        // a head is post_width / 16 neighbouring blocks: so many lanes of a
        // warp, since nthr is a multiple of 32
#pragma unroll
        for (int b = 0; b < NB; ++b)
          for (int d = p.post_width / 32; d > 0; d >>= 1) ss[b] += __shfl_xor_sync(0xFFFFFFFFu, ss[b], d);
      }
      const float inv = 1.0f / (float)p.post_width;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int j = t + b * nthr;
        if (j >= nblk) continue;
        const float r = rsqrtf(fmaf(ss[b], inv, p.eps));
        float w[16];
        load_weights(p.post_weight, p.post_width == (int)p.K ? j * 16 : (j * 16) & (p.post_width - 1), w, wide);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[b][i] = f[b][i] * r * w[i];
      }
    }
    // ------------------------------------------------ gate, residual stream
    float s = 0.0f;
    if constexpr (kStaged) {
      if (kGate) ring_gate = ring_take(ring, p, abort_flag);
      if (p.residual) ring_res = ring_take(ring, p, abort_flag);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int j = t + b * nthr;
      float x[16];
      Block16<kF32> rb, gb;
      if constexpr (kHold) {
        rb = R[b];
        if constexpr (kGate) gb = G[b];
      } else {
        load_rest(b, rb, gb);
      }
      if constexpr (kGate) {
        block_floats<kF32>(gb, x);
        if (p.gate_kind == NVFP4_GATE_LINEAR) {
#pragma unroll
          for (int i = 0; i < 16; ++i) f[b][i] *= x[i];
        } else {
          if (p.gate_kind == NVFP4_GATE_SILU) apply_gate<true>(x, f[b]);
          else apply_gate<false>(x, f[b]);
        }
      }
      block_floats<kF32>(rb, x);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        f[b][i] = fmaf(p.residual_scale, f[b][i], x[i]);
        s = fmaf(f[b][i], f[b][i], s);
      }
      if (p.residual_out && j < nblk && bounds_ok((uint64_t)((m * nblk + j + 1) * 16) <= p.row_elems, p.err))
        store_block<kF32>(const_cast<uint8_t*>(block_at(p.residual_out, m, j)), f[b], wide);
    }
    // ------------------------------------------------ norm before the next block
    if (p.pre_weight) s = row_sum<kWarpRow>(s, red[1], warps);
    else if (kStaged) __syncthreads();
    if (kStaged && threadIdx.x == 0)                     // every thread has read the row
      for (; unread > 0; --unread) ring_put(ring, p, abort_flag);
    if (p.pre_weight) {
      const float r = rsqrtf(fmaf(s, inv_k, p.eps));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int j = t + b * nthr;
        if (j >= nblk) continue;
        float w[16];
        load_weights(p.pre_weight, j * 16, w, wide);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[b][i] = f[b][i] * r * w[i];
      }
    }
    // ------------------------------------------------ outputs
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int j = t + b * nthr;
      if (j >= nblk) continue;
      if (p.out && bounds_ok((uint64_t)((m * nblk + j + 1) * 16) <= p.row_elems, p.err))
        store_block<kF32>(const_cast<uint8_t*>(block_at(p.out, m, j)), f[b], wide);
      if (p.codes) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[b][i]));
        uint32_t lo, hi;
        const uint32_t sc = quantize_values(f[b], amax, p.gs, quot, lo, hi);
        const int64_t at = m * nblk + j;
        if (bounds_ok((uint64_t)(at + 1) * 8 <= p.codes_bytes, p.err))
          reinterpret_cast<uint2*>(p.codes)[at] = make_uint2(lo, hi);
        const int64_t o = p.tc_layout ? tc_scale_offset(m, j, p.kc) : at;
        if (bounds_ok((uint64_t)o < p.scale_bytes, p.err)) p.scales[o] = (uint8_t)sc;
        // K % 64 == 32: the row's last chunk has two padding slots
        if (p.tc_layout && j == nblk - 1 && (nblk & 3) == 2) {
          const int64_t o2 = tc_scale_offset(m, j + 2, p.kc);
          if (bounds_ok((uint64_t)o2 < p.scale_bytes, p.err)) {
            p.scales[o2 - 1] = 0;
            p.scales[o2] = 0;
          }
        }
      }
    }
  };
  if constexpr (kStaged) {
    // (a row's sums lie in slots that the next row's do not use)
    int turn = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, turn ^= 2) do_row(m, red_s + turn);
    // after a wait that ran out, copies may still be on their way
    if (threadIdx.x == 0 && *abort_flag) {
      volatile int never = 0;
      for (int i = 0; i < ring.slots && i < ring.issued; ++i)
        (void)mbar_wait(ring.bars + 8 * i, (uint32_t)((ring.issued - 1 - i) / ring.slots) & 1u, &never, p.err,
                        p.drain_ns);
    }
  } else {
    const int64_t m = kWarpRow ? (int64_t)blockIdx.x * warps + (threadIdx.x >> 5) : blockIdx.x;
    if (m < p.M) do_row(m, red_s);
  }
  // padding rows of the tensor-core layout (up to 127 past M): zero scales,
  // one row a CTA
  if (p.codes && p.tc_layout) {
    const int64_t end = (p.M + 127) / 128 * 128;
    for (int64_t r = p.M + blockIdx.x; r < end; r += gridDim.x)
      for (int64_t c = threadIdx.x; c < p.kc; c += blockDim.x) {
        const int64_t o = tc_scale_offset(r, c * 4, p.kc);
        if (bounds_ok((uint64_t)o + 4 <= p.scale_bytes, p.err)) *reinterpret_cast<uint32_t*>(p.scales + o) = 0u;
      }
  }
}

namespace {

// kCtas of the kernel without slots and gate; those hold more and get fewer.
template <bool kF32, int NB, bool kWarpRow, int kThreads, int kCtas>
cudaError_t launch_norm_as(const NormParams& p, int grid, int threads, cudaStream_t st) {
  constexpr int kGated = kCtas > 3 ? 3 : kCtas, kSlotted = kCtas > 2 ? 2 : kCtas;
  if (p.slots)
    return p.gate
               ? launch_pdl(block_norm_kernel<kF32, NB, kWarpRow, true, true, kThreads, kSlotted>, grid, threads, st, p)
               : launch_pdl(block_norm_kernel<kF32, NB, kWarpRow, true, false, kThreads, kSlotted>, grid, threads, st, p);
  return p.gate
             ? launch_pdl(block_norm_kernel<kF32, NB, kWarpRow, false, true, kThreads, kGated>, grid, threads, st, p)
             : launch_pdl(block_norm_kernel<kF32, NB, kWarpRow, false, false, kThreads, kCtas>, grid, threads, st, p);
}

// Staged kernel: one CTA an SM.
template <bool kF32, int NB, int kThreads>
cudaError_t launch_norm_staged(NormParams& p, const DeviceInfo* d, int threads, cudaStream_t st) {
  auto run = [&](auto kern, std::once_flag& once, cudaError_t& attr) {
    std::call_once(once, [&] {
      attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes + 128);
    });
    if (attr != cudaSuccess) return attr;
    const int64_t row = p.K * (kF32 ? 4 : 2);
    p.ring_slots = (int)(kRingBytes / row);
    return launch_pdl_smem(kern, d->sm_count, threads, p.ring_slots * row + 128, st, p);
  };
  static std::once_flag once[2][64];
  static cudaError_t attr[2][64];
  return p.gate ? run(block_norm_kernel<kF32, NB, false, false, true, kThreads, 1, true>, once[1][d->device],
                      attr[1][d->device])
                : run(block_norm_kernel<kF32, NB, false, false, false, kThreads, 1, true>, once[0][d->device],
                      attr[0][d->device]);
}

// Staged: rows of at least 64 KB without slots whose inputs fit in the ring,
// and more than two of them an SM.  In 4 bytes, 1003 x 17408, gate, residual
// and two norms: 69.8 us, not staged 80.5 (150 rows: 21.0 and 20.1); 2048 x
// 16384: 117 and 138; 2048 x 20480, residual and norm: 109 and 116; in 2
// bytes, 1024 x 32768: 50.6 and 56.3, with gate and two norms 91.0 and 89.9.
// On shorter rows the one CTA's instructions show: 2048 x 10240 in 4 bytes,
// gate and two norms 93.2 and 86.1, 2048 x 17408 in 2 bytes 101 and 79.7.
bool staged(const NormParams& p, bool f32, const DeviceInfo* d) {
  const int64_t row = p.K * (f32 ? 4 : 2), inputs = (1 + (p.gate != nullptr) + (p.residual != nullptr)) * row;
  return !p.slots && p.M > 2 * d->sm_count && row >= kRingRow && inputs <= kRingBytes;
}

// Rows of at most 1024 elements: a warp each, 8 to a CTA.  Longer ones: a CTA
// each, with one 16-element block a thread while registers allow (K up to
// 8192), then two (18432), then four.
template <bool kF32>
cudaError_t launch_norm(NormParams& p, const DeviceInfo* d, cudaStream_t st) {
  const int nblk = (int)(p.K / 16);
  const int64_t padding = p.codes && p.tc_layout ? ceil_div(p.M, 128) * 128 - p.M : 0;
  auto ctas = [&](int64_t rows) { return (int)(rows > padding ? rows : padding); };
  if (nblk <= 64) {
    const int grid = ctas(ceil_div(p.M, 8));
    return nblk <= 32 ? launch_norm_as<kF32, 1, true, 256, 4>(p, grid, 256, st)
                      : launch_norm_as<kF32, 2, true, 256, 3>(p, grid, 256, st);
  }
  const int grid = ctas(p.M);
  auto threads = [&](int nb) { return (int)ceil_div(ceil_div(nblk, nb), 32) * 32; };
  if (nblk <= 320) return launch_norm_as<kF32, 1, false, 320, 4>(p, grid, threads(1), st);
  if (nblk <= 512) return launch_norm_as<kF32, 1, false, 512, 2>(p, grid, threads(1), st);
  if (staged(p, kF32, d)) {
    if constexpr (kF32)                            // (in 2 bytes only longer rows have 64 KB)
      if (nblk <= 2 * 576) return launch_norm_staged<kF32, 2, 576>(p, d, threads(2), st);
    return launch_norm_staged<kF32, 4, 512>(p, d, threads(4), st);
  }
  if (nblk <= 2 * 576) return launch_norm_as<kF32, 2, false, 576, 2>(p, grid, threads(2), st);
  return launch_norm_as<kF32, 4, false, 512, 1>(p, grid, threads(4), st);
}

// stalled_from: the failure-path test's first row that no copy brings, or -1.
nvfp4_status run_block_norm(const void* y, nvfp4_in_dtype dtype, int64_t M, int64_t K, int64_t y_rows,
                            const int32_t* slots, const float* slot_weights, int top_k, const float* post_weight,
                            int64_t post_width, const void* gate, nvfp4_gate gate_kind, const void* residual,
                            float residual_scale, void* residual_out, const float* pre_weight, float eps, void* out,
                            uint8_t* codes, uint8_t* block_scales, float global_scale, nvfp4_sf_layout layout,
                            int64_t stalled_from, nvfp4_stream_t stream) {
  if (!y || M < 1 || K < 32 || K % 32 != 0) return NVFP4_ERR_INVALID_ARG;
  if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
  if ((slots == nullptr) != (slot_weights == nullptr)) return NVFP4_ERR_INVALID_ARG;
  if (slots ? (top_k < 1 || y_rows < 1) : (y_rows != M)) return NVFP4_ERR_INVALID_ARG;
  if (gate_kind < NVFP4_GATE_NONE || gate_kind > NVFP4_GATE_SILU) return NVFP4_ERR_INVALID_ARG;
  if ((gate == nullptr) != (gate_kind == NVFP4_GATE_NONE)) return NVFP4_ERR_INVALID_ARG;
  if ((codes == nullptr) != (block_scales == nullptr)) return NVFP4_ERR_INVALID_ARG;
  if (!out && !codes && !residual_out) return NVFP4_ERR_INVALID_ARG;
  if (!finite_positive(eps) || !(residual_scale - residual_scale == 0.0f)) return NVFP4_ERR_INVALID_ARG;
  if (codes && (!finite_positive(global_scale) || (layout != NVFP4_SF_ROWMAJOR && layout != NVFP4_SF_TCGEN05)))
    return NVFP4_ERR_INVALID_ARG;
  if (post_weight) {
    const bool heads = post_width >= 16 && post_width <= 512 && (post_width & (post_width - 1)) == 0;
    if (post_width != K && (!heads || K % post_width != 0)) return NVFP4_ERR_INVALID_ARG;
  }
  if (K > kNormMaxK || M > (1ll << 31) - 256 || y_rows > (1ll << 31) - 256 || top_k > (1 << 16))
    return NVFP4_ERR_UNSUPPORTED;
  if (!aligned16(y) || !aligned16(post_weight) || !aligned16(gate) || !aligned16(residual) ||
      !aligned16(residual_out) || !aligned16(pre_weight) || !aligned16(out) || !aligned16(codes) ||
      !aligned16(block_scales))
    return NVFP4_ERR_ALIGNMENT;
  if (!aligned4(slots) || !aligned4(slot_weights)) return NVFP4_ERR_ALIGNMENT;
  const DeviceInfo* d = device_info();
  if (!d) return NVFP4_ERR_CUDA;
  if (d->major != 10) return NVFP4_ERR_UNSUPPORTED;
  NormParams p;
  p.y = y;
  p.M = M;
  p.K = K;
  p.y_rows = y_rows;
  p.slots = slots;
  p.slot_weights = slot_weights;
  p.top_k = top_k;
  p.post_weight = post_weight;
  p.post_width = post_weight ? (int)post_width : (int)K;
  p.gate = gate;
  p.gate_kind = (int)gate_kind;
  p.residual = residual;
  p.residual_scale = residual_scale;
  p.residual_out = residual_out;
  p.pre_weight = pre_weight;
  p.eps = eps;
  p.out = out;
  p.codes = codes;
  p.scales = block_scales;
  p.gs = global_scale;
  p.tc_layout = layout == NVFP4_SF_TCGEN05;
  p.kc = ceil_div(K, 64);
  p.codes_bytes = (uint64_t)M * (uint64_t)(K / 2);
  p.scale_bytes = codes ? nvfp4_scale_bytes(M, K, layout) : 0;
  p.row_elems = (uint64_t)M * (uint64_t)K;
  p.ahead = d->sm_count;
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = drain_timeout_ns();
  p.wide = 1;
  for (const void* q : {y, (const void*)post_weight, gate, residual, (const void*)residual_out,
                        (const void*)pre_weight, (const void*)out})
    if (reinterpret_cast<uintptr_t>(q) & 31) p.wide = 0;
  p.put_rows = stalled_from < 0 ? M : stalled_from;
  p.err = d->err_word;
  if (stalled_from >= 0 && !staged(p, dtype == NVFP4_IN_F32, d)) return NVFP4_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == NVFP4_IN_F32 ? launch_norm<true>(p, d, st) : launch_norm<false>(p, d, st));
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status nvfp4_block_norm(const void* y, nvfp4_in_dtype dtype, int64_t M, int64_t K, int64_t y_rows,
                              const int32_t* slots, const float* slot_weights, int top_k, const float* post_weight,
                              int64_t post_width, const void* gate, nvfp4_gate gate_kind, const void* residual,
                              float residual_scale, void* residual_out, const float* pre_weight, float eps, void* out,
                              uint8_t* codes, uint8_t* block_scales, float global_scale, nvfp4_sf_layout layout,
                              nvfp4_stream_t stream) {
  return run_block_norm(y, dtype, M, K, y_rows, slots, slot_weights, top_k, post_weight, post_width, gate, gate_kind,
                        residual, residual_scale, residual_out, pre_weight, eps, out, codes, block_scales, global_scale,
                        layout, -1, stream);
}

nvfp4_status nvfp4_test_block_norm_stalled(const void* y, nvfp4_in_dtype dtype, int64_t M, int64_t K,
                                           const void* residual, int64_t stalled_from, void* out,
                                           nvfp4_stream_t stream) {
  if (stalled_from < 0 || stalled_from > M) return NVFP4_ERR_INVALID_ARG;
  return run_block_norm(y, dtype, M, K, M, nullptr, nullptr, 0, nullptr, 0, nullptr, NVFP4_GATE_NONE, residual, 1.0f,
                        nullptr, nullptr, 1e-6f, out, nullptr, nullptr, 1.0f, NVFP4_SF_TCGEN05, stalled_from, stream);
}

}  // extern "C"
