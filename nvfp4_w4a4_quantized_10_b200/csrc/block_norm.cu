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

namespace nvfp4 {

constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxBlocks = 4;                                   // 16-element blocks of a thread
constexpr int kNormMaxK = kNormMaxThreads * kNormMaxBlocks * 16;    // 32768

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
  unsigned* err;
};

// A block that the same thread may overwrite later (outputs may be the
// inputs' own buffers): a plain load, not the read-only path.
template <bool kF32>
__device__ __forceinline__ void load_block_rw(const void* p, Block16<kF32>& B) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) B.v[i] = __ldcg(q + i);
}

template <bool kF32>
__device__ __forceinline__ void store_block(void* base, int64_t elem, const float (&f)[16]) {
  if constexpr (kF32) {
    float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(base) + elem);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__device__ __forceinline__ void load_weights(const float* w, int at, float (&f)[16]) {
  const float4* q = reinterpret_cast<const float4*>(w + at);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(q + i);
    f[4 * i] = v.x;
    f[4 * i + 1] = v.y;
    f[4 * i + 2] = v.z;
    f[4 * i + 3] = v.w;
  }
}

// Sum over the threads of one row: a warp, or the whole CTA.  The order is
// fixed, so results do not depend on timing.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* red, int warps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if constexpr (kWarpRow) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();                       // red may still be read from the last use
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float s = lane < warps ? red[lane] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s;
}

// NB: 16-element blocks of a thread; kWarpRow: a warp owns a row (K <= 512 NB),
// else a CTA does.
template <bool kF32, int NB, bool kWarpRow>
__global__ void __launch_bounds__(kNormMaxThreads) block_norm_kernel(const NormParams p) {
  __shared__ float red[kNormMaxThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warps = blockDim.x >> 5;
  const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x;       // thread of the row
  const int nthr = kWarpRow ? 32 : blockDim.x;
  const int nblk = (int)(p.K / 16);
  constexpr int kB = kF32 ? 64 : 32;                             // bytes of a block
  const float inv_k = 1.0f / (float)p.K;
  int64_t m = kWarpRow ? (int64_t)blockIdx.x * warps + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = kWarpRow ? (int64_t)gridDim.x * warps : gridDim.x;
  for (; m < p.M; m += step) {
    float f[NB][16];
    // ------------------------------------------------ branch
    if (p.slots == nullptr) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int j = t + b * nthr;
        Block16<kF32> B = {};
        if (j < nblk) load_block_rw<kF32>(reinterpret_cast<const uint8_t*>(p.y) + (m * nblk + j) * kB, B);
        block_floats<kF32>(B, f[b]);
      }
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
          src[c] = q0 + c < p.top_k ? __ldg(p.slots + at) : -1;
          w[c] = q0 + c < p.top_k ? __ldg(p.slot_weights + at) : 0.0f;
        }
        Block16<kF32> B[kCh][NB];
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          if (src[c] >= p.y_rows) {
            atomicCAS(p.err, 0u, kErrBounds);                    // a row y does not have: skipped
            src[c] = -1;
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int j = t + b * nthr;
            B[c][b] = Block16<kF32>{};
            if (src[c] >= 0 && j < nblk)                         // -1: a slot the router left empty
              load_block_at<kF32>(reinterpret_cast<const uint8_t*>(p.y) + (src[c] * nblk + j) * kB, B[c][b]);
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
    // the row's other inputs are in flight while the branch is normed
    Block16<kF32> R[NB], G[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int j = t + b * nthr;
      R[b] = Block16<kF32>{};
      G[b] = Block16<kF32>{};
      if (j < nblk) {
        if (p.residual) load_block_rw<kF32>(reinterpret_cast<const uint8_t*>(p.residual) + (m * nblk + j) * kB, R[b]);
        if (p.gate) load_block_rw<kF32>(reinterpret_cast<const uint8_t*>(p.gate) + (m * nblk + j) * kB, G[b]);
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
        s = row_sum<kWarpRow>(s, red, warps);
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
        load_weights(p.post_weight, p.post_width == (int)p.K ? j * 16 : (j * 16) & (p.post_width - 1), w);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[b][i] = f[b][i] * r * w[i];
      }
    }
    // ------------------------------------------------ gate, residual stream
    float s = 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int j = t + b * nthr;
      float x[16];
      if (p.gate_kind != NVFP4_GATE_NONE) {
        block_floats<kF32>(G[b], x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float a = x[i];
          if (p.gate_kind != NVFP4_GATE_LINEAR) {
            a = __frcp_rn(1.0f + expf(-x[i]));
            if (p.gate_kind == NVFP4_GATE_SILU) a *= x[i];
          }
          f[b][i] *= a;
        }
      }
      block_floats<kF32>(R[b], x);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        f[b][i] = fmaf(p.residual_scale, f[b][i], x[i]);
        s = fmaf(f[b][i], f[b][i], s);
      }
      if (p.residual_out && j < nblk && bounds_ok((uint64_t)((m * nblk + j + 1) * 16) <= p.row_elems, p.err))
        store_block<kF32>(p.residual_out, (m * nblk + j) * 16, f[b]);
    }
    // ------------------------------------------------ norm before the next block
    if (p.pre_weight) {
      s = row_sum<kWarpRow>(s, red, warps);
      const float r = rsqrtf(fmaf(s, inv_k, p.eps));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int j = t + b * nthr;
        if (j >= nblk) continue;
        float w[16];
        load_weights(p.pre_weight, j * 16, w);
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
        store_block<kF32>(p.out, (m * nblk + j) * 16, f[b]);
      if (p.codes) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[b][i]));
        uint32_t lo, hi;
        const uint32_t sc = quantize_values(f[b], amax, p.gs, lo, hi);
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
  }
  // padding rows of the tensor-core layout (up to 127 past M): zero scales
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

template <bool kF32>
cudaError_t launch_norm(const NormParams& p, const DeviceInfo* d, cudaStream_t st) {
  const int nblk = (int)(p.K / 16);
  // rows of at most 1024: a warp each, 8 to a CTA; longer ones a CTA each
  if (nblk <= 64) {
    const int64_t want = ceil_div(p.M, 8), cap = (int64_t)d->sm_count * 8;
    const int grid = (int)(want < cap ? want : cap);
    return nblk <= 32 ? launch_pdl(block_norm_kernel<kF32, 1, true>, grid, 256, st, p)
                      : launch_pdl(block_norm_kernel<kF32, 2, true>, grid, 256, st, p);
  }
  const int nb = (int)ceil_div(nblk, kNormMaxThreads);
  const int threads = (int)ceil_div(ceil_div(nblk, nb), 32) * 32;
  const int64_t cap = (int64_t)d->sm_count * (2048 / threads);
  const int grid = (int)(p.M < cap ? p.M : cap);
  if (nb == 1) return launch_pdl(block_norm_kernel<kF32, 1, false>, grid, threads, st, p);
  if (nb == 2) return launch_pdl(block_norm_kernel<kF32, 2, false>, grid, threads, st, p);
  return launch_pdl(block_norm_kernel<kF32, 4, false>, grid, threads, st, p);
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
  p.err = d->err_word;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == NVFP4_IN_F32 ? launch_norm<true>(p, d, st) : launch_norm<false>(p, d, st));
}

}  // extern "C"
