// W4A4 linear layer over experts: the grouped activation quantizer and the
// grouped GEMM.
//
//   quantize  row t of group g = NVFP4(x[row_index[t]], gs[g]), or of
//             silu(gate) * up of a row [gate | up]
//   gemm      out[t, n] = 1 / (ga[g] gw[g]) * sum_k A[t, k] W_g[n, k]
//
// Group offsets live on the device (the router wrote them), so both kernels
// build the table of groups.cuh in shared memory and take their work from it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "block_quant.cuh"
#include "common.h"
#include "gemm_host.h"
#include "gemm_kernel.cuh"
#include "groups.cuh"
#include "ptx.cuh"

namespace nvfp4 {

struct GroupedQuantParams {
  const void* x;
  int64_t M;                  // rows of x
  const int32_t* row_index;   // or NULL: row t of x
  const int32_t* offsets;
  int E;
  int64_t T;
  int nblk;                   // K / 16
  int seg;                    // warp-wide runs of 32 blocks in one work item
  int parts;                  // work items of a row
  DivU32 div_parts;
  const float* gs;
  uint8_t* codes;
  uint8_t* scales;
  uint32_t kc;
  uint64_t codes_bytes, scale_bytes;
  int wide;                   // rows start on 32-byte boundaries
  unsigned* err;
};

// One thread owns one 16-element block, as in the plain quantizer; a warp
// owns a row, or a part of one when rows are few, and walks it 32 blocks at a
// time, so that the group, the source row and the scale's place are found
// once an item and every address inside is an immediate offset.  A CTA owns a
// contiguous share of all items that the offsets name: it builds the table of
// groups, and the scale quotients of the groups it meets, once.
// Bound: HBM writes 9/16 byte an element and reads each source row once, but a
// row gathered k times is read k - 1 times from L2 and encoded k times, and
// the encoding (some 140 instructions a block) is what it waits for: 2048 rows
// of 5120 gathered 8 times take 31 us back to back (37 with cold caches; issue
// slots 59 % busy), and took 42 with a flat loop over blocks (214 instructions
// each); 16384 rows once, 37 us (5.8 TB/s).
// Three CTAs an SM: all resident, with one prologue each (4 of them with fewer
// registers took 33.1 us in the gathered case, 6 in two waves 37).
constexpr int kQuantCtas = 3;

template <bool kF32, bool kGlu>
__global__ void __launch_bounds__(256, kQuantCtas) grouped_quantize_kernel(const GroupedQuantParams p) {
  __shared__ GroupTable tab;
  __shared__ float quot[kMaxGroups][8];
  constexpr int U = kF32 || kGlu ? 2 : 4;                 // loads in flight
  constexpr int kB = kF32 ? 64 : 32;                      // bytes of a block
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  load_groups(tab, p.offsets, p.E, p.T, p.err);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t total = (uint64_t)tab.off[p.E] * p.parts;
  const uint32_t c_begin = (uint32_t)(total * blockIdx.x / gridDim.x);
  const uint32_t c_end = (uint32_t)(total * (blockIdx.x + 1) / gridDim.x);
  if (c_begin >= c_end) return;
  const int g_first = find_group(tab.off, p.E, (int)div_u32(c_begin, p.div_parts));
  const int g_last = find_group(tab.off, p.E, (int)div_u32(c_end - 1, p.div_parts));
  for (int i = threadIdx.x; i < (g_last - g_first + 1) * 8; i += 256)
    quot[i >> 3][i & 7] = scale_quotient(p.gs[g_first + (i >> 3)], i & 7);
  __syncthreads();
  const uint32_t n = c_end - c_begin;
  const uint32_t begin = c_begin + n * warp / 8, end = c_begin + n * (warp + 1) / 8;
  if (begin >= end) return;
  int g = find_group(tab.off, p.E, (int)div_u32(begin, p.div_parts));
  const int64_t src_bytes = (int64_t)p.nblk * kB * (kGlu ? 2 : 1);
  const bool wide = p.wide != 0;
  const uint32_t lane_scale = (uint32_t)(lane >> 2) * 512 + (lane & 3);
  for (uint32_t item = begin; item < end; ++item) {
    const uint32_t row = div_u32(item, p.div_parts);
    const int j0 = (int)(item - row * p.parts) * p.seg * 32 + lane;
    const int j_end = min(p.nblk, j0 - lane + p.seg * 32);
    while ((int)row >= tab.off[g + 1]) ++g;
    const float gs = p.gs[g];
    const float* q = quot[g - g_first];
    int64_t src = row;
    if (p.row_index) src = p.row_index[row];
    const bool have = src >= 0 && src < p.M;
    if (!have && lane == 0) atomicCAS(p.err, 0u, kErrBounds);   // a row that x does not have: quantized as zeros
    const uint8_t* x = reinterpret_cast<const uint8_t*>(p.x) + (have ? src : 0) * src_bytes + (int64_t)j0 * kB;
    uint2* codes = reinterpret_cast<uint2*>(p.codes) + (int64_t)row * p.nblk + j0;
    const uint32_t pos = (uint32_t)tab.blk[g] * 128u + (row - (uint32_t)tab.off[g]);
    uint8_t* scales = p.scales + (int64_t)((pos >> 7) * p.kc) * 512 + (int64_t)(j0 >> 5) * 4096 + lane_scale +
                      (pos & 31) * 16 + ((pos >> 5) & 3) * 4;
    for (int j = j0; j < j_end; j += 32 * U) {
      Block16<kF32> B[U], C[kGlu ? U : 1];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        B[u] = Block16<kF32>{};
        if constexpr (kGlu) C[u] = Block16<kF32>{};
        if (j + 32 * u < j_end && have) {
          load_block_wide<kF32>(x + 32 * kB * u, B[u], wide);
          if constexpr (kGlu) load_block_wide<kF32>(x + 32 * kB * u + (int64_t)p.nblk * kB, C[u], wide);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int ju = j + 32 * u;
        if (ju >= j_end) break;
        float f[16], amax;
        block_floats<kF32>(B[u], f);
        if constexpr (kGlu) {
          float up[16];
          block_floats<kF32>(C[u], up);
          amax = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            f[i] = silu(f[i]) * up[i];
            amax = fmaxf(amax, fabsf(f[i]));
          }
          if (amax > FLT_MAX) {                 // a product beyond FP32 counts as the largest float
            amax = FLT_MAX;
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = fminf(fmaxf(f[i], -FLT_MAX), FLT_MAX);
          }
        } else {
          amax = block_amax<kF32>(B[u]);
        }
        uint32_t lo, hi;
        const uint32_t s = quantize_values(f, amax, gs, q, lo, hi);
        if (bounds_ok((uint64_t)((int64_t)row * p.nblk + ju + 1) * 8 <= p.codes_bytes, p.err))
          codes[32 * u] = make_uint2(lo, hi);
        uint8_t* sc = scales + 4096 * u;
        if (bounds_ok((uint64_t)(sc - p.scales) < p.scale_bytes, p.err)) *sc = (uint8_t)s;
        // K % 64 == 32: the row's last chunk has two padding slots
        if (ju == p.nblk - 1 && (p.nblk & 3) == 2 && bounds_ok((uint64_t)(sc + 2 - p.scales) < p.scale_bytes, p.err))
          sc[1] = sc[2] = 0;
      }
      x += 32 * kB * U;
      codes += 32 * U;
      scales += 4096 * U;
    }
  }
}

namespace {

// Activation rows of a tile: 128 while groups are small (each CTA then keeps
// 7 pipeline stages instead of 4 in flight, which is what streams weights),
// 256 once they fill it.  The host knows only the mean rows of a group.  Both
// measured with 64 experts of 2048 x 5120, skewed groups: 8 rows a group on
// average 70.4 (128) and 80.1 us (256), 64 rows 82.0 and 84.3, 128 rows 105.6
// and 96.3, 187 rows 132 and 104.
bool grouped_small(int64_t T, int64_t E) { return T < 128 * E; }

template <int BN>
cudaError_t launch_grouped(GroupedGemmParams& p, const uint8_t* a_scales, const uint8_t* w_scales, int64_t a_blocks,
                           int64_t w_blocks, const DeviceInfo* d, cudaStream_t st, bool f32) {
  using C = Cfg<BN, false, 0, false, true, true>;
  if (!make_sf_map(&p.tmap_sfa, w_scales, w_blocks * 128, p.kc, C::kChunks) ||
      !make_sf_map(&p.tmap_sfb, a_scales, a_blocks * 128, p.kc, C::kChunks))
    return cudaErrorInvalidValue;
  // a pair of CTAs for each pair of SMs, but no more than there can be tiles
  // (the host does not know the offsets)
  const int64_t tiles = (p.M + (BN - 1) * (p.E < p.M ? p.E : p.M)) / BN * p.tiles_p;
  const int grid = 2 * (int)(tiles < d->sm_count / 2 ? tiles : d->sm_count / 2);
  return f32 ? launch<BN, false, true, 0, false, true, true>(p, d, st, grid, 2)
             : launch<BN, false, false, 0, false, true, true>(p, d, st, grid, 2);
}

nvfp4_status run_grouped_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const float* ga, const uint8_t* w_codes,
                              const uint8_t* w_scales, const float* gw, const int32_t* offsets, int E, int64_t T,
                              int64_t N, int64_t K, void* out, bool f32, const DeviceInfo* d, cudaStream_t st) {
  GroupedGemmParams p;
  std::memset(&p, 0, sizeof(p));
  p.err = d->err_word;
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = drain_timeout_ns();
  p.M = T;
  p.N = N;
  p.offsets = offsets;
  p.ga = ga;
  p.gw = gw;
  p.E = E;
  p.w_blocks = (int)ceil_div(N, 128);
  p.kc = (int)ceil_div(K, 64);
  p.kmma = p.kc;
  p.out = out;
  p.out_elems = (uint64_t)T * (uint64_t)N;
  const int64_t a_blocks = grouped_blocks(T, E), w_blocks = (int64_t)E * p.w_blocks;
  const uint64_t a_sf = (uint64_t)a_blocks * p.kc * kSfChunk, w_sf = (uint64_t)w_blocks * p.kc * kSfChunk;
  // the weight is P, 128 rows a CTA; the activations are Q
  p.rows_p = (int)(E * N);
  p.rows_q = (int)T;
  p.sf_p = w_scales;
  p.sf_q = a_scales;
  p.sf_p_bytes = w_sf;
  p.sf_q_bytes = a_sf;
  p.rb_q = (int)a_blocks;
  using C = Cfg<256, false, 0, false, true, true>;
  p.kt = (int)ceil_div(K, 64 * C::kKB);
  p.tiles_p = (int)ceil_div(N, 256);
  p.group_p = C::kGroupTiles;
  p.tma_store = (N * (f32 ? 4 : 2)) % 16 == 0 ? 1 : 0;      // output rows start on 16-byte boundaries
  if (p.tma_store && !make_out_map(&p.tmap_out, out, T, N, f32, f32 ? 32 : 64)) return NVFP4_ERR_CUDA;
  if (!make_code_map(&p.tmap_p, w_codes, p.rows_p, K, kBM, C::kRowBytes)) return NVFP4_ERR_CUDA;
  for (int i = 0; i < 4; ++i)
    if (!make_code_map(&p.tmap_q_box[i], a_codes, T, K, 16 << i, C::kRowBytes)) return NVFP4_ERR_CUDA;
  p.tmap_q = p.tmap_q_box[3];
  return cuda_status(grouped_small(T, E) ? launch_grouped<128>(p, a_scales, w_scales, a_blocks, w_blocks, d, st, f32)
                                         : launch_grouped<256>(p, a_scales, w_scales, a_blocks, w_blocks, d, st, f32));
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_grouped_scale_bytes(int64_t T, int n_groups, int64_t K) {
  if (T < 1 || n_groups < 1 || n_groups > NVFP4_MAX_GROUPS || K < 16 || K % 16 != 0) return 0;
  return (size_t)(grouped_blocks(T, n_groups) * ceil_div(K, 64) * 512);
}

nvfp4_status nvfp4_grouped_quantize(const void* x, nvfp4_in_dtype dtype, nvfp4_act act, int64_t M, int64_t K,
                                    const int32_t* row_index, const int32_t* group_offsets, int n_groups, int64_t T,
                                    const float* global_scales, uint8_t* codes, uint8_t* block_scales,
                                    nvfp4_stream_t stream) {
  if (!x || !group_offsets || !global_scales || !codes || !block_scales) return NVFP4_ERR_INVALID_ARG;
  if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
  if (act != NVFP4_ACT_NONE && act != NVFP4_ACT_SWIGLU) return NVFP4_ERR_INVALID_ARG;
  if (M < 1 || T < 1 || K < 32 || K % 32 != 0 || n_groups < 1) return NVFP4_ERR_INVALID_ARG;
  if (!row_index && M < T) return NVFP4_ERR_INVALID_ARG;
  if (n_groups > NVFP4_MAX_GROUPS || T > (1ll << 31) - 256 || M > (1ll << 31) - 256 || K > (1ll << 31) ||
      grouped_blocks(T, n_groups) * 128 >= (1ll << 32) || grouped_blocks(T, n_groups) * ceil_div(K, 64) >= (1ll << 32) ||
      T * (K / 16) >= (1ll << 31) - (1ll << 20))
    return NVFP4_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(block_scales)) return NVFP4_ERR_ALIGNMENT;
  if (!aligned4(row_index) || !aligned4(group_offsets) || !aligned4(global_scales)) return NVFP4_ERR_ALIGNMENT;
  const DeviceInfo* d = device_info();
  if (!d) return NVFP4_ERR_CUDA;
  if (d->major != 10) return NVFP4_ERR_UNSUPPORTED;
  GroupedQuantParams p;
  p.x = x;
  p.M = M;
  p.row_index = row_index;
  p.offsets = group_offsets;
  p.E = n_groups;
  p.T = T;
  // a warp an item: whole rows if they give every SM some 32 warps, else parts
  // of them
  p.nblk = (int)(K / 16);
  const int64_t nseg = ceil_div(p.nblk, 32), warps = (int64_t)d->sm_count * 32;
  p.seg = (int)(T * nseg / warps < 1 ? 1 : T * nseg / warps < nseg ? T * nseg / warps : nseg);
  p.parts = (int)ceil_div(nseg, p.seg);
  p.div_parts = make_div((uint32_t)p.parts);
  p.gs = global_scales;
  p.codes = codes;
  p.scales = block_scales;
  p.kc = (uint32_t)ceil_div(K, 64);
  p.codes_bytes = (uint64_t)T * (uint64_t)(K / 2);
  p.scale_bytes = nvfp4_grouped_scale_bytes(T, n_groups, K);
  p.wide = (reinterpret_cast<uintptr_t>(x) & 31) == 0;
  p.err = d->err_word;
  const int64_t want = ceil_div(T * p.parts, 8), cap = (int64_t)d->sm_count * kQuantCtas;
  const int grid = (int)(want < cap ? want : cap);
  cudaStream_t st = (cudaStream_t)stream;
  const bool f32 = dtype == NVFP4_IN_F32, glu = act == NVFP4_ACT_SWIGLU;
  cudaError_t e;
  if (f32) e = glu ? launch_pdl(grouped_quantize_kernel<true, true>, grid, 256, st, p)
                   : launch_pdl(grouped_quantize_kernel<true, false>, grid, 256, st, p);
  else e = glu ? launch_pdl(grouped_quantize_kernel<false, true>, grid, 256, st, p)
               : launch_pdl(grouped_quantize_kernel<false, false>, grid, 256, st, p);
  return cuda_status(e);
}

nvfp4_status nvfp4_grouped_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_global_scales,
                                const uint8_t* w_codes, const uint8_t* w_scales, const float* w_global_scales,
                                const int32_t* group_offsets, int n_groups, int64_t T, int64_t N, int64_t K, void* out,
                                nvfp4_out_dtype out_dtype, nvfp4_stream_t stream) {
  if (!a_codes || !a_scales || !a_global_scales || !w_codes || !w_scales || !w_global_scales || !group_offsets || !out)
    return NVFP4_ERR_INVALID_ARG;
  if (T < 1 || N < 1 || K < 32 || K % 32 != 0 || n_groups < 1) return NVFP4_ERR_INVALID_ARG;
  if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_F32) return NVFP4_ERR_INVALID_ARG;
  // coordinates of the stacked weight and of its scale chunks, and tile
  // counts, are 32-bit
  const int64_t lim = (1ll << 31) - 65536;
  if (n_groups > NVFP4_MAX_GROUPS || T > lim || N > lim / n_groups || K > lim ||
      (int64_t)n_groups * ceil_div(N, 128) > lim / ceil_div(K, 64) ||
      grouped_blocks(T, n_groups) > lim / ceil_div(K, 64) ||
      (T / 128 + n_groups) * ceil_div(N, 256) > lim / 2)
    return NVFP4_ERR_UNSUPPORTED;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(out))
    return NVFP4_ERR_ALIGNMENT;
  if (!aligned4(a_global_scales) || !aligned4(w_global_scales) || !aligned4(group_offsets)) return NVFP4_ERR_ALIGNMENT;
  const DeviceInfo* d = device_info();
  if (!d) return NVFP4_ERR_CUDA;
  if (d->major != 10) return NVFP4_ERR_UNSUPPORTED;
  return run_grouped_gemm(a_codes, a_scales, a_global_scales, w_codes, w_scales, w_global_scales, group_offsets,
                          n_groups, T, N, K, out, out_dtype == NVFP4_OUT_F32, d, (cudaStream_t)stream);
}

}  // extern "C"
