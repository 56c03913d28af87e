// Host side of the block-scaled GEMM entry points (nvfp4_gemm, nvfp4_linear,
// nvfp4_fused_proj, nvfp4_mx_gemm, nvfp4_gemm_noalloc) and of their K-split
// workspaces; the kernel is in gemm_kernel.cuh.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include "common.h"
#include "gemm_host.h"
#include "gemm_kernel.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

// Memory the caller declared read-only for the duration of library calls
// (nvfp4_declare_static): a GEMM whose weight codes and scales lie inside it
// loads its first weight stages before waiting on the preceding kernel.
std::mutex g_static_mu;
std::vector<std::pair<uintptr_t, uintptr_t>> g_static_ranges;   // [begin, end)

bool is_static(const void* p, size_t bytes) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p), e = b + bytes;
  std::lock_guard<std::mutex> lock(g_static_mu);
  for (const auto& r : g_static_ranges)
    if (b >= r.first && e <= r.second) return true;
  return false;
}

std::mutex g_ws_mu;
std::map<std::pair<int, cudaStream_t>, Workspace> g_ws_table;

// CTAs of a swapped GEMM's grid, at most (Cfg::kGridPerSm per SM; the
// NVFP4 bound, which also covers the MXFP4 grid).
int64_t swap_grid_cap(const DeviceInfo* d, int bn) { return (int64_t)d->sm_count * (bn <= 16 ? 2 : 1); }

}  // namespace

size_t workspace_need(const DeviceInfo* d, int bn) {
  return (size_t)2 * (size_t)swap_grid_cap(d, bn) * (size_t)bn * kBM * sizeof(uint64_t);
}

cudaError_t get_workspace(const DeviceInfo* d, cudaStream_t st, int bn, Workspace* out) {
  std::lock_guard<std::mutex> lock(g_ws_mu);
  auto it = g_ws_table.find({d->device, st});
  if (it != g_ws_table.end()) {
    if (it->second.bytes < workspace_need(d, bn)) return cudaErrorInvalidValue;   // a registered one too small
    *out = it->second;
    return cudaSuccess;
  }
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) return cudaErrorNotPermitted;
  Workspace w;
  w.bytes = workspace_need(d, 128);
  w.owned = true;
  cudaError_t e = cudaMalloc(&w.ws, w.bytes);
  if (e != cudaSuccess) return e;
  // on the call's own stream: the default stream's work is not ordered before a
  // kernel on a non-blocking one, and words cleared under a running kernel are
  // partials that its adders wait for
  e = cudaMemsetAsync(w.ws, 0, w.bytes, st);
  if (e != cudaSuccess) {
    cudaFree(w.ws);
    return e;
  }
  g_ws_table[{d->device, st}] = w;
  *out = w;
  return cudaSuccess;
}

namespace {

float alpha_of(float ga, float gw) { return (float)(1.0 / ((double)ga * (double)gw)); }

template <bool MX>
cudaError_t launch_shape(const GemmParams& p, const DeviceInfo* d, cudaStream_t st, bool swap, int bn, bool f32) {
  if (!swap) {
    // CTA pairs: 256 x 256 tiles, a persistent grid of whole pairs
    const int64_t tiles = (int64_t)p.tiles_p * p.tiles_q;
    const int pairs = (int)(tiles < d->sm_count / 2 ? tiles : d->sm_count / 2);
    return f32 ? launch<256, false, true, 0, MX, true>(p, d, st, 2 * pairs, 2)
               : launch<256, false, false, 0, MX, true>(p, d, st, 2 * pairs, 2);
  }
  if (bn == 16) return f32 ? launch<16, true, true, 0, MX>(p, d, st) : launch<16, true, false, 0, MX>(p, d, st);
  if (bn == 32) return f32 ? launch<32, true, true, 0, MX>(p, d, st) : launch<32, true, false, 0, MX>(p, d, st);
  if (bn == 64) return f32 ? launch<64, true, true, 0, MX>(p, d, st) : launch<64, true, false, 0, MX>(p, d, st);
  return f32 ? launch<128, true, true, 0, MX>(p, d, st) : launch<128, true, false, 0, MX>(p, d, st);
}

// mx: MXFP4 operands (E8M0 scales of 32-element blocks, in the same chunk
// order with 4 scales = 128 K-elements per chunk); the caller passes unit
// global scales, so alpha = 1.
nvfp4_status run_gemm(const uint8_t* a_codes, const uint8_t* a_scales, float ga, const uint8_t* w_codes,
                      const uint8_t* w_scales, const int64_t* seg_offsets, const float* seg_gs, int n_seg,
                      int64_t M, int64_t N, int64_t K, void* out, nvfp4_out_dtype out_dtype, cudaStream_t st,
                      bool mx = false, int test_stall = 0) {
  if (!a_codes || !a_scales || !w_codes || !w_scales || !out) return NVFP4_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 32 || K % 32 != 0) return NVFP4_ERR_INVALID_ARG;
  if (M > (1ll << 31) - 256 || N > (1ll << 31) - 256 || K > (1ll << 31)) return NVFP4_ERR_UNSUPPORTED;
  if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_F32) return NVFP4_ERR_INVALID_ARG;
  if (!finite_positive(ga)) return NVFP4_ERR_INVALID_ARG;
  if (n_seg < 1 || n_seg > NVFP4_MAX_SEGMENTS) return NVFP4_ERR_INVALID_ARG;
  for (int i = 0; i < n_seg; ++i)
    if (!finite_positive(seg_gs[i]) || seg_offsets[i + 1] <= seg_offsets[i]) return NVFP4_ERR_INVALID_ARG;
  if (seg_offsets[0] != 0 || seg_offsets[n_seg] != N) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16(out))
    return NVFP4_ERR_ALIGNMENT;
  const DeviceInfo* d = device_info();
  if (!d) return NVFP4_ERR_CUDA;
  if (d->major != 10) return NVFP4_ERR_UNSUPPORTED;

  GemmParams p;
  std::memset(&p, 0, sizeof(p));
  const bool f32 = out_dtype == NVFP4_OUT_F32;
  p.err = d->err_word;
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = drain_timeout_ns();
  p.M = M;
  p.N = N;
  p.n_seg = n_seg;
  p.test_stall = test_stall;
  for (int i = 0; i < n_seg; ++i) {
    p.seg_end[i] = (int)seg_offsets[i + 1];
    p.seg_alpha[i] = alpha_of(ga, seg_gs[i]);
  }
  p.w_static = is_static(w_codes, (size_t)N * (size_t)(K / 2)) &&
                       is_static(w_scales, nvfp4_scale_bytes(N, mx ? K / 2 : K, NVFP4_SF_TCGEN05))
                   ? 1 : 0;
  p.kc = (int)ceil_div(K, mx ? 128 : 64);
  p.kmma = (int)ceil_div(K, 64);
  p.out = out;
  const bool swap = M <= 128;
  int bn = 256;
  if (swap) bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  if (swap) {
    Workspace w;
    const cudaError_t e = get_workspace(d, st, bn, &w);
    if (e == cudaErrorNotPermitted) return NVFP4_ERR_UNSUPPORTED;
    if (e == cudaErrorInvalidValue) return NVFP4_ERR_INVALID_ARG;
    if (e != cudaSuccess) return cuda_status(e);
    p.ws = w.ws;
    p.ws_words = w.bytes / sizeof(uint64_t);
  }
  p.rows_p = (int)(swap ? N : M);
  p.rows_q = (int)(swap ? M : N);
  const uint8_t* codes_p = swap ? w_codes : a_codes;
  const uint8_t* codes_q = swap ? a_codes : w_codes;
  p.sf_p = swap ? w_scales : a_scales;
  p.sf_q = swap ? a_scales : w_scales;
  const int kkb = swap ? Cfg<16, true>::kKB : Cfg<256, false>::kKB;
  // normal tiles run as CTA pairs: each CTA loads 128 rows of the 256-row
  // weight tile, and the scale chunks through tensor maps
  if (!make_code_map(&p.tmap_p, codes_p, p.rows_p, K, kBM, 32 * kkb) ||
      !make_code_map(&p.tmap_q, codes_q, p.rows_q, K, swap ? bn : kBM, 32 * kkb))
    return NVFP4_ERR_CUDA;
  if (!swap) {
    const int chunks = mx ? Cfg<256, false, 0, true>::kChunks : Cfg<256, false>::kChunks;
    if (!make_sf_map(&p.tmap_sfa, p.sf_p, p.rows_p, p.kc, chunks) ||
        !make_sf_map(&p.tmap_sfb, p.sf_q, p.rows_q, p.kc, chunks))
      return NVFP4_ERR_CUDA;
  }
  // TMA stores need 16-byte aligned output rows
  p.tma_store = (!swap && (N * (f32 ? 4 : 2)) % 16 == 0) ? 1 : 0;
  if (p.tma_store && !make_out_map(&p.tmap_out, out, M, N, f32)) return NVFP4_ERR_CUDA;
  p.rb_q = (int)ceil_div(p.rows_q, 128);
  p.sf_p_bytes = (uint64_t)ceil_div(p.rows_p, 128) * p.kc * kSfChunk;
  p.sf_q_bytes = (uint64_t)p.rb_q * p.kc * kSfChunk;
  p.out_elems = (uint64_t)M * (uint64_t)N;
  p.kt = (int)ceil_div(K, 64 * kkb);
  p.tiles_p = (int)ceil_div(p.rows_p, swap ? kBM : 2 * kBM);
  p.tiles_q = (int)ceil_div(p.rows_q, bn);
  p.group_p = swap ? kGroupP : kGroupP / 2;
  return cuda_status(mx ? launch_shape<true>(p, d, st, swap, bn, f32) : launch_shape<false>(p, d, st, swap, bn, f32));
}

// ---------------------------------------------------------------------------
// Allocation-free decode GEMM (nvfp4_gemm_noalloc).  Same kernel and same
// work split as the swapped (M <= 128) path of nvfp4_gemm, but its K-split
// scratch is a fixed array in this module's static device memory instead of
// the per-stream workspace nvfp4_gemm allocates on first use.  It serves
// callers that must not allocate device memory after start-up: a serving
// engine that measures its peak memory once and hands the remainder to its
// KV cache (a later allocation can fail or eat into that cache), and code
// that cannot afford the implicit device synchronisation cudaMalloc may
// perform.
//
// Limits (the scratch is sized for them; larger inputs are rejected with
// NVFP4_ERR_UNSUPPORTED): M <= 32, at most 160 SMs.  Scratch: tagged partial
// tiles, 2 slots x 160 CTAs x (32 x 128) 64-bit words = 10 MiB.  Every word
// must be empty (zero) when a launch starts: the array is zero-initialised
// when the module loads, each launch leaves every word it used empty, and
// after a launch that timed out nvfp4_last_device_error() clears it.
constexpr int kNoAllocMaxM = 32;
constexpr int kNoAllocMaxCtas = 160;
constexpr size_t kNoAllocScratchBytes = (size_t)2 * kNoAllocMaxCtas * kNoAllocMaxM * kBM * sizeof(uint64_t);

static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];

// The array's device address on each device, resolved on the first call on
// that device with it current.  Only a successful lookup is kept, so a lookup
// that failed (for example a lazy module load under memory pressure) is tried
// again on the next call.  The address is published with release order and
// read with acquire order (clear_gemm_scratch reads it from any thread).
struct NoAllocScratch {
  std::mutex mu;
  std::atomic<uint8_t*> ptr{nullptr};
};
NoAllocScratch g_noalloc[64];

uint8_t* noalloc_scratch_ptr(int device) {
  NoAllocScratch& sc = g_noalloc[device];
  uint8_t* p = sc.ptr.load(std::memory_order_acquire);
  if (p) return p;
  std::lock_guard<std::mutex> lock(sc.mu);
  p = sc.ptr.load(std::memory_order_relaxed);
  if (p) return p;
  void* addr = nullptr;
  if (cudaGetSymbolAddress(&addr, g_noalloc_scratch) != cudaSuccess || !addr) {
    (void)cudaGetLastError();
    return nullptr;
  }
  p = static_cast<uint8_t*>(addr);
  sc.ptr.store(p, std::memory_order_release);
  return p;
}

// Quantize X then multiply.  Given activation buffers, the quantize kernel
// writes (a_codes, a_scales) and the GEMM reads them.  Without them,
// decode-sized M runs as one kernel whose epilogue warps quantize X into
// shared memory before the first MMA.  (That one-kernel form measured slower
// than the two kernels on the decode shape: every CTA quantizes the part of
// X its K range needs, so X is quantized many times over, in four warps that
// cannot hide latency, whereas the quantize kernel spreads X over the whole
// GPU once.)
constexpr int kLinearMaxM = 32;

bool linear_fused_fits(const DeviceInfo* d, int64_t M, int64_t N, int64_t K) {
  if (M > kLinearMaxM) return false;
  const int bn = M <= 16 ? 16 : 32;
  const int64_t units = ceil_div(N, kBM) * ceil_div(K, 64 * Cfg<16, true>::kKB);
  // a cooperative grid may be as small as one CTA per SM (see launch())
  const int64_t cap = decode_cooperative() ? (int64_t)d->sm_count : swap_grid_cap(d, bn);
  const int64_t grid = units < cap ? units : cap;
  const int steps = bn == 16 ? Cfg<16, true, 1>::kActSteps : Cfg<32, true, 1>::kActSteps;
  return ceil_div(units, grid) <= steps;   // steps per CTA, at most
}

template <int BN, int QX>
cudaError_t launch_linear(const GemmParams& p, const DeviceInfo* d, cudaStream_t st, bool f32) {
  return f32 ? launch<BN, true, true, QX>(p, d, st) : launch<BN, true, false, QX>(p, d, st);
}

nvfp4_status run_linear(const void* x, nvfp4_in_dtype x_dtype, int64_t M, int64_t K, float ga, const uint8_t* w_codes,
                        const uint8_t* w_scales, float gw, int64_t N, void* out, nvfp4_out_dtype out_dtype,
                        uint8_t* a_codes, uint8_t* a_scales, cudaStream_t st) {
  if (!x || !w_codes || !w_scales || !out) return NVFP4_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 32 || K % 32 != 0) return NVFP4_ERR_INVALID_ARG;
  if (x_dtype != NVFP4_IN_BF16 && x_dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
  if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_F32) return NVFP4_ERR_INVALID_ARG;
  if (!finite_positive(ga) || !finite_positive(gw)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(out)) return NVFP4_ERR_ALIGNMENT;
  if (M > (1ll << 31) - 256 || N > (1ll << 31) - 256 || K > (1ll << 31)) return NVFP4_ERR_UNSUPPORTED;
  const DeviceInfo* d = device_info();
  if (!d) return NVFP4_ERR_CUDA;
  if (d->major != 10) return NVFP4_ERR_UNSUPPORTED;
  if ((a_codes && a_scales) || !linear_fused_fits(d, M, N, K)) {
    if (!a_codes || !a_scales) return NVFP4_ERR_INVALID_ARG;
    const nvfp4_status s1 = nvfp4_quantize(x, x_dtype, M, K, ga, a_codes, a_scales, NVFP4_SF_TCGEN05, nullptr, st);
    if (s1 != NVFP4_OK) return s1;
    return nvfp4_gemm(a_codes, a_scales, ga, w_codes, w_scales, gw, M, N, K, out, out_dtype, st);
  }
  GemmParams p;
  std::memset(&p, 0, sizeof(p));
  const int bn = M <= 16 ? 16 : 32;
  Workspace w;
  const cudaError_t e0 = get_workspace(d, st, bn, &w);
  if (e0 == cudaErrorNotPermitted) return NVFP4_ERR_UNSUPPORTED;
  if (e0 == cudaErrorInvalidValue) return NVFP4_ERR_INVALID_ARG;
  if (e0 != cudaSuccess) return cuda_status(e0);
  p.ws = w.ws;
  p.ws_words = w.bytes / sizeof(uint64_t);
  constexpr int kkb = Cfg<16, true>::kKB;
  p.rows_p = (int)N;
  p.rows_q = (int)M;
  p.sf_p = w_scales;
  p.sf_q = nullptr;
  if (!make_code_map(&p.tmap_p, w_codes, p.rows_p, K, kBM, 32 * kkb)) return NVFP4_ERR_CUDA;
  p.tmap_q = p.tmap_p;                      // not read (X is quantized in the kernel)
  p.w_static = is_static(w_codes, (size_t)N * (size_t)(K / 2)) &&
                       is_static(w_scales, nvfp4_scale_bytes(N, K, NVFP4_SF_TCGEN05))
                   ? 1 : 0;
  p.out = out;
  p.tma_store = 0;
  p.err = d->err_word;
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = drain_timeout_ns();
  p.M = M;
  p.N = N;
  p.rb_q = 1;
  p.kc = (int)ceil_div(K, 64);
  p.kmma = (int)ceil_div(K, 64);
  p.kt = (int)ceil_div(K, 64 * kkb);
  p.tiles_p = (int)ceil_div(p.rows_p, kBM);
  p.tiles_q = 1;
  p.n_seg = 1;
  p.seg_end[0] = (int)N;
  p.seg_alpha[0] = alpha_of(ga, gw);
  p.x = x;
  p.x_gs = ga;
  p.K = K;
  p.sf_p_bytes = (uint64_t)ceil_div(N, 128) * p.kc * kSfChunk;
  p.out_elems = (uint64_t)M * (uint64_t)N;
  p.x_bytes = (uint64_t)M * (uint64_t)K * (x_dtype == NVFP4_IN_F32 ? 4 : 2);
  const bool f32 = out_dtype == NVFP4_OUT_F32;
  const bool xf32 = x_dtype == NVFP4_IN_F32;
  cudaError_t e;
  if (bn == 16) e = xf32 ? launch_linear<16, 2>(p, d, st, f32) : launch_linear<16, 1>(p, d, st, f32);
  else e = xf32 ? launch_linear<32, 2>(p, d, st, f32) : launch_linear<32, 1>(p, d, st, f32);
  return cuda_status(e);
}

}  // namespace

// After a launch whose bounded wait ran out, partial words may be left full;
// empty every K-split scratch of the current device (library workspaces and
// the allocation-free scratch).  Synchronous.
cudaError_t clear_gemm_scratch(int device) {
  cudaError_t first = cudaSuccess;
  {
    std::lock_guard<std::mutex> lock(g_ws_mu);
    for (auto& kv : g_ws_table)
      if (kv.first.first == device) {
        const cudaError_t e = cudaMemset(kv.second.ws, 0, kv.second.bytes);
        if (first == cudaSuccess) first = e;
      }
  }
  uint8_t* na = device >= 0 && device < 64 ? g_noalloc[device].ptr.load(std::memory_order_acquire) : nullptr;
  if (na) {
    const cudaError_t e = cudaMemset(na, 0, kNoAllocScratchBytes);
    if (first == cudaSuccess) first = e;
  }
  const cudaError_t e = cudaDeviceSynchronize();
  return first == cudaSuccess ? e : first;
}

namespace {

nvfp4_status run_gemm_noalloc(const uint8_t* a_codes, const uint8_t* a_scales, float ga, const uint8_t* w_codes,
                              const uint8_t* w_scales, float gw, int64_t M, int64_t N, int64_t K, void* out,
                              nvfp4_out_dtype out_dtype, cudaStream_t st, int test_stall = 0) {
  if (!a_codes || !a_scales || !w_codes || !w_scales || !out) return NVFP4_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 32 || K % 32 != 0) return NVFP4_ERR_INVALID_ARG;
  if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_F32) return NVFP4_ERR_INVALID_ARG;
  if (!finite_positive(ga) || !finite_positive(gw)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16(out))
    return NVFP4_ERR_ALIGNMENT;
  if (M > kNoAllocMaxM || N > (1ll << 31) - 256 || K > (1ll << 31)) return NVFP4_ERR_UNSUPPORTED;
  const DeviceInfo* d = device_info();
  if (!d) return NVFP4_ERR_CUDA;
  if (d->major != 10 || d->sm_count > kNoAllocMaxCtas || d->device >= 64) return NVFP4_ERR_UNSUPPORTED;
  // with this device current (device_info() reads the current device): the
  // scratch array's address on it, looked up once and then cached
  uint8_t* scratch = noalloc_scratch_ptr(d->device);
  if (!scratch) return NVFP4_ERR_CUDA;

  GemmParams p;
  std::memset(&p, 0, sizeof(p));
  const int bn = M <= 16 ? 16 : 32;
  // the grid's partial slots fit the scratch: 2 x (2 x SMs) x 16 x 128 words
  // for bn = 16, 2 x SMs x 32 x 128 for bn = 32; both fit for <= 160 SMs
  if (workspace_need(d, bn) > kNoAllocScratchBytes) return NVFP4_ERR_UNSUPPORTED;
  p.ws = reinterpret_cast<uint64_t*>(scratch);
  p.ws_words = kNoAllocScratchBytes / sizeof(uint64_t);
  p.rows_p = (int)N;
  p.rows_q = (int)M;
  p.sf_p = w_scales;
  p.sf_q = a_scales;
  constexpr int kkb = Cfg<16, true>::kKB;
  if (!make_code_map(&p.tmap_p, w_codes, p.rows_p, K, kBM, 32 * kkb) ||
      !make_code_map(&p.tmap_q, a_codes, p.rows_q, K, bn, 32 * kkb))
    return NVFP4_ERR_CUDA;
  p.out = out;
  p.tma_store = 0;
  p.err = d->err_word;
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = drain_timeout_ns();
  p.M = M;
  p.N = N;
  p.rb_q = (int)ceil_div(p.rows_q, 128);
  p.kc = (int)ceil_div(K, 64);
  p.kmma = (int)ceil_div(K, 64);
  p.kt = (int)ceil_div(K, 64 * kkb);
  p.tiles_p = (int)ceil_div(p.rows_p, kBM);
  p.tiles_q = 1;
  p.n_seg = 1;
  p.test_stall = test_stall;
  p.seg_end[0] = (int)N;
  p.seg_alpha[0] = alpha_of(ga, gw);
  p.sf_p_bytes = (uint64_t)ceil_div(N, 128) * p.kc * kSfChunk;
  p.sf_q_bytes = (uint64_t)p.rb_q * p.kc * kSfChunk;
  p.out_elems = (uint64_t)M * (uint64_t)N;
  cudaError_t e;
  const bool f32 = out_dtype == NVFP4_OUT_F32;
  if (bn == 16) e = f32 ? launch<16, true, true>(p, d, st) : launch<16, true, false>(p, d, st);
  else e = f32 ? launch<32, true, true>(p, d, st) : launch<32, true, false>(p, d, st);
  return cuda_status(e);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status nvfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, float a_global_scale,
                        const uint8_t* w_codes, const uint8_t* w_scales, float w_global_scale, int64_t M, int64_t N,
                        int64_t K, void* out, nvfp4_out_dtype out_dtype, nvfp4_stream_t stream) {
  const int64_t offs[2] = {0, N};
  const float gs[1] = {w_global_scale};
  return run_gemm(a_codes, a_scales, a_global_scale, w_codes, w_scales, offs, gs, 1, M, N, K, out, out_dtype,
                  (cudaStream_t)stream);
}

size_t nvfp4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 32 || K % 32 != 0) return 0;
  if (M > 128) return 0;                              // normal tiles do not split K
  const DeviceInfo* d = device_info();
  if (!d) return 0;
  const int bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  return workspace_need(d, bn);
}

nvfp4_status nvfp4_set_workspace(nvfp4_stream_t stream, void* workspace, size_t bytes) {
  const DeviceInfo* d = device_info();
  if (!d) return NVFP4_ERR_CUDA;
  const cudaStream_t st = (cudaStream_t)stream;
  std::lock_guard<std::mutex> lock(g_ws_mu);
  auto it = g_ws_table.find({d->device, st});
  if (it != g_ws_table.end() && it->second.owned) {
    // a workspace the library allocated earlier for this stream: freed once
    // the device is idle
    if (cudaDeviceSynchronize() != cudaSuccess) return cuda_status(cudaGetLastError());
    cudaFree(it->second.ws);
    g_ws_table.erase(it);
  } else if (it != g_ws_table.end()) {
    g_ws_table.erase(it);
  }
  if (!workspace) return bytes == 0 ? NVFP4_OK : NVFP4_ERR_INVALID_ARG;   // unregistered
  if (!aligned16(workspace)) return NVFP4_ERR_ALIGNMENT;
  if (bytes < workspace_need(d, 16)) return NVFP4_ERR_INVALID_ARG;
  Workspace w;
  w.ws = static_cast<uint64_t*>(workspace);
  w.bytes = bytes;
  w.owned = false;
  g_ws_table[{d->device, st}] = w;
  return NVFP4_OK;
}

nvfp4_status nvfp4_release_workspaces(void) {
  const DeviceInfo* d = device_info();
  if (!d) return NVFP4_ERR_CUDA;
  if (cudaDeviceSynchronize() != cudaSuccess) return cuda_status(cudaGetLastError());
  std::lock_guard<std::mutex> lock(g_ws_mu);
  for (auto it = g_ws_table.begin(); it != g_ws_table.end();) {
    if (it->first.first == d->device && it->second.owned) {
      cudaFree(it->second.ws);
      it = g_ws_table.erase(it);
    } else {
      ++it;
    }
  }
  return NVFP4_OK;
}

nvfp4_status nvfp4_declare_static(const void* base, size_t bytes) {
  if (!base || bytes == 0) return NVFP4_ERR_INVALID_ARG;
  const uintptr_t b = reinterpret_cast<uintptr_t>(base);
  std::lock_guard<std::mutex> lock(g_static_mu);
  g_static_ranges.emplace_back(b, b + bytes);
  return NVFP4_OK;
}

void nvfp4_forget_static(void) {
  std::lock_guard<std::mutex> lock(g_static_mu);
  g_static_ranges.clear();
}

nvfp4_status nvfp4_linear(const void* x, nvfp4_in_dtype x_dtype, int64_t M, int64_t K, float a_global_scale,
                          const uint8_t* w_codes, const uint8_t* w_scales, float w_global_scale, int64_t N, void* out,
                          nvfp4_out_dtype out_dtype, uint8_t* a_codes, uint8_t* a_scales, nvfp4_stream_t stream) {
  return run_linear(x, x_dtype, M, K, a_global_scale, w_codes, w_scales, w_global_scale, N, out, out_dtype, a_codes,
                    a_scales, (cudaStream_t)stream);
}

nvfp4_status nvfp4_fused_proj(const uint8_t* a_codes, const uint8_t* a_scales, float a_global_scale,
                              const uint8_t* w_codes, const uint8_t* w_scales, const int64_t* seg_offsets,
                              const float* seg_global_scales, int n_seg, int64_t M, int64_t K, void* out,
                              nvfp4_out_dtype out_dtype, nvfp4_stream_t stream) {
  if (!seg_offsets || !seg_global_scales || n_seg < 1 || n_seg > NVFP4_MAX_SEGMENTS) return NVFP4_ERR_INVALID_ARG;
  return run_gemm(a_codes, a_scales, a_global_scale, w_codes, w_scales, seg_offsets, seg_global_scales, n_seg, M,
                  seg_offsets[n_seg], K, out, out_dtype, (cudaStream_t)stream);
}

nvfp4_status nvfp4_mx_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                           const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, void* out,
                           nvfp4_out_dtype out_dtype, nvfp4_stream_t stream) {
  const int64_t offs[2] = {0, N};
  const float unit[1] = {1.0f};
  return run_gemm(a_codes, a_scales, 1.0f, w_codes, w_scales, offs, unit, 1, M, N, K, out, out_dtype,
                  (cudaStream_t)stream, /*mx=*/true);
}

nvfp4_status nvfp4_gemm_noalloc(const uint8_t* a_codes, const uint8_t* a_scales, float a_global_scale,
                                const uint8_t* w_codes, const uint8_t* w_scales, float w_global_scale, int64_t M,
                                int64_t N, int64_t K, void* out, nvfp4_out_dtype out_dtype, nvfp4_stream_t stream) {
  return run_gemm_noalloc(a_codes, a_scales, a_global_scale, w_codes, w_scales, w_global_scale, M, N, K, out,
                          out_dtype, (cudaStream_t)stream);
}

nvfp4_status nvfp4_test_gemm_stalled_reduction(const uint8_t* a_codes, const uint8_t* a_scales, float a_global_scale,
                                               const uint8_t* w_codes, const uint8_t* w_scales, float w_global_scale,
                                               int64_t M, int64_t N, int64_t K, void* out, nvfp4_out_dtype out_dtype,
                                               int noalloc, nvfp4_stream_t stream) {
  if (M > 128) return NVFP4_ERR_UNSUPPORTED;                 // only decode tiles split K
  if (noalloc)
    return run_gemm_noalloc(a_codes, a_scales, a_global_scale, w_codes, w_scales, w_global_scale, M, N, K, out,
                            out_dtype, (cudaStream_t)stream, /*test_stall=*/1);
  const int64_t offs[2] = {0, N};
  const float gs[1] = {w_global_scale};
  return run_gemm(a_codes, a_scales, a_global_scale, w_codes, w_scales, offs, gs, 1, M, N, K, out, out_dtype,
                  (cudaStream_t)stream, /*mx=*/false, /*test_stall=*/1);
}

}  // extern "C"
