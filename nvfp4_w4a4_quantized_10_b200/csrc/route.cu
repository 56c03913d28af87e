// Router of an expert layer: top-k experts of each token with softmax
// weights, and the counting sort of the (token, expert) pairs by expert that
// the grouped products read.
//
//   x_e = logit (NaN -> -inf, +inf -> the largest float)
//   id_j = the j-th largest finite x, ties to the lowest index
//   w_j = exp(x_id_j - x_max) / sum, over all E experts or over the selected
//   slot(m, e) = offset_e + #{m' < m : m' selects e}
//
// Both kernels are latency-bound: the bytes (logits once, 16 per pair) take a
// microsecond or two at any size met in serving.
//
// Selection: one warp a token, each lane holding E / 32 logits as ordered
// 32-bit keys; a round is one warp-wide integer maximum for the key and one
// minimum for the index (redux), so ties need no extra pass.
// Sort: an expert is taken at most once by a token, so the rank of (m, e) is
// a population count: 128 tokens set one bit each in a 128-bit mask of every
// expert (an OR is order-free, so the result does not depend on timing), and
// a pair's rank is the number of bits below its own.  Each CTA counts a
// contiguous run of tokens; the second kernel adds up the runs before it.  A
// call with few tokens runs as one CTA of one launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "common.h"
#include "groups.cuh"
#include "ptx.cuh"

namespace nvfp4 {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kSub = 128;               // tokens ranked at a time
constexpr int kMaxTopK = NVFP4_MAX_TOP_K;
constexpr int kRouteMaxChunks = 256;

struct RouteParams {
  const void* logits;
  int64_t M;
  int E, k;
  int renorm;
  int32_t* ids;
  float* weights;
  int32_t* slots;
  int32_t* row_index;
  int32_t* offsets;
  int32_t* hist;         // [chunks, E] pairs of each run of tokens
  int64_t chunk;         // tokens of a run
};

// Order-preserving key of a finite float; 0 for an expert that must not be
// taken (-inf, NaN).  -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

template <bool kF32>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  float x;
  if constexpr (kF32) x = __ldg(reinterpret_cast<const float*>(p) + i);
  else x = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p) + i) << 16);
  return x == INFINITY ? FLT_MAX : x;
}

// Exclusive prefix of `total` over the experts, by thread index (E <=
// blockDim.x): offset of expert threadIdx.x; `sum` the grand total.
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, s, d);
    if (lane >= d) s += u;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0;
  sum = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    const int u = warp_sums[w];
    if (w < warp) before += u;
    sum += u;
  }
  __syncthreads();
  return before + s - v;
}

template <bool kF32, int NV>
__global__ void __launch_bounds__(kRouteThreads) route_topk_kernel(const RouteParams p) {
  __shared__ uint32_t mask[kMaxGroups][kSub / 32];
  __shared__ int count[kMaxGroups];
  __shared__ int16_t ids_s[kSub * kMaxTopK];
  __shared__ int warp_sums[kRouteWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = p.E, k = p.k;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < E; i += kRouteThreads) count[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t m_begin = (int64_t)blockIdx.x * p.chunk;
  const int64_t m_end = m_begin + p.chunk < p.M ? m_begin + p.chunk : p.M;
  for (int64_t sub = m_begin; sub < m_end; sub += kSub) {
    const int n = (int)(m_end - sub < kSub ? m_end - sub : kSub);
    for (int i = threadIdx.x; i < E * (kSub / 32); i += kRouteThreads) (&mask[0][0])[i] = 0;
    __syncthreads();
    // the next token's logits are on their way while this one is selected
    float x[NV];
    auto load_token = [&](int ml) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        x[i] = ml < n && e < E ? load_logit<kF32>(p.logits, (sub + ml) * E + e) : -INFINITY;
      }
    };
    load_token(warp);
    for (int ml = warp; ml < n; ml += kRouteWarps) {
      const int64_t m = sub + ml;
      uint32_t key[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = order_key(x[i]);
      load_token(ml + kRouteWarps);
      // softmax over all experts: the sum before any is taken out
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) best = max(best, key[i]);
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
      const float x_max = top ? key_value(top) : 0.0f;
      float sum = 0.0f;
      if (!p.renorm) {
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += key[i] ? expf(key_value(key[i]) - x_max) : 0.0f;
      }
      int my_id = -1;
      float my_e = 0.0f;
      for (int j = 0; j < k; ++j) {
        const uint32_t kmax = __reduce_max_sync(0xFFFFFFFFu, best);
        if (kmax == 0) break;                    // nothing left that may be taken
        uint32_t at = 0xFFFFFFFFu;
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
          if (key[i] == kmax) at = lane + 32 * i;
        at = __reduce_min_sync(0xFFFFFFFFu, at);
        if (lane == j) {
          my_id = (int)at;
          my_e = expf(key_value(kmax) - x_max);
        }
        if ((at & 31) == (uint32_t)lane) {
          best = 0;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (lane + 32 * i == (int)at) key[i] = 0;
            best = max(best, key[i]);
          }
        }
      }
      if (p.renorm) sum = my_e;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      if (lane < k) {
        p.ids[m * k + lane] = my_id;
        p.weights[m * k + lane] = my_id >= 0 ? __fdiv_rn(my_e, sum) : 0.0f;
        ids_s[ml * k + lane] = (int16_t)my_id;
        if (my_id >= 0) atomicOr(&mask[my_id][ml >> 5], 1u << (ml & 31));
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * k; i += kRouteThreads) {
      const int ml = i / k, e = ids_s[i];
      int rank = -1;
      if (e >= 0) {
        rank = count[e];
#pragma unroll
        for (int w = 0; w < kSub / 32; ++w) {
          const uint32_t below = w < (ml >> 5) ? 0xFFFFFFFFu : w == (ml >> 5) ? (1u << (ml & 31)) - 1u : 0u;
          rank += __popc(mask[e][w] & below);
        }
      }
      p.slots[sub * k + i] = rank;               // rank inside this run of tokens
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      int c = 0;
#pragma unroll
      for (int w = 0; w < kSub / 32; ++w) c += __popc(mask[e][w]);
      count[e] += c;
    }
    __syncthreads();
  }
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < E; e += kRouteThreads) p.hist[(int64_t)blockIdx.x * E + e] = count[e];
    return;
  }
  // the only CTA: ranks become slots here
  int total;
  const int off = block_exclusive((int)threadIdx.x < E ? count[threadIdx.x] : 0, warp_sums, total);
  if ((int)threadIdx.x < E) {
    count[threadIdx.x] = off;
    p.offsets[threadIdx.x] = off;
  }
  if (threadIdx.x == 0) p.offsets[E] = total;
  __syncthreads();
  const int pairs = (int)(p.M * k);
  for (int i = threadIdx.x; i < pairs; i += kRouteThreads) {
    const int e = p.ids[i];
    if (e >= 0) {
      const int s = count[e] + p.slots[i];
      p.slots[i] = s;
      p.row_index[s] = i / k;
    }
    if (i >= total) p.row_index[i] = -1;
  }
}

// Second launch of a call with more than one run of tokens: every CTA adds up
// all runs' counts (for the offsets) and those before its own (for its base),
// then turns its ranks into slots.  E <= blockDim.x; blockDim.x / ep threads
// share an expert, ep the power of two >= E.
__global__ void __launch_bounds__(kRouteThreads) route_slots_kernel(const RouteParams p, int ep) {
  __shared__ int part[2][kRouteThreads];
  __shared__ int base[kMaxGroups];
  __shared__ int warp_sums[kRouteWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int E = p.E, k = p.k;
  const int64_t m_begin = (int64_t)blockIdx.x * p.chunk;
  const int64_t m_end = m_begin + p.chunk < p.M ? m_begin + p.chunk : p.M;
  const int i_end = (int)(m_end * k);
  int i = (int)(m_begin * k) + threadIdx.x;
  // the first pair of this thread is on its way while the counts are added up
  int id = -1, rank = 0;
  if (i < i_end) {
    id = __ldg(p.ids + i);
    rank = p.slots[i];
  }
  const int e = threadIdx.x & (ep - 1), q = threadIdx.x / ep, parts = kRouteThreads / ep;
  int all = 0, before = 0;
  if (e < E) {
#pragma unroll 8
    for (int c = q; c < (int)gridDim.x; c += parts) {
      const int h = __ldg(p.hist + (int64_t)c * E + e);
      all += h;
      if (c < (int)blockIdx.x) before += h;
    }
  }
  part[0][threadIdx.x] = all;
  part[1][threadIdx.x] = before;
  __syncthreads();
  all = before = 0;
  if ((int)threadIdx.x < E) {
    for (int i = 0; i < parts; ++i) {
      all += part[0][i * ep + threadIdx.x];
      before += part[1][i * ep + threadIdx.x];
    }
  }
  int total;
  const int off = block_exclusive(all, warp_sums, total);
  if ((int)threadIdx.x < E) {
    base[threadIdx.x] = off + before;
    if (blockIdx.x == 0) p.offsets[threadIdx.x] = off;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[E] = total;
  __syncthreads();
  while (i < i_end) {
    if (id >= 0) {
      const int at = base[id] + rank;
      p.slots[i] = at;
      p.row_index[at] = i / k;
    }
    if (i >= total) p.row_index[i] = -1;         // rows no pair fills
    i += kRouteThreads;
    if (i < i_end) {
      id = __ldg(p.ids + i);
      rank = p.slots[i];
    }
  }
}

namespace {

// Runs of tokens: one CTA up to 64 tokens (2 a warp: one launch), else at
// least 32 tokens a run, one for each warp, and at most one run an SM.
int64_t route_chunks(int64_t M, int sms) {
  if (M <= 64) return 1;
  const int64_t cap = sms < kRouteMaxChunks ? sms : kRouteMaxChunks;
  const int64_t c = ceil_div(M, kRouteWarps);
  return c < cap ? c : cap;
}

template <bool kF32>
cudaError_t launch_topk(const RouteParams& p, int grid, cudaStream_t st) {
  const int nv = (p.E + 31) / 32;
  if (nv <= 1) return launch_pdl(route_topk_kernel<kF32, 1>, grid, kRouteThreads, st, p);
  if (nv <= 2) return launch_pdl(route_topk_kernel<kF32, 2>, grid, kRouteThreads, st, p);
  if (nv <= 4) return launch_pdl(route_topk_kernel<kF32, 4>, grid, kRouteThreads, st, p);
  if (nv <= 8) return launch_pdl(route_topk_kernel<kF32, 8>, grid, kRouteThreads, st, p);
  return launch_pdl(route_topk_kernel<kF32, 16>, grid, kRouteThreads, st, p);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_route_workspace_bytes(int n_experts) {
  if (n_experts < 1 || n_experts > NVFP4_MAX_GROUPS) return 0;
  return (size_t)kRouteMaxChunks * (size_t)n_experts * sizeof(int32_t);
}

nvfp4_status nvfp4_route(const void* logits, nvfp4_in_dtype dtype, int64_t M, int n_experts, int top_k,
                         nvfp4_route_norm norm, int32_t* expert_ids, float* weights, int32_t* slots,
                         int32_t* row_index, int32_t* group_offsets, void* workspace, size_t workspace_bytes,
                         nvfp4_stream_t stream) {
  if (!logits || !expert_ids || !weights || !slots || !row_index || !group_offsets || !workspace)
    return NVFP4_ERR_INVALID_ARG;
  if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
  if (norm != NVFP4_ROUTE_SOFTMAX_ALL && norm != NVFP4_ROUTE_SOFTMAX_TOPK) return NVFP4_ERR_INVALID_ARG;
  if (M < 1 || n_experts < 1 || top_k < 1 || top_k > n_experts) return NVFP4_ERR_INVALID_ARG;
  if (n_experts > NVFP4_MAX_GROUPS || top_k > NVFP4_MAX_TOP_K || M > ((1ll << 31) - 65536) / top_k)
    return NVFP4_ERR_UNSUPPORTED;
  if (workspace_bytes < nvfp4_route_workspace_bytes(n_experts)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(expert_ids) || !aligned16(weights) || !aligned16(slots) ||
      !aligned16(row_index) || !aligned16(group_offsets) || !aligned16(workspace))
    return NVFP4_ERR_ALIGNMENT;
  const DeviceInfo* d = device_info();
  if (!d) return NVFP4_ERR_CUDA;
  if (d->major != 10) return NVFP4_ERR_UNSUPPORTED;
  RouteParams p;
  p.logits = logits;
  p.M = M;
  p.E = n_experts;
  p.k = top_k;
  p.renorm = norm == NVFP4_ROUTE_SOFTMAX_TOPK;
  p.ids = expert_ids;
  p.weights = weights;
  p.slots = slots;
  p.row_index = row_index;
  p.offsets = group_offsets;
  p.hist = static_cast<int32_t*>(workspace);
  p.chunk = ceil_div(M, route_chunks(M, d->sm_count));
  const int grid = (int)ceil_div(M, p.chunk);
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = dtype == NVFP4_IN_F32 ? launch_topk<true>(p, grid, st) : launch_topk<false>(p, grid, st);
  if (e == cudaSuccess && grid > 1) {
    int ep = 32;
    while (ep < n_experts) ep *= 2;
    e = launch_pdl(route_slots_kernel, grid, kRouteThreads, st, p, ep);
  }
  return cuda_status(e);
}

}  // extern "C"
