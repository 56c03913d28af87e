// Router of an expert layer: top-k experts of each token with softmax
// weights, and the counting sort of the (token, expert) pairs by expert that
// the grouped products read.
//
//   x_e = logit (NaN -> -inf, +inf -> the largest float)
//   id_j = the j-th largest finite x, ties to the lowest index
//   w_j = exp(x_id_j - x_max) / sum, over all E experts or over the selected
//   slot(m, e) = offset_e + #{m' < m : m' selects e}
//
// The bytes (logits once, 16 a pair) take a microsecond at any size met in
// serving.  8 tokens of 64 experts take 3.4 us, all latency.  16384 of 128, top
// 8, take 16.3 us: the first kernel's 550 warp instructions a token are 8 us of
// the machine's issue slots, which are busy 68 % of its time (each round of the
// selection waits for the one before); the second waits for ids and counts
// (issue slots 26 % busy).
//
// Selection: one warp a token, each lane holding E / 32 logits as ordered
// 32-bit keys; a round is one warp-wide integer maximum for the key and, for
// FP32 logits, one minimum for the index (redux), so ties need no extra pass.
// Sort: an expert is taken at most once by a token, so the rank of (m, e) is
// a population count: 128 tokens set one bit each in a 128-bit mask of every
// expert (an OR is order-free, so the result does not depend on timing), and
// a pair's rank is the number of bits below its own.  Each CTA counts a
// contiguous run of tokens; the second kernel adds up the runs before it.  A
// call with few tokens is one launch of one cluster, whose CTAs read one
// another's counts.
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
constexpr int kRouteCluster = 8;        // CTAs of a call that is one launch

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
  int32_t* hist;         // [chunks, hist_stride(E)] pairs of each run of tokens
  int64_t chunk;         // tokens of a run
};

// Order-preserving 32-bit key of a logit, 0 for an expert that must not be
// taken (-inf, NaN); -0 counts as +0, +inf as the largest float.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(fminf(__fadd_rn(x, 0.0f), FLT_MAX));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

// bf16 logits: the key's upper half says all (+inf keeps a key of its own,
// above the largest bf16), and the lower half holds the index, inverted, so
// that one maximum finds value and lowest index together.
__device__ __forceinline__ uint32_t order_key_bf16(float x, int e) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return ((b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) & 0xFFFF0000u) | (0xFFFFu - (uint32_t)e);
}

// Value of a key: bf16 keys of negative numbers have their lower half set; the
// key of +inf stands for the largest float, as in FP32.
template <bool kF32>
__device__ __forceinline__ float selected_value(uint32_t k) {
  if constexpr (kF32) return key_value(k);
  else return fminf(key_value(k & 0x80000000u ? k & 0xFFFF0000u : k | 0xFFFFu), FLT_MAX);
}

template <bool kF32>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (kF32) return reinterpret_cast<const float*>(p)[i];
  else return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

// Experts in a row of the counts of all runs: rows start on 16 bytes.
__host__ __device__ constexpr int hist_stride(int E) { return (E + 3) & ~3; }

__device__ __forceinline__ int ld_cluster(const int* p, int rank) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
  return v;
}

// By one warp: v[e] becomes the sum of v[0 .. e - 1]; returns the total.
__device__ __forceinline__ int warp_exclusive(int* v, int E) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int base = 0; base < E; base += 32) {
    const int own = base + lane < E ? v[base + lane] : 0;
    int s = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, s, d);
      if (lane >= d) s += u;
    }
    if (base + lane < E) v[base + lane] = carry + s - own;
    carry += __shfl_sync(0xFFFFFFFFu, s, 31);
  }
  return carry;
}

// kOne: the grid is one cluster, each CTA has at most kSub tokens, and ranks
// become slots here.  Else they are ranks inside the CTA's run.
// No second CTA an SM is asked for, and from 65 experts on (FP32: 33) the
// registers leave room for one: with room for two, grids smaller than the
// machine are doubled up on some SMs (8192 tokens of 128 experts 15.1 us
// instead of 11.1; 16384, a run on every SM, 15.2 instead of 16.3).  Instances
// for fewer experts have 32 registers, so two fit (bf16 of 33 to 64 experts
// spill 32 bytes): 16384 tokens of 32 experts in bf16 take 10.6 us, of 64 12.2,
// 8192 of 32 10.4.
template <bool kF32, int NV, bool kOne>
__global__ void __launch_bounds__(kRouteThreads) route_topk_kernel(const RouteParams p) {
  __shared__ uint32_t mask[kMaxGroups][kSub / 32];
  __shared__ int count[kMaxGroups];
  __shared__ int16_t ids_s[kSub * kMaxTopK];
  __shared__ int16_t rank_s[kOne ? kSub * kMaxTopK : 1];
  __shared__ int all[kOne ? kMaxGroups : 1], before[kOne ? kMaxGroups : 1];
  __shared__ int total_s;
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
      uint32_t key[NV], best = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        key[i] = kF32 ? order_key(x[i]) : order_key_bf16(x[i], lane + 32 * i);
        best = max(best, key[i]);
      }
      load_token(ml + kRouteWarps);
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
      const float x_max = top ? selected_value<kF32>(top) : 0.0f;
      float sum = 0.0f;
      if (!p.renorm) {                           // over all experts, before any is taken out
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += key[i] ? expf(selected_value<kF32>(key[i]) - x_max) : 0.0f;
      }
      uint32_t my_key = 0;                       // lane j keeps the j-th selected
      int my_id = -1;
      for (int j = 0; j < k; ++j) {
        const uint32_t kmax = j == 0 ? top : __reduce_max_sync(0xFFFFFFFFu, best);
        if (kmax == 0) break;                    // nothing left that may be taken
        int at;
        if constexpr (kF32) {
          uint32_t own = 0xFFFFFFFFu;
#pragma unroll
          for (int i = NV - 1; i >= 0; --i)
            if (key[i] == kmax) own = lane + 32 * i;
          at = (int)__reduce_min_sync(0xFFFFFFFFu, own);
        } else {
          at = 0xFFFF - (int)(kmax & 0xFFFFu);
        }
        if (lane == j) {
          my_id = at;
          my_key = kmax;
        }
        best = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (kF32 ? lane + 32 * i == at : key[i] == kmax) key[i] = 0;
          best = max(best, key[i]);
        }
      }
      const float my_e = my_id >= 0 ? expf(selected_value<kF32>(my_key) - x_max) : 0.0f;
      if (p.renorm) sum = my_e;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      if (lane < k) {
        p.ids[m * k + lane] = my_id;
        p.weights[m * k + lane] = my_id >= 0 ? __fmul_rn(my_e, __frcp_rn(sum)) : 0.0f;
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
      if constexpr (kOne) rank_s[i] = (int16_t)rank;
      else p.slots[sub * k + i] = rank;
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
  if constexpr (!kOne) {
    for (int e = threadIdx.x; e < E; e += kRouteThreads) p.hist[(int64_t)blockIdx.x * hist_stride(E) + e] = count[e];
    return;
  }
  const int ctas = gridDim.x, rank = blockIdx.x;
  int* start = count;                            // becomes each expert's first slot
  if (ctas > 1) {
    start = all;
    cluster_sync();                              // every CTA has its counts
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      int sum = 0, head = 0;
      for (int c = 0; c < ctas; ++c) {
        const int v = c == rank ? count[e] : ld_cluster(&count[e], c);
        sum += v;
        if (c < rank) head += v;
      }
      all[e] = sum;
      before[e] = head;
    }
    __syncthreads();
  }
  if (warp == 0) {
    const int t = warp_exclusive(start, E);
    if (lane == 0) total_s = t;
  }
  __syncthreads();
  const int total = total_s;
  if (rank == 0)
    for (int e = threadIdx.x; e <= E; e += kRouteThreads) p.offsets[e] = e < E ? start[e] : total;
  const int first = (int)(m_begin * k), pairs = m_begin < m_end ? (int)(m_end - m_begin) * k : 0;
  for (int i = threadIdx.x; i < pairs; i += kRouteThreads) {
    const int e = ids_s[i], slot = e >= 0 ? start[e] + (ctas > 1 ? before[e] : 0) + rank_s[i] : -1;
    p.slots[first + i] = slot;
    if (e >= 0) p.row_index[slot] = (first + i) / k;
    if (first + i >= total) p.row_index[first + i] = -1;
  }
  if (ctas > 1) cluster_sync();                  // no CTA leaves while its counts may be read
}

// Second launch of a call with more than one run of tokens: every CTA adds up
// all runs' counts (for the offsets) and those before its own (for its base),
// four experts a thread and load, then turns its ranks into slots.
__global__ void __launch_bounds__(kRouteThreads) route_slots_kernel(const RouteParams p) {
  __shared__ int all[kMaxGroups + 3];
  __shared__ int before[kMaxGroups + 3];
  __shared__ int total_s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int E = p.E, k = p.k, stride = hist_stride(E);
  for (int e = threadIdx.x; e < stride; e += kRouteThreads) all[e] = before[e] = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t m_begin = (int64_t)blockIdx.x * p.chunk;
  const int64_t m_end = m_begin + p.chunk < p.M ? m_begin + p.chunk : p.M;
  const int i_end = (int)(m_end * k);
  int i = (int)(m_begin * k) + threadIdx.x;
  // the first pair of this thread is on its way while the counts are added up
  int id = -1, rank = 0;
  if (i < i_end) {
    id = p.ids[i];
    rank = p.slots[i];
  }
  const int quads = stride / 4, at = threadIdx.x % quads, rows = kRouteThreads / quads;
  int4 sum = make_int4(0, 0, 0, 0), head = make_int4(0, 0, 0, 0);
  if ((int)threadIdx.x < rows * quads) {
#pragma unroll 4
    for (int c = threadIdx.x / quads; c < (int)gridDim.x; c += rows) {
      const int4 h = reinterpret_cast<const int4*>(p.hist + (int64_t)c * stride)[at];
      sum.x += h.x;
      sum.y += h.y;
      sum.z += h.z;
      sum.w += h.w;
      if (c < (int)blockIdx.x) {
        head.x += h.x;
        head.y += h.y;
        head.z += h.z;
        head.w += h.w;
      }
    }
    atomicAdd(&all[4 * at], sum.x);              // integer sums: any order gives the same
    atomicAdd(&all[4 * at + 1], sum.y);
    atomicAdd(&all[4 * at + 2], sum.z);
    atomicAdd(&all[4 * at + 3], sum.w);
    atomicAdd(&before[4 * at], head.x);
    atomicAdd(&before[4 * at + 1], head.y);
    atomicAdd(&before[4 * at + 2], head.z);
    atomicAdd(&before[4 * at + 3], head.w);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int t = warp_exclusive(all, E);
    if (threadIdx.x == 0) total_s = t;
  }
  __syncthreads();
  const int total = total_s;
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= E; e += kRouteThreads) p.offsets[e] = e < E ? all[e] : total;
  while (i < i_end) {
    if (id >= 0) {
      const int slot = all[id] + before[id] + rank;
      p.slots[i] = slot;
      p.row_index[slot] = i / k;
    }
    if (i >= total) p.row_index[i] = -1;         // rows no pair fills
    i += kRouteThreads;
    if (i < i_end) {
      id = p.ids[i];
      rank = p.slots[i];
    }
  }
}

namespace {

// Runs of tokens: at least 32 tokens a run, one for each warp, and at most one
// run an SM.  One launch while a cluster has a warp for each token: 256 tokens
// of 128 experts 6.6 us, in two launches 7.1 (33 tokens 5.5 and 6.2); with more
// tokens a warp it is slower (512: 9.4 and 7.1).
int64_t route_chunks(int64_t M, int sms) {
  int64_t c = ceil_div(M, kRouteWarps);
  if (M <= kRouteCluster * kRouteWarps) {
    c = c < kRouteCluster ? c : kRouteCluster;
    while (c & (c - 1)) ++c;                     // a cluster of 1, 2, 4 or 8; no CTA without tokens
    return c;
  }
  const int64_t cap = sms < kRouteMaxChunks ? sms : kRouteMaxChunks;
  return c < cap ? c : cap;
}

template <bool kF32, bool kOne>
cudaError_t launch_topk(const RouteParams& p, int grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRouteThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)grid;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kOne && grid > 1 ? 2 : 1;
  const int nv = (p.E + 31) / 32;
  if (nv <= 1) return cudaLaunchKernelEx(&cfg, route_topk_kernel<kF32, 1, kOne>, p);
  if (nv <= 2) return cudaLaunchKernelEx(&cfg, route_topk_kernel<kF32, 2, kOne>, p);
  if (nv <= 4) return cudaLaunchKernelEx(&cfg, route_topk_kernel<kF32, 4, kOne>, p);
  if (nv <= 8) return cudaLaunchKernelEx(&cfg, route_topk_kernel<kF32, 8, kOne>, p);
  return cudaLaunchKernelEx(&cfg, route_topk_kernel<kF32, 16, kOne>, p);
}

template <bool kF32>
cudaError_t launch_route(const RouteParams& p, int grid, cudaStream_t st) {
  if (grid <= kRouteCluster && p.chunk <= kSub) return launch_topk<kF32, true>(p, grid, st);
  const cudaError_t e = launch_topk<kF32, false>(p, grid, st);
  return e == cudaSuccess ? launch_pdl(route_slots_kernel, grid, kRouteThreads, st, p) : e;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_route_workspace_bytes(int n_experts) {
  if (n_experts < 1 || n_experts > NVFP4_MAX_GROUPS) return 0;
  return (size_t)kRouteMaxChunks * (size_t)hist_stride(n_experts) * sizeof(int32_t);
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
  return cuda_status(dtype == NVFP4_IN_F32 ? launch_route<true>(p, grid, st) : launch_route<false>(p, grid, st));
}

}  // extern "C"
