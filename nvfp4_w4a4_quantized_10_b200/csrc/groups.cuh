// Rows grouped by expert: the table a kernel builds from the device-resident
// group offsets.  Group g owns rows [off[g], off[g+1]); its block scales start
// at a 128-row scale block of their own, number blk[g].  Offsets are read on
// the device, because the router that wrote them runs on the same stream and
// the host never sees them.
#pragma once
#include <cstdint>

#include "../../include/nvfp4.h"
#include "ptx.cuh"

namespace nvfp4 {

constexpr int kMaxGroups = NVFP4_MAX_GROUPS;

// Most 128-row scale blocks that T rows in E groups can take: sum over the
// non-empty groups of ceil(r / 128) <= (T + 127 min(E, T)) / 128.
__host__ __device__ inline int64_t grouped_blocks(int64_t T, int64_t E) {
  return (T + 127 * (E < T ? E : T)) / 128;
}

struct GroupTable {
  int off[kMaxGroups + 1];
  int blk[kMaxGroups + 1];     // scale blocks of 128 rows before each group
  int tiles[kMaxGroups + 1];   // GEMM tiles of kTileRows rows before each group (filled if asked for)
};

// Fill the table in shared memory; called by every thread of the CTA (at
// least 64), ends with a barrier.  Offsets that do not start at 0, decrease
// or pass T are a caller's error that only the device can see: the error
// word is set and the table says that every group is empty, so no row is
// touched.
template <int kTileRows = 0>
__device__ __forceinline__ void load_groups(GroupTable& t, const int32_t* offsets, int E, int64_t T, unsigned* err) {
  bool bad = false;
  for (int i = threadIdx.x; i <= E; i += blockDim.x) {
    const int o = offsets[i];
    const int next = i < E ? offsets[i + 1] : o;
    bad |= o < 0 || next < o || next > T || (i == 0 && o != 0);
    t.off[i] = o;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicCAS(err, 0u, kErrBounds);
    for (int i = threadIdx.x; i <= E; i += blockDim.x) t.off[i] = t.blk[i] = t.tiles[i] = 0;
    __syncthreads();
    return;
  }
  auto prefix = [&](int* out, auto&& value) {
    int carry = 0;
    for (int base = 0; base < E; base += 32) {
      const int i = base + (int)(threadIdx.x & 31);
      int v = i < E ? value(t.off[i + 1] - t.off[i]) : 0;
      const int own = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if ((int)(threadIdx.x & 31) >= d) v += u;
      }
      if (i < E) out[i] = carry + v - own;
      carry += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if ((threadIdx.x & 31) == 0) out[E] = carry;
  };
  if (threadIdx.x < 32) prefix(t.blk, [](int r) { return (r + 127) >> 7; });
  if constexpr (kTileRows != 0) {
    if (threadIdx.x >= 32 && threadIdx.x < 64) prefix(t.tiles, [](int r) { return (r + kTileRows - 1) / kTileRows; });
  }
  __syncthreads();
}

// Largest g < E with prefix[g] <= v: the group that holds v, for
// prefix[0] = 0 <= v < prefix[E].  Empty groups (equal prefixes) are skipped.
__device__ __forceinline__ int find_group(const int* prefix, int E, int v) {
  int lo = 0, hi = E;        // prefix[lo] <= v < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace nvfp4
