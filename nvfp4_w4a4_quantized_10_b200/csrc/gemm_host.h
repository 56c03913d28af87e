// Host-side pieces of the block-scaled GEMMs: tensor maps, the K-split
// workspace of a stream, and the launch of one kernel instance.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "common.h"
#include "gemm_kernel.cuh"

namespace nvfp4 {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
    else
      (void)cudaGetLastError();
  });
  return fn;
}

// Codes of a [rows, K/2]-byte operand in boxes of row_bytes x box_rows, with
// the matching swizzle (128-byte rows: 128B, 64-byte rows: 64B).
inline bool make_code_map(CUtensorMap* m, const void* base, int64_t rows, int64_t K, int box_rows, int row_bytes) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  const cuuint32_t box[2] = {(cuuint32_t)row_bytes, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Block scales in the tensor-core order viewed as [chunks, 128] 32-bit words
// (one 512-byte chunk per row), boxes of `chunks` consecutive chunks.
inline bool make_sf_map(CUtensorMap* m, const void* base, int64_t rows, int64_t kc, int chunks) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {128, (cuuint64_t)(ceil_div(rows, 128) * kc)};
  const cuuint64_t strides[1] = {512};
  const cuuint32_t box[2] = {128, (cuuint32_t)chunks};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output [M, N] (bf16 or f32), boxes of box_rows rows x 128 bytes, 128B swizzle.
inline bool make_out_map(CUtensorMap* m, void* base, int64_t M, int64_t N, bool f32, int box_rows = kBM) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int64_t esz = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
  const cuuint64_t strides[1] = {(cuuint64_t)(N * esz)};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / esz), (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Swapped (decode) tiles are split over the CTAs along K; partial tiles are
// exchanged through a K-split workspace of one stream: either one the caller
// registered for that stream (nvfp4_set_workspace: caller-owned, never freed
// here) or, failing that, one the library allocates on the first swapped
// call on that stream (all words empty) and frees in
// nvfp4_release_workspaces().  One per stream, because calls on unordered
// streams may run at the same time and must not share partial words.
struct Workspace {
  uint64_t* ws = nullptr;
  size_t bytes = 0;
  bool owned = false;   // allocated (and freed) by the library
};

// The workspace of (current device, st) for a swapped GEMM with activation
// side bn; allocated here if none is registered.  cudaErrorInvalidValue: the
// registered one is too small; cudaErrorNotPermitted: st is being captured
// and there is none yet.
cudaError_t get_workspace(const DeviceInfo* d, cudaStream_t st, int bn, Workspace* out);

// Bytes of K-split workspace a swapped GEMM with activation side bn needs:
// two slots of bn x 128 words per CTA.
size_t workspace_need(const DeviceInfo* d, int bn);

template <int BN, bool SWAP, bool OUT_F32, int QX = 0, bool MX = false, bool PAIR = false, bool GROUPED = false>
cudaError_t set_smem_attr(const DeviceInfo* d) {
  using Cf = Cfg<BN, SWAP, QX, MX, PAIR, GROUPED>;
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  std::call_once(once[d->device], [&] {
    auto kern = nvfp4_gemm_kernel<BN, SWAP, OUT_F32, QX, MX, PAIR, GROUPED>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::kSmemBytes);
    // all of the SM's unified memory as shared memory: two co-resident CTAs
    // of 114 KB fit only with the full carveout, and a cooperative launch is
    // admitted against this preference
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    attr_err[d->device] = e;
  });
  return attr_err[d->device];
}

// CTAs of this kernel that can be resident on one SM (occupancy API, with the
// attributes set above), once per device; 0 if the query fails.
template <int BN, bool SWAP, bool OUT_F32, int QX = 0, bool MX = false, bool PAIR = false, bool GROUPED = false>
int resident_per_sm(const DeviceInfo* d) {
  using Cf = Cfg<BN, SWAP, QX, MX, PAIR, GROUPED>;
  static std::once_flag once[64];
  static int occ[64];
  std::call_once(once[d->device], [&] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, nvfp4_gemm_kernel<BN, SWAP, OUT_F32, QX, MX, PAIR, GROUPED>,
                                                      Cf::kThreads, Cf::kSmemBytes) != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    occ[d->device] = n;
  });
  return occ[d->device];
}

// grid: number of CTAs (0 = the persistent grid); cluster: CTAs per cluster
template <int BN, bool SWAP, bool OUT_F32, int QX = 0, bool MX = false, bool PAIR = false, bool GROUPED = false>
cudaError_t launch(const GemmParamsOf<GROUPED>& p, const DeviceInfo* d, cudaStream_t st, int grid = 0, int cluster = 1) {
  using Cf = Cfg<BN, SWAP, QX, MX, PAIR, GROUPED>;
  auto kern = nvfp4_gemm_kernel<BN, SWAP, OUT_F32, QX, MX, PAIR, GROUPED>;
  const cudaError_t ea = set_smem_attr<BN, SWAP, OUT_F32, QX, MX, PAIR, GROUPED>(d);
  if (ea != cudaSuccess) return ea;
  if (grid == 0) {
    if (SWAP) {
      const int64_t units = (int64_t)p.tiles_p * p.kt;
      int per_sm = Cf::kGridPerSm;
      if (decode_cooperative()) {
        // a cooperative grid must be resident at once: at most what the
        // occupancy API admits per SM
        const int occ = resident_per_sm<BN, SWAP, OUT_F32, QX, MX, PAIR, GROUPED>(d);
        if (occ < per_sm) per_sm = occ < 1 ? 1 : occ;
      }
      const int64_t cap = (int64_t)d->sm_count * per_sm;
      grid = (int)(units < cap ? units : cap);
    } else {
      const int tiles = p.tiles_p * p.tiles_q;
      grid = tiles < d->sm_count ? tiles : d->sm_count;
    }
  }
  // programmatic dependent launch: the kernel may start while the previous
  // kernel in the stream finishes; it waits (griddepcontrol.wait) before
  // touching anything that kernel produced
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Cf::kThreads);
  cfg.dynamicSmemBytes = Cf::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // split-K tiles: a tile's first CTA waits for partials from later CTAs,
  // so the grid (at most one CTA per SM) must be resident at once; opted in,
  // the driver guarantees that or refuses the launch
  if (SWAP && decode_cooperative()) {
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.numAttrs = 2;
  }
  if (PAIR) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace nvfp4
