// host.cuh - what the library's host sources share: error reporting, kernel
// launches, the tensor-map encoder and per-device kernel attributes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>
#include <set>
#include <utility>

#include "../../include/dg.h"

namespace dg {

// Records the thread's error text (dg_last_error) and returns `s`.
dg_status fail(dg_status s, const char* fmt, ...);

#define DG_CUDA(call)                                                                        \
  do {                                                                                       \
    cudaError_t e_ = (call);                                                                 \
    if (e_ != cudaSuccess) return fail(DG_ERR_CUDA, "%s: %s (%s:%d)", #call,                \
                                       cudaGetErrorString(e_), __FILE__, __LINE__);          \
  } while (0)

#define DG_TRY(expr)                  \
  do {                                \
    dg_status s_ = (expr);            \
    if (s_ != DG_OK) return s_;       \
  } while (0)

// One kernel launch.  With DG_PDL (programmatic dependent launch) its CTAs
// may be scheduled while the stream's previous kernel finishes: every kernel
// of the library waits (griddepcontrol.wait) before it touches memory that
// another kernel writes, so only its launch latency and its own set-up
// (barriers, tensor memory, tensor-map prefetch) overlap the predecessor's
// tail.  Optional cluster shape and cluster scheduling policy.
#ifndef DG_PDL
#define DG_PDL 1
#endif
struct Launch {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute at[3];
  Launch(dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool pdl = DG_PDL) {
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    lc.attrs = at;
    if (pdl) {
      at[lc.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[lc.numAttrs].val.programmaticStreamSerializationAllowed = 1;
      ++lc.numAttrs;
    }
  }
  Launch& cluster(unsigned x, unsigned y, unsigned z) {
    at[lc.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[lc.numAttrs].val.clusterDim.x = x;
    at[lc.numAttrs].val.clusterDim.y = y;
    at[lc.numAttrs].val.clusterDim.z = z;
    ++lc.numAttrs;
    return *this;
  }
  Launch& policy(cudaClusterSchedulingPolicy pol) {
    at[lc.numAttrs].id = cudaLaunchAttributeClusterSchedulingPolicyPreference;
    at[lc.numAttrs].val.clusterSchedulingPolicyPreference = pol;
    ++lc.numAttrs;
    return *this;
  }
  template <typename... KArgs, typename... Args>
  cudaError_t operator()(void (*k)(KArgs...), Args&&... args) {
    return cudaLaunchKernelEx(&lc, k, std::forward<Args>(args)...);
  }
};

// dg_fp8_grouped_gemm with a context's error word `err` (or null), which gets
// kDevErrTimeout when a wait of the kernel runs out.
dg_status fp8_grouped_gemm(const uint8_t* d_a, int64_t lda, const float* d_a_scale, int64_t lds, const uint8_t* d_b,
                           int64_t ldb, const float* d_b_scale, const int32_t* d_off, int64_t groups, int64_t M,
                           int64_t N, int64_t K, const float* d_row_weight, void* d_out, int32_t out_dtype, int64_t ldo,
                           int* err, cudaStream_t st);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)p;
  }
  return fn;
}

// cudaFuncSetAttribute applies to the kernel in the current device's context:
// set each (kernel, device) once, the first time a launch on that device
// needs it.
inline dg_status set_smem_attr(const void* fn, int bytes, bool max_carveout) {
  static std::mutex mu;
  static std::set<std::pair<const void*, int>> done;
  int dev = 0;
  DG_CUDA(cudaGetDevice(&dev));
  std::lock_guard<std::mutex> lock(mu);
  if (done.count({fn, dev})) return DG_OK;
  DG_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  if (max_carveout) DG_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100));
  done.insert({fn, dev});
  return DG_OK;
}

inline int device_sms() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

}  // namespace dg
