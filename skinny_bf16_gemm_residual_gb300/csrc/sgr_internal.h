// sgr_internal.h -- what the library's translation units share: per-device
// lookups defined in sgr_api.cu and the attention operators' device set-up
// defined in sgr_kv.cu.  Not part of the public interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace sgr {

namespace detail {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return (EncodeTiledFn) nullptr;
    }
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

}  // namespace detail

constexpr int kMaxDevices = 64;

// Device error word of `dev` (allocates nothing).  Returns an sgr_status.
int device_error_word(int dev, unsigned** word);

// Kernel attributes of the attention operators on `dev`; idempotent,
// allocates nothing, called by sgr_init() and by their first call.  Returns
// an sgr_status.
int kv_init_device(int dev);

}  // namespace sgr
