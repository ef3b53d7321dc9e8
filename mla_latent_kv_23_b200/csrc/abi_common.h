// Shared by the translation units that implement the C ABI: per-device state,
// the tensor-map encoder and argument helpers.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "append_slots.h"
#include "mla.h"

namespace mla {

struct DeviceInfo {
  bool ready = false;
  int sm_count = 0;
  int cc_major = 0, cc_minor = 0;
  int max_clusters = 0;  // co-resident 2-CTA clusters of the DeepSeek-V3-shape kernel
  int tree_clusters = 0;  // the same of the tree kernel of that shape
  bool small_tc = false;  // the small-latent tensor-core kernel is usable
  bool up_proj_tc = false;
  bool wgemm_tc = false;  // the weight-streaming projection kernel is usable
  bool append_tc = false;  // the slot-map append kernel is usable
  int append_clusters[kClusterSizes] = {};  // its co-resident clusters by size
  int* flags = nullptr;  // device address of the sticky device flags
};

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled, looked up by the first device_info call (null if
// the driver does not have it)
extern EncodeTiledFn g_encode;

// State of the current device, filled in at its first use.
mla_status device_info(const DeviceInfo** out);
mla_status cuda_status(cudaError_t e);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool valid_dtype(mla_dtype d) { return d == MLA_DTYPE_BF16 || d == MLA_DTYPE_FP32; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace mla
