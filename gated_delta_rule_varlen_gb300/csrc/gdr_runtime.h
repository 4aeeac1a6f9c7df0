// gdr_runtime.h -- host services that every entry point shares (defined in
// gdr_api.cu; internal to the library).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/gdr.h"

namespace gdr {

// GDR_OK when the current device is an sm_103, GDR_UNSUPPORTED for another.
gdr_status check_device();

// SM count of the current device (152 when no device answers).
int sm_count();

// The current device's error word (null on failure): a kernel whose bounded
// wait runs out writes a non-zero code there.
int* device_error_ptr();

// cu[0] == 0, non-decreasing, cu[N] == T (T below 2^31); counts 64-token chunks.
gdr_status plan_host(int64_t T, int32_t N, const int32_t* cu, int64_t* NC);

// Opened around every kernel launch: counts it and, while profiling is on,
// brackets it with a pair of CUDA events on its stream.
struct ProfScope {
  cudaStream_t st;
  bool on;
  ProfScope(const char* name, cudaStream_t s, double units = 0);
  ~ProfScope();
  ProfScope(const ProfScope&) = delete;
  ProfScope& operator=(const ProfScope&) = delete;
};

}  // namespace gdr
