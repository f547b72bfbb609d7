// What api.cu's host runtime offers to the other translation units' entry
// points: the current device's state and the cached tensor maps.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/bwgemm.h"

namespace bwg {

struct Runtime {
  int device;
  int sm_count;
  int max_smem;                   // opt-in shared memory per CTA
  unsigned long long* err;        // device error word
  unsigned long long timeout_ns;  // bound of every barrier wait
  unsigned tx_extra;              // test hook: extra bytes expected per stage (0 normally)
};

// State of the current device; BWG_ERR_UNSUPPORTED where it is not sm_103.
bwg_status runtime_device(Runtime* out);

// Tensor map of a rank-`rank` view (dimensions innermost first, strides in
// bytes for dimensions 1.., box in elements), cached by its arguments.
bool runtime_map(CUtensorMap* m, const void* ptr, CUtensorMapDataType dtype, int rank,
                 const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                 CUtensorMapSwizzle swizzle);

// BWG_OK, or BWG_ERR_CUDA with the runtime's error state cleared.
bwg_status runtime_status(cudaError_t e);

}  // namespace bwg
