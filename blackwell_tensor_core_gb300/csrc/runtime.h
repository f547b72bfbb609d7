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
  int pairs;                      // CTA pairs of the one-consumer kernels that run at once
  int pairs_2c;                   // of the two-consumer kernels
  int no_tail_split;              // 1: never cut the tiles of the last wave
  unsigned long long* trace;      // unit trace of the pair kernels, or nullptr
};

// State of the current device; BWG_ERR_UNSUPPORTED where it is not sm_103.
bwg_status runtime_device(Runtime* out);

// Tensor map of a rank-`rank` view (dimensions innermost first, strides in
// bytes for dimensions 1.., box in elements), cached by its arguments.
bool runtime_map(CUtensorMap* m, const void* ptr, CUtensorMapDataType dtype, int rank,
                 const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                 CUtensorMapSwizzle swizzle);

// The same for a row-major matrix: `inner` elements a row, `outer` rows.
inline bool runtime_map_2d(CUtensorMap* m, const void* ptr, CUtensorMapDataType dtype, uint64_t inner, uint64_t outer,
                           uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer) {
  const uint64_t dims[2] = {inner, outer};
  const uint32_t box[2] = {box_inner, box_outer};
  return runtime_map(m, ptr, dtype, 2, dims, &row_bytes, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Largest rows, columns and depths that the tiled kernels take: rounding up to
// tiles, and the first element past a tile, stay in an int.
constexpr int kMaxSize = 0x7fffffff - 1024;

inline bool is_aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// H = silu(X gate) * (X up) of at most kSmallMMaxM rows, arguments checked (see gemm_swiglu).
bwg_status run_small_m_gated(const void* X, const void* W, void* H, int dtype, bool w_nt, int M, int N, int K, int ldx,
                             int ldw, int ldh, cudaStream_t stream);

// BWG_OK, or BWG_ERR_CUDA with the runtime's error state cleared.
bwg_status runtime_status(cudaError_t e);

}  // namespace bwg
