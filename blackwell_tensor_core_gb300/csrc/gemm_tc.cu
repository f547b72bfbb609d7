// Dense and grouped kernels of the tcgen05 body (gemm_body.cuh), and their launches.
#include "gemm_body.cuh"

namespace bwg {
namespace {

template <int CG, int MC>
__global__ void __launch_bounds__(kThreads, 1) gemm_dense_kernel(const __grid_constant__ GemmParams p) {
  gemm_body<CG, MC, false, 1, kEpiPlain, false>(p, p);
}

// 512x256 tiles on a pair: warp 0 TMA, warps 1-2 MMA (one per consumer),
// warp 3 idle, warps 4-7 and 8-11 the epilogue of consumer 0 and 1.
// DYN: one cluster per unit, units claimed by cluster launch control.
template <bool DYN>
__global__ void __launch_bounds__(kThreads2C, 1)
    gemm_dense_2c_kernel(const __grid_constant__ GemmParams p) {
  gemm_body<2, 1, false, 2, kEpiPlain, DYN>(p, p);
}

template <bool SW>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_grouped_kernel(const __grid_constant__ GroupedParams p) {
  gemm_body<2, 1, true, 1, SW ? kEpiSwiglu : kEpiPlain, false>(p, p.base);
}

// Grouped, two consumers: 512-row units; the second consumer's 256 rows are
// skipped where a group has 256 rows or fewer left.
template <bool SW, bool DYN>
__global__ void __launch_bounds__(kThreads2C, 1)
    gemm_grouped_2c_kernel(const __grid_constant__ GroupedParams p) {
  gemm_body<2, 1, true, 2, SW ? kEpiSwiglu : kEpiPlain, DYN>(p, p.base);
}

}  // namespace

cudaError_t launch_gemm_1cta(const GemmParams& p, int grid, size_t smem, cudaStream_t s) {
  return launch_cluster(gemm_dense_kernel<1, 1>, p, 1, grid, smem, s);
}

cudaError_t launch_gemm_2cta(const GemmParams& p, int grid, size_t smem, cudaStream_t s) {
  return launch_cluster(gemm_dense_kernel<2, 1>, p, 2, grid, smem, s);
}

cudaError_t launch_gemm_2cta_mc(const GemmParams& p, int grid, size_t smem, cudaStream_t s) {
  return launch_cluster(gemm_dense_kernel<2, 2>, p, 4, grid, smem, s);
}

cudaError_t launch_gemm_2cta_2c(const GemmParams& p, int grid, size_t smem, cudaStream_t s,
                                bool dynamic) {
  return dynamic ? launch_two_consumer(gemm_dense_2c_kernel<true>, p, grid, smem, s)
                 : launch_two_consumer(gemm_dense_2c_kernel<false>, p, grid, smem, s);
}

cudaError_t launch_grouped_2c(const GroupedParams& p, int grid, size_t smem, cudaStream_t s,
                              bool swiglu, bool dynamic) {
  if (dynamic)
    return swiglu ? launch_two_consumer(gemm_grouped_2c_kernel<true, true>, p, grid, smem, s)
                  : launch_two_consumer(gemm_grouped_2c_kernel<false, true>, p, grid, smem, s);
  return swiglu ? launch_two_consumer(gemm_grouped_2c_kernel<true, false>, p, grid, smem, s)
                : launch_two_consumer(gemm_grouped_2c_kernel<false, false>, p, grid, smem, s);
}

cudaError_t launch_grouped_2cta(const GroupedParams& p, int grid, size_t smem, cudaStream_t s,
                                bool swiglu) {
  return swiglu ? launch_cluster(gemm_grouped_kernel<true>, p, 2, grid, smem, s)
                : launch_cluster(gemm_grouped_kernel<false>, p, 2, grid, smem, s);
}

int max_active_clusters_gemm_2c(size_t smem) {
  return occupancy_clusters(reinterpret_cast<const void*>(gemm_dense_2c_kernel<false>), 2, smem,
                            kThreads2C);
}

int max_active_clusters_grouped_2c(size_t smem) {
  return occupancy_clusters(reinterpret_cast<const void*>(gemm_grouped_2c_kernel<false, false>), 2,
                            smem, kThreads2C);
}

int max_active_clusters_gemm(int cluster, bool grouped, size_t smem) {
  const void* fn = grouped ? reinterpret_cast<const void*>(gemm_grouped_kernel<false>)
                   : cluster == 4 ? reinterpret_cast<const void*>(gemm_dense_kernel<2, 2>)
                   : cluster == 2 ? reinterpret_cast<const void*>(gemm_dense_kernel<2, 1>)
                                  : reinterpret_cast<const void*>(gemm_dense_kernel<1, 1>);
  return occupancy_clusters(fn, cluster, smem);
}

cudaError_t set_gemm_attributes(size_t smem) {
  const void* fns[] = {reinterpret_cast<const void*>(gemm_dense_kernel<1, 1>),
                       reinterpret_cast<const void*>(gemm_dense_kernel<2, 1>),
                       reinterpret_cast<const void*>(gemm_dense_kernel<2, 2>),
                       reinterpret_cast<const void*>(gemm_dense_2c_kernel<false>),
                       reinterpret_cast<const void*>(gemm_dense_2c_kernel<true>),
                       reinterpret_cast<const void*>(gemm_grouped_kernel<false>),
                       reinterpret_cast<const void*>(gemm_grouped_kernel<true>),
                       reinterpret_cast<const void*>(gemm_grouped_2c_kernel<false, false>),
                       reinterpret_cast<const void*>(gemm_grouped_2c_kernel<true, false>),
                       reinterpret_cast<const void*>(gemm_grouped_2c_kernel<false, true>),
                       reinterpret_cast<const void*>(gemm_grouped_2c_kernel<true, true>)};
  return set_max_smem(fns, smem);
}

}  // namespace bwg
