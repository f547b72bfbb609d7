// Gated kernels of the tcgen05 body (gemm_body.cuh): the products of a gated
// feed-forward block, x [gate | up], with the activation or its gradient in the
// epilogue.
#include <algorithm>
#include <cstring>

#include "gemm_body.cuh"
#include "runtime.h"

using namespace bwg;

namespace bwg {
namespace {

// 256x256 tiles, whose accumulator is one of two, so that eight epilogue warps work
// on one tile while the next is summed up.  With 512x256 tiles, which load a quarter
// less, the tensor cores wait for the epilogue at each tile's end: 8192 x 4096 x
// 8192, back to back in turn, H 300 for 322 us (K = 512: 24.6 for 30.2; K = 8192:
// 607 for 632); of another run, with gate and up kept in 8 bits 302 for 341, their
// gradient 325 for 356.  What bounds them: tensor cores and the power limit.
template <int EPI>
__global__ void __launch_bounds__(kThreads2C, 1) gated_wide_kernel(const __grid_constant__ DenseGatedParams p) {
  gemm_body<2, 1, false, 1, EPI, false>(p, p);
}

template <int EPI>
__global__ void __launch_bounds__(kThreads2C, 1) gated_grouped_kernel(const __grid_constant__ GroupedGatedParams p) {
  gemm_body<2, 1, true, 1, EPI, true>(p, p.base);
}

}  // namespace

cudaError_t launch_gated_dense(const DenseGatedParams& p, int epi, int grid, size_t smem, cudaStream_t s) {
  if (epi == kEpiSwigluKeep) return launch_pair_behind(gated_wide_kernel<kEpiSwigluKeep>, p, grid, smem, s);
  if (epi == kEpiSwigluGrad) return launch_pair_behind(gated_wide_kernel<kEpiSwigluGrad>, p, grid, smem, s);
  return launch_pair_behind(gated_wide_kernel<kEpiSwiglu>, p, grid, smem, s);
}

cudaError_t launch_gated_grouped(const GroupedGatedParams& p, int epi, int grid, size_t smem, cudaStream_t s) {
  return epi == kEpiSwigluKeep ? launch_pair_behind(gated_grouped_kernel<kEpiSwigluKeep>, p, grid, smem, s)
                               : launch_pair_behind(gated_grouped_kernel<kEpiSwigluGrad>, p, grid, smem, s);
}

cudaError_t set_gated_attributes(size_t smem) {
  const void* fns[] = {reinterpret_cast<const void*>(gated_wide_kernel<kEpiSwiglu>),
                       reinterpret_cast<const void*>(gated_wide_kernel<kEpiSwigluKeep>),
                       reinterpret_cast<const void*>(gated_wide_kernel<kEpiSwigluGrad>),
                       reinterpret_cast<const void*>(gated_grouped_kernel<kEpiSwigluKeep>),
                       reinterpret_cast<const void*>(gated_grouped_kernel<kEpiSwigluGrad>)};
  return set_max_smem(fns, smem);
}

// ---------------------------------------------------------- entry points ---

namespace {

struct GatedCall {
  int dtype;             // bwg_out_dtype of x, w and D
  int epi;
  const void* x;
  const void* const* w;  // one weight, or one an expert
  void* d;               // H [M, I], or its projections' gradients [M, 2 I]
  void* codes;
  float* scales;
  const void* dh;
  const int* offsets;    // nullptr: one group of all rows
  int G, w_nt, M, N, K, ldx, ldw, ldd, lddh;
};

bool rows16(const void* p, long long ld) { return is_aligned(p, 16) && ld % 8 == 0; }

bwg_status check_gated(const GatedCall& c) {
  if (c.dtype != BWG_OUT_BF16 && c.dtype != BWG_OUT_FP16) return BWG_ERR_INVALID_ARG;
  if (c.G < 0 || c.M < 0 || c.N < 0 || c.K < 0) return BWG_ERR_INVALID_ARG;
  if (c.G == 0 || c.M == 0 || c.N == 0) return BWG_OK;
  if (c.M > kMaxSize || c.N > kMaxSize || c.K > kMaxSize) return BWG_ERR_UNSUPPORTED;
  if (c.N % 16 != 0) return BWG_ERR_ALIGNMENT;
  const int d_cols = c.epi == kEpiSwigluGrad ? c.N : c.N / 2;
  if (c.d == nullptr || c.ldd < d_cols) return BWG_ERR_INVALID_ARG;
  if (!rows16(c.d, c.ldd)) return BWG_ERR_ALIGNMENT;
  if (c.epi == kEpiSwigluKeep) {
    if (c.codes == nullptr || c.scales == nullptr) return BWG_ERR_INVALID_ARG;
    if (!is_aligned(c.codes, 16) || !is_aligned(c.scales, 4)) return BWG_ERR_ALIGNMENT;
  }
  if (c.epi == kEpiSwigluGrad) {
    if (c.dh == nullptr || c.lddh < c.N / 2) return BWG_ERR_INVALID_ARG;
    if (!rows16(c.dh, c.lddh)) return BWG_ERR_ALIGNMENT;
  }
  if (c.K == 0) return BWG_OK;
  if (c.x == nullptr || c.w == nullptr || c.ldx < c.K || c.ldw < (c.w_nt ? c.K : c.N)) return BWG_ERR_INVALID_ARG;
  if (!rows16(c.x, c.ldx) || c.ldw % 8 != 0) return BWG_ERR_ALIGNMENT;
  for (int g = 0; g < c.G; ++g) {
    if (c.w[g] == nullptr) return BWG_ERR_INVALID_ARG;
    if (!is_aligned(c.w[g], 16)) return BWG_ERR_ALIGNMENT;
  }
  return BWG_OK;
}

bool gated_maps(const GatedCall& c, GemmParams* p, GatedExtra* x) {
  const CUtensorMapDataType t =
      c.dtype == BWG_OUT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t I = static_cast<uint64_t>(c.N / 2), M = static_cast<uint64_t>(c.M);
  const uint64_t row = static_cast<uint64_t>(c.ldd) * 2;
  if (!runtime_map_2d(&p->map_a, c.x, t, c.K, M, static_cast<uint64_t>(c.ldx) * 2, kBK, kRowsPerCta)) return false;
  if (c.epi == kEpiSwigluKeep && c.N / 2 % 16 == 0) {
    const uint64_t dims[3] = {I, M, 2}, strides[2] = {2 * I, I};
    const uint32_t box[3] = {64, 32, 1};
    if (!runtime_map(&x->map_x, c.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_64B))
      return false;
  }
  if (c.epi != kEpiSwigluGrad) return runtime_map_2d(&p->map_d, c.d, t, I, M, row, 64, 32);
  if (!runtime_map_2d(&x->map_x, c.dh, t, I, M, static_cast<uint64_t>(c.lddh) * 2, 64, 32)) return false;
  // gate's and up's gradients as two planes of I columns, so that a box at
  // the end of gate's columns stops there
  const uint64_t dims[3] = {I, M, 2}, strides[2] = {row, I * 2};
  const uint32_t box[3] = {64, 32, 1};
  return runtime_map(&p->map_d, c.d, t, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool gated_weight_map(const GatedCall& c, CUtensorMap* m, const void* w) {
  const CUtensorMapDataType t =
      c.dtype == BWG_OUT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return runtime_map_2d(m, w, t, c.w_nt ? c.K : c.N, c.w_nt ? c.N : c.K, static_cast<uint64_t>(c.ldw) * 2, 64, 64);
}

void gated_params(const GatedCall& c, const Runtime& rt, int stages, GemmParams* p, GatedExtra* x) {
  const int I = c.N / 2;
  p->err = rt.err;
  p->d_ptr = c.d;
  p->timeout_ns = rt.timeout_ns;
  p->M = c.M;
  p->N = I;
  p->K = c.K;
  p->ldd = c.ldd;
  p->box_cols = I;  // rows of whole 16 bytes
  p->num_n_tiles = (I + kTileN / 2 - 1) / (kTileN / 2);
  p->num_k_blocks = (c.K + kBK - 1) / kBK;
  p->group_m = kGroupM;
  p->stages = stages;
  p->out_dtype = c.dtype;
  p->idesc = make_idesc_f16(c.dtype == BWG_OUT_FP16 ? kFmtF16 : kFmtBF16, false, !c.w_nt, 2 * kRowsPerCta, kTileN);
  p->b_kmajor = c.w_nt ? 1 : 0;
  p->swiglu_up = I;
  p->tx_extra = rt.tx_extra;
  p->trace = rt.trace;
  p->no_tail_split = rt.no_tail_split;
  x->codes = static_cast<uint8_t*>(c.codes);
  x->scales = c.scales;
  x->blocks = (I + kInt8Block - 1) / kInt8Block;
  x->wide = I % 16 == 0 ? 1 : 0;
}

bwg_status run_gated_dense(const GatedCall& c, const Runtime& rt, cudaStream_t stream) {
  const int I = c.N / 2, n_tiles = (I + kTileN / 2 - 1) / (kTileN / 2);
  constexpr int kStages = 6;
  const int smem = dense_smem(2, kStages, false, 1);
  if (smem > rt.max_smem) return BWG_ERR_UNSUPPORTED;
  DenseGatedParams p;
  std::memset(&p, 0, sizeof(p));
  if (!gated_maps(c, &p, &p.x) || !gated_weight_map(c, &p.map_b, c.w[0])) return BWG_ERR_CUDA;
  // a pair CTA's 128 columns of a stage in one load: [K, N] as 64-column
  // groups, where gate and up both start on one; [N, K] as rows
  if (c.w_nt || I % 64 == 0) {
    const CUtensorMapDataType t =
        c.dtype == BWG_OUT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t ldb = static_cast<uint64_t>(c.ldw) * 2;
    bool ok;
    if (c.w_nt) {
      ok = runtime_map_2d(&p.map_b1, c.w[0], t, c.K, c.N, ldb, 64, 128);
    } else {
      const uint64_t dims[3] = {64, static_cast<uint64_t>(c.K), static_cast<uint64_t>(c.N / 64)};
      const uint64_t strides[2] = {ldb, 128};
      const uint32_t box[3] = {64, 64, 2};
      ok = runtime_map(&p.map_b1, c.w[0], t, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (!ok) return BWG_ERR_CUDA;
    p.b_one_box = 1;
  }
  gated_params(c, rt, kStages, &p, &p.x);
  const int tile_m = 2 * kRowsPerCta;
  p.num_m_tiles = (c.M + tile_m - 1) / tile_m;
  const long long tiles = static_cast<long long>(p.num_m_tiles) * n_tiles;
  if (tiles > 0x3fffffff) return BWG_ERR_UNSUPPORTED;
  // with pairs for all their parts, few tiles are cut
  p.workers = static_cast<int>(std::min<long long>(tiles * 2, rt.pairs));
  return runtime_status(launch_gated_dense(p, c.epi, 2 * p.workers, smem, stream));
}

bwg_status run_gated_grouped(const GatedCall& c, const Runtime& rt, cudaStream_t stream) {
  constexpr int kStages = 6;
  const int smem = dense_smem(2, kStages, false, 1);
  if (smem > rt.max_smem) return BWG_ERR_UNSUPPORTED;
  for (int g0 = 0; g0 < c.G; g0 += kMaxGroupsPerLaunch) {
    const int gn = std::min(kMaxGroupsPerLaunch, c.G - g0);
    GroupedGatedParams P;
    std::memset(&P, 0, sizeof(P));
    GemmParams& p = P.base;
    if (!gated_maps(c, &p, &P.x)) return BWG_ERR_CUDA;
    for (int i = 0; i < gn; ++i)
      if (!gated_weight_map(c, &P.map_b[i], c.w[g0 + i])) return BWG_ERR_CUDA;
    gated_params(c, rt, kStages, &p, &P.x);
    p.group_offsets = c.offsets;
    p.G = gn;
    p.g_begin = g0;
    p.G_total = c.G;
    // as in the grouped products: at most one partial row tile a group, and a
    // pair for every unit that the last wave's cut can make
    const int tile_m = 2 * kRowsPerCta;
    const long long max_tiles = (static_cast<long long>((c.M + tile_m - 1) / tile_m) + gn) * p.num_n_tiles;
    p.workers = static_cast<int>(std::min<long long>(max_tiles, rt.pairs));
    const long long pairs = max_tiles + 3LL * p.workers;
    if (2 * pairs > 0x7fffffffLL) return BWG_ERR_UNSUPPORTED;
    const cudaError_t e = launch_gated_grouped(P, c.epi, static_cast<int>(2 * pairs), smem, stream);
    if (e != cudaSuccess) return runtime_status(e);
  }
  return BWG_OK;
}

bwg_status run_gated(const GatedCall& c, cudaStream_t stream) {
  bwg_status s = check_gated(c);
  if (s != BWG_OK || c.G == 0 || c.M == 0 || c.N == 0) return s;
  Runtime rt;
  if ((s = runtime_device(&rt)) != BWG_OK) return s;
  if (c.K == 0) {
    // gate and up are zero, and so is all that is made of them
    const int d_cols = c.epi == kEpiSwigluGrad ? c.N : c.N / 2;
    cudaError_t e = launch_zero_fill(c.d, c.M, d_cols, c.ldd, 2, stream);
    if (e == cudaSuccess && c.epi == kEpiSwigluKeep) {
      const int blocks = 2 * ((c.N / 2 + kInt8Block - 1) / kInt8Block);
      e = launch_zero_fill(c.codes, c.M, c.N, c.N, 1, stream);
      if (e == cudaSuccess) e = launch_zero_fill(c.scales, c.M, blocks, blocks, 4, stream);
    }
    return runtime_status(e);
  }
  // few rows: W streams through once, as in gemm_bf16
  if (c.offsets == nullptr && c.epi == kEpiSwiglu && c.M <= kSmallMMaxM)
    return run_small_m_gated(c.x, c.w[0], c.d, c.dtype, c.w_nt != 0, c.M, c.N, c.K, c.ldx, c.ldw, c.ldd, stream);
  return c.offsets == nullptr ? run_gated_dense(c, rt, stream) : run_gated_grouped(c, rt, stream);
}

}  // namespace
}  // namespace bwg

extern "C" {

bwg_status gemm_swiglu(const void* X, const void* W, void* H, void* codes, float* scales, int dtype, int w_transposed,
                       int M, int N, int K, int ldx, int ldw, int ldh, void* stream) {
  const bool keep = codes != nullptr || scales != nullptr;
  const GatedCall c{dtype, keep ? kEpiSwigluKeep : kEpiSwiglu, X, &W, H, codes, scales, nullptr, nullptr, 1,
                    w_transposed, M, N, K, ldx, ldw, ldh, 0};
  return run_gated(c, static_cast<cudaStream_t>(stream));
}

bwg_status gemm_swiglu_grad(const void* dH, const void* X, const void* W, void* dGU, int dtype, int w_transposed,
                            int M, int N, int K, int lddh, int ldx, int ldw, int ldd, void* stream) {
  const GatedCall c{dtype, kEpiSwigluGrad, X, &W, dGU, nullptr, nullptr, dH, nullptr, 1, w_transposed, M, N, K, ldx,
                    ldw, ldd, lddh};
  return run_gated(c, static_cast<cudaStream_t>(stream));
}

bwg_status grouped_gemm_swiglu_keep(const void* X, const void* const* W, void* H, void* codes, float* scales,
                                    const int* group_offsets, int dtype, int w_transposed, int G, int M_total, int N,
                                    int K, void* stream) {
  if (G > 0 && M_total > 0 && N > 0 && group_offsets == nullptr) return BWG_ERR_INVALID_ARG;
  const GatedCall c{dtype, kEpiSwigluKeep, X, W, H, codes, scales, nullptr, group_offsets, G, w_transposed, M_total,
                    N, K, K, w_transposed ? K : N, N / 2, 0};
  return run_gated(c, static_cast<cudaStream_t>(stream));
}

bwg_status grouped_gemm_swiglu_grad(const void* dH, const void* X, const void* const* W, void* dGU,
                                    const int* group_offsets, int dtype, int w_transposed, int G, int M_total, int N,
                                    int K, void* stream) {
  if (G > 0 && M_total > 0 && N > 0 && group_offsets == nullptr) return BWG_ERR_INVALID_ARG;
  const GatedCall c{dtype, kEpiSwigluGrad, X, W, dGU, nullptr, nullptr, dH, group_offsets, G, w_transposed, M_total, N,
                    K, K, w_transposed ? K : N, N, N / 2};
  return run_gated(c, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
