// Products whose left operand is read transposed (gemm_body.cuh, TN):
// D[g] = A_g^T B_g, the gradient of a weight from a layer's input A and the
// gradient B of its output, over all rows or over each expert's.
//
// Both operands are summed over their rows, so both enter MN-major, as stored: no
// transpose.  What bounds them: tensor cores and the power limit (8192^3 in BF16
// 605 us back to back, 1.82 PFLOP/s; FP32 results 643), and where D is small
// the rate at which a slice's rows come from L2.
#include <algorithm>
#include <cstring>

#include "gemm_body.cuh"
#include "runtime.h"

using namespace bwg;

namespace bwg {
namespace {

// 512x256 tiles, sums in TMEM.
template <bool DYN>
__global__ void __launch_bounds__(kThreads2C, 1) gemm_tn_2c_kernel(const __grid_constant__ TnParams p) {
  gemm_body<2, 1, false, 2, kEpiPlain, DYN, true, false>(p, p);
}

// 256x256 tiles, sums of kChunkBlocks k-blocks joined in registers.
template <bool DYN>
__global__ void __launch_bounds__(kThreads2C, 1) gemm_tn_joined_kernel(const __grid_constant__ TnParams p) {
  gemm_body<2, 1, false, 1, kEpiPlain, DYN, true, true>(p, p);
}

// D[g] = the sum of its slices' planes, FP32 [G * splits][M][pitch], in order.
struct JoinParams {
  const float* planes;
  void* d;
  int M, N, pitch, splits, ldd;
  long long rows;  // of all groups' D
};

template <int OUT>
__global__ void __launch_bounds__(256) tn_join_kernel(const __grid_constant__ JoinParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const float* const planes = p.planes;
  void* const d = p.d;
  const int M = p.M, N = p.N, pitch = p.pitch, splits = p.splits, ldd = p.ldd, quads = pitch / 4;
  const long long rows = p.rows;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < rows * quads; i += gridDim.x * 256LL) {
    const long long row = i / quads;  // of all groups' rows of D
    const int col = static_cast<int>(i - row * quads) * 4;
    const long long g = row / M;
    const float* src = planes + (g * splits * M + (row - g * M)) * pitch + col;
    float4 s = *reinterpret_cast<const float4*>(src);
    for (int k = 1; k < splits; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(src + static_cast<long long>(k) * M * pitch);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
    if constexpr (OUT == kOutF32) {
      float* dst = static_cast<float*>(d) + row * ldd + col;
      if (col + 4 <= N) {
        *reinterpret_cast<float4*>(dst) = s;
      } else {
        for (int j = 0; col + j < N; ++j) dst[j] = v[j];
      }
    } else {
      uint16_t* dst = static_cast<uint16_t*>(d) + row * ldd + col;
      uint16_t w[4];
      for (int j = 0; j < 4; ++j)
        w[j] = static_cast<uint16_t>(OUT == kOutBF16 ? cvt_rn_bf16(v[j]) : cvt_rn_f16(v[j]));
      if (col + 4 <= N) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0] | (static_cast<uint32_t>(w[1]) << 16),
                                                    w[2] | (static_cast<uint32_t>(w[3]) << 16));
      } else {
        for (int j = 0; col + j < N; ++j) dst[j] = w[j];
      }
    }
  }
}

}  // namespace

cudaError_t launch_tn(const TnParams& p, bool joined, bool dynamic, int grid, size_t smem, cudaStream_t s) {
  if (joined)
    return dynamic ? launch_pair_behind(gemm_tn_joined_kernel<true>, p, grid, smem, s)
                   : launch_pair_behind(gemm_tn_joined_kernel<false>, p, grid, smem, s);
  return dynamic ? launch_pair_behind(gemm_tn_2c_kernel<true>, p, grid, smem, s)
                 : launch_pair_behind(gemm_tn_2c_kernel<false>, p, grid, smem, s);
}

cudaError_t set_tn_attributes(size_t smem) {
  const void* fns[] = {reinterpret_cast<const void*>(gemm_tn_2c_kernel<false>),
                       reinterpret_cast<const void*>(gemm_tn_2c_kernel<true>),
                       reinterpret_cast<const void*>(gemm_tn_joined_kernel<false>),
                       reinterpret_cast<const void*>(gemm_tn_joined_kernel<true>)};
  return set_max_smem(fns, smem);
}

// ---------------------------------------------------------- entry points ---

namespace {

struct TnCall {
  int dtype, out_dtype;
  const void* a;       // [rows, M]
  const void* b;       // [rows, N]
  void* d;             // G planes [M, N]
  const int* offsets;  // nullptr: one group of all rows
  int G, M, N, rows, lda, ldb, ldd;
  float* workspace;
  long long workspace_bytes;
};

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// How a product is cut up: tiles of 256x256 whose sums are joined in registers, or
// of 512x256, which load a quarter less for each element, and slices of each
// group's rows where D has few tiles.
struct TnPlan {
  bool joined;
  int splits;
};

// Waves of T tiles on C pairs, the last one cut as the schedule cuts it.
double tn_waves(long long T, int C, int nc) {
  const int workers = static_cast<int>(std::min<long long>(C, T * (nc == 2 ? 4 : 2)));
  const long long full = T / workers, R = T % workers;
  if (R == 0) return static_cast<double>(full);
  auto part = [&](int f, double cost) { return static_cast<double>((f * R + workers - 1) / workers) * cost; };
  const double last = nc == 2 ? std::min(part(2, kCostHalf2 / 1000.0), part(4, kCostQuarter2 / 1000.0))
                              : part(2, kCostHalf1 / 1000.0);
  return static_cast<double>(full) + std::min(1.0, last);
}

// Rows that one sum in TMEM may take.  Every step of 16 rows cuts up to 2^-23 of the
// sum, towards zero, so that sums of equal signs end short by up to rows / 16 2^-23
// (measured: 0.85 of that, 1.3e-3 at 200000 rows): at most an eighth of the result's
// rounding, 2^-11 in FP16 and 2^-8 in BF16.  FP32 results are joined at once.
int tn_max_rows(int out_dtype) {
  return out_dtype == BWG_OUT_FP32 ? kChunkBlocks * kBK : out_dtype == BWG_OUT_FP16 ? 8192 : 65536;
}

// The cheapest by an estimate in us: a tile's k-blocks, filling the ring and storing
// the tile, and for slices a launch and 8 bytes an element of every plane at 6 TB/s.
// 20011 rows of 1000 x 1416: 256x256 tiles in one slice 106 us, in three 57, 512x256
// tiles in six 50.  At 16 sizes from 256 x 256 to 4096 x 8192 the chosen form is at
// most 15% slower than the best of up to 26 (4% on average; 300 to 1500 rows are
// where it misses).
TnPlan tn_plan(int M, int N, int rows, int G, int out_dtype, int pairs, int pairs_2c) {
  // all rows may be one group's
  const int max_rows = tn_max_rows(out_dtype);
  const bool exact = out_dtype == BWG_OUT_FP32 && rows > max_rows;
  const double blocks = static_cast<double>(ceil_div(rows, kBK)) / G;
  TnPlan best{true, 1};
  double least = 0;
  for (int nc = 1; nc <= (exact ? 1 : 2); ++nc) {
    const long long tiles =
        static_cast<long long>(G) * ceil_div(M, 2 * kRowsPerCta * nc) * ceil_div(N, kTileN);
    const int all = nc == 2 ? pairs_2c : pairs;
    for (int s : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32}) {
      if (s > 1 && (blocks < 8.0 * s || tiles >= 2 * all)) break;
      if (nc == 2 && ceil_div(ceil_div(rows, kBK), s) > max_rows / kBK) continue;
      double t = tn_waves(tiles * s, all, nc) * (blocks / s * (nc == 2 ? 0.56 : 0.40) + (nc == 2 ? 4.5 : 3.0));
      if (s > 1) t += 3.0 + static_cast<double>(G) * s * M * N * 8 / 6.0e6;
      if ((nc == 1 && s == 1) || t < least) {
        least = t;
        best = TnPlan{nc == 1, s};
      }
    }
  }
  return best;
}

int tn_pitch(int N) { return (N + 3) / 4 * 4; }

long long tn_workspace(const TnPlan& plan, int M, int N, int G) {
  return plan.splits == 1 ? 0 : 4LL * G * plan.splits * M * tn_pitch(N);
}

CUtensorMapDataType map_type(int dtype) {
  return dtype == BWG_OUT_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
         : dtype == BWG_OUT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

bwg_status check_tn(const TnCall& c) {
  if (c.dtype != BWG_OUT_BF16 && c.dtype != BWG_OUT_FP16) return BWG_ERR_INVALID_ARG;
  if (c.out_dtype != BWG_OUT_BF16 && c.out_dtype != BWG_OUT_FP16 && c.out_dtype != BWG_OUT_FP32)
    return BWG_ERR_INVALID_ARG;
  if (c.G < 0 || c.M < 0 || c.N < 0 || c.rows < 0) return BWG_ERR_INVALID_ARG;
  if (c.G == 0 || c.M == 0 || c.N == 0) return BWG_OK;
  if (c.M > kMaxSize || c.N > kMaxSize || c.rows > kMaxSize) return BWG_ERR_UNSUPPORTED;
  if (c.d == nullptr || c.ldd < c.N) return BWG_ERR_INVALID_ARG;
  const int oe = c.out_dtype == BWG_OUT_FP32 ? 4 : 2;
  if (!is_aligned(c.d, 16) || static_cast<long long>(c.ldd) * oe % 16 != 0) return BWG_ERR_ALIGNMENT;
  if (c.rows == 0) return BWG_OK;
  if (c.a == nullptr || c.b == nullptr || c.lda < c.M || c.ldb < c.N) return BWG_ERR_INVALID_ARG;
  if (!is_aligned(c.a, 16) || !is_aligned(c.b, 16) || c.lda % 8 != 0 || c.ldb % 8 != 0) return BWG_ERR_ALIGNMENT;
  return BWG_OK;
}

// Windows of kBK rows, one for every row that a window can start at (see
// gemm_body): boxes of 64 columns, or (pair) of 128 as two groups of 64.
bool window_map(CUtensorMap* m, const void* p, int dtype, int cols, int rows, int ld, bool pair) {
  const uint64_t row = static_cast<uint64_t>(ld) * 2;
  const uint64_t dims[4] = {pair ? 64 : static_cast<uint64_t>(cols), static_cast<uint64_t>(kBK),
                            static_cast<uint64_t>(rows), static_cast<uint64_t>(cols / 64)};
  const uint64_t strides[3] = {row, row, 128};
  const uint32_t box[4] = {64, kBK, 1, 2};
  return runtime_map(m, p, map_type(dtype), pair ? 4 : 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bwg_status run_tn(const TnCall& c, cudaStream_t stream) {
  bwg_status s = check_tn(c);
  if (s != BWG_OK || c.G == 0 || c.M == 0 || c.N == 0) return s;
  Runtime rt;
  if ((s = runtime_device(&rt)) != BWG_OK) return s;
  const int oe = c.out_dtype == BWG_OUT_FP32 ? 4 : 2;
  if (c.rows == 0) {
    const long long all = static_cast<long long>(c.G) * c.M;
    if (all > 0x7fffffffLL) return BWG_ERR_UNSUPPORTED;
    return runtime_status(launch_zero_fill(c.d, static_cast<int>(all), c.N, c.ldd, oe, stream));
  }
  const int n_tiles = ceil_div(c.N, kTileN);
  const TnPlan plan = tn_plan(c.M, c.N, c.rows, c.G, c.out_dtype, rt.pairs, rt.pairs_2c);
  const bool joined = plan.joined;
  const int splits = plan.splits;
  const int pitch = tn_pitch(c.N);
  if (splits > 1) {
    if (c.workspace == nullptr || c.workspace_bytes < tn_workspace(plan, c.M, c.N, c.G))
      return BWG_ERR_INVALID_ARG;
    if (!is_aligned(c.workspace, 16)) return BWG_ERR_ALIGNMENT;
  }
  void* const planes = splits > 1 ? c.workspace : c.d;  // what the product writes
  const int plane_type = splits > 1 ? BWG_OUT_FP32 : c.out_dtype;
  const int plane_ld = splits > 1 ? pitch : c.ldd, pe = splits > 1 ? 4 : oe;
  const int nc = joined ? 1 : 2, stages = joined ? 6 : 4;
  const int smem = dense_smem(2, stages, false, nc);
  if (smem > rt.max_smem) return BWG_ERR_UNSUPPORTED;
  for (int g0 = 0; g0 < c.G; g0 += kMaxGroupsPerLaunch) {
    TnParams p;
    std::memset(&p, 0, sizeof(p));
    const uint64_t row = static_cast<uint64_t>(plane_ld) * pe;
    const uint64_t dims[3] = {static_cast<uint64_t>(c.N), static_cast<uint64_t>(c.M),
                              static_cast<uint64_t>(c.G) * splits};
    const uint64_t strides[2] = {row, row * c.M};
    const uint32_t box[3] = {pe == 4 ? 32u : 64u, 32, 1};
    // whole groups of 64 columns; what is left of a row takes plain boxes
    p.a_grouped = c.M / 64 * 64;
    p.b_grouped = c.N / 64 * 64;
    if (!window_map(&p.map_a, c.a, c.dtype, c.M, c.rows, c.lda, false) ||
        !window_map(&p.map_b, c.b, c.dtype, c.N, c.rows, c.ldb, false) ||
        (p.a_grouped > 0 && !window_map(&p.map_a1, c.a, c.dtype, c.M, c.rows, c.lda, true)) ||
        (p.b_grouped > 0 && !window_map(&p.map_b1, c.b, c.dtype, c.N, c.rows, c.ldb, true)) ||
        !runtime_map(&p.map_d, planes, map_type(plane_type), 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return BWG_ERR_CUDA;
    p.err = rt.err;
    p.d_ptr = planes;
    p.group_offsets = c.offsets;
    p.timeout_ns = rt.timeout_ns;
    p.M = c.M;
    p.N = c.N;
    p.K = c.rows;
    p.ldd = plane_ld;
    p.box_cols = splits > 1 ? c.N : box_columns(c.N, oe);  // a plane's rows end in whole 16 bytes
    p.num_m_tiles = ceil_div(c.M, 2 * kRowsPerCta * nc);
    p.num_n_tiles = n_tiles;
    p.group_m = kGroupM;
    p.stages = stages;
    p.out_dtype = plane_type;
    p.idesc = make_idesc_f16(c.dtype == BWG_OUT_FP16 ? kFmtF16 : kFmtBF16, true, true, 2 * kRowsPerCta, kTileN);
    p.tx_extra = rt.tx_extra;
    p.trace = rt.trace;
    p.no_tail_split = rt.no_tail_split;
    p.splits = splits;
    p.G = std::min(kMaxGroupsPerLaunch, c.G - g0);
    p.g_begin = g0;
    p.G_total = c.G;
    const long long tiles = static_cast<long long>(p.G) * splits * p.num_m_tiles * n_tiles;
    if (tiles > 0x0fffffff) return BWG_ERR_UNSUPPORTED;
    // with pairs for all their parts, few tiles are cut
    p.workers = static_cast<int>(std::min<long long>(tiles * (joined ? 2 : 4), joined ? rt.pairs : rt.pairs_2c));
    // groups differ in length: units are claimed at run time
    const bool dynamic = c.offsets != nullptr;
    const long long pairs = dynamic ? tiles + 3LL * p.workers : p.workers;
    const cudaError_t e = launch_tn(p, joined, dynamic, static_cast<int>(2 * pairs), smem, stream);
    if (e != cudaSuccess) return runtime_status(e);
  }
  if (splits == 1) return BWG_OK;
  const long long rows = static_cast<long long>(c.G) * c.M;
  const unsigned grid =
      static_cast<unsigned>(std::min<long long>((rows * (pitch / 4) + 255) / 256, 16LL * rt.sm_count));
  const JoinParams j{c.workspace, c.d, c.M, c.N, pitch, splits, c.ldd, rows};
  return runtime_status(
      launch_behind(c.out_dtype == BWG_OUT_FP32   ? tn_join_kernel<kOutF32>
                    : c.out_dtype == BWG_OUT_BF16 ? tn_join_kernel<kOutBF16>
                                                  : tn_join_kernel<kOutF16>,
                    grid, 256, 0, stream, 1, j));
}

}  // namespace
}  // namespace bwg

extern "C" {

long long bwg_tn_workspace(int M, int N, int K_total, int G, int out_dtype) {
  if (M < 1 || N < 1 || K_total < 1 || G < 1 || M > kMaxSize || N > kMaxSize || K_total > kMaxSize) return 0;
  Runtime rt;
  if (runtime_device(&rt) != BWG_OK) return 0;
  return tn_workspace(tn_plan(M, N, K_total, G, out_dtype, rt.pairs, rt.pairs_2c), M, N, G);
}

bwg_status gemm_tn(const void* A, const void* B, void* D, int dtype, int out_dtype, int M, int N, int K, int lda,
                   int ldb, int ldd, void* workspace, long long workspace_bytes, void* stream) {
  return run_tn(TnCall{dtype, out_dtype, A, B, D, nullptr, 1, M, N, K, lda, ldb, ldd, static_cast<float*>(workspace),
                       workspace_bytes},
                static_cast<cudaStream_t>(stream));
}

bwg_status grouped_gemm_tn(const void* A, const void* B, void* D, const int* group_offsets, int dtype, int out_dtype,
                           int G, int M, int N, int K_total, void* workspace, long long workspace_bytes,
                           void* stream) {
  if (G > 0 && M > 0 && N > 0 && group_offsets == nullptr) return BWG_ERR_INVALID_ARG;
  return run_tn(TnCall{dtype, out_dtype, A, B, D, group_offsets, G, M, N, K_total, M, N, N,
                       static_cast<float*>(workspace), workspace_bytes},
                static_cast<cudaStream_t>(stream));
}

}  // extern "C"
