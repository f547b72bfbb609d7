// Quantising to microscaled 4-bit floating point and reading it back
// (formats and layout: fp4.h).
//
//   nvfp4: s = e4m3(min(amax / (6 g), 448)),  code = e2m1(x / (s g))
//   mxfp4: s = 2^(max(floor(log2 amax) - 2, -127)),  code = e2m1(x / s)
// with amax the largest magnitude of the block and g the matrix's (or the
// group's) FP32 scale.  Every conversion rounds to nearest, ties to even, and
// saturates; the quotients are FP32 quotients.  A block whose scale is zero
// has zero codes; a block holding an infinity or a NaN gets a NaN scale and
// zero codes, so that all of it reads back as NaN.
//
// What bounds these kernels: HBM.  One pass: a thread owns a block, so that
// its maximum needs no exchange between threads.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/bwgemm.h"
#include "fp4.h"
#include "params.h"
#include "ptx.cuh"
#include "runtime.h"

namespace bwg {
namespace {

constexpr int kFp4MaxGroups = 1024;
constexpr int kFp4Threads = 256;

struct Fp4Params {
  const void* x;         // quantise: input; dequantise: unused
  void* y;               // dequantise: output
  uint8_t* codes;
  uint8_t* scales;
  const float* global;   // nullptr: 1
  const int* offsets;    // ragged groups: [G + 1], else nullptr
  unsigned long long* err;
  long long ldx;         // elements
  int M, K, G;
  int n_global;          // 1 or G
  int k_tiles;
  int nb;                // blocks a row
  int lanes_per_row;     // blocks a row rounded up to whole warps
};

// Group tables of a ragged matrix in shared memory: first row of each group
// (clamped into [0, M], non-decreasing) and its first scale row.
struct Groups {
  int* lo;  // [G + 1]
  int* sf;  // [G]
};

__device__ void build_groups(const Fp4Params& p, const Groups& t) {
  if (threadIdx.x < 32) {
    const int lane = static_cast<int>(threadIdx.x);
    int run = 0, carry = 0;
    bool bad = false;
    for (int g0 = 0; g0 < p.G; g0 += 32) {
      const int g = g0 + lane;
      const bool in = g < p.G;
      const int a = in ? p.offsets[g] : 0;
      const int b = in ? p.offsets[g + 1] : 0;
      if (in && ((g == 0 && a != 0) || b < a || a < 0 || b > p.M)) bad = true;
      int m = in ? max(a, b) : run;
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, m, d);
        if (lane >= d) m = max(m, y);
      }
      const int hi = min(max(m, run), p.M);
      int lo = __shfl_up_sync(0xffffffffu, hi, 1);
      if (lane == 0) lo = run;
      const int rows = in ? pad128(hi - lo) : 0;
      int incl = rows;
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      if (in) {
        t.lo[g] = lo;
        t.lo[g + 1] = hi;
        t.sf[g] = carry + incl - rows;
      }
      carry += __shfl_sync(0xffffffffu, incl, 31);
      run = __shfl_sync(0xffffffffu, hi, 31);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) atomicCAS(p.err, 0ull, kFaultBadOffsets << 56);
  }
  __syncthreads();
}

// Group and scale row of matrix row r; false: r lies in no group.
__device__ __forceinline__ bool locate(const Fp4Params& p, const Groups& t, int r, int* g, long long* row) {
  if (p.offsets != nullptr) {
    if (r >= t.lo[p.G]) return false;
    int a = 0, b = p.G - 1;
    while (a < b) {  // the last group that starts at or before r
      const int mid = (a + b + 1) >> 1;
      if (t.lo[mid] <= r)
        a = mid;
      else
        b = mid - 1;
    }
    *g = a;
    *row = static_cast<long long>(t.sf[a]) + (r - t.lo[a]);
  } else if (p.G > 1) {
    const int per = p.M / p.G;
    *g = r / per;
    *row = static_cast<long long>(*g) * pad128(per) + (r - *g * per);
  } else {
    *g = 0;
    *row = r;
  }
  return true;
}

template <class T>
__device__ __forceinline__ float bits_to_f32(uint32_t half);
template <>
__device__ __forceinline__ float bits_to_f32<__nv_bfloat16>(uint32_t half) {
  return __uint_as_float(half << 16);
}
template <>
__device__ __forceinline__ float bits_to_f32<__half>(uint32_t half) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(half)));
}

// Block of B elements of type T into FP32 and its largest magnitude.
template <class T, int B, bool VEC>
__device__ __forceinline__ float load_block(const T* src, float (&v)[B]) {
  float amax = 0.f;
  bool odd = false;  // an infinity or a NaN
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < B / 4; ++i) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(src) + i);
        v[4 * i] = q.x;
        v[4 * i + 1] = q.y;
        v[4 * i + 2] = q.z;
        v[4 * i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < B; ++i) v[i] = __ldg(reinterpret_cast<const float*>(src) + i);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    odd = m >= 0x7f800000u;
    amax = __uint_as_float(m);
  } else {
    uint32_t w[B / 2];
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < B / 8; ++i) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(src) + i);
        w[4 * i] = q.x;
        w[4 * i + 1] = q.y;
        w[4 * i + 2] = q.z;
        w[4 * i + 3] = q.w;
      }
    } else {
      const unsigned short* s = reinterpret_cast<const unsigned short*>(src);
#pragma unroll
      for (int i = 0; i < B / 2; ++i) w[i] = __ldg(s + 2 * i) | (static_cast<uint32_t>(__ldg(s + 2 * i + 1)) << 16);
    }
    // magnitudes of 16-bit floats order like their bits
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < B / 2; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    odd = m >= kInf;
    amax = bits_to_f32<T>(m);
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      v[2 * i] = bits_to_f32<T>(w[i] & 0xffffu);
      v[2 * i + 1] = bits_to_f32<T>(w[i] >> 16);
    }
  }
  return odd ? __int_as_float(0x7fffffff) : amax;
}

// 8 FP32 values as 8 e2m1 codes (nearest even, saturating).
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* q) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

__device__ __forceinline__ uint32_t cvt_e4m3(float x) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(x));
  return h & 0xffu;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(b)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xffffu)));
}

// Scales the block to codes; returns the scale byte.
template <int FMT, int B>
__device__ __forceinline__ uint32_t quantize_block(float (&v)[B], float amax, float g) {
  if (!(amax <= 3.4028235e38f)) {  // infinity or NaN in the block
#pragma unroll
    for (int i = 0; i < B; ++i) v[i] = 0.f;
    return FMT == kNvfp4 ? 0x7fu : 0xffu;
  }
  if constexpr (FMT == kMxfp4) {
    const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 2;
    const uint32_t s = static_cast<uint32_t>(max(e, 0));
    const float inv = __uint_as_float((254u - s) << 23);  // 2^(127 - s): exact
#pragma unroll
    for (int i = 0; i < B; ++i) v[i] *= inv;
    return s;
  } else {
    const uint32_t sb = cvt_e4m3(fminf(__fdiv_rn(amax, __fmul_rn(6.f, g)), 448.f));
    const float step = __fmul_rn(e4m3_to_f32(sb), g);
    if (!(step > 0.f)) {
      // zero scale: codes are zeros of x's sign
#pragma unroll
      for (int i = 0; i < B; ++i) v[i] = copysignf(0.f, v[i]);
    } else if (const float r = __frcp_rn(step); step > 1e-30f && step < 1e30f && amax * r < 1e30f) {
      // x / step in FP32 from the rounded reciprocal r: q0 = x r, then one
      // correction by the exact remainder (Markstein, 1990); nothing here
      // overflows or loses the remainder's bits
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const float q0 = v[i] * r;
        v[i] = copysignf(fmaf(fmaf(-q0, step, v[i]), r, q0), v[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < B; ++i) v[i] = __fdiv_rn(v[i], step);
    }
    return sb;
  }
}

// Warp w of the grid takes 32 consecutive blocks of one row, a lane each.
template <class T, int FMT, bool VEC>
__global__ void __launch_bounds__(kFp4Threads) quantize_kernel(const __grid_constant__ Fp4Params p) {
  constexpr int B = FMT == kNvfp4 ? 16 : 32;
  extern __shared__ int tab[];
  const Groups t{tab, tab + p.G + 1};
  if (p.offsets != nullptr) build_groups(p, t);
  const int per_row = p.lanes_per_row >> 5;
  const long long items = static_cast<long long>(p.M) * per_row;
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const long long stride = static_cast<long long>(gridDim.x) * (kFp4Threads / 32);
  for (long long w = static_cast<long long>(blockIdx.x) * (kFp4Threads / 32) + (threadIdx.x >> 5); w < items;
       w += stride) {
    const int r = static_cast<int>(w / per_row);
    const int b = static_cast<int>(w % per_row) * 32 + lane;
    int g;
    long long srow;
    const bool has = locate(p, t, r, &g, &srow);
    uint32_t sb = 0;  // blocks past the row's last: the tile's padding
    if (has && b < p.nb) {
      float v[B];
      const float amax = load_block<T, B, VEC>(static_cast<const T*>(p.x) + r * p.ldx + static_cast<long long>(b) * B, v);
      const float gs = p.global != nullptr ? __ldg(p.global + (p.n_global > 1 ? g : 0)) : 1.f;
      sb = quantize_block<FMT, B>(v, amax, gs);
      uint32_t c[B / 8];
#pragma unroll
      for (int i = 0; i < B / 8; ++i) c[i] = pack_e2m1x8(v + 8 * i);
      uint8_t* dst = p.codes + static_cast<long long>(r) * (p.K / 2) + static_cast<long long>(b) * (B / 2);
      if constexpr (B == 16)
        *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
      else
        *reinterpret_cast<uint4*>(dst) = make_uint4(c[0], c[1], c[2], c[3]);
    }
    // four neighbours' scales are one word of a tile
    sb |= __shfl_down_sync(0xffffffffu, sb, 1) << 8;
    sb |= __shfl_down_sync(0xffffffffu, sb, 2) << 16;
    if (has && (lane & 3) == 0 && (b >> 2) < p.k_tiles)
      *reinterpret_cast<uint32_t*>(p.scales + fp4_scale_offset(srow, b, p.k_tiles)) = sb;
  }
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  return pack_bf16x2(a, b);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  return pack_f16x2(a, b);
}

template <class T, int FMT, bool VEC>
__global__ void __launch_bounds__(kFp4Threads) dequantize_kernel(const __grid_constant__ Fp4Params p) {
  constexpr int B = FMT == kNvfp4 ? 16 : 32;
  extern __shared__ int tab[];
  const Groups t{tab, tab + p.G + 1};
  if (p.offsets != nullptr) build_groups(p, t);
  const int per_row = p.lanes_per_row >> 5;
  const long long items = static_cast<long long>(p.M) * per_row;
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const long long stride = static_cast<long long>(gridDim.x) * (kFp4Threads / 32);
  for (long long w = static_cast<long long>(blockIdx.x) * (kFp4Threads / 32) + (threadIdx.x >> 5); w < items;
       w += stride) {
    const int r = static_cast<int>(w / per_row);
    const int b = static_cast<int>(w % per_row) * 32 + lane;
    int g;
    long long srow;
    if (b >= p.nb || !locate(p, t, r, &g, &srow)) continue;
    const uint8_t* src = p.codes + static_cast<long long>(r) * (p.K / 2) + static_cast<long long>(b) * (B / 2);
    uint32_t c[B / 8];
    if constexpr (B == 16) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(src));
      c[0] = q.x;
      c[1] = q.y;
    } else {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(src));
      c[0] = q.x;
      c[1] = q.y;
      c[2] = q.z;
      c[3] = q.w;
    }
    const uint32_t sb = __ldg(p.scales + fp4_scale_offset(srow, b, p.k_tiles));
    float s;
    if constexpr (FMT == kNvfp4)
      s = e4m3_to_f32(sb);
    else
      s = sb == 0xffu ? __int_as_float(0x7fffffff) : sb == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(sb << 23);
    const float gs = p.global != nullptr ? __ldg(p.global + (p.n_global > 1 ? g : 0)) : 1.f;
    float v[B];
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      uint32_t h2;
      const uint16_t byte = static_cast<uint16_t>((c[i / 4] >> (8 * (i % 4))) & 0xffu);
      asm("{\n\t.reg .b8 lo, hi;\n\tmov.b16 {lo, hi}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, lo;\n\t}" : "=r"(h2) : "h"(byte));
      const __half2 h = *reinterpret_cast<const __half2*>(&h2);
      v[2 * i] = __low2float(h) * s * gs;
      v[2 * i + 1] = __high2float(h) * s * gs;
    }
    T* dst = static_cast<T*>(p.y) + r * p.ldx + static_cast<long long>(b) * B;
    if constexpr (sizeof(T) == 4) {
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < B / 4; ++i)
          reinterpret_cast<float4*>(dst)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < B; ++i) reinterpret_cast<float*>(dst)[i] = v[i];
      }
    } else {
      uint32_t o[B / 2];
#pragma unroll
      for (int i = 0; i < B / 2; ++i) o[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < B / 8; ++i)
          reinterpret_cast<uint4*>(dst)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < B; ++i)
          reinterpret_cast<unsigned short*>(dst)[i] = static_cast<unsigned short>(o[i / 2] >> (16 * (i & 1)));
      }
    }
  }
}

bwg_status check_fp4(const void* x, int dtype, int M, int K, int ldx, int format, const float* global, int n_global,
                     const int* offsets, int G, const void* codes, const void* scales, bool* empty) {
  *empty = false;
  if (dtype != BWG_OUT_BF16 && dtype != BWG_OUT_FP16 && dtype != BWG_OUT_FP32) return BWG_ERR_INVALID_ARG;
  if (format != kNvfp4 && format != kMxfp4) return BWG_ERR_INVALID_ARG;
  if (M < 0 || K < 0 || G < 1) return BWG_ERR_INVALID_ARG;
  if (offsets == nullptr && M % G != 0) return BWG_ERR_INVALID_ARG;
  if (K % 32 != 0) return BWG_ERR_ALIGNMENT;
  if (global != nullptr && (format == kMxfp4 || (n_global != 1 && n_global != G))) return BWG_ERR_INVALID_ARG;
  if (G > kFp4MaxGroups) return BWG_ERR_UNSUPPORTED;
  if (M == 0 || K == 0) {
    *empty = true;
    return BWG_OK;
  }
  if (x == nullptr || codes == nullptr || scales == nullptr || ldx < K) return BWG_ERR_INVALID_ARG;
  const uintptr_t elt = dtype == BWG_OUT_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) & (elt - 1)) || (reinterpret_cast<uintptr_t>(codes) & 15u) ||
      (reinterpret_cast<uintptr_t>(scales) & 15u))
    return BWG_ERR_ALIGNMENT;
  return BWG_OK;
}

Fp4Params make_params(const void* x, void* y, int M, int K, int ldx, int format, const float* global, int n_global,
                      const int* offsets, int G, void* codes, void* scales, const Runtime& rt) {
  Fp4Params p = {};
  p.x = x;
  p.y = y;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.global = global;
  p.n_global = n_global;
  p.offsets = offsets;
  p.err = rt.err;
  p.ldx = ldx;
  p.M = M;
  p.K = K;
  p.G = G;
  p.k_tiles = fp4_k_tiles(K, format);
  p.nb = K / fp4_block(format);
  p.lanes_per_row = (p.nb + 31) / 32 * 32;
  return p;
}

using Fp4Kernel = void (*)(Fp4Params);

template <class T, bool VEC>
Fp4Kernel pick(bool quant, int format) {
  if (quant) return format == kNvfp4 ? quantize_kernel<T, kNvfp4, VEC> : quantize_kernel<T, kMxfp4, VEC>;
  return format == kNvfp4 ? dequantize_kernel<T, kNvfp4, VEC> : dequantize_kernel<T, kMxfp4, VEC>;
}

bwg_status run_fp4(bool quant, const void* x, void* y, int dtype, int M, int K, int ldx, int format,
                   const float* global, int n_global, const int* offsets, int G, void* codes, void* scales,
                   cudaStream_t s) {
  bool empty;
  const void* mat = quant ? x : y;
  bwg_status st = check_fp4(mat, dtype, M, K, ldx, format, global, n_global, offsets, G, codes, scales, &empty);
  if (st != BWG_OK || empty) return st;
  Runtime rt;
  if ((st = runtime_device(&rt)) != BWG_OK) return st;
  const Fp4Params p = make_params(x, y, M, K, ldx, format, global, n_global, offsets, G, codes, scales, rt);
  const int elt = dtype == BWG_OUT_FP32 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(mat) & 15u) == 0 && (static_cast<long long>(ldx) * elt) % 16 == 0;
  const Fp4Kernel k = dtype == BWG_OUT_FP32   ? (vec ? pick<float, true>(quant, format) : pick<float, false>(quant, format))
                      : dtype == BWG_OUT_BF16 ? (vec ? pick<__nv_bfloat16, true>(quant, format)
                                                     : pick<__nv_bfloat16, false>(quant, format))
                                              : (vec ? pick<__half, true>(quant, format)
                                                     : pick<__half, false>(quant, format));
  const long long warps = static_cast<long long>(M) * (p.lanes_per_row / 32);
  const long long blocks = std::min<long long>((warps + kFp4Threads / 32 - 1) / (kFp4Threads / 32), rt.sm_count * 8LL);
  const size_t smem = offsets != nullptr ? (2 * static_cast<size_t>(G) + 1) * sizeof(int) : 0;
  k<<<static_cast<unsigned>(blocks), kFp4Threads, smem, s>>>(p);
  return runtime_status(cudaGetLastError());
}

}  // namespace
}  // namespace bwg

using namespace bwg;

extern "C" {

long long bwg_fp4_scale_bytes(int M, int K, int format, int G, int ragged) {
  if (M < 0 || K < 0 || G < 1 || (format != kNvfp4 && format != kMxfp4) || (!ragged && M % G != 0)) return -1;
  const long long rows = ragged ? (M + 127LL * std::min(G, M)) / 128 * 128 : static_cast<long long>(G) * pad128(M / G);
  return rows / 128 * fp4_k_tiles(K, format) * kScaleTileBytes;
}

long long bwg_fp4_scale_offset(long long row, int block, int K, int format) {
  return fp4_scale_offset(row, block, fp4_k_tiles(K, format));
}

uint32_t bwg_idesc_fp4(int format, int m, int n, int scale_id) {
  return make_idesc_fp4(format, static_cast<uint32_t>(m), static_cast<uint32_t>(n), static_cast<uint32_t>(scale_id));
}

bwg_status quantize_fp4(const void* X, int dtype, int M, int K, int ldx, int format, const float* global_scale,
                        int n_global, const int* group_offsets, int G, void* codes, void* scales, void* stream) {
  return run_fp4(true, X, nullptr, dtype, M, K, ldx, format, global_scale, n_global, group_offsets, G, codes, scales,
                 static_cast<cudaStream_t>(stream));
}

bwg_status dequantize_fp4(const void* codes, const void* scales, int format, const float* global_scale, int n_global,
                          const int* group_offsets, int G, void* Y, int dtype, int M, int K, int ldy, void* stream) {
  return run_fp4(false, nullptr, Y, dtype, M, K, ldy, format, global_scale, n_global, group_offsets, G,
                 const_cast<void*>(codes), const_cast<void*>(scales), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
