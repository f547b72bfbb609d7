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
// What bounds these kernels: HBM.  One pass: a lane owns a block, so that its
// maximum needs no exchange between lanes.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <type_traits>

#include "../../include/bwgemm.h"
#include "fp4.h"
#include "launch.h"
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
  int k_tiles;           // scale tiles along K
  int nb;                // blocks a row
  int chunks;            // units along K: U scale tiles each
  int row_blocks;        // 128-row blocks of scales; with offsets, at most that many
};

// Group tables of a ragged matrix in shared memory: first row of each group
// (clamped into [0, M], non-decreasing) and its first scale row.
struct Groups {
  int* lo;  // [G + 1]
  int* sf;  // [G + 1]
};

// Returns the 128-row blocks of scales that the groups fill.
__device__ int build_groups(const Fp4Params& p, const Groups& t) {
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
    if (lane == 0) t.sf[p.G] = carry;
    if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) atomicCAS(p.err, 0ull, kFaultBadOffsets << 56);
  }
  __syncthreads();
  return t.sf[p.G] >> 7;
}

// The rows of one 128-row block of scales: [row, end) of group g, fewer than
// 128 at a group's end; false: the block holds none.
struct RowBlock {
  int g, row, end;
};

__device__ __forceinline__ bool row_block(const Fp4Params& p, const Groups& t, int rb, RowBlock* o) {
  if (p.offsets != nullptr) {
    // the last group whose scales start at or before this block: it holds
    // the block, as empty groups share their start with the next
    int a = 0, b = p.G - 1;
    while (a < b) {
      const int mid = (a + b + 1) >> 1;
      if (t.sf[mid] <= rb * 128)
        a = mid;
      else
        b = mid - 1;
    }
    o->g = a;
    o->row = t.lo[a] + (rb * 128 - t.sf[a]);
    o->end = min(t.lo[a + 1], o->row + 128);
  } else {
    const int per = p.M / p.G, per_blocks = pad128(per) >> 7;
    o->g = rb / per_blocks;
    o->row = o->g * per + (rb - o->g * per_blocks) * 128;
    o->end = min((o->g + 1) * per, o->row + 128);
  }
  return o->row < o->end;
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

// 32 bytes in one access (sm_100 and later).
__device__ __forceinline__ void ld32(const void* p, uint32_t (&w)[8]) {
  asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
      : "l"(p));
}
__device__ __forceinline__ void st32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Words of a block of elements of E bytes, in accesses of VB bytes.
template <int E, int VB, int W>
__device__ __forceinline__ void load_words(const void* src, uint32_t (&w)[W]) {
  if constexpr (VB == 32) {
#pragma unroll
    for (int i = 0; i < W / 8; ++i)
      ld32(static_cast<const char*>(src) + 32 * i, *reinterpret_cast<uint32_t(*)[8]>(&w[8 * i]));
  } else if constexpr (VB == 16) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 q = __ldg(static_cast<const uint4*>(src) + i);
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
  } else if constexpr (E == 4) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __ldg(static_cast<const uint32_t*>(src) + i);
  } else {
    const unsigned short* s = static_cast<const unsigned short*>(src);
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __ldg(s + 2 * i) | (static_cast<uint32_t>(__ldg(s + 2 * i + 1)) << 16);
  }
}

template <int E, int VB, int W>
__device__ __forceinline__ void store_words(void* dst, const uint32_t (&w)[W]) {
  if constexpr (VB == 32) {
#pragma unroll
    for (int i = 0; i < W / 8; ++i) st32(static_cast<char*>(dst) + 32 * i, &w[8 * i]);
  } else if constexpr (VB == 16) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
      static_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else if constexpr (E == 4) {
#pragma unroll
    for (int i = 0; i < W; ++i) static_cast<uint32_t*>(dst)[i] = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 2 * W; ++i)
      static_cast<unsigned short*>(dst)[i] = static_cast<unsigned short>(w[i / 2] >> (16 * (i & 1)));
  }
}

// Larger magnitude of each half of two words of 16-bit floats, NaN winning
// (32768 x 4096 BF16 to mxfp4: 52 us; 57 on the words' bits).
template <class T>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (std::is_same<T, __half>::value)
    asm("{\n\t.reg .b32 x, y;\n\tabs.f16x2 x, %1;\n\tabs.f16x2 y, %2;\n\tmax.NaN.f16x2 %0, x, y;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
  else
    asm("{\n\t.reg .b32 x, y;\n\tabs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.NaN.bf16x2 %0, x, y;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
  return r;
}

// A block's words as FP32 values, and its largest magnitude: infinite or NaN
// where it holds an infinity or a NaN.
template <class T, int B>
__device__ __forceinline__ float unpack_block(const uint32_t* w, float (&v)[B]) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;  // magnitudes of floats order like their bits, NaN above infinity
#pragma unroll
    for (int i = 0; i < B; ++i) {
      m = max(m, w[i] & 0x7fffffffu);
      v[i] = __uint_as_float(w[i]);
    }
    return __uint_as_float(m);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      m = max_abs2<T>(m, w[i]);
      v[2 * i] = bits_to_f32<T>(w[i] & 0xffffu);
      if constexpr (std::is_same<T, __half>::value)
        v[2 * i + 1] = bits_to_f32<T>(w[i] >> 16);
      else
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    m = max_abs2<T>(m, m >> 16);
    return bits_to_f32<T>(m & 0xffffu);
  }
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

// Two FP32 operations in one instruction (sm_100 and later).
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The matrix's (or group's) scale and what a block's scale is computed from.
struct GlobalScale {
  float g, c, rc;  // g, 6 g and about 1 / (6 g)
  bool fast;       // 6 g far from the ends of FP32
};
__device__ __forceinline__ GlobalScale global_scale(const float* p) {
  GlobalScale s;
  s.g = p != nullptr ? __ldg(p) : 1.f;
  s.c = __fmul_rn(6.f, s.g);
  s.rc = rcp_approx(s.c);
  s.fast = s.c > 1e-25f && s.c < 1e25f;
  return s;
}

// Scales the block to what its codes are rounded from (nvfp4: to its negative)
// and stores the scale byte in *sb; false: left to slow_block.
//
// nvfp4's quotients are FP32's x / d from an approximate reciprocal r of d:
// q0 = x r is a few units in the last place off, its remainder x - q0 d is
// exact in an FMA, and q0 plus the remainder times r rounds to the quotient
// (Markstein, 1990; r being approximate, the codes next to every tie were compared
// with FP32 division for all 2^23 mantissas of d, and the scales for every 6 g).
// Computed as -q from -r, so that every factor is a constant of the block and a
// zero gets the sign that a flip of the codes' signs turns
// into its own, also for a zero scale (r = 0).  What could overflow or lose the
// remainder's bits goes to slow_block, out of line, which leaves registers for
// four blocks of threads an SM: 58 us for 32768 x 4096 BF16 (5.9 TB/s) against
// 75 us with that code here, 69 us with it out of line but three blocks, and
// 84 us with divisions, one value at a time.  mxfp4's multiplications: 51 us.
template <int FMT, int B>
__device__ __forceinline__ bool quantize_block(float (&v)[B], float amax, const GlobalScale& gs, uint32_t* sb) {
  if constexpr (FMT == kMxfp4) {
    const uint32_t s = static_cast<uint32_t>(max(static_cast<int>(__float_as_uint(amax) >> 23) - 2, 0));
    const float inv = __uint_as_float((254u - s) << 23);  // 2^(127 - s): exact
#pragma unroll
    for (int i = 0; i < B; ++i) v[i] *= inv;
    *sb = s;
    return amax <= 3.4028235e38f;
  } else {
    const float t0 = amax * gs.rc;
    const uint32_t s = cvt_e4m3(fminf(fmaf(fmaf(-t0, gs.c, amax), gs.rc, t0), 448.f));
    const float step = __fmul_rn(e4m3_to_f32(s), gs.g);
    const float r = step > 0.f ? rcp_approx(step) : 0.f;
    const uint64_t r2 = pair_of(-r, -r), s2 = pair_of(step, step);
#pragma unroll
    for (int i = 0; i < B; i += 2) {
      const uint64_t x2 = pair_of(v[i], v[i + 1]);
      const uint64_t q0 = mul2(x2, r2);                   // -q0
      const uint64_t q = fma2(fma2(q0, s2, x2), r2, q0);  // -q0 - (x - q0 d) r
      asm("mov.b64 {%0, %1}, %2;" : "=f"(v[i]), "=f"(v[i + 1]) : "l"(q));
    }
    *sb = s;
    return gs.fast && t0 < 1e30f;
  }
}

// One block, value by value: an infinity or a NaN in it, or magnitudes near
// the ends of FP32.  Returns the scale byte.
template <class T, int FMT>
__device__ __noinline__ uint32_t slow_block(const T* src, float g, uint8_t* codes) {
  constexpr int B = FMT == kNvfp4 ? 16 : 32;
  float amax = 0.f;
  bool finite = true;
  for (int i = 0; i < B; ++i) {
    const float a = fabsf(static_cast<float>(src[i]));
    finite = finite && a <= 3.4028235e38f;
    amax = fmaxf(amax, a);
  }
  uint32_t s;
  float step;
  if constexpr (FMT == kNvfp4) {
    s = finite ? cvt_e4m3(fminf(__fdiv_rn(amax, __fmul_rn(6.f, g)), 448.f)) : 0x7fu;
    step = __fmul_rn(e4m3_to_f32(s), g);
  } else {
    s = finite ? static_cast<uint32_t>(max(static_cast<int>(__float_as_uint(amax) >> 23) - 2, 0)) : 0xffu;
    step = 0.f;  // only blocks that are not finite come here
  }
  for (int i = 0; i < B; i += 8) {
    float q[8];
    for (int j = 0; j < 8; ++j) {
      const float x = static_cast<float>(src[i + j]);
      q[j] = !finite ? 0.f : step > 0.f ? __fdiv_rn(x, step) : copysignf(0.f, x);
    }
    *reinterpret_cast<uint32_t*>(codes + i / 2) = pack_e2m1x8(q);
  }
  return s;
}

// A unit is one 128-row block of scales x U scale tiles along K, for 8 warps.
// A warp takes rows 2 i, 2 i + 1 of each group of 32 rows (8 rows) and the 4
// blocks of a tile: its 32 scales are one 32-byte sector of the tile, its
// loads and code stores whole sectors.  All U loads of a lane are issued
// before the first is used.
template <class T, int FMT, int VB, int U>
__global__ void __launch_bounds__(kFp4Threads, 4) quantize_kernel(const __grid_constant__ Fp4Params p) {
  constexpr int B = FMT == kNvfp4 ? 16 : 32;
  constexpr int W = B * static_cast<int>(sizeof(T)) / 4;
  extern __shared__ int tab[];
  grid_dependents_launch();
  const Groups t{tab, tab + p.G + 1};
  int row_blocks = p.row_blocks;
  if (p.offsets != nullptr) row_blocks = build_groups(p, t);
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const int q = lane >> 3, h = (lane >> 2) & 1, bl = lane & 3;
  const long long units = static_cast<long long>(row_blocks) * p.chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int rb = static_cast<int>(u / p.chunks);
    const int kt0 = static_cast<int>(u - static_cast<long long>(rb) * p.chunks) * U;
    RowBlock r;
    if (!row_block(p, t, rb, &r)) continue;
    const GlobalScale gs = global_scale(p.global != nullptr ? p.global + (p.n_global > 1 ? r.g : 0) : nullptr);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int in32 = (half * (kFp4Threads / 32) + static_cast<int>(threadIdx.x >> 5)) * 2 + h;
      const int row = r.row + q * 32 + in32;
      if (row >= r.end) continue;
      const T* src = static_cast<const T*>(p.x) + row * p.ldx;
      uint32_t w[U][W];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int b = (kt0 + i) * 4 + bl;
        if (b < p.nb) load_words<sizeof(T), VB, W>(src + static_cast<long long>(b) * B, w[i]);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int b = (kt0 + i) * 4 + bl;
        uint32_t sb = 0;  // blocks past the row's last: the tile's padding
        if (b < p.nb) {
          float v[B];
          const float amax = unpack_block<T, B>(w[i], v);
          const bool done = quantize_block<FMT, B>(v, amax, gs, &sb);
          uint32_t c[B / 8];
#pragma unroll
          for (int j = 0; j < B / 8; ++j) c[j] = pack_e2m1x8(v + 8 * j) ^ (FMT == kNvfp4 ? 0x88888888u : 0u);
          uint8_t* dst = p.codes + static_cast<long long>(row) * (p.K / 2) + static_cast<long long>(b) * (B / 2);
          if constexpr (B == 16)
            *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
          else
            *reinterpret_cast<uint4*>(dst) = make_uint4(c[0], c[1], c[2], c[3]);
          if (!done) sb = slow_block<T, FMT>(src + static_cast<long long>(b) * B, gs.g, dst);
        }
        if (kt0 + i < p.k_tiles)
          p.scales[(static_cast<long long>(rb) * p.k_tiles + kt0 + i) * kScaleTileBytes + in32 * 16 + q * 4 + bl] =
              static_cast<uint8_t>(sb);
      }
    }
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

// The same units and lanes, from codes and scales to values.  mxfp4 blocks go to
// FP32 in halves, two lanes a block: lanes that store 128 bytes each, four times
// a quarter line, need 111 us for 32768 x 4096, lanes of 64 bytes 92.
template <class T, int FMT, int VB, int U>
__global__ void __launch_bounds__(kFp4Threads) dequantize_kernel(const __grid_constant__ Fp4Params p) {
  constexpr int H = FMT == kMxfp4 && sizeof(T) == 4 ? 2 : 1;  // lanes a block
  constexpr int B = (FMT == kNvfp4 ? 16 : 32) / H;            // values a lane
  constexpr int W = B * static_cast<int>(sizeof(T)) / 4;
  extern __shared__ int tab[];
  grid_dependents_launch();
  const Groups t{tab, tab + p.G + 1};
  int row_blocks = p.row_blocks;
  if (p.offsets != nullptr) row_blocks = build_groups(p, t);
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const int q = lane >> 3, h = (lane >> 2) & 1, bl = lane & 3;
  const long long units = static_cast<long long>(row_blocks) * p.chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int rb = static_cast<int>(u / p.chunks);
    const int kt0 = static_cast<int>(u - static_cast<long long>(rb) * p.chunks) * U;
    RowBlock r;
    if (!row_block(p, t, rb, &r)) continue;
    const float gs = p.global != nullptr ? __ldg(p.global + (p.n_global > 1 ? r.g : 0)) : 1.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int in32 = (half * (kFp4Threads / 32) + static_cast<int>(threadIdx.x >> 5)) * 2 + h;
      const int row = r.row + q * 32 + in32;
      if (row >= r.end) continue;
      uint32_t c[U * H][B / 8];
      uint32_t sb[U * H];
#pragma unroll
      for (int i = 0; i < U * H; ++i) {
        const int b = (kt0 * H + i) * 4 + bl;  // counts halves where H == 2
        if (b >= p.nb * H) continue;
        const uint8_t* src = p.codes + static_cast<long long>(row) * (p.K / 2) + static_cast<long long>(b) * (B / 2);
        if constexpr (B == 16) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
          c[i][0] = x.x;
          c[i][1] = x.y;
        } else {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(src));
          c[i][0] = x.x;
          c[i][1] = x.y;
          c[i][2] = x.z;
          c[i][3] = x.w;
        }
        sb[i] = __ldg(p.scales + (static_cast<long long>(rb) * p.k_tiles + kt0 + i / H) * kScaleTileBytes + in32 * 16 +
                      q * 4 + (b / H & 3));
      }
#pragma unroll
      for (int i = 0; i < U * H; ++i) {
        const int b = (kt0 * H + i) * 4 + bl;
        if (b >= p.nb * H) continue;
        float s;
        if constexpr (FMT == kNvfp4)
          s = e4m3_to_f32(sb[i]);
        else
          s = sb[i] == 0xffu ? __int_as_float(0x7fffffff)
                             : sb[i] == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(sb[i] << 23);
        uint32_t o[W];
#pragma unroll
        for (int j = 0; j < B / 2; ++j) {
          uint32_t h2;
          const uint16_t byte = static_cast<uint16_t>((c[i][j / 4] >> (8 * (j % 4))) & 0xffu);
          asm("{\n\t.reg .b8 lo, hi;\n\tmov.b16 {lo, hi}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, lo;\n\t}"
              : "=r"(h2)
              : "h"(byte));
          const __half2 v2 = *reinterpret_cast<const __half2*>(&h2);
          const float lo = __low2float(v2) * s * gs, hi = __high2float(v2) * s * gs;
          if constexpr (sizeof(T) == 4) {
            o[2 * j] = __float_as_uint(lo);
            o[2 * j + 1] = __float_as_uint(hi);
          } else {
            o[j] = pack2<T>(lo, hi);
          }
        }
        store_words<sizeof(T), VB, W>(static_cast<T*>(p.y) + row * p.ldx + static_cast<long long>(b) * B, o);
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
  if (G > kFp4MaxGroups || M > kFp4MaxSize || K > kFp4MaxSize) return BWG_ERR_UNSUPPORTED;
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
  p.row_blocks = offsets != nullptr ? static_cast<int>((M + 127LL * std::min(G, M)) / 128)
                                    : static_cast<int>(static_cast<long long>(G) * pad128(M / G) / 128);
  return p;
}

using Fp4Kernel = void (*)(Fp4Params);

// Scale tiles of a unit: 128 bytes of 16-bit input a lane, half of it on the
// larger types' side; 1 where that leaves SMs idle.
template <class T, int FMT>
constexpr int unit_tiles() {
  return (FMT == kNvfp4 ? 4 : 2) / (sizeof(T) == 4 ? 2 : 1);
}

template <class T, int FMT, int VB>
Fp4Kernel pick_unit(bool quant, bool wide) {
  constexpr int U = unit_tiles<T, FMT>();
  if (quant) return wide ? quantize_kernel<T, FMT, VB, U> : quantize_kernel<T, FMT, VB, 1>;
  return wide ? dequantize_kernel<T, FMT, VB, U> : dequantize_kernel<T, FMT, VB, 1>;
}

template <class T, int FMT>
Fp4Kernel pick_access(bool quant, bool wide, int vb) {
  return vb == 32   ? pick_unit<T, FMT, 32>(quant, wide)
         : vb == 16 ? pick_unit<T, FMT, 16>(quant, wide)
                    : pick_unit<T, FMT, 0>(quant, wide);
}

template <class T>
Fp4Kernel pick(bool quant, bool wide, int format, int vb) {
  return format == kNvfp4 ? pick_access<T, kNvfp4>(quant, wide, vb) : pick_access<T, kMxfp4>(quant, wide, vb);
}

template <class T>
int tiles_of(int format) {
  return format == kNvfp4 ? unit_tiles<T, kNvfp4>() : unit_tiles<T, kMxfp4>();
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
  Fp4Params p = make_params(x, y, M, K, ldx, format, global, n_global, offsets, G, codes, scales, rt);
  const int elt = dtype == BWG_OUT_FP32 ? 4 : 2;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(mat) | static_cast<uintptr_t>(static_cast<long long>(ldx) * elt);
  const int vb = (bits & 31u) == 0 ? 32 : (bits & 15u) == 0 ? 16 : 0;
  const int tiles = dtype == BWG_OUT_FP32   ? tiles_of<float>(format)
                    : dtype == BWG_OUT_BF16 ? tiles_of<__nv_bfloat16>(format)
                                            : tiles_of<__half>(format);
  const long long wide_units = static_cast<long long>(p.row_blocks) * ((p.k_tiles + tiles - 1) / tiles);
  const bool wide = wide_units >= 2LL * rt.sm_count;
  const int U = wide ? tiles : 1;
  p.chunks = (p.k_tiles + U - 1) / U;
  const Fp4Kernel k = dtype == BWG_OUT_FP32   ? pick<float>(quant, wide, format, vb)
                      : dtype == BWG_OUT_BF16 ? pick<__nv_bfloat16>(quant, wide, format, vb)
                                              : pick<__half>(quant, wide, format, vb);
  const long long units = static_cast<long long>(p.row_blocks) * p.chunks;
  // A block a unit: SMs that finish early go on (32768 x 4096 NVFP4 read back
  // as BF16 54 us against 58 with 8 blocks an SM that stride over the units,
  // as FP32 91 against 97).  With ragged groups, whose tables every block
  // builds, 8 an SM: there more or fewer made no difference.
  const long long blocks = std::min<long long>(units, offsets != nullptr ? rt.sm_count * 8LL : 0x7fffffffLL);
  const size_t smem = offsets != nullptr ? (2 * static_cast<size_t>(G) + 2) * sizeof(int) : 0;
  // A plain launch: blocks that start while the work before still holds some SMs
  // gather on the others, and these grids are a round or two of blocks only
  // (quantise before the experts' FC1: 275 us for both so, 260 plain).
  k<<<static_cast<unsigned>(blocks), kFp4Threads, smem, s>>>(p);
  return runtime_status(cudaGetLastError());
}

}  // namespace
}  // namespace bwg

using namespace bwg;

extern "C" {

long long bwg_fp4_scale_bytes(int M, int K, int format, int G, int ragged) {
  if (M < 0 || K < 0 || G < 1 || (format != kNvfp4 && format != kMxfp4) || (!ragged && M % G != 0)) return -1;
  if (M > kFp4MaxSize || K > kFp4MaxSize) return -1;
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
