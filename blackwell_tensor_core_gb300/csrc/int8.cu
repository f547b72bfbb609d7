// Matrices kept in 8 bits between a training step's passes: put there, read
// back, and SwiGLU's gradient from gate and up kept so.
//
//   a = largest magnitude of a block of 64 columns of a row
//   scale = a / 127,  code = rint(x * (127 / a)),  value = code * scale
//
// Both quotients are rounded to FP32 and the product with the second is rounded
// once, to the integer.  A matrix in two parts (gate and up) has blocks of its
// own in each.  A block with an infinity or a NaN in it reads back as NaN; one
// whose largest magnitude is at most 127 * 2^-128 (0.992 * 2^-121) as zero.
//
// What bounds these kernels: HBM.  One pass; four lanes share a block, 16 columns
// each (32 bytes, one load), so that its maximum takes two exchanges and a warp
// reads whole lines; two rows in flight a lane (four: 77 us in place of 68, one:
// 70).  32768 x 4096 BF16: in 68 us (6.0 TB/s), back 63 (6.6); SwiGLU's gradient
// of 32768 x 2048 83 (6.6), with H 104.  Rows that start off 16 bytes: 8192 x 4095
// in 34, back 28 (3.0 and 3.7 TB/s; a value a lane and load), 8192 x 4094 in 30 and
// 21 (two).
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <type_traits>

#include "../../include/bwgemm.h"
#include "params.h"
#include "runtime.h"
#include "swiglu.cuh"

namespace bwg {
namespace {

constexpr int kThreadsInt8 = 256;
constexpr int kRowsPerWarp = 2;   // rows in flight a lane
constexpr int kGradRows = 1;      // the same in SwiGLU's gradient
constexpr int kOddRows = 2;       // the same where nothing is aligned
constexpr int kOddCols = 256;     // and the columns that a warp takes

struct Int8Params {
  const void* x;        // quantise: the matrix; SwiGLU gradient: H's gradient
  void* y;              // read back: the matrix; SwiGLU gradient: [dgate | dup]
  void* h;              // SwiGLU gradient: H, or nullptr
  int8_t* codes;
  float* scales;
  long long ldx, ldy, ldh;  // elements
  long long rows;       // rows of parts: matrix rows x parts
  int cols;             // columns of a part
  int blocks;           // blocks of a part
  int part_bits;        // 0 or 1: log2 of the parts
  int segs;             // column segments of a part's row
  int wide;             // 16-bit matrix: 16 columns start on 32 bytes wherever a lane's do
};

template <int IN>
using Elem = std::conditional_t<IN == kOutF32, float, uint16_t>;

template <int IN>
__device__ __forceinline__ float to_float(Elem<IN> v) {
  if constexpr (IN == kOutF32)
    return v;
  else if constexpr (IN == kOutBF16)
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
  else
    return __half2float(__ushort_as_half(v));
}

template <int OUT>
__device__ __forceinline__ Elem<OUT> from_float(float v) {
  if constexpr (OUT == kOutF32)
    return v;
  else
    return static_cast<uint16_t>(OUT == kOutBF16 ? cvt_rn_bf16(v) : cvt_rn_f16(v));
}

// 32 bytes at once (sm_100 on), 32-byte aligned.
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  asm("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
      : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 8 values from 16-byte aligned memory.
template <int IN>
__device__ __forceinline__ void load8(const Elem<IN>* p, float (&v)[8]) {
  if constexpr (IN == kOutF32) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    unpack_pair(a.x, IN == kOutBF16, &v[0], &v[1]);
    unpack_pair(a.y, IN == kOutBF16, &v[2], &v[3]);
    unpack_pair(a.z, IN == kOutBF16, &v[4], &v[5]);
    unpack_pair(a.w, IN == kOutBF16, &v[6], &v[7]);
  }
}

template <int OUT>
__device__ __forceinline__ void store8(Elem<OUT>* p, const float (&v)[8]) {
  if constexpr (OUT == kOutF32) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    auto pk = [](float a, float b) { return OUT == kOutBF16 ? pack_bf16x2(a, b) : pack_f16x2(a, b); };
    *reinterpret_cast<uint4*>(p) = make_uint4(pk(v[0], v[1]), pk(v[2], v[3]), pk(v[4], v[5]), pk(v[6], v[7]));
  }
}

// The four codes of a word as floats: each byte, its sign bit turned over, as the
// low mantissa bits of 2^23, less 2^23 + 128.
__device__ __forceinline__ void codes4(uint32_t w, float* v) {
  const uint32_t b = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7540u | i)) - 8388736.0f;
}

// Where part row v of a matrix with row stride ld starts.
__device__ __forceinline__ long long part_row(const Int8Params& p, long long v, long long ld) {
  return (v >> p.part_bits) * ld + (v & ((1 << p.part_bits) - 1)) * p.cols;
}

// VEC: rows, parts and their ends lie on multiples of 8 elements in all buffers.
// A warp takes 32 / L rows at a time, L lanes a row of 16 columns each.
template <int IN, int L>
__global__ void __launch_bounds__(kThreadsInt8) quantize_int8_kernel(const Int8Params p) {
  constexpr int kR = 32 / L;
  const int lane = static_cast<int>(threadIdx.x & 31u), sub = lane % L;
  const long long rb = blockIdx.x / p.segs;
  const int seg = static_cast<int>(blockIdx.x - rb * p.segs);
  const int col = (seg * L + sub) * 16;
  const long long row0 = (rb * (kThreadsInt8 / 32) + (threadIdx.x >> 5)) * (kR * kRowsPerWarp) + lane / L;
  float v[kRowsPerWarp][16];
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    const long long row = row0 + r * kR;
    const Elem<IN>* src = static_cast<const Elem<IN>*>(p.x) + part_row(p, row, p.ldx) + col;
    if (IN != kOutF32 && p.wide) {
      uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      if (row < p.rows && col < p.cols) load32(src, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) unpack_pair(w[i], IN == kOutBF16, &v[r][2 * i], &v[r][2 * i + 1]);
      continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (row < p.rows && col + 8 * h < p.cols) load8<IN>(src + 8 * h, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[r][8 * h + i] = t[i];
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    const long long row = row0 + r * kR;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a = max_abs_nan(a, v[r][i]);
      b = max_abs_nan(b, v[r][8 + i]);
    }
    a = max_abs_nan(a, b);
    a = max_abs_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max_abs_nan(a, __shfl_xor_sync(0xffffffffu, a, 2));
    float scale, inv;
    int8_scale(a, &scale, &inv);
    if (row < p.rows && col < p.cols) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack_bytes(int8_code(v[r][4 * i], inv), int8_code(v[r][4 * i + 1], inv),
                          int8_code(v[r][4 * i + 2], inv), int8_code(v[r][4 * i + 3], inv));
      int8_t* dst = p.codes + row * p.cols + col;
      if ((p.cols & 15) == 0) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        reinterpret_cast<uint2*>(dst)[0] = make_uint2(w[0], w[1]);
        if (col + 8 < p.cols) reinterpret_cast<uint2*>(dst)[1] = make_uint2(w[2], w[3]);
      }
      if ((sub & 3) == 0) p.scales[row * p.blocks + (col >> 6)] = scale;
    }
  }
}

// Any width and stride: a warp takes four blocks of a row, two columns of each a
// lane, so that neighbouring lanes read neighbouring elements, V = 1 or 2 at a time
// (2: columns, strides and bases are even).
template <class T, int V>
struct alignas(sizeof(T) * V) Few {
  T v[V];
};

template <int IN, int V>
__global__ void __launch_bounds__(kThreadsInt8) quantize_int8_odd_kernel(const Int8Params p) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const long long rb = blockIdx.x / p.segs;
  const int seg = static_cast<int>(blockIdx.x - rb * p.segs);
  const int col = seg * kOddCols + lane * V;
  const long long row0 = (rb * (kThreadsInt8 / 32) + (threadIdx.x >> 5)) * kOddRows;
  float v[kOddRows][8];  // of block b: 2 b and 2 b + 1
#pragma unroll
  for (int r = 0; r < kOddRows; ++r) {
    const Elem<IN>* src = static_cast<const Elem<IN>*>(p.x) + part_row(p, row0 + r, p.ldx) + col;
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) {
      Few<Elem<IN>, V> t = {};
      if (row0 + r < p.rows && col + 32 * V * i < p.cols)
        t = *reinterpret_cast<const Few<Elem<IN>, V>*>(src + 32 * V * i);
#pragma unroll
      for (int j = 0; j < V; ++j) v[r][V * i + j] = to_float<IN>(t.v[j]);
    }
  }
#pragma unroll
  for (int r = 0; r < kOddRows; ++r) {
    if (row0 + r >= p.rows) break;  // the whole warp
    float a[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) a[b] = max_abs_nan(v[r][2 * b], v[r][2 * b + 1]);
    // lanes 8 b .. 8 b + 7 come to hold block b's maximum
    const bool hi = (lane & 16) != 0, mid = (lane & 8) != 0;
    float m0 = max_abs_nan(hi ? a[2] : a[0], __shfl_xor_sync(0xffffffffu, hi ? a[0] : a[2], 16));
    const float m1 = max_abs_nan(hi ? a[3] : a[1], __shfl_xor_sync(0xffffffffu, hi ? a[1] : a[3], 16));
    m0 = max_abs_nan(mid ? m1 : m0, __shfl_xor_sync(0xffffffffu, mid ? m0 : m1, 8));
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) m0 = max_abs_nan(m0, __shfl_xor_sync(0xffffffffu, m0, d));
    float scale, inv;
    int8_scale(m0, &scale, &inv);
    const int block = seg * (kOddCols / kInt8Block) + (lane >> 3);
    if ((lane & 7) == 0 && block < p.blocks) p.scales[(row0 + r) * p.blocks + block] = scale;
    int8_t* dst = p.codes + (row0 + r) * p.cols + col;
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) {
      const float f = __shfl_sync(0xffffffffu, inv, (V * i >> 1) * 8);
      Few<uint8_t, V> t;
#pragma unroll
      for (int j = 0; j < V; ++j) t.v[j] = static_cast<uint8_t>(int8_code(v[r][V * i + j], f));
      if (col + 32 * V * i < p.cols) *reinterpret_cast<Few<uint8_t, V>*>(dst + 32 * V * i) = t;
    }
  }
}

template <int OUT, int L>
__global__ void __launch_bounds__(kThreadsInt8) dequantize_int8_kernel(const Int8Params p) {
  constexpr int kR = 32 / L;
  const int lane = static_cast<int>(threadIdx.x & 31u), sub = lane % L;
  const long long rb = blockIdx.x / p.segs;
  const int seg = static_cast<int>(blockIdx.x - rb * p.segs);
  const int col = (seg * L + sub) * 16;
  const long long row0 = (rb * (kThreadsInt8 / 32) + (threadIdx.x >> 5)) * (kR * kRowsPerWarp) + lane / L;
  uint32_t w[kRowsPerWarp][4];
  float scale[kRowsPerWarp];
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    const long long row = row0 + r * kR;
    if (row < p.rows && col < p.cols) {
      const int8_t* src = p.codes + row * p.cols + col;
      if ((p.cols & 15) == 0) {
        const uint4 q = *reinterpret_cast<const uint4*>(src);
        w[r][0] = q.x, w[r][1] = q.y, w[r][2] = q.z, w[r][3] = q.w;
      } else {
        const uint2 q = reinterpret_cast<const uint2*>(src)[0];
        w[r][0] = q.x, w[r][1] = q.y;
        if (col + 8 < p.cols) {
          const uint2 q1 = reinterpret_cast<const uint2*>(src)[1];
          w[r][2] = q1.x, w[r][3] = q1.y;
        }
      }
      scale[r] = p.scales[row * p.blocks + (col >> 6)];
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    const long long row = row0 + r * kR;
    Elem<OUT>* dst = static_cast<Elem<OUT>*>(p.y) + part_row(p, row, p.ldy) + col;
    if (OUT != kOutF32 && p.wide) {
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[4];
        codes4(w[r][i], v);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          o[2 * i + j] = OUT == kOutBF16 ? pack_bf16x2(v[2 * j] * scale[r], v[2 * j + 1] * scale[r])
                                         : pack_f16x2(v[2 * j] * scale[r], v[2 * j + 1] * scale[r]);
      }
      if (row < p.rows && col < p.cols) store32(dst, o);
      continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (row < p.rows && col + 8 * h < p.cols) {
        float v[8];
        codes4(w[r][2 * h], v);
        codes4(w[r][2 * h + 1], v + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= scale[r];
        store8<OUT>(dst + 8 * h, v);
      }
    }
  }
}

template <int OUT, int V>
__global__ void __launch_bounds__(kThreadsInt8) dequantize_int8_odd_kernel(const Int8Params p) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const long long rb = blockIdx.x / p.segs;
  const int seg = static_cast<int>(blockIdx.x - rb * p.segs);
  const int col = seg * kOddCols + lane * V, block = seg * (kOddCols / kInt8Block);
  const long long row0 = (rb * (kThreadsInt8 / 32) + (threadIdx.x >> 5)) * kOddRows;
  Few<int8_t, V> c[kOddRows][8 / V];
  float scale[kOddRows][4];
#pragma unroll
  for (int r = 0; r < kOddRows; ++r) {
    const int8_t* src = p.codes + (row0 + r) * p.cols + col;
    const float* sc = p.scales + (row0 + r) * p.blocks + block;
#pragma unroll
    for (int i = 0; i < 8 / V; ++i)
      if (row0 + r < p.rows && col + 32 * V * i < p.cols)
        c[r][i] = *reinterpret_cast<const Few<int8_t, V>*>(src + 32 * V * i);
#pragma unroll
    for (int b = 0; b < 4; ++b) scale[r][b] = row0 + r < p.rows && block + b < p.blocks ? sc[b] : 0.f;
  }
#pragma unroll
  for (int r = 0; r < kOddRows; ++r) {
    Elem<OUT>* dst = static_cast<Elem<OUT>*>(p.y) + part_row(p, row0 + r, p.ldy) + col;
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) {
      Few<Elem<OUT>, V> t;
#pragma unroll
      for (int j = 0; j < V; ++j)
        t.v[j] = from_float<OUT>(static_cast<float>(c[r][i].v[j]) * scale[r][V * i >> 1]);
      if (row0 + r < p.rows && col + 32 * V * i < p.cols)
        *reinterpret_cast<Few<Elem<OUT>, V>*>(dst + 32 * V * i) = t;
    }
  }
}

// dgate and dup (and H) from H's gradient and gate and up kept in 8 bits: a lane
// takes 8 columns of a row, a warp 256.
template <int IO, bool WITH_H>
__global__ void __launch_bounds__(kThreadsInt8) swiglu_grad_int8_kernel(const Int8Params p) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const long long rb = blockIdx.x / p.segs;
  const int seg = static_cast<int>(blockIdx.x - rb * p.segs);
  const int col = (seg * 32 + lane) * 8;
  if (col >= p.cols) return;
  const long long row0 = (rb * (kThreadsInt8 / 32) + (threadIdx.x >> 5)) * kGradRows;
  uint2 cg[kGradRows], cu[kGradRows];
  uint4 dh[kGradRows];
  float sg[kGradRows], su[kGradRows];
#pragma unroll
  for (int r = 0; r < kGradRows; ++r) {
    const long long row = row0 + r;
    if (row < p.rows) {
      dh[r] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + row * p.ldx + col);
      cg[r] = *reinterpret_cast<const uint2*>(p.codes + row * 2 * p.cols + col);
      cu[r] = *reinterpret_cast<const uint2*>(p.codes + row * 2 * p.cols + p.cols + col);
      const float* sc = p.scales + row * 2 * p.blocks + (col >> 6);
      sg[r] = sc[0];
      su[r] = sc[p.blocks];
    }
  }
#pragma unroll
  for (int r = 0; r < kGradRows; ++r) {
    const long long row = row0 + r;
    if (row < p.rows) {
      float g[8], u[8], d[8], dg[8], du[8], h[8];
      codes4(cg[r].x, g);
      codes4(cg[r].y, g + 4);
      codes4(cu[r].x, u);
      codes4(cu[r].y, u + 4);
      unpack_pair(dh[r].x, IO == kOutBF16, &d[0], &d[1]);
      unpack_pair(dh[r].y, IO == kOutBF16, &d[2], &d[3]);
      unpack_pair(dh[r].z, IO == kOutBF16, &d[4], &d[5]);
      unpack_pair(dh[r].w, IO == kOutBF16, &d[6], &d[7]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] *= sg[r];
        u[i] *= su[r];
        const float s = rcp_approx(1.0f + __expf(-g[i])), t = d[i] * s;
        du[i] = t * g[i];
        dg[i] = t * u[i] * fmaf(g[i], 1.0f - s, 1.0f);
        if constexpr (WITH_H) h[i] = g[i] * s * u[i];
      }
      uint16_t* dst = static_cast<uint16_t*>(p.y) + row * p.ldy + col;
      store8<IO>(dst, dg);
      store8<IO>(dst + p.cols, du);
      if constexpr (WITH_H) store8<IO>(static_cast<uint16_t*>(p.h) + row * p.ldh + col, h);
    }
  }
}

int elt_bytes(int dtype) { return dtype == kOutF32 ? 4 : 2; }

bool known(int dtype) { return dtype == kOutBF16 || dtype == kOutF16 || dtype == kOutF32; }

// Lanes a row of `cols` columns takes, a power of two of 4 .. 32.
int row_lanes(int cols) {
  int l = 4;
  while (l < 32 && l * 16 < cols) l *= 2;
  return l;
}

// Grid of a row kernel whose warps take `rows` rows of `cols` columns at a time; 0: too large.
unsigned row_grid(Int8Params* p, int cols, int rows) {
  p->segs = (p->cols + cols - 1) / cols;
  const long long per = static_cast<long long>(kThreadsInt8 / 32) * rows;
  const long long blocks = (p->rows + per - 1) / per * p->segs;
  return blocks > 0x7fffffffLL ? 0u : static_cast<unsigned>(blocks);
}

template <int T, int L>
bool launch_rows(Int8Params p, bool back, cudaStream_t s) {
  const unsigned grid = row_grid(&p, 16 * L, 32 / L * kRowsPerWarp);
  if (grid == 0) return false;
  if (back)
    dequantize_int8_kernel<T, L><<<grid, kThreadsInt8, 0, s>>>(p);
  else
    quantize_int8_kernel<T, L><<<grid, kThreadsInt8, 0, s>>>(p);
  return true;
}

template <int T>
bool launch_type(const Int8Params& p, bool back, bool vec, cudaStream_t s) {
  if (!vec) {
    Int8Params q = p;
    const unsigned grid = row_grid(&q, kOddCols, kOddRows);
    if (grid == 0) return false;
    // two at a time: every row, part and code starts on an even element
    const bool two = p.cols % 2 == 0 && p.ldx % 2 == 0 && is_aligned(p.x, 2 * elt_bytes(T)) && is_aligned(p.codes, 2);
    if (back)
      two ? dequantize_int8_odd_kernel<T, 2><<<grid, kThreadsInt8, 0, s>>>(q)
          : dequantize_int8_odd_kernel<T, 1><<<grid, kThreadsInt8, 0, s>>>(q);
    else
      two ? quantize_int8_odd_kernel<T, 2><<<grid, kThreadsInt8, 0, s>>>(q)
          : quantize_int8_odd_kernel<T, 1><<<grid, kThreadsInt8, 0, s>>>(q);
    return true;
  }
  switch (row_lanes(p.cols)) {
    case 4: return launch_rows<T, 4>(p, back, s);
    case 8: return launch_rows<T, 8>(p, back, s);
    case 16: return launch_rows<T, 16>(p, back, s);
    default: return launch_rows<T, 32>(p, back, s);
  }
}

// Shared by both directions: m [M, N] with row stride ld in `dtype`.
bwg_status run_int8(bool back, const void* m, int dtype, int M, int N, int ld, int parts, void* codes, float* scales,
                    cudaStream_t stream) {
  if (!known(dtype) || M < 0 || N < 0 || (parts != 1 && parts != 2) || N % parts != 0) return BWG_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return BWG_OK;
  if (N > kMaxSize) return BWG_ERR_UNSUPPORTED;
  if (m == nullptr || codes == nullptr || scales == nullptr || ld < N) return BWG_ERR_INVALID_ARG;
  if (!is_aligned(m, elt_bytes(dtype)) || !is_aligned(scales, 4)) return BWG_ERR_ALIGNMENT;
  Runtime rt;
  const bwg_status s = runtime_device(&rt);
  if (s != BWG_OK) return s;
  Int8Params p = {};
  p.x = m;
  p.y = const_cast<void*>(m);
  p.codes = static_cast<int8_t*>(codes);
  p.scales = scales;
  p.ldx = p.ldy = ld;
  p.rows = static_cast<long long>(M) * parts;
  p.cols = N / parts;
  p.blocks = (p.cols + kInt8Block - 1) / kInt8Block;
  p.part_bits = parts - 1;
  const bool vec = p.cols % 8 == 0 && is_aligned(m, 16) && is_aligned(codes, 16) &&
                   static_cast<long long>(ld) * elt_bytes(dtype) % 16 == 0;
  p.wide = p.cols % 16 == 0 && is_aligned(m, 32) && ld % 16 == 0 ? 1 : 0;
  const bool ok = dtype == kOutBF16  ? launch_type<kOutBF16>(p, back, vec, stream)
                  : dtype == kOutF16 ? launch_type<kOutF16>(p, back, vec, stream)
                                     : launch_type<kOutF32>(p, back, vec, stream);
  return ok ? runtime_status(cudaGetLastError()) : BWG_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace bwg

using namespace bwg;

extern "C" {

bwg_status quantize_int8(const void* x, int dtype, int M, int N, int ldx, int parts, void* codes, float* scales,
                         void* stream) {
  return run_int8(false, x, dtype, M, N, ldx, parts, codes, scales, static_cast<cudaStream_t>(stream));
}

bwg_status dequantize_int8(const void* codes, const float* scales, int parts, void* y, int dtype, int M, int N,
                           int ldy, void* stream) {
  return run_int8(true, y, dtype, M, N, ldy, parts, const_cast<void*>(codes), const_cast<float*>(scales),
                  static_cast<cudaStream_t>(stream));
}

bwg_status swiglu_grad_int8(const void* dH, const void* codes, const float* scales, void* dGU, void* H, int dtype,
                            int M, int I, int lddh, int ldd, int ldh, void* stream) {
  if ((dtype != BWG_OUT_BF16 && dtype != BWG_OUT_FP16) || M < 0 || I < 0) return BWG_ERR_INVALID_ARG;
  if (M == 0 || I == 0) return BWG_OK;
  if (I > kMaxSize / 2) return BWG_ERR_UNSUPPORTED;
  if (dH == nullptr || codes == nullptr || scales == nullptr || dGU == nullptr || lddh < I || ldd < 2 * I ||
      (H != nullptr && ldh < I))
    return BWG_ERR_INVALID_ARG;
  if (I % 8 != 0 || !is_aligned(dH, 16) || !is_aligned(codes, 16) || !is_aligned(scales, 4) || !is_aligned(dGU, 16) ||
      lddh % 8 != 0 || ldd % 8 != 0 || (H != nullptr && (!is_aligned(H, 16) || ldh % 8 != 0)))
    return BWG_ERR_ALIGNMENT;
  Runtime rt;
  const bwg_status s = runtime_device(&rt);
  if (s != BWG_OK) return s;
  Int8Params p = {};
  p.x = dH;
  p.y = dGU;
  p.h = H;
  p.codes = static_cast<int8_t*>(const_cast<void*>(codes));
  p.scales = const_cast<float*>(scales);
  p.ldx = lddh;
  p.ldy = ldd;
  p.ldh = ldh;
  p.rows = M;
  p.cols = I;
  p.blocks = (I + kInt8Block - 1) / kInt8Block;
  const unsigned grid = row_grid(&p, 256, kGradRows);
  if (grid == 0) return BWG_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == BWG_OUT_BF16) {
    if (H != nullptr)
      swiglu_grad_int8_kernel<kOutBF16, true><<<grid, kThreadsInt8, 0, st>>>(p);
    else
      swiglu_grad_int8_kernel<kOutBF16, false><<<grid, kThreadsInt8, 0, st>>>(p);
  } else {
    if (H != nullptr)
      swiglu_grad_int8_kernel<kOutF16, true><<<grid, kThreadsInt8, 0, st>>>(p);
    else
      swiglu_grad_int8_kernel<kOutF16, false><<<grid, kThreadsInt8, 0, st>>>(p);
  }
  return runtime_status(cudaGetLastError());
}

}  // extern "C"
