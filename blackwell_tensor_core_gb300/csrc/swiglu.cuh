// SwiGLU and its gradient on FP32 values, and blocks of 64 values put into 8
// bits: the arithmetic that the gated kernels' epilogues and the passes over
// matrices kept in 8 bits share.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace bwg {

constexpr int kInt8Block = 64;  // columns that share a scale

// SwiGLU of one gate/up accumulator pair: silu(g) * u with
// silu(g) = g * sigmoid(g) = g / (1 + e^-g), using the hardware's
// approximate exponential and reciprocal (a few ulp of FP32, far below the
// final rounding to 16 bits).  For very negative g, e^-g overflows to +inf,
// the reciprocal is 0 and the result a signed zero, the function's limit.
BWG_DEV float swiglu_f32(float g, float u) { return g * rcp_approx(1.0f + __expf(-g)) * u; }

// Its gradient: with s = sigmoid(g), d(silu)/dg = s (1 + g (1 - s)).  1 - s
// loses its bits only where s is next to 1 and the product next to nothing
// beside the 1 that it is added to.
BWG_DEV void swiglu_grad_f32(float g, float u, float dh, float* dg, float* du) {
  const float s = rcp_approx(1.0f + __expf(-g));
  const float t = dh * s;
  *du = t * g;
  *dg = t * u * fmaf(g, 1.0f - s, 1.0f);
}

// Two 16-bit values of a word, BF16 or FP16.
BWG_DEV void unpack_pair(uint32_t w, bool bf16, float* lo, float* hi) {
  if (bf16) {
    *lo = __uint_as_float(w << 16);
    *hi = __uint_as_float(w & 0xFFFF0000u);
  } else {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    *lo = v.x;
    *hi = v.y;
  }
}

// max(|a|, |b|), NaN if either is one.
BWG_DEV float max_abs_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Scale and reciprocal of a block whose largest magnitude is `amax`: a / 127 and
// 127 / a, each rounded once.  Up to a = 127 * 2^-128, where 127 / a passes FP32's
// range, the block is zero; with an infinity or a NaN in it it reads back as NaN.
BWG_DEV void int8_scale(float amax, float* scale, float* inv) {
  *inv = 127.0f / amax;
  *scale = amax / 127.0f;
  if (!(*inv < __int_as_float(0x7F800000))) {  // infinite, or NaN
    *scale = amax != amax ? amax : 0.0f;
    *inv = 0.0f;
  } else if (*inv == 0.0f) {  // an infinity in the block
    *scale = __int_as_float(0x7FC00000);
  }
}

// rint(v * inv) as the low byte of a word, with one rounding: the sum with
// 1.5 * 2^23 has no bits below one, and its low byte is the code in two's
// complement (|v * inv| <= 127).
BWG_DEV uint32_t int8_code(float v, float inv) { return __float_as_uint(fmaf(v, inv, 12582912.0f)); }

BWG_DEV uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// One block of n (1 .. 64) values in registers: its codes, zero past n, and its
// scale.
BWG_DEV float keep_block(uint32_t (&v)[64], int n, uint32_t (&codes)[16]) {
  if (n < 64) {
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if (i >= n) v[i] = 0u;
  }
  // four chains: one of 64 dependent steps is slower
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 64; ++i) a[i & 3] = max_abs_nan(a[i & 3], __uint_as_float(v[i]));
  float scale, inv;
  int8_scale(max_abs_nan(max_abs_nan(a[0], a[1]), max_abs_nan(a[2], a[3])), &scale, &inv);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    codes[i] = pack_bytes(int8_code(__uint_as_float(v[4 * i]), inv), int8_code(__uint_as_float(v[4 * i + 1]), inv),
                          int8_code(__uint_as_float(v[4 * i + 2]), inv), int8_code(__uint_as_float(v[4 * i + 3]), inv));
  return scale;
}

}  // namespace bwg
