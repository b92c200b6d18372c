// What the two attention kernels over the paged NVFP4 cache share: the
// dequantization to FP16, the masks' limits and the workspace.
//
// Number format. A cached value is g * s * c with s an E4M3 scale and c an E2M1
// code; s*c has at most 6 significant bits. Both factors are placed into FP16
// by moving bits alone: the code's two exponent bits and one mantissa bit at
// the FP16 positions read as c * 2^-14 (subnormals included), the scale's seven
// bits as s * 2^-8. The kernels multiply by s * 2^7, so that the product is
// c*s * 2^-7 exactly: a multiple of 2^-17 of at most 6 * 480 * 2^-7 = 22.5. The
// factor 2^7 * g joins the softmax scale (K) and the final division (V).
// The bits read the E4M3 NaN code 0x7F as 480 and drop the sign, so no cache
// content is infinite or NaN: what a mask hides cannot reach a row's result
// through 0 * NaN.
#pragma once

#include "kernels.h"
#include "kv_common.cuh"

namespace nvfp4 {

NVFP4_DEVINL uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight codes of a word -> four FP16 pairs c * 2^-14, in the order (0,4),
// (2,6), (1,5), (3,7): the nibbles of one parity become the four high bytes of
// FP16 numbers, which two byte permutes spread over two registers.
NVFP4_DEVINL void codes_to_half(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t even = ((w << 1) & 0x0E0E0E0Eu) | ((w << 4) & 0x80808080u);
  const uint32_t odd = ((w >> 3) & 0x0E0E0E0Eu) | (w & 0x80808080u);
  p[0] = __byte_perm(even, 0, 0x2404);
  p[1] = even & 0xFF00FF00u;
  p[2] = __byte_perm(odd, 0, 0x2404);
  p[3] = odd & 0xFF00FF00u;
}

constexpr uint32_t kHalf2Exp15 = 0x78007800u;  // 2^15 in both halves

// Two E4M3 scales (low bytes of each half) -> FP16 pair s * 2^7.
NVFP4_DEVINL uint32_t scales_to_half(uint32_t two) { return hmul2((two & 0x007F007Fu) << 7, kHalf2Exp15); }

NVFP4_DEVINL float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Power of two that brings a row of BF16 queries whose largest magnitude is
// amax to [2^14, 2^15), as the exponent to add (0 for a zero or non-finite
// row). FP16 then holds every query exactly down to 2^-29 of the row's largest,
// and to 2^-40 of it below.
NVFP4_DEVINL int query_exponent(float amax) {
  const int e = (int)((__float_as_uint(amax) >> 23) & 0xFFu);
  return e == 0 || e == 255 ? 0 : 14 + 127 - e;
}
// x * 2^e for |e| up to 140 (two exact factors; a subnormal x stays one).
NVFP4_DEVINL float scale_exp2(float x, int e) {
  const int h = e / 2;
  return x * __uint_as_float((uint32_t)(127 + h) << 23) * __uint_as_float((uint32_t)(127 + e - h) << 23);
}

// Cached tokens that the new token at position `pos` sees: [lo, hi).
struct Visible {
  int32_t lo, hi;
};
NVFP4_DEVINL Visible visible(int64_t pos, int32_t len, int causal, int64_t window) {
  int64_t hi = causal ? (pos + 1 < len ? pos + 1 : len) : len;
  int64_t lo = window > 0 ? pos - window + 1 : 0;
  if (lo < 0) lo = 0;
  if (hi < lo) hi = lo;
  return Visible{(int32_t)lo, (int32_t)hi};
}

struct AttnArgs {
  const uint16_t* q;   // BF16 [total][hq][D], rows q_stride apart
  int64_t q_stride;
  KvIndex ix;
  const uint8_t* pages;
  const float *k_g, *v_g;
  float scale;         // softmax scale
  int group;           // query heads per KV head
  int causal;
  int64_t window;      // 0: no window
  uint16_t* out;       // BF16 [total][hq][D]
  float* lse;          // FP32 [total][hq] or null
  float* partial;      // workspace
  int32_t* counters;   // workspace, zero between calls
  int* status;
};

}  // namespace nvfp4
