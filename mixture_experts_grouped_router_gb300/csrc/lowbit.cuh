// Device helpers of the low-bit formats: E2M1 codes with block scales (MXFP4,
// NVFP4) and 8-bit integer codes with one bf16 scale per 32 elements.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

// Pairs of fp32 values in one 64-bit register: one instruction for two of them.
MOE_DEVINL uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

MOE_DEVINL void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

MOE_DEVINL uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

MOE_DEVINL uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

MOE_DEVINL uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 1 / t to within a bit, 2^-23 of it (t a normal float).
MOE_DEVINL float rcp_approx(float t) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

// x / t by a reciprocal and one residual step: where x / t is representable
// (a tie of the code grid, for bf16 x and scales of few bits) the result is
// exact, so that ties round as the quotient's definition says.
MOE_DEVINL float div_exact(float x, float t, float inv) {
  const float q = x * inv;
  return fmaf(fmaf(-q, t, x), inv, q);
}

// Quotients on the way to codes: x * inv (inv within 2^-23 of 1 / t) rounded to a
// multiple of the spacing of floats near `grid`, which is added for that; the
// result is that much too large.  A tie of the code grid lies on a multiple and the
// product within half a spacing of it, so that ties are met exactly.  Only where x and
// t have so few bits that no other quotient comes as near a tie.
MOE_DEVINL uint64_t snap2(uint64_t x, uint64_t inv, uint64_t grid) { return fma2(x, inv, grid); }

// Elements per scale of a 4-bit format, and columns per 512-byte scale atom
// (128 rows x 4 blocks).
__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == MOE_FP4_NV ? 16 : 32; }
__host__ __device__ constexpr int fp4_atom_cols(int fmt) { return 4 * fp4_block(fmt); }

// Byte of (padded row pr, block b) in scale atoms of `ac` atom columns.
MOE_DEVINL int64_t fp4_scale_byte(int64_t pr, int b, int ac) {
  const int rw = (int)(pr & 127);
  return ((pr >> 7) * ac + (b >> 2)) * 512 + (rw & 31) * 16 + (rw >> 5) * 4 + (b & 3);
}

// 8 values -> 8 E2M1 codes (round to nearest even, saturated at 6), value 2i in
// the low nibble of byte i.
MOE_DEVINL uint32_t cvt_e2m1x8(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// 8 E2M1 codes -> 8 values (exact).
MOE_DEVINL void e2m1x8_to_f32(uint32_t c, float *v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
    v[2 * i] = t.x;
    v[2 * i + 1] = t.y;
  }
}

// E4M3 code of v >= 0 (round to nearest even, saturated at 448) and its value.
MOE_DEVINL uint32_t e4m3_code(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}

MOE_DEVINL float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  return __half2float(__ushort_as_half((uint16_t)(h & 0xFFFFu)));
}

// 2^(code - 127), code 255: NaN.
MOE_DEVINL float e8m0_value(uint32_t code) {
  if (code == 255u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(code > 0 ? code << 23 : 1u << 22);
}

MOE_DEVINL float fp4_scale_value(uint32_t code, int fmt) {
  return fmt == MOE_FP4_NV ? e4m3_value(code) : e8m0_value(code);
}

// Scale code of a block with largest magnitude a, and the reciprocal inv of its
// scale (times g for NVFP4), or 0 where every code of the block is 0 (no magnitude,
// or a NaN / infinity, which takes the NaN scale).
//   MXFP4: t = 2^s, s = floor(log2 a) - 2 clamped to [-127, 127] (OCP MX v1.0)
//   NVFP4: E4M3(a / (6 g)) saturated at 448, g the tensor's fp32 scale; g6 = 6 g, inv6 =
//       1 / g6; a is cut to 448 g6 first, as a quotient past fp32's range has no residual
template <int FMT>
MOE_DEVINL uint32_t fp4_block_scale(float a, float g, float g6, float inv6, float &inv) {
  inv = 0.0f;
  const bool finite = a <= 3.402823466e38f;
  if (FMT == MOE_FP4_NV) {
    if (!finite) return 0x7Fu;
    const uint32_t code = e4m3_code(div_exact(fminf(a, 448.0f * g6), g6, inv6));
    const float s = e4m3_value(code) * g;
    if (s >= 1.17549435e-38f) inv = rcp_approx(s);
    return code;
  }
  if (!finite) return 0xFFu;
  if (!(a > 0.0f)) return 0u;
  const uint32_t b = __float_as_uint(a);
  const int e = (b >> 23) != 0 ? (int)(b >> 23) - 127 : (31 - __clz(b)) - 149;
  const int s = max(-127, e - 2);
  inv = __uint_as_float((uint32_t)(127 - s) << 23);
  return (uint32_t)(s + 127);
}

// Whether the tensor's scale has 8 significant bits at most, which decides how quotients
// are taken below: 32768 rows of 4096 gathered from 16384 tokens (NVFP4) 43 us linked and
// 69 direct if so, 47 and 77 if not.
MOE_DEVINL bool fp4_few_bits(float g) { return (__float_as_uint(g) & 0xFFFFu) == 0; }

// 8 values -> 8 codes, by the block's scale code and inv.  MXFP4: products with a power
// of two are exact.  NVFP4 with few bits of g: the ties are .25 to 5, met within 5 2^-23;
// near 24 floats are 2^-19 apart; a bf16 x over a scale of 12 bits (an E4M3 times g) is a
// tie or 2^-15 of itself from one.  With more bits a quotient may be nearer (of all scales
// of 24 bits 1 in 700 has a bf16 multiple that the sum would move across a tie): a residual
// step then decides as the fp32 quotient does, past which the scale's own rounding hides
// the rest (values of a saturated block are cut to 8 times the scale first: past fp32's
// range there is no residual).
template <int FMT, bool FEW>
MOE_DEVINL uint32_t fp4_codes8(const float *v, float inv, uint32_t code, float g) {
  const uint64_t inv2 = pack2(inv, inv);
  float r[8];
  if (FMT == MOE_FP4_NV && !FEW) {
    const float t = e4m3_value(code) * g;
    const uint64_t minus_t = pack2(-t, -t);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = v[j];
    if (code == 0x7Eu) {
      const float most = 8.0f * t;
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = fminf(fmaxf(r[j], -most), most);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t x = pack2(r[2 * j], r[2 * j + 1]), q = mul2(x, inv2);
      unpack2(fma2(fma2(q, minus_t, x), inv2, q), r[2 * j], r[2 * j + 1]);
    }
  } else {
    const uint64_t grid = pack2(24.0f, 24.0f), back = pack2(-24.0f, -24.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t x = pack2(v[2 * j], v[2 * j + 1]);
      unpack2(FMT == MOE_FP4_NV ? add2(snap2(x, inv2, grid), back) : mul2(x, inv2), r[2 * j],
              r[2 * j + 1]);
    }
  }
  // (a NaN or an infinity times 0 is no zero code)
  return inv == 0.0f ? 0u : cvt_e2m1x8(r);
}

// Largest magnitude of 8 bf16 values, as bf16 bits; a NaN wins over everything
// and an infinity over every number.
MOE_DEVINL uint32_t amax_bits8(const uint4 &w) {
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w);
  const __nv_bfloat162 a = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])),
                                       __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
  const uint32_t b = *reinterpret_cast<const uint32_t *>(&a);
  return max(b & 0xFFFFu, b >> 16);
}

}  // namespace moe
