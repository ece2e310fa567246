// 4-bit pages (TG_PAGES_E2M1): the places of codes and scales in a tile of 16 tokens x 128 values, and the
// conversions between values and codes.
//
// Why this layout.  K codes lie by token: the four lanes that hold a token's row of a K fragment read it in
// 16-byte pieces, 128 contiguous bytes for eight lanes.  V codes lie by block of 16 values, eight
// tokens together: a lane that holds one block of the V^T fragment reads two tokens at once, again
// 128 contiguous bytes for eight lanes.  The scales lie so that the pair a lane needs is one 16-bit load.
#pragma once

#include "../../include/tg.h"
#include "packed.cuh"
#include "ptx.cuh"

#include <cstdint>

namespace tgk {

constexpr int kTile4 = TG_TILE4_BYTES;
constexpr int kVCodes4 = 1024, kKScales4 = 2048, kVScales4 = 2176;
constexpr float kMinScale4 = 0.001953125f;  // 2^-9, the smallest e4m3 above 0

// byte offsets of token t's codes of values 8 e .. 8 e + 7 (4 bytes), and of its scale of block j
__device__ __forceinline__ int k_codes4(int t, int e) { return 64 * t + 4 * e; }
__device__ __forceinline__ int v_codes4(int t, int e) {
  return kVCodes4 + 512 * (t >> 3) + 64 * (e >> 1) + 8 * (t & 7) + 4 * (e & 1);
}
__device__ __forceinline__ int k_scale4(int t, int j) { return kKScales4 + 8 * t + j; }
__device__ __forceinline__ int v_scale4(int t, int j) { return kVScales4 + 16 * j + t; }

// the e4m3 number nearest to x >= 0 (ties to the even code, at most 448)
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ float f16_to_float(uint32_t h) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"((uint16_t)h));
  return f;
}
__device__ __forceinline__ float e4m3_to_float(uint32_t e) { return f16_to_float(e4m3x2_to_f16x2(e)); }

// the e2m1 codes of eight values, the first in the lowest bits (ties to the even code, at most 6 in magnitude, NaN as 6)
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
__device__ __forceinline__ uint32_t e2m1_of(float x) {
  uint16_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u16.u8 %0, b;\n\t}" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 15u;
}
// eight codes of a word as four f16 pairs, the lower codes first
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// the larger magnitude, NaN if either is one
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
// 1 / x, off by an ulp at most
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A block's scale from its largest magnitude (over the unit): e4m3 of a sixth of it.  Where a sixth of a bf16 number is
// halfway between two e4m3 numbers, the product with 1/6 in float32 is that, exactly (all 16 such mantissas are
// tested); any other is 2^-9 of it or more away, so the product's rounding decides nothing.
__device__ __forceinline__ uint32_t scale_of(float top) { return max(e4m3_of(top * (1.f / 6.f)), 1u); }

// A bf16 value over a scale s, by the reciprocal of s (inv): where x / s is the border of two codes the product may be
// some ulps off it, and a value that is not on the border is 2^-9 of it or more away (x has 8 significant bits,
// border times s at most 7): a multiple of 2^-14 tells them apart.
__device__ __forceinline__ float2 over_scale_exact(float2 x, float inv) {
  const float2 r = add2(mul2(x, make_float2(inv, inv)), make_float2(512.f, 512.f));
  return add2(r, make_float2(-512.f, -512.f));
}

struct Code8 {     // eight consecutive values in 4 bits
  uint32_t codes;  // a nibble each
  uint32_t scale;  // of their block of 16, e4m3
};
// eight consecutive bf16 values, their block's other eight in the neighbouring lane (lane ^ 1); to_unit: 1 / unit; odd is
// set where one of these eight is not finite
__device__ __forceinline__ Code8 encode_exact(const float2 (&x)[4], float to_unit, bool &odd) {
  float top = max_abs_nan(max_abs_nan(max_abs_nan(x[0].x, x[0].y), max_abs_nan(x[1].x, x[1].y)),
                          max_abs_nan(max_abs_nan(x[2].x, x[2].y), max_abs_nan(x[3].x, x[3].y)));
  if (!(top < __uint_as_float(0x7f800000u))) {  // infinite, or a NaN, which counts for nothing in the scale
    odd = true;
    top = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  Code8 o;
  o.scale = scale_of(top * to_unit);
  const float inv = rcp(e4m3_to_float(o.scale)) * to_unit;
  float r[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = over_scale_exact(x[e], inv);
    r[2 * e] = f.x, r[2 * e + 1] = f.y;
  }
  o.codes = e2m1x8_of(r);
  return o;
}
// what they stand for, as bf16 (exact: at most 6 significant bits)
__device__ __forceinline__ uint4 held8(Code8 c, float unit) {
  uint32_t h[4];
  e2m1x8_to_f16x2(c.codes, h);
  const float s = e4m3_to_float(c.scale) * unit;
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(f16_to_float(h[i]) * s, f16_to_float(h[i] >> 16) * s);
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// whether a unit is a power of two in [2^-60, 2^60]
inline bool unit_ok(float u) {
  if (!(u >= 0x1p-60f && u <= 0x1p60f)) return false;
  uint32_t b;
  __builtin_memcpy(&b, &u, 4);
  return (b & 0x007fffffu) == 0;
}

}  // namespace tgk
