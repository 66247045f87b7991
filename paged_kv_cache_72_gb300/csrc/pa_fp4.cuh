// The 4-bit KV pool: layout and conversions shared by its kernels.
//
// A pool is uint8 [num_blocks][num_kv_heads][P], P = B * 9 D / 16: the plane of
// one head of one block holds the E2M1 codes [B][D / 2] (head_dim 2 i in the
// low nibble of byte i), then one E4M3 scale for every 16 consecutive head_dim
// values of a token, [B / 4][D / 16][4], the last index being the token's
// position modulo 4.  value = e2m1(code) * e4m3(scale) * tensor scale.
//
// Why planes per head: a decode that splits a context over heads reads whole
// planes, B * 9 D / 16 contiguous bytes (1,152 for 16-token blocks of head_dim
// 128).  Why scales in quads of tokens: a lane of the decode takes one group of
// four consecutive tokens, whose four scales of a head_dim group are one word.
#pragma once

#include "pa_device.cuh"

namespace pa {

__host__ __device__ constexpr int fp4_row_bytes(int D) { return D / 2 + D / 16; }

__device__ __forceinline__ size_t fp4_plane(long long block, int H, int h, int plane_bytes) {
  return ((size_t)block * H + h) * (size_t)plane_bytes;
}

// Byte offset of the scale of token row r, head_dim group g, inside a plane.
template <int D>
__device__ __forceinline__ int fp4_scale_off(int B, int r, int g) {
  return B * (D / 2) + ((r >> 2) * (D / 16) + g) * 4 + (r & 3);
}

// Eight E2M1 codes in one word -> four f16x2 (byte i -> r[i], its low nibble
// in the low half).  Exact.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t x, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(x));
}

// Eight fp32 values -> eight E2M1 codes (the first in the lowest nibble), round
// to nearest even, magnitudes beyond 6 saturate.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(float x0, float x1, float x2, float x3,
                                                    float x4, float x5, float x6, float x7) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3), "f"(x4), "f"(x5), "f"(x6), "f"(x7));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// a times the low / the high half of s in both halves (the multiply selects it)
__device__ __forceinline__ uint32_t hmul2_lo(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a),
                            __low2half2(*reinterpret_cast<__half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul2_hi(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a),
                            __high2half2(*reinterpret_cast<__half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace pa
