// A paged cache of 4-bit elements: page geometry and conversions.
//
// An element is an e2m1 code (sign; 0, 0.5, 1, 1.5, 2, 3, 4, 6) times the scale
// of its 16 neighbours along the head.  A scale is never negative, so its byte
// spends no bit on a sign: five exponent bits and three of mantissa, bits 14..7
// of the same number in fp16, and the cache needs no scale per tensor beside
// it.  A product has at most 2 + 4 significant bits: exact in fp16 and in bf16.
//
// A page is one block of one KV head, contiguous: block_size rows of
// head_dim / 2 bytes of codes (byte i: element 2i in the low half, 2i + 1 in
// the high), then block_size rows of head_dim / 16 scales.  Both parts are a
// multiple of 16 bytes for every block size and head_dim, so pages are copied as
// they are (prefill: a bulk copy of each part; decode: vectors of 16 bytes).  A
// cache is [num_blocks][kv_heads][page].
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kKv4Group = 16;             // elements of a scale
constexpr float kKv4Top = 6.f;            // largest level
constexpr uint32_t kKv4MaxScale = 0xE2;   // 10240: 6 * 10240 is the largest element, 61440
constexpr uint32_t kKv4NanScale = 0xFF;   // a group with an element that is not finite: a NaN in fp16
constexpr uint32_t kKv4FirstInf = 0xF8;   // scale bytes from here on are infinite or NaN

template <int D>
struct Kv4Row {
  static constexpr int CODES = D / 2;
  static constexpr int SCALES = D / kKv4Group;
  static constexpr int BYTES = CODES + SCALES;
};

// The four element pairs of a word of eight codes, in fp16 (exact).
__device__ __forceinline__ void kv4_unpack(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Two elements as a byte of codes, nearest level, ties to the even code.
__device__ __forceinline__ uint32_t kv4_pack2(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 t, z;\n .reg .b32 zero;\n mov.b32 zero, 0;\n mov.b32 {z, _, _, _}, zero;\n"
      " cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n mov.b32 %0, {t, z, z, z};\n}\n"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// Scales as fp16: one in both halves, or two.
__device__ __forceinline__ uint32_t kv4_scale2(uint32_t byte) { return byte * 0x00800080u; }
__device__ __forceinline__ uint32_t kv4_scale_pair(uint32_t lo, uint32_t hi) { return (lo << 7) | (hi << 23); }
__device__ __forceinline__ float kv4_scale(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// Byte of the scale top / 6, rounded to nearest (even) at three mantissa bits;
// fp32's quotient decides every tie as the exact one does: top has at most 11
// significant bits, so a quotient that is no tie is at least 2^-14 away from one.
__device__ __forceinline__ uint32_t kv4_scale_byte(float top) {
  const float f = __fdiv_rn(top, kKv4Top);
  if (!(f < INFINITY)) return kKv4NanScale;  // infinite or NaN
  uint32_t b;
  if (f < 6.103515625e-05f) {  // below 2^-14 scales are 2^-17 apart
    b = (uint32_t)__float2int_rn(f * 131072.f);
  } else {
    const uint32_t u = __float_as_uint(f);
    b = ((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (112u << 3);
  }
  return b < kKv4MaxScale ? b : kKv4MaxScale;
}

__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// fp16 pair to a pair of T (exact for the cache's elements).
template <typename T>
__device__ __forceinline__ uint32_t from_half2(uint32_t h);
template <>
__device__ __forceinline__ uint32_t from_half2<__half>(uint32_t h) {
  return h;
}
template <>
__device__ __forceinline__ uint32_t from_half2<__nv_bfloat16>(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return Elem<__nv_bfloat16>::pack(f.x, f.y);
}

}  // namespace pa
