// Layout and device helpers of the paged 4-bit latent cache (the format is
// stated in include/mlaqp_kv4.h).
#pragma once

#include <cuda_runtime.h>

#include "mlaqp_kernel.cuh"

namespace mlaqp {

constexpr int kKv4CodeBytes = kLatent / 2;   // 256 per token
constexpr int kKv4RopeBytes = kRope * 2;     // 128
constexpr int kKv4Blocks = kLatent / 32;     // 16 scale bytes
constexpr int kKv4TokenBytes = kKv4CodeBytes + kKv4RopeBytes + kKv4Blocks;
constexpr int kKv4ScaleMin = 87, kKv4ScaleMax = 167, kKv4ScaleNan = 255;

constexpr unsigned kDevStatusBadIndex = 2u;
constexpr unsigned kDevStatusOutOfPages = 4u;

// Byte offsets of a token's three rows within its page of 1 << shift tokens.
__device__ __forceinline__ uint32_t kv4_code_off(uint32_t pos) { return pos * kKv4CodeBytes; }
__device__ __forceinline__ uint32_t kv4_rope_off(uint32_t pos, int shift) {
  return (static_cast<uint32_t>(kKv4CodeBytes) << shift) + pos * kKv4RopeBytes;
}
__device__ __forceinline__ uint32_t kv4_scale_off(uint32_t pos, int shift) {
  return (static_cast<uint32_t>(kKv4CodeBytes + kKv4RopeBytes) << shift) + pos * kKv4Blocks;
}

// Eight floats -> eight E2M1 codes (round to nearest even, saturating), code
// i in nibble i with its sign at bit 3 of the nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// The cache's word of eight elements: magnitudes in element order, signs in
// the order that puts those of elements 0..3 at the top of the four bytes
// and those of 4..7 four bits lower.  The sign order is the nibble order of
// the elements (4,0,5,1,6,2,7,3).
__device__ __forceinline__ uint32_t kv4_word(const float (&f)[8]) {
  const float s[8] = {f[4], f[0], f[5], f[1], f[6], f[2], f[7], f[3]};
  return (e2m1x8(f) & 0x77777777u) | (e2m1x8(s) & 0x88888888u);
}

// Four magnitudes (the low 16 bits of `mags`: nibbles 0..7) and their signs
// (the top bits of the bytes of `signs`) -> two BF16x2 registers of the plain
// code values (0, 0.5 .. 6): byte permutes look the two bytes of each value
// up in its table of eight.
__device__ __forceinline__ void kv4_bf16x4(uint32_t mags, uint32_t signs, uint32_t& lo, uint32_t& hi) {
  const uint32_t h = __byte_perm(0x3F3F3F00u, 0x40404040u, mags) | (signs & 0x80808080u);
  const uint32_t l = __byte_perm(0xC0800000u, 0xC0804000u, mags);
  lo = __byte_perm(l, h, 0x5140);
  hi = __byte_perm(l, h, 0x7362);
}

// One word of eight elements -> four BF16x2 registers in element order.
__device__ __forceinline__ void kv4_word_bf16(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t m = w & 0x77777777u;
  kv4_bf16x4(m, w, o[0], o[1]);
  kv4_bf16x4(m >> 16, w << 4, o[2], o[3]);
}

// 2^(s-127) of a scale byte as BF16 (exact), NaN for 255.
__device__ __forceinline__ uint32_t kv4_scale_clamp(uint32_t s) {
  return s == kKv4ScaleNan ? s : min(max(s, static_cast<uint32_t>(kKv4ScaleMin)), static_cast<uint32_t>(kKv4ScaleMax));
}
__device__ __forceinline__ uint32_t kv4_scale_bf16x2(uint32_t s) {
  const uint32_t b = s == kKv4ScaleNan ? 0x7FC0u : kv4_scale_clamp(s) << 7;
  return b | (b << 16);
}

__device__ __forceinline__ void st_u128(void* p, uint4 v) {
  asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

}  // namespace mlaqp
