// Page format of the 8-bit cache (device side) and the arithmetic of its codes.
//
// One block per (page of 16 tokens, KV head): 16*d key codes, 16*d value codes,
// then four fp32 words (key scale, value scale, 0, 0): 32*d + 16 bytes, so that
// one bulk copy brings codes and scales.  A value is code * scale.
//
// The element order is the attention kernel's: a lane (4*gid + tig) of a warp
// reads its tensor-core operands by 16-byte shared-memory loads without bank
// conflicts, and a 16-byte chunk is also what a placing thread produces.
//   key (t, c): a chunk holds 16 consecutive channels of one token; chunk
//     ((c/64)*2 + t%2)*32 + 4*(t/2) + (c/16)%4, byte c%16 in it.
//   value (t, c): a chunk holds 4 channels x 4 tokens; chunk
//     (c/32)*32 + 4*((c/4)%8) + t/4, byte 4*(c%4) + t%4 in it.
// The bf16 tail block of a sequence (its last L % 16 tokens) has the same
// element order at two bytes an element: 16*d keys, then 16*d values.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace oscar {

template <int D>
struct Kv8Fmt {
  static constexpr int kCodes = 16 * D;            // bytes of one code area
  static constexpr int kScales = 32 * D;           // byte offset of the scales
  static constexpr int kBlock = 32 * D + 16;
  static constexpr int kTailHalf = 16 * D;         // elements of one tail area
  static constexpr int kTailBytes = 64 * D;
};

// chunk of the key area that holds channels 16*cc .. 16*cc + 15 of token t
__device__ __forceinline__ int kv8_key_chunk(int t, int cc) {
  return ((cc >> 2) * 2 + (t & 1)) * 32 + 4 * (t >> 1) + (cc & 3);
}
// chunk of the value area that holds channels 4*cg .. 4*cg + 3 of tokens 4*tg .. 4*tg + 3
__device__ __forceinline__ int kv8_value_chunk(int tg, int cg) {
  return (cg >> 3) * 32 + 4 * (cg & 7) + tg;
}

// The largest code of a format; a block's scale is fl32(max|x| / top).
template <bool kE4m3>
__device__ __forceinline__ float kv8_top() { return kE4m3 ? 448.f : 127.f; }

// Blocks whose largest value is below 2^-100 are stored as zeros: top / max stays
// finite for every other block.
constexpr float kKv8Least = 7.888609052210118e-31f;   // 2^-100

// Four codes of x * inv, packed in order.  The product is rounded to fp32 and
// then to the code, as the format defines it (no fused multiply-add): int8 by
// adding 1.5 * 2^23 + 128, whose low byte is rint(y) + 128 (the constant is even,
// so ties go to the even code), e4m3 by the saturating conversion.  Finite x give
// |y| <= top (1 + 2^-23), which both round to top.
template <bool kE4m3>
__device__ __forceinline__ uint32_t kv8_codes4(float x0, float x1, float x2, float x3, float inv) {
  const float y0 = __fmul_rn(x0, inv), y1 = __fmul_rn(x1, inv);
  const float y2 = __fmul_rn(x2, inv), y3 = __fmul_rn(x3, inv);
  if constexpr (kE4m3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(y1), "f"(y0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(y3), "f"(y2));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    constexpr float kMagic = 12582912.f + 128.f;
    const uint32_t c0 = __float_as_uint(__fadd_rn(y0, kMagic));
    const uint32_t c1 = __float_as_uint(__fadd_rn(y1, kMagic));
    const uint32_t c2 = __float_as_uint(__fadd_rn(y2, kMagic));
    const uint32_t c3 = __float_as_uint(__fadd_rn(y3, kMagic));
    return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
  }
}

// fp16 pairs of four codes, exact.  int8: bytes 0, 2 and bytes 1, 3 read as fp16
// subnormals, (code + 128) * 2^-24.  e4m3: bytes 0, 1 and bytes 2, 3 converted.
template <bool kE4m3>
__device__ __forceinline__ void kv8_operands(uint32_t w, uint32_t& a, uint32_t& b) {
  if constexpr (kE4m3) {
    const uint16_t lo = static_cast<uint16_t>(w), hi = static_cast<uint16_t>(w >> 16);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(a) : "h"(lo));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(b) : "h"(hi));
  } else {
    a = __byte_perm(w, 0, 0x4240);
    b = __byte_perm(w, 0, 0x4341);
  }
}

// The same with int8 codes' 128 taken off (exact in fp16).
template <bool kE4m3>
__device__ __forceinline__ void kv8_signed_operands(uint32_t w, uint32_t& a, uint32_t& b) {
  kv8_operands<kE4m3>(w, a, b);
  if constexpr (!kE4m3) {
    const __half2 less = __halves2half2(__ushort_as_half(0x8080), __ushort_as_half(0x8080));   // -128 * 2^-24
    __half2 x = __hadd2(*reinterpret_cast<__half2*>(&a), less);
    __half2 y = __hadd2(*reinterpret_cast<__half2*>(&b), less);
    a = *reinterpret_cast<uint32_t*>(&x);
    b = *reinterpret_cast<uint32_t*>(&y);
  }
}

// The value of byte i of w, before the scale.
template <bool kE4m3>
__device__ __forceinline__ float kv8_code_value(uint32_t w, int i) {
  const uint32_t byte = (w >> (8 * i)) & 0xffu;
  if constexpr (kE4m3) {
    __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
    return __half2float(__half(h));
  } else {
    return static_cast<float>(static_cast<int>(byte) - 128);
  }
}

}  // namespace oscar
