// Page format of the 4-bit cache (device side) and the arithmetic of its codes.
//
// A value is code * s * g: code an e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), s the e4m3 scale of its block of 16, g the fp32 scale of its page.  A block of
// keys is one channel of the page's 16 tokens (key channels differ far more in size than
// tokens do), a block of values 16 channels of one token.  code * s has at most 6 bits
// and lies in [2^-10, 2688]: exact in fp16, so attention multiplies codes by block scales in
// fp16 without a rounding.
//
// One block of memory per (page of 16 tokens, KV head): 8*d bytes of key codes, 8*d of value
// codes, d key scales, d value scales, then four fp32 words (key scale, value scale, 0, 0):
// 18*d + 16 bytes.  The order is the attention kernel's: a lane (4*gid + tig) of a warp
// reads 32 codes by one 16-byte shared-memory load without bank conflicts.
//   key (t, c): chunk (c/64)*32 + 4*(t/2) + (c/16)%4 of 16 bytes, byte 8*(t%2) + (c%16)/2 in it,
//     low nibble for even c.
//   value (t, c): chunk (c/64)*32 + 4*((c/4)%8) + t/4, byte 8*((c/32)%2) + 2*(c%4) + (t%4)/2 in
//     it, low nibble for even t.
//   key scale of channel c: byte c.
//   value scale (t, b = c/16): byte (b/4)*64 + ((b%2)*4 + t/4)*8 + ((b/2)%2)*4 + t%4.
// The tail block of a sequence is that of the 8-bit cache.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "kv8_layout.cuh"

namespace oscar {

template <int D>
struct Kv4Fmt {
  static constexpr int kCodes = 8 * D;             // bytes of one code area
  static constexpr int kKeyScales = 16 * D;        // byte offsets
  static constexpr int kValueScales = 17 * D;
  static constexpr int kScales = 18 * D;
  static constexpr int kBlock = 18 * D + 16;
  static constexpr int kTailHalf = 16 * D;         // elements of one tail area
  static constexpr int kTailBytes = 64 * D;
};

// What the caches' kernels are made for; the first two are oscar_kv8_desc's formats.
enum KvCode { kCodeInt8 = OSCAR_KV8_INT8, kCodeE4m3 = OSCAR_KV8_E4M3, kCodeE2m1 = 2 };

template <int D, int kCode>
using KvFmt = std::conditional_t<kCode == kCodeE2m1, Kv4Fmt<D>, Kv8Fmt<D>>;

// Blocks of memory whose largest value is below 2^-97 are stored as zeros: every scale and
// quotient below stays normal.
constexpr float kKv4Least = 6.310887241768095e-30f;   // 2^-97
constexpr float kKv4Top = 2688.f;                     // 6 * 448
constexpr float kKv4BlockTop = 448.f;

// Byte of a value scale.
__device__ __forceinline__ int kv4_value_scale(int t, int b) {
  return (b >> 2) * 64 + ((b & 1) * 4 + (t >> 2)) * 8 + ((b >> 1) & 1) * 4 + (t & 3);
}

// The eight codes of a word as fp16 pairs in order, exact.
__device__ __forceinline__ void kv4_pairs(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm("{\n .reg .b8 x, y, z, u;\n mov.b32 {x, y, z, u}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, x;\n cvt.rn.f16x2.e2m1x2 %1, y;\n"
      " cvt.rn.f16x2.e2m1x2 %2, z;\n cvt.rn.f16x2.e2m1x2 %3, u;\n}\n"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}

// The four scales of a word as fp16 pairs in order, exact.
__device__ __forceinline__ void kv4_scales(uint32_t w, uint32_t& a, uint32_t& b) { kv8_operands<true>(w, a, b); }

// Eight codes of y0 .. y7 (nearest, ties to even, saturating), packed in order.
__device__ __forceinline__ uint32_t kv4_codes8(const float (&y)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}

}  // namespace oscar
