// mxfp4.cuh — the 4-bit cache format: OCP Microscaling (MX) v1.0 MXFP4.
//
// 32 consecutive elements of a row share one E8M0 byte b, the power of two
// 2^(b - 127) (255 = NaN: the whole block reads as NaN; 0 reads as 0, its
// 2^-127 being below fp32's normal range), and each element is an E2M1 code,
// sign and magnitude {0, 0.5, 1, 1.5, 2, 3, 4, 6}, two codes a byte with the
// even element in the low half. A block of the pool holds one kv-head's rows
// together: codes [num_blocks, num_kv_heads, block_size, head_dim / 2],
// scales [num_blocks, num_kv_heads, block_size, head_dim / 32], so that the
// rows a decode CTA reads of one block and head are contiguous bytes (1 KB of
// codes and 64 B of scales for 16 tokens of 128 dims).
#pragma once

#include <math_constants.h>

#include "device_common.cuh"

namespace paged {

constexpr int kMxBlock = 32;     // elements that share a scale
constexpr int kMxNan = 255;      // scale byte of a block that holds a non-finite value
// The scale exponents the writer uses: 2^(b - 127) and its inverse are normal
// fp32 numbers.
constexpr int kMxMinExp = -126, kMxMaxExp = 125;

// Scale byte of a block whose largest magnitude is amax: the largest power of
// two at most amax, divided by 4 (E2M1's largest power of two), so that the
// scaled magnitudes lie in [4, 8) and those above 6 saturate.
__device__ __forceinline__ int mx_scale_byte(float amax) {
  const int field = static_cast<int>(__float_as_uint(amax) >> 23);  // amax >= 0
  if (field == 255) return kMxNan;  // infinity or NaN in the block
  return min(max(field - 127 - 2, kMxMinExp), kMxMaxExp) + 127;
}

// 2^(127 - b): what the block's elements are multiplied by before rounding.
__device__ __forceinline__ float mx_inverse(int b) {
  return __uint_as_float(static_cast<uint32_t>(254 - b) << 23);
}

// 2^(b - 127) as fp32.
__device__ __forceinline__ float mx_scale(int b) {
  return b == kMxNan ? __uint_as_float(0x7fc00000u)
                     : __uint_as_float(static_cast<uint32_t>(b) << 23);
}

// Nonzero if some byte of w is 255.
__device__ __forceinline__ uint32_t has_ff(uint32_t w) {
  return (~w - 0x01010101u) & w & 0x80808080u;
}

// Eight scaled values -> eight codes (element 0 in the low half of byte 0),
// round to nearest even, saturating.
__device__ __forceinline__ uint32_t mx_pack8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The eight codes of a word as four f16 pairs (exact): pair j holds the low
// and the high half of byte j.
__device__ __forceinline__ void mx_unpack8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n"
      " mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n"
      " cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

}  // namespace paged
