// Microscaled matrices: the formats, where a scale lies, and the conversions
// between bf16 / fp32 values and the stored bits.
//
// A matrix [rows, cols] is codes, row by row, and one scale for every group of
// neighbouring elements of a row; a value is code * scale * g, g a power of two
// for the whole matrix (1 unless the format is nvfp4):
//   nvfp4  4-bit e2m1 codes, an e4m3 scale for 16 elements
//   fp4    4-bit e2m1 codes, a power-of-two (e8m0) scale for 32 elements
//   fp8    8-bit e4m3 codes, a power-of-two (e8m0) scale for 32 elements
// Scales lie in tiles of 128 rows x 4 groups of 512 bytes, in the order in which
// the tensor cores take them into tensor memory (lane r % 32, 32-bit column
// r / 32, the four groups side by side), so that a tile is copied as it is:
//   byte of (row r, group s) = ((r / 128) * ceil(groups / 4) + s / 4) * 512
//                              + r % 32 * 16 + r % 128 / 32 * 4 + s % 4
#pragma once

#include "common.cuh"
#include "llama_layer.h"
#include "q4.cuh"

namespace llama {

constexpr int kMxNvfp4 = LLAMA_MX_NVFP4, kMxFp4 = LLAMA_MX_FP4, kMxFp8 = LLAMA_MX_FP8;
constexpr int kMxTileRows = 128, kMxTileGroups = 4, kMxTileBytes = 512;

__host__ __device__ constexpr int mx_group(int fmt) { return fmt == kMxNvfp4 ? 16 : 32; }
__host__ __device__ constexpr int mx_bits(int fmt) { return fmt == kMxFp8 ? 8 : 4; }

// offset of row r's word of four scales in a tile
__host__ __device__ __forceinline__ constexpr int mx_scale_word(int r) {
  return (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// where the scales of groups 4 kt .. 4 kt + 3 of a row lie; ktiles = ceil(groups / 4)
__host__ __device__ __forceinline__ size_t mx_scale_at(int row, int kt, int ktiles) {
  return (static_cast<size_t>(row >> 7) * ktiles + kt) * kMxTileBytes + mx_scale_word(row);
}

// ---------------------------------------------------------------------------
// Scales.  `top` is the largest |x| of the group as the bits of an fp32 number
// (an unsigned maximum over absolute values, so an infinity or a NaN is at or
// above 0x7f800000): a group that holds one gets a NaN scale, and with it every
// product that its row enters is NaN.
// ---------------------------------------------------------------------------

// the power of two 2^(b - 127) as fp32, and its reciprocal (b 0 .. 254; exact, subnormal at the ends)
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fffffffu : b << 23);
}
__device__ __forceinline__ float e8m0_inverse(uint32_t b) {
  return __uint_as_float(b >= 254 ? 0x00400000u : (254 - b) << 23);
}

// The smallest power of two with which no element is beyond the largest code,
// 1.75 * 2^8 or 1.5 * 2^2: the exponent, one more above that significand.
template <int FMT>
__device__ __forceinline__ uint32_t e8m0_scale(uint32_t top) {
  constexpr uint32_t kCarry = FMT == kMxFp8 ? 0x1fffffu : 0x3fffffu;
  constexpr int kExp = FMT == kMxFp8 ? 8 : 2;
  if (top >= 0x7f800000u) return 255;
  const int b = static_cast<int>((top + kCarry) >> 23) - kExp;
  return b < 0 ? 0 : b;
}

// two e4m3 codes of fp32 values (nearest, ties to even, saturating), x0 in the low byte
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float x0, float x1) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(x1), "f"(x0));
  return d;
}

// e4m3 to an fp32 number
__device__ __forceinline__ float e4m3_value(uint32_t b) { return f16_lo(e4m3x2_to_f16(b & 0xFFu)); }

// nvfp4's scale, e4m3(top * sixth), sixth = 1 / (6 g), and the factor that takes elements to codes.
// BF16: the elements are bf16 numbers, whose quotients top / (6 g) are on a border of e4m3 or 2^-8 away
// from it; the product's fp32 error is rounded away by fp16's 11 bits first.
template <bool BF16>
__device__ __forceinline__ uint32_t nvfp4_scale(uint32_t top, float sixth) {
  if (top >= 0x7f800000u) return 0x7f;
  const float v = __uint_as_float(top) * sixth;
  if constexpr (BF16) {
    return f32_to_e4m3_by_f16(v);
  } else {
    return f32x2_to_e4m3(v, 0.f) & 0xFFu;
  }
}

// A group's scale byte and the factor on its elements before they are rounded to codes.
struct MxScale {
  uint32_t byte;
  float factor;
};
template <int FMT, bool BF16>
__device__ __forceinline__ MxScale mx_scale(uint32_t top, float sixth, float inv_g) {
  MxScale s;
  if constexpr (FMT == kMxNvfp4) {
    s.byte = nvfp4_scale<BF16>(top, sixth);
    s.factor = s.byte == 0 ? 0.f : __frcp_rn(e4m3_value(s.byte)) * inv_g;  // (inv_g: a power of two)
  } else {
    s.byte = e8m0_scale<FMT>(top);
    s.factor = e8m0_inverse(s.byte);
  }
  return s;
}

// Eight codes, 4 bytes (e2m1, in .x) or 8 bytes (e4m3), of elements times their group's factor.  nvfp4 of bf16 elements:
// x / (s g) is on a border of e2m1 or 2^-10 away from it and the product is off by less than 2^-19 below 8, so that rounded
// to a multiple of 2^-13 (the last bit of a sum with 1.5 * 2^10) it falls where the quotient does.  The other formats'
// factors are powers of two: exact.
template <int FMT, bool BF16>
__device__ __forceinline__ uint2 mx_codes8(const float (&x)[8], float factor) {
  constexpr float kSnap = 1536.f;
  const uint64_t f2 = f2_pack(factor, factor), up = f2_pack(kSnap, kSnap), down = f2_pack(-kSnap, -kSnap);
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t v = f2_pack(x[2 * i], x[2 * i + 1]);
    f2_unpack(FMT == kMxNvfp4 && BF16 ? f2_add(f2_fma(v, f2, up), down) : f2_mul(v, f2), y[2 * i], y[2 * i + 1]);
  }
  if constexpr (FMT == kMxFp8) {
    return make_uint2(f32x2_to_e4m3(y[0], y[1]) | f32x2_to_e4m3(y[2], y[3]) << 16,
                      f32x2_to_e4m3(y[4], y[5]) | f32x2_to_e4m3(y[6], y[7]) << 16);
  } else {
    return make_uint2(f32x8_to_e2m1(y), 0);
  }
}

// the values of eight codes
template <int FMT>
__device__ __forceinline__ void mx_values8(uint2 w, float (&v)[8]) {
  uint32_t h[4];
  if constexpr (FMT == kMxFp8) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"(static_cast<uint16_t>(w.x)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"(static_cast<uint16_t>(w.x >> 16)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2]) : "h"(static_cast<uint16_t>(w.y)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[3]) : "h"(static_cast<uint16_t>(w.y >> 16)));
  } else {
    e2m1x8_to_f16(w.x, h);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = f16_lo(h[i]);
    v[2 * i + 1] = f16_hi(h[i]);
  }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

}  // namespace llama
