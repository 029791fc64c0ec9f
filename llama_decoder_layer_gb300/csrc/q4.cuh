// The 4-bit KV-cache format: where a (token, element) of a tile lies, and the
// conversions between bf16 / fp32 values and the stored bits.
//
// A tile holds 16 tokens of one KV head: 8 D bytes of e2m1 codes, then D bytes
// of e4m3 scales, one per 16 neighbouring elements of a token.  The value of an
// element is code * scale * g, g a power of two for the whole array.  code *
// scale has at most 2 + 4 significant bits and lies on a grid of 2^-10 below
// 2688, so it is exact in bf16 and in fp16, and dividing or multiplying by g
// is exact in fp32.
//
// The order of the bytes is the one in which the decode attention's lanes take
// them (lane = 4 g + t holds rows g, g + 8 and columns 2t, 2t + 1, 2t + 8,
// 2t + 9 of an m16n8k16 operand): a lane reads its share of the codes with one
// 16-byte load per 8 keys (8 bytes at D = 64) and its scales with one load, at
// consecutive addresses over the warp, with no exchange between lanes.
//   K codes:  token row k at k * D/2, element e at byte e / 2 (low half first):
//             lane t of row k contracts over elements t * D/4 ..
//   V codes:  token k, element e at (k / 8) * 4 D + (e / W * 4 + (k % 8) / 2) * W
//             + (k % 2) * W/2 + (e % W) / 2, W = D / 8: lane (g, t) holds elements
//             g * W .. of the token pair (2t, 2t + 1) of each half
//   K scales: 8 D + ((k % 8) * 4 + s / P) * 2 P + (k / 8) * P + s % P for group s,
//             P = D / 64
//   V scales: 8 D + (s * 4 + (k % 8) / 2) * 4 + (k / 8) * 2 + k % 2
// Every token's codes and scales lie in bytes of their own, so tokens are
// written independently of one another.
#pragma once

#include "common.cuh"

namespace llama {

constexpr int kQ4Block = 16;  // tokens a tile
constexpr int kQ4Group = 16;  // elements a scale

__host__ __device__ constexpr int q4_tile_bytes(int D) { return 9 * D; }

template <int D>
__host__ __device__ __forceinline__ int q4_k_scale_at(int k, int s) {
  constexpr int P = D / 64;
  return 8 * D + ((k & 7) * 4 + s / P) * 2 * P + (k >> 3) * P + s % P;
}

template <int D>
__host__ __device__ __forceinline__ int q4_v_scale_at(int k, int s) {
  return 8 * D + (s * 4 + ((k & 7) >> 1)) * 4 + (k >> 3) * 2 + (k & 1);
}

// byte of the code of V element e of token k
template <int D>
__host__ __device__ __forceinline__ int q4_v_code_at(int k, int e) {
  constexpr int W = D / 8;
  return (k >> 3) * 4 * D + ((e / W) * 4 + ((k & 7) >> 1)) * W + (k & 1) * (W / 2) + (e % W) / 2;
}

// four bytes of e2m1 pairs -> four fp16 pairs (the low half of a byte in the low half)
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// two e4m3 bytes -> an fp16 pair (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t v) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(v)));
  return d;
}

// nearest e4m3 (at most 448, in the low byte) of the fp16 number nearest to x >= 0
__device__ __forceinline__ uint32_t f32_to_e4m3_by_f16(float x) {
  uint32_t h;
  uint16_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(0.f), "f"(x));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(h));
  return d & 0xFFu;
}

// nearest e2m1 of eight values (ties to the even code, at most 6 in size), x[0] in the lowest four bits
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&x)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

// byte of the codes of elements 8 c .. 8 c + 7 of token k (K or V), and of their scale
template <int D>
__host__ __device__ __forceinline__ int q4_code_at(bool is_v, int k, int c) {
  return is_v ? q4_v_code_at<D>(k, c * 8) : k * (D / 2) + c * 4;
}

template <int D>
__host__ __device__ __forceinline__ int q4_scale_at(bool is_v, int k, int s) {
  return is_v ? q4_v_scale_at<D>(k, s) : q4_k_scale_at<D>(k, s);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float f16_lo(uint32_t v) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(v));
  return f;
}

__device__ __forceinline__ float f16_hi(uint32_t v) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(v));
  return f;
}

// eight codes, their scale's bits and g -> eight bf16 values (exact)
__device__ __forceinline__ uint4 q4_to_bf16(uint32_t code, uint32_t s8, float g) {
  const float m = f16_lo(e4m3x2_to_f16(s8)) * g;
  const uint64_t m2 = f2_pack(m, m);
  uint32_t p[4], w[4];
  e2m1x8_to_f16(code, p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f2_mul(f2_pack(f16_lo(p[i]), f16_hi(p[i])), m2), lo, hi);
    w[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace llama
