// The 4-bit paged KV cache: quantising rows as they are written, and reading
// rows back (the format is in q4.cuh).
//
// Writing, per 16 neighbouring elements x of a token's head row:
//   s = e4m3(max |x| / (6 g)),   code_i = e2m1(x_i / (s g)),
// both to nearest, ties to even, saturating.  A NaN counts as zero in both, an
// infinity as a value beyond every scale, so the cache holds finite values
// only and a bad token cannot reach rows that do not attend to it.  s = 0
// (every |x| below 6 g 2^-10) stores zeros.
//   The rounding is that of the exact quotients: x has 8 significant bits, 6 m
// and s t (t a border between two codes) at most 8, so a quotient that is not a
// border itself is at least 2^-9 away from it, and one that is comes out of the
// fp32 division exactly.
// Reading: bf16(code * s * g), exact while it is a normal bf16.
//
// Both move 2 + 9/16 bytes an element and are bound by HBM: a thread takes one
// group of 16 (32 bytes of bf16 against 8 + 1 bytes).
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q4.cuh"

namespace llama {

namespace {

constexpr int kThreads = 256;

template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_write_q4(const CacheQ4Args a) {
  constexpr int GR = D / kQ4Group;
  const long long half = static_cast<long long>(a.T) * a.n_kv * GR;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < 2 * half;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const bool is_v = i >= half;
    const long long j = is_v ? i - half : i;
    const int s = static_cast<int>(j % GR);
    const int h = static_cast<int>((j / GR) % a.n_kv);
    const int t = static_cast<int>(j / (static_cast<long long>(GR) * a.n_kv));
    const int slot = a.slots[t];
    if (slot < 0) continue;
    if (slot >= a.num_blocks * kQ4Block) {
      if (s == 0 && h == 0 && !is_v) report_error(a.err, kErrGuard, kWhereSlot);
      continue;
    }
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? a.v : a.k) +
                               t * (is_v ? a.v_stride : a.k_stride) + h * D + s * kQ4Group;
    const float inv_g = is_v ? a.inv_v_scale : a.inv_k_scale;
    float x[16];
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 u = reinterpret_cast<const uint4*>(src)[c];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * c + 2 * e] = bf16_lo(w[e]) * inv_g;
        x[8 * c + 2 * e + 1] = bf16_hi(w[e]) * inv_g;
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] = x[e] != x[e] ? 0.f : x[e];
      amax = fmaxf(amax, fabsf(x[e]));
    }
    const uint32_t s8 = f32_to_e4m3(__fdiv_rn(amax, 6.f));
    const float sc = f16_lo(e4m3x2_to_f16(s8));
    uint32_t code[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = s8 == 0 ? 0.f : __fdiv_rn(x[8 * c + e], sc);
      code[c] = f32x8_to_e2m1(y);
    }
    const int k = slot % kQ4Block;
    uint8_t* tile = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                    (static_cast<size_t>(slot / kQ4Block) * a.n_kv + h) * q4_tile_bytes(D);
    if (!is_v) {
      *reinterpret_cast<uint2*>(tile + k * (D / 2) + s * 8) = make_uint2(code[0], code[1]);
      tile[q4_k_scale_at<D>(k, s)] = static_cast<uint8_t>(s8);
    } else {
      *reinterpret_cast<uint32_t*>(tile + q4_v_code_at<D>(k, s * 16)) = code[0];
      *reinterpret_cast<uint32_t*>(tile + q4_v_code_at<D>(k, s * 16 + 8)) = code[1];
      tile[q4_v_scale_at<D>(k, s)] = static_cast<uint8_t>(s8);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_read_q4(const CacheQ4Args a) {
  constexpr int GR = D / kQ4Group;
  const long long half = static_cast<long long>(a.T) * a.n_kv * GR;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < 2 * half;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const bool is_v = i >= half;
    const long long j = is_v ? i - half : i;
    const int s = static_cast<int>(j % GR);
    const int h = static_cast<int>((j / GR) % a.n_kv);
    const int t = static_cast<int>(j / (static_cast<long long>(GR) * a.n_kv));
    const int slot = a.slots[t];
    if (slot < 0) continue;
    if (slot >= a.num_blocks * kQ4Block) {
      if (s == 0 && h == 0 && !is_v) report_error(a.err, kErrGuard, kWhereSlot);
      continue;
    }
    const int k = slot % kQ4Block;
    const uint8_t* tile = static_cast<const uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                          (static_cast<size_t>(slot / kQ4Block) * a.n_kv + h) * q4_tile_bytes(D);
    uint32_t code[2];
    uint32_t s8;
    if (!is_v) {
      const uint2 c = *reinterpret_cast<const uint2*>(tile + k * (D / 2) + s * 8);
      code[0] = c.x;
      code[1] = c.y;
      s8 = tile[q4_k_scale_at<D>(k, s)];
    } else {
      code[0] = *reinterpret_cast<const uint32_t*>(tile + q4_v_code_at<D>(k, s * 16));
      code[1] = *reinterpret_cast<const uint32_t*>(tile + q4_v_code_at<D>(k, s * 16 + 8));
      s8 = tile[q4_v_scale_at<D>(k, s)];
    }
    const float m = f16_lo(e4m3x2_to_f16(s8)) * (is_v ? a.v_scale : a.k_scale);
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? a.v_out : a.k_out) + t * (is_v ? a.v_stride : a.k_stride) +
                         h * D + s * kQ4Group;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t p[4];
      e2m1x8_to_f16(code[c], p);
      uint4 u;
      u.x = pack_bf16x2(f16_lo(p[0]) * m, f16_hi(p[0]) * m);
      u.y = pack_bf16x2(f16_lo(p[1]) * m, f16_hi(p[1]) * m);
      u.z = pack_bf16x2(f16_lo(p[2]) * m, f16_hi(p[2]) * m);
      u.w = pack_bf16x2(f16_lo(p[3]) * m, f16_hi(p[3]) * m);
      reinterpret_cast<uint4*>(dst)[c] = u;
    }
  }
}

int grid_of(const CacheQ4Args& a) {
  const long long work = 2LL * a.T * a.n_kv * (a.head_dim / kQ4Group);
  const long long g = (work + kThreads - 1) / kThreads, cap = static_cast<long long>(num_sms()) * 16;
  return static_cast<int>(g > cap ? cap : g);
}

}  // namespace

int kv_write_q4_launch(const CacheQ4Args& a, cudaStream_t s) {
  if (a.T <= 0) return 0;
  if (a.head_dim == 128) return launch_kernel(k_kv_write_q4<128>, dim3(grid_of(a)), dim3(kThreads), 0, s, false, a);
  return launch_kernel(k_kv_write_q4<64>, dim3(grid_of(a)), dim3(kThreads), 0, s, false, a);
}

int kv_read_q4_launch(const CacheQ4Args& a, cudaStream_t s) {
  if (a.T <= 0) return 0;
  if (a.head_dim == 128) return launch_kernel(k_kv_read_q4<128>, dim3(grid_of(a)), dim3(kThreads), 0, s, false, a);
  return launch_kernel(k_kv_read_q4<64>, dim3(grid_of(a)), dim3(kThreads), 0, s, false, a);
}

}  // namespace llama
