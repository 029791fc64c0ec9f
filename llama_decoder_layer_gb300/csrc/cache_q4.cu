// The 4-bit paged KV cache: quantising rows as they are written, and reading
// rows back (the format is in q4.cuh).
//
// Writing, per 16 neighbouring elements x of a token's head row:
//   s = e4m3(max |x| / (6 g)),   code_i = e2m1(x_i / (s g)),
// both to nearest, ties to even, saturating.  A NaN counts as zero in both, an
// infinity as a value beyond every scale, so the cache holds finite values
// only and a bad token cannot reach rows that do not attend to it.  s = 0
// (every |x| below 6 g 2^-10) stores zeros.
//   The rounding is that of the exact quotients: x has 8 significant bits, a
// border t of the codes times s at most 7, so x / s either is t or is at least
// 2^-8 t >= 2^-10 away from it.  x times 1 / s in fp32 is off by less than 2^-19
// below 8; rounded to a multiple of 2^-13 it is t where the quotient is, and stays
// on its side where it is not.  (max / 6 is an fp32 division: the borders of e4m3
// times 6 have at most 7 bits, and a quotient that is one comes out exactly.)
// Reading: bf16(code * s * g), exact.
//
// Both move 2 + 9/16 bytes an element and are bound by HBM.  A thread takes
// chunks of 8 elements (16 bytes of bf16, 4 of codes), kUnroll of them kThreads
// apart with all their loads in flight, so that a warp's bf16 accesses are
// contiguous; two lanes share a scale.  (16 elements a thread, with 64-bit index
// arithmetic and an fp32 division per element, took 104 us for 32768 tokens x 8 x
// 128 written and read back.)
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q4.cuh"

namespace llama {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// n / d for n < 2^31 by one multiplication
struct FastDiv {
  uint32_t mul, shift, d;
  explicit FastDiv(uint32_t div) : mul(0), shift(0), d(div) {
    while ((1ull << shift) < div) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - div)) / div + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(__umulhi(n, mul)) + n) >> shift);
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Where chunk i of the launch's tokens x heads x D / 8 chunks lies.
template <int D>
struct Chunk {
  long long t;  // token
  int h, c, slot;
  bool ok;
};

// chunk of a token `i` from token t0 on; the slot is loaded, out-of-range ones reported
template <int D>
__device__ __forceinline__ Chunk<D> chunk_of(const CacheQ4Args& a, const FastDiv& per_token, long long t0, uint32_t i,
                                             bool is_v) {
  constexpr int C = D / 8;
  Chunk<D> x;
  const uint32_t t = per_token(i), r = i - t * per_token.d;
  x.t = t0 + t;
  x.h = r / C;
  x.c = r % C;
  x.ok = x.t < a.T;
  x.slot = x.ok ? a.slots[x.t] : -1;
  if (x.slot >= a.num_blocks * kQ4Block) {
    if (r == 0 && !is_v) report_error(a.err, kErrGuard, kWhereSlot);
    x.ok = false;
  }
  x.ok = x.ok && x.slot >= 0;
  return x;
}

// CTA (x, y): kThreads * kUnroll chunks of K (y = 0) or V, of the tokens of one
// span (so that the index arithmetic stays in 32 bits).
template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_write_q4(const CacheQ4Args a, const FastDiv per_token, int span,
                                                          int ctas_per_span) {
  const bool is_v = blockIdx.y != 0;
  const long long t0 = static_cast<long long>(blockIdx.x / ctas_per_span) * span;
  const uint32_t i0 = (blockIdx.x % ctas_per_span) * (kThreads * kUnroll) + threadIdx.x;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? a.v : a.k);
  const long long stride = is_v ? a.v_stride : a.k_stride;
  const float inv_g = is_v ? a.inv_v_scale : a.inv_k_scale;
  uint8_t* cache = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache);
  Chunk<D> x[kUnroll];
  uint4 u[kUnroll];
#pragma unroll
  for (int n = 0; n < kUnroll; ++n) {
    x[n] = chunk_of<D>(a, per_token, t0, i0 + n * kThreads, is_v);
    if (i0 + n * kThreads >= static_cast<uint32_t>(span) * per_token.d) x[n].ok = false;
    u[n] = make_uint4(0, 0, 0, 0);
    if (x[n].ok) u[n] = *reinterpret_cast<const uint4*>(src + x[n].t * stride + x[n].h * D + x[n].c * 8);
  }
#pragma unroll
  for (int n = 0; n < kUnroll; ++n) {
    float v[8] = {bf16_lo(u[n].x), bf16_hi(u[n].x), bf16_lo(u[n].y), bf16_hi(u[n].y),
                  bf16_lo(u[n].z), bf16_hi(u[n].z), bf16_lo(u[n].w), bf16_hi(u[n].w)};
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(v[e]));
    if (amax != amax) {  // rare: NaN counts as zero
      amax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = v[e] != v[e] ? 0.f : v[e];
        amax = fmaxf(amax, fabsf(v[e]));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // the group's other half is in the next lane
    const uint32_t s8 = f32_to_e4m3(__fdiv_rn(amax * inv_g, 6.f));
    const float sc = f16_lo(e4m3x2_to_f16(s8));
    const float inv = s8 == 0 ? 0.f : __frcp_rn(sc) * inv_g;
    constexpr float kSnap = 1.5f * 1024.f;  // sums with it are multiples of 2^-13 below 2^10
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = copysignf(__fadd_rn(__fmaf_rn(fabsf(v[e]), inv, kSnap), -kSnap), v[e]);
    const uint32_t code = s8 == 0 ? 0u : f32x8_to_e2m1(y);
    const int k = x[n].slot & 15, s = x[n].c >> 1;
    const uint32_t next = __shfl_down_sync(0xffffffffu, s8, 2);  // the next group's scale (K stores two at D = 128)
    if (x[n].ok) {
      uint8_t* tile = cache + (static_cast<size_t>(x[n].slot >> 4) * a.n_kv + x[n].h) * q4_tile_bytes(D);
      *reinterpret_cast<uint32_t*>(tile + q4_code_at<D>(is_v, k, x[n].c)) = code;
      if (D == 128 && !is_v) {
        if ((x[n].c & 3) == 0)
          *reinterpret_cast<uint16_t*>(tile + q4_k_scale_at<D>(k, s)) = static_cast<uint16_t>(s8 | (next << 8));
      } else if ((x[n].c & 1) == 0) {
        tile[q4_scale_at<D>(is_v, k, s)] = static_cast<uint8_t>(s8);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_read_q4(const CacheQ4Args a, const FastDiv per_token, int span,
                                                         int ctas_per_span) {
  const bool is_v = blockIdx.y != 0;
  const long long t0 = static_cast<long long>(blockIdx.x / ctas_per_span) * span;
  const uint32_t i0 = (blockIdx.x % ctas_per_span) * (kThreads * kUnroll) + threadIdx.x;
  const uint8_t* cache = static_cast<const uint8_t*>(is_v ? a.v_cache : a.k_cache);
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? a.v_out : a.k_out);
  const long long stride = is_v ? a.v_stride : a.k_stride;
  const float g = is_v ? a.v_scale : a.k_scale;
  Chunk<D> x[kUnroll];
  uint32_t code[kUnroll], s8[kUnroll];
#pragma unroll
  for (int n = 0; n < kUnroll; ++n) {
    x[n] = chunk_of<D>(a, per_token, t0, i0 + n * kThreads, is_v);
    if (i0 + n * kThreads >= static_cast<uint32_t>(span) * per_token.d) x[n].ok = false;
  }
#pragma unroll
  for (int n = 0; n < kUnroll; ++n) {
    if (!x[n].ok) continue;
    const int k = x[n].slot & 15;
    const uint8_t* tile = cache + (static_cast<size_t>(x[n].slot >> 4) * a.n_kv + x[n].h) * q4_tile_bytes(D);
    code[n] = *reinterpret_cast<const uint32_t*>(tile + q4_code_at<D>(is_v, k, x[n].c));
    s8[n] = tile[q4_scale_at<D>(is_v, k, x[n].c >> 1)];
  }
#pragma unroll
  for (int n = 0; n < kUnroll; ++n)
    if (x[n].ok)
      *reinterpret_cast<uint4*>(dst + x[n].t * stride + x[n].h * D + x[n].c * 8) = q4_to_bf16(code[n], s8[n], g);
}

// tokens a span: chunk indices within one stay below 2^30
template <typename Kernel>
int launch(Kernel kernel, const CacheQ4Args& a, cudaStream_t s) {
  const uint32_t per_token = static_cast<uint32_t>(a.n_kv) * (a.head_dim / 8);
  const long long most = (1 << 30) / static_cast<long long>(per_token);
  const int span = static_cast<int>(a.T < most ? a.T : most);
  const long long ctas = (static_cast<long long>(span) * per_token + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  const long long spans = (static_cast<long long>(a.T) + span - 1) / span;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(spans * ctas), 2), dim3(kThreads), 0, s, false, a,
                       FastDiv(per_token), span, static_cast<int>(ctas));
}

}  // namespace

int kv_write_q4_launch(const CacheQ4Args& a, cudaStream_t s) {
  if (a.T <= 0) return 0;
  return a.head_dim == 128 ? launch(k_kv_write_q4<128>, a, s) : launch(k_kv_write_q4<64>, a, s);
}

int kv_read_q4_launch(const CacheQ4Args& a, cudaStream_t s) {
  if (a.T <= 0) return 0;
  return a.head_dim == 128 ? launch(k_kv_read_q4<128>, a, s) : launch(k_kv_read_q4<64>, a, s);
}

}  // namespace llama
