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
// on its side where it is not.  For the scale likewise: the borders of e4m3 times
// 6 have at most 7 bits, so max / 6 is one or 2^-8 of it away, and max times fp32's
// 1 / 6, rounded to fp16's 11 bits, falls where the quotient does.
// Reading: bf16(code * s * g), exact.
//
// Both move 2 + 9/16 bytes an element and are bound by HBM.  A thread takes
// chunks of 8 elements (16 bytes of bf16, 4 of codes) of U tokens, always the same
// chunk of the row, with all its loads in flight; a warp's bf16 accesses are
// contiguous, two lanes share a scale.  A CTA has a whole number of rows (or a part
// of one) in its threads, so that one division finds a thread's place.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q4.cuh"

namespace llama {

namespace {

constexpr int kMaxThreads = 512;

// A launch's shape: `chunks` chunks of 8 elements a token row (K or V); a CTA
// covers `rows` rows at a time, or 1 / parts of one.
struct Shape {
  int chunks, rows, parts;
};

// This thread's chunk (head h, chunk c of it) and its first token; -1: none.
template <int D, int U>
__device__ __forceinline__ long long place(const Shape& g, int& h, int& c, bool& is_v) {
  constexpr int C = D / 8;
  const int part = blockIdx.y >> 1, row = threadIdx.x / g.chunks;
  const int r = g.parts > 1 ? part * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)
                            : static_cast<int>(threadIdx.x) - row * g.chunks;
  is_v = blockIdx.y & 1;
  h = r / C;
  c = r % C;
  if (r >= g.chunks) return -1;
  return static_cast<long long>(blockIdx.x) * g.rows * U + (g.parts > 1 ? 0 : row);
}

// the slots of this thread's tokens: -1 where there is nothing to do
template <int U>
__device__ __forceinline__ void load_slots(const CacheQ4Args& a, const Shape& g, long long t0, bool reports,
                                           int (&slot)[U]) {
#pragma unroll
  for (int n = 0; n < U; ++n) {
    const long long t = t0 + n * g.rows;
    slot[n] = t0 >= 0 && t < a.T ? a.slots[t] : -1;
  }
#pragma unroll
  for (int n = 0; n < U; ++n)
    if (slot[n] >= a.num_blocks * kQ4Block) {
      if (reports) report_error(a.err, kErrGuard, kWhereSlot);
      slot[n] = -1;
    }
}

template <int D, int U>
__global__ void __launch_bounds__(kMaxThreads) k_kv_write_q4(const CacheQ4Args a, const Shape g) {
  int h, c, slot[U];
  bool is_v;
  const long long t0 = place<D, U>(g, h, c, is_v);
  const long long stride = is_v ? a.v_stride : a.k_stride;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? a.v : a.k) + t0 * stride + h * D + c * 8;
  uint4 u[U];
#pragma unroll
  for (int n = 0; n < U; ++n) {  // before the slots are known: every row may be read
    u[n] = make_uint4(0, 0, 0, 0);
    if (t0 >= 0 && t0 + n * g.rows < a.T) u[n] = *reinterpret_cast<const uint4*>(src + n * g.rows * stride);
  }
  load_slots<U>(a, g, t0, h == 0 && c == 0 && !is_v, slot);
  const float inv_g = is_v ? a.inv_v_scale : a.inv_k_scale;
  uint8_t* cache = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + static_cast<size_t>(h) * q4_tile_bytes(D);
#pragma unroll
  for (int n = 0; n < U; ++n) {
    uint32_t w[4] = {u[n].x, u[n].y, u[n].z, u[n].w};
    __nv_bfloat162 top = __habs2(*reinterpret_cast<__nv_bfloat162*>(&w[0]));
#pragma unroll
    for (int e = 1; e < 4; ++e) top = __hmax2_nan(top, __habs2(*reinterpret_cast<__nv_bfloat162*>(&w[e])));
    float amax = __bfloat162float(__hmax_nan(__low2bfloat16(top), __high2bfloat16(top)));
    if (amax != amax) {  // rare: NaN counts as zero
      amax = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((w[e] & 0x7FFFu) > 0x7F80u) w[e] &= 0xFFFF0000u;
        if ((w[e] & 0x7FFF0000u) > 0x7F800000u) w[e] &= 0xFFFFu;
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // the group's other half is in the next lane
    const uint32_t s8 = f32_to_e4m3_by_f16(amax * (inv_g * (1.f / 6.f)));
    const float inv = s8 == 0 ? 0.f : __fdividef(inv_g, f16_lo(e4m3x2_to_f16(s8)));
    constexpr float kSnap = 1.5f * 1024.f;  // sums with it are multiples of 2^-13 below 2^10
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = bf16_lo(w[e]), hi = bf16_hi(w[e]);
      y[2 * e] = copysignf(__fadd_rn(__fmaf_rn(fabsf(lo), inv, kSnap), -kSnap), lo);
      y[2 * e + 1] = copysignf(__fadd_rn(__fmaf_rn(fabsf(hi), inv, kSnap), -kSnap), hi);
    }
    const uint32_t code = s8 == 0 ? 0u : f32x8_to_e2m1(y);
    const uint32_t next = __shfl_down_sync(0xffffffffu, s8, 2);  // the next group's scale (K stores two at D = 128)
    if (slot[n] >= 0) {
      const int k = slot[n] & 15, s = c >> 1;
      uint8_t* tile = cache + static_cast<size_t>(slot[n] >> 4) * (static_cast<size_t>(a.n_kv) * q4_tile_bytes(D));
      *reinterpret_cast<uint32_t*>(tile + q4_code_at<D>(is_v, k, c)) = code;
      if (D == 128 && !is_v) {
        if ((c & 3) == 0)
          *reinterpret_cast<uint16_t*>(tile + q4_k_scale_at<D>(k, s)) = static_cast<uint16_t>(s8 | (next << 8));
      } else if ((c & 1) == 0) {
        tile[q4_scale_at<D>(is_v, k, s)] = static_cast<uint8_t>(s8);
      }
    }
  }
}

template <int D, int U>
__global__ void __launch_bounds__(kMaxThreads) k_kv_read_q4(const CacheQ4Args a, const Shape g) {
  int h, c, slot[U];
  bool is_v;
  const long long t0 = place<D, U>(g, h, c, is_v);
  load_slots<U>(a, g, t0, h == 0 && c == 0 && !is_v, slot);
  const uint8_t* cache =
      static_cast<const uint8_t*>(is_v ? a.v_cache : a.k_cache) + static_cast<size_t>(h) * q4_tile_bytes(D);
  uint32_t code[U], s8[U];
#pragma unroll
  for (int n = 0; n < U; ++n) {
    code[n] = s8[n] = 0;
    if (slot[n] < 0) continue;
    const int k = slot[n] & 15;
    const uint8_t* tile =
        cache + static_cast<size_t>(slot[n] >> 4) * (static_cast<size_t>(a.n_kv) * q4_tile_bytes(D));
    code[n] = *reinterpret_cast<const uint32_t*>(tile + q4_code_at<D>(is_v, k, c));
    s8[n] = tile[q4_scale_at<D>(is_v, k, c >> 1)];
  }
  const long long stride = is_v ? a.v_stride : a.k_stride;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? a.v_out : a.k_out) + t0 * stride + h * D + c * 8;
  const float scale = is_v ? a.v_scale : a.k_scale;
#pragma unroll
  for (int n = 0; n < U; ++n)
    if (slot[n] >= 0) *reinterpret_cast<uint4*>(dst + n * g.rows * stride) = q4_to_bf16(code[n], s8[n], scale);
}

// U = 4 tokens a thread where that still gives every SM four CTAs, else one
template <typename K4, typename K1>
int launch(K4 four, K1 one, const CacheQ4Args& a, cudaStream_t s) {
  Shape g{};
  g.chunks = a.n_kv * (a.head_dim / 8);
  int threads = g.chunks;  // the least number of whole rows that is a number of whole warps (chunks is a multiple of 8)
  while (threads % 32) threads += g.chunks;
  if (threads <= kMaxThreads) {
    while (threads < 256 && threads * 2 <= kMaxThreads) threads *= 2;
    g.rows = threads / g.chunks;
    g.parts = 1;
  } else {
    threads = 256;
    g.rows = 1;
    g.parts = (g.chunks + threads - 1) / threads;
  }
  if (g.parts > 32767) return cudaErrorInvalidValue;
  const long long ctas = (static_cast<long long>(a.T) + g.rows - 1) / g.rows, ctas4 = (ctas + 3) / 4;
  const bool u4 = ctas4 * 2 * g.parts >= 4LL * num_sms();
  const dim3 grid(static_cast<unsigned>(u4 ? ctas4 : ctas), 2 * g.parts);
  return u4 ? launch_kernel(four, grid, dim3(threads), 0, s, false, a, g)
            : launch_kernel(one, grid, dim3(threads), 0, s, false, a, g);
}

}  // namespace

int kv_write_q4_launch(const CacheQ4Args& a, cudaStream_t s) {
  if (a.T <= 0) return 0;
  return a.head_dim == 128 ? launch(k_kv_write_q4<128, 4>, k_kv_write_q4<128, 1>, a, s)
                           : launch(k_kv_write_q4<64, 4>, k_kv_write_q4<64, 1>, a, s);
}

int kv_read_q4_launch(const CacheQ4Args& a, cudaStream_t s) {
  if (a.T <= 0) return 0;
  return a.head_dim == 128 ? launch(k_kv_read_q4<128, 4>, k_kv_read_q4<128, 1>, a, s)
                           : launch(k_kv_read_q4<64, 4>, k_kv_read_q4<64, 1>, a, s);
}

}  // namespace llama
