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
// Both move 2 + 9/16 bytes an element.  Reading is bound by HBM (131072 tokens x 8
// heads x 128: 109 us, 6.3 TB/s, 93% of the copy rate), writing by its 98
// instructions for 8 elements of 32 lanes as well (32768 tokens: 33 us, 5.2 TB/s,
// the issue slots 73% and the ALU pipe 64% busy).  A thread takes chunks of 8
// elements (16 bytes of bf16, 4 of codes) of U tokens, always the same chunk of the
// row, with all its loads in flight; a warp's bf16 accesses are contiguous, two lanes
// share a scale.  A CTA has a whole number of rows (or a part of one) in its threads,
// so that one division finds a thread's place.  The writing CTAs stay and fetch their
// next tokens while they quantise (one after the other they took 39 us, a third of
// it waiting for their rows; reading has too little to do between its loads and
// stores to gain from it).
#include "cache_rows.h"
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q4.cuh"

namespace llama {

namespace {

// This thread's chunk c of head h.
struct Place : RowPlace {
  int h, c;
};

// v, known to be the same in every lane of the warp if WHOLE
template <bool WHOLE>
__device__ __forceinline__ int warp_value(int v) {
  return WHOLE ? __shfl_sync(0xffffffffu, v, 0) : v;
}

// WHOLE: g.whole
template <int D, int U, bool WHOLE>
__device__ __forceinline__ Place place(const RowShape& g) {
  constexpr int C = D / 8;
  const int row = warp_value<WHOLE>(threadIdx.x / g.chunks);
  Place x{row_place(g, U, blockIdx.x, blockIdx.y >> 1, blockDim.x, threadIdx.x, row), 0, 0};
  if (WHOLE) x.there = true;
  x.h = x.at / C;
  x.c = x.at % C;
  return x;
}

// token t0 + n rows, or the last one
__device__ __forceinline__ uint32_t token(const CacheQ4Args& a, const RowShape& g, const Place& x, int n) {
  return min(x.t0 + n * g.rows, static_cast<uint32_t>(a.T) - 1);
}

// the slots of this thread's tokens; -1 where there is nothing to do
template <int U, bool WHOLE>
__device__ __forceinline__ void load_slots(const CacheQ4Args& a, const RowShape& g, const Place& x, bool reports,
                                           int (&slot)[U]) {
  bool past = false;
#pragma unroll
  for (int n = 0; n < U; ++n) slot[n] = a.slots[token(a, g, x, n)];
#pragma unroll
  for (int n = 0; n < U; ++n) {
    slot[n] = warp_value<WHOLE>(slot[n]);
    const bool over = slot[n] >= a.num_blocks * kQ4Block;
    past |= over;
    if (over || x.t0 + n * g.rows >= static_cast<uint32_t>(a.T) || (!WHOLE && !x.there)) slot[n] = -1;
  }
  if (past && reports) report_error(a.err, kErrGuard, kWhereSlot);
}

// What depends on the chunk alone in the places of its codes and its scale, and the step from tile to tile.
template <int D, bool V>
struct Bytes {
  int code, scale;
  __device__ __forceinline__ explicit Bytes(int c)
      : code(q4_code_at<D>(V, 0, c)), scale(q4_scale_at<D>(V, 0, c >> 1)) {}
  __device__ __forceinline__ int code_at(int k) const { return code + q4_code_at<D>(V, k, 0); }
  __device__ __forceinline__ int scale_at(int k) const { return scale + q4_scale_at<D>(V, k, 0) - 8 * D; }
};

// The signs of 8 bf16, two to a word, at bit 3 of 8 nibbles: what rounds to zero keeps its sign, which the sum with
// kSnap drops (taking the codes of absolute values and putting eight signs back cost 16 instructions more).
__device__ __forceinline__ uint32_t signs(const uint32_t (&w)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x7351), b = __byte_perm(w[2], w[3], 0x7351);  // top bytes: low halves', high
  const uint32_t lo = __byte_perm(a, b, 0x5410), hi = __byte_perm(a, b, 0x7632);
  return ((lo >> 4) & 0x08080808u) | (hi & 0x80808080u);
}

// Where the tokens of a thread go: the offset of a token's codes (of chunk 0, head 0) and the way from there to the
// scales, -1 where there is nothing to do.  If the tokens are the warp's (WHOLE), lane n finds the place of token n and
// the others take it from there.
template <int D, int U, bool WHOLE, bool V>
struct Spots {
  int slot[WHOLE ? 1 : U];

  __device__ __forceinline__ void load(const CacheQ4Args& a, const RowShape& g, const Place& x, bool reports) {
    if constexpr (WHOLE) {
      const int n = threadIdx.x % U;
      slot[0] = a.slots[token(a, g, x, n)];
      const bool over = slot[0] >= a.num_blocks * kQ4Block;
      if (over && reports) report_error(a.err, kErrGuard, kWhereSlot);
      if (over || x.t0 + n * g.rows >= static_cast<uint32_t>(a.T)) slot[0] = -1;
    } else {
      load_slots<U, false>(a, g, x, reports, slot);
    }
  }
  struct Spot {
    size_t code;
    int scale;
  };
  // (of this thread's token n; WHOLE: of the token that is the lane's, for all n)
  __device__ __forceinline__ Spot find(int n, uint32_t block_bytes) const {
    const int s = slot[WHOLE ? 0 : n], k = s & 15;
    Spot y;
    y.code = static_cast<size_t>(static_cast<uint32_t>(s) >> 4) * block_bytes + q4_code_at<D>(V, k, 0);
    y.scale = s < 0 ? -1 : q4_scale_at<D>(V, k, 0) - q4_code_at<D>(V, k, 0) + kBias;
    return y;
  }
  static constexpr int kBias = 16 * D;  // (keeps the way to the scales positive)
  static __device__ __forceinline__ Spot from(const Spot& mine, int n) {
    Spot y;
    y.code = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(mine.code), n);
    y.scale = __shfl_sync(0xffffffffu, mine.scale, n);
    return y;
  }
};

template <int D, int U, bool WHOLE, bool V>
__device__ __forceinline__ void write_rows(const CacheQ4Args& a, const RowShape& g) {
  Place x = place<D, U, WHOLE>(g);
  const long long stride = V ? a.v_stride : a.k_stride;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(V ? a.v : a.k) + x.h * D + x.c * 8;
  constexpr int C = D / 8;
  const bool reports = !V && x.there && x.h * C + x.c == (WHOLE ? static_cast<int>(threadIdx.x & 31) : 0);
  const uint32_t step = row_step(g, U, gridDim.x);
  const float inv_g = V ? a.inv_v_scale : a.inv_k_scale;
  using To = Spots<D, U, WHOLE, V>;
  // this chunk's codes and scale in the tile of token 0 of block 0 (the tokens' own part is added to them)
  uint8_t* codes = static_cast<uint8_t*>(V ? a.v_cache : a.k_cache) + static_cast<size_t>(x.h) * q4_tile_bytes(D) +
                   q4_code_at<D>(V, 0, x.c);
  const int to_scale = q4_scale_at<D>(V, 0, x.c >> 1) - q4_scale_at<D>(V, 0, 0) - q4_code_at<D>(V, 0, x.c) - To::kBias;
  const uint32_t block_bytes = static_cast<uint32_t>(a.n_kv) * q4_tile_bytes(D);
  uint4 next[U];
  To to_next;
#pragma unroll
  for (int n = 0; n < U; ++n)  // before the slots are known: every row may be read
    next[n] = *reinterpret_cast<const uint4*>(src + token(a, g, x, n) * stride);
  to_next.load(a, g, x, reports);
  for (bool more = true; more;) {
    uint4 u[U];
    const To to = to_next;
#pragma unroll
    for (int n = 0; n < U; ++n) u[n] = next[n];
    more = row_more(x, a.T, step);
    x.cta += step;
    x.t0 += step;
    if (more) {  // on their way while these are quantised
#pragma unroll
      for (int n = 0; n < U; ++n) next[n] = *reinterpret_cast<const uint4*>(src + token(a, g, x, n) * stride);
      to_next.load(a, g, x, reports);
    }
    float top[U];
    bool nan = false;
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&u[n]);
      __nv_bfloat162 m = __hmax2_nan(__habs2(w[0]), __habs2(w[1]));
      m = __hmax2_nan(m, __hmax2_nan(__habs2(w[2]), __habs2(w[3])));
      top[n] = __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
      nan |= top[n] != top[n];
    }
    if (nan) {  // rare: a NaN counts as zero
#pragma unroll
      for (int n = 0; n < U; ++n) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&u[n]);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((w[e] & 0x7FFFu) > 0x7F80u) w[e] &= 0xFFFF0000u;
          if ((w[e] & 0x7FFF0000u) > 0x7F800000u) w[e] &= 0xFFFFu;
          m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
        }
        top[n] = m;
      }
    }
    __syncwarp();
    const typename To::Spot mine = to.find(0, block_bytes);
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const float amax = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], 1));  // the group's other half: the next lane
      const uint32_t s8 = f32_to_e4m3_by_f16(amax * (inv_g * (1.f / 6.f)));
      const float inv = s8 == 0 ? 0.f : __fdividef(inv_g, f16_lo(e4m3x2_to_f16(s8)));
      constexpr float kSnap = 1.5f * 1024.f;  // sums with it are multiples of 2^-13 (|x / s| below 2^9; beyond, saturated)
      const uint64_t inv2 = f2_pack(inv, inv), up = f2_pack(kSnap, kSnap), down = f2_pack(-kSnap, -kSnap);
      const uint32_t w[4] = {u[n].x, u[n].y, u[n].z, u[n].w};
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        f2_unpack(f2_add(f2_fma(f2_pack(bf16_lo(w[e]), bf16_hi(w[e])), inv2, up), down), y[2 * e], y[2 * e + 1]);
      const uint32_t code = s8 == 0 ? 0u : (f32x8_to_e2m1(y) & 0x77777777u) | signs(w);
      const uint32_t pair = __shfl_down_sync(0xffffffffu, s8, 2);  // the next group's scale (K stores two at D = 128)
      const typename To::Spot spot = WHOLE ? To::from(mine, n) : n == 0 ? mine : to.find(n, block_bytes);
      if (spot.scale >= 0) {
        uint8_t* at = codes + spot.code;
        *reinterpret_cast<uint32_t*>(at) = code;
        at += to_scale + spot.scale;
        if (D == 128 && !V) {
          if ((x.c & 3) == 0) *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(s8 | (pair << 8));
        } else {
          if ((x.c & 1) == 0) *at = static_cast<uint8_t>(s8);
        }
      }
    }
  }
}

template <int D, int U, bool WHOLE, bool V>
__device__ __forceinline__ void read_rows(const CacheQ4Args& a, const RowShape& g) {
  const Place x = place<D, U, WHOLE>(g);
  int slot[U];
  load_slots<U, WHOLE>(a, g, x, !V && x.h == 0 && x.c == 0 && x.there, slot);
  const Bytes<D, V> at(x.c);
  const uint8_t* cache =
      static_cast<const uint8_t*>(V ? a.v_cache : a.k_cache) + static_cast<size_t>(x.h) * q4_tile_bytes(D);
  const uint32_t block_bytes = static_cast<uint32_t>(a.n_kv) * q4_tile_bytes(D);
  uint32_t code[U], s8[U];
#pragma unroll
  for (int n = 0; n < U; ++n) {
    const uint32_t from = max(slot[n], 0);  // (a skipped row reads slot 0's bytes and stores nothing)
    const uint8_t* tile = cache + static_cast<size_t>(from >> 4) * block_bytes;
    code[n] = *reinterpret_cast<const uint32_t*>(tile + at.code_at(from & 15));
    s8[n] = tile[at.scale_at(from & 15)];
  }
  const long long stride = V ? a.v_stride : a.k_stride;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(V ? a.v_out : a.k_out) + x.h * D + x.c * 8;
  const float scale = V ? a.v_scale : a.k_scale;
#pragma unroll
  for (int n = 0; n < U; ++n) {
    const uint4 v = q4_to_bf16(code[n], s8[n], scale);
    if (slot[n] >= 0) *reinterpret_cast<uint4*>(dst + token(a, g, x, n) * stride) = v;
  }
}

template <int D, int U, bool WHOLE>
__global__ void __launch_bounds__(kMaxRowThreads, WHOLE ? 2 : 1) k_kv_write_q4(const CacheQ4Args a, const RowShape g) {
  pdl_wait();
  if (blockIdx.y & 1)
    write_rows<D, U, WHOLE, true>(a, g);
  else
    write_rows<D, U, WHOLE, false>(a, g);
}

template <int D, int U, bool WHOLE>
__global__ void __launch_bounds__(kMaxRowThreads) k_kv_read_q4(const CacheQ4Args a, const RowShape g) {
  pdl_wait();
  if (blockIdx.y & 1)
    read_rows<D, U, WHOLE, true>(a, g);
  else
    read_rows<D, U, WHOLE, false>(a, g);
}

using Kernel = void (*)(const CacheQ4Args, const RowShape);

int launch(Kernel four, Kernel one, Kernel four_whole, Kernel one_whole, bool loops, const CacheQ4Args& a, cudaStream_t s) {
  const RowShape g = row_shape(a.n_kv, a.head_dim);
  if (g.parts > 32767) return cudaErrorInvalidValue;
  const RowGrid r = row_grid(g, a.T, num_sms(), loops);
  const dim3 grid(static_cast<unsigned>(r.ctas), 2 * g.parts);
  const bool u4 = r.u == 4;
  return launch_kernel(g.whole ? (u4 ? four_whole : one_whole) : (u4 ? four : one), grid, dim3(g.threads), 0, s, true, a,
                       g);
}

}  // namespace

int kv_write_q4_launch(const CacheQ4Args& a, cudaStream_t s) {
  if (a.T <= 0) return 0;
  return a.head_dim == 128 ? launch(k_kv_write_q4<128, 4, false>, k_kv_write_q4<128, 1, false>,
                                    k_kv_write_q4<128, 4, true>, k_kv_write_q4<128, 1, true>, true, a, s)
                           : launch(k_kv_write_q4<64, 4, false>, k_kv_write_q4<64, 1, false>,
                                    k_kv_write_q4<64, 4, true>, k_kv_write_q4<64, 1, true>, true, a, s);
}

int kv_read_q4_launch(const CacheQ4Args& a, cudaStream_t s) {
  if (a.T <= 0) return 0;
  return a.head_dim == 128 ? launch(k_kv_read_q4<128, 4, false>, k_kv_read_q4<128, 1, false>,
                                    k_kv_read_q4<128, 4, true>, k_kv_read_q4<128, 1, true>, false, a, s)
                           : launch(k_kv_read_q4<64, 4, false>, k_kv_read_q4<64, 1, false>,
                                    k_kv_read_q4<64, 4, true>, k_kv_read_q4<64, 1, true>, false, a, s);
}

}  // namespace llama
