// Products of microscaled matrices (the formats are in mx.cuh) on the block-scaled
// tensor-core instructions:
//   y = alpha x w^T                                    (llama_linear_mx)
//   a = silu(alpha_0 x w_gate^T) * (alpha_1 x w_up^T)  (llama_gate_up_silu_mx)
// x [M, K] and w [N, K] are codes with scales; sums are fp32 in tensor memory, and
// each result is rounded once: to bf16, or with its row's neighbours to the
// codes and scales of a microscaled matrix that the next product reads.
//
// Two kernels: whole tiles of 256 x 256 on SM pairs (k_gemm_mx_pair), and for few tiles ones of 128 x 128 with K split over a
// cluster (k_gemm_mx_split).  In both a stage of the operand ring holds 128 bytes of every row (256 e2m1 or 128 e4m3 elements,
// one swizzle row) and the scale tiles that belong to them; the issuing thread copies these into tensor memory and then issues
// the stage's four MMAs (gate_up of few tiles: eight), in order.  Up to twenty instructions a stage come from that thread, so
// everything they take is computed under control flow that is the warp's (warp_same, elect_one): their operands stay in uniform
// registers, where moving them there from lane registers cost some 50 cycles for each (70B gate_up, 4128 rows, nvfp4: 1.18 ms
// and then 0.59).
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "mx.cuh"

namespace llama {

namespace {

constexpr int BM = 128;
constexpr int kRowBytes = 128;    // of every row of a stage
constexpr int kThreads = 192;     // warp 0 copies, warp 1 MMAs, warps 2-5 epilogue
constexpr int kTmemCols = 512;
constexpr int kMaxStages = 8;
constexpr int kMaxSmemBytes = 232448;              // the opt-in limit per CTA (227 KB)
constexpr int kRingBudget = kMaxSmemBytes - 2048;  // the rest: barriers, alignment slack

enum MxEpilogue : int { kMxBf16 = 0, kMxF32 = 1, kMxSilu = 2, kMxSiluNvfp4 = 3, kMxSiluFp4 = 4, kMxSiluFp8 = 5 };

__host__ __device__ constexpr bool is_silu(int epi) { return epi >= kMxSilu; }
// the format that the output is quantised to; 0: none
__host__ __device__ constexpr int out_fmt(int epi) {
  return epi == kMxSiluNvfp4 ? kMxNvfp4 : epi == kMxSiluFp4 ? kMxFp4 : epi == kMxSiluFp8 ? kMxFp8 : 0;
}

// The tensor cores cut a sum's low bits at every step, always towards zero, so that the error grows with the steps and faster
// than that of sums rounded to nearest (against 64 bits, rms over that of the results, fp8 on SM pairs in one chain and then
// fp32: K = 2048 1.1e-7 and 0.6e-7, 8192 4.8e-7 and 1.2e-7, 28672 24e-7 and 2.7e-7; terms of one sign 190e-7 at 28672).  Results
// in fp32, and those that are quantised from it, are therefore sums of chains of no more than so many stages, which are added
// in fp32: 1.3e-7 at K = 28672, one sign 5e-7.  Few sums of 4-bit products are cut at all: exact for rows whose scales are near
// one another; where those of x spread over some ten binades, K = 28672, in one chain 39e-7 to 45e-7, in chains twice as long
// as fp8's 7e-7 to 11e-7, fp32 10e-7 to 12e-7.
template <int FMT>
constexpr int kChainStages = FMT == kMxFp8 ? 16 : 32;

// Results in bf16 round to 2^-8 of themselves.  Terms of one sign put a chain of n stages, 4 n steps of half a last place each,
// off by 2 n 2^-24: SM pairs take bf16 sums in one chain of up to 1024 stages (2^-13; longer ones are left to the other
// kernel), which takes 4-bit ones in chains of 256.
constexpr int kPairBf16Stages = 1024, kSplitBf16Stages = 256;
__host__ __device__ constexpr bool is_bf16(int epi) { return epi == kMxBf16 || epi == kMxSilu; }

// What a format makes of a stage.
template <int FMT>
struct Stage {
  static constexpr int kBits = mx_bits(FMT);
  static constexpr int kElems = kRowBytes * 8 / kBits;
  static constexpr int kTiles = kElems / mx_group(FMT) / kMxTileGroups;  // scale tiles of 128 rows
  static constexpr int kStepElems = 256 / kBits;                        // an MMA's part of K: 32 bytes of a row
  static constexpr int kSteps = kElems / kStepElems;
  static constexpr int kStepScales = kStepElems / mx_group(FMT);  // scales of a row in an MMA: 4, 2 or 1
  static constexpr int kPerTile = kMxTileGroups / kStepScales;    // MMAs that take their scales from one tile
  static constexpr bool kE8m0 = FMT != kMxNvfp4;
};

// Tensor maps: codes in boxes of up to 128 rows x 128 bytes, swizzled; for pairs also the scales, in boxes of a stage's tiles
// of 128 rows, as 8-byte elements, and the results in boxes of 32 rows x 128 bytes (4-bit codes: 64), swizzled.  What lies
// outside reads as zero and is not written.
struct MxMaps {
  CUtensorMap x, x_scales, w[2], w_scales[2], out;
};
constexpr int kScaleElems = kMxTileBytes / 8;  // of a scale tile

template <int EPI>
__device__ __forceinline__ void prefetch_maps(const MxMaps& m) {
  tma_prefetch_desc(&m.x);
  tma_prefetch_desc(&m.x_scales);
#pragma unroll
  for (int i = 0; i < (is_silu(EPI) ? 2 : 1); ++i) {
    tma_prefetch_desc(&m.w[i]);
    tma_prefetch_desc(&m.w_scales[i]);
  }
}

struct MxGemmParams {
  int M, N, kb;    // kb: stages along K
  int last_steps;  // MMAs of the last one
  // SM pairs: a tile's sums are of `chains` chains of chain_len stages, the first chain_more of them one longer
  int chains, chain_len, chain_more;
  int tiles_m, tiles_n, tiles, group_m;
  // few tiles: the ring, and its rows of x, a multiple of 32 (the MMA reads bytes of w as the rows to 128, whose results are
  // never looked at)
  int stages, a_rows;
  int meta_at;  // the barriers' place, from the ring's begin
  int recv_at;  // the receive buffer's place from the ring's begin: 0, over the ring, or behind it
  int ktiles;   // scale tiles along K
  const uint8_t *x_scales, *w_scales[2];
  float alpha[2];
  void* out;
  bool sectors;  // rows of out begin on 32 bytes
  uint8_t* out_scales;
  int out_ktiles;
  float out_inv_g, out_sixth;
  int* err;
};

__device__ __forceinline__ void tile_coords(const MxGemmParams& p, int tile, int& tm, int& tn) {
  const int group = p.group_m * p.tiles_n;
  const int g = tile / group;
  const int first_m = g * p.group_m;
  const int gm = min(p.tiles_m - first_m, p.group_m);
  const int r = tile - g * group;
  tm = first_m + r % gm;
  tn = r / gm;
}

// Tensor memory of an SM pair's CTA: two accumulators of 256 columns that share 64, then the scales of a stage.
template <int FMT>
struct PairTmem {
  static constexpr int kAcc = 192;  // from the first accumulator to the second
  static constexpr int kSa = kAcc + 256, kSb = kSa + 4 * Stage<FMT>::kTiles;
  static_assert(kSb + 8 * Stage<FMT>::kTiles <= kTmemCols, "tensor memory");
};

// ---------------------------------------------------------------------------
// Epilogue: 32 output columns of a thread's row at a time.
// ---------------------------------------------------------------------------
// 32 bytes of a thread: a whole sector of L2, which results leave first (they are not read again here).  Half sectors, 16
// bytes each, made a 256 x 256 tile of bf16 results wait 2.5 us longer.
__device__ __forceinline__ void store32(void* dst, const uint32_t* w) {
  asm volatile("st.global.L2::cache_hint.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(dst), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(policy_evict_first())
               : "memory");
}

// W words (a multiple of 8), 16-byte aligned; sectors: 32-byte aligned
template <int W>
__device__ __forceinline__ void store_words32(void* dst, const uint32_t (&w)[W], bool sectors) {
  uint4* d = static_cast<uint4*>(dst);
#pragma unroll
  for (int i = 0; i < W / 8; ++i) {
    if (sectors) {
      store32(d + 2 * i, w + 8 * i);
    } else {
      d[2 * i] = make_uint4(w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3]);
      d[2 * i + 1] = make_uint4(w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]);
    }
  }
}

// 32 results, columns n .. n + 31 of a row, to codes; `words` collects the scale words of its 128 columns.
template <int OF>
__device__ __forceinline__ void codes32(const MxGemmParams& p, int n, const float (&v)[32], uint32_t (&w)[mx_bits(OF)],
                                        uint32_t (&words)[2]) {
  constexpr int G = mx_group(OF), kGroups = 32 / G;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < G; ++e) top = max(top, abs_bits(v[g * G + e]));
    const MxScale s = mx_scale<OF, false>(top, p.out_sixth, p.out_inv_g);
    const int at = n % 128 / G + g;  // among the groups of 128 columns
    words[0] |= at < 4 ? s.byte << (at * 8) : 0u;
    words[1] |= at < 4 ? 0u : s.byte << (at * 8 - 32);
#pragma unroll
    for (int c = 0; c < G / 8; ++c) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = v[g * G + c * 8 + e];
      const uint2 u = mx_codes8<OF, false>(x, s.factor);
      const int i = g * (G / 8) + c;
      if constexpr (OF == kMxFp8) {
        w[2 * i] = u.x;
        w[2 * i + 1] = u.y;
      } else {
        w[i] = u.x;
      }
    }
  }
}

// g / (1 + exp(-g)), by the hardware's reciprocal and one Newton step to the last place.  Below -87 it is below 2^-118, and
// -87 stands for g, so that the reciprocal is a normal number.  (A NaN stays one.)
__device__ __forceinline__ float silu(float g) {
  g = g < -87.f ? -87.f : g;
  const float d = 1.0f + expf(-g);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return g * fmaf(r, fmaf(-d, r, 1.0f), r);
}

// 32 results from the accumulators v (silu: gate) and up, into v
template <int EPI>
__device__ __forceinline__ void results32(const MxGemmParams& p, float (&v)[32], const float* up) {
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = is_silu(EPI) ? silu(v[e] * p.alpha[0]) * (up[e] * p.alpha[1]) : v[e] * p.alpha[0];
}

// 32 results of a row at output column n, from the accumulators v (silu: gate) and up, stored by their thread
template <int EPI>
__device__ __forceinline__ void finish32(const MxGemmParams& p, int row, int n, float (&v)[32], const float* up,
                                         uint32_t (&words)[2]) {
  if (row >= p.M || n >= p.N) return;
  results32<EPI>(p, v, up);
  constexpr int OF = out_fmt(EPI);
  if constexpr (OF != 0) {
    uint32_t w[mx_bits(OF)];
    codes32<OF>(p, n, v, w, words);
    uint8_t* dst = static_cast<uint8_t*>(p.out) + static_cast<size_t>(row) * (p.N / 8 * mx_bits(OF)) + n / 8 * mx_bits(OF);
    if constexpr (OF == kMxFp8) store_words32(dst, w, p.sectors);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    constexpr bool kF32 = EPI == kMxF32;
    uint8_t* o = static_cast<uint8_t*>(p.out) + (static_cast<size_t>(row) * p.N + n) * (kF32 ? 4 : 2);
    uint32_t w[kF32 ? 32 : 16];
#pragma unroll
    for (int e = 0; e < (kF32 ? 32 : 16); ++e) w[e] = kF32 ? __float_as_uint(v[e]) : pack_bf16x2(v[2 * e % 32], v[(2 * e + 1) % 32]);
    if (n + 32 <= p.N) {
      store_words32(o, w, p.sectors);
    } else {  // 8, 16 or 24 columns are left
#pragma unroll
      for (int q = 0; q < (kF32 ? 8 : 4); ++q)
        if (n + q * (kF32 ? 4 : 8) < p.N)
          reinterpret_cast<uint4*>(o)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
  }
}

// A warp's results on their way to memory: 32 rows of up to 128 bytes in shared memory, swizzled as the tensor map of the
// output says, and from there by a tiled store, which writes whole lines and leaves out what lies past the last row or
// column (threads storing their own rows, 32 lines an instruction, held a 256 x 256 tile's epilogue for twice as long).  With
// two buffers one is filled while the other is read.
template <int BUFS>
struct OutBoxes {
  const CUtensorMap* map;
  uint32_t buf;  // this warp's buffers
  int row0;      // of the warp
  int next;
  // nanoseconds between a tile's boxes where another tile's MMAs run meanwhile: the results of a tile at once crowd out the
  // copies of operands (8192 x 8192, nvfp4, 32768 rows: 19.3 thousand cycles of MMAs a tile instead of 18.4)
  int pace;
  static constexpr int kBytes = 32 * 128;

  __device__ __forceinline__ uint32_t begin() {
    if ((threadIdx.x & 31) == 0) bulk_wait_read<BUFS - 1>();
    __syncwarp();
    return buf + (next & (BUFS - 1)) * kBytes;
  }
  // 16 bytes of the lane's row; rows of 128, 64 or 32 bytes
  template <int ROW>
  __device__ __forceinline__ static void put(uint32_t box, int chunk, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const int lane = threadIdx.x & 31, at = ROW == 128 ? lane & 7 : ROW == 64 ? (lane >> 1) & 3 : (lane >> 2) & 1;
    st_shared_v4(box + lane * ROW + ((chunk ^ at) << 4), a, b, c, d);
  }
  // x: the box's first element in the output's rows
  __device__ __forceinline__ void end(uint32_t box, int x) {
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      tma_store_2d(map, box, x, row0, policy_evict_first());
      bulk_commit();
    }
    ++next;
  }
};

// bf16 results: the whole 256-column tile of a warp's 32 rows, from the accumulator at taddr, 64 results of a row at a time.
// release() is called once the 64 columns shared with the other accumulator (this one's last if it is the first, its first
// if the second) are in registers.
template <int EPI, class Release>
__device__ __forceinline__ void epilogue_tile(const MxGemmParams& p, OutBoxes<2>& boxes, int tn, uint32_t taddr, int acc,
                                              const Release& release) {
  const bool any = boxes.row0 < p.M;  // a warp whose rows are all past M has nothing to do
  float keep[2][32];
  const int shared = acc == 0 ? 192 : 0;
  if (any) {
    tmem_ld32(taddr + shared, keep[0]);
    tmem_ld32(taddr + shared + 32, keep[1]);
  }
  release();
  if (!any) return;
  auto store = [&](int n, const float (&a)[32], const float (&b)[32]) {
    const uint32_t box = boxes.begin();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      boxes.put<128>(box, q, pack_bf16x2(a[8 * q], a[8 * q + 1]), pack_bf16x2(a[8 * q + 2], a[8 * q + 3]),
                     pack_bf16x2(a[8 * q + 4], a[8 * q + 5]), pack_bf16x2(a[8 * q + 6], a[8 * q + 7]));
      boxes.put<128>(box, 4 + q, pack_bf16x2(b[8 * q], b[8 * q + 1]), pack_bf16x2(b[8 * q + 2], b[8 * q + 3]),
                     pack_bf16x2(b[8 * q + 4], b[8 * q + 5]), pack_bf16x2(b[8 * q + 6], b[8 * q + 7]));
    }
    boxes.end(box, n);
  };
  if constexpr (is_silu(EPI)) {
    const int n0 = tn * 128, first = acc == 0 ? 64 : 0;  // the half whose up (gate) columns are kept
    float other[2][32];
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const int c = h == 0 ? first : 64 - first;
      if (n0 + c >= p.N) continue;
      if (h == 1 && boxes.pace > 0) __nanosleep(boxes.pace);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (h == 1) tmem_ld32(taddr + c + 32 * i + (acc == 0 ? 128 : 0), keep[i]);
        tmem_ld32(taddr + c + 32 * i + (acc == 0 ? 0 : 128), other[i]);
        // (gate, up) = (other, keep) or (keep, other)
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float g = acc == 0 ? other[i][e] : keep[i][e], u = acc == 0 ? keep[i][e] : other[i][e];
          other[i][e] = silu(g * p.alpha[0]) * (u * p.alpha[1]);
        }
      }
      store(n0 + c, other[0], other[1]);
    }
  } else {
    const int n0 = tn * 256;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int c = i == 0 ? shared : acc == 0 ? 64 * (i - 1) : 64 * i;
      if (n0 + c >= p.N) continue;
      if (i > 0) {
        if (boxes.pace > 0) __nanosleep(boxes.pace);
        tmem_ld32(taddr + c, keep[0]);
        tmem_ld32(taddr + c + 32, keep[1]);
      }
      results32<EPI>(p, keep[0], nullptr);
      results32<EPI>(p, keep[1], nullptr);
      store(n0 + c, keep[0], keep[1]);
    }
  }
}

// A warp's part of a 256 x 256 tile: 32 rows and half of the columns in registers, a row a thread, 64 neighbours twice: of
// gate and the same of up, or (no silu) all neighbours.
template <int EPI>
__device__ __forceinline__ int part_col(int half, int j) {
  return is_silu(EPI) ? 64 * half + 128 * j : 128 * half + 64 * j;
}

// v = the accumulator at taddr, or (not the first chain of the tile) v += it.  release() is called once the columns shared
// with the other accumulator are in registers: the last 64 of the first one, which only the second half has, as j = 1; the
// first 64 of the second, which the first half has, as j = 0.
template <int EPI, class Release>
__device__ __forceinline__ void add_chain(float (&v)[2][64], uint32_t taddr, int acc, int half, bool first,
                                          const Release& release) {
  auto add = [&](float (&c)[64], int j) {
    const uint32_t at = taddr + part_col<EPI>(half, j);
    if (first) {
      tmem_ld64(at, c);
      return;
    }
#pragma unroll
    for (int h = 0; h < 64; h += 16) {
      float t[16];
      tmem_ld16(at + h, t);
#pragma unroll
      for (int e = 0; e < 16; ++e) c[h + e] += t[e];
    }
  };
  if (half == acc) release();
  if (acc == 0) {
    add(v[1], 1);
    if (half != acc) release();
    add(v[0], 0);
  } else {
    add(v[0], 0);
    if (half != acc) release();
    add(v[1], 1);
  }
}

__device__ __forceinline__ float (&half_of(float (&v)[64], int i))[32] { return reinterpret_cast<float(&)[32]>(v[32 * i]); }

// fp32 or quantised results from a warp's sums, stored as boxes of 32 rows and 32 outputs, or 64.
template <int EPI>
__device__ __forceinline__ void finish_tile(const MxGemmParams& p, OutBoxes<1>& boxes, int tn, int half, float (&v)[2][64]) {
  constexpr int OF = out_fmt(EPI);
  if constexpr (EPI == kMxF32) {
    const int n0 = tn * 256 + 128 * half;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n0 + 32 * i >= p.N) break;
      if (i > 0 && boxes.pace > 0) __nanosleep(boxes.pace);
      float(&r)[32] = half_of(v[i / 2], i % 2);
      results32<EPI>(p, r, nullptr);
      const uint32_t box = boxes.begin();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        boxes.put<128>(box, q, __float_as_uint(r[4 * q]), __float_as_uint(r[4 * q + 1]), __float_as_uint(r[4 * q + 2]),
                       __float_as_uint(r[4 * q + 3]));
      boxes.end(box, n0 + 32 * i);
    }
  } else {
    constexpr int kChunks = mx_bits(OF) / 4;  // 16 bytes of 32 outputs' codes
    const int n0 = tn * 128 + 64 * half, row = boxes.row0 + (threadIdx.x & 31);
    uint32_t words[2] = {0, 0};
    if (n0 < p.N) {
      const uint32_t box = boxes.begin();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (n0 + 32 * i >= p.N) break;
        float(&r)[32] = half_of(v[0], i);
        results32<EPI>(p, r, half_of(v[1], i));
        uint32_t w[mx_bits(OF)];
        codes32<OF>(p, n0 + 32 * i, r, w, words);
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
          boxes.put<32 * kChunks>(box, i * kChunks + j, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      }
      boxes.end(box, n0 / 8 * mx_bits(OF));
    }
    if (row >= p.M) return;
    // the scales of the row's 64 outputs, a word or half of one, zeros past the last group
    if constexpr (OF == kMxNvfp4) {
      if (2 * tn + half < p.out_ktiles)
        *reinterpret_cast<uint32_t*>(p.out_scales + mx_scale_at(row, 2 * tn + half, p.out_ktiles)) = half ? words[1] : words[0];
    } else {
      *reinterpret_cast<uint16_t*>(p.out_scales + mx_scale_at(row, tn, p.out_ktiles) + 2 * half) =
          static_cast<uint16_t>(words[0] >> (16 * half));
    }
  }
}

// ---------------------------------------------------------------------------
// Persistent on SM pairs (2-CTA clusters): tiles of 256 x 256, MMAs with M = 256.  CTA r has rows 128 r .. of the tile's x
// and half of its columns of w (silu: gate on rank 0, up on rank 1) in its shared memory, the scales of its x rows and of
// all columns, and the accumulator of its rows, so that an SM loads 32 KB of codes where one alone loads 48.
// The tensor cores are what is busy (8192 cubed, nvfp4: 150 us, 7.3 PFLOP/s; 4096 x 8192 x 8192 under the profiler: 79% of the
// tensor pipe in nvfp4, 87% in fp8, seven waves of tiles of which the last is not full); in long runs the part is at its
// power limit (70B o_proj, 32768 rows, fp8: 1.20 ms at first, 1.35 over a second).
// Results in bf16 are taken from the accumulator 64 columns at a time by four warps.  For the others eight warps keep a tile's
// sums in registers, 128 columns of a row each, and add a chain's accumulator to them while the other one is filled, so that
// a chain more costs its hand-over, 0.35 us (4096 x 8192 x 8192, fp8 to fp32, four chains for one: 148 us and then 156; gate_up
// 4096 x 14336 x 4096, fp8 to fp8, two for one: 261 and 262), and a tile of few stages is done sooner than four warps finish
// it (gate_up 2004 x 16896 x 1280, nvfp4 to fp8: 61 us and then 43).
// Both CTAs' copies complete on rank 0's full barriers; one thread of rank 0 issues copies of scales and MMAs for both, and
// commits to both CTAs' barriers.
// ---------------------------------------------------------------------------
template <int FMT>
struct PairRing {
  static constexpr int kA = BM * kRowBytes, kB = 128 * kRowBytes;
  static constexpr int kSa = Stage<FMT>::kTiles * kMxTileBytes, kSb = 2 * kSa;
  static constexpr int kBytes = kA + kB + kSa + kSb;  // of a stage, a CTA
  static constexpr int kOut = 8 * OutBoxes<1>::kBytes;  // the epilogue warps' buffers: four of two, or eight of one
  static constexpr int kStages = (kRingBudget - kOut) / kBytes < kMaxStages ? (kRingBudget - kOut) / kBytes : kMaxStages;
  static constexpr int kSmem = kStages * kBytes + kOut + 2048;
};

constexpr int epilogue_warps(int epi) { return is_bf16(epi) ? 4 : 8; }
constexpr int pair_threads(int epi) { return 64 + 32 * epilogue_warps(epi); }

template <int FMT, int EPI>
__global__ void __launch_bounds__(pair_threads(EPI), 1)
    k_gemm_mx_pair(const __grid_constant__ MxMaps maps, const __grid_constant__ MxGemmParams p) {
  using S = Stage<FMT>;
  using R = PairRing<FMT>;
  using T = PairTmem<FMT>;
  constexpr int nst = R::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  const uint32_t out_buf = sbase + nst * (R::kA + R::kB), scales = out_buf + R::kOut;
  uint8_t* meta = smem_raw + pad + nst * R::kBytes + R::kOut;
  const uint32_t bar0 = smem_u32(meta);  // full[S], empty[S], tfull[2], tempty[2], drain
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meta + 8 * (2 * nst + 5));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (nst + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * nst + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * nst + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * nst + 4);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const uint32_t peer_abort = mapa_shared(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1);
  // this CTA and its peer stop waiting once either of them gives up
  auto give_up = [&]() {
    *abort_flag = 1;
    st_cluster_u32(peer_abort, 1u);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * epilogue_warps(EPI));  // of both CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_maps<EPI>(maps);
    tma_prefetch_desc(&maps.out);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist before either signals the other's
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait();
  const int npairs = static_cast<int>(gridDim.x) >> 1, first = static_cast<int>(blockIdx.x) >> 1;

  if (warp == 0) {
    // ---------------- copies (both CTAs) ----------------
    const uint64_t pol_a = policy_evict_last(), pol_b = policy_evict_first();
    int stage = 0;
    uint32_t phase = 0;
    long long used = 0;
    bool ok = true;
    for (int t = first; ok && t < p.tiles; t += npairs) {
      int tm, tn;
      tile_coords(p, t, tm, tn);
      const int xt = 2 * tm + rank;                          // this CTA's 128 rows of x
      const int w = is_silu(EPI) ? rank : 0;
      const int wt = is_silu(EPI) ? tn : 2 * tn + rank;      // and of w
      for (int kb = 0; kb < p.kb; ++kb) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t sa = sbase + stage * (R::kA + R::kB), sb = sa + R::kA;
          const uint32_t ssa = scales + stage * (R::kSa + R::kSb), ssb = ssa + R::kSa;
          const uint32_t fb = mapa_shared(full_bar(stage), 0);
          const int kx = kb * S::kTiles * kScaleElems;
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * R::kBytes);
          tma_load_2d_pair(sa, &maps.x, fb, kb * kRowBytes, xt * 128, pol_a);
          tma_load_2d_pair(sb, &maps.w[w], fb, kb * kRowBytes, wt * 128, pol_b);
          tma_load_2d_pair(ssa, &maps.x_scales, fb, kx, xt, pol_a);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            tma_load_2d_pair(ssb + i * R::kSa, &maps.w_scales[is_silu(EPI) ? i : 0], fb, kx, is_silu(EPI) ? tn : 2 * tn + i,
                             pol_b);
        }
        __syncwarp();
        ++used;
        if (++stage == nst) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0) pdl_trigger();
    if (!ok) {
      if (lane == 0) report_error(p.err, kErrTimeout, kWhereGemmProducer);
      give_up();
    }
    // rank 0's full barriers count both CTAs' bytes: after their last phases every copy has landed
    if (rank == 0)
      for (int s = 0; s < nst; ++s) {
        const long long uses = (used - s + nst - 1) / nst;
        if (uses > 0) mbar_wait(full_bar(s), static_cast<uint32_t>(uses - 1) & 1u, nullptr);
      }
  } else if (warp == 1) {
    // ---------------- MMAs (rank 0) ----------------
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_mx(2 * BM, 256, S::kBits, S::kE8m0);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      // the stages from kb to end, a tile's or (chains) a part of them, into an accumulator
      auto chain = [&](int kb, const int end) {
        if (!warp_same(mbar_wait(tempty_bar(acc ^ 1), acc ? acc_phase : acc_phase ^ 1u, abort_flag))) {
          ok = false;
          return;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * T::kAcc;
        for (const int begin = kb; kb < end; ++kb) {
          if (!warp_same(mbar_wait(full_bar(stage), phase, abort_flag))) {
            ok = false;
            return;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = sbase + stage * (R::kA + R::kB), sb = sa + R::kA;
            const uint32_t ssa = scales + stage * (R::kSa + R::kSb), ssb = ssa + R::kSa;
#pragma unroll
            for (int i = 0; i < S::kTiles; ++i) {
              tc_copy_scales<true>(tmem_base + T::kSa + 4 * i, smem_desc_scales(ssa + i * kMxTileBytes));
#pragma unroll
              for (int j = 0; j < 2; ++j)
                tc_copy_scales<true>(tmem_base + T::kSb + 8 * i + 4 * j, smem_desc_scales(ssb + j * R::kSa + i * kMxTileBytes));
            }
            const int steps = kb + 1 < p.kb ? S::kSteps : p.last_steps;
#pragma unroll
            for (int k = 0; k < S::kSteps; ++k) {
              if (k >= steps) break;
              const int i = k / S::kPerTile;
              tc_mma_mx<S::kBits, S::kStepScales, true>(d_tmem, smem_desc_sw128(sa + 32 * k), smem_desc_sw128(sb + 32 * k),
                                                        idesc_mx_scale(idesc, k % S::kPerTile * S::kStepScales),
                                                        tmem_base + T::kSa + 4 * i, tmem_base + T::kSb + 8 * i,
                                                        kb > begin || k > 0 ? 1u : 0u);
            }
            tc_commit_pair(empty_bar(stage), 3);
          }
          __syncwarp();
          if (++stage == nst) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (elect_one()) tc_commit_pair(tfull_bar(acc), 3);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      };
      for (int t = first; ok && t < p.tiles; t += npairs) {
        if constexpr (is_bf16(EPI)) {
          chain(0, p.kb);
        } else {
          for (int c = 0, kb = 0; ok && c < p.chains; ++c) {
            const int end = kb + p.chain_len + (c < p.chain_more ? 1 : 0);
            chain(kb, end);
            kb = end;
          }
        }
      }
      if (!ok) {
        if (lane == 0) report_error(p.err, kErrTimeout, kWhereGemmMma);
        give_up();
      }
      // completes in both CTAs once everything issued above has
      if (elect_one()) tc_commit_pair(drain_bar, 3);
      __syncwarp();
    }
    // no CTA frees tensor memory that the pair's MMAs may still write
    mbar_wait(drain_bar, 0, nullptr);
  } else {
    // ---------------- epilogue (both CTAs, their own rows) ----------------
    constexpr int kBufs = is_bf16(EPI) ? 2 : 1;
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tempty_lead = mapa_shared(tempty_bar(0), 0);
    OutBoxes<kBufs> boxes{&maps.out, out_buf + (warp - 2) * kBufs * OutBoxes<kBufs>::kBytes, 0, 0, 0};
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(tempty_lead + 8u * acc);
    };
    for (int t = first; ok && t < p.tiles; t += npairs) {
      int tm, tn;
      tile_coords(p, t, tm, tn);
      boxes.row0 = (2 * tm + rank) * BM + quad * 32;
      // (a stage's MMAs take some 300; fp32 results of 4096 x 8192 x 2048, fp8, whose tiles have 16 stages: 54.9 us at 16 a
      // stage, 52.6 at 40; x 8192, nvfp4, 32 stages: 83.0 and 85.5)
      boxes.pace = t + npairs >= p.tiles ? 0 : EPI == kMxF32 ? min(40 * p.chain_len, 640) : 16 * p.chain_len;
      // the next accumulator's sums, once they are there
      auto sums = [&](auto use) {
        ok = mbar_wait(tfull_bar(acc), acc_phase, abort_flag);
        if (!ok) return;
        tc_fence_after();
        use(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * T::kAcc);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      };
      if constexpr (is_bf16(EPI)) {
        sums([&](uint32_t taddr) { epilogue_tile<EPI>(p, boxes, tn, taddr, acc, release); });
      } else {
        const bool any = boxes.row0 < p.M;  // a warp whose rows are all past M has nothing to do
        float v[2][64];
#pragma unroll 1
        for (int c = 0; ok && c < p.chains; ++c)
          sums([&](uint32_t taddr) {
            if (any) add_chain<EPI>(v, taddr, acc, half, c == 0, release);
            else release();
          });
        if (ok && any) finish_tile<EPI>(p, boxes, tn, half, v);
      }
    }
    if (!ok) {
      if (lane == 0) report_error(p.err, kErrTimeout, kWhereGemmEpilogue);
      give_up();
    }
    if (lane == 0) bulk_wait_all();  // no store reads shared memory of a CTA that has left
  }

  tc_fence_before();
  cluster_sync();  // no CTA leaves while its peer may still signal its barriers
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

// ---------------------------------------------------------------------------
// Few tiles (decode batches), bound by the weights' bytes (70B down projection, nvfp4: 24.2 us for one row, 6.4 TB/s but for
// 3.5 us of set-up and exchange, 25.8 for 128 rows): tiles of 128 x 128 (silu: 64 gate and 64 up columns), K split over the
// CTAs of a cluster, CTA rank r over stages [r kb / S, (r + 1) kb / S).  Two CTAs an SM where there are more CTAs than SMs,
// which share what the SM can take in, so that SMs with two decide the time: 64 rows, K = 8192, fp8, 124 tiles 24.6 us (1.20
// times the weights' bytes at the copy rate), 170 33.6 (1.20), 300 51.9 (1.05); fewer tiles than half the SMs are split, and
// 80, which are not, leave 72 SMs without work: 19.5 (1.47).  Every 32-column chunk
// of the CTAs' accumulators goes into the shared memory of the CTA that finishes its unit (stores to another CTA need no
// round trip) and is summed there in rank order; that CTA's own part stays in its tensor memory.  Where two stages less of
// the ring leave room the chunks have a place of their own, so that a CTA need not wait for the others' MMAs before it
// stores (operands read from HBM, without either and with both: 421 x 1384 x 2080, fp8, 7.9 and 7.2 us; 128 x 4096 x 14336,
// nvfp4, 11.8 and 11.2; 128 x 8192 x 28672 28.2 and 27.5; one row of 4096 x 4096 5.5 and 5.6).
// A CTA's sums are of chains, too, where its stages are more than one's (kChain): the MMAs wait while the accumulator is added
// to the sums of the chains before it.  Those lie in tensor memory but for what the scales leave no room for.  fp8 codes
// behind gate_up that differ from 64 bits, 64 x 14336 x 4096: 33 of 3.7 million in chains of 16 stages, 21 of 11, 18 of 8
// (fp32 20), at 23.45, 23.55 and 23.7 us.  64 x 4096 x 14336 to fp32 in one chain, two and three a CTA 14.3, 14.5 and 14.85 us.
// (Tensor memory: the CTAs of a cluster, which wait for one another, hold four stages, 80 KB, or more, or else two or three
// and received chunks up to the whole budget, so that none shares an SM with a CTA of a pair, which holds all of its tensor
// memory and waits for its peer.)
// ---------------------------------------------------------------------------
constexpr int kSplitCols = 128;
constexpr int kSplitTmemCols = 256;
constexpr int kSplitMaxCluster = 8;

template <int FMT, int EPI>
struct SplitStage {
  static constexpr int kB = kSplitCols * kRowBytes;
  static constexpr int kSa = Stage<FMT>::kTiles * kMxTileBytes, kSb = kSa * (is_silu(EPI) ? 2 : 1);
  static constexpr int kUnits = is_silu(EPI) ? 2 : 4;          // 32 outputs each
  static constexpr int kChunks = is_silu(EPI) ? 2 : 1;         // accumulator chunks of a unit: gate, up
  // Tensor memory: the scales, then the sums of the chains that are done, in the place of the accumulator's columns but for
  // the first kKept chunks of 32, which stay in registers; then the accumulator.
  static constexpr int kTsa = 0, kTsb = 4 * Stage<FMT>::kTiles, kTsCols = kTsb + 4 * kChunks * Stage<FMT>::kTiles;
  static constexpr int kKept = (kTsCols + 31) / 32, kAcc = kSplitCols;
  static_assert(kAcc + kSplitCols <= kSplitTmemCols, "tensor memory");
  // stages of a chain, of which one more costs less here than on SM pairs
  static constexpr int kChain = is_bf16(EPI) ? FMT == kMxFp8 ? 32 : kSplitBf16Stages : FMT == kMxFp8 ? 12 : kChainStages<FMT>;
  __host__ __device__ static constexpr int bytes(int a_rows) { return a_rows * kRowBytes + kB + kSa + kSb; }
  // chunks that a CTA of S receives from each of the others, and the bytes of them all, `rows` accumulator rows each
  __host__ __device__ static constexpr int local_chunks(int S) { return (kUnits + S - 1) / S * kChunks; }
  __host__ __device__ static constexpr int recv_bytes(int S, int rows) { return (S - 1) * local_chunks(S) * rows * 128; }
};

// The scale bytes of a unit (32 outputs from column n on), and zeros for the groups that fill up the row's last word.
template <int OF>
__device__ __forceinline__ void store_unit_scales(const MxGemmParams& p, int row, int n, const uint32_t (&words)[2]) {
  constexpr int G = mx_group(OF), kGroups = 32 / G;
  const int g0 = n / G, at = n % 128 / G;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const uint32_t w = at + g < 4 ? words[0] : words[1];
    p.out_scales[mx_scale_at(row, (g0 + g) >> 2, p.out_ktiles) + ((g0 + g) & 3)] = static_cast<uint8_t>(w >> ((at + g & 3) * 8));
  }
  if (n + 32 >= p.N)
    for (int g = g0 + kGroups; g < 4 * p.out_ktiles; ++g) p.out_scales[mx_scale_at(row, g >> 2, p.out_ktiles) + (g & 3)] = 0;
}

// 32 columns of this CTA's sums: the accumulator's and, if there are chains before it, theirs.
template <class R>
struct OwnLoader {
  uint32_t taddr;
  bool chains;
  const float (&kept)[R::kKept][32];
  __device__ __forceinline__ void operator()(int col, float (&v)[32]) const {
    tmem_ld32(taddr + R::kAcc + col, v);
    if (!chains) return;
    if (col >= 32 * R::kKept) {
      float t[32];
      tmem_ld32(taddr + col, t);
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] += t[e];
    }
#pragma unroll
    for (int i = 0; i < R::kKept; ++i)
      if (col == 32 * i) {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] += kept[i][e];
      }
  }
};

// Adds the accumulator of a chain that is done to the sums of those before it (first: there are none).  release() is called
// once the accumulator is in registers.
template <class R, class Release>
__device__ __forceinline__ void save_chain(uint32_t taddr, bool first, float (&kept)[R::kKept][32], const Release& release) {
#pragma unroll
  for (int i = 0; i < kSplitCols / 32; ++i) {
    uint32_t a[32], b[32];
    tmem_ld32_async(taddr + R::kAcc + 32 * i, a);
    if (i >= R::kKept && !first) {
      tmem_ld32_async(taddr + 32 * i, b);
      tmem_ld_wait(b);
    }
    tmem_ld_wait(a);
    if (i + 1 == kSplitCols / 32) release();
    float v[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float sum = i < R::kKept ? kept[i % R::kKept][e] : __uint_as_float(b[e]);
      v[e] = first ? __uint_as_float(a[e]) : sum + __uint_as_float(a[e]);
    }
    if (i < R::kKept) {
#pragma unroll
      for (int e = 0; e < 32; ++e) kept[i % R::kKept][e] = v[e];
    } else {
      tmem_st32_async(taddr + 32 * i, v);
    }
  }
  tmem_st_wait();
}

// Receive buffer of CTA `to`: [source rank, without its own][local chunk][8 float4 columns][rows], so that a warp's rows are
// contiguous.
__device__ __forceinline__ uint32_t recv_at(int from, int to, int nloc, int li, int q, int row, int rows) {
  return static_cast<uint32_t>(((((from < to ? from : from - 1) * nloc + li) * 8 + q) * rows + row) * 16);
}

// The sum over the CTAs in rank order: this CTA's part from tensor memory, the others' from where they stored them.
template <class R, class Own>
struct SumLoader {
  const Own& mine;
  const uint8_t* recv;
  int ctas, rank, nloc, row, rows;
  __device__ __forceinline__ void operator()(int col, float (&v)[32]) const {
    const int c = col / 32, u = c % R::kUnits, li = u / ctas * R::kChunks + c / R::kUnits;
    float own[32];
    mine(col, own);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = 0.f;
#pragma unroll 2
    for (int s = 0; s < ctas; ++s) {
      if (s == rank) {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] += own[e];
        continue;
      }
      float4 t[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) t[q] = *reinterpret_cast<const float4*>(recv + recv_at(s, rank, nloc, li, q, row, rows));
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        v[4 * q] += t[q].x;
        v[4 * q + 1] += t[q].y;
        v[4 * q + 2] += t[q].z;
        v[4 * q + 3] += t[q].w;
      }
    }
  }
};

// unit u of tile column tn for one row; ld(column, v) gives 32 accumulator columns
template <int EPI, class Loader>
__device__ __forceinline__ void split_unit(const MxGemmParams& p, int row, int tn, int u, const Loader& ld) {
  const int n = tn * (is_silu(EPI) ? kSplitCols / 2 : kSplitCols) + 32 * u;
  if (n >= p.N) return;
  float v[32], up[32];
  uint32_t words[2] = {0, 0};
  ld(32 * u, v);
  if constexpr (is_silu(EPI)) ld(kSplitCols / 2 + 32 * u, up);
  finish32<EPI>(p, row, n, v, up, words);
  if constexpr (out_fmt(EPI) != 0) {
    if (row < p.M) store_unit_scales<out_fmt(EPI)>(p, row, n, words);
  }
}

// CHAINS: a CTA's stages may be more than a chain's.  (A kernel of its own for those that are not: with the chains' code in it
// 3 x 448 x 2048, nvfp4, takes 4.9 us and without 4.45; gate_up 64 x 28672 x 8192 53.2 and 50.8.)
template <int FMT, int EPI, bool CHAINS>
__global__ void __launch_bounds__(kThreads, 2)
    k_gemm_mx_split(const __grid_constant__ MxMaps maps, const __grid_constant__ MxGemmParams p) {
  using S = Stage<FMT>;
  using R = SplitStage<FMT, EPI>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  const int nst = p.stages, a_bytes = p.a_rows * kRowBytes, tile_bytes = a_bytes + R::kB;
  const uint32_t scales = sbase + nst * tile_bytes;
  uint8_t* meta = smem_raw + pad + p.meta_at;
  const uint32_t bar0 = smem_u32(meta);  // full[S], empty[S], tfull, recv, done, saved
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meta + 8 * (2 * nst + 4));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (nst + s); };
  const uint32_t tfull_bar = bar0 + 8u * (2 * nst), recv_bar = tfull_bar + 8, done_bar = tfull_bar + 16,
                 saved_bar = tfull_bar + 24;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int ctas = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int kb0 = rank * p.kb / ctas, kb1 = (rank + 1) * p.kb / ctas;
  // chains of chain_len stages, the first chain_more of them one longer
  const int stages = kb1 - kb0, chains = CHAINS ? (stages + R::kChain - 1) / R::kChain : 1;
  const int chain_len = stages / chains, chain_more = stages % chains;
  int tm, tn;
  tile_coords(p, static_cast<int>(blockIdx.x) / ctas, tm, tn);

  if (threadIdx.x == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(done_bar, 1);
    mbar_init(saved_bar, 4);  // an arrival of every warp that finishes rows
    // an arrival of every warp that has rows, in every other CTA
    mbar_init(recv_bar, max(ctas - 1, 1) * min((p.M - tm * BM + 31) / 32, 4));
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w[0]);
    if (is_silu(EPI)) tma_prefetch_desc(&maps.w[1]);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kSplitTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  if (ctas > 1 && p.recv_at > 0) cluster_arrive();  // this CTA's receive buffer may be written
  pdl_wait();
  // every CTA is resident (or soon will be): the next kernel may set up beside them where there is room
  if (threadIdx.x == 0) pdl_trigger();

  if (warp == 0) {
    // ---------------- copies ----------------
    const uint64_t pol_a = policy_evict_last(), pol_b = policy_evict_first();
    int stage = 0, used = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        const uint32_t sa = sbase + stage * tile_bytes, sb = sa + a_bytes;
        const uint32_t ssa = scales + stage * (R::kSa + R::kSb), ssb = ssa + R::kSa;
        const int kt = kb * S::kTiles;
        const uint32_t sbytes = min(S::kTiles, p.ktiles - kt) * kMxTileBytes;  // of the scales of 128 rows
        auto scales_of = [&](const uint8_t* all, int rt) {
          return all + (static_cast<size_t>(rt) * p.ktiles + kt) * kMxTileBytes;
        };
        mbar_arrive_expect_tx(full_bar(stage), a_bytes + R::kB + sbytes * (1 + R::kChunks));
        if constexpr (is_silu(EPI)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tma_load_2d(sb + i * R::kB / 2, &maps.w[i], full_bar(stage), kb * kRowBytes, tn * 64, pol_b);
            bulk_load(ssb + i * R::kSa, scales_of(p.w_scales[i], tn >> 1), sbytes, full_bar(stage), pol_b);
          }
        } else {
          tma_load_2d(sb, &maps.w[0], full_bar(stage), kb * kRowBytes, tn * 128, pol_b);
          bulk_load(ssb, scales_of(p.w_scales[0], tn), sbytes, full_bar(stage), pol_b);
        }
        tma_load_2d(sa, &maps.x, full_bar(stage), kb * kRowBytes, tm * BM, pol_a);
        bulk_load(ssa, scales_of(p.x_scales, tm), sbytes, full_bar(stage), pol_a);
      }
      __syncwarp();
      ++used;
      if (++stage == nst) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      if (lane == 0) report_error(p.err, kErrTimeout, kWhereGemmProducer);
      *abort_flag = 1;
    }
    // every copy has landed before shared memory is used again or left: of the stages in use, the last phase of each
    for (int s = 0; s < nst && s < used; ++s) mbar_wait(full_bar(s), static_cast<uint32_t>((used - 1 - s) / nst) & 1u, nullptr);
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    constexpr uint32_t idesc = idesc_mx(BM, is_silu(EPI) ? 64 : 128, S::kBits, S::kE8m0);
    const uint32_t gate_cols = is_silu(EPI) ? (tn & 1) * 2 : 0;  // a tile's 64 rows of w in their 128-row scale tile
    const uint32_t acc = tmem_base + R::kAcc, ts = tmem_base;  // the accumulator, the scales
    int stage = 0, first = kb0, chain = 0, end = kb0 + chain_len + (chain_more > 0 ? 1 : 0);
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (CHAINS && kb == end) {
        if (elect_one()) tc_commit(done_bar);
        __syncwarp();
        if (!warp_same(mbar_wait(saved_bar, chain & 1, abort_flag))) {
          ok = false;
          break;
        }
        ++chain;
        first = kb;
        end = kb + chain_len + (chain < chain_more ? 1 : 0);
      }
      if (!warp_same(mbar_wait(full_bar(stage), phase, abort_flag))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sa = sbase + stage * tile_bytes, sb = sa + a_bytes;
        const uint32_t ssa = scales + stage * (R::kSa + R::kSb), ssb = ssa + R::kSa;
#pragma unroll
        for (int i = 0; i < S::kTiles; ++i) {
          tc_copy_scales<false>(ts + R::kTsa + 4 * i, smem_desc_scales(ssa + i * kMxTileBytes));
#pragma unroll
          for (int j = 0; j < R::kChunks; ++j)
            tc_copy_scales<false>(ts + R::kTsb + 4 * (R::kChunks * i + j),
                                  smem_desc_scales(ssb + j * R::kSa + i * kMxTileBytes));
        }
        const int steps = kb + 1 < p.kb ? S::kSteps : p.last_steps;
#pragma unroll
        for (int k = 0; k < S::kSteps; ++k) {
          if (k >= steps) break;
          const int i = k / S::kPerTile;
#pragma unroll
          for (int j = 0; j < R::kChunks; ++j)
            tc_mma_mx<S::kBits, S::kStepScales, false>(
                acc + 64 * j, smem_desc_sw128(sa + 32 * k), smem_desc_sw128(sb + j * (R::kB / 2) + 32 * k),
                idesc_mx_scale(idesc, k % S::kPerTile * S::kStepScales), ts + R::kTsa + 4 * i,
                ts + R::kTsb + 4 * (R::kChunks * i + j) + gate_cols, kb > first || k > 0 ? 1u : 0u);
        }
        tc_commit(empty_bar(stage));
      }
      __syncwarp();
      if (++stage == nst) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      if (lane == 0) report_error(p.err, kErrTimeout, kWhereGemmMma);
      *abort_flag = 1;
    }
    // completes once everything issued above has: the accumulator is whole (or, given up, no longer written)
    if (elect_one()) tc_commit(tfull_bar);
    __syncwarp();
  }
  const int quad = warp & 3;  // tensor-memory lane quarter this warp may access
  const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
  float kept[R::kKept][32];
  if (CHAINS && warp >= 2) {
#pragma unroll 1
    for (int c = 0; c + 1 < chains; ++c) {
      if (!warp_same(mbar_wait(done_bar, c & 1, abort_flag))) {
        if (lane == 0) report_error(p.err, kErrTimeout, kWhereGemmEpilogue);
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      save_chain<R>(taddr, c == 0, kept, [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(saved_bar);
      });
    }
  }
  if (!mbar_wait(tfull_bar, 0, nullptr)) {
    if (lane == 0) report_error(p.err, kErrTimeout, kWhereGemmEpilogue);
    *abort_flag = 1;
  }
  tc_fence_after();

  const OwnLoader<R> mine{taddr, chains > 1, kept};
  if (ctas == 1) {
    __syncthreads();
    if (warp >= 2 && !*abort_flag && tm * BM + quad * 32 < p.M) {
#pragma unroll 1
      for (int u = 0; u < R::kUnits; ++u) split_unit<EPI>(p, tm * BM + quad * 32 + lane, tn, u, mine);
    }
  } else {
    const int nloc = R::local_chunks(ctas);
    const uint32_t recv = sbase + p.recv_at;
    __syncwarp();
    if (p.recv_at == 0) cluster_arrive();  // this CTA's MMAs and copies are done: its ring may be written
    cluster_wait();
    const bool has_rows = warp >= 2 && tm * BM + quad * 32 < p.M;
    const int row_in_tile = quad * 32 + lane;
    if (has_rows) {
#pragma unroll 1
      for (int c = 0; c < kSplitCols / 32; ++c) {
        const int u = c % R::kUnits, li = u / ctas * R::kChunks + c / R::kUnits, to = u % ctas;
        if (to == rank) continue;
        float v[32];
        mine(32 * c, v);
        const uint32_t dst = mapa_shared(recv + recv_at(rank, to, nloc, li, 0, row_in_tile, p.a_rows), static_cast<uint32_t>(to));
        if (tm * BM + row_in_tile < p.M) {  // (other rows' sums are never looked at)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_cluster_f4(dst + q * p.a_rows * 16, make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
        }
      }
      __syncwarp();
      if (lane < min(R::kUnits, ctas) && lane != rank) mbar_arrive_cluster(mapa_shared(recv_bar, lane));
    }
    __syncwarp();
    cluster_arrive();  // this CTA writes to no other any more
    if (has_rows && rank < R::kUnits) {
      if (!warp_same(mbar_wait_cluster(recv_bar, 0))) {
        if (lane == 0) report_error(p.err, kErrTimeout, kWhereGemmEpilogue);
        *abort_flag = 1;
      } else {
        const SumLoader<R, OwnLoader<R>> ld{mine, smem_raw + pad + p.recv_at, ctas, rank, nloc, row_in_tile, p.a_rows};
#pragma unroll 1
        for (int u = rank; u < R::kUnits; u += ctas) split_unit<EPI>(p, tm * BM + row_in_tile, tn, u, ld);
      }
    }
    __syncwarp();
    cluster_wait();  // no CTA leaves while another may write to it
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, kSplitTmemCols);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

bool encode_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, long long cols, long long rows,
               long long row_bytes, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the maps of one operand of `rows` rows (scales null: they are copied untiled)
bool operand_maps(CUtensorMap* codes, CUtensorMap* scales, const MxOperand& o, int rows, long long row_bytes, int ktiles,
                  int stage_tiles, int box_rows) {
  return encode_2d(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.codes, row_bytes, rows, row_bytes, kRowBytes, box_rows,
                   CU_TENSOR_MAP_SWIZZLE_128B) &&
         (scales == nullptr ||
          encode_2d(scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, o.scales, static_cast<long long>(ktiles) * kScaleElems,
                   (rows + kMxTileRows - 1) / kMxTileRows, static_cast<long long>(ktiles) * kMxTileBytes,
                   stage_tiles * kScaleElems, 1, CU_TENSOR_MAP_SWIZZLE_NONE));
}

template <int FMT, int EPI>
cudaError_t raise_limits() {
  static SmemLimits limits;
  return limits.raise({smem_need(k_gemm_mx_split<FMT, EPI, false>, kMaxSmemBytes),
                       smem_need(k_gemm_mx_split<FMT, EPI, true>, kMaxSmemBytes),
                       smem_need(k_gemm_mx_pair<FMT, EPI>, PairRing<FMT>::kSmem)});
}

// Clusters of S CTAs that are resident at once, of those that take an SM each.  (A cluster's SMs are of one GPC, so that the
// SMs hold fewer clusters than their number says.)
template <int FMT, int EPI>
cudaError_t max_active_pairs(int* n) {
  static ClusterLimit limit;
  return limit.get(reinterpret_cast<const void*>(k_gemm_mx_pair<FMT, EPI>), 2, pair_threads(EPI), PairRing<FMT>::kSmem, n);
}

// (the same for every kernel that takes an SM: asked of one)
cudaError_t max_active_splits(int S, int* n) {
  static ClusterLimit limits[kSplitMaxCluster + 1];
  const cudaError_t e = raise_limits<kMxFp8, kMxBf16>();
  if (e != cudaSuccess) return e;
  return limits[S].get(reinterpret_cast<const void*>(k_gemm_mx_split<kMxFp8, kMxBf16, true>), S, kThreads, kMaxSmemBytes, n);
}

// Which kernel, by estimates of both in microseconds.  tiles: of 128 x 128 for the split kernel, which splits K over S CTAs; of
// 256 x 256 for SM pairs.  Fitted to 600 random sizes; of 1000 others, bf16, fp32 and quantised results, operands from HBM, the
// chosen kernel takes 0.1% more than the better one in the mean.  It is a choice, not a prediction: a tile of gate_up takes 2.3
// us at least, and both kernels take longer than estimated there.  A stage of a pair's tile takes 0.28 and a tile 0.4 more, 0.8
// at least; a stage of a CTA of the split kernel 0.26, with two on an SM 0.44 to 0.46 and 1.3 a wave, of up to 64 rows 0.5; 5.2
// (3.2 of them besides the reads of weights) and 3.5 pass besides.  Weights are read at 5.4 TB/s by pairs and at 6.2 by the
// split kernel, 5.4 where more than 64 rows of x have more tiles than the SMs hold.  (Split and pairs: 8192 x 8192, nvfp4, 256
// rows 12.0 and 15.5, 384 rows 17.2 and 15.5; 4096 x 14336, fp8, 256 rows 18.8 and 35.3; 57344 x 8192, nvfp4, 16 rows 46.6 and
// 56.1; gate and up of 28672 x 8192, nvfp4, 128 rows 54 and 47.5.)
bool use_pairs(int M, long long tiles, int S, long long pair_tiles, int kb, double weight_bytes, int sms) {
  const long long pairs = sms / 2, waves = (pair_tiles + pairs - 1) / pairs, ctas = tiles * S;
  const double pair = std::max(2 + waves * std::max(kb * 0.28 + 0.4, 0.8), weight_bytes / 5.4e6);
  const double stages = static_cast<double>(kb) / S, wave = M > 64 ? 1.3 : 0.5;
  double split = stages * 0.26;
  if (ctas > 2 * sms) split = (ctas + 2 * sms - 1) / (2 * sms) * (stages * 0.46 + wave);
  else if (ctas > sms) split = stages * 0.44 + 1;
  split = std::max(split, weight_bytes / (M > 64 && ctas > 2 * sms ? 5.4e6 : 6.2e6));
  return pair + 3.2 < split + 3.5;
}

template <int FMT, int EPI>
int launch_typed(const MxGemmArgs& a, MxGemmParams& p, cudaStream_t s) {
  using T = Stage<FMT>;
  using R = SplitStage<FMT, EPI>;
  cudaError_t e = raise_limits<FMT, EPI>();
  if (e != cudaSuccess) return e;
  const int sms = num_sms();
  const long long row_bytes = static_cast<long long>(a.K) * T::kBits / 8;
  const int ktiles = (a.K / mx_group(FMT) + kMxTileGroups - 1) / kMxTileGroups;
  const int pair_m = (p.M + 2 * BM - 1) / (2 * BM), pair_n = is_silu(EPI) ? (p.N + 127) / 128 : (p.N + 255) / 256;
  p.tiles_m = (p.M + BM - 1) / BM;
  p.tiles_n = is_silu(EPI) ? (p.N + 63) / 64 : (p.N + 127) / 128;
  p.tiles = p.tiles_m * p.tiles_n;
  p.a_rows = p.M >= 128 ? 128 : (p.M + 31) / 32 * 32;
  const int stage_bytes = R::bytes(p.a_rows);
  // As many CTAs a tile as the SMs have room for, four stages or more each; without a split two CTAs an SM if they are more
  // than the SMs.
  int S = 1;
  for (int n = kSplitMaxCluster; n > 1 && S == 1; --n)
    if (static_cast<long long>(p.tiles) * n <= sms && p.kb >= 4 * n &&
        R::recv_bytes(n, p.a_rows) <= kRingBudget / stage_bytes * stage_bytes) {
      int room = 0;
      if ((e = max_active_splits(n, &room)) != cudaSuccess) return e;
      if (room >= p.tiles) S = n;
    }
  int pairs = 0;
  if ((e = max_active_pairs<FMT, EPI>(&pairs)) != cudaSuccess) return e;
  const bool pair = pairs > 0 && (!is_bf16(EPI) || p.kb <= kPairBf16Stages) &&
                    use_pairs(p.M, p.tiles, S, static_cast<long long>(pair_m) * pair_n, p.kb,
                              (is_silu(EPI) ? 2. : 1.) * p.N * row_bytes * (1 + 1. / 16), sms);
  MxMaps maps{};
  const int w_box = !pair && is_silu(EPI) ? 64 : 128;
  bool ok = operand_maps(&maps.x, pair ? &maps.x_scales : nullptr, a.x, a.M, row_bytes, ktiles, T::kTiles,
                         pair ? 128 : p.a_rows);
  for (int i = 0; i < (is_silu(EPI) ? 2 : 1); ++i)
    ok = ok && operand_maps(&maps.w[i], pair ? &maps.w_scales[i] : nullptr, a.w[i], a.N, row_bytes, ktiles, T::kTiles, w_box);
  if (pair) {
    constexpr bool kCodes = out_fmt(EPI) != 0, kF32 = EPI == kMxF32;
    const long long cols = kCodes ? static_cast<long long>(p.N) / 8 * mx_bits(out_fmt(EPI)) : p.N;
    const int elem = kCodes ? 1 : kF32 ? 4 : 2, box = kCodes ? 8 * mx_bits(out_fmt(EPI)) : 128;  // bytes
    ok = ok && encode_2d(&maps.out,
                         kCodes ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                         : kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         p.out, cols, p.M, cols * elem, box / elem, 32,
                         box == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                         : box == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : CU_TENSOR_MAP_SWIZZLE_32B);
  }
  if (!ok) return cudaErrorInvalidValue;
  if (pair) {
    p.tiles_m = pair_m;
    p.tiles_n = pair_n;
    p.tiles = pair_m * pair_n;
    // Raster: the tiles of as many rows of x as 32 MB of its codes hold, column by column, so that these stay in L2 while
    // the weights pass once a group.  The part is held by its power limit, and what moves least runs at the highest clock
    // (a second of calls, 12 tiles a group and then this: 70B o_proj, 32768 rows, nvfp4 664 and 658 us, fp8 1361 and 1341;
    // gate_up, 4128 rows, nvfp4 628 and 613).
    const long long group = (32LL << 20) / (2 * BM * row_bytes);
    p.group_m = group < 4 ? 4 : group < pair_m ? static_cast<int>(group) : pair_m;
    if (p.group_m > pair_m) p.group_m = pair_m;
    p.chains = is_bf16(EPI) ? 1 : (p.kb + kChainStages<FMT> - 1) / kChainStages<FMT>;
    p.chain_len = p.kb / p.chains;
    p.chain_more = p.kb % p.chains;
    return launch_kernel_cluster(k_gemm_mx_pair<FMT, EPI>, dim3(2 * (p.tiles < pairs ? p.tiles : pairs)), dim3(pair_threads(EPI)),
                                 PairRing<FMT>::kSmem, s, true, 2, maps, p);
  }
  p.group_m = p.tiles_m;
  p.ktiles = ktiles;
  p.x_scales = static_cast<const uint8_t*>(a.x.scales);
  for (int i = 0; i < 2; ++i) p.w_scales[i] = static_cast<const uint8_t*>(a.w[i].scales);
  const int ctas = p.tiles * S, budget = ctas > sms ? kMaxSmemBytes / 2 - 1024 - 2048 : kRingBudget;
  const int fill = (p.kb + S - 1) / S;  // stages that a CTA fills
  const int recv = S > 1 ? R::recv_bytes(S, p.a_rows) : 0;
  auto stages = [&](int bytes) { return std::min({bytes / stage_bytes, kMaxStages, fill}); };
  p.stages = stages(budget);
  p.meta_at = std::max(p.stages * stage_bytes, recv);
  // (a split has four stages to fill or more, so that two at least are left)
  if (S > 1 && stages(budget - recv) >= p.stages - 2) {
    p.stages = stages(budget - recv);
    p.recv_at = p.stages * stage_bytes;
    p.meta_at = p.recv_at + recv;
  }
  return launch_kernel_cluster(fill > R::kChain ? k_gemm_mx_split<FMT, EPI, true> : k_gemm_mx_split<FMT, EPI, false>, dim3(ctas),
                               dim3(kThreads), static_cast<size_t>(p.meta_at) + 2048, s, true, S, maps, p);
}

template <int FMT>
int launch_fmt(const MxGemmArgs& a, cudaStream_t s) {
  using S = Stage<FMT>;
  MxGemmParams p{};
  p.M = a.M;
  p.N = a.N;
  p.kb = static_cast<int>((static_cast<long long>(a.K) * S::kBits / 8 + kRowBytes - 1) / kRowBytes);
  p.last_steps = (a.K - (p.kb - 1) * S::kElems + S::kStepElems - 1) / S::kStepElems;
  for (int i = 0; i < 2; ++i) p.alpha[i] = a.alpha[i];
  p.out = a.out;
  const long long out_row = a.out_fmt ? static_cast<long long>(a.N) * mx_bits(a.out_fmt) / 8 : a.N * (a.out_f32 ? 4LL : 2LL);
  p.sectors = (out_row | static_cast<long long>(reinterpret_cast<uintptr_t>(a.out))) % 32 == 0;
  p.out_scales = static_cast<uint8_t*>(a.out_scales);
  if (a.out_fmt) p.out_ktiles = (a.N / mx_group(a.out_fmt) + kMxTileGroups - 1) / kMxTileGroups;
  p.out_inv_g = a.out_inv_g;
  p.out_sixth = a.out_sixth;
  p.err = a.err;
  if (!a.silu) return a.out_f32 ? launch_typed<FMT, kMxF32>(a, p, s) : launch_typed<FMT, kMxBf16>(a, p, s);
  switch (a.out_fmt) {
    case 0:
      return launch_typed<FMT, kMxSilu>(a, p, s);
    case kMxNvfp4:
      return launch_typed<FMT, kMxSiluNvfp4>(a, p, s);
    case kMxFp4:
      return launch_typed<FMT, kMxSiluFp4>(a, p, s);
    default:
      return launch_typed<FMT, kMxSiluFp8>(a, p, s);
  }
}

}  // namespace

int gemm_mx_launch(const MxGemmArgs& a, cudaStream_t s) {
  if (a.M <= 0) return 0;
  switch (a.fmt) {
    case kMxNvfp4:
      return launch_fmt<kMxNvfp4>(a, s);
    case kMxFp4:
      return launch_fmt<kMxFp4>(a, s);
    case kMxFp8:
      return launch_fmt<kMxFp8>(a, s);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace llama
