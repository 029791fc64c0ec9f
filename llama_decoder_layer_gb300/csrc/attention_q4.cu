// Paged, causal, grouped-query attention over a KV cache held in 4 bits.
//
//   o[t, h] = sum_j softmax_j(q[t, h] . K[b, h / g, j] / sqrt(d)) V[b, h / g, j],
//   j = 0 .. position(t), K and V the values of the 4-bit tiles (q4.cuh)
//
// * Sequences of one new token, or of so few that new * g <= 16 rows share a
//   pass over the keys: k_attn_q4_decode, bound by the cache's bytes up to 8 rows
//   and by the latency of its chains at 12 warps an SM with 16.  128 sequences of 512 .. 8192 tokens, 64
//   query and 8 KV heads x 128, 649 MB: 120 us, 5.4 TB/s, 80% of the copy rate (the
//   copies alone take 117, the arithmetic alone 115).  Four sequences of up to
//   131072 tokens with two new tokens each, 32 and 4 heads, 194 MB: 55 us, 3.5 TB/s.
//   - Work is the list of (sequence, KV head, block), cut into one range per CTA
//     (four an SM, three with 16 rows), whatever the lengths; every CTA finds its
//     range from the sequence lengths itself.  A (sequence, KV head) cut by a
//     border leaves partial sums (unnormalised o, maximum, sum) that
//     k_attn_q4_combine joins in order; the others are finished where they are.
//   - A CTA's four warps take the blocks of its range in turn, each through a
//     ring of its own (9 to 18 KB) filled by its lanes' asynchronous copies, across
//     the borders of sequences.  A tile's byte order makes the codes that a lane
//     copies its own operands, so a stage needs no barrier but the warp's.
//   - S^T = K Q^T and O^T = V^T P^T with m16n8k16 in fp16, fp32 sums: keys and
//     head elements on the 16-row side, the query rows on the 8-column side, so
//     a group of 8 heads wastes nothing.  Codes -> fp16 by the conversion
//     instruction (2 values each), times the scale, exact (6 significant bits).
//     (A tcgen05.mma would want the operands back in shared memory or TMEM, and
//     its 128 rows filled by 8.)
//   - q is brought to fp16 with a power of two per row that puts its largest
//     element at 2^14 (exact but for elements 2^-29 of that).  Weights are fp16
//     (relative error 2^-11), relative to a maximum that is only moved when a
//     score passes it by 2^8, times 2^6: normal fp16 down to 2^-20 of it.
// * Longer sequences: their blocks are expanded once into a 16-bit copy
//   (k_q4_expand) over which the prefill kernels of the bf16 cache run: every
//   tile is read by all query tiles, so decoding it there would repeat the work
//   and load the softmax's pipes.  Of a batch of 32 decoding sequences of up to
//   16384 tokens and two prompts of 2048 tokens, 212 us, the expansion takes 9, the
//   decode kernels (on a side stream) 60 and the prefill kernel 139.  Few new
//   tokens after many keys: the prefill kernels' keys are split over CTAs.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q4.cuh"

namespace llama {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 16;        // query rows (new tokens x group) of the decode path
constexpr int kCtasPerSm = 4;
constexpr int kRankStep = 46;       // half the share lost from one CTA of an SM to the next, in 1/1024 of the mean (0, 32,
                                    // 46, 60: 131.0, 128.7, 126.9, 129.0 us, 128 sequences of 703 MB in a graph)
constexpr int kMinShare = 8;        // blocks a CTA takes at least: two a warp
constexpr int kWholeBlocks = 64;    // pieces of up to so many blocks stay whole where the SMs hold them all
constexpr int kFewBlocks = 16384;   // blocks up to which a batch with prompts decodes in one launch, of the 16-row kernel
constexpr int kPieceCost = 6;       // what a (sequence, KV head) costs a CTA beside its blocks, in blocks
constexpr float kMaxStep = 8.f;     // log2 by which a score may pass the running maximum
constexpr float kWeightBias = 6.f;  // weights are stored times 2^6
constexpr float kMinusInf = -INFINITY;

template <int D>
constexpr int stages() { return D == 128 ? 4 : 8; }  // a power of two

// A piece that spans CTAs, for k_attn_q4_combine.
struct Cut {
  int first, last;  // its CTAs; last < 0: nothing to join
  int t0, rows, len, h, unused[2];  // (32 bytes)
};

struct Q4Params {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const uint8_t *k_cache, *v_cache;
  const int32_t *qsl, *seq_lens, *positions, *block_table;
  int T, B, max_blocks, num_blocks, nq, nkv, group, max_query_len, max_seq_len;
  int sms;
  int whole;  // every CTA takes one (sequence, KV head)
  int rows_lo, rows_hi;  // the sequences of the launch: those of so many query rows
  float scale_log2, v_scale;
  float* part_o;   // [CTA][2][kMaxRows][D]
  float2* part_ml; // [CTA][2][kMaxRows]: maximum, sum
  Cut* cut;
  int cut_by_piece;  // cut is indexed by sequence * nkv + KV head (else by the piece's first CTA)
  int* err;
};

// Blocks of a sequence on the decode path; 0 if it has no new tokens, takes the
// prefill path, or is out of bounds (*bad).
__device__ __forceinline__ int decode_blocks(const Q4Params& p, int b, int& t0, int& rows, int& len, bool& bad) {
  t0 = p.qsl[b];
  const int n = p.qsl[b + 1] - t0;
  len = p.seq_lens[b];
  rows = n * p.group;
  bad = n > p.max_query_len || t0 < 0 || t0 > p.T - n;  // n rows of q and out from t0 on, as the launch was sized for
  if (bad || n < 1 || (n > 1 && (n > kMaxRows || rows > kMaxRows)) || rows < p.rows_lo || rows > p.rows_hi) return 0;
  const int nblk = (len + kQ4Block - 1) / kQ4Block;
  bad = len < 1 || len > p.max_seq_len || nblk > p.max_blocks;
  return bad ? 0 : nblk;
}

__device__ __forceinline__ int plan_blocks(const Q4Params& p, int b) {
  int t0, rows, len;
  bool bad;
  return decode_blocks(p, b, t0, rows, len, bad);
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// bits of a where mask has ones, of b where it has zeros
template <uint32_t kMask>
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(d) : "r"(a), "r"(b), "n"(kMask));
  return d;
}

// a value that is the same in every lane, in a form the compiler can keep once per warp
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t addr) {
  static_assert(N == 2 || N == 4, "8 or 16 bytes");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}

__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// A lane's asynchronous copy of N bytes (4, 8 or 16) into its own shared memory.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// all but the newest N groups of this lane have landed
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How the units are cut into the CTAs' ranges.  An SM's warp schedulers favour the
// warps of the CTA that came first: with equal ranges the four CTAs of an SM ended
// after 86, 94, 103 and 112 us (128-sequence batch), the last ones on a half-empty
// SM.  So the CTAs of rank r (the r-th on their SM: the grid fills the SMs in
// turn) get a share that falls with r.
struct Split {
  long long total, mean;
  int per_rank, ranks;
  Split() = default;
  __device__ __forceinline__ Split(long long units, int sms) : total(units) {
    const int grid = gridDim.x;
    mean = units < 0x7fffffffLL ? (static_cast<uint32_t>(units) + grid - 1) / grid : (units + grid - 1) / grid;
    const bool ranked = grid > sms && grid % sms == 0 && mean >= 2 * kMinShare;
    per_rank = ranked ? sms : grid;
    ranks = ranked ? grid / sms : 1;
    if (mean < kMinShare) mean = kMinShare;
  }
  // the shares sum to the mean's (their parts of it are opposite in pairs, rounded down, plus one)
  __device__ __forceinline__ long long share(int r) const {
    return mean + ((mean * kRankStep * (ranks - 1 - 2 * r)) >> 10) + (ranks > 1);
  }
  __device__ __forceinline__ long long begin(int cta) const {
    long long at = 0;
#pragma unroll
    for (int r = 0; r < kCtasPerSm; ++r)
      if (r < ranks) at += min(max(cta - r * per_rank, 0), per_rank) * share(r);
    return at;
  }
  __device__ __forceinline__ int cta_of(long long unit) const {
    int r = 0;
    while (r < ranks - 1 && unit >= per_rank * share(r)) unit -= per_rank * share(r++);
    return r * per_rank + static_cast<int>(unit / share(r));
  }
};

// Where a CTA's range begins or ends.
struct Place {
  long long blocks;  // blocks before it
  long long unit;    // first unit of its piece
  int b, h, j;       // sequence, KV head, block
  int nblk;          // blocks of the sequence
};

// NT: 8-row tiles of query rows (the rows of a sequence: new token r / group, head r % group)
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? kCtasPerSm : 3) k_attn_q4_decode(const Q4Params p) {
  constexpr int TB = q4_tile_bytes(D);
  constexpr int S = stages<D>();
  constexpr int KW = D / 32;   // words of K codes a lane and 8 keys; of V codes too
  constexpr int MT = D / 16;   // 16-element tiles of the head
  constexpr int W = D / 8;     // head elements a lane holds of O
  constexpr int ROWS = 8 * NT;
  // a stage of a warp's ring: K codes of keys 0-7, 8-15, V codes of the same,
  // K scales, V scales, each a run of the lanes' own bytes
  constexpr int CB = 32 * 4 * KW, STB = 4 * CB + 2 * 128;
  extern __shared__ __align__(16) uint8_t smem[];
  float* obuf = reinterpret_cast<float*>(smem + kWarps * S * STB);      // [warp][ROWS][D]
  float2* mlbuf = reinterpret_cast<float2*>(obuf + kWarps * ROWS * D);  // [warp][ROWS]
  __shared__ long long sums[kWarps];
  __shared__ Place range[2];

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();

  // ---- the CTA's range of blocks: its first one (sequence cb, KV head ch, block cj
  // of first_n) and how many
  int cb, ch, cj = 0, first_n, count;
  long long unit = 0;      // of the piece's start
  Split split;
  if (p.whole) {  // few short pieces: one a CTA
    cb = blockIdx.x / p.nkv;
    ch = blockIdx.x - cb * p.nkv;
    int t0, rows, len;
    bool bad;
    first_n = count = uniform(decode_blocks(p, cb, t0, rows, len, bad));
    if (bad && ch == 0 && threadIdx.x == 0) report_error(p.err, kErrGuard, kWhereQueryLen);
    if (count == 0) return;
  } else {
    // Exclusive sums of the sequences' blocks (and their number, in the low 17 bits: at most 65535), a run of
    // sequences per thread.  A piece (sequence, KV head) counts kPieceCost units before those of its blocks.
    const int per = (p.B + kThreads - 1) / kThreads;
    const int bfirst = min(p.B, static_cast<int>(threadIdx.x) * per), blast = min(p.B, bfirst + per);
    long long mine = 0;
    for (int b = bfirst; b < blast; ++b) {
      int t0, rows, len;
      bool bad;
      const int n = decode_blocks(p, b, t0, rows, len, bad);
      if (n > 0) mine += (static_cast<long long>(n) << 17) + 1;
      if (bad && blockIdx.x == 0) report_error(p.err, kErrGuard, kWhereQueryLen);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    long long excl = incl - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) excl += sums[w];
      all += sums[w];
    }
    auto units_of = [&](long long v) { return ((v >> 17) + kPieceCost * (v & 0x1FFFF)) * p.nkv; };
    split = Split(units_of(all), p.sms);
    const long long begin = split.begin(blockIdx.x), end = min(split.total, split.begin(blockIdx.x + 1));
    if (threadIdx.x == 0 && !p.cut_by_piece) p.cut[blockIdx.x].last = -1;
    if (begin >= end) return;
    const long long first_unit = units_of(excl), last_unit = first_unit + units_of(mine);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const long long at = which == 0 ? begin : end - 1;  // the end by its last unit
      if (at < first_unit || at >= last_unit) continue;
      long long from = first_unit, blocks = (excl >> 17) * p.nkv;
      for (int b = bfirst; b < blast; ++b) {
        const int n = per == 1 ? static_cast<int>(mine >> 17) : plan_blocks(p, b);
        if (n == 0) continue;
        const long long units = static_cast<long long>(n + kPieceCost) * p.nkv;
        if (at < from + units) {
          Place x;
          x.b = b;
          x.nblk = n;
          x.h = static_cast<int>(static_cast<uint32_t>(at - from) / static_cast<uint32_t>(n + kPieceCost));
          x.unit = from + static_cast<long long>(x.h) * (n + kPieceCost);
          // blocks before unit `at` (for the end: before the unit after it)
          x.j = max(0, static_cast<int>(at - x.unit) + which - kPieceCost);
          x.blocks = blocks + static_cast<long long>(x.h) * n + x.j;
          range[which] = x;
          break;
        }
        from += units;
        blocks += static_cast<long long>(n) * p.nkv;
      }
    }
    __syncthreads();
    cb = uniform(range[0].b);
    ch = uniform(range[0].h);
    cj = uniform(range[0].j);
    first_n = uniform(range[0].nblk);
    count = uniform(static_cast<int>(range[1].blocks - range[0].blocks));
    unit = range[0].unit;
    if (count <= 0) return;
  }

  // ---- the warp's blocks: warp, warp + 4, ... of the range.  Lane i looks up
  // the tiles of blocks i, 32 + i, ... of those, 32 at once.
  const uint32_t ring = smem_u32(smem) + warp * S * STB;
  const int mine_n = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;
  int issued = 0;
  int pb = cb, pn = first_n, tile = 0;
  uint32_t px = static_cast<uint32_t>(ch) * pn + cj + warp + kWarps * lane;  // block within sequence pb, over its heads
  auto look_up = [&]() {
    if (issued + lane < mine_n) {
      while (px >= static_cast<uint32_t>(pn) * p.nkv) {
        px -= static_cast<uint32_t>(pn) * p.nkv;
        do pn = plan_blocks(p, ++pb);
        while (pn == 0);
      }
      const uint32_t h = px / pn, jb = px - h * pn;
      int blk = p.block_table[static_cast<size_t>(pb) * p.max_blocks + jb];
      if (blk < 0 || blk >= p.num_blocks) {
        report_error(p.err, kErrGuard, kWhereBlockTable);
        blk = 0;
      }
      tile = blk * p.nkv + h;
      px += kWarps * 32;
    }
    __syncwarp();
  };
  // the next block's copies: every lane fetches the bytes it will use
  const uint8_t* const k_lane = p.k_cache + lane * (4 * KW);
  const uint8_t* const v_lane = p.v_cache + lane * (4 * KW);
  const uint32_t ring_c = ring + lane * (4 * KW);
  const uint32_t ring_ks = ring + 4 * CB + (D == 128 ? lane : lane >> 1) * 4;
  const uint32_t ring_vs = ring + 4 * CB + 128 + ((D == 128 ? g : g >> 1) * 4 + t) * 4;
  auto issue = [&](uint32_t st) {
    if (issued < mine_n) {
      if (issued % 32 == 0) look_up();
      const size_t at = static_cast<size_t>(__shfl_sync(0xffffffffu, tile, issued % 32)) * TB;
      const uint8_t *kp = k_lane + at, *vp = v_lane + at;
      copy_async<4 * KW>(ring_c + st, kp);
      copy_async<4 * KW>(ring_c + st + CB, kp + 4 * D);
      copy_async<4 * KW>(ring_c + st + 2 * CB, vp);
      copy_async<4 * KW>(ring_c + st + 3 * CB, vp + 4 * D);
      if (lane < 8) {  // the scales, for all lanes
        copy_async<4 * KW>(ring_c + st + 4 * CB, kp + 8 * D);
        copy_async<4 * KW>(ring_c + st + 4 * CB + 128, vp + 8 * D);
      }
    }
    ++issued;
    copy_commit();
  };
  auto after = [](uint32_t st) { return st == (S - 1) * STB ? 0u : st + STB; };  // the next stage

  // ---- pieces: blocks cj .. of (cb, ch)
  int t0, rows, len, nblk;
  uint4 qu[NT][D / 32];  // row nt * 8 + g, elements t * D/4 ..
  int qpos[NT];
  auto load_q = [&]() {
    bool bad;
    nblk = uniform(decode_blocks(p, cb, t0, rows, len, bad));
    len = uniform(len);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) qu[nt][i] = make_uint4(0, 0, 0, 0);
      qpos[nt] = len - 1;
      if (r < rows) {
        const int tok = t0 + r / p.group;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (static_cast<size_t>(tok) * p.nq + ch * p.group + r % p.group) * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) qu[nt][i] = src[i];
        qpos[nt] = p.positions[tok];
      }
    }
  };
  if (NT == 1) load_q();  // before the ring is filled: behind those copies it would wait for all of them
#pragma unroll 1
  for (int i = 0; i < S; ++i) issue(i * STB);
  uint32_t stage = 0;  // of the warp's next block
  int left = count;
  int first = 0;  // index in the range of the piece's first block
  while (left > 0) {
    if (NT > 1) load_q();
    const int n = min(left, nblk - cj);
    // q as the 8-column operand
    uint32_t bq[NT][D / 8];
    float sc[NT][2];
    int lim_lo = 0x7fffffff, seen = 0;  // the least position of a row; keys that any row sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (qpos[nt] < 0 || qpos[nt] >= len)
        qpos[nt] = len - 1;  // such a row is not stored
      else if (nt * 8 + g < rows)
        seen = max(seen, qpos[nt] + 1);
      lim_lo = min(lim_lo, qpos[nt]);
      float amax = 0.f;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(qu[nt]);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -112);
      const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
      // (at least 2^-124: smaller ones give scores below 2^-60 either way)
      const float down =
          fmaxf(__uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) * p.scale_log2, 4.70197740e-38f);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) bq[nt][i] = pack_f16x2(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // this lane's score columns are rows 2t and 2t + 1
        sc[nt][c] = __shfl_sync(0xffffffffu, down, 4 * (2 * t + c));
      }
    }
    lim_lo = __reduce_min_sync(0xffffffffu, lim_lo);
    seen = __reduce_max_sync(0xffffffffu, seen);

    // thr: the unscaled score that moves the maximum, base: what is subtracted
    // from the scaled ones (the maximum less the weights' 2^6)
    float o[NT][MT][4], thr[NT][2], base[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      thr[nt][0] = thr[nt][1] = kMinusInf;
      base[nt][0] = base[nt][1] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
    }

    // N blocks of the piece, from its block i on (i, i + 4, ..)
    auto step = [&](int i, auto blocks) {
      constexpr int N = decltype(blocks)::value;
      float s[N][NT][4];
      uint32_t at[N];
#pragma unroll
      for (int x = 0; x < N; ++x) at[x] = x == 0 ? stage : after(at[x - 1]);
      copy_wait<S - N>();
      __syncwarp();  // the scales came by other lanes' copies
      // ---- S^T = K Q^T
#pragma unroll
      for (int x = 0; x < N; ++x) {
        const uint32_t st = at[x];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[x][nt][0] = s[x][nt][1] = s[x][nt][2] = s[x][nt][3] = 0.f;
        uint32_t wa[KW], wb[KW];
        lds_words(wa, ring_c + st);
        lds_words(wb, ring_c + st + CB);
        const uint32_t sw = lds_u32(ring_ks + st);
        uint32_t sa[2], sb[2];  // scales of rows g and g + 8, doubled, for the lane's first and second 16 elements
        if constexpr (D == 128) {
          const uint32_t a = e4m3x2_to_f16(sw), b = e4m3x2_to_f16(sw >> 16);
          sa[0] = __byte_perm(a, 0, 0x1010);
          sa[1] = __byte_perm(a, 0, 0x3232);
          sb[0] = __byte_perm(b, 0, 0x1010);
          sb[1] = __byte_perm(b, 0, 0x3232);
        } else {
          const uint32_t a = e4m3x2_to_f16(sw >> (16 * (lane & 1)));
          sa[0] = sa[1] = __byte_perm(a, 0, 0x1010);
          sb[0] = sb[1] = __byte_perm(a, 0, 0x3232);
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t a[4], b[4];
          e2m1x8_to_f16(wa[w], a);
          e2m1x8_to_f16(wb[w], b);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            a[y] = hmul2(a[y], sa[w / 2]);
            b[y] = hmul2(b[y], sb[w / 2]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y)  // contraction step 2w + y
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_16816(s[x][nt], a[2 * y], b[2 * y], a[2 * y + 1], b[2 * y + 1], bq[nt][4 * w + 2 * y],
                            bq[nt][4 * w + 2 * y + 1]);
        }
      }
      // ---- weights: score c of a tile is column c & 1 (row 2t + (c & 1)), key g + 8 (c >> 1)
      const int key0 = (cj + i) * kQ4Block;
      const bool edge = key0 + (N - 1) * kWarps * kQ4Block + kQ4Block - 1 > lim_lo;
      if (edge) {
#pragma unroll
        for (int x = 0; x < N; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int lim = __shfl_sync(0xffffffffu, qpos[nt], 4 * (2 * t + (c & 1)));
              if (key0 + x * kWarps * kQ4Block + g + 8 * (c >> 1) > lim) s[x][nt][c] = kMinusInf;
            }
      }
      float mx[NT][2];
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[nt][c] = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
          for (int x = 1; x < N; ++x) mx[nt][c] = fmax3(mx[nt][c], s[x][nt][c], s[x][nt][c + 2]);
          above |= mx[nt][c] > thr[nt][c];
        }
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = mx[nt][c];
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, y));
            // (v, thr and base are the same in every lane of the column)
            const float step_up = __fdividef(kMaxStep, sc[nt][c]);
            if (!(v > thr[nt][c] - step_up) && v == v) continue;  // not above the maximum (or nothing of this row yet)
            const float nb = v * sc[nt][c] - kWeightBias;
            const float a = thr[nt][c] == kMinusInf ? 0.f : fast_exp2(base[nt][c] - nb);
            thr[nt][c] = v + step_up;
            base[nt][c] = nb;
            l[nt][c] *= a;
#pragma unroll
            for (int y = 0; y < MT; ++y) {
              o[nt][y][c] *= a;
              o[nt][y][c + 2] *= a;
            }
          }
        __syncwarp();
      }
      uint32_t pw[N][NT][2];
#pragma unroll
      for (int x = 0; x < N; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            e[c] = fast_exp2(fmaf(s[x][nt][c], sc[nt][c & 1], -base[nt][c & 1]));
            l[nt][c & 1] += e[c];
          }
          pw[x][nt][0] = transpose8x8(pack_f16x2(e[0], e[1]));
          pw[x][nt][1] = transpose8x8(pack_f16x2(e[2], e[3]));
        }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int x = 0; x < N; ++x) {
        const uint32_t st = at[x];
        uint32_t v0[KW], v1[KW];
        lds_words(v0, ring_c + st + 2 * CB);
        lds_words(v1, ring_c + st + 3 * CB);
        const uint32_t sw = lds_u32(ring_vs + st);
        uint32_t s0 = e4m3x2_to_f16(sw), s1 = e4m3x2_to_f16(sw >> 16);
        const int k0 = key0 + x * kWarps * kQ4Block;
        if (edge && k0 + kQ4Block > seen) {  // tokens that no row sees may never have been written: any bytes, NaN scales
          const int k = k0 + 2 * t;
          s0 = (k < seen ? s0 & 0xFFFFu : 0u) | (k + 1 < seen ? s0 & 0xFFFF0000u : 0u);
          s1 = (k + 8 < seen ? s1 & 0xFFFFu : 0u) | (k + 9 < seen ? s1 & 0xFFFF0000u : 0u);
        }
#pragma unroll
        for (int w = 0; w < KW / 2; ++w) {
          // bytes of two tokens' codes of one element: even elements, odd elements
          uint32_t e0[4], d0[4], e1[4], d1[4];
          e2m1x8_to_f16(select_bits<0x0F0F0F0Fu>(v0[w], v0[w + KW / 2] << 4), e0);
          e2m1x8_to_f16(select_bits<0x0F0F0F0Fu>(v0[w] >> 4, v0[w + KW / 2]), d0);
          e2m1x8_to_f16(select_bits<0x0F0F0F0Fu>(v1[w], v1[w + KW / 2] << 4), e1);
          e2m1x8_to_f16(select_bits<0x0F0F0F0Fu>(v1[w] >> 4, v1[w + KW / 2]), d1);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t a0 = hmul2(e0[y], s0), a1 = hmul2(d0[y], s0), a2 = hmul2(e1[y], s1), a3 = hmul2(d1[y], s1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][4 * w + y], a0, a1, a2, a3, pw[x][nt][0], pw[x][nt][1]);
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < N; ++x) issue(at[x]);  // the stages just read take the next blocks
      stage = after(at[N - 1]);
    };
    // the warp's blocks of the piece: range indices congruent to warp
    constexpr int kStep = 2;
    int i = (warp - first) & (kWarps - 1);
    for (; i + (kStep - 1) * kWarps < n; i += kStep * kWarps) step(i, std::integral_constant<int, kStep>{});
    if (kStep > 1 && i < n) step(i, std::integral_constant<int, 1>{});

    // ---- the warps' states of the piece, joined in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = l[nt][c];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
        const int r = nt * 8 + 2 * t + c;
        if (g == 0) mlbuf[warp * ROWS + r] = make_float2(thr[nt][c] == kMinusInf ? kMinusInf : base[nt][c] + kWeightBias, v);
        float* dst = obuf + (warp * ROWS + r) * D + g * W;
#pragma unroll
        for (int y = 0; y < MT; y += 2)
          *reinterpret_cast<float4*>(dst + 2 * y) =
              make_float4(o[nt][y][c], o[nt][y][c + 2], o[nt][y + 1][c], o[nt][y + 1][c + 2]);
      }
    }
    const bool whole = cj == 0 && n == nblk;
    const int slot = cj == 0 ? 1 : 0;  // a piece that begins here, or one continued from the CTA before
    if (threadIdx.x == 0 && cj == 0 && (n < nblk || p.cut_by_piece))
      p.cut[p.cut_by_piece ? cb * p.nkv + ch : blockIdx.x] =
          Cut{static_cast<int>(blockIdx.x), n < nblk ? split.cta_of(unit + kPieceCost + nblk - 1) : -1, t0, rows, len, ch,
              {0, 0}};
    const int out_t0 = t0, out_rows = rows, out_len = len, out_h = ch;
    left -= n;
    first += n;
    unit += nblk + kPieceCost;
    cj = 0;
    if (left > 0) {  // (8 rows: the next piece's are on their way while this one is stored; 16 take too many registers)
      if (++ch == p.nkv) {
        ch = 0;
        do ++cb;
        while (plan_blocks(p, cb) == 0);
      }
      if (NT == 1) load_q();
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < out_rows * (D / 4); idx += kThreads) {
      const int r = idx / (D / 4), c4 = (idx % (D / 4)) * 4;
      float M = kMinusInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mlbuf[w * ROWS + r].x);
      const float mb = M == kMinusInf ? 0.f : M;
      float L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = mlbuf[w * ROWS + r];
        const float f = fast_exp2(ml.x - mb);
        const float4 x = *reinterpret_cast<const float4*>(obuf + (w * ROWS + r) * D + c4);
        L += ml.y * f;
        O.x += x.x * f;
        O.y += x.y * f;
        O.z += x.z * f;
        O.w += x.w * f;
      }
      if (whole) {
        const int tok = out_t0 + r / p.group;
        const int pos = p.positions[tok];
        if (pos < 0 || pos >= out_len) {
          if (out_h == 0 && c4 == 0) report_error(p.err, kErrGuard, kWhereQueryLen);
          continue;
        }
        const float inv = p.v_scale / L;
        uint2 u;
        u.x = pack_bf16x2(O.x * inv, O.y * inv);
        u.y = pack_bf16x2(O.z * inv, O.w * inv);
        *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(tok) * p.nq + out_h * p.group + r % p.group) * D + c4) =
            u;
      } else {
        const size_t at = (static_cast<size_t>(blockIdx.x) * 2 + slot) * kMaxRows + r;
        *reinterpret_cast<float4*>(p.part_o + at * D + c4) = O;
        if (c4 == 0) p.part_ml[at] = make_float2(M, L);
      }
    }
    __syncthreads();
  }
  copy_wait<0>();
}

// Joins the parts of every piece that spans CTAs, in order: 4 to 8 us, reading what the
// decode kernel just wrote (4 KB a part and 8 rows) from L2, a chain of dependent
// loads.  (Joining in the decode kernel, by the last CTA of a piece to end: 124
// instead of 120 us for 128 sequences, 78 instead of 55 for four long ones.)  Up to
// as many pieces as decode CTAs: one entry of `cut` per piece and grid.y CTAs share its rows,
// so that a few long pieces have many warps; beyond that one entry per decode CTA
// (the piece that begins in it and ends in a later one).  It lets no later kernel
// start early: CTAs of a next call's decode kernel that came one by one into
// freed slots would not be ranked by their SM (128-sequence batch 135 us instead
// of 122).
constexpr int kCombineWarps = 16;
constexpr int kCombineBatch = 2;  // parts a warp loads at once (four take registers that keep its CTAs out of the
                                  // SMs beside prefill CTAs: 226 instead of 220 us for the mixed batch)

template <int D>
__global__ void __launch_bounds__(kCombineWarps * 32) k_attn_q4_combine(const Q4Params p) {
  __shared__ float so[kCombineWarps][D];
  __shared__ float2 sml[kCombineWarps];
  pdl_wait();
  const Cut cut = p.cut[blockIdx.x];
  // (an entry per piece is written for the sequences of this launch only)
  if (p.cut_by_piece && plan_blocks(p, blockIdx.x / p.nkv) == 0) return;
  if (cut.last < 0) return;
  const int rows = cut.rows, parts = cut.last - cut.first + 1;
  const int gy = gridDim.y, y = blockIdx.y;
  const int mine = y < rows ? (rows - y + gy - 1) / gy : 0;  // rows y, y + gy, ...
  if (mine == 0) return;
  const int wpr = mine <= 1 ? 16 : mine <= 2 ? 8 : mine <= 4 ? 4 : mine <= 8 ? 2 : 1;  // warps a row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = y + (warp / wpr) * gy, sub = warp % wpr;
  constexpr int E = D / 32;
  float M = kMinusInf, L = 0.f, O[E];
#pragma unroll
  for (int e = 0; e < E; ++e) O[e] = 0.f;
  const int tok = cut.t0 + r / p.group;
  int pos = -1;
  if (r < rows) {
    pos = p.positions[tok];
    for (int i0 = sub; i0 < parts; i0 += wpr * kCombineBatch) {
      float2 ml[kCombineBatch];
      float x[kCombineBatch][E];
#pragma unroll
      for (int n = 0; n < kCombineBatch; ++n) {
        const int i = i0 + n * wpr;
        ml[n] = make_float2(kMinusInf, 0.f);
#pragma unroll
        for (int e = 0; e < E; ++e) x[n][e] = 0.f;
        if (i < parts) {
          const size_t at = (static_cast<size_t>(cut.first + i) * 2 + (i == 0 ? 1 : 0)) * kMaxRows + r;
          ml[n] = p.part_ml[at];
          const float* src = p.part_o + at * D + lane * E;
          if constexpr (E == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            x[n][0] = v.x, x[n][1] = v.y, x[n][2] = v.z, x[n][3] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            x[n][0] = v.x, x[n][1] = v.y;
          }
        }
      }
      float m = M;
#pragma unroll
      for (int n = 0; n < kCombineBatch; ++n) m = fmaxf(m, ml[n].x);
      const float mb = m == kMinusInf ? 0.f : m, a = fast_exp2(M - mb);
      M = m;
      L *= a;
#pragma unroll
      for (int e = 0; e < E; ++e) O[e] *= a;
#pragma unroll
      for (int n = 0; n < kCombineBatch; ++n) {
        const float f = fast_exp2(ml[n].x - mb);
        L += ml[n].y * f;
#pragma unroll
        for (int e = 0; e < E; ++e) O[e] += x[n][e] * f;
      }
    }
  }
  if (wpr > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = O[e];
    if (lane == 0) sml[warp] = make_float2(M, L);
    __syncthreads();
    if (sub != 0) return;
    float m = M;
    for (int w = 1; w < wpr; ++w) m = fmaxf(m, sml[warp + w].x);
    const float mb = m == kMinusInf ? 0.f : m, a = fast_exp2(M - mb);
    L *= a;
#pragma unroll
    for (int e = 0; e < E; ++e) O[e] *= a;
    for (int w = 1; w < wpr; ++w) {
      const float2 ml = sml[warp + w];
      const float f = fast_exp2(ml.x - mb);
      L += ml.y * f;
#pragma unroll
      for (int e = 0; e < E; ++e) O[e] += so[warp + w][lane * E + e] * f;
    }
  }
  if (r >= rows) return;
  if (pos < 0 || pos >= cut.len) {
    if (cut.h == 0 && lane == 0) report_error(p.err, kErrGuard, kWhereQueryLen);
    return;
  }
  const float inv = p.v_scale / L;
  uint32_t* dst = reinterpret_cast<uint32_t*>(
      p.out + (static_cast<size_t>(tok) * p.nq + cut.h * p.group + r % p.group) * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(O[e] * inv, O[e + 1] * inv);
}

// ---------------------------------------------------------------------------
// longer sequences
// ---------------------------------------------------------------------------
struct PrefillQ4 {
  const int32_t *qsl, *seq_lens, *positions, *block_table;
  int T, B, max_blocks, num_blocks, nkv, group, max_query_len, max_seq_len, prefill_blocks;
  int tile_tokens, max_items, stride;
  int32_t* base;    // [B + 1] blocks of the copy before each sequence; then the length of the work list
  uint32_t* items;  // the prefill kernels' work list
  int32_t* table;   // [B, stride] block table of the copy
  const uint8_t *k_cache, *v_cache;
  __nv_bfloat16 *k_copy, *v_copy;  // [prefill_blocks, nkv, 16, D]
  float k_scale, v_scale;
  int* err;
};

// inclusive sum of v over the CTA, and the whole sum
__device__ __forceinline__ long long cta_scan(long long v, long long* tot, long long& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) tot[warp] = v;
  __syncthreads();
  long long before = 0;
  all = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    if (w < warp) before += tot[w];
    all += tot[w];
  }
  return before + v;
}

// Blocks of sequence b on the prefill path (n new tokens); 0 if it takes the decode path or is out of bounds (*bad).
__device__ __forceinline__ long long prefill_seq_blocks(const PrefillQ4& p, int b, int& n, bool& bad) {
  const int t0 = p.qsl[b], len = p.seq_lens[b];
  n = p.qsl[b + 1] - t0;
  bad = false;
  if (n <= 1 || (n <= kMaxRows && n * p.group <= kMaxRows)) return 0;
  const long long blocks = (static_cast<long long>(len) + kQ4Block - 1) / kQ4Block;
  bad = n > p.max_query_len || t0 < 0 || t0 > p.T - n || len < 1 || len > p.max_seq_len || blocks > p.max_blocks;
  return bad ? 0 : blocks;
}

// One CTA: where each prefill sequence's blocks go in the copy, and its query
// tiles (longest causal range first within a sequence).  A sequence that is out
// of bounds or does not fit the copy is reported and left out.
__device__ __forceinline__ void plan_prefill(const PrefillQ4& p, long long* tot) {
  long long blocks_before = 0, items_before = 0, all;
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    long long blocks = 0;
    if (b < p.B) {
      bool bad;
      blocks = prefill_seq_blocks(p, b, n, bad);
      // n > max_query_len and t0 are reported by the decode kernel, which looks at every sequence
      if (bad && n <= p.max_query_len) report_error(p.err, kErrGuard, kWhereQueryLen);
    }
    const long long base = blocks_before + cta_scan(blocks, tot, all) - blocks;
    blocks_before += all;
    int tiles = 0;
    if (blocks > 0) {
      if (base + blocks > p.prefill_blocks)
        report_error(p.err, kErrGuard, kWhereQueryLen);
      else
        tiles = (n + p.tile_tokens - 1) / p.tile_tokens;
    }
    if (b < p.B) p.base[b] = static_cast<int32_t>(base < p.prefill_blocks ? base : p.prefill_blocks);
    const long long item = items_before + cta_scan(tiles, tot, all) - tiles;
    items_before += all;
    if (item + tiles > p.max_items) report_error(p.err, kErrGuard, kWhereQueryLen);  // (sequences that overlap)
    for (int j = 0; j < tiles; ++j)
      if (item + j < p.max_items)
        p.items[item + j] = (static_cast<uint32_t>(b) << 16) | static_cast<uint32_t>(tiles - 1 - j);
  }
  if (threadIdx.x == 0) {
    p.base[p.B] = static_cast<int32_t>(blocks_before < p.prefill_blocks ? blocks_before : p.prefill_blocks);
    p.base[p.B + 1] = static_cast<int32_t>(items_before < p.max_items ? items_before : p.max_items);
  }
  for (long long i = items_before + threadIdx.x; i < p.max_items; i += blockDim.x) p.items[i] = kNoPrefillItem;
}

__global__ void __launch_bounds__(1024) k_attn_q4_plan(const PrefillQ4 p) {
  __shared__ long long tot[32];
  pdl_wait();
  pdl_trigger();
  plan_prefill(p, tot);
}

// CTA (x, y): K (y = 0) or V of all KV heads of block x of the copy in bf16
// (exact), zero past the sequence's end; and the block's entry in the copy's table.
// 256 blocks of 8 heads x 128: 9.2 us for 21 MB, launch and look-up included.
// Bad positions of the sequence's tokens are reported here, by the CTAs of its
// first blocks (the prefill kernels look at the largest of a tile only).
//   PLANNED: after k_attn_q4_plan.  Else, with up to kScanSeqs sequences, every CTA
// finds its sequence itself and one more makes the plan: a launch less, and the
// expansion starts before the decode kernels fill the SMs (mixed batch above: 215
// us with the plan and the decode kernels before it, 212 so; a batch of 80 new tokens
// 20.7 and 17.5).
constexpr int kScanSeqs = 512;
constexpr int kExpandThreads = 256;

template <int D, bool V>
__device__ __forceinline__ void expand_block(const PrefillQ4& p, int s, int blk, int tokens) {
  // chunks of 8 elements, (head, token, chunk); kUnroll of a thread's loads in flight at once
  constexpr int C = D / 8, kUnroll = 4;
  const int total = p.nkv * kQ4Block * C;
  const uint8_t* tiles = (V ? p.v_cache : p.k_cache) + static_cast<size_t>(blk) * p.nkv * q4_tile_bytes(D);
  uint4* dst = reinterpret_cast<uint4*>((V ? p.v_copy : p.k_copy) + static_cast<size_t>(s) * p.nkv * kQ4Block * D);
  const float g = V ? p.v_scale : p.k_scale;
  for (int i0 = threadIdx.x; i0 < total; i0 += kExpandThreads * kUnroll) {
    uint32_t code[kUnroll], s8[kUnroll];
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
      const int i = min(i0 + n * kExpandThreads, total - 1);
      const int c = i % C, k = (i / C) % kQ4Block;
      const uint8_t* tile = tiles + (i / (C * kQ4Block)) * q4_tile_bytes(D);
      code[n] = *reinterpret_cast<const uint32_t*>(tile + q4_code_at<D>(V, k, c));
      s8[n] = k < tokens ? tile[q4_scale_at<D>(V, k, c >> 1)] : 0u;  // (unwritten tokens: any bytes; codes are finite)
    }
#pragma unroll
    for (int n = 0; n < kUnroll; ++n)
      if (i0 + n * kExpandThreads < total) dst[i0 + n * kExpandThreads] = q4_to_bf16(code[n], s8[n], g);
  }
}

template <int D, bool PLANNED>
__global__ void __launch_bounds__(kExpandThreads) k_q4_expand(const PrefillQ4 p) {
  __shared__ long long tot[kExpandThreads / 32];
  __shared__ int found[2];  // block s's sequence and its block there
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x;
  int b, j;
  if constexpr (PLANNED) {
    if (s >= p.base[p.B]) return;
    int upto = 0;  // sequences whose blocks begin at or before s: the last of them holds it
    for (int b0 = 0; b0 < p.B; b0 += kExpandThreads) {
      const int i = b0 + threadIdx.x;
      upto += __syncthreads_count(i < p.B && p.base[i] <= s);
    }
    b = upto - 1;
    j = s - p.base[b];
  } else {
    if (s == p.prefill_blocks) {
      if (blockIdx.y == 0) plan_prefill(p, tot);
      return;
    }
    if (threadIdx.x == 0) found[0] = -1;
    long long before = 0, all;
    for (int b0 = 0; b0 < p.B; b0 += kExpandThreads) {
      const int i = b0 + threadIdx.x;
      int n;
      bool bad;
      const long long blocks = i < p.B ? prefill_seq_blocks(p, i, n, bad) : 0;
      const long long base = before + cta_scan(blocks, tot, all) - blocks;
      before += all;
      if (base <= s && s < base + blocks) {
        found[0] = i;
        found[1] = static_cast<int>(s - base);
      }
      if (before > s) break;
    }
    __syncthreads();
    b = found[0];
    j = found[1];
    if (b < 0) return;
  }
  const int len = p.seq_lens[b];
  if (j >= p.stride || j * kQ4Block >= len) return;
  if (blockIdx.y == 0) {
    if (threadIdx.x == 0) p.table[static_cast<size_t>(b) * p.stride + j] = s;
    const int t0 = p.qsl[b], n = p.qsl[b + 1] - t0;
    const long long step = static_cast<long long>((len + kQ4Block - 1) / kQ4Block) * kExpandThreads;
    for (long long i = static_cast<long long>(j) * kExpandThreads + threadIdx.x; i < n; i += step) {
      const int pos = p.positions[t0 + i];
      if (pos < 0 || pos >= len) report_error(p.err, kErrGuard, kWhereQueryLen);
    }
  }
  int blk = p.block_table[static_cast<size_t>(b) * p.max_blocks + j];
  if (blk < 0 || blk >= p.num_blocks) {
    if (threadIdx.x == 0) report_error(p.err, kErrGuard, kWhereBlockTable);
    blk = 0;
  }
  if (blockIdx.y)
    expand_block<D, true>(p, s, blk, len - j * kQ4Block);
  else
    expand_block<D, false>(p, s, blk, len - j * kQ4Block);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int D, int NT>
size_t decode_smem() {
  constexpr int S = stages<D>(), ROWS = 8 * NT;
  return static_cast<size_t>(kWarps) * S * (4 * (32 * D / 8) + 2 * 128) + kWarps * ROWS * D * 4 + kWarps * ROWS * 8;
}

struct Layout {
  size_t part_o, part_ml, cut, base, items, table, k_copy, v_copy, parts, total;
  int grid, max_items, stride;
};

Layout layout(int T, int B, int max_seq_len, int prefill_blocks, int nkv, int head_dim) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  Layout L{};
  L.grid = num_sms() * kCtasPerSm;
  L.max_items = (T + 7) / 8 + B;
  L.stride = (max_seq_len + kQ4Block - 1) / kQ4Block;
  const size_t rows = static_cast<size_t>(L.grid) * 2 * kMaxRows;
  size_t off = 0;
  L.part_o = off;
  off += up(rows * head_dim * sizeof(float));
  L.part_ml = off;
  off += up(rows * sizeof(float2));
  L.cut = off;
  off += up(static_cast<size_t>(L.grid) * sizeof(Cut));
  if (prefill_blocks > 0) {
    const size_t copy = up(static_cast<size_t>(prefill_blocks) * nkv * kQ4Block * head_dim * 2);
    L.table = off;
    off += up(static_cast<size_t>(B) * L.stride * 4);
    L.k_copy = off;
    off += copy;
    L.v_copy = off;
    off += copy;
    L.parts = off;
    off += up(prefill_split_bytes(head_dim));
  }
  L.base = off;
  off += up((static_cast<size_t>(B) + 2) * 4);
  L.items = off;
  off += up(static_cast<size_t>(L.max_items) * 4);
  L.total = off;
  return L;
}

// The sequences of rows_lo .. rows_hi query rows.  alone: nothing else runs beside the kernel, so that its CTAs fill the
// SMs in turn (see Split).
template <int D, int NT>
int launch_decode(Q4Params p, int rows_lo, int rows_hi, bool alone, bool pdl, cudaStream_t s) {
  constexpr int ctas_per_sm = NT == 1 ? kCtasPerSm : 3;
  static SmemLimits limits;
  const cudaError_t attr = limits.raise({smem_need(k_attn_q4_decode<D, NT>, decode_smem<D, NT>())});
  if (attr != cudaSuccess) return attr;
  p.rows_lo = rows_lo;
  p.rows_hi = rows_hi;
  const long long pieces = static_cast<long long>(p.B) * p.nkv;
  const long long want = pieces * ((p.max_seq_len + kQ4Block - 1) / kQ4Block + kPieceCost) / kMinShare + 1;
  const int full = num_sms() * ctas_per_sm, grid = want < full ? static_cast<int>(want) : full;
  p.sms = alone ? num_sms() : grid;
  // Few short pieces are not split: finding the ranges and joining the parts cost about as much as kWholeBlocks blocks
  // (one sequence of 777 tokens, from a graph: 7.6 us split into 13 CTAs and joined, 6.9 whole, with one launch not two).
  // Beside prefill kernels, which take longer, four times as many.
  p.whole = pieces <= full && (p.max_seq_len + kQ4Block - 1) / kQ4Block <= (alone ? 1 : 4) * kWholeBlocks;
  if (p.whole)
    return launch_kernel(k_attn_q4_decode<D, NT>, dim3(static_cast<unsigned>(pieces)), dim3(kThreads),
                         decode_smem<D, NT>(), s, pdl, p);
  p.cut_by_piece = pieces <= grid;
  const cudaError_t e =
      launch_kernel(k_attn_q4_decode<D, NT>, dim3(grid), dim3(kThreads), decode_smem<D, NT>(), s, pdl, p);
  if (e != cudaSuccess) return e;
  dim3 join(grid);
  if (p.cut_by_piece) {
    const int per_piece = static_cast<int>(num_sms() / pieces);
    join = dim3(static_cast<unsigned>(pieces), per_piece < 1 ? 1 : per_piece > 8 * NT ? 8 * NT : per_piece);
  }
  return launch_kernel(k_attn_q4_combine<D>, join, dim3(kCombineWarps * 32), 0, s, true, p);
}

template <int D>
int launch_d(const AttnQ4Args& q4, const Q4Params& p, const Layout& L, cudaStream_t s) {
  const AttnArgs& a = q4.a;
  const int mq = a.max_query_len;
  if (mq <= 1 || (mq <= kMaxRows && mq * p.group <= kMaxRows))  // every sequence takes the decode path
    return max(mq, 1) * p.group <= 8 ? launch_decode<D, 1>(p, 1, 8, true, true, s)
                                     : launch_decode<D, 2>(p, 1, kMaxRows, true, true, s);

  // Longer sequences too: the decode kernels (bound by HBM) run on the side stream beside the expansion and the
  // prefill kernel (bound by its softmax and the tensor cores).
  PrefillQ4 f{};
  f.T = a.T;
  f.qsl = a.qsl;
  f.seq_lens = a.seq_lens;
  f.positions = a.positions;
  f.block_table = a.block_table;
  f.B = a.B;
  f.max_query_len = mq;
  f.max_blocks = a.max_blocks;
  f.num_blocks = a.num_blocks;
  f.nkv = a.nkv;
  f.group = p.group;
  f.max_seq_len = a.max_seq_len;
  f.prefill_blocks = q4.prefill_blocks;
  f.tile_tokens = prefill_tile_tokens(a);
  f.max_items = (a.T + f.tile_tokens - 1) / f.tile_tokens + min(a.B, q4.prefill_blocks);  // (a block a sequence at least)
  f.stride = L.stride;
  f.base = reinterpret_cast<int32_t*>(q4.ws + L.base);
  f.items = reinterpret_cast<uint32_t*>(q4.ws + L.items);
  f.table = reinterpret_cast<int32_t*>(q4.ws + L.table);
  f.k_cache = p.k_cache;
  f.v_cache = p.v_cache;
  f.k_copy = reinterpret_cast<__nv_bfloat16*>(q4.ws + L.k_copy);
  f.v_copy = reinterpret_cast<__nv_bfloat16*>(q4.ws + L.v_copy);
  f.k_scale = q4.k_scale;
  f.v_scale = q4.v_scale;
  f.err = a.err;
  SideStream* const forked = side_fork(s);
  const cudaStream_t side = forked ? forked->stream : s;
  int e;
  if (q4.prefill_blocks == 0 || a.B > kScanSeqs) {
    e = launch_kernel(k_attn_q4_plan, dim3(1), dim3(a.B < 1024 ? (a.B + 31) / 32 * 32 : 1024), 0, s, side == s, f);
    if (e == 0 && q4.prefill_blocks > 0)
      e = launch_kernel(k_q4_expand<D, true>, dim3(q4.prefill_blocks, 2), dim3(kExpandThreads), 0, s, true, f);
  } else {
    e = launch_kernel(k_q4_expand<D, false>, dim3(q4.prefill_blocks + 1, 2), dim3(kExpandThreads), 0, s, side == s, f);
  }
  // Few blocks in all: one launch for 1 .. 16 rows, not one of 8 and one of 16 rows (eight sequences each of one and of two
  // tokens beside a chunk of 64, 64 / 8 heads x 128, 8568 blocks: 19.5 us, with two 34.5; 8 / 2 x 64, 8500 blocks: 25 and
  // 23).  Many blocks of single tokens are the 8-row kernel's (262144: 60 us, the 16-row kernel takes 80 for two tokens).
  const bool few = static_cast<long long>(a.B) * a.nkv * L.stride <= kFewBlocks;
  if (e == 0) {
    if (p.group > 8 || few) {
      e = launch_decode<D, 2>(p, 1, kMaxRows, false, false, side);
    } else {
      e = launch_decode<D, 1>(p, 1, 8, false, false, side);
      if (e == 0) e = launch_decode<D, 2>(p, 9, kMaxRows, false, true, side);
    }
  }
  if (e == 0 && q4.prefill_blocks > 0) {
    AttnArgs c = a;
    c.k_cache = f.k_copy;
    c.v_cache = f.v_copy;
    c.block_table = f.table;
    c.max_blocks = L.stride;
    c.num_blocks = q4.prefill_blocks;
    e = prefill_items_launch(c, f.items, f.max_items, f.base + a.B + 1, q4.ws + L.parts, side != s, s);
  }
  if (forked) {  // join even after a failed launch, so that the caller's stream never runs ahead of the side stream
    const int j = side_join(s, forked);
    if (e == 0) e = j;
  }
  return e;
}

}  // namespace

size_t attn_q4_workspace_bytes(int T, int B, int max_seq_len, int prefill_blocks, int nkv, int head_dim) {
  return layout(T, B, max_seq_len, prefill_blocks, nkv, head_dim).total;
}

int attention_q4_launch(const AttnQ4Args& q4, cudaStream_t s) {
  const AttnArgs& a = q4.a;
  if (a.T <= 0 || a.B <= 0) return 0;
  const Layout L = layout(a.T, a.B, a.max_seq_len, q4.prefill_blocks, a.nkv, a.head_dim);
  Q4Params p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.qsl = a.qsl;
  p.seq_lens = a.seq_lens;
  p.positions = a.positions;
  p.block_table = a.block_table;
  p.T = a.T;
  p.B = a.B;
  p.max_query_len = a.max_query_len;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.nq = a.nq;
  p.nkv = a.nkv;
  p.group = a.nq / a.nkv;
  p.max_seq_len = a.max_seq_len;
  p.scale_log2 = kLog2e / sqrtf(static_cast<float>(a.head_dim)) * q4.k_scale;
  p.v_scale = q4.v_scale;
  p.part_o = reinterpret_cast<float*>(q4.ws + L.part_o);
  p.part_ml = reinterpret_cast<float2*>(q4.ws + L.part_ml);
  p.cut = reinterpret_cast<Cut*>(q4.ws + L.cut);
  p.err = a.err;
  return a.head_dim == 128 ? launch_d<128>(q4, p, L, s) : launch_d<64>(q4, p, L, s);
}

}  // namespace llama
