// Paged, causal, grouped-query attention over a KV cache held in 4 bits.
//
//   o[t, h] = sum_j softmax_j(q[t, h] . K[b, h / g, j] / sqrt(d)) V[b, h / g, j],
//   j = 0 .. position(t), K and V the values of the 4-bit tiles (q4.cuh)
//
// One CTA per (token, KV head): its four warps take the keys in turn, a lane
// D / 32 neighbouring elements, with an online softmax per warp and query head;
// the warps' states are merged in shared memory.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q4.cuh"

namespace llama {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;
constexpr int kHeads = 4;  // query heads at a time

struct Q4Params {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const uint8_t *k_cache, *v_cache;
  const int32_t *qsl, *seq_lens, *positions, *block_table;
  int T, B, max_blocks, num_blocks, nq, nkv, group, max_seq_len;
  float scale_log2, v_scale;
  int* err;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) k_attn_q4(const Q4Params p) {
  constexpr int E = D / 32;
  __shared__ float sm[kWarps][kHeads], sl[kWarps][kHeads], so[kWarps][kHeads][D];
  const int t = blockIdx.x, kvh = blockIdx.y;
  if (t >= p.qsl[p.B]) return;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.qsl[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int b = lo, n_keys = p.positions[t] + 1;
  if (n_keys < 1 || n_keys > p.seq_lens[b] || n_keys > p.max_seq_len || (n_keys + 15) / 16 > p.max_blocks) {
    if (kvh == 0 && threadIdx.x == 0) report_error(p.err, kErrGuard, kWhereQueryLen);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e0 = lane * E;
  for (int h0 = 0; h0 < p.group; h0 += kHeads) {
    float q[kHeads][E], o[kHeads][E], m[kHeads], l[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[i][e] = 0.f;
        q[i][e] = h0 + i < p.group ? __bfloat162float(p.q[(static_cast<size_t>(t) * p.nq + kvh * p.group + h0 + i) * D +
                                                          e0 + e])
                                   : 0.f;
      }
    }
    for (int j = warp; j < n_keys; j += kWarps) {
      int blk = p.block_table[static_cast<size_t>(b) * p.max_blocks + j / 16];
      if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0) report_error(p.err, kErrGuard, kWhereBlockTable);
        blk = 0;
      }
      const size_t at = (static_cast<size_t>(blk) * p.nkv + kvh) * q4_tile_bytes(D);
      const uint8_t *kt = p.k_cache + at, *vt = p.v_cache + at;
      const int k = j % 16;
      float kv[E], vv[E];
      const float ks = f16_lo(e4m3x2_to_f16(kt[q4_k_scale_at<D>(k, e0 / 16)]));
      const float vs = f16_lo(e4m3x2_to_f16(vt[q4_v_scale_at<D>(k, e0 / 16)]));
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        uint32_t h[4];
        e2m1x8_to_f16(kt[k * (D / 2) + (e0 + e) / 2] | (vt[q4_v_code_at<D>(k, e0 + e)] << 8), h);
        kv[e] = f16_lo(h[0]) * ks;
        kv[e + 1] = f16_hi(h[0]) * ks;
        vv[e] = f16_lo(h[1]) * vs;
        vv[e + 1] = f16_hi(h[1]) * vs;
      }
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[i][e], kv[e], s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale_log2;
        const float n = fmaxf(m[i], s), a = exp2f(m[i] - n), w = exp2f(s - n);
        m[i] = n;
        l[i] = l[i] * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = o[i][e] * a + w * vv[e];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (lane == 0) {
        sm[warp][i] = m[i];
        sl[warp][i] = l[i];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) so[warp][i][e0 + e] = o[i][e];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < kHeads * D; x += kWarps * 32) {
      const int i = x / D, e = x % D;
      if (h0 + i >= p.group) continue;
      float M = -INFINITY, L = 0.f, O = 0.f;
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][i]);
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(sm[w][i] - M);
        L += sl[w][i] * f;
        O += so[w][i][e] * f;
      }
      p.out[(static_cast<size_t>(t) * p.nq + kvh * p.group + h0 + i) * D + e] = __float2bfloat16_rn(O / L * p.v_scale);
    }
  }
}

}  // namespace

size_t attn_q4_workspace_bytes(int, int, int, int, int, int, int) { return 256; }

int attention_q4_launch(const AttnQ4Args& q4, cudaStream_t s) {
  const AttnArgs& a = q4.a;
  if (a.T <= 0 || a.B <= 0) return 0;
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
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.nq = a.nq;
  p.nkv = a.nkv;
  p.group = a.nq / a.nkv;
  p.max_seq_len = a.max_seq_len;
  p.scale_log2 = kLog2e / sqrtf(static_cast<float>(a.head_dim)) * q4.k_scale;
  p.v_scale = q4.v_scale;
  p.err = a.err;
  const dim3 grid(a.T, a.nkv);
  if (a.head_dim == 128) return launch_kernel(k_attn_q4<128>, grid, dim3(kWarps * 32), 0, s, false, p);
  return launch_kernel(k_attn_q4<64>, grid, dim3(kWarps * 32), 0, s, false, p);
}

}  // namespace llama
