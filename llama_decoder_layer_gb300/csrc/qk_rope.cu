// RMS norm of every query and key head, and the rotary position embedding, in
// one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w           (per head row of D elements)
//   (y_a, y_b) <- f * (y_a cos - y_b sin, y_b cos + y_a sin)  for each rotated pair
//
// Pair i of the first R = rotary_dim elements is (i, i + R/2) or, interleaved,
// (2i, 2i + 1); its angle is position * inv_freq_i, f the yarn factor.  The
// rest of the row is only normed.  Everything is fp32 between the bf16 input
// and the one rounding of the output.
//
// Bound by HBM (2 bytes read and 2 written an element).  A row sits in D / 8
// lanes, 16 bytes each, so the sum of squares is log2(D / 8) shuffles and the
// half layout's partner is R / 16 lanes away: the lanes exchange the raw bf16
// words (4 shuffles).  A CTA serves one token (or some rounds of its rows, when
// tokens are few): all its rows are requested first, kRows a thread; meanwhile
// R / 2 threads compute the token's cosines and sines, and every lane folds them
// with the norm weights into two factors per element, so that a row costs
//   y = inv * (x * (w cos) + x' * (w' sin))
// with inv = rsqrt(mean(x^2) + eps).  (Rows one after the other, each waiting for
// its load: 371 us for 32768 tokens x 72 heads x 128.)
//
// Angles: inv_freq / 2 pi is computed on the host in double and passed as two
// floats; position * (hi + lo) is reduced to a fraction of a revolution with the
// product's rounding error carried by an fma, so that an angle is good to about
// 2^-24 of a revolution plus position * 2^-48, at any position below 2^24 and
// to 2^-20 up to 2^31.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace llama {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;

struct RopeTable {
  float2 rev[kMaxPairs];  // revolutions a position (hi, lo)
};

struct QkParams {
  const uint4 *q, *k, *qw, *kw;
  uint4 *q_out, *k_out;
  const int32_t* positions;
  long long q_stride, k_stride, q_out_stride, k_out_stride;  // 16-byte chunks a token
  int nq, nkv, rot, inter;
  float eps, factor;
};

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  v[0] = bf16_lo(u.x);
  v[1] = bf16_hi(u.x);
  v[2] = bf16_lo(u.y);
  v[3] = bf16_hi(u.y);
  v[4] = bf16_lo(u.z);
  v[5] = bf16_hi(u.z);
  v[6] = bf16_lo(u.w);
  v[7] = bf16_hi(u.w);
}

// Rows of one of q and k: U rounds of them (kThreads / (D / 8) rows each) from
// round first on, already loaded in u.
template <int D, int U>
__device__ __forceinline__ void norm_rope_rows(const uint4 (&u)[U], const float (&co)[8], const float (&sn)[8],
                                               bool normed, const QkParams& p, int src, uint32_t partner_bits,
                                               int row0, int rows, uint4* out, int c) {
  constexpr int L = D / 8, R = kThreads / L;
#pragma unroll
  for (int n = 0; n < U; ++n) {
    const int row = row0 + n * R;
    uint4 v;
    if (p.inter) {
      v.x = __funnelshift_l(u[n].x, u[n].x, 16);
      v.y = __funnelshift_l(u[n].y, u[n].y, 16);
      v.z = __funnelshift_l(u[n].z, u[n].z, 16);
      v.w = __funnelshift_l(u[n].w, u[n].w, 16);
    } else {
      v.x = __shfl_sync(0xffffffffu, u[n].x, src);
      v.y = __shfl_sync(0xffffffffu, u[n].y, src);
      v.z = __shfl_sync(0xffffffffu, u[n].z, src);
      v.w = __shfl_sync(0xffffffffu, u[n].w, src);
    }
    v.x &= partner_bits;  // an element that is not rotated has no partner
    v.y &= partner_bits;
    v.z &= partner_bits;
    v.w &= partner_bits;
    float x[8], y[8];
    unpack8(u[n], x);
    unpack8(v, y);
    float inv = 1.f;
    if (normed) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      inv = rsqrtf(ss * (1.f / D) + p.eps);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = inv * fmaf(y[e], sn[e], x[e] * co[e]);
    if (row < rows)
      out[static_cast<long long>(row) * L + c] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
}

// QU: rounds of q rows loaded at once (the rows beyond them in further turns)
template <int D, int QU>
__global__ void __launch_bounds__(kThreads) k_qk_norm_rope(const __grid_constant__ RopeTable tab, const QkParams p) {
  constexpr int L = D / 8;              // lanes a row
  constexpr int R = kThreads / L;       // rows of the CTA at a time
  __shared__ float2 cs[kMaxPairs];
  const long long t = blockIdx.x;
  const int c = threadIdx.x % L, group = threadIdx.x / L;
  // the rounds of this CTA: of all q rounds, then the k rounds
  const int q_rounds = (p.nq + R - 1) / R, k_rounds = (p.nkv + R - 1) / R;
  const int share = (q_rounds + k_rounds + gridDim.y - 1) / gridDim.y;
  const int first = blockIdx.y * share, last = min(q_rounds + k_rounds, first + share);
  const uint4* q = p.q + t * p.q_stride;
  const uint4* k = p.k + t * p.k_stride;
  uint4 u[QU], uk[1];
  auto load = [&](auto& v, const uint4* x, int row0, int rows) {
#pragma unroll
    for (int n = 0; n < static_cast<int>(sizeof(v) / sizeof(v[0])); ++n) {
      const int row = row0 + n * R;
      v[n] = make_uint4(0, 0, 0, 0);
      if (row < rows) v[n] = x[static_cast<long long>(row) * L + c];
    }
  };
  const int q_last = min(last, q_rounds);          // q rounds [first, q_last)
  const int k_first = max(first, q_rounds) - q_rounds, k_last = last - q_rounds;
  const int q_end = min(p.nq, q_last * R);          // q rows of this CTA end here
  if (first < q_last) load(u, q, first * R + group, q_end);
  if (k_first < k_last) load(uk, k, k_first * R + group, p.nkv);
  const int pairs = p.rot / 2;
  if (threadIdx.x < pairs) {
    // the position in two floats (the low part is zero below 2^24)
    const int pos = p.positions[t];
    const float ph = static_cast<float>(pos);
    const float pl = static_cast<float>(static_cast<long long>(pos) - static_cast<long long>(ph));
    const float2 r = tab.rev[threadIdx.x];
    const float m = ph * r.x;
    const float e = fmaf(ph, r.x, -m) + (ph * r.y + pl * r.x);
    float sn, co;
    sincospif(2.f * ((m - rintf(m)) + e), &sn, &co);
    cs[threadIdx.x] = make_float2(co * p.factor, sn * p.factor);
  }
  __syncthreads();
  // the eight elements of this lane: rotated ones take pairs pair0 .. (half
  // layout: eight pairs and a partner lane; interleaved: four pairs of its own)
  const bool rotated = c * 8 < p.rot;
  const bool upper = !p.inter && rotated && c * 8 >= pairs;
  const int partner = !rotated || p.inter ? c : upper ? c - pairs / 8 : c + pairs / 8;
  float co[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int pair = p.inter ? c * 4 + e / 2 : c * 8 + e - (upper ? pairs : 0);
    const float2 v = rotated ? cs[pair] : make_float2(1.f, 0.f);
    co[e] = v.x;
    sn[e] = (p.inter ? !(e & 1) : !upper) ? -v.y : v.y;
  }
  const int lane = threadIdx.x & 31, src = (lane / L) * L + partner;
  const uint32_t partner_bits = rotated ? 0xffffffffu : 0u;
  // the factors with a norm's weights
  auto weighted = [&](const uint4* w, float (&cw)[8], float (&sw)[8]) {
    float wx[8], wy[8];
    const uint4 wu = w[c];
    unpack8(wu, wx);
    uint4 wv = w[partner];
    if (p.inter) {
      wv.x = __funnelshift_l(wu.x, wu.x, 16);
      wv.y = __funnelshift_l(wu.y, wu.y, 16);
      wv.z = __funnelshift_l(wu.z, wu.z, 16);
      wv.w = __funnelshift_l(wu.w, wu.w, 16);
    }
    unpack8(wv, wy);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cw[e] = co[e] * wx[e];
      sw[e] = sn[e] * wy[e];
    }
  };
  float cw[8], sw[8];
  auto factors = [&](const uint4* w) {
    if (w != nullptr) {
      weighted(w, cw, sw);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cw[e] = co[e];
        sw[e] = sn[e];
      }
    }
  };
  if (first < q_last) {
    factors(p.qw);
    uint4* out = p.q_out + t * p.q_out_stride;
    for (int r = first; r < q_last; r += QU) {
      if (r > first) load(u, q, r * R + group, q_end);
      norm_rope_rows<D, QU>(u, cw, sw, p.qw != nullptr, p, src, partner_bits, r * R + group, q_end, out, c);
    }
  }
  if (k_first < k_last) {
    factors(p.kw);
    uint4* out = p.k_out + t * p.k_out_stride;
    const int k_end = min(p.nkv, k_last * R);
    for (int r = k_first; r < k_last; ++r) {
      if (r > k_first) load(uk, k, r * R + group, k_end);
      norm_rope_rows<D, 1>(uk, cw, sw, p.kw != nullptr, p, src, partner_bits, r * R + group, k_end, out, c);
    }
  }
}

// The frequency rules, in double.  inv_i = theta^(-2i/R) by repeated
// multiplication (64 roundings, far below the table's 48 bits).
RopeTable rope_table(const LlamaQkNormRopeConfig& c) {
  RopeTable tab{};
  const int R = c.rotary_dim, pairs = R / 2;
  if (pairs == 0) return tab;
  const double two_pi = 6.283185307179586476925287;
  const double theta = c.rope_theta, f = c.rs_factor, orig = c.rs_original_max_pos;
  const double ratio = pow(theta, -2.0 / R);
  double lo = 0.0, hi = 0.0;  // yarn: the pairs between which the blend runs
  if (c.rope_scaling == LLAMA_ROPE_YARN) {
    const double per = R / (2.0 * log(theta));
    lo = fmax(floor(per * log(orig / (c.rs_high_freq_factor * two_pi))), 0.0);
    hi = fmin(ceil(per * log(orig / (c.rs_low_freq_factor * two_pi))), R - 1.0);
  }
  double inv = 1.0;
  for (int i = 0; i < pairs; ++i, inv *= ratio) {
    double v = inv;
    if (c.rope_scaling == LLAMA_ROPE_LINEAR) {
      v = inv / f;
    } else if (c.rope_scaling == LLAMA_ROPE_LLAMA3) {
      const double turns = orig * inv / two_pi;  // original context / wavelength
      const double s = fmin(fmax((turns - c.rs_low_freq_factor) /
                                     (static_cast<double>(c.rs_high_freq_factor) - c.rs_low_freq_factor), 0.0), 1.0);
      v = (1.0 - s) * inv / f + s * inv;
    } else if (c.rope_scaling == LLAMA_ROPE_YARN) {
      const double s = fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
      v = inv / f * s + inv * (1.0 - s);
    }
    v /= two_pi;
    tab.rev[i].x = static_cast<float>(v);
    tab.rev[i].y = static_cast<float>(v - static_cast<double>(tab.rev[i].x));
  }
  return tab;
}

}  // namespace

int qk_norm_rope_launch(const QkNormRopeArgs& a, cudaStream_t s) {
  if (a.T <= 0) return 0;
  const LlamaQkNormRopeConfig& c = *a.cfg;
  QkParams p{};
  p.q = static_cast<const uint4*>(a.q);
  p.k = static_cast<const uint4*>(a.k);
  p.qw = static_cast<const uint4*>(a.q_norm_w);
  p.kw = static_cast<const uint4*>(a.k_norm_w);
  p.q_out = static_cast<uint4*>(a.q_out);
  p.k_out = static_cast<uint4*>(a.k_out);
  p.positions = a.positions;
  p.q_stride = a.q_stride / 8;
  p.k_stride = a.k_stride / 8;
  p.q_out_stride = a.q_out_stride / 8;
  p.k_out_stride = a.k_out_stride / 8;
  p.nq = c.n_heads;
  p.nkv = c.n_kv_heads;
  p.rot = c.rotary_dim;
  p.inter = c.interleaved;
  p.eps = c.rms_eps;
  p.factor = c.rope_scaling == LLAMA_ROPE_YARN ? c.rs_attention_factor : 1.f;
  const RopeTable tab = rope_table(c);
  const int per = kThreads / (c.head_dim / 8);
  const int q_rounds = (p.nq + per - 1) / per, k_rounds = (p.nkv + per - 1) / per;
  // few tokens: a CTA for every round of rows of a token, so that they run side by side
  const bool split = static_cast<long long>(a.T) * (q_rounds + k_rounds) <= 8LL * num_sms();
  const dim3 grid(a.T, split ? q_rounds + k_rounds : 1);
  auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kThreads), 0, s, false, tab, p); };
  const bool one = split || q_rounds == 1;
  if (c.head_dim == 128)
    return one ? go(k_qk_norm_rope<128, 1>) : q_rounds == 2 ? go(k_qk_norm_rope<128, 2>) : go(k_qk_norm_rope<128, 4>);
  return one ? go(k_qk_norm_rope<64, 1>) : q_rounds == 2 ? go(k_qk_norm_rope<64, 2>) : go(k_qk_norm_rope<64, 4>);
}

}  // namespace llama
