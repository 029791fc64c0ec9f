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
// words (4 shuffles) and norm the partner's values themselves.  A CTA serves one
// token; its cosines and sines are computed once, by R / 2 threads, and kept in
// registers over the token's heads.
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

template <int D>
__global__ void __launch_bounds__(kThreads) k_qk_norm_rope(const __grid_constant__ RopeTable tab, const QkParams p) {
  constexpr int L = D / 8;              // lanes a row
  constexpr int R = kThreads / L;       // rows of the CTA at a time
  __shared__ float2 cs[kMaxPairs];
  const long long t = blockIdx.x;
  const int c = threadIdx.x % L, first = blockIdx.y * R + threadIdx.x / L;
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
    sn[e] = v.y;
    if (p.inter ? !(e & 1) : !upper) sn[e] = -sn[e];
  }
  const int lane = threadIdx.x & 31, src = (lane / L) * L + partner;
  const int rows = p.nq + p.nkv;
  // rows in steps of the grid's; every lane of a warp runs every step (the shuffles are warp-wide)
  for (int row0 = 0; row0 < rows; row0 += R * gridDim.y) {
    const int row = row0 + first;
    const bool ok = row < rows, is_k = row >= p.nq;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (ok) u = is_k ? p.k[t * p.k_stride + (row - p.nq) * L + c] : p.q[t * p.q_stride + row * L + c];
    const uint4* w = is_k ? p.kw : p.qw;
    float x[8], y[8];
    unpack8(u, x);
    uint4 uy;
    if (p.inter) {
      uy.x = __funnelshift_l(u.x, u.x, 16);
      uy.y = __funnelshift_l(u.y, u.y, 16);
      uy.z = __funnelshift_l(u.z, u.z, 16);
      uy.w = __funnelshift_l(u.w, u.w, 16);
    } else {
      uy.x = __shfl_sync(0xffffffffu, u.x, src);
      uy.y = __shfl_sync(0xffffffffu, u.y, src);
      uy.z = __shfl_sync(0xffffffffu, u.z, src);
      uy.w = __shfl_sync(0xffffffffu, u.w, src);
    }
    unpack8(uy, y);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!ok) continue;
    if (w != nullptr) {
      const float inv = rsqrtf(ss / static_cast<float>(D) + p.eps);
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
        x[e] = x[e] * inv * wx[e];
        y[e] = y[e] * inv * wy[e];
      }
    }
    if (rotated) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * co[e] + y[e] * sn[e];
    }
    uint4 o;
    o.x = pack_bf16x2(x[0], x[1]);
    o.y = pack_bf16x2(x[2], x[3]);
    o.z = pack_bf16x2(x[4], x[5]);
    o.w = pack_bf16x2(x[6], x[7]);
    if (is_k)
      p.k_out[t * p.k_out_stride + (row - p.nq) * L + c] = o;
    else
      p.q_out[t * p.q_out_stride + row * L + c] = o;
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
  const int rows = p.nq + p.nkv, per = kThreads / (c.head_dim / 8);
  // few tokens: a CTA for every round of rows of a token, so the rows are all in flight at once
  const int rounds = (rows + per - 1) / per;
  const int split = static_cast<long long>(a.T) * rounds <= 4LL * num_sms() ? rounds : 1;
  const dim3 grid(a.T, split);
  if (c.head_dim == 128) return launch_kernel(k_qk_norm_rope<128>, grid, dim3(kThreads), 0, s, false, tab, p);
  return launch_kernel(k_qk_norm_rope<64>, grid, dim3(kThreads), 0, s, false, tab, p);
}

}  // namespace llama
