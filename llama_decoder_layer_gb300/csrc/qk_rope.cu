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
// Bound by HBM (2 bytes read and 2 written an element): 32768 tokens x 72 heads x
// 128 take 187 us, 6.5 TB/s, 95% of the copy rate.  A row sits in D / 8
// lanes; a lane holds four rotated pairs whole (elements 4c .. and R/2 + 4c .. of
// the half layout, 8c .. of the interleaved one; eight neighbours past R), so
// that nothing but the sum of squares crosses lanes and the arithmetic runs on
// two elements an instruction.  A warp takes one token (a part of its rows, when
// tokens are few): two or four lanes' worth of cosines and sines a lane, exchanged
// through shared memory and folded with the norm weights into two factors per
// element, then its rows, kRounds of them in flight while as many are worked on:
//   y = inv * (x * (w cos) + x' * (w' sin)),  inv = rsqrt(mean(x^2) + eps)
// (A CTA of 256 threads a token, with 16-byte chunks whose partners came by
// shuffles, spent 189 instructions a chunk and took 297 us for 32768 tokens x 72
// heads x 128.)
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

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRounds = 4;  // rounds of rows (32 / (D / 8) each) loaded at once
constexpr int kCtasPerSm = 5;
constexpr int kMaxPairs = 64;

struct RopeTable {
  float2 rev[kMaxPairs];  // revolutions a position (hi, lo)
};

struct QkParams {
  const uint2 *q, *k, *qw, *kw;
  uint2 *q_out, *k_out;
  const int32_t* positions;
  long long q_stride, k_stride, q_out_stride, k_out_stride;  // 8-byte chunks a token
  int T, nq, nkv, rot;
  int parts;  // warps a token
  float eps, factor;
};

// Four pairs a lane: a[i], b[i] the elements of pair i, two pairs to a register
// pair.  Half layout: u = a0 a1 a2 a3, v = b0 b1 b2 b3; interleaved: u v = a0 b0
// a1 b1 ...
struct Pairs {
  uint64_t a[2], b[2];
};

template <bool INTER>
__device__ __forceinline__ Pairs unpack(uint2 u, uint2 v) {
  Pairs x;
  if constexpr (INTER) {
    x.a[0] = f2_pack(bf16_lo(u.x), bf16_lo(u.y));
    x.b[0] = f2_pack(bf16_hi(u.x), bf16_hi(u.y));
    x.a[1] = f2_pack(bf16_lo(v.x), bf16_lo(v.y));
    x.b[1] = f2_pack(bf16_hi(v.x), bf16_hi(v.y));
  } else {
    x.a[0] = f2_pack(bf16_lo(u.x), bf16_hi(u.x));
    x.a[1] = f2_pack(bf16_lo(u.y), bf16_hi(u.y));
    x.b[0] = f2_pack(bf16_lo(v.x), bf16_hi(v.x));
    x.b[1] = f2_pack(bf16_lo(v.y), bf16_hi(v.y));
  }
  return x;
}

template <bool INTER>
__device__ __forceinline__ void pack(const Pairs& x, uint2& u, uint2& v) {
  float a[4], b[4];
  f2_unpack(x.a[0], a[0], a[1]);
  f2_unpack(x.a[1], a[2], a[3]);
  f2_unpack(x.b[0], b[0], b[1]);
  f2_unpack(x.b[1], b[2], b[3]);
  if constexpr (INTER) {
    u = make_uint2(pack_bf16x2(a[0], b[0]), pack_bf16x2(a[1], b[1]));
    v = make_uint2(pack_bf16x2(a[2], b[2]), pack_bf16x2(a[3], b[3]));
  } else {
    u = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
    v = make_uint2(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
  }
}

// y_a = x_a aa + x_b ab,  y_b = x_b bb + x_a ba
struct Factors {
  uint64_t aa[2], ab[2], bb[2], ba[2];
};

// PARTIAL: some elements are not rotated; their lanes keep x' out of the sums (an
// infinity times a zero sine would be a NaN).
template <int D, bool INTER, bool PARTIAL>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_qk_norm_rope(const __grid_constant__ RopeTable tab, const QkParams p) {
  constexpr int L = D / 8;   // lanes a row
  constexpr int R = 32 / L;  // rows a round
  __shared__ float2 cs_all[kWarps][kMaxPairs];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % L, sub = lane / L;
  float2* cs = cs_all[warp];
  const int pairs = p.rot / 2;
  const bool rotated = !PARTIAL || c * 8 < p.rot;
  // the lane's two 8-byte chunks of a row
  const int at0 = INTER ? 2 * c : rotated ? c : p.rot / 4 + 2 * (c - p.rot / 8);
  const int at1 = INTER || !rotated ? at0 + 1 : c + p.rot / 8;
  const uint64_t keep = rotated ? ~0ull : 0ull;
  const int q_rounds = (p.nq + R - 1) / R, rounds = q_rounds + (p.nkv + R - 1) / R;
  const int share = (rounds + p.parts - 1) / p.parts;
  const long long units = static_cast<long long>(p.T) * p.parts;
  for (long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp; unit < units;
       unit += static_cast<long long>(gridDim.x) * kWarps) {
    const long long t = p.parts == 1 ? unit : unit / p.parts;
    const int first = static_cast<int>(unit - t * p.parts) * share, last = min(rounds, first + share);
    if (first >= last) continue;
    // a row of q, then of k; rounds do not mix the two
    auto load = [&](int r, uint2& u, uint2& v) {
      const bool is_k = r >= q_rounds;
      const int row = (is_k ? r - q_rounds : r) * R + sub;
      u = v = make_uint2(0, 0);
      if (r < last && row < (is_k ? p.nkv : p.nq)) {
        const uint2* src = (is_k ? p.k + t * p.k_stride : p.q + t * p.q_stride) + row * (D / 4);
        u = src[at0];
        v = src[at1];
      }
    };
    uint2 u[kRounds], v[kRounds];
#pragma unroll
    for (int n = 0; n < kRounds; ++n) load(first + n, u[n], v[n]);
    if (pairs > 0) {
      // the position in two floats (the low part is zero below 2^24)
      const int pos = p.positions[t];
      const float ph = static_cast<float>(pos);
      const float pl = static_cast<float>(static_cast<long long>(pos) - static_cast<long long>(ph));
      __syncwarp();
      for (int i = lane; i < pairs; i += 32) {
        const float2 rev = tab.rev[i];
        const float m = ph * rev.x;
        const float e = fmaf(ph, rev.x, -m) + (ph * rev.y + pl * rev.x);
        float sn, co;
        sincospif(2.f * ((m - rintf(m)) + e), &sn, &co);
        cs[i] = make_float2(co * p.factor, sn * p.factor);
      }
      __syncwarp();
    }
    Factors f;
    auto factors = [&](const uint2* w) {
      uint64_t co[2], sn[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = rotated && pairs > 0 ? cs[4 * c + 2 * i] : make_float2(1.f, 0.f);
        const float2 y = rotated && pairs > 0 ? cs[4 * c + 2 * i + 1] : make_float2(1.f, 0.f);
        co[i] = f2_pack(x.x, y.x);
        sn[i] = f2_pack(x.y, y.y);
      }
      const uint64_t minus = f2_pack(-1.f, -1.f);
      if (w != nullptr) {
        const Pairs n = unpack<INTER>(w[at0], w[at1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f.aa[i] = f2_mul(co[i], n.a[i]);
          f.bb[i] = f2_mul(co[i], n.b[i]);
          f.ab[i] = f2_mul(f2_mul(sn[i], n.b[i]), minus);
          f.ba[i] = f2_mul(sn[i], n.a[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f.aa[i] = f.bb[i] = co[i];
          f.ab[i] = f2_mul(sn[i], minus);
          f.ba[i] = sn[i];
        }
      }
    };
    auto finish = [&](int r, uint2 u0, uint2 v0) {
      const bool is_k = r >= q_rounds;
      const Pairs x = unpack<INTER>(u0, v0);
      float inv = 1.f;
      if ((is_k ? p.kw : p.qw) != nullptr) {
        uint64_t s2 = f2_mul(x.a[0], x.a[0]);
        s2 = f2_fma(x.a[1], x.a[1], s2);
        s2 = f2_fma(x.b[0], x.b[0], s2);
        s2 = f2_fma(x.b[1], x.b[1], s2);
        float s0, s1;
        f2_unpack(s2, s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        inv = rsqrtf(ss * (1.f / D) + p.eps);
      }
      const uint64_t inv2 = f2_pack(inv, inv);
      Pairs y;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t xb = PARTIAL ? x.b[i] & keep : x.b[i], xa = PARTIAL ? x.a[i] & keep : x.a[i];
        y.a[i] = f2_mul(inv2, f2_fma(x.a[i], f.aa[i], f2_mul(xb, f.ab[i])));
        y.b[i] = f2_mul(inv2, f2_fma(x.b[i], f.bb[i], f2_mul(xa, f.ba[i])));
      }
      const int row = (is_k ? r - q_rounds : r) * R + sub;
      if (row < (is_k ? p.nkv : p.nq)) {
        uint2* dst = (is_k ? p.k_out + t * p.k_out_stride : p.q_out + t * p.q_out_stride) + row * (D / 4);
        pack<INTER>(y, u0, v0);
        dst[at0] = u0;
        dst[at1] = v0;
      }
    };
    if (first < q_rounds) factors(p.qw);
    for (int r = first; r < last; r += kRounds) {
      uint2 un[kRounds], vn[kRounds];
      if (r + kRounds < last) {
#pragma unroll
        for (int n = 0; n < kRounds; ++n) load(r + kRounds + n, un[n], vn[n]);
      }
#pragma unroll
      for (int n = 0; n < kRounds; ++n) {
        if (r + n >= last) break;
        if (r + n == q_rounds || (r + n == first && first > q_rounds)) factors(p.kw);
        finish(r + n, u[n], v[n]);
      }
#pragma unroll
      for (int n = 0; n < kRounds; ++n) {
        u[n] = un[n];
        v[n] = vn[n];
      }
    }
  }
}

// The frequency rules, in double.  inv_i = theta^(-2i/R) by repeated
// multiplication: at most 63 times, each adding pow's error in the ratio (below
// 2^-52) and a rounding (2^-53), so within 2^-45.4 of its size: with inv_i / 2 pi
// up to 2^-2.65, about 2^-48 of a revolution a position.
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
  p.q = static_cast<const uint2*>(a.q);
  p.k = static_cast<const uint2*>(a.k);
  p.qw = static_cast<const uint2*>(a.q_norm_w);
  p.kw = static_cast<const uint2*>(a.k_norm_w);
  p.q_out = static_cast<uint2*>(a.q_out);
  p.k_out = static_cast<uint2*>(a.k_out);
  p.positions = a.positions;
  p.q_stride = a.q_stride / 4;
  p.k_stride = a.k_stride / 4;
  p.q_out_stride = a.q_out_stride / 4;
  p.k_out_stride = a.k_out_stride / 4;
  p.T = a.T;
  p.nq = c.n_heads;
  p.nkv = c.n_kv_heads;
  p.rot = c.rotary_dim;
  p.eps = c.rms_eps;
  p.factor = c.rope_scaling == LLAMA_ROPE_YARN ? c.rs_attention_factor : 1.f;
  const RopeTable tab = rope_table(c);
  // Few tokens: a token's rounds are shared by several warps (two rounds each at least), so that they run side by
  // side; from 16 warps an SM on, a warp a token.
  const int per = 32 / (c.head_dim / 8);
  const int rounds = (p.nq + per - 1) / per + (p.nkv + per - 1) / per;
  const long long want = 16LL * num_sms() / a.T;
  const int most = (rounds + 1) / 2;
  p.parts = want < 1 ? 1 : want > most ? most : static_cast<int>(want);
  const long long ctas = (static_cast<long long>(a.T) * p.parts + kWarps - 1) / kWarps, full = 1LL * kCtasPerSm * num_sms();
  const dim3 grid(static_cast<unsigned>(ctas < full ? ctas : full));
  auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kThreads), 0, s, true, tab, p); };
  const bool partial = p.rot < c.head_dim;
  if (c.head_dim == 128) {
    if (c.interleaved) return partial ? go(k_qk_norm_rope<128, true, true>) : go(k_qk_norm_rope<128, true, false>);
    return partial ? go(k_qk_norm_rope<128, false, true>) : go(k_qk_norm_rope<128, false, false>);
  }
  if (c.interleaved) return partial ? go(k_qk_norm_rope<64, true, true>) : go(k_qk_norm_rope<64, true, false>);
  return partial ? go(k_qk_norm_rope<64, false, true>) : go(k_qk_norm_rope<64, false, false>);
}

}  // namespace llama
