// Microscaled matrices (the formats are in mx.cuh): quantising bf16 rows,
// reading them back, and the fused residual add + RMSNorm whose output is
// quantised, for a product of microscaled matrices to read.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "mx.cuh"

namespace llama {

namespace {

constexpr int kThreads = 256;

// A thread's group: its row, its number in the row, and whether the row has it (a row's last scale word is filled up
// with zeros).  Four lanes in a row have the groups of one scale word.
struct MxPlace {
  int row, grp;
  bool there;
};
__device__ __forceinline__ MxPlace mx_place(const MxRowsArgs& a) {
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  MxPlace p;
  const uint32_t padded = static_cast<uint32_t>(a.ktiles) * kMxTileGroups;
  const bool in = i < static_cast<long long>(a.rows) * padded;
  const uint32_t n = in ? static_cast<uint32_t>(i) : 0u;
  p.row = static_cast<int>(n / padded);
  p.grp = static_cast<int>(n - static_cast<uint32_t>(p.row) * padded);
  p.there = in && p.grp < a.groups;
  if (!in) p.row = -1;
  return p;
}

// the word of four lanes' scale bytes
__device__ __forceinline__ uint32_t scale_word(uint32_t byte) {
  uint32_t w = byte << ((threadIdx.x & 3) * 8);
  w |= __shfl_xor_sync(0xffffffffu, w, 1);
  w |= __shfl_xor_sync(0xffffffffu, w, 2);
  return w;
}

__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  v[0] = bf16_lo(u.x);
  v[1] = bf16_hi(u.x);
  v[2] = bf16_lo(u.y);
  v[3] = bf16_hi(u.y);
  v[4] = bf16_lo(u.z);
  v[5] = bf16_hi(u.z);
  v[6] = bf16_lo(u.w);
  v[7] = bf16_hi(u.w);
}

// Grids of up to this many CTAs let the next kernel start at once and set up beside them (a larger grid's last CTAs would
// share their SMs with it).
constexpr unsigned kEarlyTriggerCtas = 256;

// One thread a group: its maximum needs no other lane, and only the word of scales is put together by four.  Bound by HBM
// (57344 x 8192 to nvfp4: 191 us, 6.3 TB/s, 94% of the copy rate; the issue slots 73% busy, so that maxima are taken of two
// bf16 magnitudes at a time and codes of two elements an instruction: 213 us without).  SECTORS: rows begin on 32 bytes,
// which a thread then reads at once.
template <int FMT, bool SECTORS>
__global__ void __launch_bounds__(kThreads) k_quantize_mx(const MxRowsArgs a) {
  constexpr int G = mx_group(FMT), C = G / 8;
  pdl_wait();
  if (gridDim.x <= kEarlyTriggerCtas) pdl_trigger();
  const MxPlace p = mx_place(a);
  uint32_t u[C * 4];
#pragma unroll
  for (int c = 0; c < C * 4; ++c) u[c] = 0;
  if (p.there) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + p.row * a.x_stride) + p.grp * C;
    if constexpr (SECTORS) {
#pragma unroll
      for (int c = 0; c < C; c += 2) ld_global_v8(src + c, u + 4 * c);
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint4 q = src[c];
        u[4 * c] = q.x;
        u[4 * c + 1] = q.y;
        u[4 * c + 2] = q.z;
        u[4 * c + 3] = q.w;
      }
    }
  }
  float x[C][8];
  uint32_t top = 0;  // of two bf16 magnitudes at a time
#pragma unroll
  for (int c = 0; c < C; ++c) unpack8(make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]), x[c]);
#pragma unroll
  for (int i = 0; i < 4 * C; ++i) top = __vmaxu2(top, u[i] & 0x7fff7fffu);
  top = max(top & 0xffff0000u, top << 16);
  const MxScale s = mx_scale<FMT, true>(top, a.sixth, a.inv_g);
  if (p.there) {
    uint8_t* dst = static_cast<uint8_t*>(a.codes) + static_cast<size_t>(p.row) * (a.groups * (G * mx_bits(FMT) / 8)) +
                   p.grp * (G * mx_bits(FMT) / 8);
    uint2 w[C];
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = mx_codes8<FMT, true>(x[c], s.factor);
    if constexpr (FMT == kMxNvfp4) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0].x, w[1].x);
    } else if constexpr (FMT == kMxFp4) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0].x, w[1].x, w[2].x, w[3].x);
    } else {
      if constexpr (SECTORS) {  // (codes begin on 32 bytes too)
        const uint32_t q[8] = {w[0].x, w[0].y, w[1].x, w[1].y, w[2].x, w[2].y, w[3].x, w[3].y};
        st_global_v8(dst, q);
      } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[2].x, w[2].y, w[3].x, w[3].y);
      }
    }
  }
  const uint32_t word = scale_word(p.there ? s.byte : 0u);
  if (p.row >= 0 && (threadIdx.x & 3) == 0)
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.scales) + mx_scale_at(p.row, p.grp >> 2, a.ktiles)) = word;
}

// bf16(code * scale * g), one thread a group.  Bound by HBM (57344 x 8192 of nvfp4: 180 us, 6.7 TB/s; stored in halves of
// sectors, 16 bytes at a time, 203).
template <int FMT, bool SECTORS>
__global__ void __launch_bounds__(kThreads) k_dequantize_mx(const MxRowsArgs a) {
  constexpr int G = mx_group(FMT), C = G / 8;
  pdl_wait();
  if (gridDim.x <= kEarlyTriggerCtas) pdl_trigger();
  const MxPlace p = mx_place(a);
  if (!p.there) return;
  const uint8_t* src = static_cast<const uint8_t*>(a.codes) +
                       static_cast<size_t>(p.row) * (a.groups * (G * mx_bits(FMT) / 8)) + p.grp * (G * mx_bits(FMT) / 8);
  const uint8_t byte = static_cast<const uint8_t*>(a.scales)[mx_scale_at(p.row, p.grp >> 2, a.ktiles) + (p.grp & 3)];
  uint32_t w[G * mx_bits(FMT) / 32];
  if constexpr (FMT == kMxFp8 && SECTORS) {
    ld_global_v8(src, w);
  } else if constexpr (FMT == kMxNvfp4) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < G * mx_bits(FMT) / 128; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(src)[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
  const float s = FMT == kMxNvfp4 ? e4m3_value(byte) * a.g : e8m0_value(byte);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y) + p.row * a.x_stride) + p.grp * C;
  uint32_t o[C * 4];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float v[8];
    mx_values8<FMT>(FMT == kMxFp8 ? make_uint2(w[2 * c], w[2 * c + 1]) : make_uint2(w[c], 0), v);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[4 * c + e] = pack_bf16x2(v[2 * e] * s, v[2 * e + 1] * s);
  }
#pragma unroll
  for (int c = 0; c < C; c += 2) {
    if constexpr (SECTORS) {
      st_global_v8(dst + c, o + 4 * c);
    } else {
      dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
      dst[c + 1] = make_uint4(o[4 * c + 4], o[4 * c + 5], o[4 * c + 6], o[4 * c + 7]);
    }
  }
}

// The sum over a row's chunks, ss[c] of this thread's, in an order that does not depend on T, so that a row's codes do not depend
// on the number of rows: blocks of 32 neighbouring chunks over the lanes, pairs 16 apart first, then the blocks in the same
// way, pairs 32 apart first.  A block is a warp's chunks of one c; with each exchange a lane goes on with half of its blocks
// (6 exchanges for four).
template <int T, int MAXC>
__device__ __forceinline__ float row_sum(float (&ss)[MAXC], float* red) {
  constexpr int kLanes = 32 / MAXC, kBlocks = MAXC * T / 32;  // lanes that hold a block's sum in the end, block c from c kLanes on
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = MAXC, o = 16; o > 0; o >>= 1, n = n > 1 ? n / 2 : 1) {
    const bool high = (lane & o) != 0;
    if (n > 1) {
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const float keep = high ? ss[i + n / 2] : ss[i], give = high ? ss[i] : ss[i + n / 2];
        ss[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    } else {
      ss[0] += __shfl_xor_sync(0xffffffffu, ss[0], o);
    }
  }
  float sum = ss[0];
  if constexpr (T == 32) {
#pragma unroll
    for (int o = 16; o >= kLanes; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  } else {
    if (lane % kLanes == 0) red[lane / kLanes * (T / 32) + (threadIdx.x >> 5)] = sum;
    __syncthreads();
    sum = red[lane % (kBlocks < 32 ? kBlocks : 32)];
    if constexpr (kBlocks > 32) sum += red[lane + 32];
#pragma unroll
    for (int o = (kBlocks < 32 ? kBlocks : 32) / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  return sum;
}

// The residual add and RMSNorm of rowops.cu, its output quantised: T threads a row (32: a CTA has eight rows, a warp each),
// the row in registers in chunks of 8 elements, 2 or 4 lanes a group.  The norm's fp32 result is quantised as it is, without
// a rounding to bf16 before.
template <int FMT, int T, int MAXC>
__global__ void __launch_bounds__(T == 32 ? kThreads : T) k_add_rmsnorm_mx(const MxNormArgs a) {
  constexpr int L = mx_group(FMT) / 8;  // lanes a group
  constexpr int kRows = T == 32 ? kThreads / 32 : 1;
  __shared__ float red[MAXC * T / 32];
  pdl_wait();
  if (gridDim.x <= kEarlyTriggerCtas) pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kRows + (kRows > 1 ? warp : 0), nch = a.cols >> 3;
  if (kRows > 1 && row >= a.rows) return;
  const int tid = T == 32 ? threadIdx.x & 31 : threadIdx.x;
  const size_t base = static_cast<size_t>(row) * nch;
  const uint4* x = static_cast<const uint4*>(a.x) + base;
  const uint4* res = static_cast<const uint4*>(a.res_in) + base;
  uint4 u[MAXC];  // the new residual: a bf16 tensor, and the norm is taken of that tensor
  float ss[MAXC];
#pragma unroll
  for (int c = 0; c < MAXC; ++c) u[c] = tid + c * T < nch ? x[tid + c * T] : make_uint4(0, 0, 0, 0);
  if (a.res_in != nullptr) {
    uint4 r[MAXC];
#pragma unroll
    for (int c = 0; c < MAXC; ++c) r[c] = tid + c * T < nch ? res[tid + c * T] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
      float p[8], q[8];
      unpack8(u[c], p);
      unpack8(r[c], q);
      u[c] = make_uint4(pack_bf16x2(p[0] + q[0], p[1] + q[1]), pack_bf16x2(p[2] + q[2], p[3] + q[3]),
                        pack_bf16x2(p[4] + q[4], p[5] + q[5]), pack_bf16x2(p[6] + q[6], p[7] + q[7]));
    }
  }
#pragma unroll
  for (int c = 0; c < MAXC; ++c) {
    float v[8];
    unpack8(u[c], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[c] = e == 0 ? v[0] * v[0] : fmaf(v[e], v[e], ss[c]);
  }
  // 1 / sqrt(y) = inv + low: the residual 1 - y inv^2, with the product's rounding, halved, so that the results below
  // are off by little more than their own rounding (codes near a border then fall where they should)
  const float y = row_sum<T>(ss, red) / static_cast<float>(a.cols) + a.eps;
  const float inv = rsqrtf(y), yi = y * inv;
  const float low = yi < INFINITY ? 0.5f * inv * (fmaf(-yi, inv, 1.f) - fmaf(y, inv, -yi) * inv) : 0.f;
  uint4* res_out = static_cast<uint4*>(a.res_out) + base;
  uint8_t* codes = static_cast<uint8_t*>(a.codes) + base * mx_bits(FMT);
#pragma unroll
  for (int c = 0; c < MAXC; ++c) {
    const int i = tid + c * T;
    if (c * T >= nch) break;  // the same for the whole row
    const bool there = i < nch;
    float h[8];
    uint32_t top = 0;
    if (there) {
      if (a.res_out != nullptr) res_out[i] = u[c];
      float v[8], g[8];
      unpack8(u[c], v);
      unpack8(static_cast<const uint4*>(a.gamma)[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float vg = v[e] * g[e];  // exact: 8 and 8 bits
        h[e] = fmaf(vg, inv, vg * low);
        top = max(top, abs_bits(h[e]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = 0.f;
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const MxScale s = mx_scale<FMT, false>(top, a.sixth, a.inv_g);
    if (there) {
      const uint2 w = mx_codes8<FMT, false>(h, s.factor);
      if constexpr (FMT == kMxFp8) reinterpret_cast<uint2*>(codes)[i] = w;
      else reinterpret_cast<uint32_t*>(codes)[i] = w.x;
    }
    // the scale bytes of 4 L lanes
    uint32_t word = (there ? s.byte : 0u) << ((threadIdx.x / L & 3) * 8);
#pragma unroll
    for (int o = L; o < 4 * L; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
    if (there && (threadIdx.x & (4 * L - 1)) == 0)
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.scales) + mx_scale_at(row, i / (4 * L), a.ktiles)) = word;
  }
}

// Many rows: a warp each up to 1024 elements (10099 x 192: 4.0 us; a CTA of 256 threads each 11.6), then four chunks a
// thread at most (5906 x 15840: 99 us, eight 149).  The row is kept as the bf16 numbers it is made of, four registers a
// chunk, so that an SM holds 1024 threads or more with all their loads in flight (32768 x 8192: 267 us, 7.0 TB/s; as
// floats 311).  Few rows: as many threads as chunks, for the latency (128 x 8192: 3.1 us, 256 threads 4.4).
template <int FMT>
int norm_typed(const MxNormArgs& a, cudaStream_t s) {
  const int nch = a.cols / 8;
  auto go = [&](auto kernel, int rows, int threads) {
    return launch_kernel(kernel, dim3((a.rows + rows - 1) / rows), dim3(threads), 0, s, true, a);
  };
  if (nch <= 32) return go(k_add_rmsnorm_mx<FMT, 32, 1>, 8, kThreads);
  if (a.rows <= 2 * num_sms()) {
    if (nch <= 256) return go(k_add_rmsnorm_mx<FMT, 256, 1>, 1, 256);
    if (nch <= 512) return go(k_add_rmsnorm_mx<FMT, 512, 1>, 1, 512);
    if (nch <= 1024) return go(k_add_rmsnorm_mx<FMT, 1024, 1>, 1, 1024);
    return go(k_add_rmsnorm_mx<FMT, 1024, 2>, 1, 1024);
  }
  if (nch <= 64) return go(k_add_rmsnorm_mx<FMT, 32, 2>, 8, kThreads);
  if (nch <= 128) return go(k_add_rmsnorm_mx<FMT, 32, 4>, 8, kThreads);
  if (nch <= 256) return go(k_add_rmsnorm_mx<FMT, 256, 1>, 1, 256);
  if (nch <= 512) return go(k_add_rmsnorm_mx<FMT, 256, 2>, 1, 256);
  if (nch <= 1024) return go(k_add_rmsnorm_mx<FMT, 256, 4>, 1, 256);
  return go(k_add_rmsnorm_mx<FMT, 512, 4>, 1, 512);
}

unsigned group_ctas(const MxRowsArgs& a) {
  const long long n = static_cast<long long>(a.rows) * a.ktiles * kMxTileGroups;
  return static_cast<unsigned>((n + kThreads - 1) / kThreads);
}

// bf16 rows and codes on 32 bytes (rows of codes are multiples of 16 or 32 bytes)
bool whole_sectors(const void* rows, const MxRowsArgs& a) {
  return a.x_stride % 16 == 0 && ((reinterpret_cast<uintptr_t>(rows) | reinterpret_cast<uintptr_t>(a.codes)) & 31) == 0;
}

}  // namespace

int quantize_mx_launch(int fmt, const MxRowsArgs& a, cudaStream_t s) {
  auto go = [&](auto kernel) { return launch_kernel(kernel, dim3(group_ctas(a)), dim3(kThreads), 0, s, true, a); };
  const bool whole = whole_sectors(a.x, a);
  if (fmt == kMxNvfp4) return whole ? go(k_quantize_mx<kMxNvfp4, true>) : go(k_quantize_mx<kMxNvfp4, false>);
  if (fmt == kMxFp4) return whole ? go(k_quantize_mx<kMxFp4, true>) : go(k_quantize_mx<kMxFp4, false>);
  return whole ? go(k_quantize_mx<kMxFp8, true>) : go(k_quantize_mx<kMxFp8, false>);
}

int dequantize_mx_launch(int fmt, const MxRowsArgs& a, cudaStream_t s) {
  auto go = [&](auto kernel) { return launch_kernel(kernel, dim3(group_ctas(a)), dim3(kThreads), 0, s, true, a); };
  const bool whole = whole_sectors(a.y, a);
  if (fmt == kMxNvfp4) return whole ? go(k_dequantize_mx<kMxNvfp4, true>) : go(k_dequantize_mx<kMxNvfp4, false>);
  if (fmt == kMxFp4) return whole ? go(k_dequantize_mx<kMxFp4, true>) : go(k_dequantize_mx<kMxFp4, false>);
  return whole ? go(k_dequantize_mx<kMxFp8, true>) : go(k_dequantize_mx<kMxFp8, false>);
}

int add_rmsnorm_mx_launch(int fmt, const MxNormArgs& a, cudaStream_t s) {
  return fmt == kMxNvfp4 ? norm_typed<kMxNvfp4>(a, s) : fmt == kMxFp4 ? norm_typed<kMxFp4>(a, s) : norm_typed<kMxFp8>(a, s);
}

}  // namespace llama
