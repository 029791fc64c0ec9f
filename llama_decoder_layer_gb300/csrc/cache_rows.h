// How the kernels that write and read 4-bit cache rows share a call's tokens
// among their threads.  Index arithmetic only, without CUDA: the tests compile
// it for the host.
//   A thread takes chunks of 8 elements of U tokens, always the same chunk of
// the row.  A CTA has a whole number of rows (or a part of one) in its threads.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define LLAMA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define LLAMA_HOST_DEVICE inline
#endif

namespace llama {

constexpr int kMaxRowThreads = 512;

// A launch's shape: `chunks` chunks of 8 elements a token row (K or V); a CTA
// of `threads` covers `rows` rows at a time, or 1 / parts of one.  whole: a row
// is a whole number of warps, so that its token, slot and tile are a warp's.
struct RowShape {
  int chunks, rows, parts, threads;
  bool whole;
};

inline RowShape row_shape(int n_kv, int head_dim) {
  RowShape g{};
  g.chunks = n_kv * (head_dim / 8);
  int threads = g.chunks;  // the least number of whole rows that is a number of whole warps (chunks is a multiple of 8)
  while (threads % 32) threads += g.chunks;
  if (threads <= kMaxRowThreads) {
    while (threads < 256 && threads * 2 <= kMaxRowThreads) threads *= 2;
    g.rows = threads / g.chunks;
    g.parts = 1;
  } else {  // one row, or 256 threads' part of it; the last warp's threads past the row idle
    threads = g.chunks < 256 ? (g.chunks + 31) / 32 * 32 : 256;
    g.rows = 1;
    g.parts = (g.chunks + threads - 1) / threads;
  }
  g.threads = threads;
  g.whole = g.chunks % 32 == 0 && (g.parts == 1 || g.chunks % threads == 0);
  return g;
}

// u: tokens a thread, 4 where that still gives every SM four CTAs, else 1; ctas: along x.
struct RowGrid {
  int u;
  long long ctas;
};

// loops: no more CTAs than run at once (their registers: 64 a thread, or 80 without whole rows)
inline RowGrid row_grid(const RowShape& g, int T, int sms, bool loops) {
  const long long one = (static_cast<long long>(T) + g.rows - 1) / g.rows, four = (one + 3) / 4;
  RowGrid r{};
  r.u = four * 2 * g.parts >= 4LL * sms ? 4 : 1;
  r.ctas = r.u == 4 ? four : one;
  if (loops) {
    const long long fit = static_cast<long long>(sms) * ((g.whole ? 1024 : 768) / g.threads) / (2 * g.parts);
    if (r.ctas > fit) r.ctas = fit < 1 ? 1 : fit;
  }
  return r;
}

// A thread's chunk `at` of the row, and the first of its U tokens, `rows` apart:
// t0 = cta + row.  there: it has something to do (other threads, and tokens past
// the end, load what the last ones do and store nothing).
struct RowPlace {
  uint32_t cta, t0;
  int at;
  bool there;
};

// row: thread / chunks; part: of the row, parts > 1
LLAMA_HOST_DEVICE RowPlace row_place(const RowShape& g, int U, uint32_t block, int part, int threads, int thread,
                                     int row) {
  RowPlace x;
  const int at = g.parts > 1 ? part * threads + thread : thread - row * g.chunks;
  x.at = g.whole ? at : at < g.chunks ? at : g.chunks - 1;
  x.there = x.at == at && row < g.rows;
  x.cta = block * static_cast<uint32_t>(g.rows * U);
  x.t0 = x.cta + (g.parts > 1 ? 0 : row);  // below T + rows * U < 2^32
  return x;
}

// tokens from one step of a CTA to its next
LLAMA_HOST_DEVICE uint32_t row_step(const RowShape& g, int U, uint32_t blocks) {
  return blocks * static_cast<uint32_t>(g.rows * U);  // at most 2^31 + 2^17
}

// The CTA has a step after the one at x.  By its first token, so that all of its
// threads go round together: the loop's body exchanges values over whole warps,
// whose lanes may hold rows of several tokens.
LLAMA_HOST_DEVICE bool row_more(const RowPlace& x, int T, uint32_t step) {
  return x.cta < static_cast<uint32_t>(T) && static_cast<uint32_t>(T) - x.cta > step;
}

}  // namespace llama
