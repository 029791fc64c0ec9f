// Host walk over csrc/cache_rows.h for the tests: which (token, chunk) pairs the
// threads of a launch handle, and how often the lanes of a warp go round.
#include <vector>

#include "cache_rows.h"

using namespace llama;

// out[0]: warps whose lanes leave the loop at different steps; out[1], out[2]: (token, chunk) pairs that no thread has,
// and that more than one has; out[3]: chunks out of range; out[4]: tokens a thread; out[5]: steps of the first CTA;
// out[6]: 1 if a row is whole warps; out[7]: lanes whose neighbour (lane ^ 1, or lane + 2 of a first one of four) holds
// another token or another part of the row.
extern "C" void walk(int n_kv, int head_dim, int T, int sms, int loops, long long* out) {
  const RowShape g = row_shape(n_kv, head_dim);
  const RowGrid r = row_grid(g, T, sms, loops != 0);
  const uint32_t step = row_step(g, r.u, static_cast<uint32_t>(r.ctas));
  std::vector<int> seen(static_cast<size_t>(T) * g.chunks, 0);
  for (int i = 0; i < 8; ++i) out[i] = 0;
  out[4] = r.u;
  out[6] = g.whole;
  for (long long block = 0; block < r.ctas; ++block)
    for (int part = 0; part < g.parts; ++part)
      for (int first = 0; first < g.threads; first += 32) {
        int least = 1 << 30, most = 0;
        RowPlace lanes[32];
        for (int lane = 0; lane < 32; ++lane) {
          const int thread = first + lane;
          RowPlace x = row_place(g, r.u, static_cast<uint32_t>(block), part, g.threads, thread, thread / g.chunks);
          lanes[lane] = x;
          if (x.at < 0 || x.at >= g.chunks) {
            ++out[3];
            continue;
          }
          int steps = 0;
          for (bool more = true; more;) {
            for (int n = 0; n < r.u; ++n) {
              const uint32_t t = x.t0 + n * g.rows;
              if (x.there && t < static_cast<uint32_t>(T)) ++seen[static_cast<size_t>(t) * g.chunks + x.at];
            }
            ++steps;
            more = loops && row_more(x, T, step);
            x.cta += step;
            x.t0 += step;
          }
          least = steps < least ? steps : least;
          most = steps > most ? steps : most;
          if (block == 0 && part == 0 && thread == 0) out[5] = steps;
        }
        out[0] += least != most;
        for (int lane = 0; lane < 32; ++lane) {
          const RowPlace &x = lanes[lane], &y = lanes[lane ^ 1], &z = lanes[lane + 2 < 32 ? lane + 2 : lane];
          if (!x.there) continue;
          if (y.t0 != x.t0 || y.at != (x.at ^ 1)) ++out[7];
          if (x.at % 4 == 0 && (z.t0 != x.t0 || z.at != x.at + 2)) ++out[7];
        }
      }
  for (const int n : seen) {
    out[1] += n == 0;
    out[2] += n > 1;
  }
}
