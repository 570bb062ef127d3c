// cross_runs.h — how dk and dv's sums over the queries are cut into runs, from sizes
// and lengths: shared by the host, the gradient kernels and the kernel that joins
// the runs (host-compilable).
//
// Each kernel of a call finds the number of runs for itself, and all have to find the
// same one.  So the times that are compared are whole numbers: in floating point a
// compiler may contract a product and a sum in one kernel and not in another, and
// near ties exist (497 key tiles of 56 channels, 8064 queries: two runs or three).
#pragma once

#include <cstdint>

#include "schedule.h"  // EA_HOST_DEVICE

namespace ea {

struct KvRuns {
  int batch, heads, Sk;
  int q_steps;         // steps that a key tile's sums go over
  int ctas;            // CTAs a tile takes (2: a half of the head dimension each)
  int most_runs;       // that the workspace has room for
  int sms;
  uint32_t half_step;  // time of half a step, in nanoseconds
  uint32_t run;        // of writing one run's sums of one key tile and reading them back, in 1/625 ns
};

// The plan for slices of `rows` queries, in kernels `width` columns wide.
inline KvRuns plan_kv_runs(int64_t batch, int64_t heads, int64_t Sk, int64_t rows, int64_t D, int width, int sms) {
  KvRuns k;
  const int step = width == 256 ? 64 : 128;  // queries
  k.batch = static_cast<int>(batch), k.heads = static_cast<int>(heads), k.Sk = static_cast<int>(Sk);
  k.q_steps = static_cast<int>((rows + step - 1) / step);
  k.ctas = width == 256 ? 2 : 1;
  k.sms = sms;
  k.half_step = width == 64 ? 600 : width == 128 ? 950 : 850;
  k.run = static_cast<uint32_t>(256 * D);  // 128 · D · 8 · 2 bytes at 5 TB/s: 256 / 625 · D ns
  // runs are of use where there may be fewer key tiles than SMs, or not many more
  const bool few = batch * heads * ((Sk + 127) / 128) * k.ctas < 4 * sms;
  k.most_runs = !few ? 1 : k.q_steps < 8 ? k.q_steps : 8;
  return k;
}

// The number of runs with the shortest expected time for `tiles` key tiles: rounds of
// the SMs over all (tile, run) units, each its steps and 1.5 more for its start and end,
// then the join, a launch of 3 us and the runs' bytes.  2 x 16 heads of 300 and 100 keys,
// 4096 queries of 128 channels: 64 of 152 SMs would have a tile in one run.
// (Runs are cut where there are at most 4 units an SM, 32 with the runs, so that rounds
// times half steps fit 32 bits: 64 throughout cost 0.7 us a call.)
EA_HOST_DEVICE int kv_runs(const KvRuns& k, int tiles) {
  int best = 1;
  uint64_t least = 0;
  for (int n = 1; n <= k.most_runs; ++n) {
    const uint32_t rounds = (tiles * k.ctas * n + k.sms - 1) / k.sms, steps = (k.q_steps + n - 1) / n;
    uint64_t t = uint64_t(rounds * (2 * steps + 3)) * k.half_step;
    if (n > 1) t += 3000 + k.run * uint32_t(tiles * n) / 625;
    if (n == 1 || t < least) best = n, least = t;
  }
  return best;
}

}  // namespace ea
