// cross_runs.cuh — the number of runs (cross_runs.h), found on the device, where the
// lengths are: the same in every thread of every kernel of a call.
#pragma once

#include <cuda_runtime.h>

#include "cross_runs.h"

namespace ea {
namespace {

// The number of runs with the shortest expected time: rounds of the SMs over all
// (tile, run) units, each its steps and 1.5 more for its start and end, then the join,
// a launch and the runs' bytes.  2 x 16 heads of 300 and 100 keys, 4096 queries of
// 128 channels: 64 of 152 SMs would have a tile in one run.
__device__ __forceinline__ int cross_kv_runs(const KvRuns& k, const int* lens) {
  if (k.most_runs == 1) return 1;
  int tiles = 0;
  if (lens == nullptr) {
    tiles = k.batch * ((k.Sk + 127) / 128);
  } else {
    for (int b = 0; b < k.batch; ++b) tiles += (min(max(__ldg(lens + b), 0), k.Sk) + 127) / 128;
  }
  tiles *= k.heads;
  int best = 1;
  float least = 0.f;
  for (int n = 1; n <= k.most_runs; ++n) {
    const int rounds = (tiles * k.ctas * n + k.sms - 1) / k.sms, steps = (k.q_steps + n - 1) / n;
    float t = rounds * (steps + 1.5f) * k.step_us;
    if (n > 1) t += 3.f + k.run_us * tiles * n;
    if (n == 1 || t < least) best = n, least = t;
  }
  return best;
}

}  // namespace
}  // namespace ea
