// cross_runs.h — how dk and dv's sums over the queries are cut into runs, from sizes
// and lengths: shared by the host, the gradient kernels and the kernel that joins
// the runs (host-compilable).
#pragma once

#include <cstdint>

namespace ea {

struct KvRuns {
  int batch, heads, Sk;
  int q_steps;      // steps that a key tile's sums go over
  int ctas;         // CTAs a tile takes (2: a half of the head dimension each)
  int most_runs;    // that the workspace has room for
  int sms;
  float step_us;    // of one step
  float run_us;     // of writing one run's sums of one key tile and reading them back
};

}  // namespace ea
