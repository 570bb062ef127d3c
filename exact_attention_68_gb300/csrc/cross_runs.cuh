// cross_runs.cuh — the number of runs (cross_runs.h), found on the device, where the
// lengths are: the same in every thread of every kernel of a call.
#pragma once

#include <cuda_runtime.h>

#include "cross_runs.h"

namespace ea {
namespace {

__device__ __forceinline__ int cross_kv_runs(const KvRuns& k, const int* lens) {
  if (k.most_runs == 1) return 1;
  int tiles = 0;
  if (lens == nullptr) {
    tiles = k.batch * ((k.Sk + 127) / 128);
  } else {
    for (int b = 0; b < k.batch; ++b) tiles += (min(max(__ldg(lens + b), 0), k.Sk) + 127) / 128;
  }
  return kv_runs(k, tiles * k.heads);
}

}  // namespace
}  // namespace ea
