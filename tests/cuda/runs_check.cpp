// runs_check.cpp — test-only host shim over the number of runs that cross-attention's
// gradient cuts its sums into (cross_runs.h).
#include "cross_runs.h"

extern "C" {

// The number of runs for `tiles` key tiles of a call's slices.
__attribute__((visibility("default"))) int runs_of(int64_t batch, int64_t heads, int64_t Sk, int64_t rows, int64_t D,
                                                   int width, int sms, int tiles) {
  return ea::kv_runs(ea::plan_kv_runs(batch, heads, Sk, rows, D, width, sms), tiles);
}

// The most that the workspace has room for.
__attribute__((visibility("default"))) int most_runs(int64_t batch, int64_t heads, int64_t Sk, int64_t rows, int64_t D,
                                                     int width, int sms) {
  return ea::plan_kv_runs(batch, heads, Sk, rows, D, width, sms).most_runs;
}
}
