// cross_join.h — launch entries of the kernels that join the runs that
// cross-attention's work was cut into (host-compilable).
#pragma once

#include <cstdint>
#include <cuda_runtime_api.h>

#include "cross_runs.h"

namespace ea {

constexpr int kMaxRuns = 64;  // of one tile's work

// The forward's runs: out = Σ w_r · o_r, lse = ln Σ exp(lse_r), w_r = exp(lse_r - lse).
struct JoinFwdParams {
  const float* part_o;    // [runs, rows, D]
  const float* part_lse;  // [runs, rows]
  uint16_t* out;          // [rows, D]
  float* lse;             // [rows]
  int64_t rows;
  int runs, D;
  const int* lens;        // [rows / seq_rows] keys that are there; null: some everywhere
  int64_t seq_rows;       // rows of a sequence
};
cudaError_t join_fwd_launch(const JoinFwdParams& p, bool f16, cudaStream_t stream);

// A gradient's runs: to = mul · Σ part_r.  Of keys: rows are a slice's Sk keys, the
// number of runs is found as the gradient kernel finds it (one: nothing is left to
// do); those behind the sequence's end get 0, and whole tiles of 128 of them are left
// alone.
struct JoinSumParams {
  const float* part;  // [runs, rows, D]
  uint16_t* to;       // [rows, D]
  int64_t rows;
  int runs, D;      // runs: of queries' gradients
  float mul;
  bool of_keys;
  KvRuns kv;
  const int* lens;  // null: every key is there
};
// n tensors (1 to kMaxSums) in one launch.
constexpr int kMaxSums = 3;
cudaError_t join_sum_launch(const JoinSumParams* p, int n, bool f16, cudaStream_t stream);

}  // namespace ea
