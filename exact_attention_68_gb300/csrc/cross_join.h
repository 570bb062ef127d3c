// cross_join.h — launch entries of the kernels that join the runs that
// cross-attention's work was cut into (host-compilable).
#pragma once

#include <cstdint>
#include <cuda_runtime_api.h>

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
};
cudaError_t join_fwd_launch(const JoinFwdParams& p, bool f16, cudaStream_t stream);

// A gradient's runs: to = mul · Σ part_r.  With keys (lens or Sk): rows are a
// slice's Sk keys; those behind the sequence's end get 0, and whole tiles of 128
// of them are left alone.
struct JoinSumParams {
  const float* part;  // [runs, rows, D]
  uint16_t* to;       // [rows, D]
  int64_t rows;
  int runs, D;
  float mul;
  const int* lens;  // null: every row is there
  int heads, Sk;
};
// n tensors (1 or 2) of the same sizes in one launch.
cudaError_t join_sum_launch(const JoinSumParams* p, int n, bool f16, cudaStream_t stream);

}  // namespace ea
