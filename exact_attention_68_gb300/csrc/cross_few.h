// cross_few.h — parameters and launch entries of cross-attention's kernels for few
// queries, and of its gradient for few queries and keys (host-compilable).
#pragma once

#include <cstdint>
#include <cuda_runtime_api.h>

namespace ea {

constexpr int kFewRows = 16, kFewWidth = 64;  // rows and channels of a slice that it is made for

struct FewParams {
  const uint16_t* q;  // [BH, rows, D]
  const uint16_t* k;  // [BH, Sk, D]
  const uint16_t* v;
  const int* lens;    // [BH / heads] or null
  uint16_t* out;      // [BH, rows, D]
  float* lse;         // [BH, rows]
  float* part_o;      // [runs, BH, rows, D] if runs > 1
  float* part_lse;    // [runs, BH, rows]
  int* status;
  int BH, heads, rows, Sk, D;
  int cluster;        // CTAs that share a slice's keys: 1, 2, 4 or 8
  int runs;           // into which they are cut first
  float scale_log2;
};

cudaError_t cross_few_launch(const FewParams& p, bool f16, cudaStream_t stream);

constexpr int kSmallSide = 64;  // queries and keys of a slice that the small gradient takes

struct SmallBwdParams {
  const uint16_t* q;  // [BH, rows, D]
  const uint16_t* k;  // [BH, Sk, D]
  const uint16_t* v;
  const int* lens;    // [BH / heads] or null
  const uint16_t* out;
  const float* lse;   // [BH, rows]
  const uint16_t* dout;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  float* delta;
  int* status;
  int BH, heads, rows, Sk, D;
  float scale, scale_log2;
};
cudaError_t cross_small_bwd_launch(const SmallBwdParams& p, int width, bool f16, cudaStream_t stream);

}  // namespace ea
