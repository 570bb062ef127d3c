// cross_few.h — parameters and launch entry of cross-attention's kernel for few
// queries (host-compilable).
#pragma once

#include <cstdint>
#include <cuda_runtime_api.h>

namespace ea {

constexpr int kFewRows = 32;  // rows of a slice that it is made for

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
  int groups;         // of 16 · tiles rows
  int cluster;        // CTAs that share a group's keys: 1, 2, 4 or 8
  int runs;           // into which they are cut first
  float scale_log2;
};

// width: 64, 128 or 256 columns; tiles: of 16 rows a CTA takes, 1 or 2 (256 columns: 1).
cudaError_t cross_few_launch(const FewParams& p, int width, int tiles, bool f16, cudaStream_t stream);

}  // namespace ea
