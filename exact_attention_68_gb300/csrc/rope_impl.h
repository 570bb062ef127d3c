// rope_impl.h — kernel parameters and launch entries shared by the host API of
// the heads' norm and rotation and its kernels (host-compilable).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

namespace ea {

constexpr int kRopeMaxParts = 4;
constexpr int kRopeMaxPairs = 128;

struct RopePart {
  const uint16_t* x;
  int64_t xb, xs, xh;  // strides of x
  uint16_t* y;         // [B, heads, S, D]: written by the forward, read (dy) by the backward
  uint16_t* dx;
  int64_t db, ds, dh;  // strides of dx
  const void* weight;  // [D] or null
  void* dweight;       // [D] or null
  float* sums;         // workspace: [CTAs of the grid][D], null without dweight
  int heads;
  int weight_f32, turn;
  int slot;            // which of the launch's two weight gradients, -1: none
};

struct RopeParams {
  RopePart part[kRopeMaxParts];
  uint64_t turns[kRopeMaxPairs];  // inv_freq / 2π: the fraction of a turn a position adds, times 2^64
  uint8_t axis[kRopeMaxPairs];
  const int* at;
  int64_t pb, ps, pa;  // strides of the positions
  int n_parts;
  int pairs;           // 0: no part turns
  int N, S, D;         // tokens in all, tokens of a sequence, channels
  uint64_t s_mul;      // n / S = (n · s_mul) >> s_shift for n < 2^30
  int s_shift;
  int lanes, per_warp; // of a row; rows a warp takes at once
  int split, log2_split;  // units that one token is dealt to, by heads
  int units;
  float eps, inv_d;
  int* status;
};

// How a row's channels go to threads: see rope_sm103.cu.
struct RopeShape {
  bool interleaved;
  int width;  // pairs of one vector: 8, 4, 2 or 1; 4 where interleaved
};

// Fills in lanes, per_warp, split and units; CTAs of the grid.
int rope_plan(RopeParams& p, RopeShape shape, bool bwd, int sms);

// The most CTAs that the gradient's grid has on a device of `sms` SMs.
int rope_most_ctas(int sms);

cudaError_t rope_fwd_launch(const RopeParams& p, RopeShape shape, bool f16, int ctas, cudaStream_t stream);
// Then the second kernel that adds up dweight, if any part has sums.
cudaError_t rope_bwd_launch(const RopeParams& p, RopeShape shape, bool f16, int ctas, cudaStream_t stream);

}  // namespace ea
