// rope_impl.h — kernel parameters and launch entries shared by the host API of
// the heads' norm and rotation and its kernels (host-compilable).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

namespace ea {

constexpr int kRopeMaxParts = 4;
constexpr int kRopeMaxPairs = 128;
constexpr int kRopeThreads = 256;

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
};

struct RopeParams {
  RopePart part[kRopeMaxParts];
  uint64_t turns[kRopeMaxPairs];  // inv_freq / 2π: the fraction of a turn a position adds, times 2^64
  uint8_t axis[kRopeMaxPairs];
  const int* at;
  int64_t pb, ps, pa;  // strides of the positions
  int n_parts;
  int pairs;        // 0: no part turns
  int B, S, D;
  int log2_tokens;  // tokens a CTA takes at once
  int blocks;       // of that many tokens
  int head_split;   // CTAs a block's heads are dealt to
  float eps, inv_d;
  int* status;
};

// How many channels of a row a thread takes, and how: see rope_sm103.cu.
struct RopeShape {
  bool interleaved;
  int width;  // pairs of one vector: 8, 4, 2 or 1; 4 where interleaved
};

// CTAs of the backward's grid that add to dweight.
int rope_bwd_grid(const RopeParams& p, int sms);

cudaError_t rope_fwd_launch(const RopeParams& p, RopeShape shape, bool f16, cudaStream_t stream);
cudaError_t rope_bwd_launch(const RopeParams& p, RopeShape shape, bool f16, int sms, cudaStream_t stream);

}  // namespace ea
