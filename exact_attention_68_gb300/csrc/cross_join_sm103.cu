// cross_join_sm103.cu — joins the runs that cross-attention's work is cut into
// where its tiles alone would leave SMs idle (few queries over many keys, or many
// queries over few keys).  Each run left its own fp32 result in the workspace;
// they are read once, in a fixed order, and rounded once.
//
// Bound by the workspace's bytes, which a run has just written and L2 mostly
// still holds.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cross_join.h"
#include "cross_runs.cuh"
#include "ptx.cuh"

namespace ea {
namespace {

constexpr int kJoinThreads = 256;

// One warp a row: lane r holds run r's weight (and run 32 + r's), every lane four
// (or eight) channels.
template <bool F16>
__global__ void __launch_bounds__(kJoinThreads) join_fwd_kernel(const __grid_constant__ JoinFwdParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  float e[2], m = -INFINITY;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = lane + 32 * i;
    e[i] = r < p.runs ? p.part_lse[r * p.rows + row] : -INFINITY;
    m = fmaxf(m, e[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float w[2], sum;
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = expf(e[i] - ref);
  // NaN among the runs (fmaxf passes it over) stays NaN: it is in w
  sum = w[0] + w[1];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int c0 = 0; c0 < p.D; c0 += 128) {
    const int c = c0 + lane * 4;
    const bool in = c < p.D;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* from = p.part_o + row * p.D + (in ? c : 0);
#pragma unroll 4
    for (int r = 0; r < p.runs; ++r) {
      const float wr = __shfl_sync(0xffffffffu, r < 32 ? w[0] : w[1], r & 31);
      const float4 o = *reinterpret_cast<const float4*>(from + r * p.rows * p.D);
      a.x = fmaf(wr, o.x, a.x), a.y = fmaf(wr, o.y, a.y), a.z = fmaf(wr, o.z, a.z), a.w = fmaf(wr, o.w, a.w);
    }
    if (!in) continue;
    uint2 v;
    v.x = pack_x2<F16>(a.x * inv, a.y * inv), v.y = pack_x2<F16>(a.z * inv, a.w * inv);
    *reinterpret_cast<uint2*>(p.out + row * p.D + c) = v;
  }
  if (lane == 0) p.lse[row] = m == -INFINITY && sum == 0.f ? -INFINITY : m + logf(sum);
}

struct JoinSums {
  JoinSumParams p[2];
};

// A thread takes eight channels of a row.
template <bool F16>
__global__ void __launch_bounds__(kJoinThreads) join_sum_kernel(const __grid_constant__ JoinSums ps) {
  const JoinSumParams& p = ps.p[blockIdx.y];
  const int runs = p.of_keys ? cross_kv_runs(p.kv, p.lens) : p.runs;
  if (p.of_keys && runs == 1) return;
  const int units = p.D / 8;
  const int64_t total = p.rows * units;
  for (int64_t x = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; x < total;
       x += (int64_t)gridDim.x * kJoinThreads) {
    const int64_t row = x / units;
    bool there = true;
    if (p.lens != nullptr) {
      const int64_t slice = row / p.kv.Sk;
      const int key = static_cast<int>(row - slice * p.kv.Sk);
      const int n = min(max(__ldg(p.lens + slice / p.kv.heads), 0), p.kv.Sk);
      if ((key & ~127) >= n) continue;
      there = key < n;
    }
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    if (there) {
      const float* from = p.part + x * 8;
#pragma unroll 4
      for (int r = 0; r < runs; ++r) {
        const float4* f = reinterpret_cast<const float4*>(from + r * p.rows * p.D);
        const float4 a = f[0], b = f[1];
        s[0] += a.x, s[1] += a.y, s[2] += a.z, s[3] += a.w;
        s[4] += b.x, s[5] += b.y, s[6] += b.z, s[7] += b.w;
      }
    }
    uint4 v;
    v.x = pack_x2<F16>(s[0] * p.mul, s[1] * p.mul), v.y = pack_x2<F16>(s[2] * p.mul, s[3] * p.mul);
    v.z = pack_x2<F16>(s[4] * p.mul, s[5] * p.mul), v.w = pack_x2<F16>(s[6] * p.mul, s[7] * p.mul);
    *reinterpret_cast<uint4*>(p.to + x * 8) = v;
  }
}

}  // namespace

cudaError_t join_fwd_launch(const JoinFwdParams& p, bool f16, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)), 1, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.stream = stream;
  return f16 ? cudaLaunchKernelEx(&cfg, join_fwd_kernel<true>, p) : cudaLaunchKernelEx(&cfg, join_fwd_kernel<false>, p);
}

cudaError_t join_sum_launch(const JoinSumParams* p, int n, bool f16, cudaStream_t stream) {
  JoinSums ps;
  for (int i = 0; i < 2; ++i) ps.p[i] = p[i < n ? i : 0];
  const int64_t ctas = (p->rows * (p->D / 8) + kJoinThreads - 1) / kJoinThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < 65536 ? ctas : 65536), static_cast<unsigned>(n), 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.stream = stream;
  return f16 ? cudaLaunchKernelEx(&cfg, join_sum_kernel<true>, ps) : cudaLaunchKernelEx(&cfg, join_sum_kernel<false>, ps);
}

}  // namespace ea
