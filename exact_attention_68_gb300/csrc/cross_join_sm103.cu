// cross_join_sm103.cu — joins the runs that cross-attention's work is cut into
// where its tiles alone would leave SMs idle (few queries over many keys, or many
// queries over few keys).  Each run left its own fp32 result in the workspace;
// they are read once, in a fixed order, and rounded once.
//
// Bound by the workspace's bytes, which a run has just written and L2 mostly
// still holds, and by their own start: apart and with cold caches dk and dv of 2 x 16
// heads of 300 and 100 keys take 10 us, 1024 rows of 128 channels in 16 runs 8.5.  In a
// call they are set up while the kernel before them ends.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cross_join.h"
#include "cross_runs.cuh"
#include "launch_after.cuh"
#include "ptx.cuh"

namespace ea {
namespace {

constexpr int kJoinThreads = 256;

// A CTA a row: D/4 threads side by side read a run's four channels each, as many
// groups of them as there are threads take every so many-th run, so that all runs'
// loads are in flight at once.  Each warp finds the runs' weights for itself.
constexpr int kFwdThreads = 256;
template <bool F16>
__global__ void __launch_bounds__(kFwdThreads) join_fwd_kernel(const __grid_constant__ JoinFwdParams p) {
  __shared__ float s_w[kFwdThreads / 32][kMaxRuns];
  __shared__ float4 s_sum[kFwdThreads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x;
  const int quads = p.D / 4, groups = kFwdThreads / quads;  // quads <= 64
  const int group = tid / quads, c = tid - group * quads;
  constexpr int kHeld = 8;
  float4 held[kHeld];
  wait_for_previous();
  const float* from = p.part_o + row * p.D + 4 * c;
  const int64_t stride = p.rows * p.D;
  if (group < groups) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (group + i * groups < p.runs) held[i] = __ldcg(reinterpret_cast<const float4*>(from + (group + i * groups) * stride));
  }
  float e[2], m = -INFINITY;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = lane + 32 * i;
    e[i] = r < p.runs ? __ldcg(p.part_lse + r * p.rows + row) : -INFINITY;
    m = fmaxf(m, e[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float w = expf(e[i] - ref);  // NaN among the runs, which the maximum passed over, stays
    s_w[warp][lane + 32 * i] = w;
    sum += w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncwarp();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int r, const float4& o) {
    const float w = s_w[warp][r];
    a.x = fmaf(w, o.x, a.x), a.y = fmaf(w, o.y, a.y), a.z = fmaf(w, o.z, a.z), a.w = fmaf(w, o.w, a.w);
  };
  if (group < groups) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (group + i * groups < p.runs) add(group + i * groups, held[i]);
    for (int r = group + kHeld * groups; r < p.runs; r += groups)
      add(r, __ldcg(reinterpret_cast<const float4*>(from + r * stride)));
  }
  s_sum[tid] = a;
  __syncthreads();
  if (group != 0) return;
  for (int g = 1; g < groups; ++g) {
    const float4 o = s_sum[g * quads + c];
    a.x += o.x, a.y += o.y, a.z += o.z, a.w += o.w;
  }
  // no sum: no keys, or none with a score but -inf, 0 / 0
  const bool none = sum == 0.f && p.lens != nullptr && __ldg(p.lens + row / p.seq_rows) <= 0;
  const float inv = none ? 0.f : 1.f / sum;
  uint2 v;
  v.x = pack_x2<F16>(a.x * inv, a.y * inv), v.y = pack_x2<F16>(a.z * inv, a.w * inv);
  *reinterpret_cast<uint2*>(p.out + row * p.D + 4 * c) = v;
  if (c == 0) p.lse[row] = sum == 0.f ? -INFINITY : m + logf(sum);
}

struct JoinSums {
  JoinSumParams p[kMaxSums];
};

// A thread takes eight channels of a row, a CTA as many rows as fit.  What needs no sums
// (the number of runs, found by one thread; the row's sequence) is done while the
// kernel before this one ends.
template <bool F16>
__global__ void __launch_bounds__(kJoinThreads) join_sum_kernel(const __grid_constant__ JoinSums ps) {
  const JoinSumParams& p = ps.p[blockIdx.y];
  __shared__ int s_runs;
  if (threadIdx.x == 0) s_runs = p.of_keys ? cross_kv_runs(p.kv, p.lens) : p.runs;
  const int units = p.D / 8, per_cta = kJoinThreads / units;
  const int r = static_cast<int>(threadIdx.x) / units, c = static_cast<int>(threadIdx.x) - r * units;
  const int64_t row = (int64_t)blockIdx.x * per_cta + r;
  bool mine = r < per_cta && row < p.rows, there = true;
  if (mine && p.lens != nullptr) {
    const int slice = static_cast<int>(row) / p.kv.Sk, key = static_cast<int>(row) - slice * p.kv.Sk;
    const int n = min(max(__ldg(p.lens + slice / p.kv.heads), 0), p.kv.Sk);
    there = key < n;
    mine = (key & ~127) < n;
  }
  __syncthreads();
  const int runs = s_runs;
  wait_for_previous();
  if (!mine || (p.of_keys && runs == 1)) return;
  const int64_t at = row * p.D + 8 * c;
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.f;
  if (there) {
    const float* from = p.part + at;
#pragma unroll 8
    for (int i = 0; i < runs; ++i) {
      const float4* f = reinterpret_cast<const float4*>(from + i * p.rows * p.D);
      const float4 a = __ldcg(f), b = __ldcg(f + 1);
      s[0] += a.x, s[1] += a.y, s[2] += a.z, s[3] += a.w;
      s[4] += b.x, s[5] += b.y, s[6] += b.z, s[7] += b.w;
    }
  }
  uint4 v;
  v.x = pack_x2<F16>(s[0] * p.mul, s[1] * p.mul), v.y = pack_x2<F16>(s[2] * p.mul, s[3] * p.mul);
  v.z = pack_x2<F16>(s[4] * p.mul, s[5] * p.mul), v.w = pack_x2<F16>(s[6] * p.mul, s[7] * p.mul);
  *reinterpret_cast<uint4*>(p.to + at) = v;
}

}  // namespace

cudaError_t join_fwd_launch(const JoinFwdParams& p, bool f16, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.rows), 1, 1);
  return f16 ? launch_after(join_fwd_kernel<true>, grid, kFwdThreads, stream, p)
             : launch_after(join_fwd_kernel<false>, grid, kFwdThreads, stream, p);
}

cudaError_t join_sum_launch(const JoinSumParams* p, int n, bool f16, cudaStream_t stream) {
  JoinSums ps;
  int64_t ctas = 0;
  for (int i = 0; i < kMaxSums; ++i) {
    ps.p[i] = p[i < n ? i : 0];
    // work is cut into runs only where its tiles are few: fewer rows than 4 tiles an SM
    if (ps.p[i].rows > INT32_MAX) return cudaErrorInvalidValue;
    const int per_cta = kJoinThreads / (ps.p[i].D / 8);
    const int64_t c = (ps.p[i].rows + per_cta - 1) / per_cta;
    ctas = c > ctas ? c : ctas;
  }
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(n), 1);
  return f16 ? launch_after(join_sum_kernel<true>, grid, kJoinThreads, stream, ps)
             : launch_after(join_sum_kernel<false>, grid, kJoinThreads, stream, ps);
}

}  // namespace ea
