// cross_few_sm103.cu — cross-attention of few queries (a decoder's next tokens) on
// GB300 (sm_103a): up to 16 rows a slice, the G query heads of a key head together, of up
// to 64 channels.
//
// Bound by the memory: K and V are read once for a handful of rows.  The persistent
// kernel pads them to 128 rows and pays its pipeline's start for a few steps; here
// what counts is how soon all SMs have enough loads in flight and how short the
// chain behind the last one is.  (Beyond 16 rows, or 64 channels, the persistent
// kernel is the faster one: cross_api.cu.)
//
//   A warp works by itself: it takes chunks of 32 keys, brings K
//   and V of the next ones into its own ring in shared memory (cp.async), and keeps
//   its own running maximum, sums and output for 16 rows in registers:
//   S = Q·Kᵀ and O += P·V by mma.sync m16n8k16, P from S's registers.  16 rows cost
//   what one does; the products take a fifth of the memory's time at 16 rows.
//   Keys behind the sequence's end are not read: their copies fill in zeros.
//   A slice's keys are dealt to the 4 warps of each CTA of a cluster; the CTA joins its
//   warps' parts through shared memory, the cluster its CTAs' through distributed
//   shared memory, each CTA a share of the values: one launch, no workspace.  Where
//   even clusters of 8 leave SMs idle (few slices, long keys) the keys are cut
//   into runs first, which a second kernel joins.
//
// Measured on a GB300, calls in a graph: 8 x 16 slices of one query, 300 to 1500 keys of
// 64 channels in fp16 10.7 us, 2.8 TB/s; the persistent kernel takes 13.5.  By then all of K
// and V has long been asked for; the rest is launch, length, first chunk and the two joins
// one after the other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "bwd_common.cuh"
#include "cross_common.cuh"
#include "cross_few.h"
#include "launch_after.cuh"
#include "mma_sync.cuh"
#include "ptx.cuh"

namespace ea {
namespace {

constexpr float kLn2F = 0.6931471805599453f;

enum : int { kChkFewRow = 0x5711 };

struct FewLayout {
  static constexpr int W = 64;
  static constexpr int kWarps = 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kChunk = 32;                      // keys of a warp's step
  static constexpr int kStages = 3;                      // 96 KB a CTA, two of them an SM
  static constexpr int kRow = W * 2;                     // bytes
  static constexpr int kPart = kChunk * kRow;            // K or V of a chunk
  static constexpr int kWarpRing = kStages * 2 * kPart;
  static constexpr int kRows = kFewRows;
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = kQOff + kRows * kRow;
  static constexpr int kOut = kRows * W * 4;             // one fp32 output
  // after the keys the ring holds the warps' outputs, then the CTA's
  static constexpr int kRing = kWarps * kWarpRing > (kWarps + 1) * kOut ? kWarps * kWarpRing : (kWarps + 1) * kOut;
  static constexpr int kStatOff = kRingOff + kRing;      // [warps + 1][rows] of (max, sum, rounded sum, -)
  static constexpr int kAlloc = kStatOff + (kWarps + 1) * kRows * 16;
  static_assert(kAlloc <= 232448, "shared memory budget exceeded");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (not .aligned: the loops before it leave a warp's threads at different times)
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// This CTA's shared address as that of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 r;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 r;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ void st_shared_f4(uint32_t addr, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void st_shared_f2(uint32_t addr, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// 2^(m - ref): what a part with maximum m counts against the joint one; 1 where
// neither has a finite score (its sums are then 0, or NaN, which stays)
__device__ __forceinline__ float weight_of(float m, float ref) { return ref == -INFINITY ? 1.f : ex2_approx(m - ref); }

template <bool F16>
__global__ void __launch_bounds__(FewLayout::kThreads) cross_few_kernel(const __grid_constant__ FewParams p) {
  using L = FewLayout;
  constexpr int W = L::W;
  constexpr int kUnits = W / 8;  // 16-byte units of a row
  constexpr int kFewWarps = L::kWarps, kFewThreads = L::kThreads;
  extern __shared__ __align__(128) uint8_t few_smem[];
  const uint32_t sb = smem_u32(few_smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = p.cluster > 1 ? cluster_rank() : 0u;
  if (p.runs > 1) launch_dependents();
  int x = static_cast<int>(blockIdx.x) / p.cluster;
  const int run = x % p.runs;
  const int bh = x / p.runs, rows = p.rows;
  const int len = cross_len(p.lens, bh / p.heads, p.Sk, p.status);
  const int ksteps = (p.D + 15) / 16;

  // this run's chunks, and this warp's among them
  const int chunks = (len + L::kChunk - 1) / L::kChunk, each = chunks / p.runs, more = chunks - each * p.runs;
  const int c_first = run * each + min(run, more), c_end = c_first + each + (run < more ? 1 : 0);
  const int stride = p.cluster * kFewWarps;
  const int c0 = c_first + static_cast<int>(rank) * kFewWarps + warp;

  // 16-byte unit u of row r of a tile, swizzled so that 8 rows' units fill 8 places
  auto at = [](int r, int u) -> uint32_t { return static_cast<uint32_t>(r * L::kRow + ((u ^ (r & 7)) << 4)); };
  const uint32_t ring = sb + L::kRingOff + warp * L::kWarpRing;
  const int64_t kv0 = (int64_t)bh * p.Sk * p.D;
  const int lu = lane % kUnits, lr = lane / kUnits;  // this lane's unit and row of a copy
  constexpr int kAtOnce = 32 / kUnits;
  auto fetch = [&](int c, int stage) {
    if (c < c_end && 8 * lu < p.D) {
      const uint32_t kd = ring + stage * 2 * L::kPart, vd = kd + L::kPart;
#pragma unroll
      for (int r = 0; r < L::kChunk; r += kAtOnce) {
        const int key = c * L::kChunk + r + lr;
        const bool in = key < len;
        const int64_t off = kv0 + (int64_t)(in ? key : 0) * p.D + 8 * lu;
        copy16(kd + at(r + lr, lu), p.k + off, in);
        copy16(vd + at(r + lr, lu), p.v + off, in);
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int s = 0; s < L::kStages - 1; ++s) fetch(c0 + s * stride, s);

  // Q into shared memory, zeros for rows and channels that are not; and zeros for K's
  // channels up to the next 16
  for (int i = threadIdx.x; i < L::kRows * kUnits; i += kFewThreads) {
    const int r = i / kUnits, u = i % kUnits;
    const bool in = r < rows && 8 * u < p.D;
    if (kDebugChecks && in && (bh >= p.BH || rows > L::kRows)) dbg_fail(p.status, kChkFewRow);
    const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(p.q + ((int64_t)bh * p.rows + r) * p.D + 8 * u))
                       : make_uint4(0u, 0u, 0u, 0u);
    st_shared_v4(sb + L::kQOff + at(r, u), v.x, v.y, v.z, v.w);
  }
  if (p.D % 16 != 0)
    for (int i = lane; i < L::kStages * L::kChunk; i += 32)
      st_shared_v4(ring + (i / L::kChunk) * 2 * L::kPart + at(i % L::kChunk, p.D / 8), 0u, 0u, 0u, 0u);
  __syncthreads();

  float o[kUnits][4];  // O: rows lane/4 and + 8, channels 8n + 2·(lane % 4), + 1
  float m[2], l[2], lq[2];
#pragma unroll
  for (int n = 0; n < kUnits; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) m[h] = -INFINITY, l[h] = lq[h] = 0.f;
  constexpr int kTiles = L::kChunk / 8;  // of 8 keys
  const int mi = lane >> 3, mr = lane & 7;  // matrix and row of this lane's ldmatrix address
  int stage = 0;
  for (int c = c0; c < c_end; c += stride) {
    copies_wait<L::kStages - 2>();
    __syncwarp();
    const uint32_t kt = ring + stage * 2 * L::kPart, vt = kt + L::kPart;
    float s[kTiles][4];
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < W / 16; ++kk) {
      if (kk >= ksteps) break;
      uint32_t a[4];
      ldm4(a, sb + L::kQOff + at((mi & 1) * 8 + mr, 2 * kk + (mi >> 1)));
#pragma unroll
      for (int n = 0; n < kTiles; n += 2) {
        uint32_t b[4];  // keys 8n .. +7: channels lo, hi; keys 8n + 8 ..: lo, hi
        ldm4(b, kt + at(8 * n + (mi >> 1) * 8 + mr, 2 * kk + (mi & 1)));
        mma16816<F16>(s[n], a, b[0], b[1]);
        mma16816<F16>(s[n + 1], a, b[2], b[3]);
      }
    }
    // keys that are not there
    const int left = len - c * L::kChunk;
    if (left < L::kChunk) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * n + 2 * (lane & 3) + (e & 1) >= left) s[n][e] = -INFINITY;
    }
    uint32_t pk[kTiles][2];  // P of the two rows, packed
    float alpha[2];
    bool moved = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * h], s[n][2 * h + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float to = fmaxf(m[h], mx * p.scale_log2);
      alpha[h] = m[h] == to ? 1.f : ex2_approx(m[h] - to);  // 0 from -inf
      moved = moved || (alpha[h] != 1.f && m[h] != -INFINITY);
      m[h] = to;
      const float neg = to == -INFINITY ? 0.f : -to;
      float sum = 0.f, sum_q = 0.f;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        const float p0 = ex2_approx(fmaf(s[n][2 * h], p.scale_log2, neg));
        const float p1 = ex2_approx(fmaf(s[n][2 * h + 1], p.scale_log2, neg));
        sum += p0 + p1;
        pk[n][h] = pack_x2<F16>(p0, p1);
        // what the products weigh with: it normalises the output
        if constexpr (F16) {
          const float2 q2 = f16x2_to_f32(pk[n][h]);
          sum_q += q2.x + q2.y;
        } else {
          sum_q += bf16_lo(pk[n][h]) + bf16_hi(pk[n][h]);
        }
      }
      l[h] = l[h] * alpha[h] + sum;
      lq[h] = lq[h] * alpha[h] + sum_q;
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int n = 0; n < kUnits; ++n) {
        o[n][0] *= alpha[0], o[n][1] *= alpha[0];
        o[n][2] *= alpha[1], o[n][3] *= alpha[1];
      }
    }
#pragma unroll
    for (int kg = 0; kg < kTiles / 2; ++kg) {  // 16 keys
      const uint32_t a[4] = {pk[2 * kg][0], pk[2 * kg][1], pk[2 * kg + 1][0], pk[2 * kg + 1][1]};
#pragma unroll
      for (int n = 0; n < kUnits; n += 2) {
        if (n / 2 >= ksteps) break;
        uint32_t b[4];  // channels 8n .. +7: keys lo, hi; channels 8n + 8 ..: lo, hi
        ldm4_trans(b, vt + at(16 * kg + (mi & 1) * 8 + mr, n + (mi >> 1)));
        mma16816<F16>(o[n], a, b[0], b[1]);
        mma16816<F16>(o[n + 1], a, b[2], b[3]);
      }
    }
    __syncwarp();
    fetch(c + (L::kStages - 1) * stride, stage == 0 ? L::kStages - 1 : stage - 1);
    stage = stage + 1 == L::kStages ? 0 : stage + 1;
  }
  copies_wait<0>();
  __syncthreads();  // the ring is free: it takes the warps' outputs

  const uint32_t outs = sb + L::kRingOff, stats = sb + L::kStatOff;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * h + (lane >> 2);
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {  // the row's four lanes
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], d);
      lq[h] += __shfl_xor_sync(0xffffffffu, lq[h], d);
    }
    if (r < rows) {
      if ((lane & 3) == 0) st_shared_f4(stats + (warp * L::kRows + r) * 16, make_float4(m[h], l[h], lq[h], 0.f));
#pragma unroll
      for (int n = 0; n < kUnits; ++n)
        if (8 * n < p.D)
          st_shared_f2(outs + ((warp * L::kRows + r) * W + 8 * n + 2 * (lane & 3)) * 4, o[n][2 * h], o[n][2 * h + 1]);
    }
  }
  __syncthreads();
  // the CTA's part: its warps' joined.  Where it is alone, the result.
  const uint32_t cta_out = outs + kFewWarps * L::kOut, cta_stat = stats + kFewWarps * L::kRows * 16;
  const int quads = p.D / 4;
  auto finish = [&](int r, int c, float4 a, float mx, float sum, float sum_q) {
    // no sum: no keys, or (unless the join finds out) none with a score but -inf, 0 / 0
    const float inv = sum_q == 0.f && (len == 0 || p.runs > 1) ? 0.f : 1.f / sum_q;
    a.x *= inv, a.y *= inv, a.z *= inv, a.w *= inv;
    const int64_t row = (int64_t)bh * p.rows + r;
    const float lse = (mx + log2f(sum)) * kLn2F;
    if (p.runs > 1) {
      const int64_t part = (int64_t)run * p.BH * p.rows + row;
      *reinterpret_cast<float4*>(p.part_o + part * p.D + 4 * c) = a;
      if (c == 0) p.part_lse[part] = lse;
    } else {
      uint2 v;
      v.x = pack_x2<F16>(a.x, a.y), v.y = pack_x2<F16>(a.z, a.w);
      *reinterpret_cast<uint2*>(p.out + row * p.D + 4 * c) = v;
      if (c == 0) p.lse[row] = lse;
    }
  };
  for (int i = threadIdx.x; i < rows * quads; i += kFewThreads) {
    const int r = i / quads, c = i - r * quads;
    float4 st[kFewWarps];
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      st[w] = ld_shared_f4(stats + (w * L::kRows + r) * 16);
      mx = fmaxf(mx, st[w].x);
    }
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f, sum_q = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float f = weight_of(st[w].x, mx);
      const float4 v = ld_shared_f4(outs + ((w * L::kRows + r) * W + 4 * c) * 4);
      a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
      sum = fmaf(f, st[w].y, sum), sum_q = fmaf(f, st[w].z, sum_q);
    }
    if (p.cluster == 1) {
      finish(r, c, a, mx, sum, sum_q);
    } else {
      st_shared_f4(cta_out + (r * W + 4 * c) * 4, a);
      if (c == 0) st_shared_f4(cta_stat + r * 16, make_float4(mx, sum, sum_q, 0.f));
    }
  }
  if (p.cluster == 1) return;
  cluster_sync();
  // the cluster's: each CTA a share of the values
  for (int i = static_cast<int>(rank) * kFewThreads + threadIdx.x; i < rows * quads; i += p.cluster * kFewThreads) {
    const int r = i / quads, c = i - r * quads;
    float4 st[8], v[8];
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < 8; ++w)
      if (w < p.cluster) {
        st[w] = ld_cluster_v4(map_to(cta_stat + r * 16, w));
        v[w] = ld_cluster_v4(map_to(cta_out + (r * W + 4 * c) * 4, w));
      }
#pragma unroll
    for (int w = 0; w < 8; ++w)
      if (w < p.cluster) mx = fmaxf(mx, st[w].x);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f, sum_q = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w)
      if (w < p.cluster) {
        const float f = weight_of(st[w].x, mx);
        a.x = fmaf(f, v[w].x, a.x), a.y = fmaf(f, v[w].y, a.y), a.z = fmaf(f, v[w].z, a.z), a.w = fmaf(f, v[w].w, a.w);
        sum = fmaf(f, st[w].y, sum), sum_q = fmaf(f, st[w].z, sum_q);
      }
    finish(r, c, a, mx, sum, sum_q);
  }
  cluster_sync();  // nobody leaves while others read its part
}

template <bool F16>
cudaError_t launch_few(const FewParams& p, cudaStream_t stream) {
  using L = FewLayout;
  auto kern = cross_few_kernel<F16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((long long)p.BH * p.runs * p.cluster), 1, 1);
  cfg.blockDim = dim3(L::kThreads, 1, 1);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t cross_few_launch(const FewParams& p, bool f16, cudaStream_t stream) {
  return f16 ? launch_few<true>(p, stream) : launch_few<false>(p, stream);
}

}  // namespace ea
