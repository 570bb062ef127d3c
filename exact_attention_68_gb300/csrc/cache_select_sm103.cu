// cache_select_sm103.cu — which pages of the 8-bit cache each head should read:
// an 8-bit bound on every page's scores, then the best of them.
//
// For a query row rounded to 8 bits (qi) and a page's key bounds hi >= lo,
//   Σ_d max(qi·hi, qi·lo) = Σ_d max(qi, 0)·hi + min(qi, 0)·lo
// is a product of signed bytes over twice the channels, taken with dp4a and
// exact in 32 bits (at most 256·127·127 < 2^23, also exact in fp32).  Four lanes
// share a page, 16 channels a load; query rows stay in registers while pages go
// by, each lane copying its own bounds ahead into shared memory.
//
// Bound: 2·D bytes a page and head (the page's keys and values are 2·D·page),
// read as 256-byte rows at random: 8 sequences of 50001-65536 tokens in pages of
// 16, 8 heads of 128 channels: 26.9 us for 61.6 MB, of which 9 us choosing 256 of
// 4096 pages, 64 CTAs each on its own row of scores; slope 3.1 TB/s with 20 % of the
// warps active, so that too few bytes are in flight.  One sequence of 256 pages 7.2
// us (latency of two kernels).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache_common.cuh"
#include "cache_topk.cuh"

namespace ea {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kScoreGroups = kScoreThreads / 4;  // pages at a time

// Asynchronous copies to shared memory; `bytes` of 16 are read, the rest zero.
__device__ __forceinline__ void copy_async_16(uint32_t to, const void* from, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_async_4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// UNITS: 16-channel units of a lane (1, 2 or 4: up to 64, 128, 256 channels);
// ROWS: query rows held in registers while a CTA's pages go by (more rows: once
// more over the pages, whose bounds then come from L2).
template <int UNITS, int ROWS, bool F16>
__global__ void __launch_bounds__(kScoreThreads) cache_score_kernel(const CacheSelectParams p,
                                                                    int pages_per_group) {
  __shared__ __align__(16) int8_t qpos[ROWS * 256], qneg[ROWS * 256];
  __shared__ float qa[ROWS];
  constexpr int kStages = UNITS == 4 ? 2 : 4;  // 34 KB
  __shared__ int4 ring[kStages][2 * UNITS][kScoreThreads];
  __shared__ float scale[kStages][kScoreThreads];
  const int h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & 3, group = threadIdx.x >> 2;
  const int units = p.c.pitch >> 4;
  int len, n;
  load_seq(p.s, p.c, b, threadIdx.x == 0 && blockIdx.x == 0 && h == 0, &len, &n);
  const int np = n > 0 ? (len + p.c.page - 1) >> p.c.log2_page : 0;
  const int first = blockIdx.x * kScoreGroups * pages_per_group;
  const int rows = p.G * p.s.T;
  const uint16_t* q = p.q + (static_cast<int64_t>(b) * p.c.heads + h) * rows * p.c.D;
  float* scores = p.scores + (static_cast<int64_t>(b) * p.c.heads + h) * p.s.width;
  const int stop = min(np, first + kScoreGroups * pages_per_group);
  for (int r0 = 0; first < np && r0 < rows; r0 += ROWS) {
    const int nr = min(ROWS, rows - r0);
    __syncthreads();
    for (int r = warp; r < ROWS; r += kScoreThreads / 32) {
      // one row a warp, 8 channels a lane
      const bool in = 8 * lane < p.c.D && r < nr;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (in) w = __ldg(reinterpret_cast<const uint4*>(q + static_cast<int64_t>(r0 + r) * p.c.D + 8 * lane));
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = pair_to_float2<F16>(ws[e]);
        a = fmaxf(a, fmaxf(finite_abs(x.x), finite_abs(x.y)));
      }
      a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
      const float steps = a > 0.f ? __fdiv_rn(127.f, a) : 0.f;
      uint32_t up[2] = {0u, 0u}, dn[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 x2 = pair_to_float2<F16>(ws[e >> 1]);
        float y = rintf(__fmul_rn((e & 1) ? x2.y : x2.x, steps));
        if (y != y) y = 0.f;
        const int i = static_cast<int>(fminf(fmaxf(y, -127.f), 127.f));
        up[e >> 2] |= (static_cast<uint32_t>(max(i, 0)) & 0xffu) << (8 * (e & 3));
        dn[e >> 2] |= (static_cast<uint32_t>(min(i, 0)) & 0xffu) << (8 * (e & 3));
      }
      // padding channels, to the end of the lanes' units, hold zero
      *reinterpret_cast<uint2*>(&qpos[r * 256 + 8 * lane]) = make_uint2(up[0], up[1]);
      *reinterpret_cast<uint2*>(&qneg[r * 256 + 8 * lane]) = make_uint2(dn[0], dn[1]);
      if (lane == 0) qa[r] = r < nr && (r0 + r) % p.s.T < n ? a : -1.f;  // -1: no such token
    }
    __syncthreads();
    int4 x[ROWS][UNITS], y[ROWS][UNITS];
    float a[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      a[r] = qa[r];
#pragma unroll
      for (int j = 0; j < UNITS; ++j) {
        x[r][j] = *reinterpret_cast<const int4*>(&qpos[r * 256 + (sub + 4 * j) * 16]);
        y[r][j] = *reinterpret_cast<const int4*>(&qneg[r * 256 + (sub + 4 * j) * 16]);
      }
    }
    // The pages of a group in turn: each lane copies the units it will need
    // into places of its own, kStages - 1 steps ahead; page numbers come one
    // step before that.  All lanes take all steps (the shuffles want them).
    auto page_of = [&](int k) {
      const int i = first + group + k * kScoreGroups;
      return k < pages_per_group && i < stop ? load_page(p.s, p.c, b, i, r0 == 0 && sub == 0) : -1;
    };
    int next = page_of(0);
    auto fetch = [&](int k) {
      const int g = next, at = k % kStages;
      next = page_of(k + 1);
      const int64_t gh = static_cast<int64_t>(g < 0 ? 0 : g) * p.c.heads + h;
      const int8_t* bd = p.c.k_bounds + gh * 2 * p.c.pitch;
#pragma unroll
      for (int j = 0; j < UNITS; ++j) {
        const int u = sub + 4 * j;
        const uint32_t bytes = g >= 0 && u < units ? 16u : 0u;  // 0: zeros
        const int8_t* from = bd + (bytes ? u * 16 : 0);
        copy_async_16(smem_u32(&ring[at][2 * j][threadIdx.x]), from, bytes);
        copy_async_16(smem_u32(&ring[at][2 * j + 1][threadIdx.x]), from + (bytes ? p.c.pitch : 0), bytes);
      }
      // a page that is not there scores as NaN, which no comparison takes
      if (g >= 0) copy_async_4(smem_u32(&scale[at][threadIdx.x]), p.c.k_scale + gh);
      else scale[at][threadIdx.x] = __int_as_float(0x7fffffff);
      copy_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k);
#pragma unroll 1
    for (int k = 0; k < pages_per_group; ++k) {
      const int i = first + group + k * kScoreGroups, at = k % kStages;
      fetch(k + kStages - 1);
      copy_async_wait<kStages - 1>();
      int4 hi[UNITS], lo[UNITS];
#pragma unroll
      for (int j = 0; j < UNITS; ++j) hi[j] = ring[at][2 * j][threadIdx.x], lo[j] = ring[at][2 * j + 1][threadIdx.x];
      const float ks = scale[at][threadIdx.x];
      float best = -INFINITY;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        int sum = 0;
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
          sum = __dp4a(hi[j].x, x[r][j].x, sum);
          sum = __dp4a(hi[j].y, x[r][j].y, sum);
          sum = __dp4a(hi[j].z, x[r][j].z, sum);
          sum = __dp4a(hi[j].w, x[r][j].w, sum);
          sum = __dp4a(lo[j].x, y[r][j].x, sum);
          sum = __dp4a(lo[j].y, y[r][j].y, sum);
          sum = __dp4a(lo[j].z, y[r][j].z, sum);
          sum = __dp4a(lo[j].w, y[r][j].w, sum);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (a[r] >= 0.f) best = fmaxf(best, __fmul_rn(__fmul_rn(static_cast<float>(sum), ks), a[r]));
      }
      if (sub == 0 && i < stop) scores[i] = r0 == 0 ? best : fmaxf(scores[i], best);
    }
    copy_async_wait<0>();  // the last steps' empty copies, before their places are used again
  }
  launch_dependents();
  // pages behind the sequence's end
  for (int i = max(first, np) + threadIdx.x; i < min(p.s.width, first + kScoreGroups * pages_per_group); i += kScoreThreads)
    scores[i] = -INFINITY;
}

constexpr int kPickThreads = 1024;

__global__ void __launch_bounds__(kPickThreads) cache_pick_kernel(const CacheSelectParams p) {
  const int h = blockIdx.x, b = blockIdx.y;
  const int64_t bh = static_cast<int64_t>(b) * p.c.heads + h;
  const float* scores = p.scores + bh * p.s.width;
  int* pages = p.pages + bh * p.count;
  int len, n;
  load_seq(p.s, p.c, b, false, &len, &n);
  wait_for_previous();
  int taken = 0;
  if (n > 0) {
    const int np = (len + p.c.page - 1) >> p.c.log2_page;
    const int first = (len - n) >> p.c.log2_page;  // from here on the new tokens' pages
    const int fresh = min(np - first, p.count);
    const int best = min(p.count - fresh, first);
    block_top_ascending<kPickThreads>(scores, first, best, [&](int at, int i) { pages[at] = i; });
    for (int i = threadIdx.x; i < fresh; i += kPickThreads) pages[best + i] = np - fresh + i;
    taken = best + fresh;
  }
  for (int i = taken + threadIdx.x; i < p.count; i += kPickThreads) pages[i] = -1;
}

template <int UNITS, int ROWS>
cudaError_t score(const CacheSelectParams& p, bool f16, cudaStream_t stream) {
  // the fewest pages a group with which four CTAs on each SM cover all: one wave with
  // the registers of 4 rows of 128 channels (a second wave of a few CTAs took as long as
  // the first).  Measured there; of the other variants, 64 to 189 registers, two to
  // eight CTAs fit.  The steps go by the width of the table: pages behind a sequence's end
  // cost theirs (8 sequences of 50001-65536 tokens in pages of 16: 26.9 us, under a
  // table twice as wide 39.4 us)
  const int64_t wave = 4ll * p.sms;
  auto ctas = [&](int64_t k) { return static_cast<int>((p.s.width + kScoreGroups * k - 1) / (kScoreGroups * k)); };
  const int64_t heads = static_cast<int64_t>(p.s.batch) * p.c.heads;
  int per = static_cast<int>((heads * ctas(1) + wave - 1) / wave);
  while (heads * ctas(per) > wave && ctas(per) > 1) ++per;
  const dim3 grid(ctas(per), p.c.heads, p.s.batch);
  if (f16) cache_score_kernel<UNITS, ROWS, true><<<grid, kScoreThreads, 0, stream>>>(p, per);
  else cache_score_kernel<UNITS, ROWS, false><<<grid, kScoreThreads, 0, stream>>>(p, per);
  return cudaGetLastError();
}
template <int UNITS>
cudaError_t score_rows(const CacheSelectParams& p, bool f16, cudaStream_t stream) {
  const int rows = p.G * p.s.T;
  if (rows == 1) return score<UNITS, 1>(p, f16, stream);
  if (rows <= 4 || UNITS == 4) return score<UNITS, 4>(p, f16, stream);
  return score<UNITS, UNITS == 4 ? 4 : 8>(p, f16, stream);
}

}  // namespace

cudaError_t cache_select_launch(const CacheSelectParams& p, bool f16, cudaStream_t stream) {
  const int units = p.c.pitch >> 4;
  cudaError_t e = units <= 4   ? score_rows<1>(p, f16, stream)
                  : units <= 8 ? score_rows<2>(p, f16, stream)
                               : score_rows<4>(p, f16, stream);
  if (e != cudaSuccess) return e;
  return launch_after(cache_pick_kernel, dim3(p.c.heads, p.s.batch), kPickThreads, stream, p);
}

}  // namespace ea
