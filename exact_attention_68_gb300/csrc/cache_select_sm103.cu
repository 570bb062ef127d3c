// cache_select_sm103.cu — which pages of the 8-bit cache each head should read:
// an 8-bit bound on every page's scores, then the best of them.
//
// For a query row rounded to 8 bits (qi) and a page's key bounds hi >= lo,
//   Σ_d max(qi·hi, qi·lo) = Σ_d max(qi, 0)·hi + min(qi, 0)·lo
// is a product of signed bytes over twice the channels, taken with dp4a and
// exact in 32 bits (at most 256·127·127 < 2^23, also exact in fp32).  Four lanes
// share a page, 16 channels a load.  The bounds are read once, 2·D bytes a
// page against the page's 2·D·page of keys and values.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache_common.cuh"
#include "cache_topk.cuh"

namespace ea {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kScoreGroups = kScoreThreads / 4;  // pages at a time
constexpr int kScoreRows = 32;                   // query rows in shared memory at a time
constexpr int kMaxPagesPerGroup = 4;

template <bool F16>
__global__ void __launch_bounds__(kScoreThreads) cache_score_kernel(const CacheSelectParams p,
                                                                    int pages_per_group) {
  __shared__ __align__(16) int8_t qpos[kScoreRows * 256], qneg[kScoreRows * 256];
  __shared__ float qa[kScoreRows];
  const int h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & 3, group = threadIdx.x >> 2;
  const int units = p.c.pitch >> 4;
  int len, n;
  load_seq(p.s, p.c, b, threadIdx.x == 0 && blockIdx.x == 0 && h == 0, &len, &n);
  const int np = n > 0 ? (len + p.c.page - 1) >> p.c.log2_page : 0;
  const int first = blockIdx.x * kScoreGroups * pages_per_group;
  float best[kMaxPagesPerGroup];
#pragma unroll
  for (int k = 0; k < kMaxPagesPerGroup; ++k) best[k] = -INFINITY;
  const int rows = p.G * p.s.T;
  const uint16_t* q = p.q + (static_cast<int64_t>(b) * p.c.heads + h) * rows * p.c.D;
  if (first < np) {
    for (int r0 = 0; r0 < rows; r0 += kScoreRows) {
      const int nr = min(kScoreRows, rows - r0);
      __syncthreads();
      for (int r = warp; r < nr; r += kScoreThreads / 32) {
        // one row a warp, 8 channels a lane
        const bool in = 8 * lane < p.c.D;
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
        if (8 * lane < p.c.pitch) {  // padding channels hold zero
          *reinterpret_cast<uint2*>(&qpos[r * 256 + 8 * lane]) = make_uint2(up[0], up[1]);
          *reinterpret_cast<uint2*>(&qneg[r * 256 + 8 * lane]) = make_uint2(dn[0], dn[1]);
        }
        if (lane == 0) qa[r] = (r0 + r) % p.s.T < n ? a : -1.f;  // -1: no such token
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kMaxPagesPerGroup; ++k) {
        const int i = first + k * kScoreGroups + group;
        const bool mine = k < pages_per_group && i < np;
        const int g = mine ? load_page(p.s, p.c, b, i, r0 == 0 && sub == 0) : -1;
        const int64_t gh = static_cast<int64_t>(g < 0 ? 0 : g) * p.c.heads + h;
        const int8_t* bd = p.c.k_bounds + gh * 2 * p.c.pitch;
        uint4 hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int u = sub + 4 * j;
          hi[j] = lo[j] = make_uint4(0, 0, 0, 0);
          if (g >= 0 && u < units) {
            hi[j] = __ldg(reinterpret_cast<const uint4*>(bd + u * 16));
            lo[j] = __ldg(reinterpret_cast<const uint4*>(bd + p.c.pitch + u * 16));
          }
        }
        const float ks = g >= 0 ? __ldg(p.c.k_scale + gh) : 0.f;
        for (int r = 0; r < nr; ++r) {
          const float a = qa[r];
          if (a < 0.f) continue;
          int sum = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int u = sub + 4 * j;
            if (u < units) {
              const int4 x = *reinterpret_cast<const int4*>(&qpos[r * 256 + u * 16]);
              const int4 y = *reinterpret_cast<const int4*>(&qneg[r * 256 + u * 16]);
              sum = __dp4a(static_cast<int>(hi[j].x), x.x, sum);
              sum = __dp4a(static_cast<int>(hi[j].y), x.y, sum);
              sum = __dp4a(static_cast<int>(hi[j].z), x.z, sum);
              sum = __dp4a(static_cast<int>(hi[j].w), x.w, sum);
              sum = __dp4a(static_cast<int>(lo[j].x), y.x, sum);
              sum = __dp4a(static_cast<int>(lo[j].y), y.y, sum);
              sum = __dp4a(static_cast<int>(lo[j].z), y.z, sum);
              sum = __dp4a(static_cast<int>(lo[j].w), y.w, sum);
            }
          }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if (g >= 0)
            best[k] = fmaxf(best[k], __fmul_rn(__fmul_rn(static_cast<float>(sum), ks), a));
        }
      }
    }
  }
  float* scores = p.scores + (static_cast<int64_t>(b) * p.c.heads + h) * p.s.width;
#pragma unroll
  for (int k = 0; k < kMaxPagesPerGroup; ++k) {
    const int i = first + k * kScoreGroups + group;
    if (k < pages_per_group && i < p.s.width && sub == 0) scores[i] = best[k];
  }
}

constexpr int kPickThreads = 512;

__global__ void __launch_bounds__(kPickThreads) cache_pick_kernel(const CacheSelectParams p) {
  const int h = blockIdx.x, b = blockIdx.y;
  const int64_t bh = static_cast<int64_t>(b) * p.c.heads + h;
  const float* scores = p.scores + bh * p.s.width;
  int* pages = p.pages + bh * p.count;
  int len, n;
  load_seq(p.s, p.c, b, false, &len, &n);
  int taken = 0;
  if (n > 0) {
    const int np = (len + p.c.page - 1) >> p.c.log2_page;
    const int first = (len - n) >> p.c.log2_page;  // from here on the new tokens' pages
    const int fresh = min(np - first, p.count);
    const int best = min(p.count - fresh, first);
    block_top_ascending<kPickThreads>([&](int i) { return order_key(scores[i]); }, first, best,
                                      [&](int at, int i) { pages[at] = i; });
    for (int i = threadIdx.x; i < fresh; i += kPickThreads) pages[best + i] = np - fresh + i;
    taken = best + fresh;
  }
  for (int i = taken + threadIdx.x; i < p.count; i += kPickThreads) pages[i] = -1;
}

}  // namespace

cudaError_t cache_select_launch(const CacheSelectParams& p, bool f16, cudaStream_t stream) {
  // as many pages a CTA as leave two CTAs for each of about 152 SMs
  int per = kMaxPagesPerGroup;
  while (per > 1 && static_cast<int64_t>(p.s.batch) * p.c.heads *
                            ((p.s.width + kScoreGroups * per - 1) / (kScoreGroups * per)) < 304)
    per >>= 1;
  const dim3 grid((p.s.width + kScoreGroups * per - 1) / (kScoreGroups * per), p.c.heads, p.s.batch);
  if (f16) cache_score_kernel<true><<<grid, kScoreThreads, 0, stream>>>(p, per);
  else cache_score_kernel<false><<<grid, kScoreThreads, 0, stream>>>(p, per);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache_pick_kernel<<<dim3(p.c.heads, p.s.batch), kPickThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ea
