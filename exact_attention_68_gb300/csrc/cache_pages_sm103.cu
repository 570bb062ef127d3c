// cache_pages_sm103.cu — what writes pages of the 8-bit cache: append (new keys
// and values) and evict (the tokens kept, gathered into other pages).
//
// One CTA writes one page of one head, of k or of v: it loads the tokens,
// takes the largest |x|, derives the page's power-of-two scale, writes the
// codes and, for k, the per-channel bounds.  A thread owns one 16-channel unit
// and every TPU-th token, so that a row's units lie side by side over a warp
// (whole 128-byte rows per access) and a channel's bound is a reduction over
// the threads of its unit.  Both operators move bytes and little else.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache_common.cuh"
#include "cache_topk.cuh"

namespace ea {
namespace {

// 128 threads: about half of the instructions are the same for a thread of 16
// values as for one of 64 (256 threads, 32 values each: 24 a value).
constexpr int kPageThreads = 128;
// Tokens of a thread: 64 slots over the threads of a unit (16 channels).
template <int UNITS>
constexpr int kItems = (64 + kPageThreads / UNITS - 1) / (kPageThreads / UNITS);

// Tokens of a 16-bit [rows, D] block.
template <bool F16>
struct RowSource {
  struct Raw {
    uint4 a, b;
  };
  const uint16_t* rows;  // the page's first new token
  int D;
  __device__ __forceinline__ Raw load(int t, int unit) const {
    const uint16_t* r = rows + static_cast<int64_t>(t) * D + unit * 16;
    Raw x;
    x.a = __ldg(reinterpret_cast<const uint4*>(r));
    x.b = unit * 16 + 8 < D ? __ldg(reinterpret_cast<const uint4*>(r + 8)) : make_uint4(0, 0, 0, 0);
    return x;
  }
  static __device__ __forceinline__ float2 pair(const Raw& x, int i) {
    const uint32_t w = i == 0 ? x.a.x : i == 1 ? x.a.y : i == 2 ? x.a.z : i == 3 ? x.a.w
                     : i == 4 ? x.b.x : i == 5 ? x.b.y : i == 6 ? x.b.z : x.b.w;
    return pair_to_float2<F16>(w);
  }
};

// Tokens picked out of the cache's pages.
struct CodeSource {
  struct Raw {
    uint4 w;
    float s;
  };
  const CacheView& c;
  const SeqView& s;
  const uint8_t* codes;
  const float* scales;
  const int* kept;  // positions of the page's tokens
  int b, h;
  __device__ __forceinline__ Raw load(int t, int unit) const {
    const int j = kept[t];
    const int g = j >= 0 && j < (s.width << c.log2_page)
                      ? load_page(s, c, b, j >> c.log2_page, true) : -1;
    Raw x;
    x.w = make_uint4(0, 0, 0, 0);
    x.s = 0.f;
    if (g >= 0) {
      const int64_t gh = static_cast<int64_t>(g) * c.heads + h;
      x.w = __ldg(reinterpret_cast<const uint4*>(
          codes + ((gh << c.log2_page) + (j & (c.page - 1))) * c.pitch + unit * 16));
      if (unit * 16 + 8 >= c.D) x.w.z = x.w.w = 0;  // padding channels
      x.s = __ldg(scales + gh);
    }
    return x;
  }
  static __device__ __forceinline__ float2 pair(const Raw& x, int i) {
    const uint32_t w = i < 2 ? x.w.x : i < 4 ? x.w.y : i < 6 ? x.w.z : x.w.w;
    const float2 v = half2_bits_to_float2(e4m3x2_to_f16x2((i & 1) ? w >> 16 : w & 0xffffu));
    return make_float2(v.x * x.s, v.y * x.s);
  }
};

// Writes `count` tokens from `src` to slots held .. held+count-1 of page g,
// head h; slots below `held` hold earlier tokens, which stay.
//
// Rounding keeps order, so a channel's largest code is the code of its largest
// value: the bounds cost two comparisons a value (fmaxf and fminf pass NaN
// over), and codes only meet at the end, four to a word.
template <int UNITS, class Src>
__device__ __forceinline__ void write_page(const CacheView& c, int g, int h, bool is_v, int held,
                                           int count, const Src& src) {
  __shared__ uint32_t red[kPageThreads / 32];
  __shared__ __align__(16) uint32_t top[kPageThreads * 4], bottom[kPageThreads * 4];
  // UNITS 0: any number up to 16
  constexpr int ITEMS = kItems<UNITS == 0 ? 16 : UNITS>;
  const int units = UNITS == 0 ? c.pitch >> 4 : UNITS, tpu = kPageThreads / units;
  const int unit = threadIdx.x % units, lane_t = threadIdx.x / units;
  const bool active = lane_t < tpu;
  const int64_t gh = static_cast<int64_t>(g) * c.heads + h;
  uint8_t* rows = (is_v ? c.v : c.k) + (gh << c.log2_page) * c.pitch + unit * 16;
  float* scale = (is_v ? c.v_scale : c.k_scale) + gh;
  const float was = held > 0 ? *scale : 0.f;

  typename Src::Raw raw[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    if (active && lane_t + i * tpu < count) raw[i] = src.load(lane_t + i * tpu, unit);
  float hi[16], lo[16], a = 0.f;  // k: the thread's channels' extremes; v: the largest |x|
  if (!is_v) {
#pragma unroll
    for (int e = 0; e < 16; ++e) hi[e] = -INFINITY, lo[e] = INFINITY;
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (active && lane_t + i * tpu < count) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 x = Src::pair(raw[i], e);
        if (is_v) {
          a = fmaxf(a, fmaxf(fabsf(x.x), fabsf(x.y)));
        } else {
          hi[2 * e] = fmaxf(hi[2 * e], x.x), lo[2 * e] = fminf(lo[2 * e], x.x);
          hi[2 * e + 1] = fmaxf(hi[2 * e + 1], x.y), lo[2 * e + 1] = fminf(lo[2 * e + 1], x.y);
        }
      }
    }
  }
  if (!is_v) {
#pragma unroll
    for (int e = 0; e < 16; ++e) a = fmaxf(a, fmaxf(hi[e], -lo[e]));
  }
  if (a == INFINITY) {  // infinities do not count: once more without them
    a = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (active && lane_t + i * tpu < count)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 x = Src::pair(raw[i], e);
          a = fmaxf(a, fmaxf(finite_abs(x.x), finite_abs(x.y)));
        }
  }
  // non-negative floats order as their bits
  const uint32_t wa = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = wa;
  __syncthreads();
  uint32_t ua = red[0];
#pragma unroll
  for (int w = 1; w < kPageThreads / 32; ++w) ua = max(ua, red[w]);
  const float fresh = page_scale(__uint_as_float(ua));
  const float s = held > 0 ? fmaxf(was, fresh) : fresh;
  const bool grown = held > 0 && s != was;
  uint32_t up[4], dn[4];  // ordered codes of the extremes; where there are none, up < dn
#pragma unroll
  for (int w = 0; w < 4; ++w) up[w] = 0x80808080u, dn[w] = 0x7f7f7f7fu;
  with_divider(s, [&](auto div) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int t = lane_t + i * tpu;
      if (active && t < count) {
        uint32_t q[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 x = Src::pair(raw[i], 2 * w), y = Src::pair(raw[i], 2 * w + 1);
          q[w] = pack_e4m3x2(div(x.x), div(x.y)) | (pack_e4m3x2(div(y.x), div(y.y)) << 16);
        }
        *reinterpret_cast<uint4*>(rows + static_cast<int64_t>(held + t) * c.pitch) =
            make_uint4(q[0], q[1], q[2], q[3]);
      }
    }
    if (!is_v && active) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t nan;
        up[w] = e4m3_order4(pack_e4m3x2(div(hi[4 * w]), div(hi[4 * w + 1])) |
                            (pack_e4m3x2(div(hi[4 * w + 2]), div(hi[4 * w + 3])) << 16), &nan);
        dn[w] = e4m3_order4(pack_e4m3x2(div(lo[4 * w]), div(lo[4 * w + 1])) |
                            (pack_e4m3x2(div(lo[4 * w + 2]), div(lo[4 * w + 3])) << 16), &nan);
      }
    }
  });
  if (grown) {
    // the earlier codes move to the larger scale
    const float ratio = __fdiv_rn(was, s);
    for (int t = lane_t; active && t < held; t += tpu) {
      uint4* at = reinterpret_cast<uint4*>(rows + static_cast<int64_t>(t) * c.pitch);
      const uint4 old = *at;
      uint32_t q[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t h0, h1;
        e4m3x4_to_f16(q[w], &h0, &h1);
        const float2 x = half2_bits_to_float2(h0), y = half2_bits_to_float2(h1);
        q[w] = pack_e4m3x2(x.x * ratio, x.y * ratio) | (pack_e4m3x2(y.x * ratio, y.y * ratio) << 16);
        uint32_t nan;
        const uint32_t o = e4m3_order4(q[w], &nan);
        up[w] = __vmaxs4(up[w], (o & ~nan) | (0x80808080u & nan));
        dn[w] = __vmins4(dn[w], (o & ~nan) | (0x7f7f7f7fu & nan));
      }
      *at = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
  if (!is_v && active) {
    reinterpret_cast<uint4*>(top)[lane_t * units + unit] = make_uint4(up[0], up[1], up[2], up[3]);
    reinterpret_cast<uint4*>(bottom)[lane_t * units + unit] = make_uint4(dn[0], dn[1], dn[2], dn[3]);
  }
  __syncthreads();  // bounds staged; every thread has read the old scale
  if (threadIdx.x == 0) *scale = s;
  const int words = units * 4;  // of a row of bounds
  if (!is_v && threadIdx.x < words) {
    const int w = threadIdx.x;
    uint32_t u = top[w], d = bottom[w];
    for (int t = 1; t < min(tpu, max(count, grown ? held : 0)); ++t) {
      u = __vmaxs4(u, top[t * words + w]);
      d = __vmins4(d, bottom[t * words + w]);
    }
    uint32_t* bu = reinterpret_cast<uint32_t*>(c.k_bounds + gh * 2 * c.pitch) + w;
    uint32_t* bl = bu + words;
    const bool keep = held > 0 && !grown;  // the earlier tokens' bounds still hold
    const uint32_t ou = keep ? *bu : 0u, ol = keep ? *bl : 0u;
    uint32_t ru = 0, rl = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = static_cast<int8_t>(u >> (8 * e)), y = static_cast<int8_t>(d >> (8 * e));
      const int xo = static_cast<int8_t>(ou >> (8 * e)), yo = static_cast<int8_t>(ol >> (8 * e));
      const bool none = x < y;
      int b1 = none ? 0 : bound_of_order(x, true), b0 = none ? 0 : bound_of_order(y, false);
      if (keep) b1 = none ? xo : max(b1, xo), b0 = none ? yo : min(b0, yo);
      ru |= (static_cast<uint32_t>(b1) & 0xffu) << (8 * e);
      rl |= (static_cast<uint32_t>(b0) & 0xffu) << (8 * e);
    }
    *bu = ru, *bl = rl;
  }
}

template <bool F16, int UNITS>
__global__ void __launch_bounds__(kPageThreads) cache_append_kernel(const CacheAppendParams p) {
  const bool is_v = blockIdx.x & 1;
  const int j = blockIdx.x >> 1, h = blockIdx.y, b = blockIdx.z;
  int len, n;
  if (!load_seq(p.s, p.c, b, threadIdx.x == 0, &len, &n) || n == 0) return;
  const int start = len - n, i = (start >> p.c.log2_page) + j, base = i << p.c.log2_page;
  if (base >= len) return;
  const int g = load_page(p.s, p.c, b, i, threadIdx.x == 0);
  if (g < 0) return;
  const int from = max(base, start), to = min(base + p.c.page, len);
  const int64_t row = (static_cast<int64_t>(b) * p.c.heads + h) * p.s.T + (from - start);
  const RowSource<F16> src{(is_v ? p.v : p.k) + row * p.c.D, p.c.D};
  write_page<UNITS>(p.c, g, h, is_v, from - base, to - from, src);
}

// ---------------------------------------------------------------- evict
constexpr int kPlanThreads = 1024;

// Block (h, b) with b < batch: which positions of head h stay, their weights.
// Block (0, batch): which destination pages may be written (a page that is out
// of range, in use by a source or named twice may not).
__global__ void __launch_bounds__(kPlanThreads) cache_evict_plan_kernel(const CacheEvictParams p) {
  const int h = blockIdx.x, b = blockIdx.y;
  if (b == p.s.batch) {
    if (h != 0) return;
    // used[0]: a source, or named once; used[1]: named again
    uint32_t* once = p.used;
    uint32_t* twice = p.used + p.used_words;
    for (int w = threadIdx.x; w < 2 * p.used_words; w += kPlanThreads) p.used[w] = 0;
    __syncthreads();
    for (int bb = 0; bb < p.s.batch; ++bb) {
      int len, n;
      load_seq(p.s, p.c, bb, threadIdx.x == 0, &len, &n);
      const int np = (len + p.c.page - 1) >> p.c.log2_page;
      for (int i = threadIdx.x; i < np; i += kPlanThreads) {
        const int g = load_page(p.s, p.c, bb, i, true);
        if (g >= 0) atomicOr(&once[g >> 5], 1u << (g & 31));
      }
    }
    __syncthreads();
    for (int round = 0; round < 2; ++round) {
      for (int bb = 0; bb < p.s.batch; ++bb) {
        int len, n;
        load_seq(p.s, p.c, bb, false, &len, &n);
        const int nd = (min(len, p.keep) + p.c.page - 1) >> p.c.log2_page;
        for (int i = threadIdx.x; i < p.dst_width; i += kPlanThreads) {
          const int64_t at = static_cast<int64_t>(bb) * p.dst_width + i;
          const int g = i < nd ? p.dst_table[at] : -1;
          const bool in = g >= 0 && g < p.c.pages;
          const uint32_t bit = 1u << (g & 31);
          if (round == 0) {
            if (in && (atomicOr(&once[g >> 5], bit) & bit)) atomicOr(&twice[g >> 5], bit);
          } else {
            const bool ok = in && !(twice[g >> 5] & bit);
            if (i < nd && !ok) dbg_fail(p.s.status, kChkCacheDst);
            p.dst_page[at] = ok ? g : -1;
          }
        }
      }
      __syncthreads();
    }
    return;
  }
  int len, n;
  load_seq(p.s, p.c, b, threadIdx.x == 0 && h == 0, &len, &n);
  const int left = min(len, p.keep);
  const int64_t bh = static_cast<int64_t>(b) * p.c.heads + h;
  const float* mass = p.mass + bh * (static_cast<int64_t>(p.s.width) << p.c.log2_page);
  int* kept = p.kept + bh * p.keep;
  float* out = p.mass_out + bh * (static_cast<int64_t>(p.dst_width) << p.c.log2_page);
  if (h == 0 && threadIdx.x == 0) p.new_lens[b] = left;
  if (len <= p.keep) {
    for (int j = threadIdx.x; j < len; j += kPlanThreads) {
      kept[j] = j;
      out[j] = mass[j];
    }
  } else {
    const int tail = min(p.recent, len), best = p.keep - tail;
    block_top_ascending<kPlanThreads, 16>([&](int j) { return order_key(mass[j]); }, len - tail, best,
                                      [&](int at, int j) {
                                        kept[at] = j;
                                        out[at] = mass[j];
                                      });
    for (int j = threadIdx.x; j < tail; j += kPlanThreads) {
      kept[best + j] = len - tail + j;
      out[best + j] = mass[len - tail + j];
    }
  }
  for (int j = left + threadIdx.x; j < p.keep; j += kPlanThreads) kept[j] = -1;
  for (int j = left + threadIdx.x; j < (p.dst_width << p.c.log2_page); j += kPlanThreads)
    out[j] = 0.f;
}

template <int UNITS>
__global__ void __launch_bounds__(kPageThreads) cache_evict_move_kernel(const CacheEvictParams p) {
  const bool is_v = blockIdx.x & 1;
  const int i = blockIdx.x >> 1, h = blockIdx.y, b = blockIdx.z;
  const int left = p.new_lens[b], base = i << p.c.log2_page;
  if (base >= left) return;
  const int g = p.dst_page[static_cast<int64_t>(b) * p.dst_width + i];
  if (g < 0) return;
  const CodeSource src{p.c, p.s, is_v ? p.c.v : p.c.k, is_v ? p.c.v_scale : p.c.k_scale,
                       p.kept + (static_cast<int64_t>(b) * p.c.heads + h) * p.keep + base, b, h};
  write_page<UNITS>(p.c, g, h, is_v, 0, min(p.c.page, left - base), src);
}

// The kernels know the units of 64, 128 and 256 channels at compile time.
template <class Launch>
void by_units(const CacheView& c, Launch launch) {
  switch (c.pitch >> 4) {
    case 4: return launch(std::integral_constant<int, 4>());
    case 8: return launch(std::integral_constant<int, 8>());
    case 16: return launch(std::integral_constant<int, 16>());
  }
  launch(std::integral_constant<int, 0>());
}

}  // namespace

cudaError_t cache_append_launch(const CacheAppendParams& p, bool f16, cudaStream_t stream) {
  const dim3 grid(2u * p.pages_per_seq, p.c.heads, p.s.batch);
  by_units(p.c, [&](auto u) {
    constexpr int UNITS = decltype(u)::value;
    if (f16) cache_append_kernel<true, UNITS><<<grid, kPageThreads, 0, stream>>>(p);
    else cache_append_kernel<false, UNITS><<<grid, kPageThreads, 0, stream>>>(p);
  });
  return cudaGetLastError();
}

cudaError_t cache_evict_launch(const CacheEvictParams& p, cudaStream_t stream) {
  cache_evict_plan_kernel<<<dim3(p.c.heads, p.s.batch + 1), kPlanThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid(2u * ((p.keep + p.c.page - 1) >> p.c.log2_page), p.c.heads, p.s.batch);
  by_units(p.c, [&](auto u) {
    cache_evict_move_kernel<decltype(u)::value><<<grid, kPageThreads, 0, stream>>>(p);
  });
  return cudaGetLastError();
}

}  // namespace ea
