// cache_pages_sm103.cu — what writes pages of the 8-bit cache: append (new keys
// and values) and evict (the tokens kept, gathered into other pages).
//
// One CTA writes one page of one head, of k or of v: it loads the tokens,
// takes the largest |x|, derives the page's power-of-two scale, writes the
// codes and, for k, the per-channel bounds.  A thread owns one 16-channel unit
// and every TPU-th token, so that a row's units lie side by side over a warp
// (whole 128-byte rows per access) and a channel's bound is a reduction over
// the threads of its unit.
//
// Bytes are what both cannot do without, 6·D a token and head to append and
// 4·D to move.  Measured at 8 heads of 128 channels: 2 x 8192 tokens appended in
// 21.2 us = 4.7 TB/s, about 12 instructions a value issued at 61 % of the rate;
// one token of each of 64 sequences 5.0 us (latency); 8 sequences cut to 4096
// tokens a head moved in 38 us, 134 MB as random 128-byte rows (a page's chain of
// loads, position, page, codes; 55 % of the issue rate), behind 13 us for choosing them.
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

// A thread's part of a page: one unit of 16 channels and every tpu-th token.
// UNITS 0: any number up to 16.
template <int UNITS>
struct Share {
  static constexpr int kMine = kItems<UNITS == 0 ? 16 : UNITS>;
  int units, tpu, unit, first;
  bool active;
  __device__ __forceinline__ explicit Share(int pitch) {
    units = UNITS == 0 ? pitch >> 4 : UNITS;
    tpu = kPageThreads / units;
    unit = threadIdx.x % units;
    first = threadIdx.x / units;
    active = first < tpu;
  }
};

// Largest of a non-negative value over the CTA.
__device__ __forceinline__ float block_max(float a) {
  __shared__ uint32_t red[kPageThreads / 32];
  // non-negative floats order as their bits
  const uint32_t wa = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = wa;
  __syncthreads();
  uint32_t m = red[0];
#pragma unroll
  for (int w = 1; w < kPageThreads / 32; ++w) m = max(m, red[w]);
  return __uint_as_float(m);
}

// Running extremes of the bytes of words: of the odd bytes in the high halves of
// 16-bit lanes, where the byte below decides only between equal ones, and of the
// even bytes moved there.
struct ByteMax {
  uint32_t even = 0u, odd = 0u;
  __device__ __forceinline__ void add(uint32_t w) { even = max_u16x2(even, w << 8), odd = max_u16x2(odd, w); }
  __device__ __forceinline__ uint32_t get() const { return __byte_perm(even, odd, 0x7351); }
  __device__ __forceinline__ uint32_t largest() const {
    const uint32_t m = max_u16x2(even, odd);
    return max(m >> 24, (m >> 8) & 0xffu);
  }
};
struct ByteMin {
  uint32_t even = ~0u, odd = ~0u;
  __device__ __forceinline__ void add(uint32_t w) { even = min_u16x2(even, w << 8), odd = min_u16x2(odd, w); }
  __device__ __forceinline__ uint32_t get() const { return __byte_perm(even, odd, 0x7351); }
};

// Writes a page's bounds from every thread's extremes (ordered codes of its 16
// channels; up < dn: none).  Token rows from `lanes` on hold none.  keep: the
// bounds there hold for the page's earlier tokens and are widened.
//
// Rows are parted among neighbouring lanes, four to each, and joined by shuffles;
// the rows' pitch of 5 words a unit leaves their reads without bank conflicts.
// (With one warp that read all rows an eviction's batch took 55.7 us, so 53.8.)
template <int UNITS>
__device__ __forceinline__ void write_bounds(const CacheView& c, const Share<UNITS>& sh, int64_t gh, int lanes,
                                             bool keep, const uint32_t (&up)[4], const uint32_t (&dn)[4]) {
  constexpr int kParts = UNITS == 0 ? 1 : kPageThreads / (UNITS == 0 ? 1 : UNITS * 4), kPitch = UNITS == 0 ? 4 : 5;
  __shared__ __align__(16) uint32_t top[kPageThreads * kPitch], bottom[kPageThreads * kPitch];
  const int row = sh.units * kPitch;
  if (sh.active) {
    reinterpret_cast<uint4*>(top + sh.first * row)[sh.unit] = make_uint4(up[0], up[1], up[2], up[3]);
    reinterpret_cast<uint4*>(bottom + sh.first * row)[sh.unit] = make_uint4(dn[0], dn[1], dn[2], dn[3]);
  }
  __syncthreads();
  const int words = sh.units * 4, w = threadIdx.x / kParts, part = threadIdx.x % kParts;  // words of a row of bounds
  if (w >= words) return;
  ByteMax most;
  ByteMin least;
  if constexpr (UNITS == 0) {
    for (int t = 0; t < min(sh.tpu, lanes); ++t) most.add(top[t * row + w]), least.add(bottom[t * row + w]);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int at = (t * kParts + part) * row + w;
      most.add(top[at]), least.add(bottom[at]);
    }
#pragma unroll
    for (int d = 1; d < kParts; d <<= 1) {
      most.add(__shfl_xor_sync(0xffffffffu, most.get(), d));
      least.add(__shfl_xor_sync(0xffffffffu, least.get(), d));
    }
    if (part != 0) return;
  }
  const uint32_t u = most.get(), d = least.get();
  uint32_t* bu = reinterpret_cast<uint32_t*>(c.k_bounds + gh * 2 * c.pitch) + w;
  uint32_t* bl = bu + words;
  const uint32_t ou = keep ? *bu : 0u, ol = keep ? *bl : 0u;
  uint32_t ru = 0, rl = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t x = (u >> (8 * e)) & 0xffu, y = (d >> (8 * e)) & 0xffu;
    const int xo = static_cast<int8_t>(ou >> (8 * e)), yo = static_cast<int8_t>(ol >> (8 * e));
    const bool none = x < y;
    int b1 = none ? 0 : bound_of_order(x, true), b0 = none ? 0 : bound_of_order(y, false);
    if (keep) b1 = none ? xo : max(b1, xo), b0 = none ? yo : min(b0, yo);
    ru |= (static_cast<uint32_t>(b1) & 0xffu) << (8 * e);
    rl |= (static_cast<uint32_t>(b0) & 0xffu) << (8 * e);
  }
  *bu = ru, *bl = rl;
}

// Appends `count` tokens, rows of D 16-bit values, to page g (-1: none, nothing
// is done) of head h, at slots held, held + 1, ...; the slots below hold earlier
// tokens, which stay.
//
// Rounding keeps order, so a channel's largest code is the code of its largest
// value: the bounds cost a packed maximum and minimum for two values, and codes
// only meet at the end, four to a word.
template <bool F16, int UNITS>
__device__ __forceinline__ void append_page(const CacheView& c, int g, int h, bool is_v, int held, int count,
                                            const uint16_t* src) {
  const Share<UNITS> sh(c.pitch);
  const int64_t gh = static_cast<int64_t>(g) * c.heads + h;
  uint8_t* rows = (is_v ? c.v : c.k) + (gh << c.log2_page) * c.pitch + sh.unit * 16;
  uint32_t x[Share<UNITS>::kMine][8];
#pragma unroll
  for (int i = 0; i < Share<UNITS>::kMine; ++i) {
    const int t = sh.first + i * sh.tpu;
    if (sh.active && t < count) {
      const uint16_t* r = src + static_cast<int64_t>(t) * c.D + sh.unit * 16;
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(r));
      const uint4 b = sh.unit * 16 + 8 < c.D ? __ldg(reinterpret_cast<const uint4*>(r + 8)) : make_uint4(0, 0, 0, 0);
      x[i][0] = a.x, x[i][1] = a.y, x[i][2] = a.z, x[i][3] = a.w;
      x[i][4] = b.x, x[i][5] = b.y, x[i][6] = b.z, x[i][7] = b.w;
    }
  }
  // behind the tokens' loads, which do not wait for the page's number
  if (g < 0) return;
  float* scale = (is_v ? c.v_scale : c.k_scale) + gh;
  const float was = held > 0 ? *scale : 0.f;
  constexpr uint32_t kInf = F16 ? 0x7c007c00u : 0x7f807f80u, kAbs = 0x7fff7fffu;
  uint32_t hi[8], lo[8], a2 = 0;  // k: the channels' extremes; a2: the largest |x|
#pragma unroll
  for (int e = 0; e < 8; ++e) hi[e] = kInf | ~kAbs, lo[e] = kInf;
#pragma unroll
  for (int i = 0; i < Share<UNITS>::kMine; ++i)
    if (sh.active && sh.first + i * sh.tpu < count)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (is_v) a2 = max_x2<F16>(a2, x[i][e] & kAbs);
        else hi[e] = max_x2<F16>(hi[e], x[i][e]), lo[e] = min_x2<F16>(lo[e], x[i][e]);
      }
  if (!is_v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a2 = max_x2<F16>(a2, max_x2<F16>(hi[e], lo[e] ^ ~kAbs));
  }
  const float2 af = pair_to_float2<F16>(a2);
  float a = fmaxf(af.x, af.y);
  if (a == INFINITY) {  // infinities do not count: once more without them
    a = 0.f;
#pragma unroll
    for (int i = 0; i < Share<UNITS>::kMine; ++i)
      if (sh.active && sh.first + i * sh.tpu < count)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v = pair_to_float2<F16>(x[i][e]);
          a = fmaxf(a, fmaxf(finite_abs(v.x), finite_abs(v.y)));
        }
  }
  const float fresh = page_scale(block_max(a));
  const float s = held > 0 ? fmaxf(was, fresh) : fresh;
  const bool grown = held > 0 && s != was;
  if (threadIdx.x == 0) *scale = s;  // the old one has been read: block_max is a barrier

  uint32_t up[4], dn[4];
  with_divider(s, [&](auto div) {
    auto codes = [&](uint32_t w0, uint32_t w1) {
      const float2 v0 = div(pair_to_float2<F16>(w0)), v1 = div(pair_to_float2<F16>(w1));
      return pack_e4m3x2(v0.x, v0.y) | (pack_e4m3x2(v1.x, v1.y) << 16);
    };
#pragma unroll
    for (int i = 0; i < Share<UNITS>::kMine; ++i) {
      const int t = sh.first + i * sh.tpu;
      if (sh.active && t < count)
        *reinterpret_cast<uint4*>(rows + static_cast<int64_t>(held + t) * c.pitch) =
            make_uint4(codes(x[i][0], x[i][1]), codes(x[i][2], x[i][3]), codes(x[i][4], x[i][5]),
                       codes(x[i][6], x[i][7]));
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      up[w] = e4m3_order4(codes(hi[2 * w], hi[2 * w + 1]));
      dn[w] = e4m3_order4(codes(lo[2 * w], lo[2 * w + 1]));
    }
  });
  if (grown) {
    // the earlier codes move to the larger scale
    const float ratio = __fdiv_rn(was, s);
    for (int t = sh.first; sh.active && t < held; t += sh.tpu) {
      uint4* at = reinterpret_cast<uint4*>(rows + static_cast<int64_t>(t) * c.pitch);
      const uint4 old = *at;
      uint32_t q[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t h0, h1;
        e4m3x4_to_f16(q[w], &h0, &h1);
        const float2 v0 = half2_bits_to_float2(h0), v1 = half2_bits_to_float2(h1);
        q[w] = pack_e4m3x2(v0.x * ratio, v0.y * ratio) | (pack_e4m3x2(v1.x * ratio, v1.y * ratio) << 16);
        const uint32_t o = e4m3_order4(q[w]), nan = e4m3_nan4(q[w]);
        up[w] = __vmaxu4(up[w], o & ~nan);
        dn[w] = __vminu4(dn[w], o | nan);
      }
      *at = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
  if (!is_v) write_bounds(c, sh, gh, max(count, grown ? held : 0), held > 0 && !grown, up, dn);
}

// Fills page g of head h with `count` tokens of sequence b, picked out of its
// pages; thread t < count brings the position of the t-th.
//
// Codes whose page has the new page's scale, most of them, are moved as they
// are.  The largest |code| of a token and the bounds are found among the codes.
template <int UNITS>
__device__ __forceinline__ void move_page(const CacheView& c, const SeqView& sq, int b, int g, int h, bool is_v,
                                          int count, int mine) {
  __shared__ int64_t where[64];  // byte offset of a token's row, -1: none
  __shared__ float scales[64];
  const uint8_t* codes = is_v ? c.v : c.k;
  float my_scale = 0.f;
  if (threadIdx.x < 64) {
    const int t = threadIdx.x, j = t < count ? mine : -1;
    const int from = j >= 0 && j < (sq.width << c.log2_page) ? load_page(sq, c, b, j >> c.log2_page, true) : -1;
    const int64_t fh = static_cast<int64_t>(from) * c.heads + h;
    where[t] = from < 0 ? -1 : ((fh << c.log2_page) + (j & (c.page - 1))) * c.pitch;
    if (from >= 0) my_scale = (is_v ? c.v_scale : c.k_scale)[fh];
  }
  __syncthreads();
  const Share<UNITS> sh(c.pitch);
  const int64_t gh = static_cast<int64_t>(g) * c.heads + h;
  const bool half = sh.unit * 16 + 8 >= c.D;  // the unit ends in padding channels

  uint32_t x[Share<UNITS>::kMine][4];
#pragma unroll
  for (int i = 0; i < Share<UNITS>::kMine; ++i) {
    const int t = sh.first + i * sh.tpu;
    if (sh.active && t < count) {
      const int64_t at = where[t];
      const uint4 w = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(codes + at + sh.unit * 16)) : make_uint4(0, 0, 0, 0);
      x[i][0] = w.x, x[i][1] = w.y, x[i][2] = half ? 0u : w.z, x[i][3] = half ? 0u : w.w;
    }
  }
  // the codes' loads do not wait for the scales
  if (threadIdx.x < 64) scales[threadIdx.x] = my_scale;
  __syncthreads();
  float a = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < Share<UNITS>::kMine; ++i) {
    const int t = sh.first + i * sh.tpu;
    if (sh.active && t < count) {
      ByteMax most;  // |code|
#pragma unroll
      for (int w = 0; w < 4; ++w) most.add(x[i][w] & 0x7f7f7f7fu);
      if (most.largest() == 0x7fu) {  // some are NaN, which do not count
        nan = true;
        most = ByteMax();
#pragma unroll
        for (int w = 0; w < 4; ++w) most.add(x[i][w] & 0x7f7f7f7fu & ~e4m3_nan4(x[i][w]));
      }
      a = fmaxf(a, finite_abs(half2_bits_to_float2(e4m3x2_to_f16x2(most.largest())).x * scales[t]));
    }
  }
  const float s = page_scale(block_max(a));
  if (threadIdx.x == 0) (is_v ? c.v_scale : c.k_scale)[gh] = s;
  const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));  // 1 / s, a power of two
  uint8_t* rows = (is_v ? c.v : c.k) + (gh << c.log2_page) * c.pitch + sh.unit * 16;
  ByteMax high[4];
  ByteMin low[4];
#pragma unroll
  for (int i = 0; i < Share<UNITS>::kMine; ++i) {
    const int t = sh.first + i * sh.tpu;
    if (sh.active && t < count) {
      const float f = scales[t] * inv;
      const uint32_t fb = __float_as_uint(f);
      if (f != 1.f && (fb & 0x807fffffu) == 0u && fb >= 0x33800000u && fb <= 0x47000000u) {
        // a power of two that fp16 holds: the product of a code's 4 bits is
        // exact there down to 2^-24, and below 2^-14 rounds to code 0 either way
        const uint32_t ff = pack_f16x2(f, f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t h0, h1;
          e4m3x4_to_f16(x[i][w], &h0, &h1);
          x[i][w] = pack_e4m3x2_f16(mul_f16x2(h0, ff)) | (pack_e4m3x2_f16(mul_f16x2(h1, ff)) << 16);
        }
      } else if (f != 1.f && f < INFINITY) {  // inf: codes are 0 (those of a token have |code| <= 448 / f) or NaN, and stay
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t h0, h1;
          e4m3x4_to_f16(x[i][w], &h0, &h1);
          const float2 v0 = half2_bits_to_float2(h0), v1 = half2_bits_to_float2(h1);
          x[i][w] = pack_e4m3x2(v0.x * f, v0.y * f) | (pack_e4m3x2(v1.x * f, v1.y * f) << 16);
        }
      }
      *reinterpret_cast<uint4*>(rows + static_cast<int64_t>(t) * c.pitch) =
          make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
      if (!is_v && !nan) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t o = e4m3_order4(x[i][w]);
          high[w].add(o), low[w].add(o);
        }
      } else if (!is_v) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t o = e4m3_order4(x[i][w]), no = e4m3_nan4(x[i][w]);
          high[w].add(o & ~no), low[w].add(o | no);
        }
      }
    }
  }
  if (!is_v) {
    uint32_t up[4], dn[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) up[w] = high[w].get(), dn[w] = low[w].get();
    write_bounds(c, sh, gh, count, false, up, dn);
  }
}

template <bool F16, int UNITS>
__global__ void __launch_bounds__(kPageThreads) cache_append_kernel(const CacheAppendParams p) {
  const bool is_v = blockIdx.x & 1;
  const int j = blockIdx.x >> 1, h = blockIdx.y, b = blockIdx.z;
  int len, n;
  if (!load_seq(p.s, p.c, b, threadIdx.x == 0, &len, &n) || n == 0) return;
  const int start = len - n, i = (start >> p.c.log2_page) + j;
  if (i >= (len + p.c.page - 1) >> p.c.log2_page) return;
  const int base = i << p.c.log2_page;
  const int g = load_page(p.s, p.c, b, i, threadIdx.x == 0);
  const int from = max(base, start), to = min(base + p.c.page, len);
  const int64_t row = (static_cast<int64_t>(b) * p.c.heads + h) * p.s.T + (from - start);
  append_page<F16, UNITS>(p.c, g, h, is_v, from - base, to - from, (is_v ? p.v : p.k) + row * p.c.D);
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
    // a warp takes 1024 columns of a sequence's table at a time
    auto each = [&](int width, bool report, auto visit) {
      const int blocks = (width + 1023) >> 10;
      const int64_t units = static_cast<int64_t>(blocks) * p.s.batch;
      for (int64_t u = threadIdx.x >> 5; u < units; u += kPlanThreads / 32) {
        const int bb = static_cast<int>(u / blocks), i0 = static_cast<int>(u % blocks) << 10;
        int len, n;
        load_seq(p.s, p.c, bb, report && (threadIdx.x & 31) == 0, &len, &n);
        for (int i = i0 + (threadIdx.x & 31); i < min(width, i0 + 1024); i += 32) visit(bb, len, i);
      }
      __syncthreads();
    };
    each(p.s.width, true, [&](int bb, int len, int i) {
      if (i << p.c.log2_page >= len) return;
      const int g = load_page(p.s, p.c, bb, i, true);
      if (g >= 0) atomicOr(&once[g >> 5], 1u << (g & 31));
    });
    auto dst_of = [&](int bb, int len, int i) {  // a needed destination page, or -1
      return i << p.c.log2_page < min(len, p.keep) ? p.dst_table[static_cast<int64_t>(bb) * p.dst_width + i] : -1;
    };
    each(p.dst_width, false, [&](int bb, int len, int i) {
      const int g = dst_of(bb, len, i);
      const uint32_t bit = 1u << (g & 31);
      if (g >= 0 && g < p.c.pages && (atomicOr(&once[g >> 5], bit) & bit)) atomicOr(&twice[g >> 5], bit);
    });
    each(p.dst_width, false, [&](int bb, int len, int i) {
      const int g = dst_of(bb, len, i);
      const bool ok = g >= 0 && g < p.c.pages && !(twice[g >> 5] & (1u << (g & 31)));
      if (!ok && i << p.c.log2_page < min(len, p.keep)) dbg_fail(p.s.status, kChkCacheDst);
      p.dst_page[static_cast<int64_t>(bb) * p.dst_width + i] = ok ? g : -1;
    });
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
    block_top_ascending<kPlanThreads>(mass, len - tail, best, [&](int at, int j) {
      kept[at] = j;
      out[at] = mass[j];
    });
    for (int j = threadIdx.x; j < tail; j += kPlanThreads) {
      kept[best + j] = len - tail + j;
      out[best + j] = mass[len - tail + j];
    }
  }
  launch_dependents();
  for (int j = left + threadIdx.x; j < p.keep; j += kPlanThreads) kept[j] = -1;
  for (int j = left + threadIdx.x; j < (p.dst_width << p.c.log2_page); j += kPlanThreads)
    out[j] = 0.f;
}

// Twelve CTAs an SM where 128 channels or fewer allow it, at 40 registers with a few
// spilled: more loads in flight (a batch's eviction 50.5 us, at 48 registers and ten
// CTAs 51.7; one CTA for a page's keys and values, with one look-up, 55.2).
template <int UNITS>
__global__ void __launch_bounds__(kPageThreads, UNITS == 4 || UNITS == 8 ? 12 : 7)
    cache_evict_move_kernel(const CacheEvictParams p) {
  const bool is_v = blockIdx.x & 1;
  const int i = blockIdx.x >> 1, h = blockIdx.y, b = blockIdx.z;
  wait_for_previous();
  // three loads at once: a page's time is its chain of dependent loads
  const int base = i << p.c.log2_page, at = base + static_cast<int>(threadIdx.x);
  const int left = p.new_lens[b];
  const int g = p.dst_page[static_cast<int64_t>(b) * p.dst_width + i];
  const int mine = threadIdx.x < 64 && at < p.keep
                       ? p.kept[(static_cast<int64_t>(b) * p.c.heads + h) * p.keep + at] : -1;
  if (base >= left || g < 0) return;
  move_page<UNITS>(p.c, p.s, b, g, h, is_v, min(p.c.page, left - base), mine);
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
    e = launch_after(cache_evict_move_kernel<decltype(u)::value>, grid, kPageThreads, stream, p);
  });
  return e;
}

}  // namespace ea
