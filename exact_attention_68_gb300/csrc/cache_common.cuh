// cache_common.cuh — device helpers shared by the kernels of the 8-bit cache.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "attn_cache_impl.h"
#include "ptx.cuh"

namespace ea {

// Where a device-side check of the caller's arrays failed (second status word).
enum : int { kChkCacheSeq = 0x7101, kChkCacheTable, kChkCacheList, kChkCacheDst };

constexpr float kE4M3Max = 448.f;
constexpr int kMinScaleExp = -100;

// Sequence b's length and new tokens; false (reported once per caller thread
// with `report`) if they are out of range: the sequence is left out.
__device__ __forceinline__ bool load_seq(const SeqView& s, const CacheView& c, int b, bool report,
                                         int* len, int* fresh) {
  const int L = s.lens[b];
  const int n = s.fresh != nullptr ? s.fresh[b] : s.T;
  const bool ok = n >= 0 && n <= s.T && L >= n && L <= s.width << c.log2_page;
  if (!ok && report) dbg_fail(s.status, kChkCacheSeq);
  *len = ok ? L : 0;
  *fresh = ok ? n : 0;
  return ok;
}

// Page number in column i of sequence b's table, or -1 (reported) if it is
// not a page of the pool.
__device__ __forceinline__ int load_page(const SeqView& s, const CacheView& c, int b, int i,
                                         bool report) {
  const int g = s.table[static_cast<int64_t>(b) * s.width + i];
  const bool ok = g >= 0 && g < c.pages;
  if (!ok && report) dbg_fail(s.status, kChkCacheTable);
  return ok ? g : -1;
}

// The page scale for values up to a (>= 0, finite): 2^e, e the smallest
// integer >= kMinScaleExp with a <= 448·2^e.  448 = 1.75·2^8, so with
// a = f·2^x, f in [1, 2): e = x - 8, one more if f > 1.75.
__device__ __forceinline__ float page_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (e < kMinScaleExp) e = kMinScaleExp;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Calls body with a function that divides pairs by s with one rounding each: a
// product where s is a power of two in range (its reciprocal and the quotient
// are then exact), as every scale written here is; a division for others.
template <class Body>
__device__ __forceinline__ void with_divider(float s, Body body) {
  const uint32_t u = __float_as_uint(s);
  if ((u & 0x807fffffu) == 0u && (u >> 23) >= 2u && (u >> 23) <= 252u) {
    const float inv = __uint_as_float((254u - (u >> 23)) << 23);
    body([inv](float2 x) { return __fmul2_rn(x, make_float2(inv, inv)); });
  } else {
    body([s](float2 x) { return make_float2(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s)); });
  }
}

// Two fp32 to e4m3 (nearest even, saturating): lo in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The same from a pair of fp16 values.
__device__ __forceinline__ uint32_t pack_e4m3x2_f16(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two e4m3 codes (low 16 bits) to f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
// The four codes of a word to two f16x2.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t* lo, uint32_t* hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(w));
}

__device__ __forceinline__ float2 half2_bits_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A 16-bit pair (fp16 or bf16) as two floats.
template <bool F16>
__device__ __forceinline__ float2 pair_to_float2(uint32_t w) {
  if constexpr (F16) return half2_bits_to_float2(w);
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// |x| if finite, else 0.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// Larger and smaller of two pairs of 16-bit values; a NaN loses.
template <bool F16>
__device__ __forceinline__ uint32_t max_x2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (F16) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t min_x2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (F16) asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Larger and smaller of two pairs of unsigned 16-bit values, one instruction each.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// e4m3 codes as unsigned bytes in the order of their values, four at a time:
// negative codes inverted, the others above them.
__device__ __forceinline__ uint32_t e4m3_order4(uint32_t w) {
  uint32_t neg;  // 0xff in the bytes whose sign bit is set (a permutation that spreads it)
  asm("prmt.b32 %0, %1, 0, 0xba98;" : "=r"(neg) : "r"(w));
  return w ^ (neg | 0x80808080u);
}
// 0xff in the bytes that hold NaN codes.
__device__ __forceinline__ uint32_t e4m3_nan4(uint32_t w) {
  return ((((w & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u) * 0xffu;
}

// The int8 bound of one ordered code: the value in steps of 448/127, rounded
// up (upper bound) or down.  Only 0 and ±448 are whole numbers of steps (448 =
// 2^6·7 and 127 share no factor, a code's significand has 4 bits); at the others
// a product's rounding, 2^-23 of it, is far from carrying over a whole number,
// and ±448 is clamped to ±127.
__device__ __forceinline__ int bound_of_order(uint32_t o, bool upper) {
  const uint32_t code = o & 0x80u ? o ^ 0x80u : ~o & 0xffu;
  const float y = half2_bits_to_float2(e4m3x2_to_f16x2(code)).x * (127.f / kE4M3Max);
  const int r = static_cast<int>(upper ? ceilf(y) : floorf(y));
  return max(-127, min(127, r));
}

// Floats as unsigned keys in their order; NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Programmatic dependent launch: the next kernel of the stream may be set up
// once every CTA has said so or ended; its wait ends when this grid has.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A launch that may be set up before the stream's previous kernel has ended;
// the kernel calls wait_for_previous before it uses that one's results or ends.
template <class Params>
cudaError_t launch_after(void (*kern)(Params), dim3 grid, int threads, cudaStream_t stream, const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace ea
