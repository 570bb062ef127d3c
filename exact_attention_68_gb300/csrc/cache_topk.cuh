// cache_topk.cuh — the indices of the k largest of n keys, ascending, by one
// CTA: a radix selection finds the k-th largest key, an ordered pass emits.
#pragma once

#include <cstdint>

#include "cache_common.cuh"

namespace ea {

// What block_top_ascending keeps in shared memory.
template <int THREADS>
struct TopScratch {
  static constexpr int kBins = 2048;
  int hist[kBins];
  uint32_t prefix;
  int need;
  bool all;
  int counts[THREADS / 32];
  int2 pairs[THREADS / 32];
};

// Calls emit(place, index) for the k largest of x[0] .. x[n-1] (equal ones: the
// lowest indices), places 0 .. k-1 in the order of the indices.  Whole CTA of at
// most 1024 threads; 0 < k < n.  The values' keys are held in registers, up to
// ITEMS to a thread, side by side; where n needs more than one such tile, they
// are loaded again per pass.
//
// At most three passes over 11, 11 and 10 bits: a histogram of the keys that agree
// with the digits found so far, then the digit in which the k-th largest lies.
// Floats of like size share their leading bits, so wide digits matter: with
// four passes of 8 bits the first one's atomics fell on a few bins, and 64 rows
// of 16384 weights took 36 us.  The keys still in question are a mask, which is
// empty for most warps after the first pass; the search ends as soon as all that
// are left are taken, mostly after two.
template <int THREADS, int ITEMS, class Emit>
__device__ __forceinline__ void block_top_items(TopScratch<THREADS>& sh, const float* x, int n, int k, Emit emit) {
  constexpr int kWarps = THREADS / 32, kBins = TopScratch<THREADS>::kBins, kPer = kBins / THREADS;
  static_assert(kBins % THREADS == 0 && ITEMS <= 32, "bins are shared out evenly, keys are bits of a mask");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // whole vectors to a thread where it has several keys
  const int even = (n + THREADS - 1) / THREADS, per = min(ITEMS, ITEMS % 4 == 0 ? (even + 3) / 4 * 4 : even);
  const int tile = per * THREADS;
  const bool vectors = ITEMS % 4 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  const bool one_tile = n <= tile;
  uint32_t held[ITEMS], in = 0;  // this tile's keys, and which of them there are
  auto load = [&](int base) {
    const int at = base + threadIdx.x * per, left = min(per, n - at);
    in = left <= 0 ? 0u : left >= 32 ? 0xffffffffu : (1u << left) - 1u;
#pragma unroll
    for (int j = 0; j < ITEMS; j += 4) {
      if (ITEMS % 4 == 0 && vectors && ((in >> j) & 15u) == 15u) {
        const float4 v = *reinterpret_cast<const float4*>(x + at + j);
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < ITEMS) held[j + e] = order_key(f[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < ITEMS) held[j + e] = (in >> (j + e)) & 1u ? order_key(x[at + j + e]) : 0u;
      }
    }
  };
  if (one_tile) load(0);
  uint32_t prefix = 0, open = in;  // open: keys that agree with prefix (one tile)
  int need = k;                    // of those, how many are taken
  bool all = false;                // all that agree with prefix so far
#pragma unroll 1
  for (int pass = 0; pass < 3 && !all; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digits = pass == 2 ? 0x3ff : 0x7ff;
    const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sh.hist[threadIdx.x + j * THREADS] = 0;
    __syncthreads();
    for (int base = 0; base < n; base += tile) {
      if (!one_tile) {
        load(base);
        open = in;
      }
      if (pass > 0) {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
          if ((held[j] ^ prefix) & mask) open &= ~(1u << j);
      }
      if (open != 0) {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
          if ((open >> j) & 1u) atomicAdd(&sh.hist[(held[j] >> shift) & digits], 1);
      }
    }
    __syncthreads();
    // thread t holds kPer bins, the highest first; keys in higher bins by a scan
    int c[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum += c[j] = sh.hist[kBins - 1 - (threadIdx.x * kPer + j)];
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 31) sh.counts[warp] = upto;
    __syncthreads();
    upto += __reduce_add_sync(0xffffffffu, lane < warp ? sh.counts[lane] : 0);
    int before = upto - sum;
    if (before < need && need <= upto) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (before < need && need <= before + c[j]) {
          sh.prefix = prefix | (static_cast<uint32_t>(kBins - 1 - (threadIdx.x * kPer + j)) << shift);
          sh.need = need - before;
          sh.all = need - before == c[j];
        }
        before += c[j];
      }
    }
    __syncthreads();
    prefix = sh.prefix;
    need = sh.need;
    all = sh.all;
  }
  // Keys above the k-th largest are taken, and the first `need` that equal it;
  // where the search ended early, those from the prefix up, whose missing digits
  // are zero.
  int above = 0, equal = 0;  // counts before this tile
  for (int base = 0; base < n; base += tile) {
    if (!one_tile) load(base);
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      gt |= (all ? held[j] >= prefix : held[j] > prefix) ? 1u << j : 0u;
      eq |= !all && held[j] == prefix ? 1u << j : 0u;
    }
    gt &= in, eq &= in;
    const int ng = __popc(gt), ne = __popc(eq);
    int ug = ng, ue = ne;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int og = __shfl_up_sync(0xffffffffu, ug, d), oe = __shfl_up_sync(0xffffffffu, ue, d);
      if (lane >= d) ug += og, ue += oe;
    }
    __syncthreads();  // the last tile's pairs have been read
    if (lane == 31) sh.pairs[warp] = make_int2(ug, ue);
    __syncthreads();
    const int2 w = lane < kWarps ? sh.pairs[lane] : make_int2(0, 0);
    int g = above + ug - ng + __reduce_add_sync(0xffffffffu, lane < warp ? w.x : 0);
    int e = equal + ue - ne + __reduce_add_sync(0xffffffffu, lane < warp ? w.y : 0);
    above += __reduce_add_sync(0xffffffffu, w.x);
    equal += __reduce_add_sync(0xffffffffu, w.y);
    const int at = base + threadIdx.x * per;
    for (uint32_t left = gt | eq; left != 0; left &= left - 1) {
      const int j = __ffs(left) - 1;
      if ((gt >> j) & 1u) {
        emit(g + min(e, need), at + j);
        ++g;
      } else {
        if (e < need) emit(g + e, at + j);
        ++e;
      }
    }
  }
}

// The same for any 0 <= k and n, with as few registers' keys as n needs.
template <int THREADS, class Emit>
__device__ __forceinline__ void block_top_ascending(const float* x, int n, int k, Emit emit) {
  __shared__ TopScratch<THREADS> sh;
  if (k <= 0) return;
  if (k >= n) {
    for (int i = threadIdx.x; i < n; i += THREADS) emit(i, i);
  } else if (n <= THREADS) {
    block_top_items<THREADS, 1>(sh, x, n, k, emit);
  } else if (n <= 4 * THREADS) {
    block_top_items<THREADS, 4>(sh, x, n, k, emit);
  } else {
    block_top_items<THREADS, 16>(sh, x, n, k, emit);
  }
}

}  // namespace ea
