// cache_topk.cuh — the indices of the k largest of n keys, ascending, by one
// CTA: a radix selection finds the k-th largest key, an ordered pass emits.
#pragma once

#include <cstdint>

namespace ea {

// Calls emit(place, index) for the k largest of key(0) .. key(n-1) (equal
// keys: the lowest indices), places 0 .. k-1 in the order of the indices.
// Whole CTA of at most 1024 threads; 0 <= k.  Keys are held in registers, up to
// ITEMS to a thread, side by side; where n needs more than one such tile, key()
// is called again per pass.
//
// Three passes over 11, 11 and 10 bits: a histogram of the keys that agree
// with the digits found so far, then the digit in which the k-th largest lies.
// Floats of like size share their leading bits, so wide digits matter: with
// four passes of 8 bits the first one's atomics fell on a few bins, and 64 rows
// of 16384 weights took 36 us.
template <int THREADS, int ITEMS, class Key, class Emit>
__device__ __forceinline__ void block_top_ascending(Key key, int n, int k, Emit emit) {
  constexpr int kWarps = THREADS / 32, kBins = 2048, kPer = kBins / THREADS;
  static_assert(kBins % THREADS == 0, "bins are shared out evenly");
  __shared__ int hist[kBins];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_need;
  __shared__ int counts[kWarps];
  __shared__ int2 pairs[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (k <= 0 || n <= 0) return;
  const int per = min(ITEMS, (n + THREADS - 1) / THREADS), tile = per * THREADS;
  const bool all = k >= n, one_tile = n <= tile;
  const int mine = threadIdx.x * per;
  uint32_t held[ITEMS];
  auto load = [&](int base) {
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const int i = base + mine + j;
      held[j] = j < per && i < n ? key(i) : 0u;
    }
  };
  if (one_tile) load(0);
  uint32_t prefix = 0;
  int need = k;  // of the keys that agree with prefix, how many are taken
  if (!all) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digits = pass == 2 ? 0x3ff : 0x7ff;
      const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
#pragma unroll
      for (int j = 0; j < kPer; ++j) hist[threadIdx.x + j * THREADS] = 0;
      __syncthreads();
      for (int base = 0; base < n; base += tile) {
        if (!one_tile) load(base);
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
          if (j < per && base + mine + j < n && ((held[j] ^ prefix) & mask) == 0)
            atomicAdd(&hist[(held[j] >> shift) & digits], 1);
      }
      __syncthreads();
      // thread t holds kPer bins, the highest first; keys in higher bins by a scan
      int c[kPer], sum = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) sum += c[j] = hist[kBins - 1 - (threadIdx.x * kPer + j)];
      int upto = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      if (lane == 31) counts[warp] = upto;
      __syncthreads();
      upto += __reduce_add_sync(0xffffffffu, lane < warp ? counts[lane] : 0);
      int before = upto - sum;
      if (before < need && need <= upto) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if (before < need && need <= before + c[j]) {
            sh_prefix = prefix | (static_cast<uint32_t>(kBins - 1 - (threadIdx.x * kPer + j)) << shift);
            sh_need = need - before;
          }
          before += c[j];
        }
      }
      __syncthreads();
      prefix = sh_prefix;
      need = sh_need;
    }
  }
  // keys above the k-th largest are taken, and the first `need` that equal it
  int above = 0, equal = 0;  // counts before this tile
  for (int base = 0; base < n; base += tile) {
    if (!one_tile) load(base);
    int gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const bool in = j < per && base + mine + j < n;
      gt += in && (all || held[j] > prefix);
      eq += in && !all && held[j] == prefix;
    }
    int ug = gt, ue = eq;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int og = __shfl_up_sync(0xffffffffu, ug, d), oe = __shfl_up_sync(0xffffffffu, ue, d);
      if (lane >= d) ug += og, ue += oe;
    }
    __syncthreads();  // the last tile's pairs have been read
    if (lane == 31) pairs[warp] = make_int2(ug, ue);
    __syncthreads();
    int g = above + ug - gt, e = equal + ue - eq;
    const int2 w = lane < kWarps ? pairs[lane] : make_int2(0, 0);
    g += __reduce_add_sync(0xffffffffu, lane < warp ? w.x : 0);
    e += __reduce_add_sync(0xffffffffu, lane < warp ? w.y : 0);
    above += __reduce_add_sync(0xffffffffu, w.x);
    equal += __reduce_add_sync(0xffffffffu, w.y);
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const int i = base + mine + j;
      if (j >= per || i >= n) break;
      if (all || held[j] > prefix) {
        emit(g + min(e, need), i);
        ++g;
      } else if (held[j] == prefix) {
        if (e < need) emit(g + e, i);
        ++e;
      }
    }
  }
}

}  // namespace ea
