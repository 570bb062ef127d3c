// cache_topk.cuh — the indices of the k largest of n keys, ascending, by one
// CTA: a radix selection finds the k-th largest key, an ordered pass emits.
#pragma once

#include <cstdint>

namespace ea {

// Calls emit(place, index) for the k largest of key(0) .. key(n-1) (equal
// keys: the lowest indices), places 0 .. k-1 in the order of the indices.
// key() is called up to five times per index.  Whole CTA; 0 <= k.
//
// Four passes over 8 bits each: a histogram of the keys that agree with the
// digits found so far, then the digit in which the k-th largest lies.
template <int THREADS, class Key, class Emit>
__device__ __forceinline__ void block_top_ascending(Key key, int n, int k, Emit emit) {
  constexpr int kWarps = THREADS / 32;
  __shared__ int hist[256];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_need;
  __shared__ uint32_t counts[2][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (k <= 0 || n <= 0) return;
  uint32_t prefix = 0;
  int need = k < n ? k : n;  // of the keys that agree with prefix, how many are taken
  if (k < n) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += THREADS) hist[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int i = threadIdx.x; i < n; i += THREADS) {
        const uint32_t u = key(i);
        if (((u ^ prefix) & mask) == 0) atomicAdd(&hist[(u >> shift) & 255], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // lane L holds digits 255-8L .. 248-8L, the highest first
        int c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += c[j] = hist[255 - 8 * lane - j];
        int before = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, before, d);
          if (lane >= d) before += o;
        }
        before -= sum;  // keys in higher digits
        if (before < need && need <= before + sum) {
          int rest = need - before;
          int j = 0;
          while (rest > c[j]) rest -= c[j], ++j;
          sh_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - j) << shift);
          sh_need = rest;
        }
      }
      __syncthreads();
      prefix = sh_prefix;
      need = sh_need;
    }
  }
  // keys above the k-th largest are taken, and the first `need` that equal it
  int above = 0, equal = 0;  // counts before this step's keys
  for (int i0 = 0, step = 0; i0 < n; i0 += THREADS, ++step) {
    const int i = i0 + threadIdx.x;
    const uint32_t u = i < n ? key(i) : 0u;
    const bool all = k >= n;
    const bool gt = i < n && (all || u > prefix), eq = i < n && !all && u == prefix;
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) counts[step & 1][warp] = static_cast<uint32_t>(__popc(mg)) | (static_cast<uint32_t>(__popc(me)) << 16);
    __syncthreads();
    uint32_t low = 0, total = 0;  // this step's counts, packed (each at most THREADS)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t c = counts[step & 1][w];
      if (w < warp) low += c;
      total += c;
    }
    const uint32_t below = (1u << lane) - 1u;
    const int g = above + static_cast<int>(low & 0xffffu) + __popc(mg & below);
    const int e = equal + static_cast<int>(low >> 16) + __popc(me & below);
    if (gt) emit(g + (e < need ? e : need), i);
    else if (eq && e < need) emit(g + e, i);
    above += static_cast<int>(total & 0xffffu);
    equal += static_cast<int>(total >> 16);
  }
}

}  // namespace ea
