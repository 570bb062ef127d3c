// cache_fwd_sm103.cu — attention of a few new query tokens over the 8-bit
// cache on GB300 (sm_103a).
//
// Per query row: t_j = scale·log2e·k_scale·(q·code_j), the running maximum m
// and sum l of 2^(t_j - m), and out = Σ 2^(t_j - m)·v_scale·code_j / l.
//
// What bounds it is reading the cache once: 2·D bytes a key and head, against
// 4·D·G multiply-adds (G query heads a key head) that the tensor cores take at
// 16-bit rate.  So the work is cut for bytes in flight.  The unit is a chunk
// of 64 keys of one (sequence, head), a warp's step; the chunks of all
// (sequence, head, row tile), each of these with a lead for what it costs by
// itself, stand in one line that is dealt evenly to `workers`, whatever the
// lengths.  A warp feeds itself: its lane-elected TMA
// loads bring the pages of its next K and V chunks into its own ring of
// shared memory (128-byte swizzle; columns past D read as zero; or runs of
// bytes) while it works on the current one, so no warp waits for another.
//
// Arithmetic of a chunk, 8 query rows a tile: codes become fp16 exactly; q is
// brought to fp16 by a power of two per row chosen from its largest element,
// which keeps bf16's 8 bits over 2^28 of range; Sᵀ = K·Qᵀ and Oᵀ += Vᵀ·Pᵀ are
// mma.m16n8k16 with fp32 sums, the cache as the 16-row operand: with at most 8
// rows of queries (a group of heads) no row of a tile is idle, and a code is
// converted once for up to 16 rows.  (Queries as the 16-row operand: 1676
// instructions a chunk instead of 1085, 64 sequences of 8000-16384 keys 321 us
// instead of 243.)  A 16-channel unit of a key row is one 16-byte load per lane: a lane's four
// consecutive channels of each k-step are the channels that its Q fragment
// holds, so no data moves between lanes.  V, stored like K, comes transposed
// out of ldmatrix; P crosses the lanes by movmatrix.  tcgen05 with the cache as
// its M operand, 64 keys or channels by 8 to 256 rows, would take a copy of the codes
// in fp16 in shared memory: nothing to gain up to 16 rows, where the memory is the
// bound, but it would take 17 and more in one pass, where this kernel reads and
// converts the cache once for every 16 (32 at 64 channels).
//
// Page scales of V enter P: O is kept relative to r, the running maximum of
// t + log2(v_scale), and P = 2^(t + log2 v_scale - r + 14) fits fp16 however the
// pages' scales differ; its smallest step, 2^-38 of the largest term, is far
// below the 11 bits it is rounded to.  Those 11 bits are 3 more than a bf16 output
// keeps and as many as an fp16 one (2.2e-4 from the exact output, with fp32 weights
// 2.0e-4); more would take a second product for the rest of P.
//
// m is -inf only for a row that has met no key it may see: once it has, m is at
// least kLowest, also where all its scores are -inf (l is 0, and the row NaN as
// 0 / 0) or NaN, which the maximum drops and l keeps.  So the joins may leave out
// parts with m = -inf, and a row's answer does not depend on how the work was cut.
//
// A worker that covers a segment (one sequence, head and row tile) writes the
// result; others write O, m, r, l to the workspace and a second kernel joins
// them in a fixed order.  Where segments are few or short, a cluster of CTAs has
// each segment instead and joins it through its shared memory: no second launch.
//
// Measured (8 key heads, 4 query heads each, 128 channels): 64 sequences of
// 8000-16384 keys 246 us = 6.5 TB/s, 96 % of the measured copy rate; 16 of
// 500-8192 keys 36.9 us = 4.2 TB/s (a CTA has each segment, 24 of 152 SMs none, and
// the longest end last at about 65 GB/s a CTA; dealt evenly, the second launch costs
// more than that); one of 1000 keys 8.6 us (latency).  About 1040 instructions a
// chunk, 256 of them conversions of codes.
#include <atomic>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache_common.cuh"

namespace ea {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2f = 0.6931471805599453f;
constexpr int kPShift = 14;  // P is 2^14 times the weight relative to r
constexpr float kLowest = -3.402823466e38f;  // the running maximum of a row that has met a key
constexpr int kFar = 0x7fffff00;  // position of a token that is not there (real ones stay below 2^30)
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr int kMaxCluster = kCacheMaxCluster;

enum : int { kSiteCacheK = 0x7500, kSiteCacheV = 0x7600, kChkCacheCopy = 0x7701 };

// WIDTH: 64, 128 or 256 channels; WORKER: warps of one worker (all of the
// CTA's, or 1); NT: 8-row tiles of queries in one pass; PACKED: a chunk's rows lie
// in shared memory as in the pool, one behind the other.
//
// Tiled copies swizzle rows of 64 or 128 bytes, but where a token's row is an odd
// number of 16-byte units its start is off the 32-byte sectors every other time,
// and they slow down: 48 segments of 48000 keys of 80 channels took 135 us, of 96
// channels 87.  Such rows need no swizzle, since an odd pitch keeps eight rows in
// different banks, so that whole pages come as one run of bytes: 70 to 77 us.
template <int WIDTH, int WORKER, int NT, bool PACKED>
struct CacheFwdLayout {
  static constexpr bool kPacked = PACKED;
  static constexpr int kRows = 8 * NT;
  static constexpr int kWarps = kCacheWarps<WIDTH, NT>;
  static constexpr int kRowBytes = WIDTH >= 128 ? 128 : 64;  // one swizzled row
  static constexpr int kBlocks = WIDTH / kRowBytes;          // column blocks of a chunk
  static constexpr int kBlockBytes = kCacheChunk * kRowBytes;
  static constexpr int kSlot = kBlocks * kBlockBytes;        // one chunk of K or V
  static constexpr int kSlots = 192 * 1024 / (kWarps * kSlot);
  static constexpr int kWorkers = kWarps / WORKER;           // workers of a CTA
  static constexpr int kQPitch = 2 * WIDTH;                  // bytes of a Q row
  // chunks whose page data is held: those whose K has been asked for and the current one
  static constexpr int kMeta = kSlots / 2 + 1;
  static constexpr int kJoinCols = NT == 1 ? 64 : NT == 2 ? 32 : 16;  // columns joined at a time
  static constexpr int kRingOff = 0;
  static constexpr int kQOff = kWarps * kSlots * kSlot;
  static constexpr int kQsOff = kQOff + kWorkers * kRows * kQPitch;  // row factors
  static constexpr int kMetaOff = kQsOff + kWorkers * kRows * 4;
  static constexpr int kBarOff = kMetaOff + kWarps * kMeta * 4 * 16;
  static constexpr int kMiscOff = kBarOff + kWarps * kSlots * 8;
  static constexpr int kStatOff = kMiscOff + 16;
  static constexpr int kJoinOff = kStatOff + (WORKER > 1 ? kWarps * kRows * 12 : 0);
  static constexpr int kJoinPitch = kJoinCols + 4;
  static constexpr int kEnd = kJoinOff + (WORKER > 1 ? kWarps * kRows * kJoinPitch * 4 : 0);
  static constexpr int kAlloc = kEnd + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget exceeded");
  static_assert(kSlots >= 2, "a chunk's K and V");
};

__device__ __forceinline__ void mma_f16(float2 (&c)[2], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0].x), "+f"(c[0].y), "+f"(c[1].x), "+f"(c[1].y)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values over the warp (lane: row lane/4, columns
// 2·(lane%4), +1), transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Two 16 x 16 byte matrices, transposed: a lane gets, of matrix i, column
// lane/4 (r[2i]) and lane/4 + 8 (r[2i + 1]) of rows 4·(lane%4) .. +3.
__device__ __forceinline__ void ldmatrix_b8_trans_x2(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}

__device__ __forceinline__ void tma_load_3d_plain(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                  int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// `bytes` from global memory, all multiples of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// wait_bounded behind a poll that does not suspend the thread, so that a bound
// of 0 ends the first wait whose copy has not landed yet.
__device__ __forceinline__ bool wait_copy(uint32_t bar, uint32_t parity, const WaitCtl& ctl, int site) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (ok) return true;
  if (ctl.timeout_ns == 0) {
    raise_abort(ctl, site);
    return false;
  }
  return wait_bounded(bar, parity, ctl, site);
}

// All threads of the cluster; what any wrote to shared memory before is there
// for the others after.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A float at the same place `addr` of the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, int rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr, int rank) {
  float2 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\t"
      "ld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// A row's logsumexp out of its maximum and sum in log2 units: NaN where all scores
// are -inf, -inf where there are none.
__device__ __forceinline__ float row_lse(float m, float l) {
  const float z = (m + log2f(l)) * kLn2f;
  return l == 0.f && m != -INFINITY ? __int_as_float(0x7fffffff) : z;
}

// Over the eight lanes that hold the same query rows.
__device__ __forceinline__ float keys_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float keys_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Chunks of each of sequence b's segments (0: nothing to do).
__device__ __forceinline__ int seq_chunks(const CacheFwdParams& p, int b, bool report, int* len, int* n) {
  load_seq(p.s, p.c, b, report, len, n);
  if (*n == 0) return 0;
  const int pages = (*len + p.c.page - 1) >> p.c.log2_page;
  const int read = p.list != nullptr ? min(pages, p.listed) : pages;
  // a segment without keys still has rows to write
  return max(1, ((read << p.c.log2_page) + kCacheChunk - 1) / kCacheChunk);
}

// The deal: the segments in line, sequence by sequence, each p.lead units for what
// a segment costs by itself (Q, the join, the output) and one for each chunk.  A
// worker has the chunks of an even piece of the line; without the lead the ones
// that met many short segments ended last.
struct Deal {
  int total;  // units in line
  int per;    // units of a worker
};
// Units of a segment of nc chunks.
__device__ __forceinline__ int segment_units(const CacheFwdParams& p, int nc) { return nc > 0 ? nc + p.lead : 0; }
__device__ __forceinline__ int units_per_worker(const CacheFwdParams& p, int total) {
  return max((total + p.workers - 1) / p.workers, p.min_units);
}
__device__ __forceinline__ Deal deal_chunks(const CacheFwdParams& p, bool report) {
  const int lane = threadIdx.x & 31, hr = p.c.heads * p.row_tiles;
  int sum = 0;
  for (int b = lane; b < p.s.batch; b += 32) {
    int len, n;
    sum += hr * segment_units(p, seq_chunks(p, b, report, &len, &n));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return {sum, units_per_worker(p, sum)};
}

// Writes where each sequence's segments begin in the line, and its end, for the
// join.  One warp.
__device__ __forceinline__ void write_line(const CacheFwdParams& p) {
  const int lane = threadIdx.x & 31, hr = p.c.heads * p.row_tiles;
  int before = 0;
  for (int b0 = 0; b0 < p.s.batch; b0 += 32) {
    const int b = b0 + lane;
    int len, n;
    const int mine = b < p.s.batch ? hr * segment_units(p, seq_chunks(p, b, false, &len, &n)) : 0;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    if (b < p.s.batch) p.line[b] = before + upto - mine;
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  if (lane == 0) p.line[p.s.batch] = before;
}

// A segment in the line: sequence, head and row tile.
struct Segment {
  int b, h, rt;  // sequence, head, row tile
  int first, nc; // its chunks: first .. first + nc - 1
  int len, n;
};
// The segment that holds unit `at` (< total); its chunks are counted by their
// units.  Whole warp.
__device__ __forceinline__ Segment find_segment(const CacheFwdParams& p, int at) {
  const int lane = threadIdx.x & 31, hr = p.c.heads * p.row_tiles;
  int before = 0;
  for (int b0 = 0;; b0 += 32) {
    const int b = b0 + lane;
    int len = 0, n = 0;
    const int nc = b < p.s.batch ? seq_chunks(p, b, false, &len, &n) : 0;
    int upto = segment_units(p, nc) * hr;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + upto > at);
    if (hit != 0 || b0 + 32 >= p.s.batch) {
      const int src = hit != 0 ? __ffs(hit) - 1 : 0;
      Segment s;
      s.b = b0 + src;
      s.nc = __shfl_sync(0xffffffffu, nc, src);
      s.len = __shfl_sync(0xffffffffu, len, src);
      s.n = __shfl_sync(0xffffffffu, n, src);
      const int units = segment_units(p, s.nc), base = before + __shfl_sync(0xffffffffu, upto, src) - units * hr;
      const int x = units > 0 ? (at - base) / units : 0;
      s.h = x / p.row_tiles, s.rt = x % p.row_tiles;
      s.first = base + x * units + p.lead;
      return s;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
}
// Moves to the next segment, whose chunks are counted on without its lead; false
// behind the last.
__device__ __forceinline__ bool next_segment(const CacheFwdParams& p, Segment& s) {
  s.first += s.nc;
  if (++s.rt < p.row_tiles) return true;
  s.rt = 0;
  if (++s.h < p.c.heads) return true;
  s.h = 0;
  do {
    if (++s.b >= p.s.batch) return false;
    s.nc = seq_chunks(p, s.b, false, &s.len, &s.n);
  } while (s.nc == 0);
  return true;
}

// Whether entry i >= 0 of a page list may follow the one before it: a list that
// does not ascend, or goes on behind a negative entry, breaks this somewhere.
__device__ __forceinline__ bool follows(const int* list, int i) {
  return i == 0 || (list[i - 1] >= 0 && list[i] > list[i - 1]);
}

// Row `row` (query head in the group · T + token) of a segment: its place in
// q, out (rows of D) and lse.
__device__ __forceinline__ int64_t row_place(const CacheFwdParams& p, int b, int h, int row) {
  return (static_cast<int64_t>(b) * p.c.heads + h) * (p.G * p.s.T) + row;
}

__device__ __forceinline__ uint32_t pack_16bit(bool f16, float x, float y) {
  return f16 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
}
__device__ __forceinline__ float2 unpack_16bit(bool f16, uint32_t w) {
  return f16 ? pair_to_float2<true>(w) : pair_to_float2<false>(w);
}

// The last chunks of a sequence, whose V tiles need care; rare, so kept out of
// line.  A lane has two of the chunk's 64 rows; md: the chunk's page data.  The
// writes are ordered before the TMA copy that reuses the slot by the proxy fence
// here and the warp's barrier before that copy is issued.
__device__ __forceinline__ int row_position(uint32_t md, int row) {
  return ld_volatile_shared(md + (row >> 4) * 16) + (row & 15);
}
// Address of unit i (16 channels) of a chunk's row.
template <class L>
__device__ __forceinline__ uint32_t code_at(uint32_t slot, int row, int i, int pitch) {
  if constexpr (L::kPacked) return slot + row * pitch + 16 * i;
  constexpr int kUnits = L::kRowBytes / 16;
  const int sw = kUnits == 8 ? (row & 7) : ((row >> 1) & 3);
  return slot + (i / kUnits) * L::kBlockBytes + row * L::kRowBytes + (((i % kUnits) ^ sw) << 4);
}
// Zeroes the rows that hold no token of the sequence (they may hold anything,
// and 0 · NaN is NaN); true if a row that only some of the queries may see
// (positions above first_last) holds a NaN code.
template <class L>
__device__ __noinline__ bool clear_absent(uint32_t vslot, uint32_t md, int first_last, int len, int pitch) {
  bool nan = false;
  for (int row = threadIdx.x & 31; row < kCacheChunk; row += 32) {
    const int pos = row_position(md, row);
    if (pos <= first_last) continue;
    for (int i = 0; i < pitch / 16; ++i) {
      const uint32_t at = code_at<L>(vslot, row, i, pitch);
      if (pos >= len) {
        st_shared_v4(at, 0, 0, 0, 0);
      } else {
        const uint4 w = ld_shared_v4(at);
        nan = nan || (e4m3_nan4(w.x) | e4m3_nan4(w.y) | e4m3_nan4(w.z) | e4m3_nan4(w.w)) != 0;
      }
    }
  }
  fence_proxy_async_smem();
  return nan;
}
// Zeroes the NaN codes of the rows between first_last and len.
template <class L>
__device__ __noinline__ void clear_nan(uint32_t vslot, uint32_t md, int first_last, int len, int pitch) {
  for (int row = threadIdx.x & 31; row < kCacheChunk; row += 32) {
    const int pos = row_position(md, row);
    if (pos <= first_last || pos >= len) continue;
    for (int i = 0; i < pitch / 16; ++i) {
      const uint32_t at = code_at<L>(vslot, row, i, pitch);
      const uint4 w = ld_shared_v4(at);
      st_shared_v4(at, w.x & ~e4m3_nan4(w.x), w.y & ~e4m3_nan4(w.y), w.z & ~e4m3_nan4(w.z), w.w & ~e4m3_nan4(w.w));
    }
  }
  fence_proxy_async_smem();
}
// The first position above first_last whose row holds a NaN code in channel ch.
template <class L>
__device__ __noinline__ int first_nan(uint32_t vslot, uint32_t md, int ch, int first_last, int len, int pitch) {
  int first = kFar;
  for (int row = 0; row < kCacheChunk; ++row) {
    const int pos = row_position(md, row);
    if (pos <= first_last || pos >= len) continue;
    const uint32_t w = static_cast<uint32_t>(ld_volatile_shared(code_at<L>(vslot, row, ch >> 4, pitch) + (ch & 12)));
    if (((w >> (8 * (ch & 3))) & 0x7fu) == 0x7fu) first = min(first, pos);
  }
  return first;
}

template <int WIDTH, int WORKER, int NT, bool PACKED>
__global__ void __launch_bounds__(CacheFwdLayout<WIDTH, WORKER, NT, PACKED>::kWarps * 32, 1)
    cache_fwd_kernel(const __grid_constant__ CacheFwdParams p) {
  using L = CacheFwdLayout<WIDTH, WORKER, NT, PACKED>;
  constexpr int kRows = L::kRows;
  constexpr int kKSteps = WIDTH / 64;  // 64-channel blocks of K·Qᵀ
  constexpr int kTiles = WIDTH / 16;   // 16-channel tiles of Oᵀ
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, t4 = lane & 3;
  const int worker_in_cta = warp / WORKER, wi = warp % WORKER;
  const uint32_t ring = sb + L::kRingOff + warp * L::kSlots * L::kSlot;
  const uint32_t bars = sb + L::kBarOff + warp * L::kSlots * 8;
  const uint32_t meta = sb + L::kMetaOff + warp * L::kMeta * 64;
  const uint32_t qs = sb + L::kQOff + worker_in_cta * kRows * L::kQPitch;
  const uint32_t qf = sb + L::kQsOff + worker_in_cta * kRows * 4;
  const uint32_t abort_addr = sb + L::kMiscOff;
  if (lane == 0) {
    for (int s = 0; s < L::kSlots; ++s) mbar_init(bars + 8 * s, 1);
    fence_barrier_init();
    if (warp == 0) st_volatile_shared(abort_addr, 0);
  }
  __syncthreads();
  const WaitCtl ctl{abort_addr, p.s.status, p.timeout_ns};
  const DbgBounds dbb{p.s.status, sb, smem_u32(smem_raw) + static_cast<uint32_t>(L::kAlloc), p.c.page, p.c.D,
                      p.c.pages * p.c.heads};

  const int worker = blockIdx.x * L::kWorkers + worker_in_cta;
  int begin, end;  // this worker's chunks of the line
  Segment cs;
  int cluster = 0, rank = 0;
  if constexpr (WORKER > 1) {
    cluster = p.cluster;
    if (cluster > 0) {
      // a cluster for each segment, a line of its own: every CTA an even share
      rank = blockIdx.x % cluster;
      const int seg = blockIdx.x / cluster;
      cs.rt = seg % p.row_tiles;
      cs.h = seg / p.row_tiles % p.c.heads;
      cs.b = seg / p.row_tiles / p.c.heads;
      cs.nc = seq_chunks(p, cs.b, cs.rt == 0 && cs.h == 0 && warp == 0 && rank == 0, &cs.len, &cs.n);
      cs.first = 0;
      begin = static_cast<int>(static_cast<int64_t>(cs.nc) * rank / cluster);
      end = static_cast<int>(static_cast<int64_t>(cs.nc) * (rank + 1) / cluster);
      if (cs.nc == 0) return;  // the whole cluster; a CTA without a share takes part in the join
    }
  }
  if (cluster == 0) {
    const Deal deal = deal_chunks(p, blockIdx.x == 0 && warp == 0);
    if (blockIdx.x == 0 && warp == 0) write_line(p);
    // 64 bits: worker · per may pass 2^31 (total is below 2^30)
    begin = static_cast<int>(min(static_cast<int64_t>(worker) * deal.per, static_cast<int64_t>(deal.total)));
    end = min(begin + deal.per, deal.total);
    if (begin >= end) return;  // the whole worker; with WORKER > 1 the whole CTA
    cs = find_segment(p, begin);
    begin = max(begin, cs.first);
    if (begin >= end) return;  // a piece of a lead
  }

  const int seg_rows = p.G * p.s.T;
  const int log2p = p.c.log2_page, page_mask = p.c.page - 1;
  // bytes of a row that hold channels: all that are read where rows are packed
  const int row_pitch = PACKED ? p.c.pitch : L::kBlocks * L::kRowBytes;
  const bool one_page = p.c.page == kCacheChunk;  // of a chunk

  // ---------------- fetching: chunks begin + wi, + WORKER, ... of the line
  Segment fs = cs;
  int f_at = begin + wi;      // next chunk to fetch K of
  int f_end = end;            // past the last, less the leads up to here
  int f_page = -1, f_pos = kFar;  // this lane's 16-token group (t4) of it
  bool f_have = false;
  int i_slot = 0;             // slot of the next item
  int f_meta = 0;             // page data entry of the chunk f_at
  float pend_ks = 0.f, pend_vs = 0.f;  // page data on its way
  int pend_pos = kFar, pend_meta = -1;
  int issued = 0, used = 0;   // items (K or V of a chunk)

  auto look_up = [&]() {  // pages of chunk f_at
    f_page = -1;
    f_pos = kFar;
    while (f_at < f_end && f_at >= fs.first + fs.nc) {
      next_segment(p, fs);
      f_end -= p.lead;
    }
    f_have = f_at < f_end;
    if (!f_have) return;
    const int tok = (f_at - fs.first) * kCacheChunk + 16 * t4;
    int i = tok >> log2p;
    bool in = true;
    if (p.list != nullptr) {
      in = i < p.listed;
      if (in) {
        const int* l = p.list + (static_cast<int64_t>(fs.b) * p.c.heads + fs.h) * p.listed;
        const int e = l[i];
        in = e >= 0;
        if (in && (e >= p.s.width || !follows(l, i))) {
          dbg_fail(p.s.status, kChkCacheList);
          in = false;
        }
        i = e;
      }
    }
    const int pos = in ? (i << log2p) + (tok & page_mask) : kFar;
    if (in && pos < fs.len) {
      f_page = p.s.table[static_cast<int64_t>(fs.b) * p.s.width + i];
      f_pos = pos;
    }
  };
  auto flush_pending = [&]() {
    if (pend_meta >= 0) {
      // v_scale as a power of two and a factor in [1, 2)
      const uint32_t u = __float_as_uint(pend_vs);
      const float ev = static_cast<float>(static_cast<int>((u >> 23) & 0xffu) - 127);
      const float vm = __uint_as_float((u & 0x807fffffu) | 0x3f800000u);
      if (lane < 4)
        st_shared_v4(meta + pend_meta * 64 + lane * 16, static_cast<uint32_t>(pend_pos),
                     __float_as_uint(pend_ks), __float_as_uint(ev), __float_as_uint(vm));
      pend_meta = -1;
      __syncwarp();
    }
  };
  // K (then V) of chunk f_at into the next slot; V moves on to the next chunk
  bool f_is_v = false;
  auto issue = [&]() {
    if (!f_is_v) flush_pending();
    if (!f_have) return;
    if (!f_is_v && f_pos != kFar && (f_page < 0 || f_page >= p.c.pages)) {
      dbg_fail(p.s.status, kChkCacheTable);
      f_page = -1;
      f_pos = kFar;
    }
    const bool lead = lane < 4 && ((16 * t4) & page_mask) == 0 && f_pos != kFar;
    const uint32_t leads = __ballot_sync(0xffffffffu, lead);
    const uint32_t bar = bars + 8 * i_slot;
    if (lane == 0) {
      if (leads != 0) mbar_arrive_expect_tx(bar, __popc(leads) * p.c.page * row_pitch);
      else mbar_arrive(bar);
    }
    __syncwarp();
    const int64_t gh = static_cast<int64_t>(f_page) * p.c.heads + fs.h;
    if (PACKED) {
      const uint32_t dst = ring + i_slot * L::kSlot + 16 * t4 * row_pitch, bytes = p.c.page * row_pitch;
      if (lead && dbg_smem(dbb, dst, bytes, 16, kChkCacheCopy) && dbg(gh >= 0 && gh < dbb.slices, dbb, kChkCacheCopy))
        bulk_load(dst, (f_is_v ? p.c.v : p.c.k) + gh * static_cast<int64_t>(bytes), bytes, bar);
    } else if (lead) {
#pragma unroll
      for (int cb = 0; cb < L::kBlocks; ++cb) {
        const uint32_t dst = ring + i_slot * L::kSlot + cb * L::kBlockBytes + 16 * t4 * L::kRowBytes;
        // a copy left out leaves the barrier short: the bounded wait ends the kernel
        if (dbg_tma(dbb, dst, p.c.page * L::kRowBytes, cb * L::kRowBytes, 0, static_cast<int>(gh), false, kChkCacheCopy))
          tma_load_3d_plain(dst, f_is_v ? &p.tm_v : &p.tm_k, bar, cb * L::kRowBytes, 0, static_cast<int>(gh));
      }
    }
    if (!f_is_v) {
      pend_pos = f_pos;
      pend_ks = f_pos != kFar ? __ldg(p.c.k_scale + gh) : 0.f;
      pend_vs = f_pos != kFar ? __ldg(p.c.v_scale + gh) : 1.f;
      pend_meta = f_meta;
    } else {
      f_at += WORKER;
      f_meta = (f_meta + 1) % L::kMeta;
      look_up();
    }
    f_is_v = !f_is_v;
    if (++i_slot == L::kSlots) i_slot = 0;
    ++issued;
  };
  look_up();
#pragma unroll 1
  for (int s = 0; s < L::kSlots; ++s) issue();

  // ---------------- the worker's segments
  // This lane's key of a 16-key tile; the other is row0 + 2.  Keys of a tile are
  // taken in an order in which two lanes of eight that load together are four
  // rows apart, so that the swizzle keeps them in different banks; V's rows go to
  // ldmatrix in the same order.
  const int row0 = 8 * (gid >> 2) + 4 * (gid & 1) + ((gid >> 1) & 1);
  const int vrow = (lane & 8) | ((lane & 1) << 2) | (lane & 2) | ((lane >> 2) & 1);
  int at = begin + wi, u_slot = 0, u_parity = 0, u_meta = 0;
  bool alive = true;
  int seg_at = begin;
  do {
    while (seg_at < end && seg_at >= cs.first + cs.nc) {
      next_segment(p, cs);
      end -= p.lead;
    }
    if (seg_at >= end && cluster == 0) break;
    const int seg_end = min(end, cs.first + cs.nc);
    const int h = cs.h, tile_row = cs.rt * kRows, tile_rows = min(kRows, seg_rows - tile_row);

    // ---- Q to fp16 with a power of two per row
    {
      // rows of a warp (kRows shared out, rounded up to a power of two), lanes of a row
      constexpr int kShare = (kRows + WORKER - 1) / WORKER;
      constexpr int kMine = kShare <= 1 ? 1 : kShare <= 2 ? 2 : kShare <= 4 ? 4 : kShare <= 8 ? 8 : kShare <= 16 ? 16 : 32;
      constexpr int kLanes = 32 / kMine;
      const int r = wi * kMine + lane / kLanes, part = lane % kLanes;
      const bool here = r < kRows, in = r < tile_rows;
      const uint16_t* q = p.q + row_place(p, cs.b, h, tile_row + (in ? r : 0)) * p.c.D;
      float a = 0.f;
      for (int c = 8 * part; c < p.c.D; c += 8 * kLanes) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(q + c));
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = unpack_16bit(p.f16, ws[e]);
          a = fmaxf(a, fmaxf(finite_abs(x.x), finite_abs(x.y)));
        }
      }
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
      // up = 2^(14 - e) for a in [2^e, 2^(e+1)); kept in range for tiny and huge a
      int e = static_cast<int>(__float_as_uint(a) >> 23) - 127;
      e = max(-100, e);
      const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
      for (int c = 8 * part; c < WIDTH; c += 8 * kLanes) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (in && c < p.c.D) w = __ldg(reinterpret_cast<const uint4*>(q + c));
        if (!here) continue;
        uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 x = unpack_16bit(p.f16, ws[k]);
          ws[k] = pack_f16x2(x.x * up, x.y * up);
        }
        // odd rows swap the halves of each 32 bytes: a fragment load of two
        // rows then meets every bank once
        st_shared_v4(qs + r * L::kQPitch + ((2 * c) ^ ((r & 1) << 4)), ws[0], ws[1], ws[2], ws[3]);
      }
      if (part == 0 && here)
        st_shared_f32(qf + 4 * r, p.scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23));
      if constexpr (WORKER > 1) __syncthreads();
      else __syncwarp();
    }
    // this lane's rows: 8·b + 2·t4 + i
    float2 qk[NT];
    int last[NT][2];  // last position a row may attend to; rows that are not there see every key
    auto last_of = [&](int r) {
      const int i = (tile_row + r) % p.s.T;
      return r < tile_rows && i < cs.n ? cs.len - cs.n + i : cs.len - 1;
    };
#pragma unroll
    for (int b = 0; b < NT; ++b) {
      const int r = 8 * b + 2 * t4;
      qk[b] = make_float2(ld_shared_f32(qf + 4 * r), ld_shared_f32(qf + 4 * r + 4));
      last[b][0] = last_of(r), last[b][1] = last_of(r + 1);
    }
    const int first_last = cs.len - cs.n;  // every row sees the keys up to here

    const float2 zero2 = make_float2(0.f, 0.f), none2 = make_float2(-INFINITY, -INFINITY);
    float2 o[kTiles][NT][2];  // channel 16·u + gid + 8·hf, the two rows of tile b: [u][b][hf]
#pragma unroll
    for (int u = 0; u < kTiles; ++u)
#pragma unroll
      for (int b = 0; b < NT; ++b) o[u][b][0] = o[u][b][1] = zero2;
    float2 m[NT], r[NT], l[NT];
#pragma unroll
    for (int b = 0; b < NT; ++b) m[b] = r[b] = none2, l[b] = zero2;

#pragma unroll 1
    for (; at < seg_end; at += WORKER) {
      // ---- Sᵀ = K·Qᵀ
      if (alive) alive = __all_sync(0xffffffffu, wait_copy(bars + 8 * u_slot, u_parity, ctl, kSiteCacheK));
      if (!alive) continue;
      const uint32_t kslot = ring + u_slot * L::kSlot;
      float2 s[4][NT][2];  // key row0 + 2·hf of 16-key tile g, the two rows of tile b: [g][b][hf]
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int b = 0; b < NT; ++b) s[g][b][0] = s[g][b][1] = zero2;
// rolled where registers are short (21 sequences of 996-4114 keys, 24 rows of 256
// channels: 200 us, unrolled 290 us; 128 channels or 8 rows: no change or slower)
#pragma unroll(WIDTH > 128 && NT > 1 ? 1 : kKSteps)
      for (int kb = 0; kb < kKSteps; ++kb) {
        uint32_t qw[NT][8];
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          const uint32_t qa = qs + (8 * b + gid) * L::kQPitch + kb * 128 + 32 * t4 + ((gid & 1) << 4);
          const uint4 x0 = ld_shared_v4(qa), x1 = ld_shared_v4(qa ^ 16u);
          qw[b][0] = x0.x, qw[b][1] = x0.y, qw[b][2] = x0.z, qw[b][3] = x0.w;
          qw[b][4] = x1.x, qw[b][5] = x1.y, qw[b][6] = x1.z, qw[b][7] = x1.w;
        }
        const int unit = kb * 4 + t4;  // 16 channels
        // packed rows end with the pool's channels, their last unit perhaps in padding,
        // which may hold anything (Q is zero there, but 0 · NaN is NaN)
        const bool none = PACKED && 16 * unit >= p.c.D, half = PACKED && 16 * unit + 8 >= p.c.D;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint4 kw[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            kw[hf] = none ? make_uint4(0, 0, 0, 0) : ld_shared_v4(code_at<L>(kslot, row0 + 16 * g + 2 * hf, unit, row_pitch));
            if (half) kw[hf].z = kw[hf].w = 0;
          }
          const uint32_t x[4] = {kw[0].x, kw[0].y, kw[0].z, kw[0].w}, y[4] = {kw[1].x, kw[1].y, kw[1].z, kw[1].w};
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16(x[st], &a0, &a2);
            e4m3x4_to_f16(y[st], &a1, &a3);
#pragma unroll
            for (int b = 0; b < NT; ++b) mma_f16(s[g][b], a0, a1, a2, a3, qw[b][2 * st], qw[b][2 * st + 1]);
          }
        }
      }
      ++used;
      if (++u_slot == L::kSlots) u_slot = 0, u_parity ^= 1;
      __syncwarp();
      issue();

      // ---- softmax of the chunk; the two rows of a lane's tile go in pairs
      float ev[4], vm[4];
      int gpos[4];
      bool tail = false;  // some key is hidden from some row
      int nearest = kFar;  // the chunk's first position
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint4 md = ld_shared_v4(meta + u_meta * 64 + g * 16);
        gpos[g] = static_cast<int>(md.x);
        ev[g] = __uint_as_float(md.z);
        vm[g] = __uint_as_float(md.w);
        tail = tail || gpos[g] + 15 > first_last;
        nearest = min(nearest, gpos[g]);
        const float2 ks = make_float2(__uint_as_float(md.y), __uint_as_float(md.y));
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          const float2 f = __fmul2_rn(qk[b], ks);
          s[g][b][0] = __fmul2_rn(s[g][b][0], f);
          s[g][b][1] = __fmul2_rn(s[g][b][1], f);
        }
      }
      if (tail) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int pos = gpos[g] + row0 + 2 * hf;
              if (pos > last[b][0]) s[g][b][hf].x = -INFINITY;
              if (pos > last[b][1]) s[g][b][hf].y = -INFINITY;
            }
      }
      if (p.scores != nullptr) {
        // [key][row]: the 8 rows of a key side by side
        const int64_t row_len = static_cast<int64_t>(p.row_tiles) * kRows;
        float* sc = p.scores + ((static_cast<int64_t>(cs.b) * p.c.heads + h) * p.score_cols +
                                static_cast<int64_t>(at - cs.first) * kCacheChunk + row0) * row_len + tile_row + 2 * t4;
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int b = 0; b < NT; ++b)
              *reinterpret_cast<float2*>(sc + (16 * g + 2 * hf) * row_len + 8 * b) = s[g][b][hf];
      }
      float2 mn[NT], rel[NT], beta[NT];  // -reference of m, reference of m minus that of r
      bool moved = false;
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        // a row that may see a key of the chunk
        float mx[2] = {nearest <= last[b][0] ? kLowest : -INFINITY, nearest <= last[b][1] ? kLowest : -INFINITY};
        float rx[2];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float a0 = fmaxf(s[g][b][0].x, s[g][b][1].x), a1 = fmaxf(s[g][b][0].y, s[g][b][1].y);
          const float2 av = __fadd2_rn(make_float2(a0, a1), make_float2(ev[g], ev[g]));
          mx[0] = fmaxf(mx[0], a0), mx[1] = fmaxf(mx[1], a1);
          rx[0] = g == 0 ? av.x : fmaxf(rx[0], av.x), rx[1] = g == 0 ? av.y : fmaxf(rx[1], av.y);
        }
        // references: 0 where no key has been allowed yet
        auto update = [&](float& run, float x, float& ref) {
          const float top = fmaxf(run, keys_max(x));
          ref = top == -INFINITY ? 0.f : top;
          const float f = ex2_approx(run - ref);
          moved = moved || top != run;
          run = top;
          return f;
        };
        float2 mr, rr, alpha;
        alpha.x = update(m[b].x, mx[0], mr.x), alpha.y = update(m[b].y, mx[1], mr.y);
        beta[b].x = update(r[b].x, rx[0], rr.x), beta[b].y = update(r[b].y, rx[1], rr.y);
        l[b] = __fmul2_rn(l[b], alpha);
        mn[b] = make_float2(-mr.x, -mr.y);
        rel[b] = make_float2(mr.x - rr.x + kPShift, mr.y - rr.y + kPShift);
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int u = 0; u < kTiles; ++u)
#pragma unroll
          for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) o[u][b][hf] = __fmul2_rn(o[u][b][hf], beta[b]);
      }
      uint32_t pb[4][NT][2];  // P, B fragments of the four 16-key steps
      float2 pf[NT];
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          // a page whose weights are far below the chunk's has a factor beyond
          // range; its P is held finite
          if (g == 0 || !one_page) {
            const float2 x = __fadd2_rn(make_float2(ev[g], ev[g]), rel[b]);
            pf[b] = make_float2(ex2_approx(fminf(x.x, 126.f)) * vm[g], ex2_approx(fminf(x.y, 126.f)) * vm[g]);
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float2 t = __fadd2_rn(s[g][b][hf], mn[b]);
            const float2 w = make_float2(ex2_approx(t.x), ex2_approx(t.y));
            l[b] = __fadd2_rn(l[b], w);
            const float2 pv = __fmul2_rn(w, pf[b]);
            pb[g][b][hf] = movmatrix_trans(pack_f16x2(pv.x, pv.y));
          }
        }

      // ---- Oᵀ += Vᵀ·Pᵀ
      if (alive) alive = __all_sync(0xffffffffu, wait_copy(bars + 8 * u_slot, u_parity, ctl, kSiteCacheV));
      if (!alive) continue;
      const uint32_t vslot = ring + u_slot * L::kSlot;
      if (tail) {
        const uint32_t md = meta + u_meta * 64;
        if (__any_sync(0xffffffffu, clear_absent<L>(vslot, md, first_last, cs.len, row_pitch))) {
          // A NaN code that some rows may see and others may not: the ones that
          // may get it now, then it counts as zero.
#pragma unroll
          for (int u = 0; u < kTiles; ++u)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int from = first_nan<L>(vslot, md, 16 * u + gid + 8 * hf, first_last, cs.len, row_pitch);
#pragma unroll
              for (int b = 0; b < NT; ++b) {
                if (from <= last[b][0]) o[u][b][hf].x = __int_as_float(0x7fffffff);
                if (from <= last[b][1]) o[u][b][hf].y = __int_as_float(0x7fffffff);
              }
            }
          __syncwarp();
          clear_nan<L>(vslot, md, first_last, cs.len, row_pitch);
        }
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < kTiles; u += 2) {
        if (16 * u < p.c.D) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t w[4];
            ldmatrix_b8_trans_x2(code_at<L>(vslot, 16 * g + vrow, u + (lane >> 4), row_pitch), w);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(w[2 * i], &a0, &a2);
              e4m3x4_to_f16(w[2 * i + 1], &a1, &a3);
#pragma unroll
              for (int b = 0; b < NT; ++b) mma_f16(o[u + i][b], a0, a1, a2, a3, pb[g][b][0], pb[g][b][1]);
            }
          }
        }
      }
      ++used;
      if (++u_slot == L::kSlots) u_slot = 0, u_parity ^= 1;
      if (++u_meta == L::kMeta) u_meta = 0;
      __syncwarp();
      issue();
    }
    if (end - seg_end <= p.lead) launch_dependents();  // no chunk behind: the join may be set up meanwhile
#pragma unroll
    for (int b = 0; b < NT; ++b) l[b] = make_float2(keys_sum(l[b].x), keys_sum(l[b].y));
    // row i (0, 1) of a pair
    auto of = [](const float2& v, int i) { return i ? v.y : v.x; };

    // ---- the segment's result, or this worker's part of it
    const bool whole = seg_at == cs.first && seg_end == cs.first + cs.nc;
    float* part = p.part + (2ll * worker + (seg_at == cs.first ? 1 : 0)) * kCachePartFloats<WIDTH, NT>;
    float* part_stat = part + kRows * WIDTH;
    auto live = [&](int row) { return row < tile_rows && (tile_row + row) % p.s.T < cs.n; };
    // 2^(r - 14 - m) / l: what an entry of O is multiplied by
    auto factor = [](float mm, float rr, float ll) {
      return mm == -INFINITY ? 0.f : ex2_approx(rr - mm - kPShift) / ll;
    };
    if constexpr (WORKER == 1) {
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 8 * b + 2 * t4 + i;
          const float mi = of(m[b], i), ri = of(r[b], i), li = of(l[b], i);
          if (whole) {
            if (!live(row)) continue;
            const int64_t to = row_place(p, cs.b, h, tile_row + row);
            const float w = factor(mi, ri, li);
#pragma unroll
            for (int u = 0; u < kTiles; ++u)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const int ch = 16 * u + gid + 8 * hf;
                const float x = mi == -INFINITY ? 0.f : of(o[u][b][hf], i) * w;
                if (ch < p.c.D) p.out[to * p.c.D + ch] = static_cast<uint16_t>(pack_16bit(p.f16, x, 0.f));
              }
            if (gid == 0) p.lse[to] = row_lse(mi, li);
          } else {
#pragma unroll
            for (int u = 0; u < kTiles; ++u)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) part[row * WIDTH + 16 * u + gid + 8 * hf] = of(o[u][b][hf], i);
            if (gid == 0) {
              part_stat[row] = mi;
              part_stat[kRows + row] = ri;
              part_stat[2 * kRows + row] = li;
            }
          }
        }
      __syncwarp();  // Q is rewritten for the next segment
    } else {
      // a cluster's join: O, then m, r, l, over the first warp's ring
      constexpr int kSumStat = kRows * WIDTH * 4;
      static_assert(kSumStat + kRows * 12 <= L::kSlots * L::kSlot, "a CTA's sums must fit the ring");
      // the warps' parts joined, kJoinCols columns at a time, in the order of the warps
      const uint32_t stat = sb + L::kStatOff, join = sb + L::kJoinOff;
      if (gid == 0) {
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t to = stat + (warp * kRows + 8 * b + 2 * t4 + i) * 12;
            st_shared_f32(to, of(m[b], i));
            st_shared_f32(to + 4, of(r[b], i));
            st_shared_f32(to + 8, of(l[b], i));
          }
      }
      __syncthreads();
      // Thread `row` joins the warps' statistics of its row, once for all: m, r and
      // the factor of O then stand in the first warp's place, which only it reads.
      if (threadIdx.x < kRows) {
        const int row = threadIdx.x;
        float mw[L::kWarps], M = -INFINITY, R = -INFINITY, S = 0.f;
#pragma unroll
        for (int w = 0; w < L::kWarps; ++w) {
          mw[w] = ld_shared_f32(stat + (w * kRows + row) * 12);
          M = fmaxf(M, mw[w]), R = fmaxf(R, ld_shared_f32(stat + (w * kRows + row) * 12 + 4));
        }
#pragma unroll
        for (int w = 0; w < L::kWarps; ++w)
          S += mw[w] == -INFINITY ? 0.f : ld_shared_f32(stat + (w * kRows + row) * 12 + 8) * ex2_approx(mw[w] - M);
        st_shared_f32(stat + row * 12, M);
        st_shared_f32(stat + row * 12 + 4, R);
        st_shared_f32(stat + row * 12 + 8, factor(M, R, S));
        if (cluster > 1) {
          st_shared_f32(sb + kSumStat + row * 12, M);
          st_shared_f32(sb + kSumStat + row * 12 + 4, R);
          st_shared_f32(sb + kSumStat + row * 12 + 8, S);
        } else if (!whole) {
          part_stat[row] = M;
          part_stat[kRows + row] = R;
          part_stat[2 * kRows + row] = S;
        } else if (live(row)) {
          p.lse[row_place(p, cs.b, h, tile_row + row)] = row_lse(M, S);
        }
      }
      __syncthreads();
      float beta[NT][2];
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float R = ld_shared_f32(stat + (8 * b + 2 * t4 + i) * 12 + 4);
          beta[b][i] = of(r[b], i) == -INFINITY ? 0.f : ex2_approx(of(r[b], i) - R);
        }
      // two neighbouring columns of a row per thread
      constexpr int kThreads = L::kWarps * 32, kPairs = kRows * L::kJoinCols / 2, kUPer = L::kJoinCols / 16;
#pragma unroll
      for (int c = 0; c < WIDTH / L::kJoinCols; ++c) {
#pragma unroll
        for (int u = 0; u < kUPer; ++u)
#pragma unroll
          for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              st_shared_f32(join + ((warp * kRows + 8 * b + 2 * t4 + (e & 1)) * L::kJoinPitch + 16 * u + gid + 4 * (e & 2)) * 4,
                            of(o[c * kUPer + u][b][e >> 1], e & 1) * beta[b][e & 1]);
        __syncthreads();
        for (int i = threadIdx.x; i < kPairs; i += kThreads) {
          const int row = i / (L::kJoinCols / 2), col = 2 * (i % (L::kJoinCols / 2));
          float x = 0.f, y = 0.f;
          for (int w = 0; w < L::kWarps; ++w) {
            const uint32_t from = join + ((w * kRows + row) * L::kJoinPitch + col) * 4;
            x += ld_shared_f32(from), y += ld_shared_f32(from + 4);
          }
          const int ch = L::kJoinCols * c + col;
          if (cluster > 1) {
            st_shared_f32(sb + (row * WIDTH + ch) * 4, x), st_shared_f32(sb + (row * WIDTH + ch) * 4 + 4, y);
          } else if (!whole) {
            *reinterpret_cast<float2*>(part + row * WIDTH + ch) = make_float2(x, y);
          } else if (ch < p.c.D && live(row)) {
            const float w = ld_shared_f32(stat + row * 12 + 8);
            const bool none = ld_shared_f32(stat + row * 12) == -INFINITY;
            *reinterpret_cast<uint32_t*>(p.out + row_place(p, cs.b, h, tile_row + row) * p.c.D + ch) =
                pack_16bit(p.f16, none ? 0.f : x * w, none ? 0.f : y * w);
          }
        }
        __syncthreads();
      }
      if (cluster > 1) {
        // the CTAs' sums, now at the front of each one's ring (whose copies have
        // all been used): each CTA joins every kRows · WIDTH / cluster-th pair
        cluster_barrier();
        // thread `row` first: each CTA's factor, in the place of the warps' statistics
        static_assert((kMaxCluster + 1) * 4 <= L::kWarps * 12, "a row's factors must fit its statistics");
        if (threadIdx.x < kRows) {
          const int row = threadIdx.x;
          float mk[kMaxCluster], f[kMaxCluster], M = -INFINITY, S = 0.f;
#pragma unroll
          for (int k = 0; k < kMaxCluster; ++k) {
            mk[k] = k < cluster ? ld_cluster_f32(sb + kSumStat + row * 12, k) : -INFINITY;
            f[k] = k < cluster ? ld_cluster_f32(sb + kSumStat + row * 12 + 4, k) : 0.f;
            M = fmaxf(M, mk[k]);
          }
#pragma unroll
          for (int k = 0; k < kMaxCluster; ++k) {
            if (mk[k] != -INFINITY) S += ld_cluster_f32(sb + kSumStat + row * 12 + 8, k) * ex2_approx(mk[k] - M);
            f[k] = mk[k] == -INFINITY ? 0.f : ex2_approx(f[k] - M - kPShift);
          }
#pragma unroll
          for (int k = 0; k < kMaxCluster; ++k) st_shared_f32(stat + (k * kRows + row) * 4, f[k]);
          st_shared_f32(stat + (kMaxCluster * kRows + row) * 4, M == -INFINITY ? 0.f : 1.f / S);
          if (rank == 0 && live(row)) p.lse[row_place(p, cs.b, h, tile_row + row)] = row_lse(M, S);
        }
        __syncthreads();
        for (int i = rank * kThreads + threadIdx.x; i < kRows * WIDTH / 2; i += cluster * kThreads) {
          const int row = i / (WIDTH / 2), ch = 2 * (i % (WIDTH / 2));
          if (ch >= p.c.D || !live(row)) continue;
          float2 v[kMaxCluster];
#pragma unroll
          for (int k = 0; k < kMaxCluster; ++k)
            v[k] = k < cluster ? ld_cluster_f32x2(sb + (row * WIDTH + ch) * 4, k) : make_float2(0.f, 0.f);
          float x = 0.f, y = 0.f;
#pragma unroll
          for (int k = 0; k < kMaxCluster; ++k) {
            // 0 for a CTA without keys, whose sums are 0, or far below: a NaN there stays
            const float f = ld_shared_f32(stat + (k * kRows + row) * 4);
            x += v[k].x * f, y += v[k].y * f;
          }
          const float inv = ld_shared_f32(stat + (kMaxCluster * kRows + row) * 4);
          *reinterpret_cast<uint32_t*>(p.out + row_place(p, cs.b, h, tile_row + row) * p.c.D + ch) =
              pack_16bit(p.f16, x * inv, y * inv);
        }
        cluster_barrier();  // no CTA ends while another reads its memory
      }
    }
    seg_at = seg_end;
  } while (seg_at < end);

  // after a wait that ran out: the copies still in flight land before the CTA
  // gives its shared memory back
  if (lane == 0)
    for (; used < issued; ++used) {
      wait_drain(bars + 8 * u_slot, u_parity, kDrainNs);
      if (++u_slot == L::kSlots) u_slot = 0, u_parity ^= 1;
    }
}

// Joins the parts of a segment that several workers shared.  CTA: a segment of
// the line and 32 columns; a thread takes 4 columns of a row.
constexpr int kJoinThreads = 64;

template <int WIDTH, int NT>
__global__ void __launch_bounds__(kJoinThreads * NT) cache_join_kernel(const __grid_constant__ CacheFwdParams p) {
  constexpr int kRows = 8 * NT;
  const int hr = p.c.heads * p.row_tiles;
  const int b = blockIdx.x / hr, x = blockIdx.x % hr;
  int len, n;
  load_seq(p.s, p.c, b, false, &len, &n);
  // every CTA waits, also one without work: this grid's end means the parts'
  // kernel has ended too.  lens, fresh were there before that kernel began.
  wait_for_previous();
  launch_dependents();
  const int at = p.line[b], units = (p.line[b + 1] - at) / hr, total = p.line[p.s.batch];
  if (units == 0) return;
  const int nc = units - p.lead, per = units_per_worker(p, total), first = at + x * units + p.lead;
  const int w0 = first / per, w1 = (first + nc - 1) / per;
  if (w0 == w1) return;  // one worker had it all
  const int h = x / p.row_tiles, tile_row = (x % p.row_tiles) * kRows;
  const int r = threadIdx.x / 8, col = blockIdx.y * 32 + 4 * (threadIdx.x % 8);
  if (tile_row + r >= p.G * p.s.T || (tile_row + r) % p.s.T >= n) return;
  auto part = [&](int w) { return p.part + (2ll * w + (w == w0 ? 1 : 0)) * kCachePartFloats<WIDTH, NT>; };
  float M = -INFINITY;
  for (int w = w0; w <= w1; ++w) M = fmaxf(M, part(w)[kRows * WIDTH + r]);
  float S = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M != -INFINITY) {
    for (int w = w0; w <= w1; ++w) {
      const float* q = part(w);
      const float m = q[kRows * WIDTH + r];
      if (m == -INFINITY) continue;
      S += q[kRows * WIDTH + 2 * kRows + r] * ex2_approx(m - M);
      const float f = ex2_approx(q[kRows * WIDTH + kRows + r] - M - kPShift);
      const float4 v = *reinterpret_cast<const float4*>(q + r * WIDTH + col);
      acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
    }
    acc.x /= S, acc.y /= S, acc.z /= S, acc.w /= S;
  }
  const int64_t row = row_place(p, b, h, tile_row + r);
  if (col < p.c.D)
    *reinterpret_cast<uint2*>(p.out + row * p.c.D + col) =
        make_uint2(pack_16bit(p.f16, acc.x, acc.y), pack_16bit(p.f16, acc.z, acc.w));
  if (col == 0) p.lse[row] = row_lse(M, S);
}

// mass[key] += Σ over the rows that may see the key of 2^(t - lse): one thread a
// key, whose scores lie side by side; the rows' logsumexps and last positions wait
// in shared memory.  Which rows count is a comparison of positions, not a logsumexp
// of +inf: rows that are not there were scored too, and inf - inf and NaN - inf
// would reach every key.
constexpr int kMassThreads = 128, kMassRows = 256, kMassLoads = 4;

__global__ void __launch_bounds__(kMassThreads) cache_mass_kernel(const __grid_constant__ CacheFwdParams p) {
  __shared__ __align__(16) float z[kMassRows];   // log2 units
  __shared__ __align__(16) int last[kMassRows];  // position; -1: a row that is not there or sees no key
  const int h = blockIdx.y, b = blockIdx.z;
  int len, n;
  const int nc = seq_chunks(p, b, false, &len, &n);
  const int key = blockIdx.x * kMassThreads + threadIdx.x;
  const int64_t bh = static_cast<int64_t>(b) * p.c.heads + h;
  int pos = key < nc * kCacheChunk ? key : kFar;
  if (p.list != nullptr && pos != kFar) {
    const int e = key >> p.c.log2_page;
    const int* l = p.list + bh * p.listed;
    const int i = e < p.listed ? l[e] : -1;
    pos = i < 0 || i >= p.s.width || !follows(l, e) ? kFar : (i << p.c.log2_page) + (key & (p.c.page - 1));
  }
  const bool mine = pos < len;
  float* mass = p.mass + bh * (static_cast<int64_t>(p.s.width) << p.c.log2_page) + pos;
  const float before = mine ? *mass : 0.f;
  wait_for_previous();
  if (blockIdx.x * kMassThreads >= nc * kCacheChunk) return;
  const int rows = p.G * p.s.T;
  const float* s = p.scores + (bh * p.score_cols + key) * p.score_rows;
  float sum = 0.f;
  for (int r0 = 0; r0 < rows; r0 += kMassRows) {
    __syncthreads();
    for (int r = threadIdx.x; r < kMassRows; r += kMassThreads) {
      const int i = (r0 + r) % p.s.T;
      const float w = r0 + r < rows && i < n ? p.lse[bh * rows + r0 + r] : -INFINITY;
      z[r] = w * kLog2e;
      last[r] = w == -INFINITY ? -1 : len - n + i;
    }
    __syncthreads();
    const int stop = mine ? min(kMassRows, p.score_rows - r0) : 0;  // score rows are padded to tiles of 8
    for (int r = 0; r < stop; r += 4 * kMassLoads) {
      // ordinary loads, since the scores are still being written when this kernel
      // begins; all in flight at once (one after the other: drafts 61 us, so 51 us)
      float4 t[kMassLoads];
#pragma unroll
      for (int j = 0; j < kMassLoads; ++j)
        if (r + 4 * j < stop) t[j] = *reinterpret_cast<const float4*>(s + r0 + r + 4 * j);
#pragma unroll
      for (int j = 0; j < kMassLoads; ++j) {
        if (r + 4 * j >= stop) break;
        const float4 w = *reinterpret_cast<const float4*>(z + r + 4 * j);
        const int4 e = *reinterpret_cast<const int4*>(last + r + 4 * j);
        auto weight = [&](float x, float ref, int to) { return pos <= to ? ex2_approx(x - ref) : 0.f; };
        sum += (weight(t[j].x, w.x, e.x) + weight(t[j].y, w.y, e.y)) +
               (weight(t[j].z, w.z, e.z) + weight(t[j].w, w.w, e.w));
      }
    }
  }
  if (mine) *mass = before + sum;
}

template <int WIDTH, int WORKER, int NT, bool PACKED>
cudaError_t launch_fwd(const CacheFwdParams& p, int dev, int ctas, cudaStream_t stream) {
  using L = CacheFwdLayout<WIDTH, WORKER, NT, PACKED>;
  auto kern = cache_fwd_kernel<WIDTH, WORKER, NT, PACKED>;
  static std::atomic<uint64_t> ready{0};  // devices (bits) whose copy of the kernel has its shared memory granted
  cudaError_t e = cudaSuccess;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(L::kWarps * 32);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return e;
  if (p.cluster == 0)
    e = launch_after(cache_join_kernel<WIDTH, NT>, dim3(p.s.batch * p.c.heads * p.row_tiles, WIDTH / 32),
                     kJoinThreads * NT, stream, p);
  if (e != cudaSuccess || p.mass == nullptr) return e;
  return launch_after(cache_mass_kernel, dim3((p.score_cols + kMassThreads - 1) / kMassThreads, p.c.heads, p.s.batch),
                      kMassThreads, stream, p);
}

template <int WIDTH, bool PACKED>
cudaError_t launch_width(const CacheFwdParams& p, bool warp_workers, int tiles, int dev, int ctas,
                         cudaStream_t stream) {
  auto go = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    if constexpr (NT <= kCacheWarpWorkerTiles)
      if (warp_workers) return launch_fwd<WIDTH, 1, NT, PACKED>(p, dev, ctas, stream);
    return launch_fwd<WIDTH, kCacheWarps<WIDTH, NT>, NT, PACKED>(p, dev, ctas, stream);
  };
  switch (tiles) {
    case 1: return go(std::integral_constant<int, 1>());
    case 2: return go(std::integral_constant<int, 2>());
  }
  if constexpr (WIDTH <= 64) {
    if (tiles == 3) return go(std::integral_constant<int, 3>());
    if (tiles == 4) return go(std::integral_constant<int, 4>());
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int cache_fwd_clusters(int dev, int size) {
  if (size <= 1 || size > kMaxCluster) return 0;
  constexpr int kSizes = kMaxCluster + 1;
  static std::atomic<int> known[64 * kSizes];  // one more than the answer; 0: not asked yet
  std::atomic<int>& slot = known[dev * kSizes + size];
  int n = slot.load(std::memory_order_relaxed) - 1;
  if (n >= 0) return n;
  // any of the kernels: each fills an SM with one CTA
  using L = CacheFwdLayout<128, kCacheWarps<128, 1>, 1, false>;
  auto kern = cache_fwd_kernel<128, kCacheWarps<128, 1>, 1, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(L::kWarps * 32);
  cfg.dynamicSmemBytes = L::kAlloc;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  slot.store(n + 1, std::memory_order_relaxed);
  return n;
}

cudaError_t cache_fwd_launch(const CacheFwdParams& p, int width, int tiles, bool warp_workers, int dev, int ctas,
                             cudaStream_t stream) {
  const bool packed = p.c.pitch / 16 % 2 != 0;
  auto go = [&](auto w) {
    constexpr int W = decltype(w)::value;
    return packed ? launch_width<W, true>(p, warp_workers, tiles, dev, ctas, stream)
                  : launch_width<W, false>(p, warp_workers, tiles, dev, ctas, stream);
  };
  switch (width) {
    case 64: return go(std::integral_constant<int, 64>());
    case 128: return go(std::integral_constant<int, 128>());
    case 256: return go(std::integral_constant<int, 256>());
  }
  return cudaErrorInvalidValue;
}

}  // namespace ea
