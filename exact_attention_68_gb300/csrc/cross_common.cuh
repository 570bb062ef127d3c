// cross_common.cuh — device helpers of the kernels' cross-attention forms, whose
// keys are another sequence's: units of work, lengths, and what lies behind them.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attn_bwd.h"
#include "attn_fwd.h"
#include "cross_runs.cuh"
#include "ptx.cuh"

namespace ea {
namespace {

enum : int { kChkCrossLen = 0x5701 };

// Keys of sequence b: lens[b], or all Sk.  A length outside [0, Sk] is reported
// (every build) and brought to the nearer end.
__device__ __forceinline__ int cross_len(const int* lens, int b, int Sk, int* status) {
  if (lens == nullptr) return Sk;
  const int n = __ldg(lens + b);
  if (n >= 0 && n <= Sk) return n;
  dbg_fail(status, kChkCrossLen);
  return n < 0 ? 0 : Sk;
}

// What one unit of the forward does: Q tile i of slice bh with nkv K/V tiles from
// j0 on, of whose keys those below len are there.
struct FwdUnit {
  int bh, i, j0, nkv, len;
};

// Slice and Q tile of CTA x.  Cross-attention's runs of one tile are neighbours, and
// a slice's tiles follow one another, so that what is in flight shares K and V in L2.
template <int MASK>
__device__ __forceinline__ void fwd_tile(const Fwd1QParams& p, int x, int* bh, int* i) {
  if constexpr (MASK == kMaskCross) {
    const int y = x / p.n_split;
    *bh = y / p.n_qt;
    *i = y - *bh * p.n_qt;
  } else {
    schedule_unit(p.sched, x, bh, i);
  }
}

// Run `part` of `parts` of a sequence's tiles, which are dealt evenly: first tile and
// count.  A run without tiles (no keys, or more runs than tiles) gets, with
// `some`, one of which no key is there, so that every unit has a step; *len is 0 then.
__device__ __forceinline__ void cross_run(int part, int parts, int tile, int* len, int* j0, int* n,
                                          bool some = true) {
  const int tiles = (*len + tile - 1) / tile;
  const int each = tiles / parts, more = tiles - each * parts;
  *j0 = part * each + min(part, more);
  *n = each + (part < more ? 1 : 0);
  if (*n == 0) *len = 0, *j0 = 0, *n = some ? 1 : 0;
}

// SOME: every unit has a step (cross_run).
template <int MASK, int BN, bool SOME = true>
__device__ __forceinline__ FwdUnit fwd_unit(const Fwd1QParams& p, int x) {
  FwdUnit u;
  fwd_tile<MASK>(p, x, &u.bh, &u.i);
  if constexpr (MASK == kMaskCross) {
    u.len = cross_len(p.lens, u.bh / p.heads, p.Sk, p.status);
    cross_run(x % p.n_split, p.n_split, BN, &u.len, &u.j0, &u.nkv, SOME);
  } else {
    const int n = MASK == kMaskCausal ? (u.i + 1) * (kBlockM / BN) : p.n_kt;
    u.nkv = n < p.n_kt ? n : p.n_kt;
    u.j0 = 0;
    u.len = p.S;
  }
  return u;
}

// What one unit of a gradient kernel does: tile `tile` of slice bh (of queries for
// dq, of keys for dk and dv) with n tiles of the others from first on; keys below
// len are there.  part: which run of the others, of those that are summed later.
struct BwdUnit {
  int bh, tile, first, n, len, part;
};

// dq: runs of K/V tiles of KEYS keys.  order (may be null): the sequences in the order
// in which their units are numbered.
template <int KEYS>
__device__ __forceinline__ BwdUnit cross_dq_unit(const BwdParams& p, int x, const uint8_t* order = nullptr) {
  BwdUnit u;
  const int y = x / p.q_split;
  u.part = x - y * p.q_split;
  u.bh = y / p.n_qt;
  u.tile = y - u.bh * p.n_qt;
  if (order != nullptr) {
    const int b = u.bh / p.heads;
    u.bh += (order[b] - b) * p.heads;
  }
  u.len = cross_len(p.lens, u.bh / p.heads, p.Sk, p.status);
  cross_run(u.part, p.q_split, KEYS, &u.len, &u.first, &u.n);
  return u;
}

// The sequences by falling length (whole warp, batch <= 32): a sequence's rank is the
// number of those before it.
constexpr int kMaxOrder = 32;
__device__ __forceinline__ void order_by_length(const BwdParams& p, int lane, uint8_t* order) {
  const int batch = p.BH / p.heads;
  const int len = lane < batch ? min(max(__ldg(p.lens + lane), 0), p.Sk) : -1;
  int rank = 0;
  for (int b = 0; b < batch; ++b) {
    const int other = __shfl_sync(0xffffffffu, len, b);
    rank += other > len || (other == len && b < lane) ? 1 : 0;
  }
  if (lane < batch) order[rank] = static_cast<uint8_t>(lane);
}

// Unit `round` of CTA cta: the units' numbers run to and fro over the CTAs, so that
// who had the longest of one round has the shortest of the next.
__device__ __forceinline__ int to_and_fro(int round, int cta, int ctas) {
  return round & 1 ? (round + 1) * ctas - 1 - cta : round * ctas + cta;
}

// dk and dv: runs of Q tiles of ROWS queries, at most as many as there are, of every
// key tile that has keys.  A CTA's units x, x + gridDim.x, ... are found one after the
// other, counting on from the sequence the last one was in.
struct KvWalk {
  int x, b, before;  // unit asked for; a sequence, and the units of those before it
  int runs;          // of a key tile's Q tiles
};
constexpr int kWalkBy = 8;
__device__ __forceinline__ KvWalk kv_walk(int x, int runs) { return {x, 0, 0, runs}; }
// The unit the walk is at; false: none left.  MANY: by kWalkBy sequences at a time
// where it may go that far.
template <int ROWS, bool MANY>
__device__ __forceinline__ bool cross_kv_unit(const BwdParams& p, KvWalk& w, BwdUnit* u) {
  const int batch = p.BH / p.heads;
  int tiles = 0;
  for (;; ++w.b) {
    if (w.b >= batch) return false;
    u->len = cross_len(p.lens, w.b, p.Sk, p.status);
    tiles = (u->len + 127) / 128;
    const int units = p.heads * tiles * w.runs;
    if (w.x - w.before < units) break;
    w.before += units;
    if constexpr (MANY) {
      // Eight sequences further at least, whatever their lengths: these are asked for
      // together.  A length out of range is reported where its queries are.
      const int each = p.heads * w.runs;
      while (w.x - w.before >= each * kWalkBy * p.n_kt && w.b + kWalkBy < batch) {
        int sum = 0;
#pragma unroll
        for (int i = 1; i <= kWalkBy; ++i) sum += (min(max(__ldg(p.lens + w.b + i), 0), p.Sk) + 127) / 128;
        w.before += each * sum;
        w.b += kWalkBy;
      }
    }
  }
  const int y = w.x - w.before, z = y / w.runs;
  u->part = y - z * w.runs;
  const int h = z / tiles;
  u->bh = w.b * p.heads + h;
  u->tile = z - h * tiles;
  int rows = p.S;
  cross_run(u->part, w.runs, ROWS, &rows, &u->first, &u->n);
  return true;
}

// Zeroes dk and dv of the key tiles without keys (columns first_col .. +cols), dealt to
// the grid's CTAs: `threads` threads of each, tid this one's number.
__device__ __forceinline__ void cross_zero_tiles(const BwdParams& p, int cta, int ctas, int tid, int threads,
                                                 int first_col, int cols) {
  cols = min(cols, p.d_cols - first_col);
  if (p.lens == nullptr || cols <= 0) return;
  const int units = cols / 8;
  for (int x = cta; x < p.BH * p.n_kt; x += ctas) {
    const int bh = x / p.n_kt, j = x - bh * p.n_kt;
    if (j * 128 < cross_len(p.lens, bh / p.heads, p.Sk, p.status)) continue;
    const int64_t row0 = (int64_t)bh * p.Sk + j * 128;
    for (int c = tid; c < min(128, p.Sk - j * 128) * units; c += threads) {
      const int64_t at = (row0 + c / units) * p.d_cols + first_col + (c % units) * 8;
      *reinterpret_cast<uint4*>(p.dk + at) = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(p.dv + at) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

// The bounds of key rows for the debug checks.
template <int MASK>
__device__ __forceinline__ DbgBounds key_bounds(DbgBounds d, int Sk) {
  if (MASK == kMaskCross) d.rows = Sk;
  return d;
}

// Zeroes the rows from `live` on of a tile of `rows` rows x CHUNKS 64-column blocks
// (whole warp, after the tile has landed, before a product reads it).  What a
// padded batch holds behind a sequence's end may be NaN or infinite, and the
// weight 0 it gets would not silence that in a product.  Rows past the tensor's
// end are zero already (`padded` false).
template <int CHUNKS>
__device__ __forceinline__ void clear_tail(uint32_t tile, int rows, int live, bool padded, int lane,
                                           const DbgBounds& dbb, int site) {
  if (!padded || live >= rows) return;
  const int from = max(live, 0) * 128, to = rows * 128;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c)
    for (int at = from + lane * 16; at < to; at += 32 * 16) {
      const uint32_t addr = tile + c * to + at;
      if (dbg_smem(dbb, addr, 16, 16, site)) st_shared_v4(addr, 0u, 0u, 0u, 0u);
    }
  fence_proxy_async_smem();
  __syncwarp();
}

// P enters dv's product times this, and dv is divided by it: fp16 holds values below
// 2^-14 in steps of 2^-24 only, and weights are as small as one over the keys.
template <bool F16>
constexpr float kPTimes = F16 ? 4096.f : 1.f;

// 32 columns of this thread's row of an fp32 TMEM accumulator, times mul, to
// columns x0 .. of the row at `to` (none: zeros).  Call with the full warp.
__device__ __forceinline__ void store_part(uint32_t taddr, float* to, int x0, float mul, bool valid,
                                           const DbgBounds& dbb, int bh, int row, int site,
                                           bool none = false) {
  uint32_t o[32];
  __syncwarp();  // the last call's stores were by row
  tmem_ld_32x32b_x32(taddr, o);
  tmem_ld_wait();
  reg_fence(o);
  if (!valid) return;
  if (none) {
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = 0u;
  }
#pragma unroll
  for (int e = 0; e < 32; e += 4)
    if (x0 + e < dbb.cols && dbg_row(dbb, bh, row, x0 + e, 4, site))
      *reinterpret_cast<float4*>(to + x0 + e) =
          make_float4(__uint_as_float(o[e]) * mul, __uint_as_float(o[e + 1]) * mul,
                      __uint_as_float(o[e + 2]) * mul, __uint_as_float(o[e + 3]) * mul);
}

}  // namespace
}  // namespace ea
