// cross_common.cuh — device helpers of the kernels' cross-attention forms, whose
// keys are another sequence's: units of work, lengths, and what lies behind them.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attn_bwd.h"
#include "attn_fwd.h"
#include "ptx.cuh"

namespace ea {
namespace {

enum : int { kChkCrossLen = 0x7101, kChkCrossPart = 0x7102 };

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
// count.  A run without tiles (no keys, or more runs than tiles) gets one of which no
// key is there, so that every unit has a step; *len is 0 then.
__device__ __forceinline__ void cross_run(int part, int parts, int tile, int* len, int* j0, int* n) {
  const int tiles = (*len + tile - 1) / tile;
  const int each = tiles / parts, more = tiles - each * parts;
  *j0 = part * each + min(part, more);
  *n = each + (part < more ? 1 : 0);
  if (*n == 0) *len = 0, *j0 = 0, *n = 1;
}

template <int MASK, int BN>
__device__ __forceinline__ FwdUnit fwd_unit(const Fwd1QParams& p, int x) {
  FwdUnit u;
  fwd_tile<MASK>(p, x, &u.bh, &u.i);
  if constexpr (MASK == kMaskCross) {
    u.len = cross_len(p.lens, u.bh / p.heads, p.Sk, p.status);
    cross_run(x % p.n_split, p.n_split, BN, &u.len, &u.j0, &u.nkv);
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

// dq: runs of K/V tiles of KEYS keys.
template <int KEYS>
__device__ __forceinline__ BwdUnit cross_dq_unit(const BwdParams& p, int x) {
  BwdUnit u;
  const int y = x / p.q_split;
  u.part = x - y * p.q_split;
  u.bh = y / p.n_qt;
  u.tile = y - u.bh * p.n_qt;
  u.len = cross_len(p.lens, u.bh / p.heads, p.Sk, p.status);
  cross_run(u.part, p.q_split, KEYS, &u.len, &u.first, &u.n);
  return u;
}

// dk and dv: runs of Q tiles of ROWS queries, at most as many as there are.
template <int ROWS>
__device__ __forceinline__ BwdUnit cross_kv_unit(const BwdParams& p, int x) {
  BwdUnit u;
  const int y = x / p.kv_split;
  u.part = x - y * p.kv_split;
  u.bh = y / p.n_kt;
  u.tile = y - u.bh * p.n_kt;
  u.len = cross_len(p.lens, u.bh / p.heads, p.Sk, p.status);
  int rows = p.S;
  cross_run(u.part, p.kv_split, ROWS, &rows, &u.first, &u.n);
  return u;
}

// The gradient of 128 keys that are not there: dk = dv = 0 (whole CTA of `threads`).
__device__ __forceinline__ void cross_no_keys(uint16_t* dk, uint16_t* dv, int64_t row0, int rows,
                                              int d_cols, int first_col, int cols, int threads) {
  cols = min(cols, d_cols - first_col);
  if (cols <= 0) return;
  const int units = cols / 8;
  for (int c = threadIdx.x; c < rows * units; c += threads) {
    const int64_t at = (row0 + c / units) * d_cols + first_col + (c % units) * 8;
    *reinterpret_cast<uint4*>(dk + at) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(dv + at) = make_uint4(0u, 0u, 0u, 0u);
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

// 32 columns of this thread's row of an fp32 TMEM accumulator, times mul, to
// columns x0 .. of the row at `to`.  Call with the full warp.
__device__ __forceinline__ void store_part(uint32_t taddr, float* to, int x0, float mul, bool valid,
                                           const DbgBounds& dbb, int bh, int row, int site) {
  uint32_t o[32];
  tmem_ld_32x32b_x32(taddr, o);
  tmem_ld_wait();
  reg_fence(o);
  if (!valid) return;
#pragma unroll
  for (int e = 0; e < 32; e += 4)
    if (x0 + e < dbb.cols && dbg_row(dbb, bh, row, x0 + e, 4, site))
      *reinterpret_cast<float4*>(to + x0 + e) =
          make_float4(__uint_as_float(o[e]) * mul, __uint_as_float(o[e + 1]) * mul,
                      __uint_as_float(o[e + 2]) * mul, __uint_as_float(o[e + 3]) * mul);
}

}  // namespace
}  // namespace ea
