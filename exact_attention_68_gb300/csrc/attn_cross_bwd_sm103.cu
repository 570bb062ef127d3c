// attn_cross_bwd_sm103.cu — gradient of cross-attention on GB300 (sm_103a), head
// dimensions up to 128 (above: attn_bwd256_sm103.cu).  The formulas are
// attn_bwd_sm103.cu's, without a causal mask and with lens[b] keys:
//
//   dS = P ⊙ (dP − delta),   dq = scale·dS·k,   dk = scale·dSᵀ·q,   dv = Pᵀ·dout,
//   P = exp(scale·q·kᵀ − lse),  dP = dout·vᵀ,  delta_i = rowsum(dout ⊙ out)_i.
//
// As there a dq kernel owns 128 query rows and walks the keys, and a dk/dv kernel
// owns 128 key rows and walks the queries, so that no sum depends on scheduling; the
// tiles, the split of the elementwise work over two warpgroups and the order of
// the products are the same.  Why other kernels: here a tile may meet very few of
// the others (a prompt of 300 tokens is three), and a CTA a tile then spends most
// of its time on its start and its end.  With kernels of that kind a tile of three
// steps took 13.5 us, of which the steps are 4.  So:
//
//   One CTA an SM, which takes units (a tile, or a run of its steps) one after the
//   other.  The rings run on: a unit's own rows (Q and dO, or K and V) come through
//   them ahead of its steps, and the MMA warp copies them into tensor memory
//   (tcgen05.cp) as soon as the last unit's products have been issued, so that the
//   next unit's first scores are being computed while this one's sums are stored.
//   Only the first product into the sums waits for them to have been read.
//   Sums are staged in the ring's next place and stored with TMA.
//
// Bound by: where a tile meets few of the others, the hand-over from unit to unit (dq: 6.5
// us a unit of two steps on average); else the exchange between the elementwise warps
// and the warp that issues products, and at 64 channels that warp itself.
// Measured on a GB300, both kernels and the joins, calls in a graph: 2 x 16 heads,
// 4096 queries, 300 and 100 keys of 128 channels 83.9 us (dq 44, dk and dv 38); 8 x 16
// heads, 500 queries, 300 to 1500 keys of 64 channels 94.6 us; 2 x 16 heads on 4 of
// keys, 4000 queries, 6000 keys of 128 channels 936 us, 1050 TFLOP/s of the formula's
// five products.  One CTA a tile: 156, 131 and 1022 us.
//
// Roles as there: warps 0-7 elementwise, warp 8 issues tcgen05.mma, warp 9 feeds the
// rings.  The dk/dv kernel is set up on each SM as the dq kernel, whose delta it
// reads, leaves it.  All waits between warps are bounded mbarrier waits: a role that gave up
// does not come back, and nobody waits for it for ever.
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_bwd.h"
#include "bwd_common.cuh"
#include "cross_common.cuh"
#include "launch_after.cuh"
#include "ptx.cuh"
#include "umma.cuh"

namespace ea {
namespace {

constexpr float kLog2eX = 1.4426950408889634f;
constexpr uint64_t kDrainLimitNsX = 1000000000ull;
constexpr int kRowsX = 128;             // of a tile
constexpr int kBlockX = kRowsX * 128;   // one 64-column, 128-row swizzled block
constexpr uint32_t kTmemColsX = 512;

enum : int {
  kSiteXqProd = 0x7100, kSiteXqMmaQ = 0x7200, kSiteXqMmaKV = 0x7300, kSiteXqMmaP = 0x7400,
  kSiteXqMmaFree = 0x7500, kSiteXqElemS = 0x7600, kSiteXqElemO = 0x7700, kSiteXqElemD = 0x7800,
  kSiteXkProd = 0x7900, kSiteXkMmaKV = 0x7a00, kSiteXkMmaQ = 0x7b00, kSiteXkMmaP = 0x7c00,
  kSiteXkMmaFree = 0x7d00, kSiteXkElemS = 0x7e00, kSiteXkElemO = 0x7f00
};
// debug-check sites (-DATTN_DEBUG)
enum : int { kChkXRow = 0x5601, kChkXSTmem, kChkXStat, kChkXLoadA, kChkXLoadB, kChkXMmaA, kChkXMmaB };

// A 128-row K-major tile of D columns in shared memory (its descriptor d) into D/2
// columns of tensor memory from `to` on, two 16-bit values a column.
template <int D>
__device__ __forceinline__ void copy_tile(uint32_t to, uint64_t d) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    tmem_cp_128x256b(to + kk * 8, d + (((kk >> 2) * kBlockX + (kk & 3) * 32) >> 4));
}

// A read-only load that stays where it is written: asked for here, used behind waits.
__device__ __forceinline__ float ldg_now(const float* ptr) {
  float r;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(r) : "l"(ptr));
  return r;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
  return r;
}

// ============================================================== dq kernel
// TMEM: half h of a K/V tile (64 keys) has S in [128h, +64), dP in [128h + 64, +64);
// dQ [256, 256+D); Q [384, 384+D/2), dO [384+D/2, 384+D).

template <int D>
struct XqLayout {
  static constexpr int kTile = kRowsX * D * 2;
  static constexpr int kChunks = D / 64;
  // Of a unit the K ring carries Q, then the K tiles, then a place for dQ on its way
  // out; the V ring dO, out, then the V tiles.
  static constexpr int kKStages = D == 128 ? 3 : 6;
  static constexpr int kVStages = D == 128 ? 4 : 6;
  static constexpr int kKOff = 0;
  static constexpr int kVOff = kKOff + kKStages * kTile;
  static constexpr int kPartOff = kVOff + kVStages * kTile;  // float [2][128] delta halves
  static constexpr int kBarOff = kPartOff + 2 * kRowsX * 4;
  static constexpr int kKFull = 0;
  static constexpr int kKEmpty = kKFull + kKStages;
  static constexpr int kVFull = kKEmpty + kKStages;
  static constexpr int kVEmpty = kVFull + kVStages;
  static constexpr int kSFull = kVEmpty + kVStages;  // [2] S_h and dP_h computed
  static constexpr int kPFull = kSFull + 2;          // [2] dS_h stored (128 arrivals)
  static constexpr int kOFull = kPFull + 2;          // dQ final
  static constexpr int kOFree = kOFull + 1;          // dQ read, its place in the ring too (256 arrivals)
  static constexpr int kStat = kOFree + 1;           // a unit's delta halves written (256 arrivals)
  static constexpr int kDrain = kStat + 1;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // tmem base, abort flag
  static constexpr int kOrderOff = kMiscOff + 16;          // uint8 [kMaxOrder]
  static constexpr int kAlloc = kOrderOff + kMaxOrder + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget exceeded");
  static constexpr uint32_t kDqCol = 256, kQCol = 384, kDoCol = 384 + D / 2;
};

// ORDERED: units of long sequences first.  TWO: dS enters its product in two terms, the
// 16-bit value and what rounding to it left, which has its place behind it.
template <int D, bool F16, bool ORDERED, bool TWO>
__global__ void __launch_bounds__(kBwdThreads, 1) cross_dq_kernel(const __grid_constant__ BwdParams p) {
  using L = XqLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto bar = [sb](int idx) -> uint32_t { return sb + L::kBarOff + 8u * idx; };
  const uint32_t tmem_slot = sb + L::kMiscOff;
  const uint32_t abort_addr = sb + L::kMiscOff + 4;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const DbgBounds dbb{p.status, sb, smem_u32(smem_raw) + static_cast<uint32_t>(L::kAlloc), p.S,
                      p.d_cols, p.BH};
  const DbgBounds dbk = key_bounds<kMaskCross>(dbb, p.Sk);
  const int n_units = p.BH * p.n_qt * p.q_split;
  const int x0 = static_cast<int>(blockIdx.x), step = static_cast<int>(gridDim.x);
  const uint8_t* order = ORDERED ? smem_raw + (sb - smem_u32(smem_raw)) + L::kOrderOff : nullptr;
  BwdUnit unit0{};
  if constexpr (ORDERED) {
    if (warp == 9) order_by_length(p, lane, smem_raw + (sb - smem_u32(smem_raw)) + L::kOrderOff);
  } else {
    unit0 = cross_dq_unit<kRowsX>(p, x0);  // the grid has no more CTAs than units
  }
  // this CTA's unit `round`
  auto unit_at = [&](int round) { return ORDERED ? to_and_fro(round, x0, step) : x0 + round * step; };

  if (threadIdx.x == 0) {
    launch_dependents();
#pragma unroll
    for (int s = 0; s < L::kKStages; ++s) mbar_init(bar(L::kKFull + s), 1), mbar_init(bar(L::kKEmpty + s), 1);
#pragma unroll
    for (int s = 0; s < L::kVStages; ++s) mbar_init(bar(L::kVFull + s), 1), mbar_init(bar(L::kVEmpty + s), 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) mbar_init(bar(L::kSFull + h), 1), mbar_init(bar(L::kPFull + h), 128);
    mbar_init(bar(L::kOFull), 1);
    mbar_init(bar(L::kOFree), 256);
    mbar_init(bar(L::kStat), 256);
    mbar_init(bar(L::kDrain), 1);
    st_volatile_shared(abort_addr, 0);
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, kTmemColsX);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = static_cast<uint32_t>(ld_volatile_shared(tmem_slot));
  const WaitCtl ctl{abort_addr, p.status, p.timeout_ns};
  if constexpr (ORDERED) unit0 = cross_dq_unit<kRowsX>(p, x0, order);

  if (warp < 8) {
    // ======================= elementwise: delta, dS, dQ out =======================
    const int g = warp >> 2;  // half of every K/V tile this warpgroup takes
    const int wq = warp & 3;  // TMEM lane quarter
    const int row = wq * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem_base + lane_bits + 128 * g;
    const uint32_t tP = tS + 64;
    const float sl2 = p.scale_log2;

    BwdUnit un = unit0;
    int steps = 0;           // K/V tiles of the units before this one
    int kpos = 0, vpos = 0;  // and ring positions
    bool ok = true;
    auto lse_of = [&](const BwdUnit& u) {
      const int grow = u.tile * kRowsX + row;
      return grow < p.S && dbg_row(dbb, u.bh, grow, 0, 0, kChkXRow) ? ldg_now(p.lse + (int64_t)u.bh * p.S + grow) : 0.f;
    };
    float lse = lse_of(un);
    for (int unit = 0;; ++unit) {
      const int grow = un.tile * kRowsX + row;
      const bool valid = grow < p.S;
      const float lse2 = lse * kLog2eX;
      // delta = rowsum(dout ⊙ out), half a row a thread, from the tiles in the V ring
      const int s0 = vpos % L::kVStages, s1 = (vpos + 1) % L::kVStages;
      ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kVFull + s0), (vpos / L::kVStages) & 1, ctl, kSiteXqElemD | 1));
      if (ok) ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kVFull + s1), ((vpos + 1) / L::kVStages) & 1, ctl, kSiteXqElemD | 2));
      if (!ok) break;
      float part = 0.f;
#pragma unroll
      for (int u = 0; u < D / 16; ++u) {  // 16-byte units of the half
        const int col = g * (D / 16) + u;
        const uint32_t off = (col >> 3) * kBlockX + row * 128 + (((col & 7) ^ (row & 7)) << 4);
        if (dbg_smem(dbb, sb + L::kVOff + s0 * L::kTile + off, 16, 16, kChkXStat) &&
            dbg_smem(dbb, sb + L::kVOff + s1 * L::kTile + off, 16, 16, kChkXStat))
          part += dot8<F16>(ld_shared_v4(sb + L::kVOff + s1 * L::kTile + off), ld_shared_v4(sb + L::kVOff + s0 * L::kTile + off));
      }
      // (all have read the last unit's halves: its dQ, which has been waited for, took
      // the dS of every row)
      st_shared_f32(sb + L::kPartOff + 4 * (g * kRowsX + row), part);
      mbar_arrive(bar(L::kStat));
      ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kStat), unit & 1, ctl, kSiteXqElemD));
      if (!ok) break;
      const float delta = ld_shared_f32(sb + L::kPartOff + 4 * row) + ld_shared_f32(sb + L::kPartOff + 4 * (kRowsX + row));
      if (g == 0 && valid && un.part == 0 && dbg_row(dbb, un.bh, grow, 0, 0, kChkXRow))
        p.delta[(int64_t)un.bh * p.S + grow] = delta;
      for (int j = 0; j < un.n; ++j) {
        ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kSFull + g), (steps + j) & 1, ctl,
                                                  kSiteXqElemS | (g << 7) | (j & 0x7f)));
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t s[2][32], dp[2][32];
        if (!dbg_warp(dbg_tmem(dbb, tS, 64, warp, kChkXSTmem) && dbg_tmem(dbb, tP, 64, warp, kChkXSTmem))) {
          ok = false;
          break;
        }
        tmem_ld_32x32b_x32(tS, s[0]);
        tmem_ld_32x32b_x32(tS + 32, s[1]);
        tmem_ld_32x32b_x32(tP, dp[0]);
        tmem_ld_32x32b_x32(tP + 32, dp[1]);
        tmem_ld_wait();
        reg_fence(s[0]);
        reg_fence(s[1]);
        reg_fence(dp[0]);
        reg_fence(dp[1]);
        // key columns of this half that are there: 0 .. lim
        const int lim = un.len - 1 - ((un.first + j) * kRowsX + 64 * g);
        uint32_t pk[32], rest[TWO ? 32 : 1];
        // with or without keys that are not: most steps pay for no comparison.  (A row
        // behind the last query is zero in Q and dO and never stored.)
        auto weigh = [&](auto masked) {
          constexpr bool kMasked = decltype(masked)::value;
#pragma unroll
          for (int e2 = 0; e2 < 32; ++e2) {
            const int h = e2 >> 4;
            const int e = (2 * e2) & 31;
            const float2 x2 = __ffma2_rn(make_float2(__uint_as_float(s[h][e]), __uint_as_float(s[h][e + 1])),
                                         make_float2(sl2, sl2), make_float2(-lse2, -lse2));
            const float2 dd = __fadd2_rn(make_float2(__uint_as_float(dp[h][e]), __uint_as_float(dp[h][e + 1])),
                                         make_float2(-delta, -delta));
            float2 ds = __fmul2_rn(make_float2(ex2_approx(x2.x), ex2_approx(x2.y)), dd);
            if (kMasked) {  // such a key may make S and dP anything
              if (2 * e2 > lim) ds.x = 0.f;
              if (2 * e2 + 1 > lim) ds.y = 0.f;
            }
            pk[e2] = pack_x2<F16>(ds.x, ds.y);
            if constexpr (TWO) rest[e2] = rest_x2<F16>(ds, pk[e2]);
          }
        };
        if (lim < 63) weigh(std::true_type{});  // the same in every thread of the warpgroup
        else weigh(std::false_type{});
        tmem_st_32x32b_x32(tS, pk);
        if constexpr (TWO) tmem_st_32x32b_x32(tS + 32, rest);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(bar(L::kPFull + g));
      }
      if (!ok) break;
      steps += un.n;
      kpos += 1 + un.n;
      vpos += 2 + un.n;
      const int x = unit_at(unit + 1);
      const bool more = x < n_units;
      const BwdUnit nu = more ? cross_dq_unit<kRowsX>(p, x, order) : un;
      if (more) lse = lse_of(nu);

      // dQ · scale → 16-bit → the ring's next place, swizzled → TMA store
      const int st = kpos % L::kKStages;
      ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kKFull + st), (kpos / L::kKStages) & 1, ctl, kSiteXqElemO | 0x80));
      if (ok) ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kOFull), unit & 1, ctl, kSiteXqElemO));
      if (!ok) break;
      ++kpos;
      tc_fence_after_sync();
      const uint32_t tQ = tmem_base + lane_bits + L::kDqCol;
      if (p.q_split > 1) {  // this run's sum, to be added to the others
        const int64_t at = (((int64_t)un.part * p.BH + un.bh) * p.S + grow) * p.d_cols;
#pragma unroll 1
        for (int c = g * (D / 64); c < (g + 1) * (D / 64); ++c)
          store_part(tQ + c * 32, p.part_dq + at, c * 32, 1.f, valid, dbb, un.bh, grow, kChkStore);
      } else {
        for (int c = g; c < L::kChunks; c += 2)
          store_chunk<F16>(tQ + c * 64, sb + L::kKOff + st * L::kTile + c * kBlockX, row, p.scale, &p.tm_dq, c * 64,
                           un.tile * kRowsX, un.bh, wq, lane, dbb);
        if (lane == 0) {
          tma_store_commit();
          tma_store_wait_read();
        }
        __syncwarp();
      }
      tc_fence_before_sync();
      mbar_arrive(bar(L::kOFree));
      if (!more) break;
      un = nu;
    }
    if (lane == 0) tma_store_wait_all();
    tc_fence_before_sync();
  } else if (warp == 9) {
    // ======================= TMA producer: Q and dO, then K and V tiles =======================
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_q);
      tma_prefetch_desc(&p.tm_do);
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
      tma_prefetch_desc(&p.tm_dq);
      tma_prefetch_desc(&p.tm_out);
      const uint64_t pol_kv = l2_policy_evict_last();
      const uint64_t pol_q = l2_policy_evict_first();
      int k_issued = 0, v_issued = 0;  // ring positions, counted over all units
      bool ok = true;
      // one tile into the next position of a ring
      auto put = [&](int& issued, int stages, int full, int empty, int off, const CUtensorMap* map,
                     const DbgBounds& d, int y, int z, uint64_t pol, int site, int chk) {
        const int st = issued % stages;
        if (!wait_bounded(bar(empty + st), ((issued / stages) & 1) ^ 1, ctl, site)) return false;
        mbar_arrive_expect_tx(bar(full + st), L::kTile);
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c) {
          // a skipped copy leaves the stage's transaction count short: the
          // consumer's bounded wait then ends the kernel
          const uint32_t dst = sb + off + st * L::kTile + c * kBlockX;
          if (dbg_tma(d, dst, kBlockX, c * 64, y, z, false, chk))
            tma_load_3d(dst, map, bar(full + st), c * 64, y, z, pol);
        }
        ++issued;
        return true;
      };
      auto put_k = [&](const CUtensorMap* map, const DbgBounds& d, int y, int z, uint64_t pol) {
        return put(k_issued, L::kKStages, L::kKFull, L::kKEmpty, L::kKOff, map, d, y, z, pol,
                   kSiteXqProd | (k_issued & 0x7f), kChkXLoadA);
      };
      auto put_v = [&](const CUtensorMap* map, const DbgBounds& d, int y, int z, uint64_t pol) {
        return put(v_issued, L::kVStages, L::kVFull, L::kVEmpty, L::kVOff, map, d, y, z, pol,
                   kSiteXqProd | 0x80 | (v_issued & 0x7f), kChkXLoadB);
      };
      BwdUnit un = unit0;
      for (int unit = 0; ok;) {
        ok = put_v(&p.tm_do, dbb, un.tile * kRowsX, un.bh, pol_q) &&
             put_k(&p.tm_q, dbb, un.tile * kRowsX, un.bh, pol_q) &&
             put_v(&p.tm_out, dbb, un.tile * kRowsX, un.bh, pol_q);
        for (int j = 0; j < un.n && ok; ++j)
          ok = put_k(&p.tm_k, dbk, (un.first + j) * kRowsX, un.bh, pol_kv) &&
               put_v(&p.tm_v, dbk, (un.first + j) * kRowsX, un.bh, pol_kv);
        if (ok) {  // the way out
          const int st = k_issued % L::kKStages;
          ok = wait_bounded(bar(L::kKEmpty + st), ((k_issued / L::kKStages) & 1) ^ 1, ctl, kSiteXqProd | (k_issued & 0x7f));
          if (ok) mbar_arrive(bar(L::kKFull + st)), ++k_issued;
        }
        const int x = unit_at(++unit);
        if (x >= n_units) break;
        un = cross_dq_unit<kRowsX>(p, x, order);
      }
      if (ok) {
        // every stage released by the tensor core before this CTA may exit
        for (int i = max(k_issued - L::kKStages, 0); i < k_issued && ok; ++i)
          ok = wait_bounded(bar(L::kKEmpty + i % L::kKStages), (i / L::kKStages) & 1, ctl, kSiteXqProd | 0x7f);
        for (int i = max(v_issued - L::kVStages, 0); i < v_issued && ok; ++i)
          ok = wait_bounded(bar(L::kVEmpty + i % L::kVStages), (i / L::kVStages) & 1, ctl, kSiteXqProd | 0xff);
      }
      if (!ok) {
        for (int i = max(k_issued - L::kKStages, 0); i < k_issued; ++i)
          wait_drain(bar(L::kKFull + i % L::kKStages), (i / L::kKStages) & 1, kDrainLimitNsX);
        for (int i = max(v_issued - L::kVStages, 0); i < v_issued; ++i)
          wait_drain(bar(L::kVFull + i % L::kVStages), (i / L::kVStages) & 1, kDrainLimitNsX);
      }
    }
  } else {
    // ======================= tcgen05 issuer (warp 8) =======================
    // The whole warp runs the issue code; each product and commit is predicated on
    // the elected lane.
    const bool leader = elect_one();
    constexpr uint32_t kIdescSP = instr_desc_16bit(kRowsX, 64, false, false, F16);  // 64 keys
    constexpr uint32_t kIdescQ = instr_desc_16bit(kRowsX, D, false, true, F16);
    constexpr uint32_t kTileUnits = L::kTile >> 4;
    constexpr uint32_t kHalfUnits = (64 * 128) >> 4;  // 64 rows of a 128-byte-row block
    const uint64_t dk = smem_desc_sw128(sb + L::kKOff, 16, 1024);
    const uint64_t dv = smem_desc_sw128(sb + L::kVOff, 16, 1024);
    const uint64_t dk_mn = smem_desc_sw128(sb + L::kKOff, kBlockX, 1024);
    auto wait_warp = [&](uint32_t b, uint32_t parity, int site) {
      return __all_sync(0xffffffffu, wait_bounded(b, parity, ctl, site));
    };
    // SP(h): S_h = Q · K[64h, 64h+64)ᵀ and dP_h = dO · V[64h, 64h+64)ᵀ of the K and V
    // tiles in ring positions kp and vp; A (Q, dO) from TMEM, 8 columns per K step of 16
    auto issue_sp = [&](int kp, int vp, int h) {
      const int ks = kp % L::kKStages, vs = vp % L::kVStages;
      if (!dbg_smem(dbb, sb + L::kKOff + ks * L::kTile, L::kTile, 1024, kChkXMmaA) ||
          !dbg_smem(dbb, sb + L::kVOff + vs * L::kTile, L::kTile, 1024, kChkXMmaB))
        return;  // S_h never completes: the elementwise warps' bounded wait ends the kernel
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kBlockX + (kk & 3) * 32) >> 4;
        mma_ts_p(leader, tmem_base + 128 * h, tmem_base + L::kQCol + kk * 8,
                 dk + ks * kTileUnits + h * kHalfUnits + off, kIdescSP, kk > 0 ? 1u : 0u);
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kBlockX + (kk & 3) * 32) >> 4;
        mma_ts_p(leader, tmem_base + 128 * h + 64, tmem_base + L::kDoCol + kk * 8,
                 dv + vs * kTileUnits + h * kHalfUnits + off, kIdescSP, kk > 0 ? 1u : 0u);
      }
      mma_commit_p(leader, bar(L::kSFull + h));
    };
    // G(h): dQ += dS_h · K[64h, 64h+64) (16 key rows per step)
    auto issue_g = [&](int kp, int h, bool first) {
      const int ks = kp % L::kKStages;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int r = 0; r <= (TWO ? 1 : 0); ++r)
          mma_ts_p(leader, tmem_base + L::kDqCol, tmem_base + 128 * h + 32 * r + kk * 8,
                   dk_mn + ks * kTileUnits + (4 * h + kk) * (2048 >> 4), kIdescQ,
                   (first && kk == 0 && r == 0) ? 0u : 1u);
    };
    auto k_full = [&](int kp) {
      return wait_warp(bar(L::kKFull + kp % L::kKStages), (kp / L::kKStages) & 1, kSiteXqMmaKV | (kp & 0x7f));
    };
    auto v_full = [&](int vp) {
      return wait_warp(bar(L::kVFull + vp % L::kVStages), (vp / L::kVStages) & 1, kSiteXqMmaKV | 0x80 | (vp & 0x7f));
    };
    BwdUnit un = unit0;
    int kpos = 0, vpos = 0, steps = 0;  // the unit's first ring positions
    bool ok = true;
    // tile j of the unit has landed; what lies behind the keys' end is silenced, as dQ's
    // product multiplies it by dS = 0
    auto wait_kv = [&](int j) {
      const bool r = k_full(kpos + 1 + j) && v_full(vpos + 2 + j);
      if (r)
        clear_tail<L::kChunks>(sb + L::kKOff + ((kpos + 1 + j) % L::kKStages) * L::kTile, kRowsX,
                               un.len - (un.first + j) * kRowsX, un.len < p.Sk, lane, dbb, kChkXMmaA);
      return r;
    };
    for (int unit = 0;; ++unit) {
      // Q and dO into tensor memory.  The products that read the last unit's are
      // complete: this warp has waited for the dS of its last step, which came after them.
      ok = k_full(kpos) && v_full(vpos);
      if (!ok) break;
      tc_fence_after_sync();
      if (leader && dbg_smem(dbb, sb + L::kKOff + (kpos % L::kKStages) * L::kTile, L::kTile, 1024, kChkXMmaA) &&
          dbg_smem(dbb, sb + L::kVOff + (vpos % L::kVStages) * L::kTile, L::kTile, 1024, kChkXMmaB)) {
        copy_tile<D>(tmem_base + L::kQCol, dk + (kpos % L::kKStages) * kTileUnits);
        mma_commit(bar(L::kKEmpty + kpos % L::kKStages));
        copy_tile<D>(tmem_base + L::kDoCol, dv + (vpos % L::kVStages) * kTileUnits);
      }
      __syncwarp();
      ok = wait_kv(0);
      if (!ok) break;
      tc_fence_after_sync();
      issue_sp(kpos + 1, vpos + 2, 0);
      issue_sp(kpos + 1, vpos + 2, 1);
      mma_commit_p(leader, bar(L::kVEmpty + (vpos + 2) % L::kVStages));
      if (unit > 0) {  // the last unit's dQ has been read, and its place in the ring
        ok = wait_warp(bar(L::kOFree), (unit - 1) & 1, kSiteXqMmaFree);
        if (!ok) break;
        if (leader) mbar_arrive(bar(L::kKEmpty + (kpos - 1) % L::kKStages));
        tc_fence_after_sync();
      }
      for (int j = 0; j < un.n && ok; ++j) {
        const int kp = kpos + 1 + j, vp = vpos + 2 + j;
        const bool more = j + 1 < un.n;
        if (more) ok = wait_kv(j + 1);
        if (ok) ok = wait_warp(bar(L::kPFull + 0), (steps + j) & 1, kSiteXqMmaP | (j & 0x7f));
        if (!ok) break;
        if (j == 0) {
          // dO has been copied (the scores that have been read came after it) and, once
          // every delta is written, read: its place and out's are free
          ok = wait_warp(bar(L::kStat), unit & 1, kSiteXqMmaP | 0xff);
          if (!ok) break;
          if (leader) {
            mbar_arrive(bar(L::kVEmpty + vpos % L::kVStages));
            mbar_arrive(bar(L::kVEmpty + (vpos + 1) % L::kVStages));
          }
        }
        tc_fence_after_sync();
        issue_g(kp, 0, j == 0);
        if (more) issue_sp(kp + 1, vp + 1, 0);
        ok = wait_warp(bar(L::kPFull + 1), (steps + j) & 1, kSiteXqMmaP | 0x80 | (j & 0x7f));
        if (!ok) break;
        tc_fence_after_sync();
        issue_g(kp, 1, false);
        mma_commit_p(leader, bar(L::kKEmpty + kp % L::kKStages));  // K_j: last read by G(j, 1)
        if (more) {
          issue_sp(kp + 1, vp + 1, 1);
          mma_commit_p(leader, bar(L::kVEmpty + (vp + 1) % L::kVStages));  // V: last read by SP(·, 1)
        }
      }
      if (!ok) break;
      mma_commit_p(leader, bar(L::kOFull));
      steps += un.n;
      kpos += 2 + un.n;
      vpos += 2 + un.n;
      const int x = unit_at(unit + 1);
      if (x >= n_units) {  // the last one's way out
        ok = wait_warp(bar(L::kOFree), unit & 1, kSiteXqMmaFree);
        if (ok && leader) mbar_arrive(bar(L::kKEmpty + (kpos - 1) % L::kKStages));
        break;
      }
      un = cross_dq_unit<kRowsX>(p, x, order);
    }
    if (leader) {
      mma_commit(bar(L::kDrain));
      wait_drain(bar(L::kDrain), 0, kDrainLimitNsX);
    }
    __syncwarp();
  }

  __syncthreads();
  if (warp == 8) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, kTmemColsX);
  }
}

// ============================================================== dk/dv kernel
// Each Q tile is four 32-query sub-steps, warpgroup b taking those t ≡ b (mod 2); the last
// one two where no query is in the other two.
// TMEM: buffer b's Sᵀ [64b, 64b+32) and dPᵀ [64b+32, 64b+64); K [128, 128+D/2),
// V [128+D/2, 128+D); dV [256, 256+D), dK [256+D, 256+2D).

template <int D>
struct XkLayout {
  static constexpr int kTile = kRowsX * D * 2;
  static constexpr int kChunks = D / 64;
  // Ring positions of two tiles each: of a unit first K and V, then its Q and dO tiles,
  // then a place for dV and dK on their way out
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kStatBytes = 2 * kRowsX * 4;    // (−lse·log2e, −delta) per query row
  static constexpr int kQOff = 0;
  static constexpr int kDoOff = kQOff + kStages * kTile;
  static constexpr int kStatOff = kDoOff + kStages * kTile;
  static constexpr int kBarOff = kStatOff + kStages * kStatBytes;
  static constexpr int kFull = 0;
  static constexpr int kEmpty = kFull + kStages;
  static constexpr int kSFull = kEmpty + kStages;   // [2] Sᵀ and dPᵀ of buffer b computed
  static constexpr int kPFull = kSFull + 2;         // [2] Pᵀ and dSᵀ of buffer b stored (128)
  static constexpr int kOFull = kPFull + 2;         // dK, dV final
  static constexpr int kOFree = kOFull + 1;         // dK, dV read, their place in the ring too (256 arrivals)
  static constexpr int kDrain = kOFree + 1;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kAlloc = kMiscOff + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget exceeded");
  static constexpr uint32_t kKCol = 128, kVCol = 128 + D / 2, kDvCol = 256, kDkCol = 256 + D;
};

// Sub-steps of a unit.  (128 slices of one query over 1500 keys of 64 channels: 48.5 us
// against 56.0 with all four.)
__device__ __forceinline__ int sub_steps(const BwdUnit& u, int S) {
  return 4 * u.n - (S - (u.first + u.n - 1) * kRowsX <= 64 ? 2 : 0);
}

// MANY: more sequences between a CTA's units than are worth looking at one by one.  TWO:
// P and dS in two terms, as in the dq kernel.
template <int D, bool F16, bool MANY, bool TWO>
__global__ void __launch_bounds__(kBwdThreads, 1) cross_dkdv_kernel(const __grid_constant__ BwdParams p) {
  using L = XkLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint8_t* smem_gen = smem_raw + (sb - smem_u32(smem_raw));  // same window, generic
  auto bar = [sb](int idx) -> uint32_t { return sb + L::kBarOff + 8u * idx; };
  const uint32_t tmem_slot = sb + L::kMiscOff;
  const uint32_t abort_addr = sb + L::kMiscOff + 4;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const DbgBounds dbb{p.status, sb, smem_u32(smem_raw) + static_cast<uint32_t>(L::kAlloc), p.S,
                      p.d_cols, p.BH};
  const DbgBounds dbk = key_bounds<kMaskCross>(dbb, p.Sk);
  // this CTA's units, those of key tiles that have keys
  const int runs = cross_kv_runs(p.kv, p.lens);
  KvWalk walk0 = kv_walk(static_cast<int>(blockIdx.x), runs);
  BwdUnit unit0{};
  const bool any = cross_kv_unit<kRowsX, MANY>(p, walk0, &unit0);
  auto next_unit = [&](KvWalk& w, BwdUnit* un) {
    w.x += static_cast<int>(gridDim.x);
    return cross_kv_unit<kRowsX, MANY>(p, w, un);
  };

  // This kernel is set up on each SM as the dq kernel leaves it; what waits for delta
  // does so before the first bounded wait that depends on it, and all before the end.
  if (threadIdx.x == 0) {
    launch_dependents();
#pragma unroll
    for (int s = 0; s < L::kStages; ++s) mbar_init(bar(L::kFull + s), 1), mbar_init(bar(L::kEmpty + s), 1);
#pragma unroll
    for (int b = 0; b < 2; ++b) mbar_init(bar(L::kSFull + b), 1), mbar_init(bar(L::kPFull + b), 128);
    mbar_init(bar(L::kOFull), 1);
    mbar_init(bar(L::kOFree), 256);
    mbar_init(bar(L::kDrain), 1);
    st_volatile_shared(abort_addr, 0);
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, kTmemColsX);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = static_cast<uint32_t>(ld_volatile_shared(tmem_slot));
  const WaitCtl ctl{abort_addr, p.status, p.timeout_ns};

  if (warp < 8) {
    // ======================= elementwise: Pᵀ, dSᵀ, dK and dV out =======================
    const int g = warp >> 2;            // TMEM buffer (quarters g and g+2) of this warpgroup
    const int wq = warp & 3;
    const int r = wq * 32 + lane;       // key row within the tile (TMEM lane)
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem_base + lane_bits + 64 * g;
    const uint32_t tP = tS + 32;
    const float sl2 = p.scale_log2;
    KvWalk walk = walk0;
    BwdUnit un = unit0;
    int subs = 0, pos = 0;  // sub-steps and ring positions of the units before this one
    bool ok = true;
    wait_for_previous();
    for (int unit = 0; any; ++unit) {
      const int gk = un.tile * kRowsX + r;  // key row in the sequence
      const bool there = gk < un.len;
      const int end = sub_steps(un, p.S);
      for (int t = g; t < end; t += 2) {
        const int it = t >> 2, q = t & 3;
        ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kSFull + g), ((subs + t) >> 1) & 1, ctl,
                                                  kSiteXkElemS | (g << 7) | (t & 0x7f)));
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t s[32], dp[32];
        if (!dbg_warp(dbg_tmem(dbb, tS, 32, warp, kChkXSTmem) && dbg_tmem(dbb, tP, 32, warp, kChkXSTmem))) {
          ok = false;
          break;
        }
        tmem_ld_32x32b_x32(tS, s);
        tmem_ld_32x32b_x32(tP, dp);
        tmem_ld_wait();
        reg_fence(s);
        reg_fence(dp);
        // query columns of this quarter that are there: 0 .. hi; none for a key that is not
        const int hi = there ? p.S - 1 - ((un.first + it) * kRowsX + 32 * q) : -1;
        // (−lse·log2e, −delta) of this quarter's 32 query columns, two columns per load
        const float4* stat = reinterpret_cast<const float4*>(
            smem_gen + L::kStatOff + ((pos + 1 + it) % L::kStages) * L::kStatBytes + 8 * 32 * q);
        uint32_t ppk[16], dpk[16], prest[TWO ? 16 : 1], drest[TWO ? 16 : 1];
        auto weigh = [&](auto masked) {
          constexpr bool kMasked = decltype(masked)::value;
#pragma unroll
          for (int e2 = 0; e2 < 16; ++e2) {
            const int c = 2 * e2;
            const float4 sd = stat[e2];  // -lse2[c], -delta[c], -lse2[c+1], -delta[c+1]
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                        make_float2(sl2, sl2), make_float2(sd.x, sd.z));
            float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            const float2 dd = __fadd2_rn(make_float2(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1])),
                                         make_float2(sd.y, sd.w));
            float2 ds = __fmul2_rn(make_float2(p0, p1), dd);
            if (kMasked) {  // a key that is not there may make S and dP anything
              if (c > hi) p0 = 0.f, ds.x = 0.f;
              if (c + 1 > hi) p1 = 0.f, ds.y = 0.f;
            }
            const float2 pt = F16 ? __fmul2_rn(make_float2(p0, p1), make_float2(kPTimes<F16>, kPTimes<F16>))
                                  : make_float2(p0, p1);
            ppk[e2] = pack_x2<F16>(pt.x, pt.y);
            dpk[e2] = pack_x2<F16>(ds.x, ds.y);
            if constexpr (TWO) {
              prest[e2] = rest_x2<F16>(pt, ppk[e2]);
              drest[e2] = rest_x2<F16>(ds, dpk[e2]);
            }
          }
        };
        if (__any_sync(0xffffffffu, hi < 31)) weigh(std::true_type{});
        else weigh(std::false_type{});
        tmem_st_32x32b_x16(tS, ppk);
        tmem_st_32x32b_x16(tP, dpk);
        if constexpr (TWO) {
          tmem_st_32x32b_x16(tS + 16, prest);
          tmem_st_32x32b_x16(tP + 16, drest);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(bar(L::kPFull + g));
      }
      if (!ok) break;
      subs += end;
      pos += 1 + un.n;

      // warpgroup 0 stores dV, 1 stores dK · scale, by way of the ring's next place
      const int st = pos % L::kStages;
      ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kFull + st), (pos / L::kStages) & 1, ctl, kSiteXkElemO | 0x80));
      if (ok) ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kOFull), unit & 1, ctl, kSiteXkElemO));
      if (!ok) break;
      ++pos;
      tc_fence_after_sync();
      const uint32_t tAcc = tmem_base + lane_bits + (g == 0 ? L::kDvCol : L::kDkCol);
      if (runs > 1) {  // this run's sum, to be added to the others
        float* to = (g == 0 ? p.part_dv : p.part_dk) +
                    (((int64_t)un.part * p.BH + un.bh) * p.Sk + gk) * p.d_cols;
#pragma unroll 1
        for (int c = 0; c < 2 * L::kChunks; ++c)
          store_part(tAcc + c * 32, to, c * 32, g == 0 ? 1.f / kPTimes<F16> : 1.f, there, dbk, un.bh, gk, kChkStore);
      } else {
#pragma unroll 1
        for (int c = 0; c < L::kChunks; ++c)
          store_chunk<F16>(tAcc + c * 64, sb + (g == 0 ? L::kQOff : L::kDoOff) + st * L::kTile + c * kBlockX, r,
                           g == 0 ? 1.f / kPTimes<F16> : p.scale, g == 0 ? &p.tm_dv : &p.tm_dk, c * 64, un.tile * kRowsX,
                           un.bh, wq, lane, dbk, !there);
        if (lane == 0) {
          tma_store_commit();
          tma_store_wait_read();
        }
        __syncwarp();
      }
      tc_fence_before_sync();
      mbar_arrive(bar(L::kOFree));
      if (!next_unit(walk, &un)) break;
    }
    if (ok)
      cross_zero_tiles(p, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), threadIdx.x, 256, 0, D);
    if (lane == 0) tma_store_wait_all();
    tc_fence_before_sync();
  } else if (warp == 9) {
    // ======================= producer: K and V, then Q, dO and statistics per Q tile =======================
    const uint64_t pol_q = l2_policy_evict_last(), pol_kv = l2_policy_evict_first();
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
      tma_prefetch_desc(&p.tm_q);
      tma_prefetch_desc(&p.tm_do);
      tma_prefetch_desc(&p.tm_dk);
      tma_prefetch_desc(&p.tm_dv);
    }
    int issued = 0;  // ring positions, counted over all units
    bool ok = true;
    KvWalk walk = walk0;
    BwdUnit un = unit0;
    for (bool more = any; more && ok; more = next_unit(walk, &un)) {
      const int64_t row0 = (int64_t)un.bh * p.S;
      for (int it = -1; it <= un.n; ++it) {  // -1: the unit's K and V; un.n: the way out
        const int st = issued % L::kStages;
        ok = __all_sync(0xffffffffu, wait_bounded(bar(L::kEmpty + st), ((issued / L::kStages) & 1) ^ 1,
                                                  ctl, kSiteXkProd | (issued & 0xff)));
        if (!ok) break;
        if (it == un.n) {
          if (lane == 0) mbar_arrive(bar(L::kFull + st));
          ++issued;
          __syncwarp();
          continue;
        }
        const int y = (it < 0 ? un.tile : un.first + it) * kRowsX;
        if (issued == 1) wait_for_previous();
        if (it >= 0) {
          // per-query-row statistics of the Q tile; rows past the end read as 0
          const uint32_t stat = sb + L::kStatOff + st * L::kStatBytes;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int c = lane + 32 * t;
            const bool in = y + c < p.S && dbg_row(dbb, un.bh, y + c, 0, 0, kChkXStat);
            st_shared_f32x2(stat + 8 * c, in ? -(p.lse[row0 + y + c] * kLog2eX) : 0.f,
                            in ? -p.delta[row0 + y + c] : 0.f);
          }
          __syncwarp();
        }
        if (lane == 0) {
          const CUtensorMap* ma = it < 0 ? &p.tm_k : &p.tm_q;
          const CUtensorMap* mb = it < 0 ? &p.tm_v : &p.tm_do;
          const DbgBounds& d = it < 0 ? dbk : dbb;
          const uint64_t pol = it < 0 ? pol_kv : pol_q;
          mbar_arrive_expect_tx(bar(L::kFull + st), 2 * L::kTile);
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c) {
            // a skipped copy leaves the stage's transaction count short: the
            // consumer's bounded wait then ends the kernel
            const uint32_t da = sb + L::kQOff + st * L::kTile + c * kBlockX;
            const uint32_t db = sb + L::kDoOff + st * L::kTile + c * kBlockX;
            if (dbg_tma(d, da, kBlockX, c * 64, y, un.bh, false, kChkXLoadA))
              tma_load_3d(da, ma, bar(L::kFull + st), c * 64, y, un.bh, pol);
            if (dbg_tma(d, db, kBlockX, c * 64, y, un.bh, false, kChkXLoadB))
              tma_load_3d(db, mb, bar(L::kFull + st), c * 64, y, un.bh, pol);
          }
        }
        ++issued;
        __syncwarp();
      }
      if (!ok) break;
    }
    if (lane == 0) {
      if (ok) {
        for (int i = max(issued - L::kStages, 0); i < issued && ok; ++i)
          ok = wait_bounded(bar(L::kEmpty + i % L::kStages), (i / L::kStages) & 1, ctl, kSiteXkProd | 0xff);
      }
      if (!ok) {
        for (int i = max(issued - L::kStages, 0); i < issued; ++i)
          wait_drain(bar(L::kFull + i % L::kStages), (i / L::kStages) & 1, kDrainLimitNsX);
      }
    }
    __syncwarp();
  } else {
    // ======================= tcgen05 issuer (warp 8) =======================
    const bool leader = elect_one();
    constexpr uint32_t kIdescSP = instr_desc_16bit(kRowsX, 32, false, false, F16);  // 32 queries
    constexpr uint32_t kIdescG = instr_desc_16bit(kRowsX, D, false, true, F16);
    constexpr uint32_t kTileUnits = L::kTile >> 4;
    constexpr uint32_t kQuarterUnits = (32 * 128) >> 4;  // 32 rows of a 128-byte-row block
    const uint64_t dq = smem_desc_sw128(sb + L::kQOff, 16, 1024);
    const uint64_t ddo = smem_desc_sw128(sb + L::kDoOff, 16, 1024);
    const uint64_t dq_mn = smem_desc_sw128(sb + L::kQOff, kBlockX, 1024);
    const uint64_t ddo_mn = smem_desc_sw128(sb + L::kDoOff, kBlockX, 1024);
    auto wait_warp = [&](uint32_t b, uint32_t parity, int site) {
      return __all_sync(0xffffffffu, wait_bounded(b, parity, ctl, site));
    };
    auto full = [&](int at, int site) {
      return wait_warp(bar(L::kFull + at % L::kStages), (at / L::kStages) & 1, site | (at & 0xff));
    };
    int pos = 0;  // the unit's first ring position: K and V, then its Q tiles
    // SP(t): Sᵀ = K · Q[32q, 32q+32)ᵀ and dPᵀ = V · dO[32q, 32q+32)ᵀ into
    // buffer t & 1; A (K, V) from TMEM, 8 columns per K step of 16
    auto issue_sp = [&](int t) {
      const int b = t & 1, q = t & 3, st = (pos + 1 + (t >> 2)) % L::kStages;
      if (!dbg_smem(dbb, sb + L::kQOff + st * L::kTile, L::kTile, 1024, kChkXMmaA) ||
          !dbg_smem(dbb, sb + L::kDoOff + st * L::kTile, L::kTile, 1024, kChkXMmaB))
        return;  // S never completes: the elementwise warps' bounded wait ends the kernel
      const uint32_t bq = st * kTileUnits + q * kQuarterUnits;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kBlockX + (kk & 3) * 32) >> 4;
        mma_ts_p(leader, tmem_base + 64 * b, tmem_base + L::kKCol + kk * 8, dq + bq + off, kIdescSP,
                 kk > 0 ? 1u : 0u);
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kBlockX + (kk & 3) * 32) >> 4;
        mma_ts_p(leader, tmem_base + 64 * b + 32, tmem_base + L::kVCol + kk * 8, ddo + bq + off, kIdescSP,
                 kk > 0 ? 1u : 0u);
      }
      mma_commit_p(leader, bar(L::kSFull + b));
    };
    // G(t): dV += Pᵀ · dO[32q, 32q+32), dK += dSᵀ · Q[32q, 32q+32)
    auto issue_g = [&](int t) {
      const int b = t & 1, q = t & 3, st = (pos + 1 + (t >> 2)) % L::kStages;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const uint32_t bo = st * kTileUnits + (2 * q + kk) * (2048 >> 4);
#pragma unroll
        for (int r = 0; r <= (TWO ? 1 : 0); ++r) {
          const uint32_t a = 64 * b + 16 * r + kk * 8;
          const uint32_t acc = (t == 0 && kk == 0 && r == 0) ? 0u : 1u;
          mma_ts_p(leader, tmem_base + L::kDvCol, tmem_base + a, ddo_mn + bo, kIdescG, acc);
          mma_ts_p(leader, tmem_base + L::kDkCol, tmem_base + a + 32, dq_mn + bo, kIdescG, acc);
        }
      }
    };
    KvWalk walk = walk0;
    BwdUnit un = unit0;
    int subs = 0;
    bool ok = true;
    for (int unit = 0; any; ++unit) {
      const int end = sub_steps(un, p.S);
      // K and V into tensor memory: the products that read the last unit's are
      // complete, as this warp has waited for the P of its last sub-steps
      ok = full(pos, kSiteXkMmaKV);
      if (!ok) break;
      tc_fence_after_sync();
      if (leader && dbg_smem(dbb, sb + L::kQOff + (pos % L::kStages) * L::kTile, L::kTile, 1024, kChkXMmaA)) {
        copy_tile<D>(tmem_base + L::kKCol, dq + (pos % L::kStages) * kTileUnits);
        copy_tile<D>(tmem_base + L::kVCol, ddo + (pos % L::kStages) * kTileUnits);
        mma_commit(bar(L::kEmpty + pos % L::kStages));
      }
      __syncwarp();
      if (unit == 0) wait_for_previous();
      ok = full(pos + 1, kSiteXkMmaQ);
      if (!ok) break;
      tc_fence_after_sync();
      issue_sp(0);
      issue_sp(1);
      if (unit > 0) {  // the last unit's sums have been read
        ok = wait_warp(bar(L::kOFree), (unit - 1) & 1, kSiteXkMmaFree);
        if (!ok) break;
        if (leader) mbar_arrive(bar(L::kEmpty + (pos - 1) % L::kStages));
        tc_fence_after_sync();
      }
      for (int t = 0; t < end && ok; ++t) {
        const int b = t & 1;
        const int t2 = t + 2;
        // the sub-step issued after this one opens Q tile t2 / 4: its stage must have
        // landed (normally long before this P, so waited for first)
        if ((t2 & 3) == 0 && t2 < end) ok = full(pos + 1 + (t2 >> 2), kSiteXkMmaQ);
        if (ok) ok = wait_warp(bar(L::kPFull + b), ((subs + t) >> 1) & 1, kSiteXkMmaP | (b << 7) | (t & 0x7f));
        if (!ok) break;
        tc_fence_after_sync();
        issue_g(t);
        if ((t & 3) == 3 || t == end - 1) mma_commit_p(leader, bar(L::kEmpty + (pos + 1 + (t >> 2)) % L::kStages));  // Q, dO done
        if (t2 < end) issue_sp(t2);
      }
      if (!ok) break;
      mma_commit_p(leader, bar(L::kOFull));
      subs += end;
      pos += 2 + un.n;
      if (!next_unit(walk, &un)) {  // the last one's way out
        ok = wait_warp(bar(L::kOFree), unit & 1, kSiteXkMmaFree);
        if (ok && leader) mbar_arrive(bar(L::kEmpty + (pos - 1) % L::kStages));
        break;
      }
    }
    if (leader) {
      mma_commit(bar(L::kDrain));
      wait_drain(bar(L::kDrain), 0, kDrainLimitNsX);
    }
    __syncwarp();
  }

  __syncthreads();
  if (warp == 8) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, kTmemColsX);
  }
}

template <int D, bool F16, bool TWO>
cudaError_t launch_cross(const BwdParams& p, cudaStream_t stream) {
  // Long sequences first where a CTA takes few units, which may differ much: a decoder's
  // ragged batch, 3.4 units a CTA, 93.3 us against 99.4 for the gradient (in their own
  // order the SMs were active for 69 % of the dq kernel's time); two prompts, 6.7 units a
  // CTA, 87.6 against 85.4, since the order has to be found and kept.
  const long long q_units = (long long)p.BH * p.n_qt * p.q_split;
  const bool ordered = p.lens != nullptr && p.BH / p.heads <= kMaxOrder && q_units < 5ll * p.sms;
  auto kdq = ordered ? cross_dq_kernel<D, F16, true, TWO> : cross_dq_kernel<D, F16, false, TWO>;
  // Whether a CTA passes eight sequences and more from one unit to its next.  10000
  // sequences of one tile: 744 us against 1512, whose walk alone took longer than the
  // work; in every call, 300 sequences of 8 heads of 3 tiles 218 us against 204.
  const bool many = p.lens != nullptr && 8ll * p.heads * p.n_kt <= p.sms;
  auto kkv = many ? cross_dkdv_kernel<D, F16, true, TWO> : cross_dkdv_kernel<D, F16, false, TWO>;
  cudaError_t e = cudaFuncSetAttribute(kdq, cudaFuncAttributeMaxDynamicSharedMemorySize, XqLayout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kkv, cudaFuncAttributeMaxDynamicSharedMemorySize, XkLayout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  auto ctas = [&](long long units) { return dim3(static_cast<unsigned>(units < p.sms ? units : p.sms), 1, 1); };
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = ctas(q_units);
  cfg.blockDim = dim3(kBwdThreads, 1, 1);
  cfg.stream = stream;
  cfg.dynamicSmemBytes = XqLayout<D>::kAlloc;
  e = cudaLaunchKernelEx(&cfg, kdq, p);
  if (e != cudaSuccess) return e;
  return launch_after(kkv, ctas((long long)p.BH * p.n_kt * p.kv.most_runs), kBwdThreads, stream, p, XkLayout<D>::kAlloc);
}

template <int D, bool F16>
cudaError_t launch_terms(const BwdParams& p, cudaStream_t stream) {
  return two_terms(p) ? launch_cross<D, F16, true>(p, stream) : launch_cross<D, F16, false>(p, stream);
}

}  // namespace

cudaError_t cross_bwd_launch(const BwdParams& p, int D, bool f16, cudaStream_t stream) {
  if (D == 64) return f16 ? launch_terms<64, true>(p, stream) : launch_terms<64, false>(p, stream);
  if (D == 128) return f16 ? launch_terms<128, true>(p, stream) : launch_terms<128, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ea
