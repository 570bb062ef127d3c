// rope_sm103.cu — the heads' norm and rotation and their gradient (sm_103a);
// include/attn_rope.h has the formulas.
//
// Bound by the memory: a training step's rows are read once and written once
// (the gradient reads two tensors), about 8 operations a value.  So the kernels
// are shaped by three things: full-width loads and stores, enough of them in
// flight, and few instructions a value.
//
//   A warp works by itself, on one unit after the other: a token's heads of all
//   parts, or a share of them where tokens are few.  It finds the angles of the
//   token once, for all heads, into shared memory: a sine and a cosine cost about
//   as much as a row's 16 values.
//   A lane holds 16 values of a row, in pairs: `width` pairs to a vector, both
//   channels of each, so that the rotation needs no exchange.  A row takes
//   D/16 neighbouring lanes, whatever that number is (the sums over a row are
//   shuffles that stop at its last lane), and a warp as many rows as fit.
//   Rows come through a ring in shared memory that each lane fills and reads for
//   itself (cp.async, no barrier), two slots ahead and across units: up to 64 KB in
//   flight on an SM (16 warps, slots of 2 KB), 96 KB in the gradient (12 warps, x and
//   dy in 4 KB), without registers to hold them.
//   Units are dealt to the warps of one full grid, each the same number of them.
//
// Angles.  A position adds the fraction inv_freq / 2π of a turn.  It is kept as
// a 64-bit integer in units of 2^-64 turns: position times it, modulo 2^64, is
// the angle without whole turns, exactly, at any position; the top 32 bits then
// go to sincospif.
//
// The gradient of the weights: each thread adds up its channels over all rows
// that it takes, the CTA adds its threads' sums in a fixed order, and a second
// kernel, set up while the first ends, the CTAs'.
//
// Measured on a GB300, calls in a graph.  2 x 4096 tokens of 32 + 8 + 8 heads of 128
// channels: 39 us, 5.1 TB/s, 77 % of what a plain copy gets; the gradient 61.5 us, 4.6
// TB/s.  12720 tokens of 3 x 16 heads of 72 channels in neighbouring pairs: 51 and 81
// us, 52 % and 43 %: a row of 144 bytes fills four and a half lanes, and both run at
// half of the issue slots with the latency of shared memory in between.  One token of 16
// sequences: 8 us, a chain of positions, angles, rows and stores.  Pairs half a row
// apart that 8 does not divide go in narrower vectors: of the first case 60, 62 and 63
// pairs in place of 64 take 44, 55 and 108 us (75, 101 and 245 the gradient); one pair a
// vector has no asynchronous copies, and its gradient spills 48 bytes.  A CTA for eight
// tokens with its rows in registers took 60 us for the first; one row a lane, 42 to
// 47; rings of 2 or 4 and other numbers of CTAs, 40 to 52.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "bwd_common.cuh"
#include "launch_after.cuh"
#include "ptx.cuh"
#include "rope_impl.h"

namespace ea {
namespace {

enum : int { kChkRopeRow = 0x6101 };

template <int N>
struct Vec;  // N 16-bit values
template <> struct Vec<8> { using T = uint4; };
template <> struct Vec<4> { using T = uint2; };
template <> struct Vec<2> { using T = uint32_t; };
template <> struct Vec<1> { using T = uint16_t; };

template <bool F16>
__device__ __forceinline__ float2 widen(uint32_t x) {
  if constexpr (F16) return f16x2_to_f32(x);
  else return make_float2(bf16_lo(x), bf16_hi(x));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <bool F16>
__device__ __forceinline__ float weight_at(const RopePart& q, int d) {
  if (q.weight_f32) return __ldg(static_cast<const float*>(q.weight) + d);
  const uint32_t w = __ldg(static_cast<const unsigned short*>(q.weight) + d);
  return widen<F16>(w).x;
}

// The sums of each v over a row's `lanes` lanes, in every one of them.  t: this lane's
// place in its row, first: the row's first lane, even: lanes is a power of two.
// Lanes behind the last row pass through with sums of their own.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int t, int lanes, int first, bool even) {
  if (even) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      if (off >= lanes) break;  // the same in every lane
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    }
    return;
  }
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    if (off >= lanes) break;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float o = __shfl_down_sync(0xffffffffu, v[i], off);
      if (t + off < lanes) v[i] += o;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], first);
}

// 4, 8 or 16 bytes global -> shared, asynchronous; 2 bytes at once.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else if constexpr (BYTES == 2)
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst), "h"(*static_cast<const uint16_t*>(src)) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Threads of a CTA (warps share nothing but the weights and, in the gradient,
// the sum of theirs), CTAs that are to fit an SM, and rows that a ring holds.
template <bool BWD>
struct RopeTile {
  static constexpr int kThreads = BWD ? 128 : 64;
  static constexpr int kCtas = BWD ? 3 : 8;
  static constexpr int kRing = 3;
  static constexpr int kRows = 2;  // of a lane at once
};

// float4 of a unit's angles: of each pair cos, cos, -sin, sin where a float2 is a
// pair; else the cosines, the sines and the negative sines (two pairs: cos, cos, sin,
// sin, then the negative ones).
template <int VW>
struct RopeTurns {
  static constexpr int kUnit = VW == 1 ? 1 : VW == 2 ? 2 : 3 * VW / 4;
};

template <bool F16, bool INTER, int VW, bool BWD>
__global__ void __launch_bounds__(RopeTile<BWD>::kThreads, RopeTile<BWD>::kCtas)
    rope_kernel(const __grid_constant__ RopeParams p) {
  using RT = RopeTile<BWD>;
  // A lane's 16 values of a row: NU units of VW pairs.  Where pairs are half a row
  // apart unit u's first channels are a .. a+VW-1, the second ones b ..; where they
  // are neighbours the unit is the 2·VW channels from a on.
  constexpr int NU = 8 / VW;
  constexpr int LV = INTER ? 2 * VW : VW;   // values of one load
  constexpr int NL = INTER ? 1 : 2;         // loads of a unit
  // In registers a unit is VW float2: the first channels of two pairs each, then
  // the second ones; of one pair where VW is 1 (kByPair).
  constexpr bool kByPair = VW == 1;
  constexpr int kWarps = RT::kThreads / 32;
  constexpr int kVecs = NU * NL * (BWD ? 2 : 1);  // loads of a row
  constexpr int kTurn = RopeTurns<VW>::kUnit;
  using LT = typename Vec<LV>::T;
  constexpr int kRows = RT::kRows;
  __shared__ LT s_ring[kWarps][RT::kRing][kRows][kVecs][32];
  // (indexed by lane: constant memory would serve one lane after the other)
  __shared__ uint64_t s_fraction[kRopeMaxPairs];
  extern __shared__ float4 s_dyn[];  // weights [parts][4 · lanes], then per warp the angles [NU · kTurn · lanes]

  // (the shuffle tells the compiler that the warp's number, and with it all that says
  // where a warp is, is the same in every lane)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int lanes = p.lanes;
  const bool even = (lanes & (lanes - 1)) == 0;
  const int mine = lane / lanes;  // row of the warp's; per_warp: none
  const int t = lane - mine * lanes, first = mine * lanes;
  const int units = p.D / (2 * VW);
  int ca[NU], cb[NU];  // this lane's channels
  bool in[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = t + i * lanes;
    in[i] = u < units && mine < p.per_warp;
    ca[i] = INTER ? u * 2 * VW : u * VW < p.pairs ? u * VW : p.pairs + u * VW;
    cb[i] = INTER ? 0 : ca[i] + (u * VW < p.pairs ? p.pairs : p.D / 2 - p.pairs);
  }
  // channel of value e (0 .. 2·VW-1, in the order of the float2) of unit i
  auto channel = [&](int i, int e) {
    if constexpr (INTER) return ca[i] + (e < VW ? 2 * e : 2 * (e - VW) + 1);
    else return e < VW ? ca[i] + e : cb[i] + e - VW;
  };
  // weights so that lanes read 16 bytes side by side (8 where VW is 1)
  constexpr int kW = VW == 1 ? 2 : 4;
  auto w_at = [&](int i, int e) { return ((i * (2 * VW / kW) + e / kW) * lanes + t) * kW + e % kW; };
  float* s_w = reinterpret_cast<float*>(s_dyn);
  float4* s_turn = s_dyn + (p.n_parts * 4 + warp * NU * kTurn) * lanes;
  float2 acc[BWD ? 2 : 1][NU][VW];
  if constexpr (BWD) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e) acc[k][i][e] = both(0.f);
  }

  const uint32_t ring = smem_u32(&s_ring[warp][0][0][0][lane]);
  // Where a warp is: a unit's part, the first head of its rows there, and the
  // token; and this lane's first row, to read (x, and dy in y) or to write (to).
  const int stride = gridDim.x * kWarps, step = kRows * p.per_warp * p.split;
  const int64_t plane = (int64_t)p.S * p.D;
  struct Place {
    int unit, part, h, b, s;
    const uint16_t *x, *y;
    uint16_t* to;
  };
  auto token = [&](Place& c) {
    const int n = c.unit >> p.log2_split;
    c.b = static_cast<int>((static_cast<uint64_t>(n) * p.s_mul) >> p.s_shift);
    c.s = n - c.b * p.S;
    c.part = 0;
  };
  auto enter = [&](Place& c, bool reads) {
    const RopePart& q = p.part[c.part];
    c.h = (c.unit & (p.split - 1)) * kRows * p.per_warp;
    const int h = c.h + mine;
    const int64_t at = ((int64_t)c.b * q.heads + h) * plane + (int64_t)c.s * p.D;
    if (reads) {
      c.x = q.x + c.b * q.xb + c.s * q.xs + h * q.xh;
      if constexpr (BWD) c.y = q.y + at;
    } else {
      c.to = BWD ? q.dx + c.b * q.db + c.s * q.ds + h * q.dh : q.y + at;
    }
  };
  // on to rows that are there: a share of a unit may have none of a part
  auto settle = [&](Place& c, bool reads) {
    while (c.unit < p.units && c.h >= p.part[c.part].heads) {
      if (++c.part == p.n_parts) {
        c.unit += stride;
        token(c);
      }
      enter(c, reads);
    }
  };
  auto start = [&](bool reads) {
    Place c;
    c.unit = static_cast<int>(blockIdx.x) * kWarps + warp;
    token(c);
    enter(c, reads);
    settle(c, reads);
    return c;
  };
  auto next = [&](Place& c, bool reads) {
    const RopePart& q = p.part[c.part];
    c.h += step;
    if (c.h >= q.heads) return settle(c, reads);
    if (reads) {
      c.x += step * q.xh;
      if constexpr (BWD) c.y += step * plane;
    } else {
      c.to += BWD ? step * q.dh : step * plane;
    }
  };
  auto load = [&](const Place& c, int slot) {
    if (c.unit < p.units) {
      const RopePart& q = p.part[c.part];
      const bool read_x = !BWD || q.weight != nullptr;
      if (kDebugChecks && (c.b < 0 || c.s < 0 || c.s >= p.S || c.b * (int64_t)p.S + c.s >= p.N)) {
        dbg_fail(p.status, kChkRopeRow);
      } else {
        const uint32_t at = ring + slot * (kRows * kVecs * 32) * static_cast<int>(sizeof(LT));
        const int64_t next_x = p.per_warp * q.xh, next_y = p.per_warp * plane;
#pragma unroll
        for (int j = 0; j < kRows; ++j)
#pragma unroll
          for (int i = 0; i < NU; ++i)
            if (in[i] && c.h + mine + j * p.per_warp < q.heads) {
#pragma unroll
              for (int k = 0; k < NL; ++k) {
                const uint32_t dst = at + ((j * kVecs + i * NL + k) * 32) * static_cast<int>(sizeof(LT));
                const int d = k == 0 ? ca[i] : cb[i];
                if (read_x) copy_async<LV * 2>(dst, c.x + j * next_x + d);
                if constexpr (BWD) copy_async<LV * 2>(dst + NU * NL * 32 * sizeof(LT), c.y + j * next_y + d);
              }
            }
      }
    }
    copy_commit();
  };

  // positions of the next unit's token, asked for while this one's rows are worked on
  constexpr int kAngles = kRopeMaxPairs / 32;  // of a lane
  int pos[kAngles];
  uint32_t axes = 0;  // a byte each
#pragma unroll
  for (int k = 0; k < kAngles; ++k)
    if (lane + 32 * k < p.pairs) axes |= static_cast<uint32_t>(p.axis[lane + 32 * k]) << (8 * k);
  auto ask = [&](int unit) {
    if (unit >= p.units) return;
    const int n = unit >> p.log2_split;
    const int b = static_cast<int>((static_cast<uint64_t>(n) * p.s_mul) >> p.s_shift), s = n - b * p.S;
    const int* at = p.at + b * p.pb + s * p.ps;
#pragma unroll
    for (int k = 0; k < kAngles; ++k)
      if (lane + 32 * k < p.pairs) pos[k] = __ldg(at + (axes >> (8 * k) & 255) * p.pa);
  };
  auto turn_token = [&]() {
    float* to = reinterpret_cast<float*>(s_turn);
#pragma unroll
    for (int k = 0; k < kAngles; ++k) {
      const int i = lane + 32 * k;
      if (i >= p.pairs) break;
      const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos[k])) * s_fraction[i];
      // turns · 2^64, signed: half turns are its top 32 bits / 2^31
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn, &cs);
      if constexpr (BWD) sn = -sn;
      // pair i is pair i % VW of unit i / VW
      const int u = i / VW, e = i % VW, ui = u / lanes, ut = u - ui * lanes;
      auto place = [&](int c, int f) { return ((ui * kTurn + c) * lanes + ut) * 4 + f; };
      if constexpr (kByPair) {
        *reinterpret_cast<float4*>(to + place(e, 0)) = make_float4(cs, cs, -sn, sn);
      } else if constexpr (VW == 2) {
        to[place(0, e)] = cs, to[place(0, 2 + e)] = sn, to[place(1, e)] = -sn;
      } else {
        to[place(e / 4, e % 4)] = cs;
        to[place(VW / 4 + e / 4, e % 4)] = sn;
        to[place(2 * (VW / 4) + e / 4, e % 4)] = -sn;
      }
    }
  };

  Place ahead = start(true), here = start(false);
#pragma unroll
  for (int s = 0; s < RT::kRing - 1; ++s) {
    load(ahead, s);
    if (ahead.unit < p.units) next(ahead, true);
  }
  if (p.pairs > 0) ask(here.unit);
  // (what a row waits for longest, its loads and positions, is on its way)
  for (int i = tid; i < p.pairs; i += RT::kThreads) s_fraction[i] = p.turns[i];
  if (mine == 0 && warp == 0)
    for (int q = 0; q < p.n_parts; ++q)
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int e = 0; e < 2 * VW; ++e)
          s_w[q * 16 * lanes + w_at(i, e)] =
              p.part[q].weight && in[i] ? weight_at<F16>(p.part[q], channel(i, e)) : 1.f;
  __syncthreads();
  int slot = 0, last_unit = -1;
  while (here.unit < p.units) {
    if (p.pairs > 0 && here.unit != last_unit) {
      __syncwarp();
      turn_token();
      ask(here.unit + stride);
      __syncwarp();
    }
    last_unit = here.unit;
    load(ahead, slot == 0 ? RT::kRing - 1 : slot - 1);
    if (ahead.unit < p.units) next(ahead, true);
    copy_wait<RT::kRing - 1>();
    const RopePart& q = p.part[here.part];
    const bool norm = q.weight != nullptr;
    const int left = q.heads - here.h, rows_in = left - mine;  // this lane's row j is there if j · per_warp is less
    uint16_t* const to0 = here.to;
    const int64_t next_to = p.per_warp * (BWD ? q.dh : plane);
    const float* weights = s_w + here.part * 16 * lanes;
    const LT(&landed)[kRows][kVecs][32] = s_ring[warp][slot];
    slot = slot + 1 == RT::kRing ? 0 : slot + 1;
    next(here, false);
    if (!norm && !q.turn) {  // only laid out
#pragma unroll
      for (int j = 0; j < kRows; ++j)
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int k = 0; k < NL; ++k)
            if (in[i] && j * p.per_warp < rows_in)
              *reinterpret_cast<LT*>(to0 + j * next_to + (k == 0 ? ca[i] : cb[i])) =
                  landed[j][(BWD ? NU * NL : 0) + i * NL + k][lane];
      continue;
    }

    // J rows of this lane side by side: their weights and angles are read once
    auto work = [&](auto rows) {
      constexpr int J = decltype(rows)::value;
      // the rows as float2; a lane's unit that is not there counts as zero (all of a
      // row that is not there may hold anything: nobody else reads its sums)
      auto widened = [&](int v0, float2(&f)[J][NU][VW]) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int i = 0; i < NU; ++i) {
            LT v[NL];
#pragma unroll
            for (int k = 0; k < NL; ++k) v[k] = landed[j][v0 + i * NL + k][lane];
            if constexpr (VW == 1) {
              f[j][i][0] = make_float2(widen<F16>(v[0]).x, widen<F16>(v[NL - 1]).x);
            } else if constexpr (INTER) {
              const uint32_t* wd = reinterpret_cast<const uint32_t*>(&v[0]);
#pragma unroll
              for (int e = 0; e < VW / 2; ++e) {
                const float2 a = widen<F16>(wd[2 * e]), b = widen<F16>(wd[2 * e + 1]);
                f[j][i][e] = make_float2(a.x, b.x), f[j][i][VW / 2 + e] = make_float2(a.y, b.y);
              }
            } else {
#pragma unroll
              for (int k = 0; k < NL; ++k) {
                const uint32_t* wd = reinterpret_cast<const uint32_t*>(&v[k]);
#pragma unroll
                for (int e = 0; e < LV / 2; ++e) f[j][i][k * (LV / 2) + e] = widen<F16>(wd[e]);
              }
            }
            if (NU > 1 && !in[i]) {
#pragma unroll
              for (int e = 0; e < VW; ++e) f[j][i][e] = both(0.f);
            }
          }
      };
      // y = R(z), or dz = R^T dy (the table holds the other way's sines), in place
      auto turned = [&](float2(&f)[J][NU][VW]) {
        if (!q.turn) return;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const int pair = (t + i * lanes) * VW;
          if (pair >= p.pairs) continue;
          const float4* from = s_turn + i * kTurn * lanes + t;
          if constexpr (VW == 1) {
            const float4 c = from[0];  // cos, cos, -sin, sin
#pragma unroll
            for (int j = 0; j < J; ++j) {
              const float2 z = f[j][i][0];
              f[j][i][0] = __ffma2_rn(z, make_float2(c.x, c.y), __fmul2_rn(make_float2(z.y, z.x), make_float2(c.z, c.w)));
            }
          } else {
            // whether pair e of the unit is turned: all are but in the last one of
            // neighbouring pairs
            auto there = [&](int e) { return !INTER || pair + e < p.pairs; };
#pragma unroll
            for (int c = 0; c < VW / 2; ++c) {
              float2 cs, sn, ns;
              if constexpr (VW == 2) {
                const float4 v = from[0], o = from[lanes];
                cs = make_float2(v.x, v.y), sn = make_float2(v.z, v.w), ns = make_float2(o.x, o.y);
              } else {
                const float4 cv = from[(c / 2) * lanes], sv = from[(VW / 4 + c / 2) * lanes],
                             nv = from[(2 * (VW / 4) + c / 2) * lanes];
                cs = c & 1 ? make_float2(cv.z, cv.w) : make_float2(cv.x, cv.y);
                sn = c & 1 ? make_float2(sv.z, sv.w) : make_float2(sv.x, sv.y);
                ns = c & 1 ? make_float2(nv.z, nv.w) : make_float2(nv.x, nv.y);
              }
#pragma unroll
              for (int j = 0; j < J; ++j) {
                const float2 a = f[j][i][c], b = f[j][i][VW / 2 + c];
                const float2 a1 = __ffma2_rn(a, cs, __fmul2_rn(b, ns)), b1 = __ffma2_rn(a, sn, __fmul2_rn(b, cs));
                f[j][i][c] = make_float2(there(2 * c) ? a1.x : a.x, there(2 * c + 1) ? a1.y : a.y);
                f[j][i][VW / 2 + c] = make_float2(there(2 * c) ? b1.x : b.x, there(2 * c + 1) ? b1.y : b.y);
              }
            }
          }
        }
      };
      float2 w[NU][VW];
      auto read_weights = [&]() {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          if constexpr (VW == 1) {
            w[i][0] = *reinterpret_cast<const float2*>(weights + w_at(i, 0));
          } else {
#pragma unroll
            for (int e = 0; e < VW / 2; ++e) {
              const float4 v = *reinterpret_cast<const float4*>(weights + w_at(i, 4 * e));
              w[i][2 * e] = make_float2(v.x, v.y), w[i][2 * e + 1] = make_float2(v.z, v.w);
            }
          }
        }
      };
      auto store = [&](const float2(&f)[J][NU][VW]) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j * p.per_warp >= rows_in) continue;
          uint16_t* to = to0 + j * next_to;
#pragma unroll
          for (int i = 0; i < NU; ++i) {
            if (!in[i]) continue;
            const float2(&r)[VW] = f[j][i];
            if constexpr (VW == 1) {
              to[ca[i]] = static_cast<uint16_t>(pack_x2<F16>(r[0].x, 0.f));
              to[cb[i]] = static_cast<uint16_t>(pack_x2<F16>(r[0].y, 0.f));
            } else if constexpr (INTER) {
              LT v;
              uint32_t* wd = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
              for (int e = 0; e < VW / 2; ++e) {
                wd[2 * e] = pack_x2<F16>(r[e].x, r[VW / 2 + e].x);
                wd[2 * e + 1] = pack_x2<F16>(r[e].y, r[VW / 2 + e].y);
              }
              *reinterpret_cast<LT*>(to + ca[i]) = v;
            } else {
#pragma unroll
              for (int k = 0; k < NL; ++k) {
                LT v;
                uint32_t* wd = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                for (int e = 0; e < LV / 2; ++e) wd[e] = pack_x2<F16>(r[k * (LV / 2) + e].x, r[k * (LV / 2) + e].y);
                *reinterpret_cast<LT*>(to + (k == 0 ? ca[i] : cb[i])) = v;
              }
            }
          }
        }
      };

      float2 x[J][NU][VW];
      if (!BWD || norm) widened(0, x);
      if constexpr (!BWD) {
        if (norm) {
          float ss[J];
#pragma unroll
          for (int j = 0; j < J; ++j) {
            float2 s2 = both(0.f);
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
              for (int e = 0; e < VW; ++e) s2 = __ffma2_rn(x[j][i][e], x[j][i][e], s2);
            ss[j] = s2.x + s2.y;
          }
          row_sums(ss, t, lanes, first, even);
          read_weights();
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const float2 f = both(rsqrtf(fmaf(ss[j], p.inv_d, p.eps)));
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
              for (int e = 0; e < VW; ++e) x[j][i][e] = __fmul2_rn(x[j][i][e], __fmul2_rn(f, w[i][e]));
          }
        }
        turned(x);
        store(x);
      } else {
        float2 g[J][NU][VW];
        widened(NU * NL, g);
        turned(g);
        if (norm) {
          read_weights();
          float sums[2 * J];
#pragma unroll
          for (int j = 0; j < J; ++j) {
            float2 s2 = both(0.f), g2 = both(0.f);
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
              for (int e = 0; e < VW; ++e) {
                s2 = __ffma2_rn(x[j][i][e], x[j][i][e], s2);
                g2 = __ffma2_rn(__fmul2_rn(g[j][i][e], w[i][e]), x[j][i][e], g2);
              }
            sums[2 * j] = s2.x + s2.y, sums[2 * j + 1] = g2.x + g2.y;
          }
          row_sums(sums, t, lanes, first, even);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const float f = rsqrtf(fmaf(sums[2 * j], p.inv_d, p.eps));
            const float c = f * f * sums[2 * j + 1] * p.inv_d;  // mean(g ⊙ x·r)·r
            auto add = [&](float2(&to_acc)[NU][VW]) {
              if (j * p.per_warp >= rows_in) return;
#pragma unroll
              for (int i = 0; i < NU; ++i)
#pragma unroll
                for (int e = 0; e < VW; ++e)
                  to_acc[i][e] = __ffma2_rn(g[j][i][e], __fmul2_rn(x[j][i][e], both(f)), to_acc[i][e]);
            };
            if (q.slot == 0) add(acc[0]);
            else if (q.slot == 1) add(acc[1]);
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
              for (int e = 0; e < VW; ++e) {
                const float2 d = __ffma2_rn(g[j][i][e], w[i][e], __fmul2_rn(x[j][i][e], both(-c)));
                g[j][i][e] = __fmul2_rn(d, both(f));
              }
          }
        }
        store(g);
      }
    };
    if (left > p.per_warp) work(std::integral_constant<int, kRows>{});
    else work(std::integral_constant<int, 1>{});
  }
  copy_wait<0>();

  if constexpr (BWD) {
    launch_dependents();
    // the CTA's sum of each channel: the rows of its warps in their order
    __shared__ float s_acc[RT::kThreads * 16];
    for (int q = 0; q < p.n_parts; ++q) {
      const RopePart& part = p.part[q];
      if (part.sums == nullptr) continue;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int e = 0; e < 2 * VW; ++e)
          if (in[i]) {
            const float2 v = part.slot == 0 ? acc[0][i][e / 2] : acc[1][i][e / 2];
            s_acc[(warp * p.per_warp + mine) * p.D + channel(i, e)] = e & 1 ? v.y : v.x;
          }
      __syncthreads();
      for (int d = tid; d < p.D; d += RT::kThreads) {
        float s = 0.f;
        for (int r = 0; r < kWarps * p.per_warp; ++r) s += s_acc[r * p.D + d];
        part.sums[(int64_t)blockIdx.x * p.D + d] = s;
      }
    }
  }
}

// dweight[d] = Σ over CTAs: 32 channels a block, 32 runs of CTAs added in order.
struct RopeSums {
  RopeParams p;
  int ctas;
};
template <bool F16>
__global__ void __launch_bounds__(1024) rope_dweight_kernel(const __grid_constant__ RopeSums ps) {
  const RopeParams& p = ps.p;
  const int ctas = ps.ctas;
  const RopePart& q = p.part[blockIdx.y];
  if (q.sums == nullptr) {
    wait_for_previous();
    return;
  }
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + c;
  float v = 0.f;
  wait_for_previous();
  if (d < p.D)
#pragma unroll 8
    for (int i = r; i < ctas; i += 32) v += q.sums[(int64_t)i * p.D + d];
  s[r][c] = v;
  __syncthreads();
  if (r == 0 && d < p.D) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][c];
    if (q.weight_f32) static_cast<float*>(q.dweight)[d] = v;
    else static_cast<uint16_t*>(q.dweight)[d] = static_cast<uint16_t>(pack_x2<F16>(v, 0.f));
  }
}

template <bool F16, bool INTER, int VW, bool BWD>
cudaError_t launch(const RopeParams& p, int ctas, cudaStream_t stream) {
  constexpr int kThreads = RopeTile<BWD>::kThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  // weights of each part, angles of each warp's token
  constexpr int kTurns = 8 / VW * RopeTurns<VW>::kUnit;  // float4 of a lane
  cfg.dynamicSmemBytes = static_cast<size_t>(p.n_parts * 4 + kThreads / 32 * kTurns) * p.lanes * 16;
  cfg.stream = stream;
  auto kern = rope_kernel<F16, INTER, VW, BWD>;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool F16, bool BWD>
cudaError_t launch_shape(const RopeParams& p, RopeShape s, int ctas, cudaStream_t stream) {
  if (s.interleaved) return launch<F16, true, 4, BWD>(p, ctas, stream);
  switch (s.width) {
    case 8: return launch<F16, false, 8, BWD>(p, ctas, stream);
    case 4: return launch<F16, false, 4, BWD>(p, ctas, stream);
    case 2: return launch<F16, false, 2, BWD>(p, ctas, stream);
    case 1: return launch<F16, false, 1, BWD>(p, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int rope_plan(RopeParams& p, RopeShape shape, bool bwd, int sms) {
  const int units = p.D / (2 * shape.width), per_lane = 8 / shape.width;
  p.lanes = (units + per_lane - 1) / per_lane;
  p.per_warp = 32 / p.lanes;
  const int warps = bwd ? RopeTile<true>::kThreads / 32 : RopeTile<false>::kThreads / 32;
  const int resident = sms * warps * (bwd ? RopeTile<true>::kCtas : RopeTile<false>::kCtas);
  int groups = 0;
  const int rows = RopeTile<false>::kRows * p.per_warp;  // of a pass
  for (int i = 0; i < p.n_parts; ++i) groups += (p.part[i].heads + rows - 1) / rows;
  // few tokens: their rows are dealt to several warps, each of which finds the angles
  p.log2_split = 0;
  while (((int64_t)p.N << (p.log2_split + 1)) <= resident && (2 << p.log2_split) <= groups) ++p.log2_split;
  p.split = 1 << p.log2_split;
  p.units = p.N << p.log2_split;
  // every warp the same number of units, as near as it goes
  const int rounds = (p.units + resident - 1) / resident;
  const int used = (p.units + rounds - 1) / rounds;
  return (used + warps - 1) / warps;
}

int rope_most_ctas(int sms) { return sms * RopeTile<true>::kCtas; }

cudaError_t rope_fwd_launch(const RopeParams& p, RopeShape shape, bool f16, int ctas, cudaStream_t stream) {
  return f16 ? launch_shape<true, false>(p, shape, ctas, stream) : launch_shape<false, false>(p, shape, ctas, stream);
}

cudaError_t rope_bwd_launch(const RopeParams& p, RopeShape shape, bool f16, int ctas, cudaStream_t stream) {
  cudaError_t e = f16 ? launch_shape<true, true>(p, shape, ctas, stream) : launch_shape<false, true>(p, shape, ctas, stream);
  if (e != cudaSuccess) return e;
  bool any = false;
  for (int i = 0; i < p.n_parts; ++i) any = any || p.part[i].sums != nullptr;
  if (!any) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((p.D + 31) / 32), static_cast<unsigned>(p.n_parts), 1);
  const RopeSums sums = {p, ctas};
  return f16 ? launch_after(rope_dweight_kernel<true>, grid, 1024, stream, sums)
             : launch_after(rope_dweight_kernel<false>, grid, 1024, stream, sums);
}

}  // namespace ea
