// rope_sm103.cu — the heads' norm and rotation and their gradient (sm_103a);
// include/attn_rope.h has the formulas.
//
// Bound by the memory: a training step's rows are read once and written once
// (the gradient reads two tensors), about 8 operations a value.  So the kernels
// are shaped by three things: full-width loads and stores, enough of them in
// flight, and few instructions a value.
//
//   A CTA takes a block of tokens (1 to 8) of one part and all its heads.  The
//   angles of the block's tokens are found once, into shared memory, and serve
//   every head: sine and cosine cost about as much as a row of 16 channels.
//   A thread holds `width` pairs of a row, both channels of each, so that the
//   rotation needs no exchange: two 16-byte loads where pairs are half a row
//   apart, one where they are neighbours.  Rows go to D/16 (or D/8) neighbouring
//   lanes, whatever that number is: the sums over a row are shuffles that stop at
//   its last lane.  Rows are dealt token first, head second, so that a warp's
//   stores run on through y, where a head's tokens follow one another.
//   The next row's loads are issued before this row is worked on.
//
// Angles.  A position adds the fraction inv_freq / 2π of a turn.  It is kept as
// a 64-bit integer in units of 2^-64 turns: position times it, modulo 2^64, is
// the angle without whole turns, exactly, at any position; the top 32 bits then
// go to sincospif.
//
// The gradient of the weights: each thread adds up its channels over all rows
// that its CTA takes, the CTA adds its threads' sums in a fixed order, and a
// second kernel the CTAs'.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "bwd_common.cuh"
#include "ptx.cuh"
#include "rope_impl.h"

namespace ea {
namespace {

constexpr int kMaxTokens = 8;  // of a block
enum : int { kChkRopeRow = 0x6101, kChkRopeCopy = 0x6102 };

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

template <bool F16, int N>
__device__ __forceinline__ void unpack(const typename Vec<N>::T& v, float (&f)[N]) {
  if constexpr (N == 1) {
    f[0] = widen<F16>(v).x;
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 x = widen<F16>(w[i]);
      f[2 * i] = x.x, f[2 * i + 1] = x.y;
    }
  }
}

template <bool F16, int N>
__device__ __forceinline__ typename Vec<N>::T pack(const float (&f)[N]) {
  if constexpr (N == 1) {
    return static_cast<uint16_t>(pack_x2<F16>(f[0], 0.f));
  } else {
    typename Vec<N>::T v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_x2<F16>(f[2 * i], f[2 * i + 1]);
    return v;
  }
}

template <bool F16>
__device__ __forceinline__ float weight_at(const RopePart& q, int d) {
  if (q.weight_f32) return __ldg(static_cast<const float*>(q.weight) + d);
  const uint32_t w = __ldg(static_cast<const unsigned short*>(q.weight) + d);
  return widen<F16>(w).x;
}

// The sum of v over a row's `lanes` lanes, in every one of them.  t: this lane's
// place in its row, first: the row's first lane.  Lanes behind the last row pass
// through with sums of their own.
__device__ __forceinline__ float row_sum(float v, int t, int lanes, int first) {
  for (int off = 1; off < lanes; off <<= 1) {
    const float o = __shfl_down_sync(0xffffffffu, v, off);
    if (t + off < lanes) v += o;
  }
  return __shfl_sync(0xffffffffu, v, first);
}

// One thread's pairs of a row: unit i of NU holds VW pairs.  Where pairs are half a
// row apart their first channels are a .. a+VW-1, the second ones b ..; where
// they are neighbours the unit is the 2·VW channels from a on.
template <bool INTER, int VW>
struct Unit {
  int a, b;     // first channel of either half (b unused if INTER)
  int pair;     // index of the first pair
  bool in;      // whether the unit exists
};



template <bool F16, bool INTER, int VW, bool BWD>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int NU = VW >= 4 ? 1 : 4 / VW;  // units of a thread: a row fits a warp
  constexpr int LV = INTER ? 2 * VW : VW;   // values of one load
  constexpr int NL = INTER ? 1 : 2;         // loads of a unit
  using LT = typename Vec<LV>::T;
  __shared__ float2 s_turn[kMaxTokens * kRopeMaxPairs];  // cos, sin
  __shared__ int2 s_tok[kMaxTokens];                     // batch, token; batch -1: behind the last
  __shared__ float s_w[2 * kRopeMaxPairs];

  const RopePart& q = p.part[blockIdx.y];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = 1 << p.log2_tokens;
  const int split = blockIdx.x % p.head_split, grid = gridDim.x / p.head_split;
  const int rows = q.heads << p.log2_tokens;
  const bool norm = q.weight != nullptr;

  // ---- a part that is only laid out: 16-byte copies
  if (!norm && !q.turn) {
    const int lanes = p.D / 8;
    for (int block = blockIdx.x / p.head_split; block < p.blocks; block += grid) {
      const int total = rows * lanes;
      for (int c = split * kRopeThreads + tid; c < total; c += p.head_split * kRopeThreads) {
        const int row = c / lanes, col = (c - row * lanes) * 8;
        const int n = (block << p.log2_tokens) + (row & (T - 1)), h = row >> p.log2_tokens;
        if (n >= p.B * p.S) continue;
        const int b = n / p.S, s = n - b * p.S;
        if (kDebugChecks && (h >= q.heads || col + 8 > p.D)) {
          dbg_fail(p.status, kChkRopeCopy);
          continue;
        }
        uint16_t* y = q.y + (((int64_t)b * q.heads + h) * p.S + s) * p.D + col;
        if constexpr (BWD) {
          *reinterpret_cast<uint4*>(q.dx + b * q.db + s * q.ds + h * q.dh + col) =
              __ldcs(reinterpret_cast<const uint4*>(y));
        } else {
          *reinterpret_cast<uint4*>(y) =
              __ldcs(reinterpret_cast<const uint4*>(q.x + b * q.xb + s * q.xs + h * q.xh + col));
        }
      }
    }
    return;
  }

  const int pairs = q.turn ? p.pairs : 0;
  const int units = p.D / (2 * VW);
  const int lanes = (units + NU - 1) / NU;  // of a row, at most 32
  const int per_warp = 32 / lanes;
  const int mine = lane / lanes;            // row of the warp's rows; per_warp: none
  const int t = lane - mine * lanes, first = mine * lanes;
  Unit<INTER, VW> unit[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = t + i * lanes;
    unit[i].in = u < units;
    unit[i].pair = u * VW;
    if constexpr (INTER) {
      unit[i].a = u * 2 * VW;
      unit[i].b = 0;
    } else {
      const bool turned = u * VW < pairs;
      unit[i].a = turned ? u * VW : 2 * pairs + (u * VW - pairs);
      unit[i].b = unit[i].a + (turned ? pairs : p.D / 2 - pairs);
    }
  }
  if (norm)
    for (int d = tid; d < p.D; d += kRopeThreads) s_w[d] = weight_at<F16>(q, d);
  __syncthreads();
  // the weights of this thread's channels: the first VW of a unit are its first half
  float w[NU][2 * VW];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 2 * VW; ++e) {
      const int d = INTER || e < VW ? unit[i].a + e : unit[i].b + e - VW;
      w[i][e] = norm && unit[i].in ? s_w[d] : 1.f;
    }
  float acc[BWD ? NU : 1][2 * VW];
  if constexpr (BWD) {
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < 2 * VW; ++e) acc[i][e] = 0.f;
  }

  const int stride = p.head_split * (kRopeThreads / 32) * per_warp;
  const int row0 = (split * (kRopeThreads / 32) + warp) * per_warp + mine;
  for (int block = blockIdx.x / p.head_split; block < p.blocks; block += grid) {
    // ---- the block's tokens and their angles
    __syncthreads();
    if (tid < T) {
      const int n = (block << p.log2_tokens) + tid;
      const int b = n / p.S;
      s_tok[tid] = n < p.B * p.S ? make_int2(b, n - b * p.S) : make_int2(-1, 0);
    }
    for (int c = tid; c < pairs << p.log2_tokens; c += kRopeThreads) {
      const int tok = c / pairs, i = c - tok * pairs;
      const int n = (block << p.log2_tokens) + tok;
      if (n >= p.B * p.S) break;
      const int b = n / p.S, s = n - b * p.S;
      const int64_t at = __ldg(p.at + b * p.pb + s * p.ps + p.axis[i] * p.pa);
      const uint64_t turn = static_cast<uint64_t>(at) * p.turns[i];
      // turns · 2^64, signed: half turns are its top 32 bits / 2^31
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn, &cs);
      s_turn[c] = make_float2(cs, sn);
    }
    __syncthreads();

    LT xv[NU][NL], gv[NU][NL];
    int tok = 0;
    auto load = [&](int row) {
      const int tk = row & (T - 1), h = row >> p.log2_tokens;
      const int2 bs = s_tok[tk];
      if (mine >= per_warp || row >= rows || bs.x < 0) return -1;
      if (kDebugChecks && (h >= q.heads || bs.x >= p.B || bs.y >= p.S)) {
        dbg_fail(p.status, kChkRopeRow);
        return -1;
      }
      const uint16_t* x = q.x + bs.x * q.xb + bs.y * q.xs + h * q.xh;
      const uint16_t* y = q.y + (((int64_t)bs.x * q.heads + h) * p.S + bs.y) * p.D;
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int k = 0; k < NL; ++k) {
          if (!unit[i].in) continue;
          const int d = k == 0 ? unit[i].a : unit[i].b;
          if (!BWD || norm) xv[i][k] = __ldcs(reinterpret_cast<const LT*>(x + d));
          if constexpr (BWD) gv[i][k] = __ldcs(reinterpret_cast<const LT*>(y + d));
        }
      return tk;
    };
    tok = load(row0);
    for (int row = row0; row - mine < rows; row += stride) {
      const int tk = tok, h = row >> p.log2_tokens;
      float x[NU][2 * VW], g[NU][2 * VW];
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int k = 0; k < NL; ++k) {
          float f[LV];
          const bool there = tk >= 0 && unit[i].in;
          if (!BWD || norm) {
            unpack<F16, LV>(xv[i][k], f);
#pragma unroll
            for (int e = 0; e < LV; ++e) x[i][k * LV + e] = there ? f[e] : 0.f;
          }
          if constexpr (BWD) {
            unpack<F16, LV>(gv[i][k], f);
#pragma unroll
            for (int e = 0; e < LV; ++e) g[i][k * LV + e] = there ? f[e] : 0.f;
          }
        }
      tok = load(row + stride);  // the next row's, while this one is worked on

      // y = R(z), or dz = R^T dy, in place in `f`
      auto turned = [&](float(&f)[NU][2 * VW]) {
        if (pairs == 0 || tk < 0) return;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          if (!unit[i].in || unit[i].pair >= pairs) continue;
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            if (INTER && unit[i].pair + e >= pairs) continue;
            const float2 cs = s_turn[tk * pairs + unit[i].pair + e];
            const float sn = BWD ? -cs.y : cs.y;
            float& a = f[i][INTER ? 2 * e : e];
            float& c = f[i][INTER ? 2 * e + 1 : VW + e];
            const float a1 = a * cs.x - c * sn;
            c = a * sn + c * cs.x;
            a = a1;
          }
        }
      };
      if constexpr (!BWD) {
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int e = 0; e < 2 * VW; ++e) ss = fmaf(x[i][e], x[i][e], ss);
          ss = row_sum(ss, t, lanes, first);
          const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
#pragma unroll
          for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int e = 0; e < 2 * VW; ++e) x[i][e] *= r * w[i][e];
        }
        turned(x);
      } else {
        turned(g);
        if (norm) {
          float ss = 0.f, sg = 0.f;
#pragma unroll
          for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int e = 0; e < 2 * VW; ++e) {
              ss = fmaf(x[i][e], x[i][e], ss);
              sg = fmaf(g[i][e] * w[i][e], x[i][e], sg);
            }
          ss = row_sum(ss, t, lanes, first);
          sg = row_sum(sg, t, lanes, first);
          const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
          const float c = r * r * sg * p.inv_d;  // mean(g ⊙ x·r)·r
#pragma unroll
          for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int e = 0; e < 2 * VW; ++e) {
              if (tk >= 0) acc[i][e] = fmaf(g[i][e], x[i][e] * r, acc[i][e]);
              g[i][e] = r * (g[i][e] * w[i][e] - x[i][e] * c);
            }
        }
      }
      if (tk >= 0) {
        const int2 bs = s_tok[tk];
        uint16_t* to = BWD ? q.dx + bs.x * q.db + bs.y * q.ds + h * q.dh
                           : q.y + (((int64_t)bs.x * q.heads + h) * p.S + bs.y) * p.D;
        float(&f)[NU][2 * VW] = BWD ? g : x;
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int k = 0; k < NL; ++k) {
            if (!unit[i].in) continue;
            float o[LV];
#pragma unroll
            for (int e = 0; e < LV; ++e) o[e] = f[i][k * LV + e];
            *reinterpret_cast<LT*>(to + (k == 0 ? unit[i].a : unit[i].b)) = pack<F16, LV>(o);
          }
      }
    }
  }

  if constexpr (BWD) {
    if (q.sums == nullptr) return;
    // the CTA's sum of each channel: rows of the warps, in their order
    __shared__ float s_acc[kRopeThreads * 16];  // [rows of a pass][D]
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < 2 * VW; ++e)
        if (mine < per_warp && unit[i].in)
          s_acc[(warp * per_warp + mine) * p.D +
                (INTER || e < VW ? unit[i].a + e : unit[i].b + e - VW)] = acc[i][e];
    __syncthreads();
    for (int d = tid; d < p.D; d += kRopeThreads) {
      float s = 0.f;
      for (int r = 0; r < (kRopeThreads / 32) * per_warp; ++r) s += s_acc[r * p.D + d];
      q.sums[(int64_t)blockIdx.x * p.D + d] = s;
    }
  }
}

// dweight[d] = Σ over CTAs: 32 channels a block, 32 runs of CTAs added in order.
template <bool F16>
__global__ void __launch_bounds__(1024) rope_dweight_kernel(const __grid_constant__ RopeParams p, int ctas) {
  const RopePart& q = p.part[blockIdx.y];
  if (q.sums == nullptr) return;
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + c;
  float v = 0.f;
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

template <bool F16, bool INTER, int VW>
cudaError_t launch(const RopeParams& p, bool bwd, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(p.n_parts), 1);
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = stream;
  return bwd ? cudaLaunchKernelEx(&cfg, rope_kernel<F16, INTER, VW, true>, p)
             : cudaLaunchKernelEx(&cfg, rope_kernel<F16, INTER, VW, false>, p);
}

template <bool F16>
cudaError_t launch_shape(const RopeParams& p, RopeShape s, bool bwd, int ctas, cudaStream_t stream) {
  if (s.interleaved) return launch<F16, true, 4>(p, bwd, ctas, stream);
  switch (s.width) {
    case 8: return launch<F16, false, 8>(p, bwd, ctas, stream);
    case 4: return launch<F16, false, 4>(p, bwd, ctas, stream);
    case 2: return launch<F16, false, 2>(p, bwd, ctas, stream);
    case 1: return launch<F16, false, 1>(p, bwd, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int rope_bwd_grid(const RopeParams& p, int sms) {
  const int64_t most = static_cast<int64_t>(sms) * 4;
  const int64_t all = static_cast<int64_t>(p.blocks) * p.head_split;
  return static_cast<int>(all < most ? all : most / p.head_split * p.head_split);
}

cudaError_t rope_fwd_launch(const RopeParams& p, RopeShape shape, bool f16, cudaStream_t stream) {
  const int ctas = p.blocks * p.head_split;
  return f16 ? launch_shape<true>(p, shape, false, ctas, stream) : launch_shape<false>(p, shape, false, ctas, stream);
}

cudaError_t rope_bwd_launch(const RopeParams& p, RopeShape shape, bool f16, int sms, cudaStream_t stream) {
  const int ctas = rope_bwd_grid(p, sms);
  cudaError_t e = f16 ? launch_shape<true>(p, shape, true, ctas, stream) : launch_shape<false>(p, shape, true, ctas, stream);
  if (e != cudaSuccess) return e;
  bool any = false;
  for (int i = 0; i < p.n_parts; ++i) any = any || p.part[i].sums != nullptr;
  if (!any) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.D + 31) / 32), static_cast<unsigned>(p.n_parts), 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = stream;
  return f16 ? cudaLaunchKernelEx(&cfg, rope_dweight_kernel<true>, p, ctas)
             : cudaLaunchKernelEx(&cfg, rope_dweight_kernel<false>, p, ctas);
}

}  // namespace ea
