// cross_small_bwd_sm103.cu — gradient of cross-attention where a slice has at most 64
// queries and 64 keys (sm_103a): one CTA a slice, one launch.
//
// Such a slice is less than one tile of the kernels of attn_cross_bwd_sm103.cu, whose
// two launches and pipelines cost more than its work; bound by the latency of
// load, three dependent products and store.  It also has so few weights that their
// rounding to 16 bits does not average out in the sums: here P and dS enter their
// products as two 16-bit terms each (a value and what its rounding left, together 16
// bits or more), which a kernel of this size has the time for.
//
// (Rounded once, the gradients of such slices were up to 1.5 times as far from the
// definition as those of a plain form in the same types.)
//
//   q, k, v and dout lie in shared memory, 128-byte-swizzled rows; S = q·kᵀ and dP =
//   dout·vᵀ by mma.sync in 16 x 32 tiles of 8 warps; P and dS from the registers to
//   shared memory; then dq, dk, dv, each warp a 16-row tile and half of the channels.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "bwd_common.cuh"
#include "cross_common.cuh"
#include "cross_few.h"
#include "mma_sync.cuh"
#include "ptx.cuh"

namespace ea {
namespace {

constexpr int kSmallThreads = 256;
enum : int { kChkSmallRow = 0x5721 };

template <int W>
struct SmallLayout {
  static constexpr int kRow = W * 2;                   // bytes
  static constexpr int kTile = kSmallSide * kRow;
  static constexpr int kPairRow = kSmallSide * 2;
  static constexpr int kPair = kSmallSide * kPairRow;  // a 64 x 64 matrix of 16-bit values
  static constexpr int kQ = 0, kDo = kTile, kK = 2 * kTile, kV = 3 * kTile;
  static constexpr int kP = 4 * kTile;                 // P, its rest, dS, its rest
  static constexpr int kStat = kP + 4 * kPair;         // (lse·log2e, delta) of a row
  static constexpr int kAlloc = kStat + kSmallSide * 8;
  static_assert(kAlloc <= 232448, "shared memory budget exceeded");
};

template <int W, bool F16>
__global__ void __launch_bounds__(kSmallThreads) cross_small_bwd_kernel(const __grid_constant__ SmallBwdParams p) {
  using L = SmallLayout<W>;
  constexpr int kUnits = W / 8;
  extern __shared__ __align__(128) uint8_t small_smem[];
  const uint32_t sb = smem_u32(small_smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int mi = lane >> 3, mr = lane & 7;
  const int bh = static_cast<int>(blockIdx.x);
  const int len = cross_len(p.lens, bh / p.heads, p.Sk, p.status);
  const int64_t q0 = (int64_t)bh * p.rows, k0 = (int64_t)bh * p.Sk;
  auto at = [](int r, int u) -> uint32_t { return static_cast<uint32_t>(r * L::kRow + ((u ^ (r & 7)) << 4)); };
  auto pair_at = [](int r, int u) -> uint32_t { return static_cast<uint32_t>(r * L::kPairRow + ((u ^ (r & 7)) << 4)); };

  // rows and channels that are not there are zero (keys behind the end are not read);
  // delta from out and dout on the way: a row's units lie in neighbouring lanes
  for (int i = tid; i < kSmallSide * kUnits; i += kSmallThreads) {
    const int r = i / kUnits, u = i % kUnits;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const bool q_in = r < p.rows && 8 * u < p.D, k_in = r < len && 8 * u < p.D;
    if (kDebugChecks && ((q_in && (q0 + r) >= (int64_t)p.BH * p.rows) || (k_in && (k0 + r) >= (int64_t)p.BH * p.Sk)))
      dbg_fail(p.status, kChkSmallRow);
    auto read = [&](const uint16_t* t, int64_t row, bool in) {
      return in ? __ldg(reinterpret_cast<const uint4*>(t + row * p.D + 8 * u)) : z;
    };
    const uint4 qv = read(p.q, q0 + r, q_in), dv = read(p.dout, q0 + r, q_in), ov = read(p.out, q0 + r, q_in);
    const uint4 kv = read(p.k, k0 + r, k_in), vv = read(p.v, k0 + r, k_in);
    st_shared_v4(sb + L::kQ + at(r, u), qv.x, qv.y, qv.z, qv.w);
    st_shared_v4(sb + L::kDo + at(r, u), dv.x, dv.y, dv.z, dv.w);
    st_shared_v4(sb + L::kK + at(r, u), kv.x, kv.y, kv.z, kv.w);
    st_shared_v4(sb + L::kV + at(r, u), vv.x, vv.y, vv.z, vv.w);
    float d = dot8<F16>(ov, dv);
#pragma unroll
    for (int off = kUnits / 2; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (u == 0) {
      const float lse = r < p.rows ? __ldg(p.lse + q0 + r) : 0.f;
      st_shared_f32x2(sb + L::kStat + 8 * r, lse * 1.4426950408889634f, d);
      if (r < p.rows) p.delta[q0 + r] = d;
    }
  }
  __syncthreads();

  const int ksteps = (p.D + 15) / 16;
  const int row_tiles = (p.rows + 15) / 16, key_tiles = (len + 15) / 16;
  // ---- S and dP: rows 16·(warp / 2) .., keys 32·(warp % 2) ..
  {
    const int rt = warp >> 1, kt = (warp & 1) * 2;
    float s[4][4], dp[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = dp[n][e] = 0.f;
    if (rt < row_tiles && kt < key_tiles)
      for (int kk = 0; kk < ksteps; ++kk) {
        uint32_t a[4], d[4], b[4];
        const uint32_t own = at(16 * rt + (mi & 1) * 8 + mr, 2 * kk + (mi >> 1));
        ldm4(a, sb + L::kQ + own);
        ldm4(d, sb + L::kDo + own);
#pragma unroll
        for (int n = 0; n < 4; n += 2) {
          const uint32_t theirs = at(16 * kt + 8 * n + (mi >> 1) * 8 + mr, 2 * kk + (mi & 1));
          ldm4(b, sb + L::kK + theirs);
          mma16816<F16>(s[n], a, b[0], b[1]);
          mma16816<F16>(s[n + 1], a, b[2], b[3]);
          ldm4(b, sb + L::kV + theirs);
          mma16816<F16>(dp[n], d, b[0], b[1]);
          mma16816<F16>(dp[n + 1], d, b[2], b[3]);
        }
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 16 * rt + 8 * h + (lane >> 2);
      const float lse2 = ld_shared_f32(sb + L::kStat + 8 * r), delta = ld_shared_f32(sb + L::kStat + 8 * r + 4);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int key = 16 * kt + 8 * n + 2 * (lane & 3);
        float pv[2], ds[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = r < p.rows && key + e < len;
          pv[e] = in ? ex2_approx(fmaf(s[n][2 * h + e], p.scale_log2, -lse2)) : 0.f;
          ds[e] = in ? pv[e] * (dp[n][2 * h + e] - delta) : 0.f;
        }
        auto put = [&](int which, float a, float b) {  // the values, then what their rounding left
          const uint32_t hi = pack_x2<F16>(a, b);
          const uint32_t lo = rest_x2<F16>(make_float2(a, b), hi);
          const uint32_t to = sb + L::kP + which * L::kPair + pair_at(r, key >> 3) + 2 * (key & 7);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(hi) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + L::kPair), "r"(lo) : "memory");
        };
        put(0, pv[0], pv[1]);
        put(2, ds[0], ds[1]);
      }
    }
  }
  __syncthreads();

  // ---- the gradients: a 16-row tile (of queries or keys) and half of the channels a warp
  const int tile = warp >> 1, unit0 = (warp & 1) * (kUnits / 2);
  constexpr int kN = kUnits / 2;  // 8-channel blocks
  // rows from `live` on get 0: their weights are, but 0 times a query or dout that is not
  // finite is not
  auto store = [&](const float(&c)[kN][4], uint16_t* to, int64_t first, int rows, int live, float mul) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 16 * tile + 8 * h + (lane >> 2);
      if (r >= rows) continue;
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const int ch = 8 * (unit0 + n) + 2 * (lane & 3);
        if (ch < p.D)
          *reinterpret_cast<uint32_t*>(to + (first + r) * p.D + ch) =
              r < live ? pack_x2<F16>(c[n][2 * h] * mul, c[n][2 * h + 1] * mul) : 0u;
      }
    }
  };
  // c += M (rows of this tile) · B over `steps` 16-row steps of B; the matrix and its
  // rest, transposed for sums over queries
  auto product = [&](float(&c)[kN][4], int which, bool transposed, int b_tile, int steps) {
    __syncwarp();  // the last one's stores were by row
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[n][e] = 0.f;
    for (int kk = 0; kk < steps; ++kk) {
      uint32_t a[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t m = sb + L::kP + (which + t) * L::kPair;
        if (transposed) ldm4_trans(a[t], m + pair_at(16 * kk + (mi >> 1) * 8 + mr, 2 * tile + (mi & 1)));
        else ldm4(a[t], m + pair_at(16 * tile + (mi & 1) * 8 + mr, 2 * kk + (mi >> 1)));
      }
#pragma unroll
      for (int n = 0; n < kN; n += 2) {
        uint32_t b[4];
        ldm4_trans(b, sb + b_tile + at(16 * kk + (mi & 1) * 8 + mr, unit0 + n + (mi >> 1)));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          mma16816<F16>(c[n], a[t], b[0], b[1]);
          mma16816<F16>(c[n + 1], a[t], b[2], b[3]);
        }
      }
    }
  };
  float c[kN][4];
  if (tile < row_tiles) {
    product(c, 2, false, L::kK, key_tiles);
    store(c, p.dq, q0, p.rows, p.rows, p.scale);
  }
  if (16 * tile < p.Sk) {
    product(c, 2, true, L::kQ, tile < key_tiles ? row_tiles : 0);
    store(c, p.dk, k0, p.Sk, len, p.scale);
    product(c, 0, true, L::kDo, tile < key_tiles ? row_tiles : 0);
    store(c, p.dv, k0, p.Sk, len, 1.f);
  }
}

template <int W, bool F16>
cudaError_t launch_small(const SmallBwdParams& p, cudaStream_t stream) {
  auto kern = cross_small_bwd_kernel<W, F16>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallLayout<W>::kAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.BH), 1, 1);
  cfg.blockDim = dim3(kSmallThreads, 1, 1);
  cfg.dynamicSmemBytes = SmallLayout<W>::kAlloc;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t cross_small_bwd_launch(const SmallBwdParams& p, int width, bool f16, cudaStream_t stream) {
  if (width == 64) return f16 ? launch_small<64, true>(p, stream) : launch_small<64, false>(p, stream);
  if (width == 128) return f16 ? launch_small<128, true>(p, stream) : launch_small<128, false>(p, stream);
  return f16 ? launch_small<256, true>(p, stream) : launch_small<256, false>(p, stream);
}

}  // namespace ea
