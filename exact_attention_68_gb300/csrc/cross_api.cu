// cross_api.cu — the C ABI declared in include/attn_cross.h: argument checks, how
// the work is cut, tensor maps, workspaces, launch.
//
// No mask goes by the query, so the G query heads that share a key head are one
// slice of G·Sq rows: [batch, q_heads, Sq, D] is [batch·heads, G·Sq, D] as it lies
// in memory.  The kernels see slices of `rows` queries and Sk keys.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "attn_bwd.h"
#include "attn_cross.h"
#include "attn_fwd.h"
#include "attn_host.h"
#include "cross_few.h"
#include "cross_join.h"
#include "tmap.h"

namespace {

using ea::aligned;
using ea::any_overlap;
using ea::Span;

constexpr size_t kNoSpace = 16;  // the size that says no workspace is needed

struct Sizes {
  int64_t BH, rows, Sk, D;
  uint64_t q_bytes, k_bytes, row_bytes;  // q; k; one fp32 a query
};

// The sizes of a call; touches no CUDA API.
attn_status_t check_sizes(const attn_cross_t* c, Sizes* s) {
  if (!c || c->batch < 1 || c->heads < 1 || c->q_heads < 1 || c->Sq < 1 || c->Sk < 1 || c->head_dim < 1)
    return ATTN_ERR_INVALID_ARG;
  if (c->head_dim > 256 || c->head_dim % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  constexpr int64_t most = INT32_MAX - 128;
  if (c->q_heads % c->heads != 0 || c->batch > most || c->heads > most || c->q_heads > most || c->Sq > most ||
      c->Sk > most)
    return ATTN_ERR_INVALID_ARG;
  const int64_t G = c->q_heads / c->heads;
  s->BH = c->batch * c->heads;
  if (s->BH > INT32_MAX || G > most / c->Sq) return ATTN_ERR_INVALID_ARG;
  s->rows = G * c->Sq;
  s->Sk = c->Sk;
  s->D = c->head_dim;
  // a CTA for each tile, half of the head dimension and run of them
  const int64_t tiles = s->rows > s->Sk ? (s->rows + 127) / 128 : (s->Sk + 127) / 128;
  if (s->BH > INT32_MAX / 2 / tiles) return ATTN_ERR_INVALID_ARG;
  const int64_t longest = s->rows > s->Sk ? s->rows : s->Sk;
  if (s->BH > (int64_t(1) << 50) / (longest * s->D)) return ATTN_ERR_INVALID_ARG;
  s->q_bytes = static_cast<uint64_t>(s->BH * s->rows * s->D) * 2;
  s->k_bytes = static_cast<uint64_t>(s->BH * s->Sk * s->D) * 2;
  s->row_bytes = static_cast<uint64_t>(s->BH * s->rows) * 4;
  return ATTN_OK;
}

attn_status_t check_values(float scale, int dtype) {
  if (!std::isfinite(scale) || !(scale > 0.f) || (dtype != ATTN_BF16 && dtype != ATTN_F16)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// Into how many runs the `steps` of each of `units` pieces of work are cut, each
// run on one of `sms` SMs: the number with the shortest expected time.  A run costs
// its steps and `start` more of them; joining costs a launch and the bytes of the
// runs' results, written and read.
int runs_of(int64_t units, int64_t steps, int sms, double step_us, double start, double bytes_per_run) {
  int best = 1;
  double least = 0;
  const int64_t most = steps < ea::kMaxRuns ? steps : ea::kMaxRuns;
  for (int64_t n = 1; n <= most; ++n) {
    if (n > 1 && units > INT32_MAX / 2 / n) break;
    const double waves = static_cast<double>((units * n + sms - 1) / sms);
    double t = waves * (static_cast<double>((steps + n - 1) / n) + start) * step_us;
    if (n > 1) t += 3.0 + 2.0 * static_cast<double>(n) * bytes_per_run / 5e6;
    if (n == 1 || t < least * 0.97) {
      best = static_cast<int>(n);
      least = t;
    }
    if (units * n >= 4 * sms) break;  // more runs would only add joins
  }
  return best;
}

// The plans.  Each is one function and not inlined: a workspace query and the call
// compare the same times, which a compiler that contracts products and sums in one copy
// and not in the other could settle differently.
struct FwdPlan {
  bool few;     // the kernel for few queries
  int cluster;  // its CTAs a slice
  int width, bn, n_qt, n_kt, runs;
  size_t space;
};
__attribute__((noinline)) FwdPlan plan_fwd(const Sizes& s, int sms) {
  FwdPlan f;
  // Few queries of up to 64 channels.  Against the persistent kernel, 16 rows: 128
  // slices of 1500 keys 11.5 us and 13.6, 4 slices of 16384 keys 10.3 and 9.9 (one row
  // 8.3 and 9.7), 256 of 2000 keys 25.2 and 30.3, 16 of 300 keys 6.1 and 6.7.  Two tiles
  // of 16 rows: 16.0 and 13.9, 12.7 and 10.3, 30.8 and 30.3, 8.4 and 6.6; 128 channels,
  // one row: 18.5 and 15.7, 10.8 and 10.6, 44.3 and 42.9, 6.9 and 7.4; 256 channels: 47
  // and 34, 38 and 13.
  f.few = s.rows <= ea::kFewRows && s.D <= ea::kFewWidth;
  if (f.few) {
    const int64_t slices = s.BH;
    // As many CTAs as the SMs hold at once (two each), not more:
    // 128 slices of 64 channels, 300 to 1500 keys, took 14.1 us with one a slice, 11.4
    // with two, 14.2 with four, 22.4 with eight.  A cluster of up to 8 shares a
    // slice; where those leave half of the SMs idle, and there are chunks of keys for
    // more, the keys are cut into runs.
    const int64_t resident = 2 * sms, chunks = (s.Sk + 127) / 128;
    f.cluster = 1, f.runs = 1;
    while (f.cluster < 8 && slices * f.cluster * 2 <= resident && f.cluster * 2 <= chunks) f.cluster *= 2;
    if (f.cluster == 8) {
      int64_t n = resident / (slices * 8);
      if (n > chunks / 16) n = chunks / 16;
      if (n > ea::kMaxRuns) n = ea::kMaxRuns;
      if (n > 2) f.runs = static_cast<int>(n);
    }
    f.space = f.runs > 1 ? static_cast<size_t>(f.runs) * s.BH * s.rows * (s.D + 1) * 4 : kNoSpace;
    return f;
  }
  f.width = ea::forward_head_dim(s.D);
  f.bn = f.width > 128 ? 64 : 128;
  f.n_qt = static_cast<int>((s.rows + ea::kBlockM - 1) / ea::kBlockM);
  f.n_kt = static_cast<int>((s.Sk + f.bn - 1) / f.bn);
  f.runs = runs_of(s.BH * f.n_qt, f.n_kt, sms, f.bn == 64 ? 0.45 : 0.7, 3.0,
                   static_cast<double>(s.BH) * s.rows * s.D * 4);
  f.space = f.runs > 1 ? static_cast<size_t>(f.runs) * s.BH * s.rows * (s.D + 1) * 4 : kNoSpace;
  return f;
}

struct BwdPlan {
  bool small;  // a CTA a slice
  int width, n_qt, n_kt, q_split;
  ea::KvRuns kv;
  size_t dq_space, dk_space, space;  // dk_space: of dk and of dv each
};
__attribute__((noinline)) BwdPlan plan_bwd(const attn_cross_t& c, const Sizes& s, int sms) {
  BwdPlan b;
  std::memset(&b, 0, sizeof(b));
  b.width = ea::kernel_head_dim(s.D);
  // Less than a tile both ways: a CTA a slice.  64 queries and keys, 16 slices of 64
  // channels 5.8 us against 10.4, 512 of them 16.1 against 30.4; of 128 channels 9.0
  // against 12.3 and 26.3 against 38.2.
  b.small = s.rows <= ea::kSmallSide && s.Sk <= ea::kSmallSide;
  if (b.small) {
    b.space = kNoSpace;
    return b;
  }
  const int step = b.width == 256 ? 64 : 128;  // keys of a step
  b.n_qt = static_cast<int>((s.rows + 127) / 128);
  b.n_kt = static_cast<int>((s.Sk + 127) / 128);
  const double us = b.width == 64 ? 1.0 : 1.4;
  b.q_split = runs_of(s.BH * b.n_qt, (s.Sk + step - 1) / step, sms, us, 4.0, static_cast<double>(s.BH) * s.rows * s.D * 4);
  b.kv = ea::plan_kv_runs(c.batch, c.heads, s.Sk, s.rows, s.D, b.width, sms);
  b.dq_space = b.q_split > 1 ? static_cast<size_t>(b.q_split) * s.BH * s.rows * s.D * 4 : 0;
  b.dk_space = b.kv.most_runs > 1 ? static_cast<size_t>(b.kv.most_runs) * s.BH * s.Sk * s.D * 4 : 0;
  b.space = b.dq_space + 2 * b.dk_space;
  if (b.space < kNoSpace) b.space = kNoSpace;
  return b;
}

attn_status_t check_space(const void* workspace, size_t bytes, size_t need) {
  if (need <= kNoSpace) return ATTN_OK;
  if (!workspace || bytes < need) return ATTN_ERR_INVALID_ARG;
  return aligned(workspace, 16) ? ATTN_OK : ATTN_ERR_MISALIGNED;
}

attn_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return ATTN_OK;
  (void)cudaGetLastError();
  return ea::cuda_failure(static_cast<int>(e));
}

}  // namespace

extern "C" {

size_t attn_cross_fwd_workspace(const attn_cross_t* sizes) {
  Sizes s;
  if (check_sizes(sizes, &s) != ATTN_OK) return 0;
  int sms = 0;
  return ea::device_sms(&sms) == ATTN_OK ? plan_fwd(s, sms).space : 0;
}

size_t attn_cross_bwd_workspace(const attn_cross_t* sizes) {
  Sizes s;
  if (check_sizes(sizes, &s) != ATTN_OK) return 0;
  int sms = 0;
  return ea::device_sms(&sms) == ATTN_OK ? plan_bwd(*sizes, s, sms).space : 0;
}

attn_status_t attn_cross_fwd(const attn_cross_t* sizes, const void* q, const void* k, const void* v,
                             const int32_t* lens, void* out, float* lse, float scale, attn_dtype_t dtype,
                             void* workspace, size_t workspace_bytes, uint64_t wait_timeout_ns,
                             cudaStream_t stream) {
  Sizes s;
  attn_status_t st = check_sizes(sizes, &s);
  if (st == ATTN_OK) st = check_values(scale, dtype);
  if (st != ATTN_OK) return st;
  if (!q || !k || !v || !out || !lse) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(lens, 4))
    return ATTN_ERR_MISALIGNED;
  const Span spans[7] = {{q, s.q_bytes, false}, {k, s.k_bytes, false}, {v, s.k_bytes, false},
                         {lens, static_cast<uint64_t>(sizes->batch) * 4, false}, {out, s.q_bytes, true},
                         {lse, s.row_bytes, true}, {workspace, workspace_bytes, true}};
  if (any_overlap(spans, 7)) return ATTN_ERR_INVALID_ARG;
  int* status = nullptr;
  int sms = 0;
  st = ea::current_status_words(&status);
  if (st == ATTN_OK) st = ea::device_sms(&sms);
  if (st != ATTN_OK) return st;
  const FwdPlan f = plan_fwd(s, sms);
  st = check_space(workspace, workspace_bytes, f.space);
  if (st != ATTN_OK) return st;

  const bool f16 = dtype == ATTN_F16;
  ea::JoinFwdParams j;
  float* const part_o = f.runs > 1 ? static_cast<float*>(workspace) : nullptr;
  float* const part_lse = f.runs > 1 ? part_o + static_cast<int64_t>(f.runs) * s.BH * s.rows * s.D : nullptr;
  j.part_o = part_o, j.part_lse = part_lse;
  j.out = static_cast<uint16_t*>(out), j.lse = lse;
  j.rows = s.BH * s.rows;
  j.runs = f.runs, j.D = static_cast<int>(s.D);
  j.lens = lens, j.seq_rows = sizes->heads * s.rows;
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (f.few) {
    ea::FewParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.lens = lens;
    p.out = j.out, p.lse = lse;
    p.part_o = part_o, p.part_lse = part_lse;
    p.status = status;
    p.BH = static_cast<int>(s.BH), p.heads = static_cast<int>(sizes->heads), p.rows = static_cast<int>(s.rows);
    p.Sk = static_cast<int>(s.Sk), p.D = j.D;
    p.cluster = f.cluster, p.runs = f.runs;
    p.scale_log2 = scale_log2;
    cudaError_t e = ea::cross_few_launch(p, f16, stream);
    if (e == cudaSuccess && f.runs > 1) e = ea::join_fwd_launch(j, f16, stream);
    return launched(e);
  }
  ea::Fwd1QParams p;
  std::memset(&p, 0, sizeof(p));
  if (!ea::encode_bhsd_16bit(&p.tm_k, k, s.BH, s.Sk, s.D, f.bn, f16) ||
      !ea::encode_bhsd_16bit(&p.tm_v, v, s.BH, s.Sk, s.D, f.bn, f16) ||
      !ea::encode_bhsd_16bit(&p.tm_o, out, s.BH, s.rows, s.D, 32, f16) ||
      !ea::encode_bhsd_16bit(&p.tm_q, q, s.BH, s.rows, s.D, 128, f16))
    return ea::cuda_failure(ea::kErrTensorMap);
  p.q = static_cast<const uint16_t*>(q);
  p.lse = lse;
  p.status = status;
  p.BH = static_cast<int>(s.BH);
  p.S = static_cast<int>(s.rows);
  p.d_cols = static_cast<int>(s.D);
  p.n_qt = f.n_qt;
  p.n_kt = f.n_kt;
  p.scale_log2 = scale_log2;
  p.timeout_ns = wait_timeout_ns;
  p.Sk = static_cast<int>(s.Sk);
  p.lens = lens;
  p.heads = static_cast<int>(sizes->heads);
  p.n_split = f.runs;
  p.part_o = part_o, p.part_lse = part_lse;
  cudaError_t e = f.width <= 128 ? ea::fwd1qp_launch(p, f.width, ea::kMaskCross, f16, stream)
                                 : ea::fwd1q_launch(p, f.width, ea::kMaskCross, f16, stream);
  if (e == cudaSuccess && f.runs > 1) e = ea::join_fwd_launch(j, f16, stream);
  return launched(e);
}

attn_status_t attn_cross_bwd(const attn_cross_t* sizes, const void* q, const void* k, const void* v,
                             const int32_t* lens, const void* out, const float* lse, const void* dout,
                             void* dq, void* dk, void* dv, float* delta, float scale, attn_dtype_t dtype,
                             void* workspace, size_t workspace_bytes, uint64_t wait_timeout_ns,
                             cudaStream_t stream) {
  Sizes s;
  attn_status_t st = check_sizes(sizes, &s);
  if (st == ATTN_OK) st = check_values(scale, dtype);
  if (st != ATTN_OK) return st;
  if (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv || !delta) return ATTN_ERR_INVALID_ARG;
  const void* by16[8] = {q, k, v, out, dout, dq, dk, dv};
  for (const void* a : by16)
    if (!aligned(a, 16)) return ATTN_ERR_MISALIGNED;
  if (!aligned(lse, 4) || !aligned(delta, 4) || !aligned(lens, 4)) return ATTN_ERR_MISALIGNED;
  const Span spans[12] = {{q, s.q_bytes, false}, {k, s.k_bytes, false}, {v, s.k_bytes, false},
                          {lens, static_cast<uint64_t>(sizes->batch) * 4, false}, {out, s.q_bytes, false},
                          {lse, s.row_bytes, false}, {dout, s.q_bytes, false}, {dq, s.q_bytes, true},
                          {dk, s.k_bytes, true}, {dv, s.k_bytes, true}, {delta, s.row_bytes, true},
                          {workspace, workspace_bytes, true}};
  if (any_overlap(spans, 12)) return ATTN_ERR_INVALID_ARG;
  int* status = nullptr;
  int sms = 0;
  st = ea::current_status_words(&status);
  if (st == ATTN_OK) st = ea::device_sms(&sms);
  if (st != ATTN_OK) return st;
  const BwdPlan b = plan_bwd(*sizes, s, sms);
  st = check_space(workspace, workspace_bytes, b.space);
  if (st != ATTN_OK) return st;

  const bool f16 = dtype == ATTN_F16;
  if (b.small) {
    ea::SmallBwdParams p;
    p.q = static_cast<const uint16_t*>(q), p.k = static_cast<const uint16_t*>(k), p.v = static_cast<const uint16_t*>(v);
    p.lens = lens;
    p.out = static_cast<const uint16_t*>(out), p.lse = lse, p.dout = static_cast<const uint16_t*>(dout);
    p.dq = static_cast<uint16_t*>(dq), p.dk = static_cast<uint16_t*>(dk), p.dv = static_cast<uint16_t*>(dv);
    p.delta = delta;
    p.status = status;
    p.BH = static_cast<int>(s.BH), p.heads = static_cast<int>(sizes->heads), p.rows = static_cast<int>(s.rows);
    p.Sk = static_cast<int>(s.Sk), p.D = static_cast<int>(s.D);
    p.scale = scale, p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    return launched(ea::cross_small_bwd_launch(p, b.width, f16, stream));
  }
  ea::BwdParams p;
  std::memset(&p, 0, sizeof(p));
  auto map = [&](CUtensorMap* m, const void* t, int64_t n, uint32_t box) {
    return ea::encode_bhsd_16bit(m, t, s.BH, n, s.D, box, f16);
  };
  if (!map(&p.tm_q, q, s.rows, 128) || !map(&p.tm_k, k, s.Sk, 128) || !map(&p.tm_v, v, s.Sk, 128) ||
      !map(&p.tm_do, dout, s.rows, 128) || !map(&p.tm_out, out, s.rows, 128) || !map(&p.tm_dq, dq, s.rows, 32) || !map(&p.tm_dk, dk, s.Sk, 32) ||
      !map(&p.tm_dv, dv, s.Sk, 32))
    return ea::cuda_failure(ea::kErrTensorMap);
  if (b.width == 256 && (!map(&p.tm_q64, q, s.rows, 64) || !map(&p.tm_k64, k, s.Sk, 64) ||
                         !map(&p.tm_v64, v, s.Sk, 64) || !map(&p.tm_do64, dout, s.rows, 64)))
    return ea::cuda_failure(ea::kErrTensorMap);
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.out = static_cast<const uint16_t*>(out);
  p.dout = static_cast<const uint16_t*>(dout);
  p.dk = static_cast<uint16_t*>(dk);
  p.dv = static_cast<uint16_t*>(dv);
  p.lse = lse;
  p.delta = delta;
  p.status = status;
  p.BH = static_cast<int>(s.BH);
  p.S = static_cast<int>(s.rows);
  p.d_cols = static_cast<int>(s.D);
  p.scale = scale;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.timeout_ns = wait_timeout_ns;
  p.Sk = static_cast<int>(s.Sk);
  p.lens = lens;
  p.heads = static_cast<int>(sizes->heads);
  p.sms = sms;
  p.n_qt = b.n_qt, p.n_kt = b.n_kt;
  p.q_split = b.q_split, p.kv = b.kv;
  p.part_dq = static_cast<float*>(workspace);
  p.part_dk = p.part_dq + b.dq_space / 4;
  p.part_dv = p.part_dk + b.dk_space / 4;
  cudaError_t e = b.width == 256 ? ea::bwd256_launch(p, ea::kMaskCross, f16, stream)
                                 : ea::cross_bwd_launch(p, b.width, f16, stream);
  ea::JoinSumParams j[ea::kMaxSums];
  std::memset(j, 0, sizeof(j));
  int sums = 0;
  if (b.q_split > 1) {
    ea::JoinSumParams& r = j[sums++];
    r.part = p.part_dq, r.to = static_cast<uint16_t*>(dq);
    r.rows = s.BH * s.rows, r.runs = b.q_split, r.D = p.d_cols, r.mul = scale;
  }
  for (int i = 0; i < 2 && b.kv.most_runs > 1; ++i) {
    ea::JoinSumParams& r = j[sums++];
    r.part = i == 0 ? p.part_dk : p.part_dv;
    r.to = i == 0 ? p.dk : p.dv;
    r.rows = s.BH * s.Sk, r.D = p.d_cols, r.mul = i == 0 ? scale : 1.f;
    r.of_keys = true, r.kv = b.kv, r.lens = lens;
  }
  if (e == cudaSuccess && sums) e = ea::join_sum_launch(j, sums, f16, stream);
  return launched(e);
}

}  // extern "C"
