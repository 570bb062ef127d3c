// attn_bwd.h — parameters and launch entry of the attention backward kernels,
// shared by the host API and the kernel translation unit (no device code).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

#include "cross_runs.h"
#include "schedule.h"

namespace ea {

// Both backward kernels: warps 0-7 elementwise (two groups of four warps, one
// per half of a tile's 128 columns), warp 8 tcgen05 issuer, warp 9 producer.
constexpr int kBwdThreads = 320;

struct BwdParams {
  CUtensorMap tm_q;   // q as (D, S, B·H), box 64 x 128 rows, 128-byte swizzle
  CUtensorMap tm_k;   // k, same box
  CUtensorMap tm_v;   // v, same box
  CUtensorMap tm_do;  // dout, same box
  CUtensorMap tm_dq;  // dq, box 64 x 32 rows (one warp's rows)
  CUtensorMap tm_dk;  // dk, same
  CUtensorMap tm_dv;  // dv, same
  CUtensorMap tm_out; // out, box 64 x 128 rows (cross-attention's dq kernel)
  // 256-column kernels only (head dimension above 128): boxes of 64 columns x
  // 64 rows, for the 64-key (K, V) and 64-query (Q, dout) steps
  CUtensorMap tm_q64;
  CUtensorMap tm_k64;
  CUtensorMap tm_v64;
  CUtensorMap tm_do64;
  const uint16_t* q;     // 16-bit [B·H, S, d_cols]: rows read into TMEM by the dq kernel
  const uint16_t* k;     // 16-bit [B·H, S, d_cols]: rows read into TMEM by the dk/dv kernel
  const uint16_t* v;     // 16-bit [B·H, S, d_cols]: rows read into TMEM by the dk/dv kernel
  const uint16_t* out;   // 16-bit [B·H, S, d_cols]: forward output (rows read for delta)
  const uint16_t* dout;  // 16-bit [B·H, S, d_cols]
  const float* lse;      // [B·H, S]: natural-log logsumexp saved by the forward
  uint16_t* dk;          // 16-bit [B·H, Sk, d_cols] (kMaskCross: rows without keys are zeroed)
  uint16_t* dv;
  float* delta;          // [B·H, S]: rowsum(dout ⊙ out), written by the dq kernel
  int* status;           // device status word pair (error bits, first wait site)
  int BH, S;
  int d_cols;            // the tensors' head dimension (<= the kernel's D, a multiple
                         // of 8); the kernel's columns past it are zero
  int n_t;               // ceil(S / 128): tiles along the sequence
  UnitSchedule sched;    // CTA index -> (b·H + h, unit level): the level of a Q tile i
                         // is i, of a K/V tile j is n_t - 1 - j (both cost level + 1
                         // tile-steps under the causal mask)
  float scale;           // softmax scale
  float scale_log2;      // scale · log2(e)
  uint64_t timeout_ns;
  // kMaskCross only (attn_fwd.h).  Rows of a slice are the G·Sq queries of the heads
  // that share its key head, S of them in n_qt tiles.
  int Sk;               // keys of a slice: k, v, dk, dv are (D, Sk, BH)
  const int* lens;      // [BH / heads] keys that are there; null: all Sk
  int heads;            // key heads of one sequence
  int sms;              // of the device
  int n_qt, n_kt;       // ceil(S / 128), ceil(Sk / 128)
  int q_split;          // runs of K/V tiles that a Q tile's dq is summed over
  KvRuns kv;            // the runs of Q tiles that a K/V tile's dk, dv are summed over
  float* part_dq;       // [q_split, BH, S, d_cols] if q_split > 1: each run's sum, unscaled
  float* part_dk;       // [runs, BH, Sk, d_cols] if there are several: the same of dk and dv
  float* part_dv;
};

// kMaskCross: whether P and dS enter their products in two 16-bit terms each, as in the
// kernel of at most 64 queries and keys.  Rounded once, a gradient is 1.4 times as far
// from the definition as the plain form's, its own rounding and theirs; but where a call
// has few queries a handful of weights decide: of calls with at most 512, 40 of 1152
// gradients were 1.5 to 2.1 times as far off, of larger ones 1 of 1584 (1.53).  Two terms
// cost 128 slices of one query over 1500 keys of 64 channels 55.8 us against 50.0, of
// 128 channels 79.9 against 73.4, of 256 224 against 207.
inline bool two_terms(const BwdParams& p) { return p.S <= 128 && (long long)p.BH * p.S <= 512; }

// Launches the dq kernel (which also writes delta) and then the dk/dv kernel
// on `stream`.  f16: the 16-bit tensors are fp16 (else bf16).
cudaError_t bwd_launch(const BwdParams& p, int D, bool causal, bool f16, cudaStream_t stream);

// Cross-attention's dq and dk/dv kernels for head dimensions up to 128.
cudaError_t cross_bwd_launch(const BwdParams& p, int D, bool f16, cudaStream_t stream);

// The same for head dimensions above 128 (kernels 256 columns wide): the dq
// kernel, then the dk/dv kernel with one CTA per K/V tile and half of the
// head dimension.
cudaError_t bwd256_launch(const BwdParams& p, int mask, bool f16, cudaStream_t stream);

}  // namespace ea
