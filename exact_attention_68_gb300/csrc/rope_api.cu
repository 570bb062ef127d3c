// rope_api.cu — the C ABI declared in include/attn_rope.h: argument checks,
// the angles' fixed-point fractions, launch.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "attn_host.h"
#include "attn_rope.h"
#include "rope_impl.h"

static_assert(ea::kRopeMaxParts == ATTN_ROPE_MAX_PARTS, "parts of a call");

namespace {

using ea::aligned;
using ea::overlaps;

constexpr size_t kNoSpace = 16;  // the size that says no workspace is needed

// A tensor [B, S, heads, D] by its strides, in bytes from its first value to behind its last.
struct View {
  const void* p;
  int64_t b, s, h;
};

// Strides a view may have: what they span stays below 2^60 values, so that extents in
// bytes fit 64 bits.
bool strides_ok(int64_t b, int64_t s, int64_t h, int64_t B, int64_t S, int64_t H) {
  constexpr int64_t most = int64_t(1) << 58;
  auto spans = [](int64_t stride, int64_t n) { return stride >= 0 && stride % 8 == 0 && stride <= most / n; };
  return spans(b, B) && spans(s, S) && spans(h, H);
}
uint64_t extent(const View& v, int64_t B, int64_t S, int64_t H, int64_t D) {
  return static_cast<uint64_t>((B - 1) * v.b + (S - 1) * v.s + (H - 1) * v.h + D) * 2;
}

// Whether no two of a view's values share a place: each stride, from the
// smallest on, goes past all that the smaller ones reach.
bool separate(const View& v, int64_t B, int64_t S, int64_t H, int64_t D) {
  int64_t stride[3] = {v.b, v.s, v.h}, size[3] = {B, S, H};
  int64_t reach = D;
  for (int done = 0; done < 3; ++done) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (size[i] > 1 && (at < 0 || stride[i] < stride[at])) at = i;
    if (at < 0) return true;
    if (stride[at] < reach) return false;
    reach += stride[at] * (size[at] - 1);
    size[at] = 1;
  }
  return true;
}

// Whether two views, as parts of a packed tensor are, share no place; neither has two
// values in one place (separate).  They lie apart as ranges, or do so in each block of
// the outermost dimension: its stride T is that of both, and block i of both lies
// within the same T values.
bool apart(const View& a, int64_t ha, const View& b, int64_t hb, int64_t B, int64_t S, int64_t D) {
  const char *pa = static_cast<const char*>(a.p), *pb = static_cast<const char*>(b.p);
  if (pb < pa) return apart(b, hb, a, ha, B, S, D);
  const int64_t delta = (pb - pa) / 2;
  const int64_t sa[3] = {a.b, a.s, a.h}, sb[3] = {b.b, b.s, b.h}, na[3] = {B, S, ha}, nb[3] = {B, S, hb};
  bool done[3] = {false, false, false};
  int64_t ra = D, rb = D;  // what a block reaches
  for (int i = 0; i < 3; ++i) ra += (na[i] - 1) * sa[i], rb += (nb[i] - 1) * sb[i];
  for (;;) {
    if (delta >= ra) return true;
    int top = -1;
    int64_t T = 0;
    for (int i = 0; i < 3; ++i) {
      const int64_t stride = na[i] > 1 ? sa[i] : nb[i] > 1 ? sb[i] : 0;
      if (!done[i] && stride > T) top = i, T = stride;
    }
    if (top < 0 || (na[top] > 1 && nb[top] > 1 && sa[top] != sb[top])) return false;
    ra -= (na[top] - 1) * sa[top], rb -= (nb[top] - 1) * sb[top];
    if (ra > T || delta + rb > T) return false;
    done[top] = true;
  }
}

attn_status_t check_sizes(const attn_rope_part_t* parts, int n, int64_t B, int64_t S, int64_t D) {
  if (!parts || n < 1 || n > ATTN_ROPE_MAX_PARTS) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || S < 1 || D < 1) return ATTN_ERR_INVALID_ARG;
  if (D > 256 || D % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  constexpr int64_t tokens = (int64_t(1) << 30) - 1;
  if (B > tokens || S > tokens / B) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (parts[i].heads < 1 || parts[i].heads > 65535 || parts[i].heads > INT32_MAX / (B * S)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

attn_status_t check(const attn_rope_part_t* parts, int n, const attn_rope_t* rope,
                    const attn_rope_positions_t* at, int64_t B, int64_t S, int64_t D, float eps, int dtype,
                    bool bwd, const void* workspace, uint64_t space) {
  attn_status_t s = check_sizes(parts, n, B, S, D);
  if (s != ATTN_OK) return s;
  if (dtype != ATTN_BF16 && dtype != ATTN_F16) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return ATTN_ERR_INVALID_ARG;
  bool turn = false;
  for (int i = 0; i < n; ++i) {
    const attn_rope_part_t& q = parts[i];
    const bool reads_x = !bwd || q.weight;
    if ((reads_x && !q.x) || !q.y || (bwd && !q.dx)) return ATTN_ERR_INVALID_ARG;
    if ((q.turn != 0 && q.turn != 1) || (q.weight_f32 != 0 && q.weight_f32 != 1)) return ATTN_ERR_INVALID_ARG;
    if (bwd && q.dweight && !q.weight) return ATTN_ERR_INVALID_ARG;
    if (reads_x && !strides_ok(q.stride_b, q.stride_s, q.stride_h, B, S, q.heads)) return ATTN_ERR_INVALID_ARG;
    if (bwd && (!strides_ok(q.dx_stride_b, q.dx_stride_s, q.dx_stride_h, B, S, q.heads) ||
                !separate({q.dx, q.dx_stride_b, q.dx_stride_s, q.dx_stride_h}, B, S, q.heads, D)))
      return ATTN_ERR_INVALID_ARG;
    if ((reads_x && !aligned(q.x, 16)) || !aligned(q.y, 16) || (bwd && !aligned(q.dx, 16)) ||
        !aligned(q.weight, 4) || (bwd && !aligned(q.dweight, 4)))
      return ATTN_ERR_MISALIGNED;
    turn = turn || q.turn;
  }
  if (turn) {
    if (!rope || !at || !at->at || (rope->pairs > 0 && !rope->inv_freq)) return ATTN_ERR_INVALID_ARG;
    if (rope->pairs < 0 || rope->pairs > D / 2) return ATTN_ERR_INVALID_ARG;
    if (rope->interleaved != 0 && rope->interleaved != 1) return ATTN_ERR_INVALID_ARG;
    if (at->axes < 1 || at->axes > ATTN_ROPE_MAX_AXES) return ATTN_ERR_INVALID_ARG;
    constexpr int64_t most = int64_t(1) << 40;
    if (at->stride_b < 0 || at->stride_s < 0 || at->stride_a < 0 || at->stride_b > most || at->stride_s > most ||
        at->stride_a > most / 8 || (B - 1) > most / (at->stride_b + 1) || (S - 1) > most / (at->stride_s + 1))
      return ATTN_ERR_INVALID_ARG;
    if (!aligned(at->at, 4)) return ATTN_ERR_MISALIGNED;
    for (int64_t i = 0; i < rope->pairs; ++i) {
      if (!std::isfinite(rope->inv_freq[i]) || std::fabs(rope->inv_freq[i]) > 1048576.0) return ATTN_ERR_INVALID_ARG;
      if (rope->axis && rope->axis[i] >= at->axes) return ATTN_ERR_INVALID_ARG;
    }
  }
  // a tensor that is written overlaps nothing that is read, nor another one
  const uint64_t pos_bytes = turn ? static_cast<uint64_t>((B - 1) * at->stride_b + (S - 1) * at->stride_s +
                                                          (at->axes - 1) * at->stride_a + 1) * 4
                                  : 0;
  for (int i = 0; i < n; ++i) {
    const attn_rope_part_t& q = parts[i];
    const uint64_t yn = static_cast<uint64_t>(B * q.heads * S * D) * 2;
    const View dx = {q.dx, q.dx_stride_b, q.dx_stride_s, q.dx_stride_h};
    const void* w = bwd ? q.dx : q.y;
    const uint64_t wn = bwd ? extent(dx, B, S, q.heads, D) : yn;
    const uint64_t gn = bwd && q.dweight ? static_cast<uint64_t>(D) * (q.weight_f32 ? 4 : 2) : 0;
    // the workspace is written too
    auto in_space = [&](const void* p, uint64_t bytes) {
      return workspace && space && p && bytes && overlaps(workspace, space, p, bytes);
    };
    if (bwd && (in_space(w, wn) || in_space(q.dweight, gn) || in_space(q.y, yn) || in_space(q.weight, static_cast<uint64_t>(D) * (q.weight_f32 ? 4 : 2)) ||
                (q.weight && in_space(q.x, extent({q.x, q.stride_b, q.stride_s, q.stride_h}, B, S, q.heads, D))) ||
                (turn && in_space(at->at, pos_bytes))))
      return ATTN_ERR_INVALID_ARG;
    auto hit = [&](const void* p, uint64_t bytes) {
      return p && bytes && (overlaps(w, wn, p, bytes) || (gn && overlaps(q.dweight, gn, p, bytes)));
    };
    if (turn && hit(at->at, pos_bytes)) return ATTN_ERR_INVALID_ARG;
    if (gn && overlaps(q.dweight, gn, w, wn)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < n; ++j) {
      const attn_rope_part_t& r = parts[j];
      if (!bwd || r.weight) {
        const View x = {r.x, r.stride_b, r.stride_s, r.stride_h};
        if (hit(r.x, extent(x, B, S, r.heads, D))) return ATTN_ERR_INVALID_ARG;
      }
      if (hit(r.weight, static_cast<uint64_t>(D) * (r.weight_f32 ? 4 : 2))) return ATTN_ERR_INVALID_ARG;
      const uint64_t rn = static_cast<uint64_t>(B * r.heads * S * D) * 2;
      if (bwd ? hit(r.y, rn) : (j != i && hit(r.y, rn))) return ATTN_ERR_INVALID_ARG;
      if (!bwd || j <= i) continue;
      const View other = {r.dx, r.dx_stride_b, r.dx_stride_s, r.dx_stride_h};
      const uint64_t on = extent(other, B, S, r.heads, D);
      if (overlaps(w, wn, r.dx, on) && !apart(dx, q.heads, other, r.heads, B, S, D)) return ATTN_ERR_INVALID_ARG;
      if (r.dweight) {
        const uint64_t dn = static_cast<uint64_t>(D) * (r.weight_f32 ? 4 : 2);
        if (hit(r.dweight, dn)) return ATTN_ERR_INVALID_ARG;
      }
      if (gn && overlaps(q.dweight, gn, r.dx, on)) return ATTN_ERR_INVALID_ARG;
    }
  }
  return ATTN_OK;
}

// f radians as a fraction of a turn in units of 2^-64, modulo one turn.  f / 2π
// in two doubles: the product with the rounded 1/2π, and what that and the
// product's rounding left out.
uint64_t turn_fraction(double f) {
  constexpr double inv = 0x1.45f306dc9c883p-3, inv_low = -0x1.6b01ec5417056p-57;  // 1/2π and the rest
  const double hi = f * inv;
  const double lo = std::fma(f, inv, -hi) + f * inv_low;
  const double part = hi - std::rint(hi);  // exact
  const int64_t a = std::llrint(part * 0x1p62), b = std::llrint(lo * 0x1p64);
  return (static_cast<uint64_t>(a) << 2) + static_cast<uint64_t>(b);
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// Sizes, and the division of a token's number by S as a product: with l bits of S,
// ceil(2^(30 + l) / S) is off by less than one in 2^(30 + l) / S, which no token
// below 2^30 sees.
void set_sizes(ea::RopeParams& p, int64_t B, int64_t S, int64_t D) {
  p.N = static_cast<int>(B * S), p.S = static_cast<int>(S), p.D = static_cast<int>(D);
  p.inv_d = 1.f / static_cast<float>(D);
  int l = 0;
  while ((int64_t(1) << l) < S) ++l;
  p.s_shift = 30 + l;
  p.s_mul = ((uint64_t(1) << p.s_shift) + S - 1) / S;
}

// The vectors that a call's rows go in.  Pairs half a row apart: vectors that divide
// the turned half and the rest's.  All parts of a launch go the same way.
ea::RopeShape shape_of(int64_t D, bool turn, int pairs, bool interleaved) {
  if (turn && interleaved) return {true, 4};
  return {false, gcd(gcd(8, pairs), static_cast<int>(D) / 2 - pairs)};
}

// Parts of one launch: at most two whose weights have a gradient, which a thread
// adds up in registers.
int parts_of_launch(const attn_rope_part_t* parts, int n, bool bwd) {
  int weighted = 0;
  for (int i = 0; i < n; ++i)
    if (bwd && parts[i].dweight && ++weighted > 2) return i;
  return n;
}

// One launch of n parts.  With `need`, only adds the workspace it needs to *need.
attn_status_t launch(const attn_rope_part_t* parts, int n, const attn_rope_t* rope, const attn_rope_positions_t* at,
                     int64_t B, int64_t S, int64_t D, float eps, int dtype, int sms, int* status, float* sums,
                     size_t* need, bool bwd, cudaStream_t stream) {
  ea::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  set_sizes(p, B, S, D);
  p.n_parts = n;
  p.eps = eps;
  p.status = status;
  bool turn = false;
  int slot = 0;
  for (int i = 0; i < n; ++i) {
    const attn_rope_part_t& q = parts[i];
    ea::RopePart& r = p.part[i];
    r.x = static_cast<const uint16_t*>(q.x);
    r.xb = q.stride_b, r.xs = q.stride_s, r.xh = q.stride_h;
    r.y = static_cast<uint16_t*>(q.y);
    r.weight = q.weight;
    r.weight_f32 = q.weight_f32;
    r.heads = static_cast<int>(q.heads);
    r.slot = -1;
    if (bwd) {
      r.dx = static_cast<uint16_t*>(q.dx);
      r.db = q.dx_stride_b, r.ds = q.dx_stride_s, r.dh = q.dx_stride_h;
      r.dweight = q.dweight;
      if (q.dweight) r.slot = slot++;
    }
    r.turn = q.turn && rope && rope->pairs > 0;
    turn = turn || r.turn;
  }
  if (turn) {
    p.pairs = static_cast<int>(rope->pairs);
    p.at = at->at;
    p.pb = at->stride_b, p.ps = at->stride_s, p.pa = at->stride_a;
  }
  const ea::RopeShape shape = shape_of(D, turn, p.pairs, turn && rope->interleaved);
  const int ctas = ea::rope_plan(p, shape, bwd, sms);
  if (need) {
    *need += static_cast<size_t>(slot) * ctas * D * 4;
    return ATTN_OK;
  }
  if (turn)
    for (int i = 0; i < p.pairs; ++i) {
      p.turns[i] = turn_fraction(rope->inv_freq[i]);
      p.axis[i] = rope->axis ? rope->axis[i] : 0;
    }
  for (int i = 0; i < n; ++i)
    if (p.part[i].slot >= 0) p.part[i].sums = sums + static_cast<int64_t>(p.part[i].slot) * ctas * D;
  const cudaError_t e = bwd ? ea::rope_bwd_launch(p, shape, dtype == ATTN_F16, ctas, stream)
                            : ea::rope_fwd_launch(p, shape, dtype == ATTN_F16, ctas, stream);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return ea::cuda_failure(static_cast<int>(e));
  }
  return ATTN_OK;
}

attn_status_t run(const attn_rope_part_t* parts, int n, const attn_rope_t* rope,
                  const attn_rope_positions_t* at, int64_t B, int64_t S, int64_t D, float eps, int dtype,
                  void* workspace, size_t space, bool bwd, cudaStream_t stream) {
  int* status = nullptr;
  int sms = 0;
  attn_status_t st = ea::current_status_words(&status);
  if (st == ATTN_OK) st = ea::device_sms(&sms);
  if (st != ATTN_OK) return st;
  float* sums = static_cast<float*>(workspace);
  size_t need = 0;
  for (int i = 0, m; bwd && i < n; i += m) {
    m = parts_of_launch(parts + i, n - i, bwd);
    launch(parts + i, m, rope, at, B, S, D, eps, dtype, sms, status, nullptr, &need, bwd, stream);
  }
  if (need && (!workspace || space < need)) return ATTN_ERR_INVALID_ARG;
  if (need && !aligned(workspace, 16)) return ATTN_ERR_MISALIGNED;
  // launches follow one another on the stream: they share the workspace
  for (int i = 0, m; i < n && st == ATTN_OK; i += m) {
    m = parts_of_launch(parts + i, n - i, bwd);
    st = launch(parts + i, m, rope, at, B, S, D, eps, dtype, sms, status, sums, nullptr, bwd, stream);
  }
  return st;
}

}  // namespace

extern "C" {

attn_status_t attn_rope_fwd(const attn_rope_part_t* parts, int n, const attn_rope_t* rope,
                            const attn_rope_positions_t* positions, int64_t B, int64_t S, int64_t D,
                            float eps, attn_dtype_t dtype, cudaStream_t stream) {
  const attn_status_t s = check(parts, n, rope, positions, B, S, D, eps, dtype, false, nullptr, 0);
  if (s != ATTN_OK) return s;
  return run(parts, n, rope, positions, B, S, D, eps, dtype, nullptr, 0, false, stream);
}

size_t attn_rope_bwd_workspace(const attn_rope_part_t* parts, int n, int64_t B, int64_t S, int64_t D) {
  if (check_sizes(parts, n, B, S, D) != ATTN_OK) return 0;
  bool any = false;
  for (int i = 0; i < n; ++i) any = any || parts[i].dweight;
  if (!any) return kNoSpace;
  int sms = 0;
  if (ea::device_sms(&sms) != ATTN_OK) return 0;
  // the number of CTAs goes by the rotation too, which is not told here: the most
  // that any has
  size_t bytes = 0;
  for (int i = 0; i < n; ++i)
    if (parts[i].dweight) bytes += static_cast<size_t>(ea::rope_most_ctas(sms)) * D * 4;
  return bytes < kNoSpace ? kNoSpace : bytes;
}

attn_status_t attn_rope_bwd(const attn_rope_part_t* parts, int n, const attn_rope_t* rope,
                            const attn_rope_positions_t* positions, int64_t B, int64_t S, int64_t D,
                            float eps, attn_dtype_t dtype, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  const attn_status_t s = check(parts, n, rope, positions, B, S, D, eps, dtype, true, workspace, workspace_bytes);
  if (s != ATTN_OK) return s;
  return run(parts, n, rope, positions, B, S, D, eps, dtype, workspace, workspace_bytes, true, stream);
}

}  // extern "C"
