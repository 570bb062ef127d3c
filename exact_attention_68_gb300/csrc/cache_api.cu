// cache_api.cu — the C ABI declared in include/attn_cache.h: argument checks,
// tensor maps, workspaces, launch.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "attn_cache.h"
#include "attn_cache_impl.h"
#include "attn_host.h"
#include "tmap.h"

namespace {

using ea::aligned;
using ea::any_overlap;
using ea::Span;

int64_t pitch_of(int64_t D) { return (D + 15) / 16 * 16; }

// The pool and the sequences of a call; touches no CUDA API.
attn_status_t check_cache(const attn_cache_t* c, const attn_cache_seqs_t* s) {
  if (!c || !s) return ATTN_ERR_INVALID_ARG;
  if (c->pages < 1 || c->heads < 1 || c->head_dim < 1 || s->batch < 1 || s->width < 1)
    return ATTN_ERR_INVALID_ARG;
  if (c->head_dim > 256 || c->head_dim % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64) return ATTN_ERR_UNSUPPORTED;
  if (c->heads > 65535 || s->batch > 65534 || c->pages > INT32_MAX || s->width > INT32_MAX)
    return ATTN_ERR_INVALID_ARG;
  if (c->pages * c->heads > INT32_MAX / c->page || s->width > (1 << 30) / c->page)
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}
attn_status_t check_pointers(const attn_cache_t* c, const attn_cache_seqs_t* s) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->k_bounds || !s->table || !s->lens)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_bounds, 16)) return ATTN_ERR_MISALIGNED;
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(s->table, 4) ||
      !aligned(s->lens, 4) || !aligned(s->fresh, 4))
    return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

// The pool's and the sequences' buffers as spans (8 of them).
int cache_spans(const attn_cache_t* c, const attn_cache_seqs_t* s, bool pool_written, Span* out) {
  const uint64_t rows = static_cast<uint64_t>(c->pages * c->heads);
  const uint64_t pitch = static_cast<uint64_t>(pitch_of(c->head_dim));
  out[0] = {c->k, rows * c->page * pitch, pool_written};
  out[1] = {c->v, rows * c->page * pitch, pool_written};
  out[2] = {c->k_scale, rows * 4, pool_written};
  out[3] = {c->v_scale, rows * 4, pool_written};
  out[4] = {c->k_bounds, rows * 2 * pitch, pool_written};
  out[5] = {s->table, static_cast<uint64_t>(s->batch * s->width) * 4, false};
  out[6] = {s->lens, static_cast<uint64_t>(s->batch) * 4, false};
  out[7] = {s->fresh, static_cast<uint64_t>(s->batch) * 4, false};
  return 8;
}

ea::CacheView view_of(const attn_cache_t* c) {
  ea::CacheView v;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.k_bounds = c->k_bounds;
  v.pages = static_cast<int>(c->pages);
  v.heads = static_cast<int>(c->heads);
  v.D = static_cast<int>(c->head_dim);
  v.pitch = static_cast<int>(pitch_of(c->head_dim));
  v.page = static_cast<int>(c->page);
  v.log2_page = c->page == 16 ? 4 : c->page == 32 ? 5 : 6;
  return v;
}

ea::SeqView seqs_of(const attn_cache_seqs_t* s, int64_t T, int* status) {
  ea::SeqView v;
  v.table = s->table;
  v.lens = s->lens;
  v.fresh = s->fresh;
  v.batch = static_cast<int>(s->batch);
  v.width = static_cast<int>(s->width);
  v.T = static_cast<int>(T);
  v.status = status;
  return v;
}

// The passes over a head's keys that `rows` query rows need, and the 8-row
// tiles of one: as few passes as registers allow, as few tiles as those need.
int64_t passes_of(int64_t rows, int width) {
  const int64_t per = ea::kCacheTileRows * ea::cache_max_tiles(width);
  return (rows + per - 1) / per;
}
int tiles_of(int64_t rows, int width) {
  const int64_t per = passes_of(rows, width) * ea::kCacheTileRows;
  return static_cast<int>((rows + per - 1) / per);
}

// What a segment costs besides its chunks (Q, the join, the output), in a worker's
// chunks.  480 segments of 1 to 32 chunks, a CTA a worker: 52.8 us at 0, 44.7 at 4,
// 31.0 at 12, 30.3 at 16, 31.3 at 24; 960 of two tiles, a warp a worker: 99 us at 0,
// 79 at 1, 72 at 2, but 720 of 3 chunks 21.9, 19.8 and 22.0.
constexpr int kWarpLead = 1, kCtaLead = 16;

// Sizes of the queries; touches no CUDA API.
attn_status_t check_queries(const attn_cache_t* c, const attn_cache_seqs_t* s, int64_t q_heads,
                            int64_t T) {
  if (q_heads < 1 || T < 1 || T > ATTN_CACHE_MAX_TOKENS || q_heads > INT32_MAX / 64 ||
      q_heads % c->heads != 0)
    return ATTN_ERR_INVALID_ARG;
  // query rows and the chunks of the longest call are counted in 32 bits
  const int64_t chunks = (s->width * c->page + ea::kCacheChunk - 1) / ea::kCacheChunk;
  const int64_t segments = s->batch * c->heads * passes_of(q_heads / c->heads * T, ea::cache_kernel_width(c->head_dim));  // < 2^52
  if (s->batch * q_heads > INT32_MAX / T || segments > (1ll << 30) / (chunks + kCtaLead)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// Entries of a page list: their tokens are counted in 32 bits.
constexpr int64_t kMaxListed = INT32_MAX / 64;

// Keys of a head in the score workspace: whole chunks.
int64_t score_cols(const attn_cache_t* c, const attn_cache_seqs_t* s, int64_t listed, bool has_list) {
  const int64_t pages = has_list && listed < s->width ? listed : s->width;
  return (pages * c->page + ea::kCacheChunk - 1) / ea::kCacheChunk * ea::kCacheChunk;
}

// How the chunks are dealt.  With more short segments than SMs a warp is a
// worker: nothing has to be joined but at a worker's two ends.  Otherwise a CTA is
// one: its warps' results are joined in shared memory, a twelfth of the parts go
// through the workspace.  320 segments of 8, 32 chunks: a warp each 19, 43 us, a
// CTA 21, 40 us; 720 of 3, 16 chunks 18, 48 and 30, 51 us; 1024 of 16, 32, 64 chunks 64,
// 101, 181 and 68, 96, 168 us, of 2 to 32 chunks 70 and 79 us.
constexpr int64_t kShortSegment = 16;
// Sizes here are those of the table, since lengths are on the device: under a table of
// 2048 pages one sequence of 1000 keys takes 13.1 us (tight 8.7), 720 segments of up to 3
// chunks 32.5 (18.9), 16 sequences of 500-8192 keys 37.6 (37.0).
struct Plan {
  int width, tiles, passes, ctas, workers;
  int cluster;
  bool warp_workers;
};
// Steps of a warp up to which a segment is left to its own cluster: that saves
// the deal and the join, about 5 us and a launch, and one CTA streams at about
// twice its even share of the memory's rate, so that lengths may differ by two
// before it loses; fewer with two tiles, whose products bound the step, and where
// the clusters leave a quarter of the SMs empty.  128 segments of 2048, 4096, 8192
// keys: 14, 28, 46 us, dealt 19, 32, 54 us; of 128 to 2048, 256 to 4096, 512 to 8192
// keys 14, 22, 38 and 18, 23, 37 us; 32 segments of 64 listed pages, clusters of 4: 12.7
// us, dealt 18 us; 48 segments of 4096, 8192 keys, clusters of 2: 15, 24 us, dealt 17, 22
// us.
constexpr int64_t kSegmentSteps = 12, kTilesSegmentSteps = 8, kFewSegmentSteps = 4;
Plan plan_of(const attn_cache_t* c, const attn_cache_seqs_t* s, int64_t listed, int64_t q_heads, int64_t T,
             int dev, int sms) {
  Plan p;
  p.width = ea::cache_kernel_width(c->head_dim);
  const int64_t rows = q_heads / c->heads * T;
  p.tiles = tiles_of(rows, p.width);
  p.passes = static_cast<int>(passes_of(rows, p.width));
  const int warps = ea::cache_kernel_warps(p.width, p.tiles);
  const int64_t segments = s->batch * c->heads * p.passes;
  const int64_t chunks = score_cols(c, s, listed, listed > 0) / ea::kCacheChunk;  // at most, of a segment
  // a cluster for each segment: the largest of which all find their place at once
  // (of 8 CTAs 15 or 16 on 152 SMs; one cluster that has to wait doubles the time)
  // and that leaves each CTA four chunks of the longest segment
  int cluster = 1;
  while (cluster < ea::kCacheMaxCluster && chunks >= 8 * cluster &&
         segments <= ea::cache_fwd_clusters(dev, 2 * cluster))
    cluster *= 2;
  const int64_t steps = 4 * segments * cluster < 3 * sms ? kFewSegmentSteps
                        : p.tiles > 1                   ? kTilesSegmentSteps
                                                        : kSegmentSteps;
  p.cluster = segments <= sms && chunks <= steps * warps * cluster ? cluster : 0;
  p.warp_workers = p.cluster == 0 && p.tiles <= ea::kCacheWarpWorkerTiles &&
                   segments > sms &&
                   chunks <= kShortSegment * (segments >= static_cast<int64_t>(sms) * warps / 2 ? 2 : 1);
  p.ctas = p.cluster > 0 ? static_cast<int>(segments) * p.cluster : sms;
  p.workers = p.cluster > 0 ? 0 : p.warp_workers ? sms * warps : sms;
  return p;
}

// Two parts for each worker: the segment it begins in and the one it ends in.
size_t part_bytes(const Plan& p) {
  const size_t floats = p.tiles * (p.width == 64    ? ea::kCachePartFloats<64, 1>
                                   : p.width == 128 ? ea::kCachePartFloats<128, 1>
                                                    : ea::kCachePartFloats<256, 1>);
  return 2 * static_cast<size_t>(p.workers) * floats * 4;  // a multiple of 16
}

// The line's sequences, where there is one.
size_t line_bytes(const Plan& p, const attn_cache_seqs_t* s) {
  return p.cluster > 0 ? 0 : (static_cast<size_t>(s->batch + 1) * 4 + 15) / 16 * 16;
}

// Rows of the score workspace: whole tiles.
size_t score_rows(const Plan& p) { return static_cast<size_t>(p.passes) * p.tiles * ea::kCacheTileRows; }

// The current device and its number of SMs (asked for once per device).
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];
bool sm_count(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) return false;
  *sms = g_sms[*dev].load(std::memory_order_relaxed);
  if (*sms > 0) return true;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess || *sms < 1) return false;
  g_sms[*dev].store(*sms, std::memory_order_relaxed);
  return true;
}

// The current device's status words.  They stay where they are once they are
// there, so the set-up behind them (a lock, a device call) is gone through
// once per device.
std::atomic<int*> g_status[kMaxDevices];
attn_status_t status_words(int** status) {
  int dev = -1;
  const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices;
  if (known && (*status = g_status[dev].load(std::memory_order_acquire)) != nullptr) return ATTN_OK;
  const attn_status_t s = ea::current_status_words(status);
  if (s == ATTN_OK && known) g_status[dev].store(*status, std::memory_order_release);
  return s;
}

// The attention's workspace: parts, then scores; 16 bytes, which no kernel
// touches, where there are neither.
constexpr size_t kNoSpace = 16;
size_t fwd_bytes(const Plan& plan, const attn_cache_t* c, const attn_cache_seqs_t* s, int64_t listed, bool with_mass) {
  const size_t keys = static_cast<size_t>(s->batch * c->heads) * score_cols(c, s, listed, listed > 0);
  return kNoSpace + line_bytes(plan, s) + part_bytes(plan) + (with_mass ? keys * score_rows(plan) * 4 : 0);
}

// (channel, slot, page·head) map of a pool's codes; the box is one swizzled
// row (64 or 128 bytes) by one page.  Channels past head_dim read as zero.
bool encode_codes(CUtensorMap* map, void* base, const ea::CacheView& c, int width) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = ea::tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page),
                              static_cast<cuuint64_t>(c.pages) * c.heads};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.pitch),
                                 static_cast<cuuint64_t>(c.page) * c.pitch};
  const cuuint32_t box[3] = {width >= 128 ? 128u : 64u, static_cast<cuuint32_t>(c.page), 1u};
  const cuuint32_t step[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             width >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

attn_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return ATTN_OK;
  (void)cudaGetLastError();
  return ea::cuda_failure(static_cast<int>(e));
}

}  // namespace

extern "C" {

attn_status_t attn_cache_append(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                                const void* k, const void* v, int64_t T, attn_dtype_t dtype,
                                cudaStream_t stream) {
  if (dtype != ATTN_BF16 && dtype != ATTN_F16) return ATTN_ERR_INVALID_ARG;
  attn_status_t s = check_cache(cache, seqs);
  if (s != ATTN_OK) return s;
  if (!k || !v || T < 1 || T > (1 << 30)) return ATTN_ERR_INVALID_ARG;
  const int64_t per_seq = (T + cache->page - 2) / cache->page + 1;
  if (seqs->batch * cache->heads > INT32_MAX / 2 / per_seq) return ATTN_ERR_INVALID_ARG;  // the grid
  s = check_pointers(cache, seqs);
  if (s != ATTN_OK) return s;
  if (!aligned(k, 16) || !aligned(v, 16)) return ATTN_ERR_MISALIGNED;
  Span spans[10];
  int n = cache_spans(cache, seqs, true, spans);
  const uint64_t bytes = static_cast<uint64_t>(seqs->batch * cache->heads) * T * cache->head_dim * 2;
  spans[n++] = {k, bytes, false};
  spans[n++] = {v, bytes, false};
  if (any_overlap(spans, n)) return ATTN_ERR_INVALID_ARG;
  int* status = nullptr;
  s = status_words(&status);
  if (s != ATTN_OK) return s;
  ea::CacheAppendParams p;
  p.c = view_of(cache);
  p.s = seqs_of(seqs, T, status);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.pages_per_seq = static_cast<int>(per_seq);
  return launched(ea::cache_append_launch(p, dtype == ATTN_F16, stream));
}

size_t attn_cache_fwd_workspace(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                                int64_t listed, int64_t q_heads, int64_t T, int with_mass) {
  int dev = -1, sms = 0;
  if (check_cache(cache, seqs) != ATTN_OK || listed < 0 || listed > kMaxListed ||
      check_queries(cache, seqs, q_heads, T) != ATTN_OK || !sm_count(&dev, &sms))
    return 0;
  return fwd_bytes(plan_of(cache, seqs, listed, q_heads, T, dev, sms), cache, seqs, listed, with_mass != 0);
}

attn_status_t attn_cache_fwd(const attn_cache_t* cache, const attn_cache_seqs_t* seqs, const void* q,
                             const int32_t* pages, int64_t listed, void* out, float* lse, float* mass,
                             int64_t q_heads, int64_t T, float scale, attn_dtype_t dtype,
                             void* workspace, size_t workspace_bytes, uint64_t wait_timeout_ns,
                             cudaStream_t stream) {
  if (dtype != ATTN_BF16 && dtype != ATTN_F16) return ATTN_ERR_INVALID_ARG;
  attn_status_t s = check_cache(cache, seqs);
  if (s != ATTN_OK) return s;
  if (!q || !out || !lse) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (pages ? (listed < 1 || listed > kMaxListed) : listed != 0) return ATTN_ERR_INVALID_ARG;
  s = check_queries(cache, seqs, q_heads, T);
  if (s != ATTN_OK) return s;
  s = check_pointers(cache, seqs);
  if (s != ATTN_OK) return s;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4) ||
      !aligned(mass, 4) || !aligned(pages, 4))
    return ATTN_ERR_MISALIGNED;
  int* status = nullptr;
  s = status_words(&status);
  if (s != ATTN_OK) return s;
  int dev = -1, sms = 0;
  if (!sm_count(&dev, &sms)) return ATTN_ERR_CUDA;
  const Plan plan = plan_of(cache, seqs, listed, q_heads, T, dev, sms);
  const size_t need = fwd_bytes(plan, cache, seqs, listed, mass != nullptr);
  if (need > kNoSpace && (!workspace || workspace_bytes < need)) return ATTN_ERR_INVALID_ARG;
  Span spans[14];
  int n = cache_spans(cache, seqs, false, spans);
  const uint64_t rows = static_cast<uint64_t>(seqs->batch * q_heads * T);
  const uint64_t heads = static_cast<uint64_t>(seqs->batch * cache->heads);
  spans[n++] = {q, rows * cache->head_dim * 2, false};
  spans[n++] = {pages, heads * listed * 4, false};
  spans[n++] = {out, rows * cache->head_dim * 2, true};
  spans[n++] = {lse, rows * 4, true};
  spans[n++] = {mass, heads * seqs->width * cache->page * 4, true};
  spans[n++] = {workspace, need, true};
  if (any_overlap(spans, n)) return ATTN_ERR_INVALID_ARG;

  // the tensor maps are encoded by a driver call, which wants a context on this thread
  const cudaError_t bound = ea::current_device_bound(&dev);
  if (bound != cudaSuccess) return ea::cuda_failure(static_cast<int>(bound));
  ea::CacheFwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = view_of(cache);
  p.s = seqs_of(seqs, T, status);
  if (!encode_codes(&p.tm_k, p.c.k, p.c, plan.width) || !encode_codes(&p.tm_v, p.c.v, p.c, plan.width))
    return ea::cuda_failure(ea::kErrTensorMap);
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.list = pages;
  p.listed = static_cast<int>(listed);
  p.G = static_cast<int>(q_heads / cache->heads);
  p.f16 = dtype == ATTN_F16;
  p.row_tiles = plan.passes;
  p.score_rows = static_cast<int>(score_rows(plan));
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.cluster = plan.cluster;
  p.workers = plan.workers;
  p.lead = plan.cluster > 0 ? 0 : plan.warp_workers ? kWarpLead : kCtaLead;
  p.min_units = p.lead + (plan.warp_workers ? 1 : 4);
  char* space = static_cast<char*>(workspace);
  p.line = reinterpret_cast<int*>(space);
  p.part = reinterpret_cast<float*>(space + line_bytes(plan, seqs));
  p.mass = mass;
  p.score_cols = static_cast<int>(score_cols(cache, seqs, listed, pages != nullptr));
  p.scores = mass ? reinterpret_cast<float*>(space + line_bytes(plan, seqs) + part_bytes(plan)) : nullptr;
  p.timeout_ns = wait_timeout_ns;
  return launched(ea::cache_fwd_launch(p, plan.width, plan.tiles, plan.warp_workers, dev, plan.ctas, stream));
}

attn_status_t attn_cache_select(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                                const void* q, int64_t q_heads, int64_t T, attn_dtype_t dtype,
                                int64_t count, int32_t* pages, float* scores, cudaStream_t stream) {
  if (dtype != ATTN_BF16 && dtype != ATTN_F16) return ATTN_ERR_INVALID_ARG;
  attn_status_t s = check_cache(cache, seqs);
  if (s != ATTN_OK) return s;
  if (!q || !pages || !scores || count < 1 || count > INT32_MAX / 64) return ATTN_ERR_INVALID_ARG;
  s = check_queries(cache, seqs, q_heads, T);
  if (s != ATTN_OK) return s;
  s = check_pointers(cache, seqs);
  if (s != ATTN_OK) return s;
  if (!aligned(q, 16) || !aligned(pages, 4) || !aligned(scores, 4)) return ATTN_ERR_MISALIGNED;
  Span spans[11];
  int n = cache_spans(cache, seqs, false, spans);
  const uint64_t heads = static_cast<uint64_t>(seqs->batch * cache->heads);
  spans[n++] = {q, static_cast<uint64_t>(seqs->batch * q_heads * T) * cache->head_dim * 2, false};
  spans[n++] = {pages, heads * count * 4, true};
  spans[n++] = {scores, heads * seqs->width * 4, true};
  if (any_overlap(spans, n)) return ATTN_ERR_INVALID_ARG;
  int* status = nullptr;
  s = status_words(&status);
  if (s != ATTN_OK) return s;
  int dev = -1, sms = 0;
  if (!sm_count(&dev, &sms)) return ATTN_ERR_CUDA;
  ea::CacheSelectParams p;
  p.sms = sms;
  p.c = view_of(cache);
  p.s = seqs_of(seqs, T, status);
  p.q = static_cast<const uint16_t*>(q);
  p.G = static_cast<int>(q_heads / cache->heads);
  p.count = static_cast<int>(count);
  p.pages = pages;
  p.scores = scores;
  return launched(ea::cache_select_launch(p, dtype == ATTN_F16, stream));
}

size_t attn_cache_evict_workspace(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                                  int64_t dst_width) {
  if (check_cache(cache, seqs) != ATTN_OK || dst_width < 1 || dst_width > (1 << 30) / cache->page) return 0;
  const size_t words = static_cast<size_t>((cache->pages + 31) / 32);
  return (2 * words * 4 + static_cast<size_t>(seqs->batch * dst_width) * 4 + 15) / 16 * 16;
}

attn_status_t attn_cache_evict(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                               const float* mass, const int32_t* dst_table, int64_t dst_width,
                               int64_t keep, int64_t recent, int32_t* kept, int32_t* new_lens,
                               float* mass_out, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  attn_status_t s = check_cache(cache, seqs);
  if (s != ATTN_OK) return s;
  if (!mass || !dst_table || !kept || !new_lens || !mass_out || !workspace) return ATTN_ERR_INVALID_ARG;
  if (dst_width < 1 || dst_width > (1 << 30) / cache->page || keep < 1 || keep > dst_width * cache->page ||
      recent < 0 || recent > keep)
    return ATTN_ERR_INVALID_ARG;
  const int64_t per_seq = (keep + cache->page - 1) / cache->page;
  if (seqs->batch * cache->heads > INT32_MAX / 2 / per_seq) return ATTN_ERR_INVALID_ARG;  // the grid
  s = check_pointers(cache, seqs);
  if (s != ATTN_OK) return s;
  if (!aligned(workspace, 16) || !aligned(mass, 4) || !aligned(dst_table, 4) || !aligned(kept, 4) ||
      !aligned(new_lens, 4) || !aligned(mass_out, 4))
    return ATTN_ERR_MISALIGNED;
  const size_t need = attn_cache_evict_workspace(cache, seqs, dst_width);
  if (workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
  Span spans[14];
  int n = cache_spans(cache, seqs, true, spans);
  const uint64_t heads = static_cast<uint64_t>(seqs->batch * cache->heads);
  spans[n++] = {mass, heads * seqs->width * cache->page * 4, false};
  spans[n++] = {dst_table, static_cast<uint64_t>(seqs->batch * dst_width) * 4, false};
  spans[n++] = {kept, heads * keep * 4, true};
  spans[n++] = {new_lens, static_cast<uint64_t>(seqs->batch) * 4, true};
  spans[n++] = {mass_out, heads * dst_width * cache->page * 4, true};
  spans[n++] = {workspace, need, true};
  if (any_overlap(spans, n)) return ATTN_ERR_INVALID_ARG;
  int* status = nullptr;
  s = status_words(&status);
  if (s != ATTN_OK) return s;
  ea::CacheEvictParams p;
  p.c = view_of(cache);
  p.s = seqs_of(seqs, 0, status);
  p.s.fresh = nullptr;
  p.mass = mass;
  p.dst_table = dst_table;
  p.dst_width = static_cast<int>(dst_width);
  p.keep = static_cast<int>(keep);
  p.recent = static_cast<int>(recent);
  p.kept = kept;
  p.new_lens = new_lens;
  p.mass_out = mass_out;
  p.used_words = static_cast<int>((cache->pages + 31) / 32);
  p.used = static_cast<uint32_t*>(workspace);
  p.dst_page = static_cast<int*>(workspace) + 2 * p.used_words;
  return launched(ea::cache_evict_launch(p, stream));
}

}  // extern "C"
