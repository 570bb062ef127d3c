// attn_cache_impl.h — kernel parameters and launch entries shared by the host
// API of the 8-bit cache and its kernel translation units (host-compilable).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

namespace ea {

// The pool of pages (see include/attn_cache.h for the layout).
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int8_t* k_bounds;
  int pages, heads;
  int D, pitch;         // channels, bytes of one row
  int page, log2_page;  // token slots of a page
};

// The sequences of a call.
struct SeqView {
  const int* table;
  const int* lens;
  const int* fresh;  // may be null: T new tokens each
  int batch, width, T;
  int* status;
};

struct CacheAppendParams {
  CacheView c;
  SeqView s;
  const uint16_t* k;  // [batch, heads, T, D]
  const uint16_t* v;
  int pages_per_seq;  // pages T tokens can touch
};
cudaError_t cache_append_launch(const CacheAppendParams& p, bool f16, cudaStream_t stream);

struct CacheEvictParams {
  CacheView c;
  SeqView s;
  const float* mass;
  const int* dst_table;
  int dst_width;
  int keep, recent;
  int* kept;
  int* new_lens;
  float* mass_out;
  uint32_t* used;   // workspace: two bits per page of the pool, [2][words]
  int used_words;
  int* dst_page;    // workspace: dst_table after its checks, -1: not to be written
};
cudaError_t cache_evict_launch(const CacheEvictParams& p, cudaStream_t stream);

struct CacheSelectParams {
  CacheView c;
  SeqView s;
  const uint16_t* q;  // [batch, heads·G, T, D]
  int G;
  int count;
  int* pages;     // [batch, heads, count]
  float* scores;  // [batch, heads, width]
  int sms;        // of the device
};
cudaError_t cache_select_launch(const CacheSelectParams& p, bool f16, cudaStream_t stream);

// Tokens of one chunk, the unit of work of the attention: one warp's step.
constexpr int kCacheChunk = 64;
// Query rows of a tile; a pass over a (sequence, head)'s keys takes as many
// tiles as their sums leave registers for.  Measured at 128 channels, 128
// segments of 4096 keys: 1 tile 27 us, 2 tiles 32 us; 24 rows in two passes of 2
// tiles 58 us (in one pass of 3, which spills, 79 us when two took 63).  At 64
// channels 32 rows in one pass 40.5 us, in two 43.7 us; at 256 channels 16 rows in one
// 82 us, in two 92 us.
constexpr int kCacheTileRows = 8;
// Tiles up to which a warp may be a worker of its own: each worker's Q takes
// shared memory from the rings.
constexpr int kCacheWarpWorkerTiles = 2;
inline int cache_max_tiles(int width) { return width <= 64 ? 4 : 2; }

struct CacheFwdParams {
  CUtensorMap tm_k, tm_v;  // (channel, slot, page·head), box: a swizzled row x one page
  CacheView c;
  SeqView s;
  const uint16_t* q;   // [batch, heads·G, T, D]
  uint16_t* out;
  float* lse;
  const int* list;     // [batch, heads, listed] or null
  int listed;
  bool f16;            // q and out are fp16 (else bf16)
  int G, row_tiles;    // query heads per key head; passes over a head's keys
  float scale_log2;
  int cluster;         // CTAs of the cluster that has a segment; 0: chunks are dealt to workers
  int workers;         // parts the chunks of all (sequence, head, row tile) are dealt to
  int lead;            // what a segment costs by itself, in chunks
  int min_units;       // fewest chunks, with a lead, worth a worker of their own
  int* line;           // workspace: first unit of each sequence in the line, then its end
  float* part;         // workspace: partial results, two slots per worker
  float* scores;       // workspace: scaled scores in log2 units, or null (no mass)
  int score_cols;      // keys of a head in `scores`
  int score_rows;      // rows of a key
  float* mass;         // [batch, heads, width·page] or null
  uint64_t timeout_ns;
};
// Floats of one partial result of `rows` query rows: O [rows][width], then m, r, l [rows] each.
template <int WIDTH, int TILES>
constexpr int kCachePartFloats = kCacheTileRows * TILES * (WIDTH + 3);
// Width of the kernel that runs a head dimension: 64, 128 or 256.
inline int cache_kernel_width(int64_t D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// Warps of one CTA of that kernel: as many as the registers of a tile's sums allow.
template <int WIDTH, int TILES>
constexpr int kCacheWarps = (TILES == 1 ? 12 : 8) / (WIDTH <= 128 ? 1 : 2);
inline int cache_kernel_warps(int width, int tiles) { return (tiles == 1 ? 12 : 8) / (width <= 128 ? 1 : 2); }

// CTAs of the largest cluster, and how many clusters of `size` the device holds
// at once (asked for once per device; it depends on how its SMs are grouped, which
// differs between devices of one kind).
constexpr int kCacheMaxCluster = 8;
int cache_fwd_clusters(int dev, int size);

// tiles: 8-row tiles of one pass.
cudaError_t cache_fwd_launch(const CacheFwdParams& p, int width, int tiles, bool warp_workers, int dev, int ctas,
                             cudaStream_t stream);

}  // namespace ea
