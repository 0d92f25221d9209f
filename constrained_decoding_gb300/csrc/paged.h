// Rotary positions and the 8-bit paged K/V cache: launch arguments and
// launchers of pcd_k_rope, pcd_k_kv_append and pcd_k_paged_attention.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

namespace pcd {

// Records `detail` as pcd_last_error's text of this thread and returns `code`.
int set_error(int code, const char* detail);

// Rotation of pairs: F[i] is pair i's angle per position as a fraction of a
// turn in units of 2^-64.
struct RopeSpec {
  const int64_t* freqs = nullptr;  // device, rot / 2 entries; nullptr: no rotation
  int rot = 0;                     // rotated channels: the first rot of a head, even
  int interleaved = 0;             // pairs (2i, 2i + 1), else (i, i + rot / 2)
  float amp = 1.f;                 // factor on cos and sin
  int transpose = 0;               // the transposed rotation
};

struct RopeKArgs {
  const void* x;
  void* y;
  int dtype, n_tok, heads, dim;
  int64_t x_tok, x_head, y_tok, y_head;  // strides in elements
  RopeSpec rope;
  const int32_t* pos;  // per token, or nullptr: base + token
  int base;
};
int launch_rope(const RopeKArgs& a, int sms, cudaStream_t s);

// The cache: codes of (page, KV head, slot, channel), channels contiguous,
// and one scale for each (page, KV head).
struct PagesView {
  uint8_t *k, *v;
  float *ks, *vs;                             // [n_pages][Hkv]
  int64_t page_stride, head_stride, tok_stride;  // bytes
  int n_pages, page_log2, Hkv, dim, format;
};

// Ragged sequences: query (or new) rows q_off[s] .. q_off[s + 1), kv_len[s]
// tokens in the cache with them included, their pages the first entries of the
// table_width at table[s * table_stride].
struct SeqView {
  const int32_t *q_off, *kv_len, *table;
  int n_seq, n_tok, table_stride, table_width;
};

struct AppendArgs {
  PagesView c;
  SeqView q;
  const void *k, *v;
  int dtype;
  int64_t k_tok, k_head, v_tok, v_head;  // elements
  RopeSpec rope;
  const int32_t* pos;  // per new token, or nullptr: its place in the cache
  int* err;
};
int launch_kv_append(const AppendArgs& a, int sms, cudaStream_t s);

// How a call is cut up.  rows: query rows of a work item (8 or 16: warp MMA,
// 256: tcgen05).  n_splits: ranges that every item's keys are divided into, walked
// by a thread-block cluster that joins them (cluster) or joined by a second
// kernel; with stream, CTAs that share the blocks of all items evenly.  parts:
// of a row for that kernel, as far as the host knows.  alternate: items of one
// tcgen05 tile give their key blocks to two pipelines in turn.
constexpr int kTileRowsLog = 8, kTileRows = 1 << kTileRowsLog;  // query rows of an item of the tcgen05 kernel
struct PagedPlan {
  int rows, n_splits, cluster, stream, parts, alternate;
};

struct PagedAttnArgs {
  PagesView c;
  SeqView q;
  const void* x;  // queries [n_tok][Hq][dim]
  void* out;
  float* lse;     // [n_tok][Hq] or nullptr
  int dtype, Hq, G, causal;
  int64_t x_tok, x_head, out_tok, out_head;  // elements
  float scale_log2;                          // softmax scale x log2(e)
  PagedPlan plan;
  // scratch: states (O, then M and l) of rows cut by ranges, [n_splits][n_tok][Hq], or by the ends of
  // stretches, [2 n_splits][16], and then where a row's are
  float* part_o;
  float2* part_ml;
  int2* part_at;
  int* err;
  uint64_t wait_ns;  // limit of a pipeline's waits
};
void plan_paged_attention(int n_tok, int n_seq, int G, int Hkv, int64_t max_kv, int sms, PagedPlan* p);
int launch_paged_attention(const PagedAttnArgs& a, cudaStream_t s);
int launch_paged_attention_tiles(const PagedAttnArgs& a, cudaStream_t s);  // plan.rows == 256, without the join

}  // namespace pcd
