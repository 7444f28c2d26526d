// Attention over a paged key/value cache: what the planning, row-block and
// combine kernels share.
//
// For query row t of head h, with the keys s that are visible to it,
//
//     x_s = scale * q . k_s      lse = log sum_s exp(x_s)      out = sum_s exp(x_s - lse) v_s
//
// (out = 0 and lse = -inf when none is visible). The kernels hold x in units
// of log 2 and keep a running maximum and sum per row, so the keys are read in
// one pass and any cut of them into pieces can be joined afterwards.
#pragma once

#include <cuda_fp16.h>

#include "internal.h"

namespace saib {

// One call's arguments, as the kernels see them.
struct AttendParams {
  const void* q;
  int64_t q_stride_token, q_stride_head;  // elements
  const void* k;
  const void* v;
  int64_t k_stride_page, k_stride_token, k_stride_head;
  int64_t v_stride_page, v_stride_token, v_stride_head;
  int64_t num_pages;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t bt_width;
  const int32_t* seq_lens;         // [num_reqs] (paged form)
  const int32_t* query_start_loc;  // [num_reqs + 1]
  const int32_t* indices;          // [num_tokens, topk] (selected form), else nullptr
  int64_t indices_stride;
  int32_t topk;
  int32_t num_reqs, num_tokens;
  int32_t num_heads, num_kv_heads, group;
  float scale_log2;                // scale * log2(e)
  int32_t window;                  // INT32_MAX: no window
  int32_t sinks;
  void* out;                       // [num_tokens, num_heads, head_dim]
  float* lse;                      // nullable [num_tokens, num_heads]
  // workspace
  int32_t* req_entry;              // [num_reqs + 1] first entry of each request
  int64_t* entry_cost;             // [max_entries + 1] exclusive prefix of the entries' costs
  int4* bound;                     // [grid + 1] first piece of each CTA: entry, kv head, tile, request
  float* part_o;                   // [2 * grid, rows, head_dim] unnormalised pieces
  float2* part_ml;                 // [2 * grid, rows] their maximum and sum
  int32_t max_entries;
  int32_t grid;                    // CTAs of the row-block launch
  int32_t rows;                    // query rows of a unit
  int32_t tile;                    // keys of a tile
  uint32_t* dev_error;
  uint64_t wait_ns;
};

// A unit is one kv head's block of `rows` query rows of one request (rows are
// (token, head of the group) pairs in that order); an entry is a unit without
// its kv head. The tiles of a unit cover the keys that some row of it sees:
// first the tiles of the first `sinks` keys (when a window hides what follows
// them), then those of the window up to the last row's own position.
struct UnitTiles {
  int32_t first;  // tiles of the sinks
  int32_t skip;   // tiles between them and the window's
  int32_t count;  // all tiles of the unit
  int32_t p_lo, p_hi;  // positions of the unit's first and last token

  __device__ __forceinline__ int32_t tile(int32_t i) const { return i < first ? i : i + skip; }
};

struct ReqShape {
  int32_t q0;    // first token row
  int32_t nq;    // new tokens
  int32_t keys;  // keys, the new ones among them
};

// Lengths of request b, clamped to what the buffers hold.
__device__ __forceinline__ ReqShape request_shape(const AttendParams& p, int32_t b, bool report) {
  int32_t a = p.query_start_loc[b], e = p.query_start_loc[b + 1];
  int64_t n = p.seq_lens ? p.seq_lens[b] : 0;
  const int64_t most = static_cast<int64_t>(p.bt_width) * kPageTokens;
  const bool bad = a < 0 || e < a || e > p.num_tokens || n < 0 || n > most;
  if (bad && report) set_error(p.dev_error, IDX_DEV_BAD_LEN);
  a = min(max(a, 0), p.num_tokens);
  e = min(max(e, a), p.num_tokens);
  n = n < 0 ? 0 : (n > most ? most : n);
  return ReqShape{a, e - a, static_cast<int32_t>(n)};
}

__device__ __forceinline__ int32_t request_entries(const AttendParams& p, const ReqShape& r) {
  return static_cast<int32_t>((static_cast<int64_t>(r.nq) * p.group + p.rows - 1) / p.rows);
}

__device__ __forceinline__ UnitTiles unit_tiles(const AttendParams& p, const ReqShape& r, int32_t u) {
  UnitTiles t;
  const int64_t row0 = static_cast<int64_t>(u) * p.rows;
  const int64_t total = static_cast<int64_t>(r.nq) * p.group;
  const int64_t row1 = row0 + p.rows < total ? row0 + p.rows : total;
  const int32_t ahead = r.keys - r.nq;
  t.p_lo = ahead + static_cast<int32_t>(row0 / p.group);
  t.p_hi = ahead + static_cast<int32_t>((row1 - 1) / p.group);
  if (t.p_hi < 0) {
    t.first = t.skip = t.count = 0;
    return t;
  }
  const int32_t end = t.p_hi / p.tile + 1;
  const int64_t lo = static_cast<int64_t>(t.p_lo) - p.window + 1;
  const int32_t start = lo > 0 ? static_cast<int32_t>(lo) / p.tile : 0;
  int32_t first = (p.sinks + p.tile - 1) / p.tile;
  first = first < start ? first : start;
  t.first = first;
  t.skip = start - first;
  t.count = end - t.skip;
  return t;
}

// Tiles of streaming that starting and ending a unit cost its CTA.
constexpr int kUnitOverhead = 1;

// Launchers.
idx_status launch_attend_plan(const AttendParams& p, cudaStream_t s);
idx_status launch_attend_rows(const AttendParams& p, int head_dim, bool half, int mt, cudaStream_t s);
idx_status launch_attend_combine(const AttendParams& p, int head_dim, bool half, cudaStream_t s);

}  // namespace saib
