// C entry points of the attention calls: argument checks, the choice of a
// kernel, the workspace and the launches.
#include <math.h>

#include <algorithm>

#include "attend.cuh"

namespace saib {

namespace {

constexpr int kRowsCtasPerSm = 2;
// Keys of a request; a window that wide hides nothing. Positions less windows less keys fit in
// 32 bits.
constexpr int32_t kMostKeys = 1 << 30;
constexpr int64_t kMostRows = INT32_MAX - 1024;  // num_tokens * num_heads
constexpr uint64_t kWaitNs = 2000000000ull;  // give-up time of a pipeline wait

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct AttendWs {
  size_t req_entry, entry_cost, bound, part_o, part_ml, total;
};

int64_t entry_bound(int64_t num_tokens, int64_t num_reqs, int64_t group, int64_t rows) {
  return (num_tokens * group + rows - 1) / rows + num_reqs;
}

AttendWs attend_ws(int64_t num_reqs, int64_t max_entries, int64_t grid, int64_t rows,
                   int64_t head_dim) {
  AttendWs w{};
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = off;
    off = round_up(off + bytes, 256);
    return o;
  };
  w.req_entry = take(4 * static_cast<size_t>(num_reqs + 1));
  w.entry_cost = take(8 * static_cast<size_t>(max_entries + 1));
  w.bound = take(16 * static_cast<size_t>(grid + 1));
  w.part_o = take(4 * static_cast<size_t>(2 * grid * rows * head_dim));
  w.part_ml = take(8 * static_cast<size_t>(2 * grid * rows));
  w.total = off;
  return w;
}

// How a call is run: query rows per unit, keys per tile, CTAs.
struct Variant {
  int mt;  // row-block kernel: 16-row blocks per unit; 0: tensor-memory kernel
  int32_t rows, tile_log2, grid, overhead, min_cost;
};

// (At least two tiles a CTA; four with a list: 64-key tiles, one token over 1000 keys 12.7 us
// with four, 11.5 with two; lists of 512 11.5 and 13.4, where four leaves them uncut.)
Variant rows_variant(int mt, int head_dim, bool selected) {
  return Variant{mt, 16 * mt, rows_tile_keys(head_dim) == 64 ? 6 : 7,
                 kRowsCtasPerSm * device_sm_count(), 1, selected ? 4 : 2};
}

// Whether a list's units go to a warp each or to a CTA each, by what they take on a GB300 in
// tenths of a microsecond: a warp takes 1.1 us a sub-tile (16 keys at D = 128, 32 at 64) and 1.7 a
// unit, rounds of units one after another; a CTA's four warps share the sub-tiles at 0.9 each, but
// stand still for 2.6 between units, and up to `grid` units are cut evenly. (us, warp /
// CTA, D = 128, 8 kv heads: 2400 tokens with lists of 32: 64 / 206, 512: 594 / 610; 256 tokens,
// 128: 25 / 42, 2048: 288 / 219; 64 tokens, 512: 40 / 33, 2048: 144 / 69; one kv head, 8000
// tokens, 512: 260 / 278; D = 64: 141 / 160, 2048: 526 / 450.)
bool warp_per_list(const AttendParams& p, int head_dim, const Variant& v) {
  const int64_t sub = (p.topk + rows_tile_keys(head_dim) / 4 - 1) / (rows_tile_keys(head_dim) / 4);
  const int64_t one = static_cast<int64_t>(p.num_tokens) * p.num_kv_heads;
  const int64_t by_warp = one * ((p.group + 15) / 16), by_cta = one * ((p.group + v.rows - 1) / v.rows);
  const int64_t warps = 4 * v.grid;
  const int64_t warp_time = (by_warp + warps - 1) / warps * (11 * sub + 17) + 40;
  const int64_t cta_time = by_cta <= v.grid ? 10 * by_cta * sub / warps + 130
                                            : by_cta * (9 * sub / 4 + 26) / v.grid + 80;
  return warp_time < cta_time;
}

// Blocks of a cluster that share each of `units` units of at most `tiles` tiles, with no plan, no
// partial results in memory and no second launch; 0 where cutting all tiles evenly over the device
// is faster. A block takes 0.9 us a tile and 4; the cut's blocks take fewer tiles, but 11 more (for a
// list, whose units are cut late, 15). us, cut / cluster, D = 128, 8 kv heads: one request of 1000
// keys 11.5 / 6.2, 6000: 16.0 / 14.5, 12 000: 18.6 / 24.3; 16 of 1000: 19.1 / 13.3, of 3000: 40 /
// 35; 4 tokens with lists of 512: 18.1 / 6.2, 32 with 2048: 37 / 32. `most` bounds a block's tiles
// where lengths may differ, for only the cut evens them out.
int cluster_blocks(int64_t units, int64_t tiles, int64_t slack, int64_t most, const Variant& v) {
  int c = kMostCluster;
  while (c > 1 && (units * c > v.grid || c >= 2 * tiles)) c /= 2;
  const int64_t one = (tiles + c - 1) / c;
  return units * c <= v.grid && one <= most && one <= tiles * units / v.grid + slack ? c : 0;
}

constexpr int64_t kLittleTiles = 12;  // a block's

Variant tc_variant() { return Variant{0, kRowsTc, 7, device_sm_count(), 3, 4}; }

// What the largest call of at most these sizes needs. Fewer kv heads make larger groups and so more
// entries (8 bytes each): one kv head is counted with.
size_t most_workspace(int64_t num_tokens, int64_t num_reqs, int64_t num_heads, int64_t head_dim) {
  size_t most = 0;
  for (const Variant& v : {rows_variant(1, head_dim, true), rows_variant(2, head_dim, true), tc_variant()}) {
    const size_t n = attend_ws(num_reqs, entry_bound(num_tokens, num_reqs, num_heads, v.rows), v.grid,
                               v.rows, head_dim)
                         .total;
    most = n > most ? n : most;
  }
  return most;
}

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

// The checks that both forms share.
idx_status check_attend(const idx_attend* a) {
  if (!a) return IDX_ERR_INVALID_ARG;
  if (a->dtype != IDX_BF16 && a->dtype != IDX_FP16) return IDX_ERR_UNSUPPORTED;
  if (a->head_dim != 64 && a->head_dim != 128) return IDX_ERR_UNSUPPORTED;
  if (a->num_tokens < 0 || a->num_reqs < 0 || a->num_heads < 1 || a->num_kv_heads < 1)
    return IDX_ERR_INVALID_ARG;
  if (a->num_heads % a->num_kv_heads != 0) return IDX_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a->num_tokens) * a->num_heads > kMostRows) return IDX_ERR_UNSUPPORTED;
  if (!(a->scale > 0.f) || !isfinite(a->scale)) return IDX_ERR_INVALID_ARG;
  if (a->num_pages < 1 || a->num_pages > INT32_MAX || a->bt_width < 1 ||
      a->bt_width > kMostKeys / kPageTokens || a->bt_stride < a->bt_width)
    return IDX_ERR_INVALID_ARG;
  if (a->num_tokens == 0 || a->num_reqs == 0) return IDX_OK;
  if (!a->q || !a->k || !a->v || !a->out || !a->block_table || !a->query_start_loc)
    return IDX_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->out, 16) ||
      !aligned(a->block_table, 4) || !aligned(a->query_start_loc, 4) || !aligned(a->lse, 4))
    return IDX_ERR_INVALID_ARG;
  if (!stride_ok(a->q_stride_token) || !stride_ok(a->q_stride_head) ||
      !stride_ok(a->k_stride_page) || !stride_ok(a->k_stride_token) ||
      !stride_ok(a->k_stride_head) || !stride_ok(a->v_stride_page) ||
      !stride_ok(a->v_stride_token) || !stride_ok(a->v_stride_head))
    return IDX_ERR_INVALID_ARG;
  if ((!a->workspace && a->workspace_bytes) || !aligned(a->workspace, 256))
    return IDX_ERR_INVALID_ARG;
  return IDX_OK;
}

AttendParams attend_params(const idx_attend* a) {
  AttendParams p{};
  p.q = a->q;
  p.q_stride_token = a->q_stride_token;
  p.q_stride_head = a->q_stride_head;
  p.k = a->k;
  p.v = a->v;
  p.k_stride_page = a->k_stride_page;
  p.k_stride_token = a->k_stride_token;
  p.k_stride_head = a->k_stride_head;
  p.v_stride_page = a->v_stride_page;
  p.v_stride_token = a->v_stride_token;
  p.v_stride_head = a->v_stride_head;
  p.num_pages = a->num_pages;
  p.block_table = a->block_table;
  p.bt_stride = a->bt_stride;
  p.bt_width = a->bt_width;
  p.query_start_loc = a->query_start_loc;
  p.num_reqs = a->num_reqs;
  p.num_tokens = a->num_tokens;
  p.num_heads = a->num_heads;
  p.num_kv_heads = a->num_kv_heads;
  p.group = a->num_heads / a->num_kv_heads;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.window = kMostKeys;
  p.out = a->out;
  p.lse = a->lse;
  p.dev_error = a->dev_error;
  p.wait_ns = kWaitNs;
  return p;
}

void set_variant(AttendParams* p, const Variant& v) {
  p->rows = v.rows;
  p->tile_log2 = v.tile_log2;
  p->sinks_tiles = static_cast<int32_t>((static_cast<int64_t>(p->sinks) + (1 << v.tile_log2) - 1) >>
                                        v.tile_log2);
  p->grid = v.grid;
  p->unit_overhead = v.overhead;
  p->min_cost = v.min_cost;
}

idx_status place_workspace(AttendParams* p, const idx_attend* a, const Variant& v) {
  if (p->cluster && !a->workspace) return IDX_OK;
  p->max_entries =
      static_cast<int32_t>(entry_bound(a->num_tokens, a->num_reqs, p->group, v.rows));
  const AttendWs w = attend_ws(a->num_reqs, p->max_entries, v.grid, v.rows, a->head_dim);
  if (a->workspace_bytes < w.total) return IDX_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  p->req_entry = reinterpret_cast<int32_t*>(ws + w.req_entry);
  p->entry_cost = reinterpret_cast<int64_t*>(ws + w.entry_cost);
  p->bound = reinterpret_cast<int4*>(ws + w.bound);
  p->part_o = reinterpret_cast<float*>(ws + w.part_o);
  p->part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  return IDX_OK;
}

}  // namespace
}  // namespace saib

using namespace saib;

extern "C" {

idx_status indexer_attend_workspace_bytes(int32_t num_tokens, int32_t num_reqs, int32_t num_heads,
                                          int32_t num_kv_heads, int32_t head_dim, size_t* bytes) {
  if (!bytes || num_tokens < 0 || num_reqs < 0 || num_heads < 1 || num_kv_heads < 1 ||
      num_heads % num_kv_heads != 0)
    return IDX_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) ||
      static_cast<int64_t>(num_tokens) * num_heads > kMostRows)
    return IDX_ERR_UNSUPPORTED;
  *bytes = most_workspace(num_tokens, num_reqs, num_heads, head_dim);
  return IDX_OK;
}

idx_status indexer_attend_paged(const idx_attend* a, void* stream) {
  idx_status st = check_attend(a);
  if (st != IDX_OK) return st;
  if (a->window < 0 || a->sinks < 0 || a->max_query_len < 0) return IDX_ERR_INVALID_ARG;
  if (a->num_tokens == 0 || a->num_reqs == 0) return IDX_OK;
  if (!a->seq_lens || !aligned(a->seq_lens, 4)) return IDX_ERR_INVALID_ARG;
  AttendParams p = attend_params(a);
  p.seq_lens = a->seq_lens;
  if (a->window > 0) {
    p.window = std::min(a->window, kMostKeys);
    p.sinks = a->sinks;
  }
  const int64_t longest =
      a->max_query_len > 0 ? std::min(a->max_query_len, a->num_tokens) : a->num_tokens;
  // The row-block kernel holds 16 rows at once and reads K and V again for the next 16; from
  // 17 rows on the tensor-memory kernel is faster (24 requests of 8000 keys, 8 kv heads of 128:
  // 15 rows 132 against 140 us, 20 rows 173 against 142).
  const bool half = a->dtype == IDX_FP16;
  CUtensorMap kmap, vmap;
  const bool tc =
      longest * p.group > 16 && attend_tc_maps(p, a->head_dim, half, &kmap, &vmap);
  const Variant v = tc ? tc_variant() : rows_variant(1, a->head_dim, false);
  set_variant(&p, v);
  // (a window's tiles: those of the sinks, and the window and the new tokens, cut at both ends)
  const int64_t tile = int64_t{1} << v.tile_log2;
  const int64_t tiles =
      std::min((a->bt_width * int64_t{kPageTokens} + tile - 1) / tile,
               p.sinks_tiles + (p.window + longest + tile - 1) / tile + 1);
  if (!tc && longest * p.group <= v.rows) {
    const int64_t units = static_cast<int64_t>(a->num_reqs) * p.num_kv_heads;
    p.cluster = cluster_blocks(units, tiles, 10, 16, v);
    if (p.cluster) p.grid = static_cast<int32_t>(units * p.cluster);
  }
  if ((st = place_workspace(&p, a, v)) != IDX_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.cluster) return launch_attend_rows(p, a->head_dim, half, v.mt, s);
  // The chunk kernel's blocks plan for themselves when there is little work: a launch less is 4 us
  // less of the host's time, which is what such calls take (100 tokens of a first prompt: 33 us a
  // call, then 29; on the device 256 tokens 20.9, then 15.7). The cuts of the planning kernel are
  // finer (26 requests of up to 9000 keys 130 us, else 134).
  const bool little = int64_t{p.max_entries} * p.num_kv_heads * tiles <= kLittleTiles * v.grid;
  p.self_plan = (!tc || little) && a->num_reqs <= kSelfPlanReqs &&
                longest * p.group <= kSelfPlanEntries * int64_t{v.rows};
  if (!p.self_plan && (st = launch_attend_plan(p, s)) != IDX_OK) return st;
  st = tc ? launch_attend_tc(p, a->head_dim, half, kmap, vmap, s)
          : launch_attend_rows(p, a->head_dim, half, v.mt, s);
  if (st != IDX_OK) return st;
  return launch_attend_combine(p, a->head_dim, half, s);
}

idx_status indexer_attend_selected(const idx_attend* a, void* stream) {
  idx_status st = check_attend(a);
  if (st != IDX_OK) return st;
  if (a->topk < 1 || a->indices_stride < a->topk) return IDX_ERR_INVALID_ARG;
  if (a->num_tokens == 0 || a->num_reqs == 0) return IDX_OK;
  if (!a->indices || !aligned(a->indices, 4)) return IDX_ERR_INVALID_ARG;
  AttendParams p = attend_params(a);
  p.indices = a->indices;
  p.indices_stride = a->indices_stride;
  p.topk = a->topk;
  p.same_strides = p.k_stride_page == p.v_stride_page && p.k_stride_token == p.v_stride_token;
  const Variant v = rows_variant(p.group <= 16 ? 1 : 2, a->head_dim, true);
  set_variant(&p, v);
  if (v.mt == 1) {
    const int64_t tile = int64_t{1} << v.tile_log2;
    const int64_t units = static_cast<int64_t>(a->num_tokens) * p.num_kv_heads;
    p.cluster = cluster_blocks(units, (a->topk + tile - 1) / tile, 14, INT32_MAX, v);
    if (p.cluster) p.grid = static_cast<int32_t>(units * p.cluster);
  }
  if ((st = place_workspace(&p, a, v)) != IDX_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = a->dtype == IDX_FP16;
  if (!p.cluster && warp_per_list(p, a->head_dim, v)) {
    p.rows = 16;
    p.tile_log2 = a->head_dim == 64 ? 5 : 4;
    return launch_attend_lists(p, a->head_dim, half, s);
  }
  if ((st = launch_attend_rows(p, a->head_dim, half, v.mt, s)) != IDX_OK || p.cluster) return st;
  return launch_attend_combine(p, a->head_dim, half, s);
}

}  // extern "C"
