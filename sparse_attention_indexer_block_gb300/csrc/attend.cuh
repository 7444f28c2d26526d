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

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

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
  int32_t same_strides;            // K's and V's pages and tokens lie alike (selected form)
  int32_t num_reqs, num_tokens;
  int32_t num_heads, num_kv_heads, group;
  float scale_log2;                // scale * log2(e)
  int32_t window;                  // (2^30: none)
  int32_t sinks;
  int32_t sinks_tiles;             // tiles that hold them
  void* out;                       // [num_tokens, num_heads, head_dim]
  float* lse;                      // nullable [num_tokens, num_heads]
  // workspace
  int32_t* req_entry;              // [num_reqs + 1] first entry of each request
  int64_t* entry_cost;             // [max_entries + 1] exclusive prefix of the entries' costs
  int4* bound;                     // [grid + 1] first piece of each CTA: entry, kv head, tile, request
  float* part_o;                   // [2 * grid, rows, head_dim] unnormalised pieces
  float2* part_ml;                 // [2 * grid, rows] their maximum and sum
  int32_t max_entries;
  int32_t self_plan;               // the CTAs work `bound` out for themselves
  int32_t min_cost;                // least work of a CTA (a tile: 1, of a tree tile_cost)
  int32_t cluster;                 // row-block kernel: blocks that share a unit; 0: a plan cuts
  int32_t cluster_entries;         // trees: clusters of a request's kv head
  int32_t tile_cost, narrow_cost;  // trees: what a tile costs, and one of a unit of at most 128 rows
  int32_t grid;                    // CTAs of the row-block launch
  int32_t rows;                    // query rows of a unit
  int32_t tile_log2;               // keys of a tile
  int32_t unit_overhead;           // what a unit's start and end cost, in the same measure
  uint32_t* dev_error;
  uint64_t wait_ns;
  // a tree's: the new tokens that each of them sees (bit j of a row's words: new token j of its
  // request), and their positions (nullptr without a window)
  const int32_t* masks;            // [num_tokens, mask_words]
  int64_t mask_stride;
  int32_t mask_words;
  const int32_t* positions;        // [num_tokens]
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
  // positions of the unit's first and last token; of a tree the lowest that a new token can have,
  // and the last key
  int32_t p_lo, p_hi;

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
  return (r.nq * p.group + p.rows - 1) / p.rows;
}

// (All in 32 bits: num_tokens * num_heads and the table's tokens fit with room for a tile.)
// kTree: any row of a request may see any of its new tokens, so its units have the same tiles.
template <bool kTree>
__device__ __forceinline__ UnitTiles unit_tiles(const AttendParams& p, const ReqShape& r, int32_t u) {
  UnitTiles t;
  const int32_t row0 = u * p.rows;
  const int32_t row1 = min(row0 + p.rows, r.nq * p.group);
  const int32_t ahead = r.keys - r.nq;
  t.p_lo = kTree ? ahead : ahead + row0 / p.group;
  t.p_hi = kTree ? r.keys - 1 : ahead + (row1 - 1) / p.group;
  if (t.p_hi < 0) {
    t.first = t.skip = t.count = 0;
    return t;
  }
  const int32_t end = (t.p_hi >> p.tile_log2) + 1;
  const int32_t lo = max(t.p_lo, 0) - p.window + 1;
  const int32_t start = max(lo, 0) >> p.tile_log2;
  t.first = min(p.sinks_tiles, start);
  t.skip = start - t.first;
  t.count = end - t.skip;
  return t;
}

// What a tile of entry u costs a CTA.
template <bool kTree>
__device__ __forceinline__ int32_t tile_cost(const AttendParams& p, const ReqShape& r, int32_t u) {
  if (!kTree) return 1;
  return r.nq * p.group - u * p.rows > 128 ? p.tile_cost : p.narrow_cost;
}

// A piece: tiles [t0, t1) of a unit.
struct Piece {
  int32_t req, head;  // request, kv head
  int32_t row0;       // first row of the unit: (token - q0) * group + head of the group
  int32_t rows;       // rows that exist
  int32_t q0;         // first token of the request (selected form: the token)
  int32_t ahead;      // position of the request's first new token
  UnitTiles tiles;
  int32_t t0, t1;

  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles.count; }
};

// Token, head and position of a unit's row.
__device__ __forceinline__ void row_place(const AttendParams& p, const Piece& u, int r,
                                          int64_t* token, int* head, int32_t* pos) {
  const int32_t row = u.row0 + r;
  const int32_t i = row / p.group;
  *token = static_cast<int64_t>(u.q0) + i;
  *head = u.head * p.group + (row - i * p.group);
  *pos = u.ahead + i;
}

// The n lowest bits of a word, n clamped to [0, 32].
__device__ __forceinline__ uint32_t low_bits(int32_t n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// What a row of a tree sees: the keys before the new tokens (with a window, those that it leaves),
// and the new tokens that its mask names.
struct TreeRow {
  const int32_t* mask;  // nullptr: a row that does not exist, which sees nothing
  int32_t ahead, keys;  // the request's keys without and with its new tokens
  int32_t pos;

  TreeRow() = default;
  __device__ __forceinline__ TreeRow(const AttendParams& p, const Piece& u, int64_t token, bool there)
      : mask(nullptr), ahead(u.ahead), keys(u.tiles.p_hi + 1), pos(0) {
    if (!there) return;
    mask = p.masks + token * p.mask_stride;
    if (p.positions) pos = max(min(max(p.positions[token], ahead), keys - 1), 0);
  }

  // Bit i: key s0 + i.
  __device__ __forceinline__ uint32_t sees(const AttendParams& p, int32_t s0) const {
    if (!mask) return 0;
    uint32_t see = low_bits(ahead - s0);
    if (p.positions) see &= ~low_bits(pos - p.window + 1 - s0) | low_bits(p.sinks - s0);
    const int32_t c = s0 - ahead;  // new token of bit 0
    if (c > -32) {
      const int32_t w = c >> 5;
      const uint32_t lo = w >= 0 && w < p.mask_words ? mask[w] : 0;
      const uint32_t hi = w + 1 < p.mask_words ? mask[w + 1] : 0;
      see |= __funnelshift_r(lo, hi, c & 31) & low_bits(keys - s0);
    }
    return see;
  }
};

// The pieces of a CTA's range in the paged form, in order; with kFirstLast, a
// first piece that begins inside its unit comes last. (The CTAs of one request
// and kv head then all begin at its first keys and read them at the same time:
// from HBM once, from L2 otherwise.)
template <bool kFirstLast, bool kTree>
struct PieceWalk {
  int4 cur, end;
  ReqShape shape;   // of request cur.w
  int32_t entries;  // its entries
  bool done, stale;
  int later;        // kFirstLast: 2 to be passed over, 1 to come, 0 none

  PieceWalk() = default;
  __device__ __forceinline__ PieceWalk(const AttendParams& p, const int4& from, const int4& to)
      : cur(from), end(to), done(from.w >= p.num_reqs), stale(true),
        later(kFirstLast && from.z > 0 && !(from.x == to.x && from.y == to.y && from.w == to.w) ? 2
                                                                                              : 0) {}
  // with the first request's shape at hand
  __device__ __forceinline__ PieceWalk(const AttendParams& p, const int4& from, const int4& to,
                                       const ReqShape& first)
      : PieceWalk(p, from, to) {
    shape = first;
    entries = request_entries(p, first);
    stale = false;
  }

  __device__ __forceinline__ bool next(const AttendParams& p, Piece* u) {
    for (;;) {
      if (done) {
        if (!kFirstLast || later != 1) return false;
        cur = p.bound[blockIdx.x];
        end = make_int4(cur.x, cur.y, INT32_MAX, cur.w);
        stale = true;
        later = 0;
      }
      const bool last = cur.w == end.w && cur.y == end.y && cur.x == end.x;
      if (last && end.z <= cur.z) {
        done = true;
        continue;
      }
      if (stale) {
        shape = request_shape(p, cur.w, false);
        entries = request_entries(p, shape);
        stale = false;
      }
      u->req = cur.w;
      u->head = cur.y;
      u->row0 = cur.x * p.rows;
      u->rows = min(p.rows, shape.nq * p.group - u->row0);
      u->q0 = shape.q0;
      u->ahead = shape.keys - shape.nq;
      u->tiles = unit_tiles<kTree>(p, shape, cur.x);
      u->t0 = cur.z;
      u->t1 = last ? min(end.z, u->tiles.count) : u->tiles.count;
      done = last;
      if (!last) {
        cur.z = 0;
        if (++cur.x == entries) {
          cur.x = 0;
          if (++cur.y == p.num_kv_heads) {
            cur.y = 0;
            do {
              if (++cur.w == p.num_reqs) {
                done = true;
                break;
              }
              shape = request_shape(p, cur.w, false);
              entries = request_entries(p, shape);
            } while (entries == 0);
          }
        }
      }
      if (kFirstLast && later == 2) {
        later = 1;
        continue;
      }
      return true;
    }
  }
};

// A pair of T values with its infinities and NaNs replaced by 0.
template <typename T>
__device__ __forceinline__ uint32_t clear_nonfinite(uint32_t v) {
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  if ((v & kExp) == kExp) v &= 0xffff0000u;
  if ((v & (kExp << 16)) == kExp << 16) v &= 0xffffu;
  return v;
}

// Bits of v whose 16-bit halves are infinities or NaNs (their top bits, else 0).
template <typename T>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t v) {
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr uint32_t kExp = kHalf ? 0x7c007c00u : 0x7f807f80u;
  return ((v & kExp) + (kHalf ? 0x04000400u : 0x00800080u)) & 0x80008000u;
}

// Two fp32 values as a pair of T, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 16 bytes, asynchronously; `valid` false: zeros, and src is not read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr float kLn2 = 0.693147180559945309f;

// A row's weights are exp2(x - m) with m, which the kernels keep and pass on as its maximum, the
// largest score less kTopWeight: the largest weight is 2^kTopWeight. bf16 has the exponents of fp32
// and needs no more than 1. fp16 has no values below 2^-24: beside a weight of 1, those below 2^-25
// are lost to the second product, though not to the sum (65 536 keys 17.5 nats below one more: most
// of their 1.6e-3 of the output). Beside 2^15 they are lost below 2^-40 of the largest.
template <typename T>
constexpr float kTopWeight = std::is_same<T, __half>::value ? 15.f : 0.f;

// The chunk kernel raises m (and rescales the row's accumulator) only when a weight would pass the
// last one's largest by 2^8: bf16's then stay below 2^8, with the same relative precision, and
// fp16's, whose largest is first 2^7, below 2^15.
constexpr float kLazyRaise = 8.f;
template <typename T>
constexpr float kTopWeightTc = kTopWeight<T> == 0.f ? 0.f : kTopWeight<T> - kLazyRaise;

// lse of a row whose weights exp2(x - m) sum up to l (scaled by 2^-kTop, as m is moved by it: then
// nothing is added to the logarithm's error).
template <int kTop>
__device__ __forceinline__ float row_lse(float m, float l) {
  constexpr float kDown = 1.f / static_cast<float>(1 << kTop);
  return ((m + static_cast<float>(kTop)) + log2f(l * kDown)) * kLn2;
}

// Keys of a tile of the row-block kernel: 4 KB of K per warp either way.
__host__ __device__ constexpr int rows_tile_keys(int head_dim) { return head_dim == 64 ? 128 : 64; }

constexpr int kTileTc = 128;   // keys of a tensor-memory kernel's tile: two pages
constexpr int kRowsTc = 256;   // its query rows: two accumulators of 128

// a / b for a >= 0, b > 0, in 32 bits where both fit (a fifth of the time).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// CTAs that take part in work of cost `all` in `units` units: as many as have
// min_cost each, and where it costs at most a quarter of them, a number that
// cuts equal units alike or not at all (a cut costs a join, a CTA's second piece
// 7 us without copies in flight).
__device__ __forceinline__ int64_t cutters(const AttendParams& p, int64_t all, int64_t units) {
  const int64_t most = max(min(quotient(all, p.min_cost), static_cast<int64_t>(p.grid)), int64_t{1});
  if (units < 1 || units > most) return most;
  const int64_t n = quotient(most, units) * units;
  return 4 * n >= 3 * most ? n : most;
}

// Position of cut c of n.
__device__ __forceinline__ int64_t cut_position(int64_t all, int64_t n, int c) {
  if (c >= n) return all;
  const int64_t q = quotient(all, n);
  return q * c + quotient((all - q * n) * c, n);
}

// Inclusive sum of v over the block's threads; *total gets the sum of all.
template <int kThreads>
__device__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = lane < kThreads / 32 ? warp_sums[lane] : 0;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += o;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[kThreads / 32 - 1];
  return v + (warp ? warp_sums[warp - 1] : 0);
}

// The same from the costs of whole requests (cost[b]: exclusive prefix of
// their units' costs for one kv head), which a CTA works out for itself
// when there are few requests.
template <bool kTree>
__device__ inline int4 cut_at_request(const AttendParams& p, const int64_t* cost, int64_t units,
                                      int c) {
  const int64_t all = cost[p.num_reqs] * p.num_kv_heads, n = cutters(p, all, units);
  const int64_t pos = cut_position(all, n, c);
  if (pos >= all) return make_int4(0, 0, 0, p.num_reqs);
  int lo = 0, hi = p.num_reqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cost[mid] * p.num_kv_heads <= pos) lo = mid; else hi = mid - 1;
  }
  const int64_t one = cost[lo + 1] - cost[lo], rest = pos - cost[lo] * p.num_kv_heads;
  int32_t head = static_cast<int32_t>(quotient(rest, one));
  int64_t off = rest - head * one;
  const ReqShape r = request_shape(p, lo, false);
  int32_t u = 0, tiles, of_tile;
  for (;; ++u) {
    of_tile = tile_cost<kTree>(p, r, u);
    tiles = unit_tiles<kTree>(p, r, u).count;
    if (off < tiles * of_tile + p.unit_overhead) break;
    off -= tiles * of_tile + p.unit_overhead;
  }
  // a cut near a unit's end moves there (by at most a sixteenth of a CTA's work)
  int32_t t = static_cast<int32_t>(max(off - p.unit_overhead, int64_t{0})) / of_tile;
  const int64_t near = quotient(all, n) / 16 / of_tile;
  if (t <= near) t = 0;
  if (t > 0 && tiles - t <= near) {
    t = 0;
    if (++u == request_entries(p, r)) {
      u = 0;
      if (++head == p.num_kv_heads) {
        head = 0;
        do ++lo;
        while (lo < p.num_reqs && cost[lo + 1] == cost[lo]);
      }
    }
  }
  return make_int4(u, head, t, lo);
}

// Requests, and entries of each, up to which the CTAs plan for themselves: one
// scan of the requests' costs each, against a launch of the planning kernel
// (4 us).
constexpr int kSelfPlanReqs = 512, kSelfPlanEntries = 8;
constexpr int kMostCluster = 8;
constexpr int kMostTreeCluster = 16;  // (more than eight where the device has room for them)

// The cuts at both ends of a CTA's range and its first request's shape, by its
// kThreads threads; `cost` has room for num_reqs + 1. p.bound gets them too, for the join.
template <int kThreads, bool kTree>
__device__ void self_plan(const AttendParams& p, int cta, int64_t* cost, int64_t* sums, int4* cuts,
                          ReqShape* first) {
  constexpr int kEntryShift = 40;  // one scan for both sums: costs below, entries above
  int64_t carry = 0, total;
  for (int b0 = 0; b0 < p.num_reqs; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int64_t n = 0;
    if (b < p.num_reqs) {
      const ReqShape r = request_shape(p, b, cta == 0);
      const int32_t e = request_entries(p, r);
      for (int32_t i = 0; i < e; ++i)
        n += unit_tiles<kTree>(p, r, i).count * tile_cost<kTree>(p, r, i) + p.unit_overhead;
      n += static_cast<int64_t>(e) << kEntryShift;
    }
    const int64_t incl = carry + block_scan<kThreads>(n, sums, &total);
    if (b < p.num_reqs) cost[b + 1] = incl & ((int64_t{1} << kEntryShift) - 1);
    carry += total;
  }
  const int64_t units = (carry >> kEntryShift) * p.num_kv_heads;
  if (threadIdx.x == 0) cost[0] = 0;
  __syncthreads();
  if (threadIdx.x < 2) {
    const int4 at = cut_at_request<kTree>(p, cost, units, cta + threadIdx.x);
    cuts[threadIdx.x] = at;
    if (threadIdx.x == 0 && at.w < p.num_reqs) *first = request_shape(p, at.w, false);
    if (threadIdx.x == 0 || cta == p.grid - 1) p.bound[cta + threadIdx.x] = at;
  }
  __syncthreads();
}

// Raises the kernel's limit of dynamic shared memory, once per device (any host
// thread; doing it twice is harmless). kRegs: registers a thread that the kernel
// must have been built with (0: any).
template <int kBytes, int kRegs, typename Kernel>
inline cudaError_t allow_smem(Kernel* kernel, std::atomic<bool>* configured) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  if (cached && configured[dev].load(std::memory_order_acquire)) return cudaSuccess;
  if (kRegs) {
    cudaFuncAttributes a;
    if ((e = cudaFuncGetAttributes(&a, kernel)) != cudaSuccess) return e;
    if (a.numRegs != kRegs) return cudaErrorInvalidConfiguration;
  }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e == cudaSuccess && cached) configured[dev].store(true, std::memory_order_release);
  return e;
}

// Clusters of kMostTreeCluster blocks of a tree's row-block kernel that the current device runs at once
// (0: none can be placed).
int attend_wide_clusters(int head_dim, bool half);

// Launchers.
idx_status launch_attend_plan(const AttendParams& p, cudaStream_t s);
idx_status launch_attend_rows(const AttendParams& p, int head_dim, bool half, int mt, cudaStream_t s);
// The chunk kernel's tensor maps of the caches; false when their strides suit none.
bool attend_tc_maps(const AttendParams& p, int head_dim, bool half, CUtensorMap* kmap,
                    CUtensorMap* vmap);
idx_status launch_attend_tc(const AttendParams& p, int head_dim, bool half, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, cudaStream_t s);
// The join of the chunk kernel's pieces of trees (launch_attend_combine: of all others).
idx_status launch_attend_join(const AttendParams& p, int head_dim, bool half, cudaStream_t s);
idx_status launch_attend_lists(const AttendParams& p, int head_dim, bool half, cudaStream_t s);
idx_status launch_attend_combine(const AttendParams& p, int head_dim, bool half, cudaStream_t s);

}  // namespace saib
