// The pages of the caches: copies between pages, forks of requests (shared
// full pages, a copied last one), freeing, and compaction of a pool. A page is
// free when no block-table row holds it, i.e. when its reference count is 0;
// pages are handed out lowest first, so every result is a function of the
// tables alone.
#include <algorithm>

#include "internal.h"

namespace saib {

namespace {

constexpr int kScanThreads = 1024;
constexpr int kCopyThreads = 128;
constexpr int kCopyLoads = 4;                           // 16-byte loads in flight per thread
constexpr int kChunk = kCopyThreads * 16 * kCopyLoads;  // bytes of a page that a CTA copies at once
constexpr int kCopyCtasPerSm = 16;
constexpr int kPoolsPerLaunch = 64;            // pools in one launch's parameters

struct Pools {
  uint8_t* base[kPoolsPerLaunch];
  int64_t stride[kPoolsPerLaunch];
  int32_t bytes[kPoolsPerLaunch];
  int32_t chunk0[kPoolsPerLaunch + 1];  // exclusive prefix of the pools' chunks
  int32_t num;
};

struct Tables {
  int32_t* block_table;
  int64_t bt_stride;
  int32_t bt_width, num_rows;
  int32_t* seq_lens;
  int32_t* ref_counts;
  int32_t num_pages;
  uint32_t* err;
};

// Moves of a compaction, as its second launch leaves them.
struct Moves {
  const int32_t* count;  // moves
  int32_t* remap;        // nullptr: no tables to follow
};

// Pages that a row of n keys holds, n clamped to the table's width.
__device__ __forceinline__ int32_t row_pages(const Tables& t, int32_t n, bool* part) {
  const int64_t most = static_cast<int64_t>(t.bt_width) * kPageTokens;
  if (n < 0 || n > most) {
    set_error(t.err, IDX_DEV_BAD_LEN);
    n = n < 0 ? 0 : static_cast<int32_t>(most);
  }
  if (part) *part = (n % kPageTokens) != 0;
  return (n + kPageTokens - 1) / kPageTokens;
}

// Exclusive sum of v over the block; *total gets the sum of all.
__device__ int block_exclusive(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int s = v;
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = lane < warps ? warp_sums[lane] : 0;
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += o;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[warps - 1];
  return s - v + (warp ? warp_sums[warp - 1] : 0);
}

// ---------------------------------------------------------------------------
// copies
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Pages src[i] of every pool to dst[i], in chunks of 8 KB spread over the grid
// (16 small CTAs an SM, four 16-byte loads in flight per thread: 3000 pages of
// 74 KB at 6.1 TB/s read and written, 128 KB at 6.5, 8 KB at 5.5; two loads and
// 256 threads: 5.5, 5.6, 4.4); with moves.remap, the tables follow the moves of
// a compaction first. Bound by HBM: each byte is read and written once.
__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const Pools pools, const int32_t* src, const int32_t* dst, int32_t n,
                      const Tables t, const Moves moves) {
  pdl_wait();
  pdl_trigger();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
  if (moves.count) n = *moves.count;
  if (moves.remap) {
    volatile int32_t* remap = moves.remap;
    // an entry of a moved page reads as -2 - move until its own thread below has put the new
    // page there; both lead to the same page
    const auto place = [&](int32_t page) -> int32_t {
      const int32_t v = remap[page];
      return v <= -2 ? dst[-2 - v] : v;
    };
    for (int64_t i = me; i < static_cast<int64_t>(t.num_rows) * t.bt_width; i += step) {
      const int32_t row = static_cast<int32_t>(i / t.bt_width);
      const int32_t col = static_cast<int32_t>(i % t.bt_width);
      if (col >= row_pages(t, t.seq_lens[row], nullptr)) continue;
      int32_t* e = t.block_table + row * t.bt_stride + col;
      const int32_t page = *e;
      if (page < 0 || page >= t.num_pages) {
        set_error(t.err, IDX_DEV_BAD_BLOCK);
        continue;
      }
      const int32_t to = place(page);
      if (to < 0) set_error(t.err, IDX_DEV_BAD_REF);
      else if (to != page) *e = to;
    }
    for (int64_t i = me; i < n; i += step) {
      t.ref_counts[dst[i]] = t.ref_counts[src[i]];
      t.ref_counts[src[i]] = 0;
      remap[src[i]] = dst[i];
    }
  }
  const int32_t per_page = pools.chunk0[pools.num];
  const int64_t tasks = static_cast<int64_t>(n) * per_page;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int32_t i = static_cast<int32_t>(task / per_page);
    const int32_t part = static_cast<int32_t>(task % per_page);
    const int32_t a = src[i], b = dst[i];
    if (a < 0 || b < 0 || a == b) continue;
    if (a >= t.num_pages || b >= t.num_pages) {
      if (threadIdx.x == 0) set_error(t.err, IDX_DEV_BAD_BLOCK);
      continue;
    }
    int lo = 0, hi = pools.num - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pools.chunk0[mid] <= part) lo = mid; else hi = mid - 1;
    }
    const int32_t off = (part - pools.chunk0[lo]) * kChunk + threadIdx.x * 16;
    const uint8_t* from = pools.base[lo] + a * pools.stride[lo] + off;
    uint8_t* to = pools.base[lo] + b * pools.stride[lo] + off;
    constexpr int kStep = kCopyThreads * 16;
    uint4 v[kCopyLoads];
#pragma unroll
    for (int e = 0; e < kCopyLoads; ++e)
      if (off + e * kStep < pools.bytes[lo])
        v[e] = ld_stream(reinterpret_cast<const uint4*>(from + e * kStep));
#pragma unroll
    for (int e = 0; e < kCopyLoads; ++e)
      if (off + e * kStep < pools.bytes[lo]) *reinterpret_cast<uint4*>(to + e * kStep) = v[e];
  }
}

// ---------------------------------------------------------------------------
// forks
// ---------------------------------------------------------------------------

// Block 0 hands out the children's fresh pages (the k-th fork that needs one
// gets the k-th lowest free page) and writes their lengths and the copies to
// make; block 1 + i gives child i its parent's full pages. The counts that the
// other blocks raise are of pages in use, so block 0 sees the same free pages
// whenever it looks. Bound by latency: a scan of the reference counts up to
// the last page handed out.
__global__ void __launch_bounds__(kScanThreads)
    fork_pages_kernel(const Tables t, const int32_t* parents, const int32_t* children, int32_t n,
                      int32_t* copy_src, int32_t* copy_dst) {
  pdl_wait();
  pdl_trigger();
  const auto rows_ok = [&](int32_t a, int32_t b) {
    return a >= 0 && a < t.num_rows && b >= 0 && b < t.num_rows && a != b;
  };
  if (blockIdx.x > 0) {
    const int32_t i = blockIdx.x - 1, a = parents[i], b = children[i];
    if (!rows_ok(a, b)) return;
    bool part = false;
    int32_t full = row_pages(t, t.seq_lens[a], &part);
    if (part) --full;
    for (int32_t c = threadIdx.x; c < full; c += kScanThreads) {
      const int32_t page = t.block_table[a * t.bt_stride + c];
      t.block_table[b * t.bt_stride + c] = page;
      if (page >= 0 && page < t.num_pages) atomicAdd(t.ref_counts + page, 1);
      else set_error(t.err, IDX_DEV_BAD_BLOCK);
    }
    return;
  }
  // Pages of child i's parent, whether its last one is a partial one (to be copied), and whether
  // that one lies outside the pools; `report`: sets the error bits.
  struct Parent {
    int32_t pages = 0, last = 0;
    bool ok = false, part = false, bad = false;
    __device__ __forceinline__ bool copied() const { return part && !bad; }
  };
  const auto parent_of = [&](int32_t i, bool report) -> Parent {
    Parent q;
    if (i >= n) return q;
    q.ok = rows_ok(parents[i], children[i]);
    if (!q.ok) {
      if (report) set_error(t.err, IDX_DEV_BAD_ROW);
      return q;
    }
    q.pages = row_pages(t, t.seq_lens[parents[i]], &q.part);
    if (q.part) {
      q.last = t.block_table[parents[i] * t.bt_stride + q.pages - 1];
      q.bad = q.last < 0 || q.last >= t.num_pages;
      if (q.bad && report) set_error(t.err, IDX_DEV_BAD_BLOCK);
    }
    return q;
  };
  __shared__ int sums[32];
  int need_all = 0, total;
  for (int32_t i0 = 0; i0 < n; i0 += kScanThreads) {
    const int32_t i = i0 + threadIdx.x;
    if (i < n) {
      copy_src[i] = -1;
      copy_dst[i] = -1;
    }
    block_exclusive(parent_of(i, true).copied(), sums, &total);
    need_all += total;
  }
  // the lowest free pages, in order, into copy_dst
  int found = 0;
  constexpr int kPer = 4;
  for (int64_t p0 = 0; p0 < t.num_pages && found < need_all; p0 += kScanThreads * kPer) {
    const int64_t page = p0 + threadIdx.x * kPer;
    bool zero[kPer];
    int cnt = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      zero[e] = page + e < t.num_pages && t.ref_counts[page + e] == 0;
      cnt += zero[e];
    }
    int k = found + block_exclusive(cnt, sums, &total);
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (zero[e]) {
        if (k < need_all) copy_dst[k] = static_cast<int32_t>(page + e);
        ++k;
      }
    found += total;
  }
  __syncthreads();
  int base = 0;
  for (int32_t i0 = 0; i0 < n; i0 += kScanThreads) {
    const int32_t i = i0 + threadIdx.x;
    const Parent q = parent_of(i, false);
    const int k = base + block_exclusive(q.copied(), sums, &total);
    base += total;
    if (!q.ok) continue;
    int32_t len = q.part ? t.seq_lens[parents[i]] : q.pages * kPageTokens;
    if (q.copied() && k < found) {
      const int32_t fresh = copy_dst[k];
      copy_src[k] = q.last;
      t.block_table[children[i] * t.bt_stride + q.pages - 1] = fresh;
      t.ref_counts[fresh] = 1;
    } else if (q.part) {
      if (!q.bad) set_error(t.err, IDX_DEV_NO_PAGE);
      len = (q.pages - 1) * kPageTokens;
    }
    t.seq_lens[children[i]] = len;
  }
}

// ---------------------------------------------------------------------------
// freeing and compaction
// ---------------------------------------------------------------------------

// One block per row: its pages lose a reference, its length becomes 0.
__global__ void __launch_bounds__(kScanThreads)
    free_pages_kernel(const Tables t, const int32_t* rows) {
  pdl_wait();
  pdl_trigger();
  const int32_t row = rows[blockIdx.x];
  if (row < 0 || row >= t.num_rows) {
    if (threadIdx.x == 0) set_error(t.err, IDX_DEV_BAD_ROW);
    return;
  }
  const int32_t pages = row_pages(t, t.seq_lens[row], nullptr);
  for (int32_t c = threadIdx.x; c < pages; c += kScanThreads) {
    const int32_t page = t.block_table[row * t.bt_stride + c];
    if (page < 0 || page >= t.num_pages) {
      set_error(t.err, IDX_DEV_BAD_BLOCK);
    } else if (atomicSub(t.ref_counts + page, 1) <= 0) {
      atomicAdd(t.ref_counts + page, 1);
      set_error(t.err, IDX_DEV_BAD_REF);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) t.seq_lens[row] = 0;
}

// Pages in use of each block's kScanThreads pages.
__global__ void __launch_bounds__(kScanThreads)
    count_live_kernel(const int32_t* refs, int32_t num_pages, int32_t* counts) {
  pdl_wait();
  pdl_trigger();
  const int64_t page = static_cast<int64_t>(blockIdx.x) * kScanThreads + threadIdx.x;
  const int n = __syncthreads_count(page < num_pages && refs[page] > 0);
  if (threadIdx.x == 0) counts[blockIdx.x] = n;
}

// With n pages in use: the i-th of those at n or past it moves to the i-th free
// page below n. A thread per page ranks its page among the used ones below it;
// a used page past n has as many movers before it as used pages less those
// below n, a free page below n as many holes before it as pages less used ones.
__global__ void __launch_bounds__(kScanThreads)
    plan_moves_kernel(const int32_t* refs, int32_t num_pages, const int32_t* counts,
                      int32_t blocks, int32_t* remap, int32_t* src, int32_t* dst, int32_t* num_live,
                      int32_t* num_moves) {
  __shared__ int sums[32];
  pdl_wait();
  pdl_trigger();
  // used pages before this block's, and all
  int before = 0, all = 0, total;
  for (int b = threadIdx.x; b < blocks; b += kScanThreads) {
    const int c = counts[b];
    all += c;
    if (b < static_cast<int>(blockIdx.x)) before += c;
  }
  block_exclusive(all, sums, &total);
  all = total;
  block_exclusive(before, sums, &total);
  before = total;
  // used pages below `all`
  int low = 0;
  const int cut = all / kScanThreads;
  for (int b = threadIdx.x; b < cut && b < blocks; b += kScanThreads) low += counts[b];
  const int64_t at = static_cast<int64_t>(cut) * kScanThreads + threadIdx.x;
  if (at < all && refs[at] > 0) ++low;
  block_exclusive(low, sums, &total);
  low = total;
  const int64_t page = static_cast<int64_t>(blockIdx.x) * kScanThreads + threadIdx.x;
  const bool live = page < num_pages && refs[page] > 0;
  const int rank = before + block_exclusive(live, sums, &total);
  if (page < num_pages) {
    int32_t to = live ? static_cast<int32_t>(page) : -1;
    if (live && page >= all) {
      const int i = rank - low;
      src[i] = static_cast<int32_t>(page);
      to = -2 - i;
    } else if (!live && page < all) {
      dst[page - rank] = static_cast<int32_t>(page);
    }
    remap[page] = to;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *num_live = all;
    *num_moves = all - low;
  }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

idx_status check_pools(const idx_page_pool* pools, int32_t num_pools, int64_t num_pages) {
  if (num_pools < 0 || (num_pools > 0 && !pools) || num_pages < 1 || num_pages > INT32_MAX / 2)
    return IDX_ERR_INVALID_ARG;
  for (int32_t i = 0; i < num_pools; ++i) {
    const idx_page_pool& q = pools[i];
    if (!q.base || q.page_bytes < 1 || q.page_stride < q.page_bytes) return IDX_ERR_INVALID_ARG;
    if (!aligned(q.base, 16) || q.page_bytes % 16 || q.page_stride % 16) return IDX_ERR_INVALID_ARG;
    if (q.page_bytes > (1 << 28)) return IDX_ERR_UNSUPPORTED;
  }
  return IDX_OK;
}

idx_status check_tables(const Tables& t) {
  if (!t.block_table || !t.seq_lens || !t.ref_counts || t.num_rows < 1 || t.bt_width < 1 ||
      t.bt_width > INT32_MAX / kPageTokens || t.bt_stride < t.bt_width)
    return IDX_ERR_INVALID_ARG;
  if (!aligned(t.block_table, 4) || !aligned(t.seq_lens, 4) || !aligned(t.ref_counts, 4))
    return IDX_ERR_INVALID_ARG;
  return IDX_OK;
}

// Copies of n pages in every pool (n, or *moves.count of them), with the
// tables of a compaction in the first launch.
idx_status launch_copies(const idx_page_pool* pools, int32_t num_pools, const int32_t* src,
                         const int32_t* dst, int32_t n, const Tables& t, Moves moves,
                         cudaStream_t s) {
  int32_t first = 0;
  do {
    Pools q{};
    q.num = std::min(num_pools - first, kPoolsPerLaunch);
    for (int i = 0; i < q.num; ++i) {
      q.base[i] = static_cast<uint8_t*>(pools[first + i].base);
      q.stride[i] = pools[first + i].page_stride;
      q.bytes[i] = static_cast<int32_t>(pools[first + i].page_bytes);
      q.chunk0[i + 1] = q.chunk0[i] + (q.bytes[i] + kChunk - 1) / kChunk;
    }
    const int64_t tasks = std::max<int64_t>(1, static_cast<int64_t>(n) * q.chunk0[q.num]);
    const unsigned grid =
        static_cast<unsigned>(std::min<int64_t>(tasks, int64_t{kCopyCtasPerSm} * device_sm_count()));
    const idx_status st = cuda_status(
        launch_pdl(copy_pages_kernel, grid, kCopyThreads, 0, s, q, src, dst, n, t, moves));
    if (st != IDX_OK) return st;
    moves.remap = nullptr;
    first += q.num;
  } while (first < num_pools);
  return IDX_OK;
}

struct CompactWs {
  size_t counts, src, dst, moves, total;
  int32_t blocks;
};

CompactWs compact_ws(int64_t num_pages) {
  CompactWs w{};
  w.blocks = static_cast<int32_t>((num_pages + kScanThreads - 1) / kScanThreads);
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  w.counts = take(4 * static_cast<size_t>(w.blocks));
  w.src = take(4 * static_cast<size_t>(num_pages));
  w.dst = take(4 * static_cast<size_t>(num_pages));
  w.moves = take(4);
  w.total = off;
  return w;
}

}  // namespace
}  // namespace saib

using namespace saib;

extern "C" {

idx_status indexer_copy_pages(const idx_page_pool* pools, int32_t num_pools, int64_t num_pages,
                              const int32_t* src, const int32_t* dst, int32_t n,
                              uint32_t* dev_error, void* stream) {
  const idx_status st = check_pools(pools, num_pools, num_pages);
  if (st != IDX_OK) return st;
  if (n < 0) return IDX_ERR_INVALID_ARG;
  if (n == 0 || num_pools == 0) return IDX_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return IDX_ERR_INVALID_ARG;
  Tables t{};
  t.num_pages = static_cast<int32_t>(num_pages);
  t.err = dev_error;
  return launch_copies(pools, num_pools, src, dst, n, t, Moves{}, static_cast<cudaStream_t>(stream));
}

idx_status indexer_fork_pages(const idx_page_pool* pools, int32_t num_pools, int64_t num_pages,
                              int32_t* block_table, int64_t bt_stride, int32_t bt_width,
                              int32_t num_rows, int32_t* seq_lens, int32_t* ref_counts,
                              const int32_t* parents, const int32_t* children, int32_t n,
                              int32_t* copy_src, int32_t* copy_dst, uint32_t* dev_error,
                              void* stream) {
  idx_status st = check_pools(pools, num_pools, num_pages);
  if (st != IDX_OK) return st;
  const Tables t{block_table, bt_stride,  bt_width, num_rows,
                 seq_lens,    ref_counts, static_cast<int32_t>(num_pages), dev_error};
  if ((st = check_tables(t)) != IDX_OK) return st;
  if (n < 0 || n > num_rows) return IDX_ERR_INVALID_ARG;
  if (n == 0) return IDX_OK;
  if (!parents || !children || !copy_src || !copy_dst || !aligned(parents, 4) ||
      !aligned(children, 4) || !aligned(copy_src, 4) || !aligned(copy_dst, 4))
    return IDX_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = cuda_status(launch_pdl(fork_pages_kernel, 1 + n, kScanThreads, 0, s, t, parents, children, n,
                              copy_src, copy_dst));
  if (st != IDX_OK || num_pools == 0) return st;
  return launch_copies(pools, num_pools, copy_src, copy_dst, n, t, Moves{}, s);
}

idx_status indexer_free_pages(const int32_t* block_table, int64_t bt_stride, int32_t bt_width,
                              int32_t num_rows, int32_t* seq_lens, int32_t* ref_counts,
                              int64_t num_pages, const int32_t* rows, int32_t n,
                              uint32_t* dev_error, void* stream) {
  if (num_pages < 1 || num_pages > INT32_MAX / 2) return IDX_ERR_INVALID_ARG;
  const Tables t{const_cast<int32_t*>(block_table), bt_stride,  bt_width,
                 num_rows,                          seq_lens,   ref_counts,
                 static_cast<int32_t>(num_pages),   dev_error};
  const idx_status st = check_tables(t);
  if (st != IDX_OK) return st;
  if (n < 0 || n > num_rows) return IDX_ERR_INVALID_ARG;
  if (n == 0) return IDX_OK;
  if (!rows || !aligned(rows, 4)) return IDX_ERR_INVALID_ARG;
  return cuda_status(launch_pdl(free_pages_kernel, n, kScanThreads, 0,
                                static_cast<cudaStream_t>(stream), t, rows));
}

idx_status indexer_compact_workspace_bytes(int64_t num_pages, size_t* bytes) {
  if (!bytes || num_pages < 1 || num_pages > INT32_MAX / 2) return IDX_ERR_INVALID_ARG;
  *bytes = compact_ws(num_pages).total;
  return IDX_OK;
}

idx_status indexer_compact_pages(const idx_page_pool* pools, int32_t num_pools, int64_t num_pages,
                                 int32_t* block_table, int64_t bt_stride, int32_t bt_width,
                                 int32_t num_rows, const int32_t* seq_lens, int32_t* ref_counts,
                                 int32_t* remap, int32_t* num_live, void* workspace,
                                 size_t workspace_bytes, uint32_t* dev_error, void* stream) {
  idx_status st = check_pools(pools, num_pools, num_pages);
  if (st != IDX_OK) return st;
  const Tables t{block_table, bt_stride, bt_width, num_rows, const_cast<int32_t*>(seq_lens),
                 ref_counts,  static_cast<int32_t>(num_pages), dev_error};
  if ((st = check_tables(t)) != IDX_OK) return st;
  if (!remap || !num_live || !workspace || !aligned(workspace, 256) || !aligned(remap, 4) ||
      !aligned(num_live, 4))
    return IDX_ERR_INVALID_ARG;
  const CompactWs w = compact_ws(num_pages);
  if (workspace_bytes < w.total) return IDX_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* counts = reinterpret_cast<int32_t*>(ws + w.counts);
  int32_t* src = reinterpret_cast<int32_t*>(ws + w.src);
  int32_t* dst = reinterpret_cast<int32_t*>(ws + w.dst);
  int32_t* moves = reinterpret_cast<int32_t*>(ws + w.moves);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = cuda_status(launch_pdl(count_live_kernel, w.blocks, kScanThreads, 0, s, ref_counts,
                              t.num_pages, counts));
  if (st != IDX_OK) return st;
  st = cuda_status(launch_pdl(plan_moves_kernel, w.blocks, kScanThreads, 0, s, ref_counts,
                              t.num_pages, counts, w.blocks, remap, src, dst, num_live, moves));
  if (st != IDX_OK) return st;
  return launch_copies(pools, num_pools, src, dst, t.num_pages, t, Moves{moves, remap}, s);
}

}  // extern "C"
