// Trees of drafted tokens: what they ask of attention, and the accepted path
// kept in the caches.
#include <algorithm>
#include <memory>
#include <new>

#include "internal.h"

namespace saib {

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---------------------------------------------------------------------------
// masks, positions and paths
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 128;
constexpr int kPlanNodes = 2048;  // nodes of a request whose parents fit in shared memory
constexpr int kChain = 32;        // nodes of a chain that do
constexpr int kPathWidth = 1024;  // widest path that a warp writes together

struct PlanParams {
  const int32_t* parents;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  int32_t num_tokens, window, sinks;
  int32_t* masks;
  int32_t mask_words;
  int32_t* positions;
  int32_t* paths;
  int32_t path_width;
  uint32_t* err;
};

// A thread per node walks up to the root. A parent's index is below its child's, so
// the walk ends, and it meets the mask's words in descending order: each is collected
// in a register and written once. Chains of up to kChain nodes are kept in shared memory,
// from which the warp writes its nodes' paths together (256 trees of 64 to 160 nodes, paths
// of 24: 5.9 us; each thread its own 8.2). Bound by the walk's dependent reads of shared
// memory and the rows written.
__global__ void __launch_bounds__(kPlanThreads) plan_tree_kernel(const PlanParams p) {
  __shared__ int32_t near[kPlanNodes];
  __shared__ int32_t chains[kPlanThreads][kChain + 1], nodes[kPlanThreads];
  pdl_wait();
  pdl_trigger();
  const int32_t b = blockIdx.x, lane = threadIdx.x & 31;
  int32_t q0 = p.query_start_loc[b], q1 = p.query_start_loc[b + 1];
  const int32_t keys = p.seq_lens[b];
  const bool first = threadIdx.x == 0 && blockIdx.y == 0;
  if (first && (q0 < 0 || q1 < q0 || q1 > p.num_tokens || keys < q1 - q0))
    set_error(p.err, IDX_DEV_BAD_LEN);
  q0 = min(max(q0, 0), p.num_tokens);
  q1 = min(max(q1, q0), p.num_tokens);
  const int32_t nq = q1 - q0, ahead = max(keys, 0) - nq;
  if (nq == 0) return;
  if (first && nq > 32 * static_cast<int64_t>(p.mask_words)) set_error(p.err, IDX_DEV_OVERFLOW);
  const int32_t* const parents = p.parents + q0;
  const bool fits = nq <= kPlanNodes;
  if (fits) {
    for (int32_t i = threadIdx.x; i < nq; i += kPlanThreads) near[i] = parents[i];
    __syncthreads();
  }
  const auto parent = [&](int32_t i) -> int32_t {
    const int32_t v = fits ? near[i] : parents[i];
    return v < i ? max(v, -1) : -1;
  };
  // (a warp's nodes together: some of the last may not exist)
  for (int32_t i0 = blockIdx.y * kPlanThreads + threadIdx.x - lane; i0 < nq; i0 += gridDim.y * kPlanThreads) {
    const int32_t i = i0 + lane;
    const int64_t t = static_cast<int64_t>(q0) + i;
    int32_t* const chain = chains[threadIdx.x];
    int32_t n = 0;  // nodes of the chain
    if (i < nq) {
      const int32_t own = fits ? near[i] : parents[i];
      if (own < -1 || own >= i) set_error(p.err, IDX_DEV_BAD_ROW);
      for (int32_t j = i; j >= 0; j = parent(j), ++n)
        if (n < kChain) chain[n] = j;
      const int32_t depth = n - 1;
      p.positions[t] = ahead + depth;
      if (p.paths && n > p.path_width) set_error(p.err, IDX_DEV_OVERFLOW);
      int32_t* const mask = p.masks + t * p.mask_words;
      int32_t word = p.mask_words - 1;
      uint32_t bits = 0;
      const auto name = [&](int32_t j, int32_t up) {
        if (p.window > 0 && up >= p.window && ahead + depth - up >= p.sinks) return;
        const int32_t w = j >> 5;
        if (w >= p.mask_words) return;
        for (; word > w; --word) {
          mask[word] = static_cast<int32_t>(bits);
          bits = 0;
        }
        bits |= 1u << (j & 31);
      };
      if (n <= kChain) {
        for (int32_t up = 0; up < n; ++up) name(chain[up], up);
      } else {
        for (int32_t j = i, up = 0; j >= 0; j = parent(j), ++up) name(j, up);
      }
      for (; word >= 0; --word) {
        mask[word] = static_cast<int32_t>(bits);
        bits = 0;
      }
      if (p.paths && (n > kChain || p.path_width > kPathWidth)) {
        int32_t* const path = p.paths + t * p.path_width;
        int32_t up = 0;
        for (int32_t j = i; j >= 0 && up < p.path_width; j = parent(j), ++up) path[up] = max(ahead + j, -1);
        for (; up < p.path_width; ++up) path[up] = -1;
      }
    }
    if (p.paths && p.path_width <= kPathWidth) {
      nodes[threadIdx.x] = n;
      __syncwarp();
      const uint32_t width = p.path_width, all = min(32, nq - i0) * width;
      const uint32_t inverse = 0xffffffffu / width + 1;  // e / width = e * inverse >> 32 for these e
      int32_t* const path = p.paths + (static_cast<int64_t>(q0) + i0) * width;
      const int warp0 = threadIdx.x - lane;
#pragma unroll 4
      for (uint32_t e = lane; e < all; e += 32) {
        const uint32_t r = width == 1 ? e : __umulhi(e, inverse), c = e - r * width;
        const int32_t of = nodes[warp0 + r];
        const int32_t j = chains[warp0 + r][min(c, static_cast<uint32_t>(kChain))];
        if (of <= kChain) path[e] = static_cast<int32_t>(c) < of ? max(ahead + j, -1) : -1;
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------
// the accepted path
// ---------------------------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kMoves = 64;            // of a round
constexpr int kMoveLoads = 8;         // loads in flight per thread
constexpr int kPoolsPerLaunch = 48;   // pools in one launch's parameters
constexpr int kMostBlocks = 8;        // of a request

struct MovePools {
  uint8_t* base[kPoolsPerLaunch];
  int64_t page_stride[kPoolsPerLaunch], token_stride[kPoolsPerLaunch], piece_stride[kPoolsPerLaunch];
  int32_t columns[kPoolsPerLaunch];      // of a piece
  int32_t column0[kPoolsPerLaunch + 1];  // exclusive prefix of the pools' columns
  uint8_t wide[kPoolsPerLaunch];         // a column has 16 bytes (else 4)
  int32_t num;
};

struct CommitParams {
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t bt_width;
  int32_t* seq_lens;
  const int32_t* query_start_loc;
  const int32_t* accepted;
  int64_t accepted_stride;
  int32_t max_accepted;
  int32_t num_pages;
  int32_t blocks;      // of a request: a cluster
  int32_t last;        // the call's last launch: lengths and references follow
  int32_t* ref_counts;
  uint32_t* err;
};

// Moves a column's bytes for n moves (from[i] and to[i]: page and token; a page of -1: none). A list
// is ascending and entry i is at least i, so a later move never reads what an earlier one has
// written; no other thread touches the column.
template <typename V>
__device__ __forceinline__ void move_column(uint8_t* at, int64_t page_stride, int64_t token_stride,
                                            const int2* from, const int2* to, int32_t n) {
  for (int32_t i0 = 0; i0 < n; i0 += kMoveLoads) {
    V x[kMoveLoads];
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e)
      if (i0 + e < n && from[i0 + e].x >= 0)
        x[e] = *reinterpret_cast<const V*>(at + from[i0 + e].x * page_stride +
                                           from[i0 + e].y * token_stride);
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e)
      if (i0 + e < n && from[i0 + e].x >= 0)
        *reinterpret_cast<V*>(at + to[i0 + e].x * page_stride + to[i0 + e].y * token_stride) = x[e];
  }
}

// A cluster per request: its blocks share the columns (16 or 4 bytes of a token) of all pools; the
// first one writes the length, once all have read it, and drops the references of the pages that the
// row no longer holds. Bound by the latency of a chain of loads (lengths, list, table, data).
__global__ void __launch_bounds__(kMoveThreads)
    commit_tree_kernel(const __grid_constant__ CommitParams p, const __grid_constant__ MovePools pools) {
  __shared__ int2 from[kMoves], to[kMoves];
  __shared__ int32_t end;
  pdl_wait();
  pdl_trigger();
  const int32_t b = blockIdx.x / p.blocks, rank = blockIdx.x % p.blocks;
  const bool first = rank == 0 && threadIdx.x == 0;
  const int32_t keys = p.seq_lens[b];
  const int64_t new_tokens = static_cast<int64_t>(p.query_start_loc[b + 1]) - p.query_start_loc[b];
  if (p.blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const bool ok = new_tokens >= 0 && keys >= new_tokens &&
                  keys <= static_cast<int64_t>(p.bt_width) * kPageTokens;
  const int32_t nq = ok ? static_cast<int32_t>(new_tokens) : 0, ahead = keys - nq;
  const int32_t* const list = p.accepted + b * p.accepted_stride;
  const int32_t* const bt = p.block_table + b * p.bt_stride;
  const int32_t most = min(p.max_accepted, nq);
  int32_t kept = 0;
  for (int32_t i0 = 0; i0 < most; i0 += kMoves) {
    if (threadIdx.x == 0) end = kMoves;
    __syncthreads();
    if (threadIdx.x < kMoves) {
      const int32_t i = i0 + threadIdx.x;
      const int32_t a = i < most ? list[i] : -1;
      const int32_t before = i > 0 && i < most ? list[i - 1] : -1;
      int2 src = make_int2(-1, 0), dst = make_int2(0, 0);
      if (a > before && a < nq) {
        if (a != i) {
          src = make_int2(bt[(ahead + a) / kPageTokens], (ahead + a) % kPageTokens);
          dst = make_int2(bt[(ahead + i) / kPageTokens], (ahead + i) % kPageTokens);
          if (src.x < 0 || src.x >= p.num_pages || dst.x < 0 || dst.x >= p.num_pages) {
            set_error(p.err, IDX_DEV_BAD_BLOCK);
            src.x = -1;
          }
        }
      } else {
        atomicMin(&end, static_cast<int32_t>(threadIdx.x));
      }
      from[threadIdx.x] = src;
      to[threadIdx.x] = dst;
    }
    __syncthreads();
    const int32_t n = end;
    kept = i0 + n;
    for (int32_t col = rank * kMoveThreads + threadIdx.x; col < pools.column0[pools.num];
         col += p.blocks * kMoveThreads) {
      int lo = 0, hi = pools.num - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pools.column0[mid] <= col) lo = mid; else hi = mid - 1;
      }
      const int32_t at = col - pools.column0[lo], piece = at / pools.columns[lo];
      uint8_t* const base = pools.base[lo] + piece * pools.piece_stride[lo] +
                            (at - piece * pools.columns[lo]) * (pools.wide[lo] ? 16 : 4);
      if (pools.wide[lo])
        move_column<uint4>(base, pools.page_stride[lo], pools.token_stride[lo], from, to, n);
      else
        move_column<uint32_t>(base, pools.page_stride[lo], pools.token_stride[lo], from, to, n);
    }
    if (n < kMoves) break;
    __syncthreads();
  }
  // every thread has read the length (a block alone whose lists are empty has met no barrier yet)
  if (p.blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else __syncthreads();
  if (rank != 0 || !p.last) return;
  if (!ok) {
    if (first) set_error(p.err, IDX_DEV_BAD_LEN);
    return;
  }
  if (first && kept < p.max_accepted && list[kept] >= 0) set_error(p.err, IDX_DEV_BAD_ROW);
  const int32_t left = ahead + kept;
  const auto pages = [](int32_t k) { return (k + kPageTokens - 1) / kPageTokens; };
  if (p.ref_counts) {
    for (int32_t c = pages(left) + threadIdx.x; c < pages(keys); c += kMoveThreads) {
      const int32_t page = bt[c];
      if (page < 0 || page >= p.num_pages) {
        set_error(p.err, IDX_DEV_BAD_BLOCK);
      } else if (atomicSub(p.ref_counts + page, 1) <= 0) {
        atomicAdd(p.ref_counts + page, 1);
        set_error(p.err, IDX_DEV_BAD_REF);
      }
    }
  }
  if (first) p.seq_lens[b] = left;
}

// Whether two pools begin at the same place: moved twice, a token would end up where another's is.
bool same_pool_twice(const idx_token_pool* pools, int32_t n) {
  const std::unique_ptr<uintptr_t[]> at(n > 1 ? new (std::nothrow) uintptr_t[n] : nullptr);
  if (!at) return false;
  for (int32_t i = 0; i < n; ++i) at[i] = reinterpret_cast<uintptr_t>(pools[i].base);
  std::sort(at.get(), at.get() + n);
  return std::adjacent_find(at.get(), at.get() + n) != at.get() + n;
}

}  // namespace
}  // namespace saib

using namespace saib;

extern "C" {

idx_status indexer_plan_tree(const int32_t* parents, const int32_t* seq_lens,
                             const int32_t* query_start_loc, int32_t num_reqs, int32_t num_tokens,
                             int32_t window, int32_t sinks, int32_t* masks, int32_t mask_words,
                             int32_t* positions, int32_t* paths, int32_t path_width,
                             uint32_t* dev_error, void* stream) {
  if (num_reqs < 0 || num_tokens < 0 || window < 0 || sinks < 0 || mask_words < 1 ||
      path_width < 0 || (paths && path_width < 1))
    return IDX_ERR_INVALID_ARG;
  if (num_reqs == 0 || num_tokens == 0) return IDX_OK;
  if (!parents || !seq_lens || !query_start_loc || !masks || !positions || !aligned(parents, 4) ||
      !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(masks, 4) ||
      !aligned(positions, 4) || !aligned(paths, 4))
    return IDX_ERR_INVALID_ARG;
  const PlanParams p{parents, seq_lens, query_start_loc, num_tokens, window,     sinks,
                     masks,   mask_words, positions,     paths,      path_width, dev_error};
  cudaLaunchConfig_t cfg = {};
  // (a block's nodes; more of a request's go round)
  const int64_t most = std::min<int64_t>(32 * static_cast<int64_t>(mask_words), num_tokens);
  cfg.gridDim = dim3(num_reqs, static_cast<unsigned>(std::min<int64_t>(
                                   (most + kPlanThreads - 1) / kPlanThreads, 64)));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, plan_tree_kernel, p));
}

idx_status indexer_commit_tree(const idx_token_pool* pools, int32_t num_pools, int64_t num_pages,
                               const int32_t* block_table, int64_t bt_stride, int32_t bt_width,
                               int32_t num_reqs, int32_t* seq_lens, const int32_t* query_start_loc,
                               const int32_t* accepted, int64_t accepted_stride,
                               int32_t max_accepted, int32_t* ref_counts, uint32_t* dev_error,
                               void* stream) {
  if (num_pools < 0 || (num_pools && !pools) || num_pages < 1 || num_pages > INT32_MAX / 2 ||
      num_reqs < 0 || num_reqs > INT32_MAX / kMostBlocks || bt_width < 1 || bt_width > INT32_MAX / kPageTokens || bt_stride < bt_width ||
      max_accepted < 0 || accepted_stride < max_accepted)
    return IDX_ERR_INVALID_ARG;
  for (int32_t i = 0; i < num_pools; ++i) {
    const idx_token_pool& t = pools[i];
    if (!t.base || !aligned(t.base, 4) || t.pieces < 1 || t.piece_bytes < 4 || t.piece_bytes % 4 ||
        t.page_stride < 0 || t.page_stride % 4 || t.token_stride < 0 || t.token_stride % 4 ||
        t.piece_stride < 0 || t.piece_stride % 4 ||
        static_cast<int64_t>(t.pieces) * t.piece_bytes > INT32_MAX)
      return IDX_ERR_INVALID_ARG;
  }
  if (same_pool_twice(pools, num_pools)) return IDX_ERR_INVALID_ARG;
  if (num_reqs == 0) return IDX_OK;
  if (!block_table || !seq_lens || !query_start_loc || (max_accepted && !accepted) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) ||
      !aligned(accepted, 4) || !aligned(ref_counts, 4))
    return IDX_ERR_INVALID_ARG;
  CommitParams p{block_table,  bt_stride,    bt_width, seq_lens, query_start_loc, accepted, accepted_stride,
                 max_accepted, static_cast<int32_t>(num_pages), 1, 0, ref_counts, dev_error};
  int32_t first = 0;
  do {
    MovePools q{};
    q.num = std::min(num_pools - first, kPoolsPerLaunch);
    int64_t columns = 0;
    for (int32_t i = 0; i < q.num; ++i) {
      const idx_token_pool& t = pools[first + i];
      q.base[i] = static_cast<uint8_t*>(t.base);
      q.page_stride[i] = t.page_stride;
      q.token_stride[i] = t.token_stride;
      q.piece_stride[i] = t.piece_stride;
      q.wide[i] = aligned(t.base, 16) && (t.page_stride | t.token_stride | t.piece_bytes |
                                          (t.pieces > 1 ? t.piece_stride : 0)) % 16 == 0;
      q.columns[i] = t.piece_bytes / (q.wide[i] ? 16 : 4);
      columns += static_cast<int64_t>(q.columns[i]) * t.pieces;
      if (columns > INT32_MAX) return IDX_ERR_UNSUPPORTED;
      q.column0[i + 1] = static_cast<int32_t>(columns);
    }
    first += q.num;
    p.last = first >= num_pools;
    p.blocks = 1;
    while (p.blocks < kMostBlocks && int64_t{p.blocks} * kMoveThreads < columns) p.blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_reqs) * p.blocks);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(p.blocks), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const idx_status st = cuda_status(cudaLaunchKernelEx(&cfg, commit_tree_kernel, p, q));
    if (st != IDX_OK) return st;
  } while (first < num_pools);
  return IDX_OK;
}

}  // extern "C"
