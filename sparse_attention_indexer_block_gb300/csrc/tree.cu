// Trees of drafted tokens: what they ask of attention, and the accepted path
// kept in the caches.
#include <algorithm>

#include "internal.h"

namespace saib {

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---------------------------------------------------------------------------
// masks, positions and paths
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 128;
constexpr int kPlanNodes = 2048;  // nodes of a request whose parents fit in shared memory

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

// A thread per node walks up to the root. A parent's index is below its
// child's, so the walk ends, and it meets the mask's words in descending order:
// each is collected in a register and written once. Bound by the walk's
// dependent reads (shared memory) and, for many nodes, the rows written.
__global__ void __launch_bounds__(kPlanThreads) plan_tree_kernel(const PlanParams p) {
  __shared__ int32_t near[kPlanNodes];
  pdl_wait();
  pdl_trigger();
  const int32_t b = blockIdx.x;
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
  for (int32_t i = blockIdx.y * kPlanThreads + threadIdx.x; i < nq; i += gridDim.y * kPlanThreads) {
    const int64_t t = static_cast<int64_t>(q0) + i;
    const int32_t own = parents[i];
    if (own < -1 || own >= i) set_error(p.err, IDX_DEV_BAD_ROW);
    int32_t depth = 0;
    {
      int32_t* const path = p.paths ? p.paths + t * p.path_width : nullptr;
      int32_t n = 0;
      for (int32_t j = i; j >= 0; j = parent(j), ++n)
        if (path && n < p.path_width) path[n] = max(ahead + j, -1);
      depth = n - 1;
      if (path) {
        if (n > p.path_width) set_error(p.err, IDX_DEV_OVERFLOW);
        for (; n < p.path_width; ++n) path[n] = -1;
      }
    }
    p.positions[t] = ahead + depth;
    int32_t* const mask = p.masks + t * p.mask_words;
    int32_t word = p.mask_words - 1;
    uint32_t bits = 0;
    for (int32_t j = i, up = 0; j >= 0; j = parent(j), ++up) {
      if (p.window > 0 && up >= p.window && ahead + depth - up >= p.sinks) continue;
      const int32_t w = j >> 5;
      if (w >= p.mask_words) continue;
      for (; word > w; --word) {
        mask[word] = static_cast<int32_t>(bits);
        bits = 0;
      }
      bits |= 1u << (j & 31);
    }
    for (; word >= 0; --word) {
      mask[word] = static_cast<int32_t>(bits);
      bits = 0;
    }
  }
}

// ---------------------------------------------------------------------------
// the accepted path
// ---------------------------------------------------------------------------

constexpr int kMoveThreads = 128;
constexpr int kMoveLoads = 4;         // loads in flight per thread
constexpr int kPoolsPerLaunch = 48;   // pools in one launch's parameters

struct MovePools {
  uint8_t* base[kPoolsPerLaunch];
  int64_t page_stride[kPoolsPerLaunch], token_stride[kPoolsPerLaunch], piece_stride[kPoolsPerLaunch];
  int32_t pieces[kPoolsPerLaunch], piece_bytes[kPoolsPerLaunch];
  uint8_t wide[kPoolsPerLaunch];  // 16 bytes at once (else 4)
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
  int32_t* ref_counts;
  uint32_t* err;
};

struct TreeShape {
  int32_t keys, nq;  // keys, the tree's nodes among them
  bool ok;
};

__device__ __forceinline__ TreeShape tree_shape(const CommitParams& p, int32_t b) {
  const int32_t keys = p.seq_lens[b];
  const int64_t nq = static_cast<int64_t>(p.query_start_loc[b + 1]) - p.query_start_loc[b];
  const bool ok = nq >= 0 && keys >= nq && keys <= static_cast<int64_t>(p.bt_width) * kPageTokens;
  return TreeShape{keys, static_cast<int32_t>(ok ? nq : 0), ok};
}

// Whether entry i of a list continues it.
__device__ __forceinline__ bool continues(const int32_t* list, int32_t i, int32_t nq) {
  const int32_t a = list[i];
  return a >= 0 && a < nq && (i == 0 || a > list[i - 1]);
}

// Moves the bytes of a thread's columns for n moves from place from[i] to to[i] (byte offsets in
// the pool, -1: none). A list is ascending and entry i is at least i, so a later move never reads
// what an earlier one has written, and no thread reads another's columns.
template <typename V>
__device__ __forceinline__ void move_columns(uint8_t* base, int64_t piece_stride, int32_t pieces,
                                             int32_t piece_bytes, const int64_t* from,
                                             const int64_t* to, int32_t n) {
  const int32_t per = piece_bytes / static_cast<int32_t>(sizeof(V));
  for (int32_t col = threadIdx.x; col < per * pieces; col += kMoveThreads) {
    const int32_t piece = col / per;
    uint8_t* const at = base + piece * piece_stride + (col - piece * per) * sizeof(V);
    for (int32_t i0 = 0; i0 < n; i0 += kMoveLoads) {
      V x[kMoveLoads];
#pragma unroll
      for (int e = 0; e < kMoveLoads; ++e)
        if (i0 + e < n && from[i0 + e] >= 0) x[e] = *reinterpret_cast<const V*>(at + from[i0 + e]);
#pragma unroll
      for (int e = 0; e < kMoveLoads; ++e)
        if (i0 + e < n && from[i0 + e] >= 0) *reinterpret_cast<V*>(at + to[i0 + e]) = x[e];
    }
  }
}

// Block (request, pool): the accepted tokens to the tree's first places.
__global__ void __launch_bounds__(kMoveThreads)
    move_tokens_kernel(const __grid_constant__ CommitParams p, const __grid_constant__ MovePools pools) {
  __shared__ int64_t from[kMoveThreads], to[kMoveThreads];
  __shared__ int32_t end;
  pdl_wait();
  pdl_trigger();
  const int32_t b = blockIdx.x, pool = blockIdx.y;
  const TreeShape r = tree_shape(p, b);
  if (!r.ok) return;
  const int32_t ahead = r.keys - r.nq;
  const int32_t* const list = p.accepted + b * p.accepted_stride;
  const int32_t* const bt = p.block_table + b * p.bt_stride;
  const int32_t most = min(p.max_accepted, r.nq);
  for (int32_t i0 = 0; i0 < most; i0 += kMoveThreads) {
    if (threadIdx.x == 0) end = kMoveThreads;
    __syncthreads();
    const int32_t i = i0 + threadIdx.x;
    const bool in = i < most && continues(list, i, r.nq);
    if (!in) atomicMin(&end, static_cast<int32_t>(threadIdx.x));
    int64_t a = -1, c = -1;
    if (in && list[i] != i) {
      const int32_t s = ahead + list[i], d = ahead + i;
      const int32_t sp = bt[s / kPageTokens], dp = bt[d / kPageTokens];
      if (sp >= 0 && sp < p.num_pages && dp >= 0 && dp < p.num_pages) {
        a = sp * pools.page_stride[pool] + (s % kPageTokens) * pools.token_stride[pool];
        c = dp * pools.page_stride[pool] + (d % kPageTokens) * pools.token_stride[pool];
      } else {
        set_error(p.err, IDX_DEV_BAD_BLOCK);
      }
    }
    from[threadIdx.x] = a;
    to[threadIdx.x] = c;
    __syncthreads();
    const int32_t n = end;
    if (pools.wide[pool])
      move_columns<uint4>(pools.base[pool], pools.piece_stride[pool], pools.pieces[pool],
                          pools.piece_bytes[pool], from, to, n);
    else
      move_columns<uint32_t>(pools.base[pool], pools.piece_stride[pool], pools.pieces[pool],
                             pools.piece_bytes[pool], from, to, n);
    if (n < kMoveThreads) return;
    __syncthreads();
  }
}

// A warp per request: its new length, and the references of the pages that it no longer holds.
__global__ void __launch_bounds__(kMoveThreads) commit_lens_kernel(const CommitParams p, int32_t num_reqs) {
  pdl_wait();
  pdl_trigger();
  const int32_t b = (blockIdx.x * kMoveThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (b >= num_reqs) return;
  const TreeShape r = tree_shape(p, b);
  if (!r.ok) {
    if (lane == 0) set_error(p.err, IDX_DEV_BAD_LEN);
    return;
  }
  const int32_t* const list = p.accepted + b * p.accepted_stride;
  int32_t n = 0;
  for (int32_t i0 = 0; i0 < p.max_accepted; i0 += 32) {
    const int32_t i = i0 + lane;
    const bool in = i < p.max_accepted && continues(list, i, r.nq);
    const uint32_t all = __ballot_sync(0xffffffffu, in);
    if (all != 0xffffffffu) {
      n = i0 + __ffs(~all) - 1;
      break;
    }
    n = i0 + 32;
  }
  if (lane == 0 && n < p.max_accepted && list[n] >= 0) set_error(p.err, IDX_DEV_BAD_ROW);
  const int32_t left = r.keys - r.nq + n;
  const auto pages = [](int32_t k) { return (k + kPageTokens - 1) / kPageTokens; };
  if (p.ref_counts) {
    for (int32_t c = pages(left) + lane; c < pages(r.keys); c += 32) {
      const int32_t page = p.block_table[b * p.bt_stride + c];
      if (page < 0 || page >= p.num_pages) {
        set_error(p.err, IDX_DEV_BAD_BLOCK);
      } else if (atomicSub(p.ref_counts + page, 1) <= 0) {
        atomicAdd(p.ref_counts + page, 1);
        set_error(p.err, IDX_DEV_BAD_REF);
      }
    }
  }
  __syncwarp();
  if (lane == 0) p.seq_lens[b] = left;
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
      num_reqs < 0 || bt_width < 1 || bt_width > INT32_MAX / kPageTokens || bt_stride < bt_width ||
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
  if (num_reqs == 0) return IDX_OK;
  if (!block_table || !seq_lens || !query_start_loc || (max_accepted && !accepted) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) ||
      !aligned(accepted, 4) || !aligned(ref_counts, 4))
    return IDX_ERR_INVALID_ARG;
  const CommitParams p{block_table, bt_stride,       bt_width,     seq_lens,
                       query_start_loc, accepted,    accepted_stride, max_accepted,
                       static_cast<int32_t>(num_pages), ref_counts, dev_error};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t first = 0; max_accepted && first < num_pools; first += kPoolsPerLaunch) {
    MovePools q{};
    const int32_t n = std::min(num_pools - first, kPoolsPerLaunch);
    for (int32_t i = 0; i < n; ++i) {
      const idx_token_pool& t = pools[first + i];
      q.base[i] = static_cast<uint8_t*>(t.base);
      q.page_stride[i] = t.page_stride;
      q.token_stride[i] = t.token_stride;
      q.piece_stride[i] = t.piece_stride;
      q.pieces[i] = t.pieces;
      q.piece_bytes[i] = t.piece_bytes;
      q.wide[i] = aligned(t.base, 16) &&
                  (t.page_stride | t.token_stride | (t.pieces > 1 ? t.piece_stride : 0) | t.piece_bytes) % 16 == 0;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_reqs, n);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const idx_status st = cuda_status(cudaLaunchKernelEx(&cfg, move_tokens_kernel, p, q));
    if (st != IDX_OK) return st;
  }
  const unsigned grid = static_cast<unsigned>((num_reqs + kMoveThreads / 32 - 1) / (kMoveThreads / 32));
  return cuda_status(launch_pdl(commit_lens_kernel, grid, kMoveThreads, 0, s, p, num_reqs));
}

}  // extern "C"
