// Attention over a paged key/value cache: the split of the work over the CTAs,
// the row-block kernel (mma.sync, one query block of 16 or 32 rows per unit)
// and the join of units that several CTAs share. The same row-block kernel
// attends to a list of selected tokens.
#include "attend.cuh"

namespace saib {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kWarps = 4;        // of a row-block CTA
constexpr int kStages = 3;       // sub-tiles in flight per warp

// ---------------------------------------------------------------------------
// small helpers
// ---------------------------------------------------------------------------

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Request of an entry: the last one whose first entry is not past it.
__device__ __forceinline__ int entry_request(const int32_t* req_entry, int n, int32_t e) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (req_entry[mid] <= e) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Where CTA c of `grid` begins. A unit costs its tiles and p.unit_overhead; the
// units, in the order request, kv head, entry, are cut into `grid` ranges of
// equal cost. A cut inside a unit's overhead leaves the unit whole to the CTA
// that begins there.
__device__ int4 cut_at(const AttendParams& p, int c) {
  const int64_t all = p.entry_cost[p.req_entry[p.num_reqs]] * p.num_kv_heads;
  const int64_t pos = cut_position(all, cutters(p, all, 0), c);
  if (pos >= all) return make_int4(0, 0, 0, p.num_reqs);
  int lo = 0, hi = p.num_reqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.entry_cost[p.req_entry[mid]] * p.num_kv_heads <= pos) lo = mid; else hi = mid - 1;
  }
  const int32_t e0 = p.req_entry[lo], e1 = p.req_entry[lo + 1];
  const int64_t base = p.entry_cost[e0], cost = p.entry_cost[e1] - base;
  const int64_t rest = pos - base * p.num_kv_heads;
  const int32_t head = static_cast<int32_t>(quotient(rest, cost));
  const int64_t at = base + rest - head * cost;
  int32_t a = e0, b = e1 - 1;
  while (a < b) {
    const int32_t mid = (a + b + 1) >> 1;
    if (p.entry_cost[mid] <= at) a = mid; else b = mid - 1;
  }
  const int32_t off = static_cast<int32_t>(at - p.entry_cost[a]) - p.unit_overhead;
  return make_int4(a - e0, head, off > 0 ? off : 0, lo);
}

// One CTA: entries of the requests, their costs and the CTAs' cuts. Bound by
// the latency of a few dependent loads and scans.
__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const AttendParams p) {
  __shared__ int64_t sums[32];
  pdl_wait();
  pdl_trigger();
  int64_t carry = 0, total;
  for (int b0 = 0; b0 < p.num_reqs; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    const int64_t n = b < p.num_reqs ? request_entries(p, request_shape(p, b, true)) : 0;
    const int64_t incl = carry + block_scan<kPlanThreads>(n, sums, &total);
    // offsets that are not ascending could ask for more entries than there is room for
    if (b < p.num_reqs) {
      if (incl > p.max_entries) set_error(p.dev_error, IDX_DEV_BAD_LEN);
      p.req_entry[b] = static_cast<int32_t>(min(incl - n, static_cast<int64_t>(p.max_entries)));
    }
    carry += total;
  }
  const int32_t entries = static_cast<int32_t>(min(carry, static_cast<int64_t>(p.max_entries)));
  if (threadIdx.x == 0) {
    p.req_entry[p.num_reqs] = entries;
    p.entry_cost[0] = 0;
  }
  __syncthreads();
  carry = 0;
  for (int e0 = 0; e0 < entries; e0 += kPlanThreads) {
    const int e = e0 + threadIdx.x;
    int64_t cost = 0;
    if (e < entries) {
      const int b = entry_request(p.req_entry, p.num_reqs, e);
      cost = unit_tiles(p, request_shape(p, b, false), e - p.req_entry[b]).count + p.unit_overhead;
    }
    const int64_t incl = carry + block_scan<kPlanThreads>(cost, sums, &total);
    if (e < entries) p.entry_cost[e + 1] = incl;
    carry += total;
  }
  __syncthreads();
  for (int c = threadIdx.x; c <= p.grid; c += kPlanThreads) p.bound[c] = cut_at(p, c);
}

// ---------------------------------------------------------------------------
// row-block kernel
// ---------------------------------------------------------------------------

// Cuts of the selected form, where every unit has the same tiles: unit =
// (token * head blocks + block) * kv heads + kv head.
__device__ __forceinline__ int32_t selected_tiles(const AttendParams& p) {
  return (p.topk + (1 << p.tile_log2) - 1) >> p.tile_log2;
}
__device__ __forceinline__ int2 selected_cut(const AttendParams& p, int64_t units, int c) {
  const int64_t cost = selected_tiles(p) + p.unit_overhead;
  const int64_t all = units * cost, pos = cut_position(all, cutters(p, all, units), c);
  const int64_t unit = quotient(pos, cost);
  const int32_t off = static_cast<int32_t>(pos - unit * cost) - p.unit_overhead;
  return make_int2(static_cast<int32_t>(unit), off > 0 ? off : 0);
}
__device__ __forceinline__ int64_t selected_units(const AttendParams& p) {
  return static_cast<int64_t>(p.num_tokens) * ((p.group + p.rows - 1) / p.rows) * p.num_kv_heads;
}

// Request of a token row, or -1 when it lies in none.
__device__ __forceinline__ int token_request(const AttendParams& p, int32_t t) {
  // (equal numbers of tokens per request: two loads side by side instead of a chain)
  const int guess = static_cast<int>(static_cast<int64_t>(t) * p.num_reqs / p.num_tokens);
  if (p.query_start_loc[guess] <= t && t < p.query_start_loc[guess + 1]) return guess;
  int lo = 0, hi = p.num_reqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.query_start_loc[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return t >= p.query_start_loc[lo] && t < p.query_start_loc[lo + 1] ? lo : -1;
}

template <int D, int MT>
struct RowsCfg {
  static constexpr int kRows = 16 * MT;
  static constexpr int kSub = rows_tile_keys(D) / kWarps;  // keys of a warp's sub-tile
  static constexpr int kSubBytes = kSub * D * 2;           // of K or V: 4 KB
  static constexpr int kStageBytes = 2 * kSubBytes;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kPad = 4;  // floats between the joined rows, against bank conflicts
  static constexpr int kJoin = kWarps * kRows * (D + kPad) * 4;
  static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin) + kQ;
};

// Byte offset of 16-byte chunk c of row r in a tile of rows of D 16-bit values:
// chunks are XORed with the row, so that eight rows' equal chunks lie in
// different banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return r * (D * 2) + ((c ^ (r & 7)) << 4);
}

// Whether the token at pos sees key k.
__device__ __forceinline__ bool sees(const AttendParams& p, int32_t pos, int32_t k) {
  return k <= pos && (k < p.sinks || pos - k < p.window);
}

// One sub-tile of kSub keys (K at shared address kt, V kSubBytes on) against 16
// * MT query rows by one warp: scores, running maxima m and sums l, and the
// accumulators o. k_at, v_at: the lane's fragment addresses within a 16-key
// block for step & 3; q_of(f, mt, kk): query fragments; valid: bit per key (a
// list's); all: every row sees every key; s0: the first key's position; rpos: the
// positions of the lane's rows.
template <typename T, int D, int MT, bool kSel, typename QOf>
__device__ __forceinline__ void score_subtile(const AttendParams& p, const uint8_t* smem, uint32_t kt,
                                              const uint32_t (&k_at)[4], const uint32_t (&v_at)[4],
                                              const QOf& q_of, uint32_t valid, bool all, int32_t s0,
                                              const int32_t (&rpos)[MT][2],
                                              float (&o)[MT][D / 8][4], float (&m)[MT][2],
                                              float (&l)[MT][2]) {
  using C = RowsCfg<D, MT>;
  constexpr int kSteps = D / 16, kSub = C::kSub, kTiles8 = kSub / 8;  // 8-key column blocks
  const int lane = threadIdx.x & 31;
  // (two sums per block of scores where there are few, to shorten the chain of products)
  constexpr int kSplit = kTiles8 == 2 ? 2 : 1;
  float s[kSplit][MT][kTiles8][4];
#pragma unroll
  for (int f = 0; f < kSplit; ++f)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int n = 0; n < kTiles8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[f][mt][n][e] = 0.f;
#pragma unroll
  for (int kk = 0; kk < kSteps; ++kk) {
    uint32_t qa[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      q_of(qa[mt], mt, kk);
    }
#pragma unroll
    for (int b = 0; b < kSub / 16; ++b) {
      uint32_t f[4];
      ldsm4(f, kt + k_at[kk & 3] + (kk >> 2) * 128 + b * 16 * (D * 2));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma16816<T>(s[kk % kSplit][mt][2 * b], qa[mt], f[0], f[1]);
        mma16816<T>(s[kk % kSplit][mt][2 * b + 1], qa[mt], f[2], f[3]);
      }
    }
  }
  uint32_t pa[MT][kSub / 16][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float alpha[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // the row's scores of keys 8 n + 2 (lane % 4) + e
      float x[kTiles8][2];
#pragma unroll
      for (int n = 0; n < kTiles8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = s[0][mt][n][2 * h + e];
          if (kSplit == 2) y += s[kSplit - 1][mt][n][2 * h + e];
          x[n][e] = y * p.scale_log2;
        }
      if (!all) {
#pragma unroll
        for (int n = 0; n < kTiles8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = n * 8 + 2 * (lane & 3) + e;
            if (!(kSel ? (valid >> key) & 1 : sees(p, rpos[mt][h], s0 + key)))
              x[n][e] = -INFINITY;
          }
      }
      float mx = fmaxf(x[0][0], x[0][1]);
#pragma unroll
      for (int n = 1; n < kTiles8; ++n) mx = max3(mx, x[n][0], x[n][1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      const float far = __shfl_xor_sync(0xffffffffu, mx, 2);
      mx = kTopWeight<T> == 0.f ? max3(mx, far, m[mt][h])
                                : fmaxf(fmaxf(mx, far) - kTopWeight<T>, m[mt][h]);
      const float base = mx == -INFINITY ? 0.f : mx;
      alpha[h] = exp2_approx(m[mt][h] - base);
      m[mt][h] = mx;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < kTiles8; ++n) {
        const float a = exp2_approx(x[n][0] - base), b = exp2_approx(x[n][1] - base);
        sum += a + b;
        // the weights are rounded to T for the second product (half a step of T each);
        // their sum is of the unrounded ones
        pa[mt][n >> 1][2 * (n & 1) + h] = pack2<T>(a, b);
      }
      l[mt][h] = l[mt][h] * alpha[h] + sum;
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[mt][n][0] *= alpha[0];
        o[mt][n][1] *= alpha[0];
        o[mt][n][2] *= alpha[1];
        o[mt][n][3] *= alpha[1];
      }
    }
  }
  const auto v_frag = [&](uint32_t(&f)[4], int b, int cc) {
    ldsm4_t(f, kt + v_at[cc & 3] + (cc >> 2) * 128 + b * 16 * (D * 2));
  };
  // A key that some rows see and others do not: a weight of 0 times an infinity or NaN
  // would reach the rows that do not, so such values are left out of the product and
  // added to the rows that see them. (A list's keys are seen by all rows or none, and
  // read as zeros where they are seen by none.)
  bool odd = false;
  if (!kSel && !all) {
#pragma unroll 1
    for (int b = 0; b < kSub / 16; ++b)
#pragma unroll
      for (int cc = 0; cc < kSteps; ++cc) {
        uint32_t f[4];
        v_frag(f, b, cc);
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= nonfinite_bits<T>(f[e]) != 0;
      }
    odd = __any_sync(0xffffffffu, odd);
  }
#pragma unroll
  for (int b = 0; b < kSub / 16; ++b)
#pragma unroll
    for (int cc = 0; cc < kSteps; ++cc) {
      uint32_t f[4];
      v_frag(f, b, cc);
      if (odd) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = clear_nonfinite<T>(f[e]);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma16816<T>(o[mt][2 * cc], pa[mt][b], f[0], f[1]);
        mma16816<T>(o[mt][2 * cc + 1], pa[mt][b], f[2], f[3]);
      }
    }
  if (odd) {
    const T* v = reinterpret_cast<const T*>(smem + (kt + C::kSubBytes - smem_u32(smem)));
#pragma unroll 1
    for (int key = 0; key < kSub; ++key)
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x =
              static_cast<float>(v[chunk_at<D>(key, n) / 2 + 2 * (lane & 3) + e]);
          if (!isfinite(x)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (sees(p, rpos[mt][h], s0 + key)) o[mt][n][2 * h + e] += x;
          }
        }
  }
}

__device__ __forceinline__ int cluster_rank() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address, in the cluster's window, of a shared-memory address of this block in block `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ float cluster_load(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Per unit of 16 * MT query rows of one kv head: the four warps take a quarter
// of every tile's keys each (16 at D = 128, 32 at D = 64), with a ring of kStages sub-tiles of K and V per
// warp that its own lanes fill with 16-byte asynchronous copies (so no warp
// waits for another inside a piece), products by mma.sync m16n8k16, running
// maximum and sum per row; the warps' results are joined through shared memory
// at the end of the piece. Bound by HBM (or L2) bytes of K and V when few rows
// share a key: 4 * D bytes of a key feed 4 * D * 16 * MT multiply-adds.
//
// kCluster, for calls of few short units: nothing is planned, every unit (the
// units of every request and kv head) belongs to a cluster whose blocks take equal
// ranges of its tiles and join their results in each other's shared memory, so
// that one launch does all.
template <typename T, int D, int MT, bool kSel, bool kCluster>
__global__ void __launch_bounds__(kWarps * 32, 2) attend_rows_kernel(const AttendParams p) {
  using C = RowsCfg<D, MT>;
  constexpr int kChunks = D / 8;         // 16-byte chunks of a row
  constexpr int kSteps = D / 16;
  constexpr int kSub = C::kSub, kTile = kWarps * kSub;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];
  __shared__ uint32_t s_valid[kWarps][kStages];
  __shared__ float2 s_part[kCluster ? C::kRows : 1];  // maximum and sum of the block's rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = blockIdx.x;
  const uint32_t ring = smem_u32(smem) + warp * (kStages * C::kStageBytes);
  uint8_t* q_smem = smem + (C::kSmem - C::kQ);
  const uint32_t q_addr = smem_u32(q_smem);

  pdl_wait();
  pdl_trigger();

  // this CTA's range of the units
  int64_t unit = 0, unit_end = 0;
  int32_t first_tile = 0, last_tile = 0, req_token = -1, req = -1;
  const int rank = kCluster ? cluster_rank() : 0;
  const int64_t mine = kCluster ? cta / p.cluster : 0;  // this cluster's unit, or request and kv head
  ReqShape shape{};
  if constexpr (kCluster) {
    if (kSel) {
      unit = mine;
      unit_end = mine + 1;
    } else {
      req = static_cast<int32_t>(mine / p.num_kv_heads);
      shape = request_shape(p, req, cta == req * p.num_kv_heads * p.cluster);
      unit_end = request_entries(p, shape);
    }
  } else if constexpr (kSel) {
    const int64_t units = selected_units(p);
    const int2 a = selected_cut(p, units, cta), b = selected_cut(p, units, cta + 1);
    unit = a.x;
    unit_end = b.x;
    first_tile = a.y;
    last_tile = b.y;
  }
  PieceWalk<false> walk;
  if constexpr (!kSel && !kCluster) {
    if (p.self_plan) {
      __shared__ int64_t sums[32];
      __shared__ int4 cuts[2];
      __shared__ ReqShape first;
      self_plan<kWarps * 32>(p, cta, reinterpret_cast<int64_t*>(smem), sums, cuts, &first);
      walk = PieceWalk<false>(p, cuts[0], cuts[1], first);
    } else {
      walk = PieceWalk<false>(p, p.bound[cta], p.bound[cta + 1]);
    }
  }

  for (;;) {
    Piece u;
    if constexpr (kSel) {
      const bool last = unit >= unit_end;
      if (unit > unit_end || (last && last_tile <= first_tile)) break;
      const int blocks = (p.group + p.rows - 1) / p.rows;
      const int64_t tb = unit / p.num_kv_heads;
      const int32_t token = static_cast<int32_t>(tb / blocks);
      u.head = static_cast<int32_t>(unit % p.num_kv_heads);
      u.row0 = static_cast<int32_t>(tb % blocks) * p.rows;
      u.rows = min(p.rows, p.group - u.row0);
      u.q0 = token;
      u.ahead = 0;
      if (token != req_token) {
        req = token_request(p, token);
        req_token = token;
      }
      u.req = req;
      u.tiles = UnitTiles{0, 0, selected_tiles(p), 0, 0};
      u.t0 = first_tile;
      u.t1 = last ? last_tile : u.tiles.count;
      ++unit;
      first_tile = 0;
    } else if constexpr (kCluster) {
      if (unit >= unit_end) break;
      const int32_t entry = static_cast<int32_t>(unit++);
      u.req = req;
      u.head = static_cast<int32_t>(mine % p.num_kv_heads);
      u.row0 = entry * p.rows;
      u.rows = min(p.rows, shape.nq * p.group - u.row0);
      u.q0 = shape.q0;
      u.ahead = shape.keys - shape.nq;
      u.tiles = unit_tiles(p, shape, entry);
    } else {
      if (!walk.next(p, &u)) break;
    }
    if constexpr (kCluster) {
      u.t0 = u.tiles.count * rank / p.cluster;
      u.t1 = u.tiles.count * (rank + 1) / p.cluster;
    }
    const bool whole = u.whole();

    if (!kSel || u.req >= 0) {
      const int32_t p_lo = u.tiles.p_lo, p_hi = u.tiles.p_hi;
      int32_t rpos[MT][2];  // positions of this thread's rows
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = mt * 16 + h * 8 + (lane >> 2);
          int64_t token;
          int head;
          row_place(p, u, r, &token, &head, &rpos[mt][h]);
          if (r >= u.rows) rpos[mt][h] = INT32_MIN;
        }

      float o[MT][D / 8][4];
      float m[MT][2], l[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
        m[mt][0] = m[mt][1] = -INFINITY;
        l[mt][0] = l[mt][1] = 0.f;
      }

      // ---- copies: a pass of the warp copies 32 / kChunks rows of K and of V. Where sub-tile
      // j's keys lie is read one (list entries: two) sub-tiles before its copies are issued.
      constexpr int kPerPass = 32 / kChunks;
      const int c = lane % kChunks, h0 = lane / kChunks;
      // chunk_at of the lane's row and chunk in pass 0; pass i XORs and adds constants
      const uint32_t lane_at = chunk_at<D>(h0, c);
      const T* const k_lane = static_cast<const T*>(p.k) + u.head * p.k_stride_head + c * 8;
      const T* const v_lane = static_cast<const T*>(p.v) + u.head * p.v_stride_head + c * 8;
      const int32_t* const bt = p.block_table + static_cast<int64_t>(u.req) * p.bt_stride;
      const int32_t* const list =
          kSel ? p.indices + static_cast<int64_t>(u.q0) * p.indices_stride : nullptr;
      const int32_t w_lo = max(p_lo, 0) - p.window, w_hi = max(p_hi, 0) - p.window;
      const auto first_key = [&](int j) -> int32_t { return u.tiles.tile(j) * kTile + warp * kSub; };
      const auto load_index = [&](int j) -> int32_t {
        const int at = j * kTile + warp * kSub + (lane & (kSub - 1));
        return j < u.t1 && at < p.topk ? list[at] : -1;
      };
      const auto load_page = [&](int j, int32_t idx) -> int32_t {
        if constexpr (kSel) {
          if (idx < 0) return -1;
          return idx < p.bt_width * kPageTokens ? bt[idx / kPageTokens] : -1;
        } else {
          if (j >= u.t1) return 0;
          const int32_t s0 = first_key(j);
          return s0 <= p_hi ? bt[s0 / kPageTokens] : 0;
        }
      };
      const auto issue = [&](int j, int stage, int32_t idx, int32_t page) {
        if (j < u.t1) {
          const uint32_t dst = ring + stage * C::kStageBytes;
          const bool ok = (!kSel || idx >= 0) && page >= 0 && page < p.num_pages;
          const auto at = [&](int i) -> uint32_t {
            return dst + i * kPerPass * (D * 2) + (lane_at ^ (((i * kPerPass) & 7) << 4));
          };
          if constexpr (kSel) {
            if (idx >= 0 && !ok) set_error(p.dev_error, IDX_DEV_BAD_BLOCK);
            uint32_t valid = __ballot_sync(0xffffffffu, ok);
            if (kSub < 32) valid &= (1u << (kSub & 31)) - 1;
            if (lane == 0) s_valid[warp][stage] = valid;
            const int64_t pg = ok ? page : 0;
            const int32_t tok = ok ? idx & (kPageTokens - 1) : 0;
            const int64_t k_at = pg * p.k_stride_page + tok * p.k_stride_token;
            const int64_t v_at = p.same_strides ? k_at : pg * p.v_stride_page + tok * p.v_stride_token;
#pragma unroll
            for (int i = 0; i < kSub / kPerPass; ++i) {
              const int key = i * kPerPass + h0;
              const int64_t ka = __shfl_sync(0xffffffffu, k_at, key);
              const int64_t va = p.same_strides ? ka : __shfl_sync(0xffffffffu, v_at, key);
              const bool v = (valid >> key) & 1;
              cp_async16(at(i), k_lane + ka, v);
              cp_async16(at(i) + C::kSubBytes, v_lane + va, v);
            }
          } else {
            const int32_t s0 = first_key(j);
            // (what the table says of a page that no row sees may be out of date)
            if (!ok && s0 <= p_hi && (s0 + kSub - 1 > w_lo || s0 < p.sinks))
              set_error(p.dev_error, IDX_DEV_BAD_BLOCK);
            const int64_t pg = ok ? page : 0;
            const int32_t tok = (s0 & (kPageTokens - 1)) + h0;
            const T* kp = k_lane + (pg * p.k_stride_page + tok * p.k_stride_token);
            const T* vp = v_lane + (pg * p.v_stride_page + tok * p.v_stride_token);
            const int64_t k_step = kPerPass * p.k_stride_token, v_step = kPerPass * p.v_stride_token;
            // (every key of most sub-tiles is one that some row sees)
            if (ok && s0 + kSub - 1 <= p_hi && (s0 > w_lo || s0 + kSub <= p.sinks)) {
#pragma unroll
              for (int i = 0; i < kSub / kPerPass; ++i) {
                cp_async16(at(i), kp, true);
                cp_async16(at(i) + C::kSubBytes, vp, true);
                kp += k_step;
                vp += v_step;
              }
            } else {
#pragma unroll
              for (int i = 0; i < kSub / kPerPass; ++i) {
                const int32_t s = s0 + i * kPerPass + h0;
                const bool v = ok && s <= p_hi && (s > w_lo || s < p.sinks);
                cp_async16(at(i), kp, v);
                cp_async16(at(i) + C::kSubBytes, vp, v);
                kp += k_step;
                vp += v_step;
              }
            }
          }
        }
        cp_commit();
      };
      int32_t idx1 = 0, idx2 = 0, page1;  // of the next sub-tile to issue (and the list entry after)
      if constexpr (kSel) {
        idx1 = load_index(u.t0);
        idx2 = load_index(u.t0 + 1);
      }
      page1 = load_page(u.t0, idx1);
      int next = u.t0, stage_in = 0;
      const auto issue_next = [&] {
        const int32_t idx = idx1, page = page1;
        if constexpr (kSel) {
          idx1 = idx2;
          idx2 = load_index(next + 2);
        }
        page1 = load_page(next + 1, idx1);
        issue(next, stage_in, idx, page);
        ++next;
        stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
      };
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) issue_next();

      // ---- queries (the first keys are on their way): shared memory, then fragments
      for (int i = threadIdx.x; i < C::kRows * kChunks; i += kWarps * 32) {
        const int r = i / kChunks, c = i % kChunks;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < u.rows) {
          int64_t token;
          int head, pos;
          row_place(p, u, r, &token, &head, &pos);
          v = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                              token * p.q_stride_token + head * p.q_stride_head +
                                              c * 8);
        }
        *reinterpret_cast<uint4*>(q_smem + chunk_at<D>(r, c)) = v;
      }
      __syncthreads();
      uint32_t qf[MT == 1 ? kSteps : 1][4];
      const auto q_frag = [&](uint32_t(&f)[4], int mt, int kk) {
        const int m = lane >> 3, r = mt * 16 + (m & 1) * 8 + (lane & 7);
        ldsm4(f, q_addr + chunk_at<D>(r, 2 * kk + (m >> 1)));
      };
      if constexpr (MT == 1) {
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) q_frag(qf[kk], 0, kk);
      }

      // ---- fragments: addresses of the 16-key blocks' chunks within a sub-tile, for step & 3
      const int g = lane >> 3, r7 = lane & 7;
      uint32_t k_at[4], v_at[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        k_at[q] = chunk_at<D>((g >> 1) * 8 + r7, 2 * q + (g & 1));
        v_at[q] = C::kSubBytes + chunk_at<D>((g & 1) * 8 + r7, 2 * q + (g >> 1));
      }
      const auto q_of = [&](uint32_t(&f)[4], int mt, int kk) {
        if constexpr (MT == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = qf[kk][e];
        } else {
          q_frag(f, mt, kk);
        }
      };
      int stage = 0;
      for (int j = u.t0; j < u.t1; ++j) {
        cp_wait<kStages - 2>();
        __syncwarp();
        issue_next();  // into the sub-tile that the last round read
        const int32_t s0 = kSel ? 0 : first_key(j);
        uint32_t valid = 0xffffffffu;
        bool any, all;
        if constexpr (kSel) {
          valid = s_valid[warp][stage];
          any = valid != 0;
          all = valid == (0xffffffffu >> (32 - kSub));
        } else {
          any = s0 <= p_hi && (s0 + kSub - 1 > w_lo || s0 < p.sinks);
          all = s0 + kSub - 1 <= p_lo && (s0 > w_hi || s0 + kSub <= p.sinks);
        }
        if (any) {
          score_subtile<T, D, MT, kSel>(p, smem, ring + stage * C::kStageBytes, k_at, v_at, q_of,
                                        valid, all, s0, rpos, o, m, l);
        }
        __syncwarp();
        stage = stage + 1 == kStages ? 0 : stage + 1;
      }
      cp_wait<0>();
      __syncthreads();  // the rings are free: the warps' results go there

      // ---- join of the four warps
      float* const join = reinterpret_cast<float*>(smem);
      constexpr int kPitch = D + C::kPad;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = mt * 16 + h * 8 + (lane >> 2);
          float sum = l[mt][h];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if ((lane & 3) == 0) {
            s_m[warp][r] = m[mt][h];
            s_l[warp][r] = sum;
          }
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2*>(join + (warp * C::kRows + r) * kPitch + n * 8 +
                                       2 * (lane & 3)) =
                make_float2(o[mt][n][2 * h], o[mt][n][2 * h + 1]);
        }
      __syncthreads();
      const auto write_row = [&](int r, int d, float mx, float sum, const float4& v) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        int64_t token;
        int head, pos;
        row_place(p, u, r, &token, &head, &pos);
        const int64_t at = token * p.num_heads + head;
        const uint2 b = make_uint2(pack2<T>(v.x * inv, v.y * inv), pack2<T>(v.z * inv, v.w * inv));
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + at * D + d) = b;
        if (d == 0 && p.lse) p.lse[at] = row_lse<static_cast<int>(kTopWeight<T>)>(mx, sum);
      };
      for (int i = threadIdx.x; i < u.rows * (D / 4); i += kWarps * 32) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][r]);
        const float base = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = exp2_approx(s_m[w][r] - base);
          const float4 a =
              *reinterpret_cast<const float4*>(join + (w * C::kRows + r) * kPitch + d);
          sum += f * s_l[w][r];
          v.x += f * a.x;
          v.y += f * a.y;
          v.z += f * a.z;
          v.w += f * a.w;
        }
        if constexpr (kCluster) {
          // (where the thread's first summand was)
          *reinterpret_cast<float4*>(join + r * kPitch + d) = v;
          if (d == 0) s_part[r] = make_float2(mx, sum);
        } else if (whole) {
          write_row(r, d, mx, sum, v);
        } else {
          const int64_t slot = 2 * static_cast<int64_t>(cta) + (u.t0 == 0 ? 1 : 0);
          *reinterpret_cast<float4*>(p.part_o + (slot * p.rows + r) * D + d) = v;
          if (d == 0) p.part_ml[slot * p.rows + r] = make_float2(mx, sum);
        }
      }
      if constexpr (kCluster) {
        // ---- join of the cluster's blocks, in their order; each writes a share of the unit
        cluster_sync();
        for (int i = rank * (kWarps * 32) + threadIdx.x; i < u.rows * (D / 4);
             i += p.cluster * (kWarps * 32)) {
          const int r = i / (D / 4), d = i % (D / 4) * 4;
          const uint32_t part_at = smem_u32(&s_part[r]), o_at = smem_u32(join + r * kPitch + d);
          float bm[kMostCluster], bl[kMostCluster];
          float4 bo[kMostCluster];
#pragma unroll
          for (int b = 0; b < kMostCluster; ++b) {
            bm[b] = -INFINITY;
            bl[b] = 0.f;
            bo[b] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (b < p.cluster) {
              const uint32_t at = cluster_addr(part_at, b);
              bm[b] = cluster_load(at);
              bl[b] = cluster_load(at + 4);
              bo[b] = cluster_load4(cluster_addr(o_at, b));
            }
          }
          float mx = -INFINITY;
#pragma unroll
          for (int b = 0; b < kMostCluster; ++b) mx = fmaxf(mx, bm[b]);
          const float base = mx == -INFINITY ? 0.f : mx;
          float sum = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int b = 0; b < kMostCluster; ++b) {
            const float f = exp2_approx(bm[b] - base);
            sum += f * bl[b];
            v.x += f * bo[b].x;
            v.y += f * bo[b].y;
            v.z += f * bo[b].z;
            v.w += f * bo[b].w;
          }
          write_row(r, d, mx, sum, v);
        }
        cluster_sync();  // (the results are read before their memory is used again)
      }
      __syncthreads();
    }

  }
}

// The selected form with a warp per unit of 16 query rows, for many tokens: no
// unit is cut, no warp waits for another, and a warp's ring goes on from one unit
// to the next, whose list and pages are looked up while the last one is scored
// (a CTA per unit stands still for 4 us between units). 8000 tokens, one kv head
// of 128, lists of 128: 76 us against 130 with a CTA per unit. Bound by the
// latency of a sub-tile's dependent products with two warps a scheduler (1.1 us
// for 8 KB), then by the reads of K and V rows from L2.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 2) attend_lists_kernel(const AttendParams p) {
  using C = RowsCfg<D, 1>;
  constexpr int kChunks = D / 8, kSteps = D / 16, kSub = C::kSub, kPerPass = 32 / kChunks;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_valid[kWarps][kStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ring = smem_u32(smem) + warp * (kStages * C::kStageBytes);
  pdl_wait();
  pdl_trigger();
  const int blocks = (p.group + 15) / 16;
  const int64_t units = selected_units(p);
  const int64_t all_warps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int32_t unit0 = static_cast<int32_t>(cut_position(units, all_warps, static_cast<int>(w)));
  const int32_t unit1 = static_cast<int32_t>(cut_position(units, all_warps, static_cast<int>(w) + 1));
  if (unit0 >= unit1) return;
  const int32_t tiles = (p.topk + kSub - 1) / kSub;

  // The request of a token, looked up when the last one's tokens end.
  struct Found {
    int32_t req = -1, begin = 0, end = 0;
    __device__ __forceinline__ void find(const AttendParams& p, int32_t token) {
      if (token >= begin && token < end) return;
      req = token_request(p, token);
      begin = req < 0 ? token : p.query_start_loc[req];
      end = req < 0 ? token + 1 : p.query_start_loc[req + 1];
    }
  };

  // ---- copies, ahead of the scores: list entries two sub-tiles before their copies are issued,
  // pages one
  Found ahead;
  int32_t unit_in = unit0, tile_in = 0, head_in = 0;
  const int32_t* list = nullptr;
  const int32_t* bt = nullptr;
  const auto enter = [&] {
    const int32_t tb = unit_in / p.num_kv_heads, token = tb / blocks;
    head_in = unit_in - tb * p.num_kv_heads;
    ahead.find(p, token);
    list = p.indices + static_cast<int64_t>(token) * p.indices_stride;
    bt = p.block_table + static_cast<int64_t>(max(ahead.req, 0)) * p.bt_stride;
  };
  enter();
  int32_t idx1 = -1, head1 = 0, idx0 = -1, page0 = -1, head0 = 0;
  const int32_t* bt1 = bt;
  bool there1 = false, there0 = false;
  // moves every sub-tile one step on: its list entries, then its pages
  const auto look = [&] {
    idx0 = idx1;
    head0 = head1;
    there0 = there1;
    page0 = idx1 >= 0 && idx1 < p.bt_width * kPageTokens ? bt1[idx1 / kPageTokens] : -1;
    there1 = unit_in < unit1;
    idx1 = -1;
    if (there1) {
      const int at = tile_in * kSub + (lane & (kSub - 1));
      if (ahead.req >= 0 && at < p.topk) idx1 = list[at];
      head1 = head_in;
      bt1 = bt;
      if (++tile_in == tiles) {
        tile_in = 0;
        if (++unit_in < unit1) enter();
      }
    }
  };
  const int c = lane % kChunks, h0 = lane / kChunks;
  const uint32_t lane_at = chunk_at<D>(h0, c);
  int stage_in = 0;
  const auto issue = [&] {
    if (there0) {
      const uint32_t dst = ring + stage_in * C::kStageBytes;
      const bool ok = idx0 >= 0 && page0 >= 0 && page0 < p.num_pages;
      if (idx0 >= 0 && !ok) set_error(p.dev_error, IDX_DEV_BAD_BLOCK);
      uint32_t valid = __ballot_sync(0xffffffffu, ok);
      if (kSub < 32) valid &= (1u << (kSub & 31)) - 1;
      if (lane == 0) s_valid[warp][stage_in] = valid;
      const int64_t pg = ok ? page0 : 0;
      const int32_t tok = ok ? idx0 & (kPageTokens - 1) : 0;
      const int64_t k_row = pg * p.k_stride_page + tok * p.k_stride_token;
      const int64_t v_row = p.same_strides ? k_row : pg * p.v_stride_page + tok * p.v_stride_token;
      const T* const k_lane = static_cast<const T*>(p.k) + head0 * p.k_stride_head + c * 8;
      const T* const v_lane = static_cast<const T*>(p.v) + head0 * p.v_stride_head + c * 8;
#pragma unroll
      for (int i = 0; i < kSub / kPerPass; ++i) {
        const int key = i * kPerPass + h0;
        const int64_t ka = __shfl_sync(0xffffffffu, k_row, key);
        const int64_t va = p.same_strides ? ka : __shfl_sync(0xffffffffu, v_row, key);
        const bool v = (valid >> key) & 1;
        const uint32_t at =
            dst + i * kPerPass * (D * 2) + (lane_at ^ (((i * kPerPass) & 7) << 4));
        cp_async16(at, k_lane + ka, v);
        cp_async16(at + C::kSubBytes, v_lane + va, v);
      }
    }
    cp_commit();
    stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
    look();
  };
  look();
  look();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  uint32_t k_at[4], v_at[4];
  const int g = lane >> 3, r7 = lane & 7;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    k_at[q] = chunk_at<D>((g >> 1) * 8 + r7, 2 * q + (g & 1));
    v_at[q] = C::kSubBytes + chunk_at<D>((g & 1) * 8 + r7, 2 * q + (g >> 1));
  }
  const int32_t rpos[1][2] = {};  // (a list's keys are seen by every row)
  Found here;
  int stage = 0;
  for (int32_t unit = unit0; unit < unit1; ++unit) {
    const int32_t tb = unit / p.num_kv_heads, kv_head = unit - tb * p.num_kv_heads;
    const int32_t token = tb / blocks, row0 = (tb - token * blocks) * 16;
    here.find(p, token);
    // ---- queries straight into fragments: rows lane / 4 and 8 on, column pairs
    uint32_t qf[kSteps][4];
    const int row = lane >> 2, rows = min(16, p.group - row0);
    const T* const q = static_cast<const T*>(p.q) + token * p.q_stride_token +
                       static_cast<int64_t>(kv_head * p.group + row0) * p.q_stride_head + 2 * (lane & 3);
#pragma unroll
    for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = row + (e & 1) * 8;
        qf[kk][e] = r < rows ? *reinterpret_cast<const uint32_t*>(q + r * p.q_stride_head + kk * 16 +
                                                                  (e >> 1) * 8)
                             : 0u;
      }
    const auto q_of = [&](uint32_t(&f)[4], int, int kk) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = qf[kk][e];
    };
    float o[1][D / 8][4], m[1][2] = {{-INFINITY, -INFINITY}}, l[1][2] = {};
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[0][n][e] = 0.f;
    for (int j = 0; j < tiles; ++j) {
      cp_wait<kStages - 2>();
      __syncwarp();
      issue();  // into the sub-tile that the last round read
      const uint32_t valid = s_valid[warp][stage];
      if (valid)
        score_subtile<T, D, 1, true>(p, smem, ring + stage * C::kStageBytes, k_at, v_at, q_of, valid,
                                     valid == (0xffffffffu >> (32 - kSub)), 0, rpos, o, m, l);
      __syncwarp();
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    if (here.req < 0) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = l[0][h];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int r = row + 8 * h;
      if (r < rows) {
        const int64_t at = static_cast<int64_t>(token) * p.num_heads + kv_head * p.group + row0 + r;
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + at * D) + (lane & 3);
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          dst[n * 4] = pack2<T>(o[0][n][2 * h] * inv, o[0][n][2 * h + 1] * inv);
        if ((lane & 3) == 0 && p.lse)
          p.lse[at] = row_lse<static_cast<int>(kTopWeight<T>)>(m[0][h], sum);
      }
    }
  }
  cp_wait<0>();
}

// ---------------------------------------------------------------------------
// join of the pieces of units that several CTAs share
// ---------------------------------------------------------------------------

constexpr int kCombineWarps = 4;

// Rows that one warp joins: 1 of a row-block kernel's unit, 4 of 256.
__host__ __device__ constexpr int combine_rows(int32_t rows) { return rows > 64 ? 4 : 1; }

// Block (c, y): the unit whose first piece ends CTA c's range, a warp for
// combine_rows of its rows. Only cuts inside a unit leave work. The lanes look
// at 32 following CTAs' cuts at once, then at their pieces' maxima and sums, so
// that the accumulators' loads do not wait for one another; the pieces are
// joined in the order of the CTAs, so the result does not depend on timing.
// Bound by latency: four dependent loads (one request of 8000 keys, 8 units
// of 31 pieces: 3 us; piece by piece 10).
template <typename T, int D, bool kSel, int kRows>
__global__ void __launch_bounds__(kCombineWarps * 32) attend_combine_kernel(const AttendParams p) {
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int r0 = (blockIdx.y * kCombineWarps + (threadIdx.x >> 5)) * kRows;
  constexpr int kV = D / 32;
  // (four rows a warp: the chunk kernel's)
  constexpr int kTop = static_cast<int>(kRows > 1 ? kTopWeightTc<T> : kTopWeight<T>);
  using Vec = typename std::conditional<kV == 4, float4, float2>::type;
  pdl_wait();
  pdl_trigger();
  Piece u;
  // a cut as (unit, tile) with the unit as three numbers
  const auto cut = [&](int at) -> int4 {
    if constexpr (kSel) {
      const int2 x = selected_cut(p, selected_units(p), at);
      return make_int4(x.x, 0, x.y, 0);
    } else {
      return p.bound[at];
    }
  };
  const auto same = [](const int4& a, const int4& b) {
    return a.x == b.x && a.y == b.y && a.w == b.w;
  };
  const int4 here = cut(c), next = cut(c + 1);
  if (next.z == 0 || (same(here, next) && here.z > 0)) return;
  if constexpr (kSel) {
    const int blocks = (p.group + p.rows - 1) / p.rows;
    const int64_t tb = next.x / p.num_kv_heads;
    u.q0 = static_cast<int32_t>(tb / blocks);
    u.head = next.x % p.num_kv_heads;
    u.row0 = static_cast<int32_t>(tb % blocks) * p.rows;
    u.rows = min(p.rows, p.group - u.row0);
    u.ahead = 0;
    if (token_request(p, u.q0) < 0) return;
  } else {
    if (next.w >= p.num_reqs) return;
    const ReqShape q = request_shape(p, next.w, false);
    u.q0 = q.q0;
    u.head = next.y;
    u.row0 = next.x * p.rows;
    u.rows = min(p.rows, q.nq * p.group - u.row0);
    u.ahead = 0;
  }
  if (r0 >= u.rows) return;
  // (rows past the unit's last are worked out from the last one's and not written)
  const auto row_of = [&](int k) { return min(r0 + k, u.rows - 1); };
  const auto piece = [&](int64_t slot, int k) {
    return *reinterpret_cast<const Vec*>(p.part_o + (slot * p.rows + row_of(k)) * D + lane * kV);
  };
  // the first piece is the last of CTA c, the others the first of theirs
  const int64_t slot0 = 2 * static_cast<int64_t>(c) + 1;
  float mx[kRows], sum[kRows], v[kRows][kV];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const float2 ml = p.part_ml[slot0 * p.rows + row_of(k)];
    const Vec x = piece(slot0, k);
    mx[k] = ml.x;
    sum[k] = ml.y;
#pragma unroll
    for (int e = 0; e < kV; ++e) v[k][e] = reinterpret_cast<const float*>(&x)[e];
  }
  for (int c0 = c + 1; c0 < p.grid; c0 += 32) {
    const int cc = c0 + lane;
    bool in = false, empty = false;
    if (cc < p.grid) {
      const int4 a = cut(cc), b = cut(cc + 1);
      in = same(a, next) && a.z > 0;
      empty = same(b, next) && b.z == a.z;
    }
    const uint32_t all = __ballot_sync(0xffffffffu, in);
    const uint32_t full = __ballot_sync(0xffffffffu, in && !empty);
    float f[kRows];  // the lane's piece's factors
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (in && !empty) ml = p.part_ml[2 * static_cast<int64_t>(cc) * p.rows + row_of(k)];
      float top = ml.x;
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      top = fmaxf(top, mx[k]);
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = exp2_approx(mx[k] - base);
      f[k] = exp2_approx(ml.x - base);
      float add = f[k] * ml.y;
#pragma unroll
      for (int d = 16; d; d >>= 1) add += __shfl_xor_sync(0xffffffffu, add, d);
      sum[k] = sum[k] * keep + add;
      mx[k] = top;
#pragma unroll
      for (int e = 0; e < kV; ++e) v[k][e] *= keep;
    }
    const int n = full ? 32 - __clz(full) : 0;
    // the loads of several pieces side by side (where there is none: the first again, unused)
    constexpr int kAtOnce = 8 / kRows;
    for (int i = 0; i < n; i += kAtOnce) {
      Vec x[kAtOnce][kRows];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a)
#pragma unroll
        for (int k = 0; k < kRows; ++k)
          x[a][k] = piece(full >> (i + a) & 1 ? 2 * static_cast<int64_t>(c0 + i + a) : slot0, k);
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a)
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          const float w = __shfl_sync(0xffffffffu, f[k], i + a);
          if (full >> (i + a) & 1) {
#pragma unroll
            for (int e = 0; e < kV; ++e) v[k][e] += w * reinterpret_cast<const float*>(&x[a][k])[e];
          }
        }
    }
    if (all != 0xffffffffu) break;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (r0 + k >= u.rows) break;
    const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
    int64_t token;
    int head, pos;
    row_place(p, u, r0 + k, &token, &head, &pos);
    const int64_t out = token * p.num_heads + head;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + out * D + lane * kV);
#pragma unroll
    for (int e = 0; e < kV; e += 2) dst[e / 2] = pack2<T>(v[k][e] * inv, v[k][e + 1] * inv);
    if (lane == 0 && p.lse) p.lse[out] = row_lse<kTop>(mx[k], sum[k]);
  }
}

template <typename T, int D, int MT, bool kSel>
idx_status launch_rows_as(const AttendParams& p, cudaStream_t s) {
  using C = RowsCfg<D, MT>;
  const auto kernel = attend_rows_kernel<T, D, MT, kSel, false>;
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = allow_smem<C::kSmem, 0>(kernel, configured);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_pdl(kernel, p.grid, kWarps * 32, C::kSmem, s, p));
}

template <typename T, int D, bool kSel>
idx_status launch_cluster_as(const AttendParams& p, cudaStream_t s) {
  using C = RowsCfg<D, 1>;
  const auto kernel = attend_rows_kernel<T, D, 1, kSel, true>;
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = allow_smem<C::kSmem, 0>(kernel, configured);
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(p.cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

template <typename T, int D>
idx_status launch_lists_as(const AttendParams& p, cudaStream_t s) {
  using C = RowsCfg<D, 1>;
  const auto kernel = attend_lists_kernel<T, D>;
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = allow_smem<C::kRing, 0>(kernel, configured);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_pdl(kernel, p.grid, kWarps * 32, C::kRing, s, p));
}

template <typename T, int D>
idx_status launch_rows_d(const AttendParams& p, int mt, cudaStream_t s) {
  if (p.cluster)
    return p.indices ? launch_cluster_as<T, D, true>(p, s) : launch_cluster_as<T, D, false>(p, s);
  if (!p.indices) return launch_rows_as<T, D, 1, false>(p, s);
  return mt == 1 ? launch_rows_as<T, D, 1, true>(p, s) : launch_rows_as<T, D, 2, true>(p, s);
}

template <typename T, int D>
idx_status launch_combine_as(const AttendParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int per_block = kCombineWarps * combine_rows(p.rows);
  cfg.gridDim = dim3(p.grid, (p.rows + per_block - 1) / per_block);
  cfg.blockDim = dim3(kCombineWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = p.indices                  ? attend_combine_kernel<T, D, true, 1>
                      : combine_rows(p.rows) > 1 ? attend_combine_kernel<T, D, false, 4>
                                                 : attend_combine_kernel<T, D, false, 1>;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

}  // namespace

idx_status launch_attend_plan(const AttendParams& p, cudaStream_t s) {
  return cuda_status(launch_pdl(attend_plan_kernel, 1, kPlanThreads, 0, s, p));
}

idx_status launch_attend_rows(const AttendParams& p, int head_dim, bool half, int mt,
                              cudaStream_t s) {
  if (half)
    return head_dim == 64 ? launch_rows_d<__half, 64>(p, mt, s)
                          : launch_rows_d<__half, 128>(p, mt, s);
  return head_dim == 64 ? launch_rows_d<__nv_bfloat16, 64>(p, mt, s)
                        : launch_rows_d<__nv_bfloat16, 128>(p, mt, s);
}

idx_status launch_attend_lists(const AttendParams& p, int head_dim, bool half, cudaStream_t s) {
  if (half)
    return head_dim == 64 ? launch_lists_as<__half, 64>(p, s) : launch_lists_as<__half, 128>(p, s);
  return head_dim == 64 ? launch_lists_as<__nv_bfloat16, 64>(p, s)
                        : launch_lists_as<__nv_bfloat16, 128>(p, s);
}

idx_status launch_attend_combine(const AttendParams& p, int head_dim, bool half, cudaStream_t s) {
  if (half)
    return head_dim == 64 ? launch_combine_as<__half, 64>(p, s)
                          : launch_combine_as<__half, 128>(p, s);
  return head_dim == 64 ? launch_combine_as<__nv_bfloat16, 64>(p, s)
                        : launch_combine_as<__nv_bfloat16, 128>(p, s);
}

}  // namespace saib
