// Attention of chunks of new tokens over a paged cache on the tcgen05 tensor
// cores: blocks of 256 query rows of one kv head against tiles of 128 keys.
#include <cudaTypedefs.h>

#include <mutex>

#include "attend.cuh"

namespace saib {

namespace {

constexpr int kThreads = 384;
constexpr int kSlotRows = 128;       // rows of one accumulator (a slot)
// Registers per thread after the split: warps 0-3 and warps 4-11. 128 * 72 +
// 256 * 216 = 384 * 168, what the block is launched with.
constexpr int kRegsLaunch = 168, kRegsFeed = 72, kRegsSoftmax = 216;
static_assert(128 * kRegsFeed + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");
constexpr int kTmemCols = 512;
constexpr uint32_t kOddUnits = 8;
constexpr int kPieces = 4;  // pieces that the walk may be ahead

template <int D>
struct TcCfg {
  // At D = 64 the accumulators leave room for the weights beside the scores: the next tile's scores
  // are then computed while this one's weights are (2 x 8192 tokens, 64/8 heads: 1056 -> 1030 us;
  // windowed prefill 146 -> 140 us; units of 128 rows 99 -> 82 us). At D = 128 the weights lie over
  // the scores, and the second product begins with the first half of a tile's keys.
  static constexpr bool kAhead = D == 64;
  // Tensor memory: scores of slot i at 128 i, its accumulator at kColO + D i, its weights at
  // kColP + kStepP i
  static constexpr int kColO = 256;
  static constexpr int kColP = kAhead ? kColO + 2 * D : 0, kStepP = kAhead ? 64 : 128;
  static constexpr int kSlotBytes = kSlotRows * D * 2;
  static constexpr int kQ = 2 * kSlotBytes;
  static constexpr int kStage = kTileTc * D * 2;
  // Stages of K and of V. While tile j's V is in use, K of j + 1 and j + 2 and V of j + 1 and
  // j + 2 are in flight (K of j is done by then).
  static constexpr int kKStages = D == 128 ? 2 : 5;
  static constexpr int kVStages = D == 128 ? 3 : 5;
  static constexpr int kHalf = kTileTc * 128;  // 64 of the D values of 128 rows
  static constexpr int kSmem = 1024 + kQ + (kKStages + kVStages) * kStage;
  static constexpr int kV0 = kQ + kKStages * kStage;  // first V stage
};

struct TcBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[5], k_empty[5];
  uint64_t v_full[5], v_empty[5], v_ok[5];  // v_ok: edge tiles cleared (or none)
  uint64_t s_full[2], o_full[2];   // o_full: a unit's last product, with kAhead every tile's
  uint64_t s_read[2];              // kAhead: scores are in registers
  uint64_t p_half[2], p_full[2];   // weights of keys 0-63 (not with kAhead) and of all
  uint64_t done;
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  Piece piece[kPieces];  // what the CTA works on, in order; req -1: no more
  int4 cut_end;          // kSelfPlan: where this CTA's range ends
  uint32_t tmem_base;
  int abort_flag;
  uint32_t odd[kOddUnits];  // 1 + the last unit whose edge tiles held infinities or NaNs
};

// Instruction descriptor of kind::f16 with fp32 D: A K-major, B K-major or (kTransB) MN-major.
template <typename T>
__host__ __device__ constexpr uint32_t f16_idesc(int M, int N, bool trans_b) {
  constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : 1u;
  return (1u << 4) | (kType << 7) | (kType << 10) | ((trans_b ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Shared-memory descriptor of an MN-major operand stored with the 128-byte
// swizzle: 64 values of the MN dimension per 128-byte row, eight rows (K) per
// 1024-byte atom, atoms of the next eight rows 1024 bytes on (SBO), the next 64
// values kHalf bytes on (LBO).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lbo >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t x,
                                            int32_t y, int32_t z, int32_t w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t v;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(v));
  return v != 0;
}

// A place in the ring of stages: fills go round it in order.
template <int kStages>
struct Ring {
  int stage = 0;
  uint32_t phase = 0;  // parity of the current round

  __device__ __forceinline__ void step() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// Lane 4a + i's chunk j goes to lane 4a + j's chunk i.
__device__ __forceinline__ void transpose4(uint4 (&w)[4], int lane) {
  const auto swap = [&](uint4& a, uint4& b, int mask) {
    // the lower lane of a pair keeps a and gets the other's a as b, the upper the reverse
    const bool up = lane & mask;
    const uint4 give = up ? a : b;
    const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, mask),
                                 __shfl_xor_sync(0xffffffffu, give.y, mask),
                                 __shfl_xor_sync(0xffffffffu, give.z, mask),
                                 __shfl_xor_sync(0xffffffffu, give.w, mask));
    if (up) a = got; else b = got;
  };
  swap(w[0], w[1], 1);
  swap(w[2], w[3], 1);
  swap(w[0], w[2], 2);
  swap(w[1], w[3], 2);
}

// Whether some row of the unit does not see some key of the tile.
__device__ __forceinline__ bool edge_tile(const AttendParams& p, const UnitTiles& t, int32_t tile) {
  const int32_t s0 = tile * kTileTc;
  return !(s0 + kTileTc - 1 <= t.p_lo && (s0 > t.p_hi - p.window || s0 + kTileTc <= p.sinks));
}

// The n lowest bits of a word, n clamped to [0, 32].
__device__ __forceinline__ uint32_t low_bits(int32_t n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// The infinities and NaNs that were left out of the edge tiles' products, for
// a row that sees them: added to the row where it was written.
template <typename T, int D>
__device__ __noinline__ void add_nonfinite(const AttendParams& p, const Piece u, int32_t pos,
                                           T* out, float* part) {
  const int32_t* bt = p.block_table + static_cast<int64_t>(u.req) * p.bt_stride;
  for (int j = u.t0; j < u.t1; ++j) {
    const int32_t tile = u.tiles.tile(j);
    if (!edge_tile(p, u.tiles, tile)) continue;
    for (int i = 0; i < kTileTc; ++i) {
      const int32_t key = tile * kTileTc + i;
      if (key > pos || (key >= p.sinks && pos - key >= p.window)) continue;
      const int32_t page = bt[key / kPageTokens];
      if (page < 0 || page >= p.num_pages) continue;
      const T* v = static_cast<const T*>(p.v) + page * p.v_stride_page +
                   (key % kPageTokens) * p.v_stride_token + u.head * p.v_stride_head;
      for (int e = 0; e < D; ++e) {
        const float x = static_cast<float>(v[e]);
        if (isfinite(x)) continue;
        if (out) out[e] = static_cast<T>(static_cast<float>(out[e]) + x);
        else part[e] += x;
      }
    }
  }
}

// One CTA per SM walks its range of units. Per unit and tile,
//   S = Q K^T (two slots of 128 rows), P = exp2(S * scale - m), O += P V
// with S, O in tensor memory and P written over S (D = 64: beside it) as the
// second product's A operand, so that scores and weights never leave the SM:
//   warp 0      walks the CTA's pieces and hands them to the other warps; TMA:
//               the tile's two K and two V pages into rings of stages
//   warp 1      one thread issues the products: while one slot's softmax runs,
//               the other slot's products keep the tensor pipe busy
//   warps 2, 3  load a unit's queries; clear infinities and NaNs in the edge
//               tiles' V (a weight of 0 would turn them into NaNs)
//   warps 4-7, 8-11  softmax of slot 0, 1: a thread per row, running maximum
//               raised lazily, row sums in fp32, accumulators written out
// Tiles of 128 keys read K and V once per 256 rows; with fewer rows than 129 in
// a unit slot 1 idles. A tile of both slots costs the tensor pipe 2048 cycles at
// D = 128 and some 1200 at D = 64, the exponentials 1050; it takes 2900 and 2050,
// for a row's chain of scores, maximum, exponentials and products is longer than
// either, and two slots do not hide all of it.
//
// kSelfPlan: the blocks work out their ranges themselves. (A kernel of its own: with the code in
// one, the others take 5 % longer.)
template <typename T, int D, bool kSelfPlan>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using C = TcCfg<D>;
  constexpr int KS = C::kKStages, VS = C::kVStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TcBars bars;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t q_addr = base, k_addr = base + C::kQ, v_addr = base + C::kV0;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* const abort_flag = &bars.abort_flag;

  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    mbar_init(&bars.q_full, 64);
    mbar_init(&bars.q_empty, 1);
    for (int i = 0; i < 5; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.v_empty[i], 1);
      mbar_init(&bars.v_ok[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_half[i], 4);
      mbar_init(&bars.p_full[i], 4);
      mbar_init(&bars.o_full[i], 1);
      mbar_init(&bars.s_read[i], 4);
    }
    mbar_init(&bars.done, 1);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&bars.piece_full[i], 1);
      mbar_init(&bars.piece_empty[i], kThreads / 32 - 1);
    }
    bars.abort_flag = 0;
    for (uint32_t i = 0; i < kOddUnits; ++i) bars.odd[i] = 0;
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 1) tmem_alloc(&bars.tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // All of tensor memory is this block's, so it begins at address 0 (a constant makes the
  // products' issue cheaper).
  constexpr uint32_t tmem = 0;
  if (bars.tmem_base != 0) {
    if (threadIdx.x == 0) set_error(p.dev_error, IDX_DEV_INTERNAL);
    __syncthreads();
    if (warp == 1) tmem_dealloc(bars.tmem_base, kTmemCols);
    return;
  }
  pdl_wait();
  pdl_trigger();
  if constexpr (kSelfPlan) {
    __shared__ int64_t sums[32];
    __shared__ int4 cuts[2];
    __shared__ ReqShape first;
    // (the costs lie where the queries will: written by these threads too, not by TMA; the cuts
    // are in p.bound as well)
    self_plan<kThreads>(p, blockIdx.x, reinterpret_cast<int64_t*>(smem), sums, cuts, &first);
    if (threadIdx.x == 0) bars.cut_end = cuts[1];
  }
  Piece u;

  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait(bar, parity, abort_flag, p.dev_error, p.wait_ns);
  };
  // of a whole warp, which goes on together or not at all
  const auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(bar, parity));
  };

  // The next piece, for a whole warp; false when there is none (or the wait gave up). The walk
  // costs some 2000 cycles a piece (loads and divisions that depend on one another), so the loading
  // thread, which is ahead of all others, does it for them.
  Ring<kPieces> pieces;
  const auto next_piece = [&]() -> bool {
    if (!wait_warp(&bars.piece_full[pieces.stage], pieces.phase)) return false;
    u = bars.piece[pieces.stage];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.piece_empty[pieces.stage]);
    pieces.step();
    return u.req >= 0;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFeed));
    if (warp == 0) {
      if (lane == 0) {
        // ---------------------------------------------------------------- TMA
        Ring<KS> ka;
        Ring<VS> va;
        int64_t tiles = 0;  // K issued
        int64_t v_tiles = 0;
        int filled = 0;  // places of the ring of pieces
        bool ok = true;
        PieceWalk<true> walk(p, p.bound[blockIdx.x],
                             kSelfPlan ? bars.cut_end : p.bound[blockIdx.x + 1]);
        while (ok) {
          if (!walk.next(p, &u)) u.req = -1;
          if (filled < kPieces) ++filled;
          else if (!(ok = wait(&bars.piece_empty[pieces.stage], pieces.phase ^ 1))) break;
          bars.piece[pieces.stage] = u;
          mbar_arrive(&bars.piece_full[pieces.stage]);
          pieces.step();
          if (u.req < 0) break;
          const int32_t* bt = p.block_table + static_cast<int64_t>(u.req) * p.bt_stride;
          const auto pages_of = [&](int j) -> int2 {
            if (j >= u.t1) return make_int2(-1, -1);
            const int32_t c = u.tiles.tile(j) * 2;
            // (the second page may lie past the request's last)
            return make_int2(bt[c], (c + 1) * kPageTokens <= u.tiles.p_hi ? bt[c + 1] : -1);
          };
          // Whether some row of the unit sees a key of page c. Of the others nothing is loaded:
          // their keys are masked, and what the table says of them may be out of date.
          const int32_t before = max(u.tiles.p_lo, 0) - p.window;
          const auto needed = [&](int32_t c) -> bool {
            const int32_t s = c * kPageTokens;
            return s <= u.tiles.p_hi && (s + kPageTokens - 1 > before || s < p.sinks);
          };
          int2 next = pages_of(u.t0);
          for (int j = u.t0; ok && j < u.t1; ++j) {
            int2 pg = next;
            next = pages_of(j + 1);
            const int32_t first = u.tiles.tile(j) * 2;
            const bool a = needed(first), b = needed(first + 1);
            // a page outside the cache is read as the one past its last, of which every value is
            // out of the map's bounds: zeros
            const auto place = [&](int32_t page, bool use) -> int32_t {
              if (page >= 0 && page < p.num_pages) return page;
              if (use) set_error(p.dev_error, IDX_DEV_BAD_BLOCK);
              return static_cast<int32_t>(p.num_pages);
            };
            pg.x = place(pg.x, a);
            pg.y = place(pg.y, b);
            const uint32_t bytes = (static_cast<uint32_t>(a) + b) * kPageTokens * D * 2;
            const auto fill = [&](uint32_t dst, const CUtensorMap* map, uint64_t* bar) {
              if (bytes) mbar_arrive_expect_tx(bar, bytes);
              else mbar_arrive(bar);
#pragma unroll
              for (int h = 0; h < D / 64; ++h) {
                if (a) tma_load_4d(dst + h * C::kHalf, map, h * 64, 0, u.head, pg.x, bar);
                if (b)
                  tma_load_4d(dst + h * C::kHalf + kPageTokens * 128, map, h * 64, 0, u.head, pg.y,
                              bar);
              }
            };
            if (tiles >= KS && !(ok = wait(&bars.k_empty[ka.stage], ka.phase ^ 1))) break;
            fill(k_addr + ka.stage * C::kStage, &kmap, &bars.k_full[ka.stage]);
            ++tiles;
            ka.step();
            if (v_tiles >= VS && !(ok = wait(&bars.v_empty[va.stage], va.phase ^ 1))) break;
            fill(v_addr + va.stage * C::kStage, &vmap, &bars.v_full[va.stage]);
            ++v_tiles;
            va.step();
          }
        }
        if (!ok) {
          // gave up: the copies in flight land before the block leaves
          int dummy = 0;
          for (int64_t f = tiles < KS ? 0 : tiles - KS; f < tiles; ++f)
            mbar_wait(&bars.k_full[f % KS], (f / KS) & 1, &dummy, p.dev_error, p.wait_ns);
          for (int64_t f = v_tiles < VS ? 0 : v_tiles - VS; f < v_tiles; ++f)
            mbar_wait(&bars.v_full[f % VS], (f / VS) & 1, &dummy, p.dev_error, p.wait_ns);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------- products
      // The whole warp walks; one elected lane issues. (Descriptors from warp-uniform values
      // with constant steps: computed by a single diverged thread, they cost 140 cycles a
      // product to issue, against 64 to execute.) What this warp does between a wait and its
      // products delays every chain behind it, so the lanes vote on their waits once a tile: after
      // a wait that gave up, the tile's products still run, on whatever is there.
      constexpr uint32_t kDescQK = f16_idesc<T>(128, kTileTc, false);
      constexpr uint32_t kDescPV = f16_idesc<T>(128, D, true);
      const uint64_t q_desc = sw128_kmajor_desc(q_addr), k_desc = sw128_kmajor_desc(k_addr);
      const uint64_t v_desc = sw128_mnmajor_desc(v_addr, C::kHalf);
      Ring<KS> ka;
      Ring<VS> va;
      uint32_t q_phase = 0, p_phase = 0, r_phase = 0;  // (bit i: slot i)
      bool ok = true, issued = false;
      const auto qk = [&](int slot, int stage) {
        const uint32_t d = tmem + slot * 128;
        const uint64_t a = q_desc + slot * (C::kSlotBytes >> 4);
        const uint64_t b = k_desc + stage * (C::kStage >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss(d, a + (((kk >> 2) * (kSlotRows * 128) + (kk & 3) * 32) >> 4),
                     b + (((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4), kDescQK, kk > 0);
        mma_commit(&bars.s_full[slot]);
      };
      const auto pv = [&](int slot, int stage, int half, bool first) {
        const uint32_t d = tmem + C::kColO + slot * D, a = tmem + C::kColP + slot * C::kStepP;
        const uint64_t b = v_desc + stage * (C::kStage >> 4);
#pragma unroll
        for (int i = 0; i < kTileTc / 32; ++i) {
          const int kk = half * (kTileTc / 32) + i;
          mma_f16_ts(d, a + kk * 8, b + kk * (2048 >> 4), kDescPV, !first || kk > 0);
        }
      };
      while (ok && next_piece()) {
        const int n = u.t1 - u.t0;
        if (n <= 0) continue;
        const int slots = u.rows > kSlotRows ? 2 : 1;
        issued = true;
        ok = wait(&bars.q_full, q_phase) && ok;
        q_phase ^= 1;
        ok = wait(&bars.k_full[ka.stage], ka.phase) && ok;
        // the scores of a tile; its last slot frees K, the last tile's the queries
        const auto scores = [&](int slot, bool last_tile) {
          qk(slot, ka.stage);
          if (slot == slots - 1) {
            mma_commit(&bars.k_empty[ka.stage]);
            if (last_tile) mma_commit(&bars.q_empty);
          }
        };
        // (This and the loops over slots below stay rolled: the code of all roles shares the
        // instruction cache. Unrolled, a window of 1024 + 16 takes 367 us instead of 356 at D = 64.)
#pragma unroll 1
        for (int slot = 0; slot < slots; ++slot) {
          if (C::kAhead && slot == 1) {
            // half a tile later than slot 0's: the exponentials of one slot then fall into the
            // other's waits (5 % faster than beginning together)
            ok = wait(&bars.s_read[0], r_phase & 1) && ok;
            tc_fence_after();
          }
          if (elect_one()) scores(slot, n == 1);
          __syncwarp();
        }
        ka.step();
        if constexpr (C::kAhead) {
          // Slot 1 is half a tile behind: scores of slot 0's next tile, products of slot 1's last
          // weights, scores of its next tile, products of slot 0's weights.
          const auto next_scores = [&](int slot, bool last_tile) {
            ok = wait(&bars.s_read[slot], (r_phase >> slot) & 1) && ok;
            r_phase ^= 1u << slot;
            tc_fence_after();
            if (elect_one()) scores(slot, last_tile);
            __syncwarp();
          };
          const auto products = [&](int slot, int stage, bool first) {
            ok = wait(&bars.p_full[slot], (p_phase >> slot) & 1) && ok;
            p_phase ^= 1u << slot;
            tc_fence_after();
            if (elect_one()) {
              pv(slot, stage, 0, first);
              pv(slot, stage, 1, first);
              mma_commit(&bars.o_full[slot]);
              if (slot == slots - 1) mma_commit(&bars.v_empty[stage]);
            }
            __syncwarp();
          };
          int sv = 0;
          // (the last round has slot 1's products alone)
          for (int j = 0; j < n + slots - 1; ++j) {
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const bool more = j + 1 < n;
            if (more) ok = wait(&bars.k_full[ka.stage], ka.phase) && ok;
#pragma unroll 1
            for (int half = 0; half < slots; ++half) {
              if (more) next_scores(half, j + 2 == n);
              const int of = half + 1 == slots ? j : j - 1;  // the tile whose weights are due
              if (of == j && j < n) {
                sv = va.stage;
                ok = wait(&bars.v_ok[sv], va.phase) && ok;
                va.step();
              }
              if (of >= 0 && of < n) products(slots - 1 - half, sv, of == 0);
            }
            if (more) ka.step();
          }
          // (the last scores were read before their weights came)
          r_phase ^= slots == 2 ? 3u : 1u;
        } else {
          for (int j = 0; j < n; ++j) {
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const int sv = va.stage;
            const bool more = j + 1 < n;
            ok = wait(&bars.v_ok[sv], va.phase) && ok;
            va.step();
#pragma unroll 1
            for (int slot = 0; slot < slots; ++slot) {
              const uint32_t parity = (p_phase >> slot) & 1;
              p_phase ^= 1u << slot;
              ok = wait(&bars.p_half[slot], parity) && ok;
              tc_fence_after();
              if (elect_one()) pv(slot, sv, 0, j == 0);
              __syncwarp();
              if (more && slot == 0) ok = wait(&bars.k_full[ka.stage], ka.phase) && ok;
              ok = wait(&bars.p_full[slot], parity) && ok;
              tc_fence_after();
              if (elect_one()) {
                pv(slot, sv, 1, j == 0);
                if (more) scores(slot, j + 2 == n);
                else mma_commit(&bars.o_full[slot]);
                if (slot == slots - 1) mma_commit(&bars.v_empty[sv]);
              }
              __syncwarp();
            }
            if (more) ka.step();
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (issued) {
        // every product completes before tensor memory is released
        if (elect_one()) {
          mma_commit(&bars.done);
          int dummy = 0;
          mbar_wait(&bars.done, 0, &dummy, p.dev_error, p.wait_ns);
        }
        __syncwarp();
      }
    } else {
      // ------------------------------------------- queries, V of edge tiles
      const int tid = threadIdx.x - 64;
      Ring<VS> va;
      uint32_t unit = 0, q_phase = 0;
      bool ok = true;
      while (ok && next_piece()) {
        const int n = u.t1 - u.t0;
        if (n <= 0) continue;
        if (unit > 0) {
          if (!(ok = wait_warp(&bars.q_empty, q_phase))) break;
          q_phase ^= 1;
        }
        // a lane places a row; D / 8 lanes copy it
        constexpr int kChunks = D / 8, kRowsAtOnce = 32 / kChunks;
        const int most = u.rows > kSlotRows ? kRowsTc : kSlotRows;
        const int c = lane % kChunks;
        for (int r0 = (warp - 2) * 32; r0 < most; r0 += 64) {
          int64_t token = 0;
          int head = 0, pos;
          const int row = r0 + lane;
          if (row < u.rows) row_place(p, u, row, &token, &head, &pos);
          const int64_t from = token * p.q_stride_token + head * p.q_stride_head;
          const uint32_t to = q_addr + (r0 / kSlotRows) * C::kSlotBytes;
#pragma unroll 8
          for (int i = 0; i < 32; i += kRowsAtOnce) {
            const int k = i + lane / kChunks, rr = r0 % kSlotRows + k;
            const int64_t at = __shfl_sync(0xffffffffu, from, k);
            cp_async16(to + (c >> 3) * (kSlotRows * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4),
                       static_cast<const T*>(p.q) + at + c * 8, r0 + k < u.rows);
          }
        }
        cp_commit();
        cp_wait<0>();
        fence_proxy_async_shared();
        mbar_arrive(&bars.q_full);
        for (int j = 0; j < n; ++j) {
          const int32_t tile = u.tiles.tile(u.t0 + j);
          const int stage = va.stage;
          if (!(ok = wait_warp(&bars.v_full[stage], va.phase))) break;
          va.step();
          if (!edge_tile(p, u.tiles, tile)) {
            if (lane == 0) mbar_arrive(&bars.v_ok[stage]);
            continue;
          }
          uint4* v = reinterpret_cast<uint4*>(smem + C::kV0 + stage * C::kStage);
          bool seen = false;
          constexpr int kAtOnce = 8;
          static_assert(C::kStage / 16 % (64 * kAtOnce) == 0, "whole rounds");
#pragma unroll 1
          for (int i0 = tid; i0 < C::kStage / 16; i0 += 64 * kAtOnce) {
            uint32_t hit = 0;
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
              const uint4 x = v[i0 + e * 64];
              hit |= nonfinite_bits<T>(x.x) | nonfinite_bits<T>(x.y) | nonfinite_bits<T>(x.z) |
                     nonfinite_bits<T>(x.w);
            }
            if (!hit) continue;
#pragma unroll 1
            for (int i = i0; i < i0 + 64 * kAtOnce; i += 64) {
              const uint4 x = v[i];
              const uint4 y = make_uint4(clear_nonfinite<T>(x.x), clear_nonfinite<T>(x.y),
                                         clear_nonfinite<T>(x.z), clear_nonfinite<T>(x.w));
              if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) {
                v[i] = y;
                const int32_t key = tile * kTileTc + (i >> 3) % kTileTc;
                seen |= key <= u.tiles.p_hi && (key < p.sinks || max(u.tiles.p_lo, 0) - key < p.window);
              }
            }
          }
          if (seen) *reinterpret_cast<volatile uint32_t*>(&bars.odd[unit % kOddUnits]) = unit + 1;
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.v_ok[stage]);
        }
        ++unit;
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // -------------------------------------------------------------- softmax
    const int slot = (warp - 4) >> 2;
    const int r = slot * kSlotRows + (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lanes + slot * 128, o_col = lanes + C::kColO + slot * D;
    const uint32_t p_col = lanes + C::kColP + slot * C::kStepP;
    const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2);
    uint32_t s_phase = 0, o_phase = 0, unit = 0;
    bool ok = true;
    while (ok && next_piece()) {
      const int n = u.t1 - u.t0;
      const uint32_t this_unit = unit;
      if (n > 0) ++unit;
      if (slot == 1 && u.rows <= kSlotRows) continue;
      int64_t token;
      int head, pos;
      row_place(p, u, r, &token, &head, &pos);
      if (r >= u.rows) pos = INT32_MIN;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int32_t tile = u.tiles.tile(u.t0 + j);
        if (!(ok = wait_warp(&bars.s_full[slot], s_phase))) break;
        s_phase ^= 1;
        tc_fence_after();
        float s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + c * 32, s[c]);
        tmem_ld_wait();
        if (C::kAhead) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.s_read[slot]);
        }
        if (edge_tile(p, u.tiles, tile)) {
          // bit i of a word: key s0 + i is seen (i <= hi and (i > lo or i < first))
          const int32_t s0 = tile * kTileTc;
          const int32_t hi = max(pos, -1) - s0, lo = max(pos, -1) - p.window - s0;
          const int32_t first = p.sinks - s0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t see = low_bits(hi + 1 - 32 * c) &
                                 (~low_bits(lo + 1 - 32 * c) | low_bits(first - 32 * c));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see >> i & 1)) s[c][i] = -INFINITY;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = fmaxf(s[c][0], s[c][1]);
#pragma unroll
          for (int i = 2; i < 32; i += 2) mx[c] = max3(mx[c], s[c][i], s[c][i + 1]);
        }
        const float top =
            fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2 - kTopWeightTc<T>;
        float alpha = 1.f;
        if (top > m + kLazyRaise) {
          alpha = exp2_approx(m - top);
          m = top;
          l *= alpha;
        }
        const auto rescale = [&] {
          if (j == 0 || !__any_sync(0xffffffffu, alpha != 1.f)) return;
          // (rare: short code, which would push the rest out of the instruction cache)
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld32(o_col + c * 32, o);
            tmem_ld_wait();
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * alpha);
            tmem_st32(o_col + c * 32, w);
          }
        };
        if (!C::kAhead) rescale();
        const float sub = m == -INFINITY ? 0.f : -m;
        const uint64_t sub2 = pack_f32x2(sub, sub);
        uint64_t sum2[2] = {0, 0};
        uint32_t w2[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t(&w)[32] = w2[c];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float(&v)[32] = s[2 * c + (i >> 4)];
            const int e = (i & 15) * 2;
            const float2 x = unpack_f32x2(fma_f32x2(pack_f32x2(v[e], v[e + 1]), scale2, sub2));
            const float a = exp2_approx(x.x), b = exp2_approx(x.y);
            sum2[i & 1] = add_f32x2(sum2[i & 1], pack_f32x2(a, b));
            // the weights are rounded to T for the second product (half a step of T
            // each); their sum is of the unrounded ones
            w[i] = pack2<T>(a, b);
          }
          if (C::kAhead) {
            if (c == 0) continue;
            if (j > 0) {
              // the last tile's products are done with its weights and with the accumulator
              if (!(ok = wait_warp(&bars.o_full[slot], o_phase))) break;
              o_phase ^= 1;
              tc_fence_after();
              rescale();
            }
            tmem_st32(p_col, w2[0]);
          }
          tmem_st32(p_col + c * 32, w);
          if (!C::kAhead || c == 1) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c ? &bars.p_full[slot] : &bars.p_half[slot]);
          }
        }
        if (C::kAhead && !ok) break;
        const float2 sum = unpack_f32x2(add_f32x2(sum2[0], sum2[1]));
        l += sum.x + sum.y;
      }
      if (!ok) break;
      // ------------------------------------------------------- accumulators
      if (n > 0) {
        if (!(ok = wait_warp(&bars.o_full[slot], o_phase))) break;
        o_phase ^= 1;
        tc_fence_after();
      }
      const bool odd =
          n > 0 && *reinterpret_cast<volatile uint32_t*>(&bars.odd[this_unit % kOddUnits]) ==
                       this_unit + 1;
      const bool whole = u.whole();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t at = token * p.num_heads + head;
      const int64_t part = (2 * static_cast<int64_t>(blockIdx.x) + (u.t0 == 0 ? 1 : 0)) * p.rows + r;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        if (n > 0) {
          tmem_ld32(o_col + c * 32, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (whole) {
          // four lanes exchange 16-byte chunks, so that together they write 64 bytes of one row
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = make_uint4(pack2<T>(o[8 * i] * inv, o[8 * i + 1] * inv),
                              pack2<T>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                              pack2<T>(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                              pack2<T>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
          __syncwarp();
          transpose4(w, lane);
          uint4* const out = reinterpret_cast<uint4*>(p.out);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int from = (lane & ~3) + i;
            const int64_t row = __shfl_sync(0xffffffffu, at, from);
            if (r - lane + from < u.rows) out[row * (D / 8) + c * 4 + (lane & 3)] = w[i];
          }
        } else if (r < u.rows) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + part * D + c * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        __syncwarp();
      }
      if (r < u.rows) {
        if (!whole) p.part_ml[part] = make_float2(m, l);
        else if (p.lse) p.lse[at] = row_lse<static_cast<int>(kTopWeightTc<T>)>(m, l);
      }
      if (odd) {
        __threadfence_block();  // (the row was written by four lanes)
        __syncwarp();
        if (r < u.rows)
          add_nonfinite<T, D>(p, u, pos, whole ? static_cast<T*>(p.out) + at * D : nullptr,
                              p.part_o + part * D);
        __syncwarp();
      }
      tc_fence_before();
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Map of a cache: [64 tokens of a page][64 of the head_dim values] boxes of one
// head and page.
bool encode_map(CUtensorMap* map, const void* base, bool half, int head_dim, int64_t tok,
                int64_t head, int64_t page, int64_t heads, int64_t pages) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!encode) return false;
  // (the stride of a dimension of one entry is never used; it only has to be valid)
  if (heads == 1) head = tok;
  if (pages == 1) page = tok;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(head_dim), kPageTokens,
                              static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(2 * tok), static_cast<cuuint64_t>(2 * head),
                                 static_cast<cuuint64_t>(2 * page)};
  const cuuint32_t box[4] = {64, kPageTokens, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode(map,
                half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, bool kSelfPlan>
idx_status launch_tc_as(const AttendParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        cudaStream_t s) {
  using C = TcCfg<D>;
  const auto kernel = attend_tc_kernel<T, D, kSelfPlan>;
  // (the register split hands out what the launch holds, no more)
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = allow_smem<C::kSmem, kRegsLaunch>(kernel, configured);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_pdl(kernel, p.grid, kThreads, C::kSmem, s, p, kmap, vmap));
}

template <typename T, int D>
idx_status launch_tc_d(const AttendParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                       cudaStream_t s) {
  return p.self_plan ? launch_tc_as<T, D, true>(p, kmap, vmap, s)
                     : launch_tc_as<T, D, false>(p, kmap, vmap, s);
}

bool map_stride_ok(int64_t stride, int64_t entries) {
  return entries == 1 || (stride > 0 && stride < (int64_t{1} << 38));
}

}  // namespace

bool attend_tc_maps(const AttendParams& p, int head_dim, bool half, CUtensorMap* kmap,
                    CUtensorMap* vmap) {
  return map_stride_ok(p.k_stride_token, 2) && map_stride_ok(p.v_stride_token, 2) &&
         map_stride_ok(p.k_stride_head, p.num_kv_heads) &&
         map_stride_ok(p.v_stride_head, p.num_kv_heads) &&
         map_stride_ok(p.k_stride_page, p.num_pages) &&
         map_stride_ok(p.v_stride_page, p.num_pages) &&
         encode_map(kmap, p.k, half, head_dim, p.k_stride_token, p.k_stride_head, p.k_stride_page,
                    p.num_kv_heads, p.num_pages) &&
         encode_map(vmap, p.v, half, head_dim, p.v_stride_token, p.v_stride_head, p.v_stride_page,
                    p.num_kv_heads, p.num_pages);
}

idx_status launch_attend_tc(const AttendParams& p, int head_dim, bool half, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, cudaStream_t s) {
  if (half)
    return head_dim == 64 ? launch_tc_d<__half, 64>(p, kmap, vmap, s)
                          : launch_tc_d<__half, 128>(p, kmap, vmap, s);
  return head_dim == 64 ? launch_tc_d<__nv_bfloat16, 64>(p, kmap, vmap, s)
                        : launch_tc_d<__nv_bfloat16, 128>(p, kmap, vmap, s);
}

}  // namespace saib
