// New tokens into the caches: keys and values with the position rotation on
// the way, and index keys into an MXFP4 cache.
#include <algorithm>

#include "attend.cuh"

namespace saib {

namespace {

constexpr int kThreads = 128;
constexpr int kManyHeads = 5;  // heads of a lane

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---------------------------------------------------------------------------
// keys and values
// ---------------------------------------------------------------------------

struct AppendParams {
  idx_append a;
  int32_t splits;       // blocks that share a token, or
  int32_t tokens_log2;  // tokens that share a block
};

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (std::is_same<T, __half>::value) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  } else {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
}

// Two 16-byte chunks of a head, x and y, turned by eight angles: pairs (x[i], y[i]), or
// (interleaved) neighbours, x holding the first four pairs. Products and differences in fp32; one
// rounding to T at the end.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void turn(uint4* x, uint4* y, const float (&c)[8], const float (&s)[8]) {
  uint32_t* const a = reinterpret_cast<uint32_t*>(x);
  uint32_t* const b = reinterpret_cast<uint32_t*>(y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInterleaved) {
      const float2 u = unpack2<T>(a[i]), v = unpack2<T>(b[i]);
      a[i] = pack2<T>(u.x * c[i] - u.y * s[i], u.y * c[i] + u.x * s[i]);
      b[i] = pack2<T>(v.x * c[4 + i] - v.y * s[4 + i], v.y * c[4 + i] + v.x * s[4 + i]);
    } else {
      const float2 u = unpack2<T>(a[i]), v = unpack2<T>(b[i]);
      const int e = 2 * i;
      a[i] = pack2<T>(u.x * c[e] - v.x * s[e], u.y * c[e + 1] - v.y * s[e + 1]);
      b[i] = pack2<T>(v.x * c[e] + u.x * s[e], v.y * c[e + 1] + u.y * s[e + 1]);
    }
  }
}

// A token's heads (its queries', keys', values') go round its groups of D / 16 lanes, a lane holding
// two 16-byte chunks of a head: the two halves of eight pairs, whose angles it reads once for all
// its heads. A token has a part of a block, a block, or several of them. The first heads are asked
// for before the token's slot and position are there (16011 tokens of 64/8 heads of 64: 51.3 us
// instead of 55.6), three a lane at a time (50.0; four 52.9). Bound by HBM: 49.4 us, 6.7 TB/s.
template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kUnits = D / 16, kGroups = kThreads / kUnits, kGroupsLog2 = D == 64 ? 5 : 4, kAtOnce = 3;
  static_assert(kGroups == 1 << kGroupsLog2, "groups");
  const idx_append& a = p.a;
  pdl_wait();
  pdl_trigger();
  const int unit = threadIdx.x % kUnits, groups = kGroups >> p.tokens_log2;  // of a token
  const int group = threadIdx.x / kUnits & (groups - 1);
  int block = blockIdx.x, split = 0;
  if (p.splits > 1) {
    block = blockIdx.x / p.splits;
    split = blockIdx.x - block * p.splits;
  }
  const int64_t t =
      (static_cast<int64_t>(block) << p.tokens_log2) + (threadIdx.x / kUnits >> (kGroupsLog2 - p.tokens_log2));
  if (t >= a.num_tokens) return;
  const int step = groups * p.splits;
  const int queries = a.rotary && a.q ? a.num_heads : 0;
  const int keys = queries + a.num_kv_heads, heads = keys + a.num_kv_heads;
  const bool turned = a.rotary && unit < a.rotary_dim / 16;
  // the lane's chunks of a rotated head (of others: 2 unit and the next)
  const int c0 = turned && !kInterleaved ? unit : 2 * unit;
  const int c1 = turned && !kInterleaved ? unit + a.rotary_dim / 16 : 2 * unit + 1;
  const T* const q = static_cast<const T*>(a.q) + t * a.q_stride_token;
  const T* const k = static_cast<const T*>(a.k) + t * a.k_stride_token;
  const T* const v = static_cast<const T*>(a.v) + t * a.v_stride_token;
  uint4 x[kAtOnce], y[kAtOnce];
  const auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int h = h0 + i * step;
      if (h >= heads) break;
      const T* const from = h < queries ? q + h * a.q_stride_head
                            : h < keys  ? k + (h - queries) * a.k_stride_head
                                        : v + (h - keys) * a.v_stride_head;
      x[i] = *(reinterpret_cast<const uint4*>(from) + (h < keys ? c0 : 2 * unit));
      y[i] = *(reinterpret_cast<const uint4*>(from) + (h < keys ? c1 : 2 * unit + 1));
    }
  };
  int h0 = split * groups + group;
  load(h0);
  int64_t slot = a.slot_mapping[t];
  int64_t pos = a.rotary ? a.positions[t] : 0;
  const bool first = unit == 0 && group == 0 && split == 0;
  float c[8], s[8];
  if (a.rotary) {
    const int64_t in = min(max(pos, int64_t{0}), a.num_positions - 1);
    if (first && in != pos && slot >= 0 && slot < a.num_pages * kPageTokens)
      set_error(a.dev_error, IDX_DEV_BAD_LEN);
    if (turned) {
      const float4* row = reinterpret_cast<const float4*>(a.rotary + in * a.rotary_stride) + 2 * unit;
      const float4* sin = row + a.rotary_dim / 8;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<float4*>(c + 4 * i) = __ldg(row + i);
        *reinterpret_cast<float4*>(s + 4 * i) = __ldg(sin + i);
      }
    }
  }
  if (slot >= a.num_pages * kPageTokens) {
    if (first) set_error(a.dev_error, IDX_DEV_BAD_BLOCK);
    slot = -1;
  }
  const int64_t page = slot < 0 ? 0 : slot / kPageTokens, at = slot < 0 ? 0 : slot % kPageTokens;
  T* const q_out = static_cast<T*>(a.q_out) + t * a.q_out_stride_token;
  T* const k_out = static_cast<T*>(a.k_cache) + page * a.k_cache_stride_page + at * a.k_cache_stride_token;
  T* const v_out = static_cast<T*>(a.v_cache) + page * a.v_cache_stride_page + at * a.v_cache_stride_token;
  for (;;) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int h = h0 + i * step;
      if (h >= heads || (h >= queries && slot < 0)) break;
      T* const to = h < queries ? q_out + h * a.q_out_stride_head
                    : h < keys  ? k_out + (h - queries) * a.k_cache_stride_head
                                : v_out + (h - keys) * a.v_cache_stride_head;
      if (turned && h < keys) turn<T, kInterleaved>(&x[i], &y[i], c, s);
      *(reinterpret_cast<uint4*>(to) + (h < keys ? c0 : 2 * unit)) = x[i];
      *(reinterpret_cast<uint4*>(to) + (h < keys ? c1 : 2 * unit + 1)) = y[i];
    }
    h0 += kAtOnce * step;
    if (h0 >= heads) break;
    load(h0);
  }
}

template <typename T, int D>
idx_status launch_append(const AppendParams& p, cudaStream_t s) {
  const auto kernel = p.a.interleaved ? append_kernel<T, D, true> : append_kernel<T, D, false>;
  const unsigned blocks = (static_cast<unsigned>(p.a.num_tokens) + (1u << p.tokens_log2) - 1) >> p.tokens_log2;
  return cuda_status(launch_pdl(kernel, blocks * p.splits, kThreads, 0, s, p));
}

// ---------------------------------------------------------------------------
// index keys, MXFP4
// ---------------------------------------------------------------------------

// Eight values to e2m1 codes (value 2i in the low half of byte i), round to nearest even,
// saturating.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// The larger magnitude of each half of two bf16 pairs; NaN where either is one.
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr int kInsertAtOnce = 2;  // tokens in flight per 16 lanes

// Sixteen lanes a token, eight values each; four lanes hold a block of 32 and its
// largest magnitude. The scale is a power of two, so the products are exact and the
// codes those of the definition. Magnitudes, products by the scale and the values that
// a code stands for are worked out on bf16 pairs (a value from two byte tables): with
// each value by itself the instructions, not the reads and writes, bound it.
__global__ void __launch_bounds__(kThreads)
    insert_mxfp4_kernel(const __nv_bfloat16* __restrict__ k, int64_t k_stride,
                        const int64_t* __restrict__ slots, int64_t n, uint8_t* __restrict__ cache,
                        int64_t num_pages, __nv_bfloat16* __restrict__ values, uint32_t* err) {
  constexpr int kLanes = 16, kAtOnce = kInsertAtOnce, kTokens = kThreads / kLanes;
  constexpr uint32_t kAbs = 0x7fff7fffu;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % kLanes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTokens;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kTokens; base < n; base += kAtOnce * step) {
    const int64_t t0 = base + threadIdx.x / kLanes;
    uint4 raw[kAtOnce];
    int64_t slot[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t t = t0 + u * step;
      raw[u] = make_uint4(0, 0, 0, 0);
      slot[u] = -1;
      if (t < n) {
        raw[u] = *(reinterpret_cast<const uint4*>(k + t * k_stride) + lane);
        slot[u] = slots[t];
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t t = t0 + u * step;
      uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      // bits of the block's largest magnitude
      const auto largest = [&]() -> uint32_t {
        uint32_t m = larger2(larger2(w[0] & kAbs, w[1] & kAbs), larger2(w[2] & kAbs, w[3] & kAbs));
        m = larger2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = larger2(m, __shfl_xor_sync(0xffffffffu, m, 2));
        return max(m & 0xffffu, m >> 16);
      };
      uint32_t top = largest();
      if (__any_sync(0xffffffffu, top > 0x7f80u)) {  // a NaN counts as 0
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((w[i] & 0x7fffu) > 0x7f80u) w[i] &= 0xffff0000u;
          if ((w[i] & 0x7fff0000u) > 0x7f800000u) w[i] &= 0xffffu;
        }
        top = largest();
      }
      // floor(log2 top) + 127 is the exponent field (0 for subnormals, whose E is 0 too)
      const uint32_t e = max(static_cast<int32_t>(top >> 7) - 2, 0);
      const uint32_t down = (254 - e) * 0x00800080u;  // 2^(127 - e), twice
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                         *reinterpret_cast<const __nv_bfloat162*>(&down));
        const uint32_t v = *reinterpret_cast<const uint32_t*>(&y);
        x[2 * i] = __uint_as_float(v << 16);
        x[2 * i + 1] = __uint_as_float(v & 0xffff0000u);
      }
      uint32_t code = e2m1x8(x);
      if (top == 0) code = 0;  // (no signs of zeros)
      if (t >= n) continue;
      const bool bad = slot[u] >= num_pages * kPageTokens;
      if (bad && lane == 0) set_error(err, IDX_DEV_BAD_BLOCK);
      const bool written = slot[u] >= 0 && !bad;
      if (written) {
        // (entries are 68 bytes, so only 4-byte aligned)
        uint8_t* const entry = cache + slot[u] * kMxTokenBytes;
        reinterpret_cast<uint32_t*>(entry)[lane] = code;
        if ((lane & 3) == 0) entry[kDim / 2 + (lane >> 2)] = static_cast<uint8_t>(e);
      }
      if (values) {
        // codes 0 to 7 are 0, 0.5, 1, 1.5, 2, 3, 4, 6: bytes of their bf16 forms
        const uint32_t m = written ? code & 0x77777777u : 0, sign = written ? code & 0x88888888u : 0;
        const uint32_t lo[2] = {__byte_perm(0xc0800000u, 0xc0804000u, m), __byte_perm(0xc0800000u, 0xc0804000u, m >> 16)};
        const uint32_t hi[2] = {__byte_perm(0x3f3f3f00u, 0x40404040u, m), __byte_perm(0x3f3f3f00u, 0x40404040u, m >> 16)};
        // 2^(e - 127), which is subnormal for e = 0
        const uint32_t up = e ? e * 0x00800080u : 0x00400040u;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v = __byte_perm(lo[i >> 1], hi[i >> 1], i & 1 ? 0x7362 : 0x5140);
          v |= (sign << (28 - 8 * i) & 0x80000000u) >> 16 | (sign << (24 - 8 * i) & 0x80000000u);
          const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                           *reinterpret_cast<const __nv_bfloat162*>(&up));
          o[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
        *(reinterpret_cast<uint4*>(values + t * kDim) + lane) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// A stride of a dimension of n entries (of one entry it is never used); `written`: entries apart.
bool stride_ok(int64_t s, int64_t n, bool written) {
  return n <= 1 || (s >= (written ? 1 : 0) && s % 8 == 0);
}

}  // namespace
}  // namespace saib

using namespace saib;

extern "C" {

idx_status indexer_append_kv(const idx_append* a, void* stream) {
  if (!a) return IDX_ERR_INVALID_ARG;
  if (a->dtype != IDX_BF16 && a->dtype != IDX_FP16) return IDX_ERR_UNSUPPORTED;
  if (a->head_dim != 64 && a->head_dim != 128) return IDX_ERR_UNSUPPORTED;
  const bool rotate = a->rotary != nullptr, queries = rotate && a->q;
  if (a->num_tokens < 0 || a->num_kv_heads < 1 || a->num_heads < (queries ? 1 : 0) ||
      a->num_pages < 1 || a->num_pages > INT32_MAX)
    return IDX_ERR_INVALID_ARG;
  // (heads of a token as 32-bit numbers, blocks of a launch)
  if (a->num_heads > 1 << 20 || a->num_kv_heads > 1 << 20 || a->num_tokens > 1 << 28)
    return IDX_ERR_UNSUPPORTED;
  if (rotate) {
    if (a->rotary_dim < 16 || a->rotary_dim % 16 || a->rotary_dim > a->head_dim)
      return IDX_ERR_UNSUPPORTED;
    if (a->interleaved != 0 && a->interleaved != 1) return IDX_ERR_INVALID_ARG;
    if (a->num_positions < 1 || a->rotary_stride < a->rotary_dim || a->rotary_stride % 4 ||
        !aligned(a->rotary, 16))
      return IDX_ERR_INVALID_ARG;
  }
  if (a->num_tokens == 0) return IDX_OK;
  if (!a->k || !a->v || !a->slot_mapping || !a->k_cache || !a->v_cache || !aligned(a->k, 16) ||
      !aligned(a->v, 16) || !aligned(a->slot_mapping, 8) || !aligned(a->k_cache, 16) ||
      !aligned(a->v_cache, 16))
    return IDX_ERR_INVALID_ARG;
  if (rotate && (!a->positions || !aligned(a->positions, 4))) return IDX_ERR_INVALID_ARG;
  const int64_t n = a->num_tokens, kv = a->num_kv_heads;
  if (queries && (!a->q_out || !aligned(a->q, 16) || !aligned(a->q_out, 16) ||
                  !stride_ok(a->q_stride_token, n, false) ||
                  !stride_ok(a->q_stride_head, a->num_heads, false) ||
                  !stride_ok(a->q_out_stride_token, n, true) ||
                  !stride_ok(a->q_out_stride_head, a->num_heads, true)))
    return IDX_ERR_INVALID_ARG;
  if (!stride_ok(a->k_stride_token, n, false) || !stride_ok(a->k_stride_head, kv, false) ||
      !stride_ok(a->v_stride_token, n, false) || !stride_ok(a->v_stride_head, kv, false) ||
      !stride_ok(a->k_cache_stride_page, a->num_pages, true) ||
      !stride_ok(a->k_cache_stride_token, kPageTokens, true) ||
      !stride_ok(a->k_cache_stride_head, kv, true) ||
      !stride_ok(a->v_cache_stride_page, a->num_pages, true) ||
      !stride_ok(a->v_cache_stride_token, kPageTokens, true) ||
      !stride_ok(a->v_cache_stride_head, kv, true))
    return IDX_ERR_INVALID_ARG;
  AppendParams p{*a, 1, 0};
  if (!rotate) p.a.rotary_dim = p.a.interleaved = 0;
  const int heads = (queries ? a->num_heads : 0) + 2 * a->num_kv_heads;
  const int groups = kThreads / (a->head_dim / 16);
  const int rounds = (heads + groups - 1) / groups;  // of a block alone
  // few tokens: a block a round, up to 12 blocks an SM (576 tokens of 64/8 heads of 128: 5.1 us
  // interleaved, 4.7 not; 8 blocks: 5.5, 4.5; 16: 5.3, 5.4); many: so many tokens a block that a lane has some heads (us, one token a block / here:
  // 16011 of 64/8 heads of 64 52.8 / 49.4, 14903 of 16/8 of 128 47.1 / 38.8, 11394 of 9/3 of 64
  // 22.0 / 10.7; three heads a lane: 49.3, 39.5, 10.1, eight: 50.8, 38.8, 9.8)
  const int64_t room = int64_t{12} * device_sm_count() / a->num_tokens;
  p.splits = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(rounds, room)));
  if (room < 1)
    while (groups >> p.tokens_log2 > 1 && heads < kManyHeads * (groups >> p.tokens_log2)) ++p.tokens_log2;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->dtype == IDX_FP16)
    return a->head_dim == 64 ? launch_append<__half, 64>(p, s) : launch_append<__half, 128>(p, s);
  return a->head_dim == 64 ? launch_append<__nv_bfloat16, 64>(p, s)
                           : launch_append<__nv_bfloat16, 128>(p, s);
}

idx_status indexer_insert_keys_mxfp4(const void* k, int64_t k_stride, const int64_t* slot_mapping,
                                     int64_t num_tokens, int32_t head_dim, uint8_t* index_cache,
                                     int64_t num_pages, void* values, uint32_t* dev_error,
                                     void* stream) {
  if (num_tokens < 0 || num_pages < 0) return IDX_ERR_INVALID_ARG;
  if (head_dim != kDim) return IDX_ERR_UNSUPPORTED;
  if (num_tokens == 0) return IDX_OK;
  if (!k || !slot_mapping || !index_cache || !aligned(k, 16) || !aligned(slot_mapping, 8) ||
      !aligned(index_cache, 16) || !aligned(values, 16) || k_stride < kDim || k_stride % 8)
    return IDX_ERR_INVALID_ARG;
  // few tokens: one a group of lanes; many: kInsertAtOnce, and no second round
  const int64_t blocks = (num_tokens + kThreads / 16 - 1) / (kThreads / 16);
  const int64_t grid = std::max(std::min(blocks, int64_t{4} * device_sm_count()),
                                (blocks + kInsertAtOnce - 1) / kInsertAtOnce);
  return cuda_status(launch_pdl(insert_mxfp4_kernel,
                                static_cast<unsigned>(std::min<int64_t>(grid, INT32_MAX)),
                                kThreads, 0, static_cast<cudaStream_t>(stream),
                                static_cast<const __nv_bfloat16*>(k), k_stride, slot_mapping,
                                num_tokens, index_cache, num_pages,
                                static_cast<__nv_bfloat16*>(values), dev_error));
}

}  // extern "C"
