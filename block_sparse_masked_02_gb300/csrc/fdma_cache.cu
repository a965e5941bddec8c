// Writing tokens into a paged key/value cache and reading sequences back.
//
// Both move rows of d values between packed tokens and cache slots and are bound by
// memory traffic (or, for a few tokens, by the latency of token -> sequence -> page ->
// row).  All rows of a call, T tokens times Hkv heads times K and V, form one line of which
// a warp takes PASSES times those that its lanes move at once: bf16 four times two or four rows
// (LPR = 16 or 8 lanes a row, eight values a lane), e4m3 twice four or eight (8 or 4 lanes a row, 16
// values a lane, so that codes too move 16 bytes at a time).  The sequence is searched once for them,
// and every row's load is issued before the first is used.  (Four passes: eight, with fewer warps
// on an SM, took 60 instead of 52 us for 82 thousand tokens of four bf16 heads with some of them in L2; with none
// there it takes 54 us, 6.2 TB/s read and written.  Quantising 19 thousand tokens of eight heads took 23 us, 5.1 TB/s.)
//
// e4m3: with m = max |x| of a row, e is the least integer with m <= 448 * 2^e, taken from
// m's bits: 448 = 1.75 * 2^8, so e = E - 8 where m = f * 2^E has f <= 1.75 and E - 7
// otherwise.  x * 2^-e is exact, so each value is rounded once.
#include "fdma_paged.cuh"

namespace fdma {
namespace {

template <bool FP8>
struct Move {
  static constexpr int kPasses = FP8 ? 2 : 4, kValues = FP8 ? 16 : 8, kVec = kValues / 8;
};
constexpr int kCacheThreads = 128;

struct MoveParams {
  CacheView c;
  const uint16_t* k_new;  // append: (T, Hkv, d), strides in elements
  const uint16_t* v_new;
  int64_t kn[2], vn[2];
  uint16_t* k_out;  // gather: (T, Hkv, d) contiguous
  uint16_t* v_out;
  const int32_t* cu;
  const int32_t* first;
  int T;
  unsigned check_blocks;  // see check_offsets
  int* err;
};

// The sequence of packed token t: the largest b with cu[b] <= t, or -1 where t is behind (or
// before) all of them.  The warp's lanes try 32 places at a time.
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, n = B + 1;  // the answer is in [lo, lo + n) or is lo - 1
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && cu[lo + i] <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) return lo - 1;
    const int last = 31 - __clz(m);
    if (step == 1) {
      const int b = lo + last;
      return b < B ? b : -1;
    }
    lo += last * step + 1;  // cu[lo - 1] <= t
    n = min(step - 1, n - last * step - 1);
  }
  return lo - 1 < B ? lo - 1 : -1;
}

// The same for one lane, by halving.
__device__ __forceinline__ int find_from_start(const int32_t* cu, int B, int t) {
  if (cu[0] > t) return -1;
  int lo = 0, hi = B;  // cu[lo] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo < B ? lo : -1;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Quantises 16 values of a row that LPR lanes hold; returns the codes, e + 127 in `be`.  Every lane of
// the warp calls it.
template <int LPR>
__device__ __forceinline__ uint4 quantise16(const uint4 (&x)[2], uint32_t& be) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  constexpr uint32_t kAbs = 0x7fff7fffu;
  // largest magnitude of the row, as bf16 bits, two values at a time
  uint32_t m2 = w[0] & kAbs;
#pragma unroll
  for (int i = 1; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & kAbs);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
  uint32_t m = max(m2 & 0xffffu, m2 >> 16);
  if (__any_sync(0xffffffffu, m >= 0x7f80u)) {  // a row with infinities or NaN: its largest finite one
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
      m = max(m, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  // m = (1 + mant / 128) * 2^(E - 127), 1.75 = 1 + 96 / 128 (bf16 subnormals fall to the clamp)
  const int E = static_cast<int>(m >> 7), up = (m & 0x7fu) > 96u ? 1 : 0;
  const int b = min(max(E - 8 + up, 1), 246);
  be = static_cast<uint32_t>(b);
  // 2^-(b - 127): exact in bf16 but for products below 2^-126, which become codes of zero either way
  const uint32_t inv = static_cast<uint32_t>(254 - b) * 0x00800080u;
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t y = mul_bf16x2(w[i], inv);
    const float lo = __uint_as_float(y << 16), hi = __uint_as_float(y & 0xffff0000u);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    h[i] = r;
  }
  return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}

// (code -> f16 -> bf16 are exact, and so is the product with a power of two down to bf16's least step, 2^-133;
// below, with scale bytes 1 and 2, it is rounded once, to nearest even.)
__device__ __forceinline__ uint4 dequantise8(uint2 q, uint32_t be) {
  const uint32_t s = (__float_as_uint(exp_scale(be)) >> 16) * 0x10001u;
  uint32_t f[4], r[4];
  e4m3x4_to_f16x4(q.x, f[0], f[1]);
  e4m3x4_to_f16x4(q.y, f[2], f[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(f[i]));
    r[i] = mul_bf16x2(pack_bf16x2(lo, hi), s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// One row of the line: which token, kv head and tensor.
struct Row {
  int64_t tok;
  int g;
  bool is_v, real;
};

// The i-th row of a warp whose first is row rem of the 2 * Hkv of token tok0.  ONE: a warp's rows
// are always one token's.
template <bool ONE>
__device__ __forceinline__ Row warp_row(const MoveParams& p, int64_t tok0, int rem, int i) {
  Row r;
  int x = rem + i, t = 0;
  const int per = 2 * p.c.Hkv;
  if (!ONE && x >= per) {
    t = x / per;
    x -= t * per;
  }
  r.tok = tok0 + t;
  r.real = ONE || r.tok < p.T;
  r.is_v = x >= p.c.Hkv;
  r.g = r.is_v ? x - p.c.Hkv : x;
  return r;
}

// The sequence of token t, which is not before one of sequence b (of token b's search); -1: none.
__device__ __forceinline__ int seq_from(const MoveParams& p, int b, int t) {
  if (b < 0) return find_from_start(p.cu, p.c.B, t);
  while (b < p.c.B && p.cu[b + 1] <= t) ++b;
  return b < p.c.B ? b : -1;
}

// Reports offsets that do not begin at 0 or later, run backwards or end behind T.  (The lookups see only the sequences
// of tokens that are there.)  The first warps of the first check_blocks blocks share them, beside the search: with more
// warps, or at the end with a pair in registers, 50 us of quantisation took 2 us more.
__device__ __forceinline__ void check_offsets(const MoveParams& p) {
  if (blockIdx.x >= p.check_blocks || threadIdx.x >= 32) return;
  bool bad = false;
  for (int64_t i = blockIdx.x * 32 + threadIdx.x; i < p.c.B; i += static_cast<int64_t>(gridDim.x) * 32)
    bad |= p.cu[i] > p.cu[i + 1] || p.cu[i] < 0 || p.cu[i + 1] > p.T;
  if (bad) atomicCAS(p.err, 0, FDMA_ERR_INVALID);
}

// Page of position pos of sequence b, or -1 (reported).
__device__ __forceinline__ int page_at(const MoveParams& p, int b, int pos) {
  const int pg = p.c.table[static_cast<int64_t>(b) * p.c.table_stride + (pos >> p.c.page_shift)];
  if (pg >= 0 && pg < p.c.num_pages) return pg;
  atomicCAS(p.err, 0, FDMA_ERR_INVALID);
  return -1;
}

// Where a token's rows lie in the cache, as byte offsets of kv head 0.
struct Slot {
  int64_t tok = -1;
  bool owned = false;  // a sequence has the token
  bool paged = false;  // and its position has a slot
  int64_t k, v, ke, ve;
};

template <bool FP8>
__device__ __forceinline__ void set_slot(const MoveParams& p, Slot& s, int pg, int pos) {
  const int64_t at = pos & ((1 << p.c.page_shift) - 1);
  s.paged = true;
  s.k = pg * p.c.ks[0] + at * p.c.ks[1];
  s.v = pg * p.c.vs[0] + at * p.c.vs[1];
  if (FP8) {
    s.ke = pg * p.c.kes[0] + at * p.c.kes[1];
    s.ve = pg * p.c.ves[0] + at * p.c.ves[1];
  }
}

template <bool FP8, int LPR, bool ONE>
__global__ void __launch_bounds__(kCacheThreads) kv_append_kernel(const __grid_constant__ MoveParams p) {
  constexpr int RPP = 32 / LPR, PASSES = Move<FP8>::kPasses, VEC = Move<FP8>::kVec;
  const int lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  int64_t tok0;
  int rem;
  if (ONE) {  // a warp's rows divide a token's
    const uint32_t per = static_cast<uint32_t>(2 * p.c.Hkv) / (RPP * PASSES), t = w / per;
    tok0 = t;
    rem = static_cast<int>(w - t * per) * (RPP * PASSES);
  } else {
    const int64_t first = static_cast<int64_t>(w) * (RPP * PASSES);
    tok0 = first / (2 * p.c.Hkv);
    rem = static_cast<int>(first - tok0 * (2 * p.c.Hkv));
  }
  if (tok0 >= p.T) return;  // (never a block's first warp)
  check_offsets(p);
  const int col = (lane % LPR) * Move<FP8>::kValues;
  const bool in = col < p.c.d;
  // the rows themselves do not depend on the slot: load them while it is looked up
  uint4 x[PASSES][VEC];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const Row r = warp_row<ONE>(p, tok0, rem, i * RPP + lane / LPR);
    const uint4* src = reinterpret_cast<const uint4*>((r.is_v ? p.v_new : p.k_new) + r.tok * (r.is_v ? p.vn[0] : p.kn[0]) +
                                                      r.g * (r.is_v ? p.vn[1] : p.kn[1]) + col);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[i][e] = in && r.real ? __ldg(src + e) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int b0 = find_seq(p.cu, p.c.B, static_cast<int>(tok0), lane);
  Slot s;
  auto look_up = [&](int64_t tok) {
    s = Slot{};
    s.tok = tok;
    const int t = static_cast<int>(tok), b = seq_from(p, b0, t);
    if (b < 0) return;  // behind the last sequence
    // (cu[b] <= t < cu[b + 1] whatever cu holds, so the position is below k_len)
    const int kl = p.c.k_len[b], pos = kl < 0 ? -1 : kl - (p.cu[b + 1] - t);
    if (pos < 0 || kl > p.c.max_pages << p.c.page_shift) {
      atomicCAS(p.err, 0, FDMA_ERR_INVALID);
      return;
    }
    const int pg = page_at(p, b, pos);
    if (pg >= 0) set_slot<FP8>(p, s, pg, pos);
  };
  look_up(tok0);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const Row r = warp_row<ONE>(p, tok0, rem, i * RPP + lane / LPR);
    uint32_t be = 0;
    uint4 q = x[i][0];
    if constexpr (FP8) q = quantise16<LPR>(x[i], be);
    if (!r.real) continue;
    if (!ONE && r.tok != s.tok) look_up(r.tok);
    if (!s.paged) continue;
    uint8_t* dst = const_cast<uint8_t*>(r.is_v ? p.c.v : p.c.k) + (r.is_v ? s.v : s.k) +
                   r.g * (r.is_v ? p.c.vs[2] : p.c.ks[2]);
    if (in) *reinterpret_cast<uint4*>(dst + col * (FP8 ? 1 : 2)) = q;
    if (FP8) {
      if (col == 0)
        const_cast<uint8_t*>(r.is_v ? p.c.ve : p.c.ke)[(r.is_v ? s.ve : s.ke) + r.g * (r.is_v ? p.c.ves[2] : p.c.kes[2])] =
            static_cast<uint8_t>(be);
    }
  }
}

template <bool FP8, int LPR, bool ONE>
__global__ void __launch_bounds__(kCacheThreads) kv_gather_kernel(const __grid_constant__ MoveParams p) {
  constexpr int RPP = 32 / LPR, PASSES = Move<FP8>::kPasses;
  const int lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  int64_t tok0;
  int rem;
  if (ONE) {  // a warp's rows divide a token's
    const uint32_t per = static_cast<uint32_t>(2 * p.c.Hkv) / (RPP * PASSES), t = w / per;
    tok0 = t;
    rem = static_cast<int>(w - t * per) * (RPP * PASSES);
  } else {
    const int64_t first = static_cast<int64_t>(w) * (RPP * PASSES);
    tok0 = first / (2 * p.c.Hkv);
    rem = static_cast<int>(first - tok0 * (2 * p.c.Hkv));
  }
  if (tok0 >= p.T) return;  // (never a block's first warp)
  check_offsets(p);
  const int col = (lane % LPR) * Move<FP8>::kValues;
  const bool in = col < p.c.d;
  const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.page_shift;
  const int b0 = find_seq(p.cu, p.c.B, static_cast<int>(tok0), lane);
  uint4 x[PASSES];
  uint32_t be[PASSES];
  uint32_t store = 0;  // bit i: pass i has a row to write
  Slot s;
  auto look_up = [&](int64_t tok) {
    s = Slot{};
    s.tok = tok;
    const int t = static_cast<int>(tok), b = seq_from(p, b0, t);
    if (b < 0) return;
    s.owned = true;
    const int64_t at = static_cast<int64_t>(p.first != nullptr ? p.first[b] : 0) + (t - p.cu[b]);
    const int kl = p.c.k_len[b];
    if (kl < 0 || kl > cap) atomicCAS(p.err, 0, FDMA_ERR_INVALID);
    if (at < 0 || at >= min(static_cast<int64_t>(kl), cap)) return;
    const int pg = page_at(p, b, static_cast<int>(at));
    if (pg >= 0) set_slot<FP8>(p, s, pg, static_cast<int>(at));
  };
  look_up(tok0);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const Row r = warp_row<ONE>(p, tok0, rem, i * RPP + lane / LPR);
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    be[i] = 127;
    if (!r.real) continue;
    if (!ONE && r.tok != s.tok) look_up(r.tok);
    if (!s.owned) continue;
    store |= 1u << i;
    if (!s.paged || !in) continue;
    const uint8_t* src = (r.is_v ? p.c.v : p.c.k) + (r.is_v ? s.v : s.k) + r.g * (r.is_v ? p.c.vs[2] : p.c.ks[2]);
    x[i] = __ldg(reinterpret_cast<const uint4*>(src + col * (FP8 ? 1 : 2)));
    if (FP8)
      be[i] = (r.is_v ? p.c.ve : p.c.ke)[(r.is_v ? s.ve : s.ke) + r.g * (r.is_v ? p.c.ves[2] : p.c.kes[2])];
  }
  if (!in) return;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    if (!((store >> i) & 1u)) continue;
    const Row r = warp_row<ONE>(p, tok0, rem, i * RPP + lane / LPR);
    uint4* dst = reinterpret_cast<uint4*>((r.is_v ? p.v_out : p.k_out) + (r.tok * p.c.Hkv + r.g) * p.c.d + col);
    if (FP8) be[i] = scale_byte(be[i]);
    dst[0] = FP8 ? dequantise8(make_uint2(x[i].x, x[i].y), be[i]) : x[i];
    if (FP8) dst[1] = dequantise8(make_uint2(x[i].z, x[i].w), be[i]);
  }
}

struct Append {
  template <bool FP8, int LPR, bool ONE>
  static auto kernel() {
    return kv_append_kernel<FP8, LPR, ONE>;
  }
};
struct Gather {
  template <bool FP8, int LPR, bool ONE>
  static auto kernel() {
    return kv_gather_kernel<FP8, LPR, ONE>;
  }
};

// A warp's rows are one token's where they divide its 2 * Hkv (the usual head counts); that form needs
// no division a row and one lookup a warp.
template <typename K>
void launch_move(bool fp8, int d, int Hkv, unsigned blocks, const MoveParams& p, cudaStream_t stream, K) {
  const int rows = d > 64 ? 8 : 16;  // of a warp
  const bool one = 2 * Hkv % rows == 0;
  void (*kern)(MoveParams);
  if (d > 64)
    kern = fp8 ? (one ? K::template kernel<true, 8, true>() : K::template kernel<true, 8, false>())
               : (one ? K::template kernel<false, 16, true>() : K::template kernel<false, 16, false>());
  else
    kern = fp8 ? (one ? K::template kernel<true, 4, true>() : K::template kernel<true, 4, false>())
               : (one ? K::template kernel<false, 8, true>() : K::template kernel<false, 8, false>());
  kern<<<blocks, kCacheThreads, 0, stream>>>(p);
}

int64_t move_blocks(int T, int Hkv, int d) {
  const int64_t rows = static_cast<int64_t>(T) * 2 * Hkv, per = (d > 64 ? 8 : 16) * (kCacheThreads / 32);
  return (rows + per - 1) / per;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

int validate_cache(const fdma_kv_cache* c) {
  if (c == nullptr) return FDMA_ERR_INVALID;
  if (c->B < 0 || c->Hkv <= 0 || c->d <= 0 || c->num_pages < 0 || c->page_size <= 0 || c->max_pages < 0 ||
      c->table_stride < 0)
    return FDMA_ERR_INVALID;
  if (c->cache_type != FDMA_CACHE_BF16 && c->cache_type != FDMA_CACHE_E4M3) return FDMA_ERR_INVALID;
  const bool fp8 = c->cache_type == FDMA_CACHE_E4M3;
  if (c->d > 128 || c->d % (fp8 ? 16 : 8) != 0) return FDMA_ERR_UNSUPPORTED;
  if (c->B > (1 << 30) || c->Hkv > (1 << 20)) return FDMA_ERR_UNSUPPORTED;  // (B + 1 and 2 * Hkv are formed in 32 bits)
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0) return FDMA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->max_pages) * c->page_size > (1 << 30)) return FDMA_ERR_UNSUPPORTED;
  if (c->B == 0) return FDMA_OK;
  if (c->page_table == nullptr || c->k_len == nullptr) return c->max_pages == 0 && c->k_len ? FDMA_OK : FDMA_ERR_INVALID;
  if (c->num_pages == 0) return FDMA_OK;
  if (c->k == nullptr || c->v == nullptr) return FDMA_ERR_INVALID;
  if (!aligned16(c->k) || !aligned16(c->v)) return FDMA_ERR_UNSUPPORTED;
  const int per16 = fp8 ? 16 : 8;
  for (const int64_t* st : {c->k_stride, c->v_stride})
    for (int i = 0; i < 3; ++i) {
      if (st[i] < 0) return FDMA_ERR_INVALID;
      if (st[i] % per16 != 0) return FDMA_ERR_UNSUPPORTED;
    }
  if (fp8) {
    if (c->k_exp == nullptr || c->v_exp == nullptr) return FDMA_ERR_INVALID;
    for (const int64_t* st : {c->k_exp_stride, c->v_exp_stride})
      for (int i = 0; i < 3; ++i)
        if (st[i] < 0) return FDMA_ERR_INVALID;
  }
  return FDMA_OK;
}

CacheView cache_view(const fdma_kv_cache& c) {
  CacheView v{};
  const int es = c.cache_type == FDMA_CACHE_E4M3 ? 1 : 2;
  v.k = static_cast<const uint8_t*>(c.k);
  v.v = static_cast<const uint8_t*>(c.v);
  v.ke = c.k_exp;
  v.ve = c.v_exp;
  for (int i = 0; i < 3; ++i) {
    v.ks[i] = c.k_stride[i] * es;
    v.vs[i] = c.v_stride[i] * es;
    v.kes[i] = c.k_exp_stride[i];
    v.ves[i] = c.v_exp_stride[i];
  }
  v.table = c.page_table;
  v.table_stride = c.table_stride;
  v.k_len = c.k_len;
  v.B = c.B;
  v.Hkv = c.Hkv;
  v.d = c.d;
  v.num_pages = c.num_pages;
  v.max_pages = c.max_pages;
  while ((1 << v.page_shift) < c.page_size) ++v.page_shift;
  return v;
}

}  // namespace fdma

using namespace fdma;

extern "C" {

int fdma_kv_append(const fdma_kv_cache* c, const void* k_new, const int64_t kn[2], const void* v_new,
                   const int64_t vn[2], const int32_t* cu, int T, void* stream) {
  const int st = validate_cache(c);
  if (st != FDMA_OK) return st;
  if (T < 0) return FDMA_ERR_INVALID;
  if (T == 0 || c->B == 0) return FDMA_OK;
  if (k_new == nullptr || v_new == nullptr || cu == nullptr || kn == nullptr || vn == nullptr) return FDMA_ERR_INVALID;
  if (!aligned16(k_new) || !aligned16(v_new)) return FDMA_ERR_UNSUPPORTED;
  for (int i = 0; i < 2; ++i) {
    if (kn[i] < 0 || vn[i] < 0) return FDMA_ERR_INVALID;
    if (kn[i] % 8 != 0 || vn[i] % 8 != 0) return FDMA_ERR_UNSUPPORTED;
  }
  // distinct slots must be distinct memory
  for (int i = 0; i < 3; ++i) {
    const int n = i == 0 ? c->num_pages : i == 1 ? c->page_size : c->Hkv;
    if (n > 1 && (c->k_stride[i] == 0 || c->v_stride[i] == 0)) return FDMA_ERR_INVALID;
    if (n > 1 && c->cache_type == FDMA_CACHE_E4M3 && (c->k_exp_stride[i] == 0 || c->v_exp_stride[i] == 0))
      return FDMA_ERR_INVALID;
  }
  const int64_t blocks = move_blocks(T, c->Hkv, c->d);
  if (blocks > 0x1fffffff) return FDMA_ERR_UNSUPPORTED;
  MoveParams p{};
  p.c = cache_view(*c);
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  for (int i = 0; i < 2; ++i) {
    p.kn[i] = kn[i];
    p.vn[i] = vn[i];
  }
  p.cu = cu;
  p.T = T;
  p.check_blocks = (static_cast<unsigned>(c->B) + 31) / 32;
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  launch_move(c->cache_type == FDMA_CACHE_E4M3, c->d, c->Hkv, static_cast<unsigned>(blocks), p,
              static_cast<cudaStream_t>(stream), Append{});
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

int fdma_kv_gather(const fdma_kv_cache* c, const int32_t* cu, const int32_t* first, int T, void* k_out, void* v_out,
                   void* stream) {
  const int st = validate_cache(c);
  if (st != FDMA_OK) return st;
  if (T < 0) return FDMA_ERR_INVALID;
  if (T == 0 || c->B == 0) return FDMA_OK;
  if (cu == nullptr || k_out == nullptr || v_out == nullptr) return FDMA_ERR_INVALID;
  if (!aligned16(k_out) || !aligned16(v_out)) return FDMA_ERR_UNSUPPORTED;
  const int64_t blocks = move_blocks(T, c->Hkv, c->d);
  if (blocks > 0x1fffffff) return FDMA_ERR_UNSUPPORTED;
  MoveParams p{};
  p.c = cache_view(*c);
  p.cu = cu;
  p.first = first;
  p.T = T;
  p.check_blocks = (static_cast<unsigned>(c->B) + 31) / 32;
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  launch_move(c->cache_type == FDMA_CACHE_E4M3, c->d, c->Hkv, static_cast<unsigned>(blocks), p,
              static_cast<cudaStream_t>(stream), Gather{});
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

}  // extern "C"
