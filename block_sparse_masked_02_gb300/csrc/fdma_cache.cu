// Writing tokens into a paged key/value cache and reading sequences back.
//
// Both move rows of d values between packed tokens and cache slots and are bound by
// memory traffic (or, for a few tokens, by the latency of token -> sequence -> page ->
// row).  One warp serves one token and up to kHeadsPerWarp kv heads: the search for the
// token's sequence and its page is made once for all of them, lanes 0..15 then move the
// K rows and lanes 16..31 the V rows, eight values a lane, every row's load issued before
// the first is used.
//
// e4m3: with m = max |x| of a row, e is the least integer with m <= 448 * 2^e, taken from
// m's bits: 448 = 1.75 * 2^8, so e = E - 8 where m = f * 2^E has f <= 1.75 and E - 7
// otherwise.  x * 2^-e is exact, so each value is rounded once.
#include "fdma_paged.cuh"

namespace fdma {
namespace {

constexpr int kHeadsPerWarp = 4;
constexpr int kCacheThreads = 256;

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

// Byte offset of (page of position pos, slot in it) for strides st (page, token, head) and
// head g; pg: the page.
__device__ __forceinline__ int64_t slot_offset(const CacheView& c, const int64_t* st, int pg, int pos, int g) {
  return pg * st[0] + (pos & ((1 << c.page_shift) - 1)) * st[1] + g * st[2];
}

// Quantises eight values of a row whose 16 lanes hold it all; returns the codes, e + 127 in `be`.
__device__ __forceinline__ uint2 quantise8(uint4 x, uint32_t& be) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = 0;  // largest finite magnitude, as bf16 bits
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
    m = max(m, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  // m = (1 + mant / 128) * 2^(E - 127), 1.75 = 1 + 96 / 128 (bf16 subnormals fall to the clamp)
  const int E = static_cast<int>(m >> 7), up = (m & 0x7fu) > 96u ? 1 : 0;
  const int b = min(max(E - 8 + up, 1), 246);
  be = static_cast<uint32_t>(b);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);  // 2^-(b - 127)
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16) * inv, hi = __uint_as_float(w[i] & 0xffff0000u) * inv;
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    h[i] = r;
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ uint4 dequantise8(uint2 q, uint32_t be) {
  const float s = exp_scale(be);
  const uint32_t h[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t f = e4m3x2_to_f16x2(h[i]);
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(f));
    r[i] = pack_bf16x2(lo * s, hi * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool FP8>
__global__ void __launch_bounds__(kCacheThreads) kv_append_kernel(const MoveParams p) {
  const int lane = threadIdx.x & 31;
  const int groups = (p.c.Hkv + kHeadsPerWarp - 1) / kHeadsPerWarp;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kCacheThreads + threadIdx.x) >> 5;
  const int64_t tok = w / groups;
  if (tok >= p.T) return;
  const int t = static_cast<int>(tok), g0 = static_cast<int>(w % groups) * kHeadsPerWarp;
  const bool is_v = lane >= 16;
  const int col = (lane & 15) * 8;
  const bool in = col < p.c.d;
  // the rows themselves do not depend on the slot: load them while it is looked up
  const uint16_t* src = (is_v ? p.v_new : p.k_new) + t * (is_v ? p.vn[0] : p.kn[0]) + col;
  const int64_t sh = is_v ? p.vn[1] : p.kn[1];
  uint4 x[kHeadsPerWarp];
#pragma unroll
  for (int i = 0; i < kHeadsPerWarp; ++i) {
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (in && g0 + i < p.c.Hkv) x[i] = __ldg(reinterpret_cast<const uint4*>(src + (g0 + i) * sh));
  }
  const int b = find_seq(p.cu, p.c.B, t, lane);
  if (b < 0) return;  // behind the last sequence
  const int pos = p.c.k_len[b] - (p.cu[b + 1] - t);
  int pg = -1;
  if (pos >= 0 && (pos >> p.c.page_shift) < p.c.max_pages)
    pg = p.c.table[static_cast<int64_t>(b) * p.c.table_stride + (pos >> p.c.page_shift)];
  if (pg < 0 || pg >= p.c.num_pages) {
    if (lane == 0) atomicCAS(p.err, 0, FDMA_ERR_INVALID);
    return;
  }
  uint8_t* dst = const_cast<uint8_t*>(is_v ? p.c.v : p.c.k);
  const int64_t* st = is_v ? p.c.vs : p.c.ks;
#pragma unroll
  for (int i = 0; i < kHeadsPerWarp; ++i) {
    const int g = g0 + i;
    if (g >= p.c.Hkv) break;
    if (FP8) {
      uint32_t be;
      const uint2 q = quantise8(x[i], be);
      if (in) *reinterpret_cast<uint2*>(dst + slot_offset(p.c, st, pg, pos, g) + col) = q;
      if ((lane & 15) == 0)
        const_cast<uint8_t*>(is_v ? p.c.ve : p.c.ke)[slot_offset(p.c, is_v ? p.c.ves : p.c.kes, pg, pos, g)] =
            static_cast<uint8_t>(be);
    } else if (in) {
      *reinterpret_cast<uint4*>(dst + slot_offset(p.c, st, pg, pos, g) + col * 2) = x[i];
    }
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kCacheThreads) kv_gather_kernel(const MoveParams p) {
  const int lane = threadIdx.x & 31;
  const int groups = (p.c.Hkv + kHeadsPerWarp - 1) / kHeadsPerWarp;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kCacheThreads + threadIdx.x) >> 5;
  const int64_t tok = w / groups;
  if (tok >= p.T) return;
  const int t = static_cast<int>(tok), g0 = static_cast<int>(w % groups) * kHeadsPerWarp;
  const bool is_v = lane >= 16;
  const int col = (lane & 15) * 8;
  const int b = find_seq(p.cu, p.c.B, t, lane);
  if (b < 0) return;
  const int64_t pos64 = static_cast<int64_t>(p.first != nullptr ? p.first[b] : 0) + (t - p.cu[b]);
  const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.page_shift;
  const int kl = p.c.k_len[b];
  if ((kl < 0 || kl > cap) && lane == 0) atomicCAS(p.err, 0, FDMA_ERR_INVALID);
  int pg = -1;
  const int pos = static_cast<int>(pos64);
  if (pos64 >= 0 && pos64 < min(static_cast<int64_t>(kl), cap)) {
    pg = p.c.table[static_cast<int64_t>(b) * p.c.table_stride + (pos >> p.c.page_shift)];
    if (pg < 0 || pg >= p.c.num_pages) {
      if (lane == 0) atomicCAS(p.err, 0, FDMA_ERR_INVALID);
      pg = -1;
    }
  }
  if (col >= p.c.d) return;
  const uint8_t* src = is_v ? p.c.v : p.c.k;
  const uint8_t* ex = is_v ? p.c.ve : p.c.ke;
  const int64_t* st = is_v ? p.c.vs : p.c.ks;
  const int64_t* es = is_v ? p.c.ves : p.c.kes;
  uint16_t* dst = (is_v ? p.v_out : p.k_out) + (tok * p.c.Hkv + g0) * p.c.d + col;
  uint4 x[kHeadsPerWarp];
  uint32_t be[kHeadsPerWarp];
#pragma unroll
  for (int i = 0; i < kHeadsPerWarp; ++i) {
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    be[i] = 127;
    if (pg >= 0 && g0 + i < p.c.Hkv) {
      const uint8_t* a = src + slot_offset(p.c, st, pg, pos, g0 + i);
      if (FP8) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(a + col));
        x[i].x = q.x;
        x[i].y = q.y;
        be[i] = ex[slot_offset(p.c, es, pg, pos, g0 + i)];
      } else {
        x[i] = __ldg(reinterpret_cast<const uint4*>(a + col * 2));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kHeadsPerWarp; ++i) {
    if (g0 + i >= p.c.Hkv) break;
    *reinterpret_cast<uint4*>(dst + i * p.c.d) = FP8 ? dequantise8(make_uint2(x[i].x, x[i].y), be[i]) : x[i];
  }
}

int64_t move_blocks(int T, int Hkv) {
  const int64_t warps = static_cast<int64_t>(T) * ((Hkv + kHeadsPerWarp - 1) / kHeadsPerWarp);
  return (warps * 32 + kCacheThreads - 1) / kCacheThreads;
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
  const int64_t blocks = move_blocks(T, c->Hkv);
  if (blocks > 0x7fffffff) return FDMA_ERR_UNSUPPORTED;
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
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  auto kern = c->cache_type == FDMA_CACHE_E4M3 ? kv_append_kernel<true> : kv_append_kernel<false>;
  kern<<<static_cast<unsigned>(blocks), kCacheThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
  const int64_t blocks = move_blocks(T, c->Hkv);
  if (blocks > 0x7fffffff) return FDMA_ERR_UNSUPPORTED;
  MoveParams p{};
  p.c = cache_view(*c);
  p.cu = cu;
  p.first = first;
  p.T = T;
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  auto kern = c->cache_type == FDMA_CACHE_E4M3 ? kv_gather_kernel<true> : kv_gather_kernel<false>;
  kern<<<static_cast<unsigned>(blocks), kCacheThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

}  // extern "C"
