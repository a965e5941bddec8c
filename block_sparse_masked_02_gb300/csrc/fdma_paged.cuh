// What the kernels over a paged key/value cache share: their parameter block, the
// key tiles that a group of query rows sees, and the division of all those tiles
// into equal runs, one per CTA.
//
// An item is one (sequence, kv head, block of ROWS packed query rows); a packed row
// is (token, head of the group), the group's heads of one token next to each other,
// so that one token's heads share the keys that are fetched for them.  An item's key
// tiles are kKeyTile wide and aligned to multiples of it: first the tiles that hold
// visible sinks, then the tiles from the window's lower edge (or 0) to the last
// visible key.  All items' tiles, in the order (sequence, kv head, row block, tile),
// form one line that is cut into runs of equal length, one for each CTA: ragged
// batches, causal chunks and one very long sequence all load the machine evenly, and
// what is needed of the workspace does not depend on any length.  A CTA's run ends
// inside an item at most twice (its first item may have begun in an earlier CTA, its
// last may go on in the next ones); those pieces go to the workspace as fp32 sums with
// their running maximum and weight and are joined by a second kernel.
#pragma once

#include <atomic>

#include "../../include/fdma_paged.h"
#include "fdma_internal.h"
#include "fdma_ptx.cuh"

namespace fdma {

constexpr int kPagedCtas = 152;  // one CTA per SM
constexpr float kPLog2e = 1.4426950408889634f;
constexpr float kPLn2 = 0.6931471805599453f;

constexpr int kItemCost = 2;
constexpr int64_t kMaxRun = 1 << 30;  // places of a CTA's run (of a chunk: a quarter of an hour): more is refused

struct CacheView {
  const uint8_t* k;  // strides in bytes: page, token, head
  const uint8_t* v;
  int64_t ks[3], vs[3];
  const uint8_t* ke;
  const uint8_t* ve;
  int64_t kes[3], ves[3];
  const int32_t* table;
  int64_t table_stride;
  const int32_t* k_len;
  int B, Hkv, d, page_shift, num_pages, max_pages;
};

struct PagedParams {
  CacheView c;
  const uint16_t* q;
  int64_t q_t, q_h;  // elements
  const int32_t* cu;
  int T, max_q, Hq, G;
  int causal, window, sinks;
  float scale_log2;
  uint16_t* out;  // (T, Hq, d)
  float* lse;     // (Hq, T)
  float* part_o;  // [cta][2][ROWS][D]
  float2* part_ml;  // [cta][2][ROWS]: running maximum (log2 units) and weight sum
  int4* desc;     // [cta]: the split item that begins in this CTA: (sequence, kv head, row block, slot | pieces << 1)
  int* err;
  int min_run;  // least length of a run
  int plan_lanes;  // lanes that share a sequence when the line is laid out: a power of two, at most 32
  int box;      // chunk kernel: rows of a TMA box of the cache (0: no TMA)
};

// One sequence as the kernels use it: every value inside its bounds whatever the arrays hold.  Tokens that are left
// out (outside [0, T), behind max_q) do not move the others: packed token t stays at position
// k_len - (cu[b + 1] - t).  A sequence whose k_len is out of range has no rows.
struct Seq {
  int q0;    // first packed token
  int nq;    // new tokens
  int klen;  // keys, the new tokens among them
  int pos0;  // position of token q0 (negative: that row is before the first key); pos0 + nq <= klen
};

__device__ __forceinline__ Seq load_seq(const PagedParams& p, int b, bool report) {
  Seq s;
  const int a = p.cu[b], e = p.cu[b + 1], kl = p.c.k_len[b];
  const int cap = p.c.max_pages << p.c.page_shift;
  s.klen = min(max(kl, 0), cap);
  s.q0 = min(max(a, 0), p.T);
  s.nq = kl == s.klen ? min(max(min(e, p.T) - s.q0, 0), p.max_q) : 0;
  // (far below the first key, as far as a row's number reaches, is the same as further)
  s.pos0 = s.nq > 0 ? max(s.klen - (e - s.q0), -(1 << 30)) : 0;
  if (report && (a != s.q0 || e != s.q0 + s.nq || kl != s.klen)) atomicCAS(p.err, 0, FDMA_ERR_INVALID);
  return s;
}

struct Span {
  int lo, hi;   // visible to some row: keys lo .. hi-1 ...
  int sink_hi;  // ... and 0 .. sink_hi-1 (sink_hi <= lo)
  int sink_tiles, main0, tiles;
};

// Keys seen by the tokens [i0, i1) of a sequence (i1 > i0).
template <int KT>
__device__ __forceinline__ Span key_span(const PagedParams& p, const Seq& s, int i0, int i1) {
  Span r;
  const int first = max(s.pos0 + i0, 0);
  r.hi = p.causal ? max(s.pos0 + i1, 0) : s.klen;
  r.lo = p.window > 0 ? max(first - p.window + 1, 0) : 0;
  r.sink_hi = p.window > 0 ? min(p.sinks, r.lo) : 0;
  if (r.hi <= 0) {
    r.sink_tiles = r.main0 = r.tiles = 0;
    r.lo = r.hi = r.sink_hi = 0;
    return r;
  }
  r.sink_tiles = (r.sink_hi + KT - 1) / KT;
  r.main0 = max(r.lo / KT, r.sink_tiles);
  r.tiles = r.sink_tiles + (r.hi + KT - 1) / KT - r.main0;
  return r;
}

// The keys that the row at position pos sees: j < hi and (j >= lo or j < sinks).
struct RowKeys {
  int lo, hi;
};
__device__ __forceinline__ RowKeys row_keys(const PagedParams& p, const Seq& s, int pos) {
  RowKeys r;
  r.hi = p.causal ? pos + 1 : s.klen;
  r.lo = p.window > 0 ? pos - p.window + 1 : 0;
  return r;
}

// The tile of the span that holds key j, which some row sees.
template <int KT>
__device__ __forceinline__ int tile_of(int sink_tiles, int main0, int j) {
  const int t = j / KT;
  return t < sink_tiles ? t : t - main0 + sink_tiles;
}

// Position on the line of tiles.
template <int ROWS, int KT>
struct Cursor {
  int b, g, rt, t;
  int left;  // places of the run from this tile on
  Seq s;
  Span r;

  __device__ __forceinline__ void span(const PagedParams& p) {
    const int i0 = rt * ROWS / p.G, i1 = min((rt * ROWS + ROWS - 1) / p.G + 1, s.nq);
    r = key_span<KT>(p, s, i0, i1);
  }
  __device__ __forceinline__ int key0() const { return (t < r.sink_tiles ? t : r.main0 + (t - r.sink_tiles)) * KT; }
  __device__ __forceinline__ bool last_tile() const { return t + 1 == r.tiles; }
  // Places of the run that are left when the current tile is done (the tiles t .. t + n - 1 of the item).
  __device__ __forceinline__ int left_after(int n) const { return left - n - (t + n == r.tiles ? kItemCost : 0); }
  // The next tile of the line; the caller knows that the run goes on.
  __device__ __forceinline__ void next(const PagedParams& p) {
    if (++t < r.tiles) return;
    t = 0;
    for (;;) {
      if ((rt + 1) * ROWS < s.nq * p.G) {
        ++rt;
        span(p);
      } else {
        const bool had_one_block = rt == 0;
        rt = 0;
        if (g + 1 < p.c.Hkv) {
          ++g;
          if (!had_one_block) span(p);
        } else {
          g = 0;
          do {
            if (++b >= p.c.B) return;  // not reached while tiles are left
            s = load_seq(p, b, false);
          } while (s.nq == 0);
          span(p);
        }
      }
      if (r.tiles > 0) return;
    }
  }
};

// Places of the rt-th item of a kv head.
template <int ROWS, int KT>
__device__ __forceinline__ int item_places(const PagedParams& p, const Seq& s, int rt) {
  const int r0 = rt * ROWS;
  if (r0 >= s.nq * p.G) return 0;
  const int k = key_span<KT>(p, s, r0 / p.G, min((r0 + ROWS - 1) / p.G + 1, s.nq)).tiles;
  return k > 0 ? k + kItemCost : 0;
}

// a / b, a >= 0 and b > 0.  (A 64-bit division takes 400 cycles, and every CTA waits for these.)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

struct PlanSmem {
  int64_t warp_sum[32];
  int64_t total;
  int b, g, rt, t;
  Seq s;
};

// Finds this CTA's run: every thread of the CTA calls it (NT threads).  False where it has no
// tiles; else c stands on the first of them.  quota: the run length of all CTAs.
// A sequence's items are counted by plan_lanes lanes together (by one, a chunk's 16 to 32 row blocks took
// 6 us before the first load).  Places are counted in 64 bits: 1.5 million tokens of 64 heads on one kv head over
// themselves have 2^31.
template <int ROWS, int KT, int NT>
__device__ __forceinline__ bool plan_run(const PagedParams& p, PlanSmem* sm, Cursor<ROWS, KT>& c, int& quota) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, L = p.plan_lanes, sub = lane & (L - 1);
  const unsigned group = (L == 32 ? 0xffffffffu : (1u << L) - 1u) << (lane & -L);
  const int per = (p.c.B + NT / L - 1) / (NT / L);
  const int b0 = min(tid / L * per, p.c.B), b1 = min(b0 + per, p.c.B);
  // places of a kv head of a sequence, in every lane of the group
  auto seq_places = [&](const Seq& s) {
    int64_t n = 0;
    for (int rt = sub; rt * ROWS < s.nq * p.G; rt += L) n += item_places<ROWS, KT>(p, s, rt);
    for (int o = 1; o < L; o <<= 1) n += __shfl_xor_sync(group, n, o);
    return n;
  };
  int64_t mine = 0;
  Seq s{};  // the last one, and its places: usually a group has one sequence
  int64_t n = 0;
  for (int b = b0; b < b1; ++b) {
    s = load_seq(p, b, blockIdx.x == 0);
    n = seq_places(s);
    mine += n * p.c.Hkv;
  }
  __syncwarp();
  int64_t x = sub == 0 ? mine : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm->warp_sum[warp] = x;
  __syncthreads();
  int64_t before = x - mine, total = 0;  // (x holds the group's places in every lane of it)
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += sm->warp_sum[w];
    total += sm->warp_sum[w];
  }
  const int64_t run = max(quotient(total + kPagedCtas - 1, kPagedCtas), static_cast<int64_t>(p.min_run));
  if (run > kMaxRun) {
    if (blockIdx.x == 0 && tid == 0) atomicCAS(p.err, 0, FDMA_ERR_UNSUPPORTED);
    return false;
  }
  quota = static_cast<int>(run);
  const int64_t start = static_cast<int64_t>(blockIdx.x) * quota;
  if (start >= before && start < before + mine) {  // (one group of lanes)
    int64_t left = start - before;
    for (int b = b0; b < b1; ++b) {
      if (b1 - b0 > 1) {
        s = load_seq(p, b, false);
        n = seq_places(s);
      }
      if (left >= n * p.c.Hkv) {
        left -= n * p.c.Hkv;
        continue;
      }
      const int g = static_cast<int>(quotient(left, n));
      int64_t t = left - g * n;
      for (int rt = sub;; rt += L) {
        const int k = item_places<ROWS, KT>(p, s, rt);
        int64_t sum = k;
        for (int o = 1; o < L; o <<= 1) {
          const int64_t y = __shfl_up_sync(group, sum, o, L);
          if (sub >= o) sum += y;
        }
        if (t >= sum - k && t < sum) {
          sm->b = b;
          sm->g = g;
          sm->rt = rt;
          sm->t = static_cast<int>(t - (sum - k));
          sm->s = s;
        }
        const int64_t all = __shfl_sync(group, sum, L - 1, L);
        if (t < all) break;
        t -= all;
      }
      break;
    }
  }
  __syncthreads();
  if (start >= total) return false;
  c.b = sm->b;
  c.g = sm->g;
  c.rt = sm->rt;
  c.t = sm->t;
  c.s = sm->s;
  c.span(p);
  c.left = static_cast<int>(min(static_cast<int64_t>(quota), total - start));
  if (c.t >= c.r.tiles) {  // between two items: the run's tiles begin with the next
    c.left -= c.r.tiles + kItemCost - c.t;
    c.t = c.r.tiles - 1;
    if (c.left <= 0) return false;
    c.next(p);
  }
  return true;
}

// Rows that see no key at all because their row block has no tiles: out = 0, lse = -inf.
// Called by every thread of every CTA; the sequences are dealt out over the CTAs.
template <int ROWS>
__device__ __forceinline__ void write_empty_blocks(const PagedParams& p) {
  for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
    const Seq s = load_seq(p, b, false);
    if (p.causal ? s.pos0 >= 0 : s.klen > 0) continue;  // every row sees a key
    for (int r0 = 0; r0 < s.nq * p.G; r0 += ROWS) {
      const int i0 = r0 / p.G, i1 = min((r0 + ROWS - 1) / p.G + 1, s.nq);
      if (key_span<128>(p, s, i0, i1).tiles > 0) continue;
      const int r1 = min(r0 + ROWS, s.nq * p.G), nr = (r1 - r0) * p.c.Hkv, vec = p.c.d >> 3;
      for (int e = threadIdx.x; e < nr * vec; e += blockDim.x) {
        const int x = e / vec, r = r0 + x % (r1 - r0), h = x / (r1 - r0) * p.G + r % p.G, t = s.q0 + r / p.G;
        *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(t) * p.Hq + h) * p.c.d + (e % vec) * 8) =
            make_uint4(0u, 0u, 0u, 0u);
        if (e % vec == 0) p.lse[static_cast<int64_t>(h) * p.T + t] = -__int_as_float(0x7f800000);
      }
    }
  }
}

// The table's entry for key j: looked up a step ahead of its use, so nothing may depend on it yet.
__device__ __forceinline__ int table_entry(const PagedParams& p, int b, int j) {
  return p.c.table[static_cast<int64_t>(b) * p.c.table_stride + (j >> p.c.page_shift)];
}
constexpr int kNoKeys = -0x7fffffff - 1;  // in place of an entry that is not needed

// The page that an entry names, or -1 where it names none (reported) or is not needed.
__device__ __forceinline__ int checked_page(const PagedParams& p, int entry) {
  if (entry >= 0 && entry < p.c.num_pages) return entry;
  if (entry != kNoKeys) atomicCAS(p.err, 0, FDMA_ERR_INVALID);
  return -1;
}

__device__ __forceinline__ float paged_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A scale byte as it counts: what no append writes (0, 247 to 255) as the nearest that one does.  So every value is
// finite in bf16, and in a product with a weight of 0 adds nothing.
__device__ __forceinline__ uint32_t scale_byte(uint32_t e) { return min(max(e, 1u), 246u); }
// 2^(e - 127) of a scale byte
__device__ __forceinline__ float exp_scale(uint32_t e) { return __uint_as_float(e == 0 ? 0x00400000u : e << 23); }

// Four e4m3 codes (low byte first) as f16, exact (NaN stays NaN).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// ---- Values that are not finite, in keys that only some rows of a block see.  In the product with
// V their weight 0 would still make the other rows NaN, so they are set to zero in shared memory, and
// at the end of the item the rows that do see them add them (a weight is positive, so an infinity
// or NaN is all that is left of the sum).  A CTA adds those of its own tiles only: its sums enter the
// join with the weight of the keys it saw, which is 0 where a row saw none of them.

// Clears what is not finite in two bf16.
__device__ __forceinline__ void clear_odd_bf16x2(uint32_t& w) {
  uint32_t keep = 0xffffffffu;
  if ((w & 0x7f80u) == 0x7f80u) keep &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) keep &= 0x0000ffffu;
  w &= keep;
}
// Clears NaN codes (0x7f, 0xff) in four e4m3.
__device__ __forceinline__ void clear_odd_e4m3x4(uint32_t& w) {
  w &= ~(((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu);
}

// The rest of it is out of line: in line, what hardly ever runs pushed the loops out of the
// instruction cache (a 2048-token chunk took 205 instead of 185 us).

// Which keys of an item somebody sees (j < sink_hi, or lo <= j < hi), and which everybody
// (j < all_hi, and j >= all_lo or j < sinks).
struct SeenKeys {
  int lo, hi, sink_hi, all_lo, all_hi, sinks;
};

// Clears them in `count` (a multiple of N) 16-byte pieces of shared memory, `step` bytes and `dj` keys
// apart, of keys that not every row sees, and zeroes those of keys that no row sees; true if values
// were cleared that some row sees.
template <bool FP8, int N = 4>
__device__ __forceinline__ bool mend_pieces(uint32_t at, int step, int count, int j, int dj, const SeenKeys s) {
  bool found = false;
#pragma unroll 1
  for (int i = 0; i < count; i += N, at += N * step, j += N * dj) {
    uint32_t v[N][4], sum[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v[e][0]), "=r"(v[e][1]), "=r"(v[e][2]), "=r"(v[e][3])
                   : "r"(at + e * step)
                   : "memory");
    }
    uint32_t any = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      sum[e] = 0;
      // an exponent (a code) of all ones carries into the sign bit's place
#pragma unroll
      for (int w = 0; w < 4; ++w)
        sum[e] |= FP8 ? (v[e][w] & 0x7f7f7f7fu) + 0x01010101u : (v[e][w] & 0x7f807f80u) + 0x00800080u;
      sum[e] &= FP8 ? 0x80808080u : 0x80008000u;
      const int k = j + e * dj;
      if (k < s.all_hi && (k >= s.all_lo || k < s.sinks)) sum[e] = 0;
      if (!(k < s.sink_hi || (k >= s.lo && k < s.hi))) {
        v[e][0] = v[e][1] = v[e][2] = v[e][3] = 0u;
        sum[e] = 1;
      }
      any |= sum[e];
    }
    if (any == 0) continue;
    found |= any > 1u;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (sum[e] == 0) continue;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (FP8) clear_odd_e4m3x4(v[e][w]);
        else clear_odd_bf16x2(v[e][w]);
      }
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + e * step), "r"(v[e][0]), "r"(v[e][1]), "r"(v[e][2]),
                   "r"(v[e][3])
                   : "memory");
    }
  }
  return found;
}

template <bool FP8, int N = 4>
__device__ __noinline__ bool mend_pieces_apart(uint32_t at, int step, int count, int j, int dj, const SeenKeys s) {
  return mend_pieces<FP8, N>(at, step, count, j, dj, s);
}

// What a row adds: keys lo .. hi-1 but those between mid and from, in the tiles t0 .. t1 of KT keys.
struct OddKeys {
  int b, g, lo, mid, from, hi, sink_tiles, main0, t0, t1;
};

// Adds the values that are not finite of the keys that a row (rlo, rhi) sees to columns
// col .. col + n - 1 of its result: bf16 at out, or (out NULL) fp32 at part, column c at
// part[(c / 4) * part_step + c % 4].
template <bool FP8, int KT>
__device__ __noinline__ void add_odd_values(const PagedParams& p, const OddKeys& k, int rlo, int rhi, int col, int n,
                                            uint16_t* out, float* part, int64_t part_step) {
#pragma unroll 1
  for (int j = k.lo < k.mid ? k.lo : k.from; j < k.hi; j = j + 1 == k.mid ? k.from : j + 1) {
    const int t = tile_of<KT>(k.sink_tiles, k.main0, j);
    if (t < k.t0 || t > k.t1 || !(j < rhi && (j >= rlo || j < p.sinks))) continue;
    const int pg = table_entry(p, k.b, j);
    if (pg < 0 || pg >= p.c.num_pages) continue;
    const uint8_t* src = p.c.v + pg * p.c.vs[0] + static_cast<int64_t>(j & ((1 << p.c.page_shift) - 1)) * p.c.vs[1] +
                         k.g * p.c.vs[2];
#pragma unroll 1
    for (int c = col; c < min(col + n, p.c.d); ++c) {
      const uint32_t w = FP8 ? ((src[c] & 0x7fu) == 0x7fu ? 0x7fc0u : 0u) : reinterpret_cast<const uint16_t*>(src)[c];
      if ((w & 0x7f80u) != 0x7f80u) continue;
      const float v = __uint_as_float(w << 16);
      if (out != nullptr) out[c] = static_cast<uint16_t>(pack_bf16x2(__uint_as_float(out[c] << 16) + v, 0.f));
      else part[(c >> 2) * part_step + (c & 3)] += v;
    }
  }
}

// cp.async of 16 bytes; src_bytes 0 fills with zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

int validate_cache(const fdma_kv_cache* c);
CacheView cache_view(const fdma_kv_cache& c);
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Lets a kernel use smem_bytes of shared memory on the current device and checks that it was compiled
// with at least min_regs registers; done once for each kernel and device (bit `device` of ready).
template <typename K>
inline cudaError_t set_up_once(std::atomic<uint64_t>& ready, K* kern, int smem_bytes, int min_regs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (ready.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs < min_regs) return cudaErrorInvalidConfiguration;
  ready.fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

// Attention kernels: the token kernel with its join, and the chunk kernel without.
constexpr int kChunkItemRows = 256;
cudaError_t launch_paged_token(bool fp8, const PagedParams& p, cudaStream_t stream);
cudaError_t launch_paged_chunk(bool fp8, const PagedParams& p, cudaStream_t stream);

}  // namespace fdma
