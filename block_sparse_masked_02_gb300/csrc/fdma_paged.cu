// Attention of few new tokens a sequence (decoding, a handful of drafted tokens) over a
// paged cache, and the host side of fdma_paged_fwd.
//
// An item is a kv head's query rows of one sequence, at most 8 * NT of them.  Every key and
// value is read from HBM once and takes part in 4 * d flops a row, so with few rows the kernel
// is bound by memory, and its work is to keep enough loads in flight with few instructions:
// each warp of the one CTA on an SM runs its own ring of cp.async stages of 16 or 32 keys' K and V
// rows (192 KB on an SM at d = 128), with no barrier between warps inside the loop, and the
// ring runs on across items, so that a batch of short sequences streams like one long one.
// page_size is a multiple of 16, so a group of 16 keys lies in one page.  32 sequences of 257 to 8191 keys,
// 8 kv heads of 128, bf16, a token each: a call of 97 us, 5.7 TB/s of keys and values, 84 % of a plain copy's rate.
//
// Each warp keeps its own running maximum, weight sum and output for its keys (online
// softmax), and they are joined at the end of the item.  The products are mma.sync with the
// keys (then the head dim) as the 16 rows of A and eight query rows as the columns of B:
//   S^T = K Q^T,    O^T += V^T P^T,
// so eight rows, the usual group of one token, waste nothing; P^T becomes the B operand by one
// 8 x 8 transpose of 16-bit values in registers.  At so few rows the tensor pipe is idle most of
// the time whichever instruction feeds it, and this one takes K and V as they lie in shared
// memory.
//
// e4m3 caches: codes become f16 exactly (one conversion for two), so the products run in f16.
// q is scaled by a power of two per row to [2^14, 2^15), which is exact but for parts below
// 2^-31 of the row's largest (f16's least step, 2^-24, is 2^-38 of 2^14, and a bf16 number has eight bits).  The key's scale multiplies S; the value's scale multiplies P,
// as 2^(e - r + 15) with r the largest e so far of the keys that the row sees (its output is kept in
// units of 2^(r - 15)), so that P stays in f16's range: a weight keeps 11 bits, or 2^(r - e - 40) where
// that is more, at most 2^-24 because e and r are at most 16 apart.  A row that sees scales further
// apart ("wide") goes on in fp32 products of its own, in units of 1: with f16 weights a large value would
// take the weights of all others away, in columns where it is 0 and where its own weight is 0 too.
// What a row gets so depends on the keys that it sees alone.  Value rows of zeros do not make it wide.
// (A unit for each row instead of one for a warp: 26.1 against 24.8 us for a token over two sequences of 65 thousand keys, 58.6
// against 54.1 for 16 rows of 16 sequences of 4096 keys, 8 kv heads; the first case with all rows wide: 81 us.)
// A key is half the bytes and has the conversions on top, so a warp takes 32 keys a step: two
// independent chains of products and half the bookkeeping a key.
#include <cmath>

#include <cuda_fp16.h>

#include "fdma_paged.cuh"

namespace fdma {

namespace {

// Packed rows up to which the token kernel runs.  With 17 to 24 rows (8 kv heads, d 128) of 16
// sequences of 4096 keys it took 69 us and the chunk kernel 59 (e4m3: 81 and 73; of one sequence of
// 32768 keys 41 and 40, e4m3 42 and 42), with 9 to 16 rows 57 and 59 (e4m3 59 and 73).
constexpr int kTokenRows = 16;
constexpr float kNInf = -__builtin_huge_valf();
constexpr float kMostF = 3.402823466e38f;  // the largest fp32 number
constexpr int kNarrow = 16;  // value scales of an f16 row are at most 2^16 apart

// The largest value scale byte that a row has seen in the low half, 255 less the least one in the high half (0: none):
// both grow, so a maximum by halves takes more keys in.
__device__ __forceinline__ uint32_t scale_span(uint32_t most, uint32_t least) { return most | (255u - least) << 16; }
__device__ __forceinline__ bool wide_span(uint32_t s) { return (s & 0xffffu) + (s >> 16) > 255u + kNarrow; }

// (The following two hardly ever run: out of line, so that the loop stays in the instruction cache.)
// True if the `pieces` 16-byte pieces of codes at `at` are zeros.
__device__ __noinline__ bool zero_row(uint32_t at, int pieces) {
  uint32_t any = 0;
#pragma unroll 1
  for (int c = 0; c < pieces; ++c) {
    uint32_t x, y, z, w;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x), "=r"(y), "=r"(z), "=r"(w) : "r"(at + c * 16) : "memory");
    any |= x | y | z | w;
  }
  return (any & 0x7f7f7f7fu) == 0;
}
// Of 32 keys' scale bytes, those that a row with these first and last keys sees, but for those in `none`.  The
// eight lanes of a row (lane & 3 the same) call it together.
__device__ __noinline__ uint32_t seen_span(const uint8_t* bytes, int first, int end, int sinks, unsigned none) {
  uint32_t x = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = static_cast<int>(lane_id() >> 2) + 8 * i;
    const uint32_t b = bytes[k];
    if (b != 0 && !((none >> k) & 1u) && k < end && (k >= first || k < sinks)) x = __vmaxu2(x, scale_span(b, b));
  }
#pragma unroll
  for (int i = 4; i < 32; i <<= 1) x = __vmaxu2(x, __shfl_xor_sync(0xffffffffu, x, i));
  return x;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Over the eight lanes that hold a query row (lane & 3 the same).
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// The 8 x 8 matrix of 16-bit values that the warp holds as (row lane / 4, columns 2 * (lane & 3) + {0, 1}),
// transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// D: 64 or 128, the head dim's padded width (columns past d are read as zeros); NT: eights of rows.
template <int D, bool FP8, int NT>
struct TokCfg {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kGroups = FP8 ? 2 : 1;       // 16-key groups of a warp's step
  static constexpr int kStep = 16 * kGroups;        // keys of a warp's step
  static constexpr int kKeys = kWarps * kStep;      // keys of a tile
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowB = FP8 ? D : 2 * D;     // bytes of a row in shared memory
  static constexpr int kHalfB = kStep * kRowB;      // a step's K (or V)
  static constexpr int kStages = kHalfB == 4096 ? 3 : 5;
  static constexpr int kWarpB = kStages * 2 * kHalfB;
  // columns joined at a time: [kWarps][kRows][kCols] fp32 within 32 KB
  static constexpr int kFit = 32768 / (kWarps * kRows * 4);
  static constexpr int kCols = kFit >= D ? D : kFit >= 64 ? 64 : 32;
  static constexpr int kOffMerge = kWarps * kWarpB;
  static constexpr int kOffMl = kOffMerge + kWarps * kRows * kCols * 4;  // [kWarps][kRows] (maximum, sum)
  static constexpr int kOffExp = kOffMl + kWarps * kRows * 8;            // [kWarps][kStages][2][kStep] scale bytes (e4m3)
  static constexpr int kOffPlan = kOffExp + (FP8 ? kWarps * kStages * 2 * kStep : 0);
  static constexpr int kTotal = kOffPlan + static_cast<int>(sizeof(PlanSmem));
  static_assert(kTotal <= 232448, "shared memory of one CTA");
};

// Byte offset of 16-byte chunk c of key row r: the chunks of a row are exchanged so that the
// eight rows of an ldmatrix (and the 32 lanes of the e4m3 key reads) touch different banks.
template <int ROWB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return r * ROWB + ((ROWB == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7)) << 4);
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(TokCfg<D, FP8, NT>::kThreads, 1)
    paged_token_kernel(const __grid_constant__ PagedParams p) {
  using L = TokCfg<D, FP8, NT>;
  constexpr int ROWS = L::kRows, NST = L::kStages, ROWB = L::kRowB, W = L::kWarps, KG = L::kGroups, STEP = L::kStep;
  constexpr int CPR = ROWB / 16;  // 16-byte chunks of a row
  constexpr int RPP = 32 / CPR;   // rows that a warp copies at a time
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q4 = lane & 3, n8 = lane >> 2;
  PlanSmem* plan = reinterpret_cast<PlanSmem*>(smem + L::kOffPlan);
  float* merge = reinterpret_cast<float*>(smem + L::kOffMerge);
  float2* sml = reinterpret_cast<float2*>(smem + L::kOffMl);
  uint8_t* sexp = smem + L::kOffExp + warp * NST * 2 * STEP;
  const uint32_t ring = smem_u32(smem) + warp * L::kWarpB;

  Cursor<ROWS, L::kKeys> lc;  // the tile that is loaded next
  int quota;
  const bool any = plan_run<ROWS, L::kKeys, L::kThreads>(p, plan, lc, quota);
  if (tid == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  write_empty_blocks<ROWS>(p);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up; it waits for the end
  if (!any) return;
  Cursor<ROWS, L::kKeys> cc = lc;  // the tile that is computed next

  // ---- loads: stage (x mod NST) of this warp's ring takes its step's keys of tile x
  const int chunk = lane % CPR, crow = lane / CPR;
  const uint32_t cbytes = chunk * 16 < p.c.d * (FP8 ? 1 : 2) ? 16u : 0u;
  const int pmask = (1 << p.c.page_shift) - 1;
  uint32_t exp_pend[2] = {127, 127};
  bool seen_pend = false;
  auto some_seen = [&](const Span& r, int j0, int n) { return j0 < r.sink_hi || (j0 < r.hi && j0 + n > r.lo); };
  // a group's page is looked up (a step ahead) only where some row sees one of its keys
  int lentry[KG];
  auto look_up = [&]() {
#pragma unroll
    for (int g = 0; g < KG; ++g) {
      const int j0 = lc.key0() + warp * STEP + g * 16;
      lentry[g] = some_seen(lc.r, j0, 16) ? table_entry(p, lc.b, j0) : kNoKeys;
    }
  };
  look_up();
  int lstage = 0;
  bool more = true, pending = false;  // tiles to load; scale bytes still in registers
  auto load_next = [&]() {
    if (FP8 && pending) {
      uint8_t* e = sexp + (lstage == 0 ? NST - 1 : lstage - 1) * 2 * STEP;
      // (not when they are loaded: nothing may wait for them there)
      e[lane] = static_cast<uint8_t>(scale_byte(exp_pend[0]));
      e[STEP + lane] = static_cast<uint8_t>(seen_pend ? scale_byte(exp_pend[1]) : 0u);
    }
    pending = more;
    if (more) {
      const int js = lc.key0() + warp * STEP;
      int pgs[KG];
#pragma unroll
      for (int g = 0; g < KG; ++g) pgs[g] = checked_page(p, lentry[g]);
      if (some_seen(lc.r, js, STEP)) {
#pragma unroll
        for (int g = 0; g < KG; ++g) {
          const int j0 = js + g * 16;
          const int64_t pg = pgs[g];
          const uint32_t dst = ring + lstage * 2 * L::kHalfB;
          const uint8_t* kb = p.c.k + pg * p.c.ks[0] + ((j0 & pmask) + crow) * p.c.ks[1] + lc.g * p.c.ks[2] + chunk * 16;
          const uint8_t* vb = p.c.v + pg * p.c.vs[0] + ((j0 & pmask) + crow) * p.c.vs[1] + lc.g * p.c.vs[2] + chunk * 16;
          if (pg >= 0 && j0 >= lc.r.lo && j0 + 16 <= lc.r.hi) {  // all 16 keys
#pragma unroll
            for (int i = 0; i < 16 / RPP; ++i) {
              const uint32_t at = swz<ROWB>(g * 16 + i * RPP + crow, chunk);
              cp_async16(dst + at, kb, cbytes);
              cp_async16(dst + L::kHalfB + at, vb, cbytes);
              kb += RPP * p.c.ks[1];
              vb += RPP * p.c.vs[1];
            }
          } else {  // some, or none (zeros)
#pragma unroll 1
            for (int i = 0; i < 16 / RPP; ++i) {
              const int j = j0 + i * RPP + crow;
              const uint32_t at = swz<ROWB>(g * 16 + i * RPP + crow, chunk);
              const bool ok = pg >= 0 && (j < lc.r.sink_hi || (j >= lc.r.lo && j < lc.r.hi));
              cp_async16(dst + at, ok ? kb : p.c.k, ok ? cbytes : 0u);
              cp_async16(dst + L::kHalfB + at, ok ? vb : p.c.v, ok ? cbytes : 0u);
              kb += RPP * p.c.ks[1];
              vb += RPP * p.c.vs[1];
            }
          }
        }
      }
      if (FP8) {  // (a step has a lane for each of its keys)
        const int j = js + lane;
        const int64_t pg = lane < 16 ? pgs[0] : pgs[KG - 1];
        exp_pend[0] = exp_pend[1] = 0;
        seen_pend = false;
        if (pg >= 0 && (j < lc.r.sink_hi || (j >= lc.r.lo && j < lc.r.hi))) {
          exp_pend[0] = p.c.ke[pg * p.c.kes[0] + (j & pmask) * p.c.kes[1] + lc.g * p.c.kes[2]];
          exp_pend[1] = p.c.ve[pg * p.c.ves[0] + (j & pmask) * p.c.ves[1] + lc.g * p.c.ves[2]];
          seen_pend = true;
        }
      }
      lstage = lstage + 1 == NST ? 0 : lstage + 1;
      lc.left = lc.left_after(1);
      more = lc.left > 0;
      if (more) {
        lc.next(p);
        look_up();
      }
    }
    cp_async_commit();
  };

  uint32_t qf[NT][D / 16][2];  // Q^T as B operands: rows n8 of each eight
  float rowfac[NT][2];         // of rows 2 * q4 + {0, 1}: log2(e) * scale; e4m3: what undoes the row's power of two
  int rlo[NT][2], rhi[NT][2];  // their keys
  float o[NT][D / 16][4];      // O^T: head dim n8 (+ 8; e4m3: 2 * n8 + {0, 1}) of each 16, rows 2 * q4 + {0, 1}
  float m[NT][2], l[NT][2];
  int full_lo = 0, full_hi = 0;  // keys that every row sees
  bool any_wide = false;         // e4m3: some row of the warp is wide
  uint32_t span[NT][2];          // e4m3: value scales of the keys that the row has seen (scale_span)
  int seg0 = 0;                  // tile of the item at which this CTA began
  int stage = 0;
  bool first_seg = true, begin = true;
  bool odd = false;  // this warp cleared values that are not finite

  // (the first NST - 1 turns only load: the item's query rows come in at the same time)
#pragma unroll 1
  for (int x = 1 - NST;; ++x) {
    if (begin) {
      // ---- a new item: its query rows, and an empty softmax
      begin = false;
      seg0 = cc.t;
      const int rows = cc.s.nq * p.G - cc.rt * ROWS;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int pr = nt * 8 + n8, R = cc.rt * ROWS + pr;
        const bool in = pr < rows;
        const int i = in ? R / p.G : 0;
        const uint16_t* src = p.q + (cc.s.q0 + i) * p.q_t + (cc.g * p.G + (in ? R - i * p.G : 0)) * p.q_h;
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // the pair's columns: with e4m3 a lane's key bytes are D / 4 adjacent ones, so the
            // order of the columns inside the product is that of those bytes
            const int col = FP8 ? q4 * (D / 4) + s * 4 + e * 2 : s * 16 + e * 8 + q4 * 2;
            const uint32_t w = in && col < p.c.d ? __ldg(reinterpret_cast<const uint32_t*>(src + col)) : 0u;
            qf[nt][s][e] = w;
            top = max(top, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
          }
        float fac = p.scale_log2;
        if (FP8) {
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // q * 2^up has its largest part in [2^14, 2^15) (below, where that is subnormal)
          const int E = static_cast<int>(top >> 7);
          const int up = E == 255 ? 0 : 14 + 127 - max(E, 1);
          const float f1 = __uint_as_float(static_cast<uint32_t>(127 + up / 2) << 23);
          const float f2 = __uint_as_float(static_cast<uint32_t>(127 + up - up / 2) << 23);
          fac = 1.f / f1 / f2;
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t w = qf[nt][s][e];
              qf[nt][s][e] =
                  pack_f16x2(__uint_as_float(w << 16) * f1 * f2, __uint_as_float(w & 0xffff0000u) * f1 * f2);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // (row 2 * q4 + e of this eight is row n8 of lane 4 * (2 * q4 + e))
          rowfac[nt][e] = FP8 ? __shfl_sync(0xffffffffu, fac, 4 * (2 * q4 + e)) : fac;
          const int pe = nt * 8 + 2 * q4 + e, Re = cc.rt * ROWS + pe;
          // (a row past the last is treated like the last: nothing is stored for it)
          const RowKeys rk = row_keys(p, cc.s, cc.s.pos0 + (pe < rows ? Re / p.G : cc.s.nq - 1));
          rlo[nt][e] = rk.lo;
          rhi[nt][e] = rk.hi;
          m[nt][e] = kNInf;
          l[nt][e] = 0.f;
          span[nt][e] = 0;
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][c][e] = 0.f;
      }
      {
        const int i0 = cc.rt * ROWS / p.G, i1 = min((cc.rt * ROWS + ROWS - 1) / p.G, cc.s.nq - 1);
        full_hi = row_keys(p, cc.s, cc.s.pos0 + i0).hi;
        full_lo = row_keys(p, cc.s, cc.s.pos0 + i1).lo;
      }
      odd = any_wide = false;
    }
    if (x >= 0) cp_async_wait<NST - 2>();
    __syncwarp();
    load_next();
    if (x < 0) continue;

    const int j0 = cc.key0() + warp * STEP;
    if (some_seen(cc.r, j0, STEP)) {
      const uint32_t sk = ring + stage * 2 * L::kHalfB, sv = sk + L::kHalfB;
      const bool masked = j0 < full_lo || j0 + STEP > full_hi;
      // ---- S^T = K Q^T: keys j0 + 16 * g + n8 (+ 8), rows 2 * q4 + {0, 1} of each eight
      float s[KG][NT][4];
#pragma unroll
      for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[g][nt][e] = 0.f;
      if (FP8) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int g = 0; g < KG; ++g) {
            const uint4 wa = lds128(sk + swz<ROWB>(g * 16 + n8, q4 * (D / 64) + c));
            const uint4 wb = lds128(sk + swz<ROWB>(g * 16 + n8 + 8, q4 * (D / 64) + c));
            const uint32_t aw[4] = {wa.x, wa.y, wa.z, wa.w}, bw[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t a[4];
              e4m3x4_to_f16x4(aw[e], a[0], a[2]);
              e4m3x4_to_f16x4(bw[e], a[1], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<true>(s[g][nt], a, qf[nt][c * 4 + e][0], qf[nt][c * 4 + e][1]);
            }
          }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int g = 0; g < KG; ++g) {
            uint32_t a[4];
            ldsm4(a, sk + swz<ROWB>(g * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * ks + (lane >> 4)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(s[g][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
          }
      }
      float kf[KG][2];    // scales of keys n8, n8 + 8 of each group
      uint32_t vx[KG][2];  // and their values' scale bytes (0: not there, or a row of zeros)
      const uint8_t* ex = sexp + stage * 2 * STEP;
      float grow[NT][2];   // what the output's unit changes by
      bool plain = false;  // every key is there and no larger than any row's unit, no row is wide
      if (FP8) {
        uint32_t ve = ex[STEP + lane];
        uint32_t least = __reduce_min_sync(0xffffffffu, ve);
        plain = least > 1;
        if (least <= 1) {  // 1: what rows of zeros are written with, which never count
          if (ve == 1 && zero_row(sv + lane * ROWB, CPR)) sexp[stage * 2 * STEP + STEP + lane] = static_cast<uint8_t>(ve = 0);
          __syncwarp();
          least = __reduce_min_sync(0xffffffffu, ve != 0 ? ve : 255u);
        }
        const uint32_t step_span = scale_span(__reduce_max_sync(0xffffffffu, ve), least);
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            kf[g][e] = exp_scale(ex[g * 16 + n8 + 8 * e]) * p.scale_log2;
            vx[g][e] = ex[STEP + g * 16 + n8 + 8 * e];
          }
        bool grows = false, widens = false;
        uint32_t now[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            now[nt][r] = __vmaxu2(span[nt][r], step_span);
            grows |= now[nt][r] != span[nt][r];
            widens |= wide_span(now[nt][r]);
            grow[nt][r] = 1.f;
          }
        if (__any_sync(0xffffffffu, grows)) {
          // A row's keys have the step's span where those that every row sees have it.  (Keys that a single token does
          // not see are not there.)
          if (masked && cc.s.nq > 1) {
            const int j = j0 + lane;
            if (!(j < full_hi && (j >= full_lo || j < p.sinks))) ve = 0;
            widens |= step_span != scale_span(__reduce_max_sync(0xffffffffu, ve),
                                              __reduce_min_sync(0xffffffffu, ve != 0 ? ve : 255u));
          }
          if (__builtin_expect(!__any_sync(0xffffffffu, widens), 1)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int r = 0; r < 2; ++r) {  // the output's unit grows
                const int up = static_cast<int>((now[nt][r] & 0xffffu) - (span[nt][r] & 0xffffu));
                grow[nt][r] = __uint_as_float(static_cast<uint32_t>(127 - min(up, 127)) << 23);
                span[nt][r] = now[nt][r];
              }
          } else {
            unsigned none = 0;
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
              widens = false;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const uint32_t x = seen_span(ex + STEP, rlo[nt][r] - j0, rhi[nt][r] - j0, p.sinks - j0, none);
                  if (pass == 0 || (wide_span(now[nt][r]) && !wide_span(span[nt][r])))
                    now[nt][r] = __vmaxu2(span[nt][r], x);
                  widens |= wide_span(now[nt][r]) && !wide_span(span[nt][r]);
                }
              // (rows of zeros with any other scale make no row wide)
              if (pass == 1 || !__any_sync(0xffffffffu, widens)) break;
              none = __ballot_sync(0xffffffffu, zero_row(sv + lane * ROWB, CPR));
            }
            bool wide = false, over = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                // the output's unit grows, or becomes 1 (two factors: 2^-141 is not a normal number)
                const uint32_t old = span[nt][r], to = now[nt][r];
                const int up = static_cast<int>(old & 0xffffu) - (wide_span(to) ? 142 : static_cast<int>(to & 0xffffu));
                const int x = wide_span(old) ? 0 : max(up, -200);
                grow[nt][r] = __uint_as_float((127 + x / 2) << 23) * __uint_as_float((127 + x - x / 2) << 23);
                span[nt][r] = to;
                wide |= wide_span(to);
                over |= __vmaxu2(to, step_span) != to;  // unseen keys, rows of zeros that did not count
              }
            any_wide = __any_sync(0xffffffffu, wide);
            plain &= !__any_sync(0xffffffffu, over);
          }
        }
        plain &= !any_wide;
      }
      uint32_t up[NT][2];
      if (FP8) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) up[nt][r] = (142u - (span[nt][r] & 0xffffu)) << 23;
      }
      // ---- softmax of these keys
      uint32_t pb[KG][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float alpha[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // row 2 * q4 + r
          float mx = kNInf;
#pragma unroll
          for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // (e4m3: the two factors first, as either alone may take the sum out of fp32's range; together they are too
              // large only where the score is at least 2^95, or 0)
              float u = s[g][nt][2 * e + r] * (FP8 ? fminf(kf[g][e] * rowfac[nt][r], kMostF) : rowfac[nt][r]);
              if (masked) {
                const int j = j0 + g * 16 + n8 + 8 * e;
                if (!(j < rhi[nt][r] && (j >= rlo[nt][r] || j < p.sinks))) u = kNInf;
              }
              s[g][nt][2 * e + r] = u;
              mx = fmaxf(mx, u);
            }
          mx = fmaxf(m[nt][r], row_max(mx));
          const float base = mx == kNInf ? 0.f : mx;
          alpha[r] = paged_ex2(m[nt][r] - base);
          m[nt][r] = mx;
          float sum = 0.f;
#pragma unroll
          for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float w = paged_ex2(s[g][nt][2 * e + r] - base);
              sum += w;
              s[g][nt][2 * e + r] = w;
            }
          l[nt][r] = l[nt][r] * alpha[r] + sum;
          if (FP8) alpha[r] *= grow[nt][r];
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            o[nt][c][0] *= alpha[0];
            o[nt][c][1] *= alpha[1];
            o[nt][c][2] *= alpha[0];
            o[nt][c][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float a = s[g][nt][2 * h], b = s[g][nt][2 * h + 1];
            if (FP8) {  // times 2^(e - r + 15), at most 2^15
              const uint32_t e = vx[g][h] << 23;
              a *= __uint_as_float(e + up[nt][0]);
              b *= __uint_as_float(e + up[nt][1]);
            }
            pb[g][nt][h] = FP8 ? pack_f16x2(a, b) : transpose8(pack_bf16x2(a, b));
          }
      }
      if (FP8) {
        if (!plain) {  // (keys that a row does not see have weight 0 and any scale, rows of zeros any scale too)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int g = 0; g < KG; ++g)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float f[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const int e = static_cast<int>(vx[g][h]) + 142 - static_cast<int>(span[nt][r] & 0xffffu);
                  f[r] = wide_span(span[nt][r]) ? 0.f : __uint_as_float(static_cast<uint32_t>(min(max(e, 0), 142)) << 23);
                }
                pb[g][nt][h] = pack_f16x2(s[g][nt][2 * h] * f[0], s[g][nt][2 * h + 1] * f[1]);
              }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) pb[g][nt][h] = transpose8(pb[g][nt][h]);
      }
      if (FP8 && any_wide) {
        // ---- the wide rows' part of O: weights, scales and products in fp32, key by key (of weight 0: not
        // seen, where some keys are not; their values may be NaN here)
#pragma unroll 1
        for (int k = 0; k < STEP; ++k) {
          const float sc = exp_scale(ex[STEP + k]);
          float wr[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float a = k & 8 ? s[0][nt][2 + r] : s[0][nt][r], b = k & 8 ? s[KG - 1][nt][2 + r] : s[KG - 1][nt][r];
              wr[nt][r] = __shfl_sync(0xffffffffu, k & 16 ? b : a, (k & 7) * 4 + q4);
              if (!wide_span(span[nt][r])) wr[nt][r] = 0.f;
            }
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint16_t code;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(code) : "r"(sv + swz<ROWB>(k, c) + 2 * n8) : "memory");
            uint32_t f16, none;
            e4m3x4_to_f16x4(code, f16, none);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f16));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const bool skip = masked && wr[nt][r] == 0.f;
                o[nt][c][r] += skip ? 0.f : wr[nt][r] * (v.x * sc);
                o[nt][c][2 + r] += skip ? 0.f : wr[nt][r] * (v.y * sc);
              }
          }
        }
      }
      if (masked && cc.s.nq > 1) {
        // a lane's column of 16-byte pieces (rows eight apart have theirs exchanged alike)
        bool found = false;
        const SeenKeys seen{cc.r.lo, cc.r.hi, cc.r.sink_hi, full_lo, full_hi, p.sinks};
        if (STEP == 32) {
          for (int r = crow; r < 8; r += RPP)
            found |= mend_pieces_apart<FP8>(sv + swz<ROWB>(r, chunk), 8 * ROWB, 4, j0 + r, 8, seen);
        } else {
          for (int r = crow; r < 16; r += RPP)  // (four times the same piece)
            found |= mend_pieces_apart<FP8>(sv + swz<ROWB>(r, chunk), 0, 4, j0 + r, 0, seen);
        }
        odd |= __any_sync(0xffffffffu, found);
        __syncwarp();
      }
      // ---- O^T += V^T P^T
      if (FP8) {
        const int vr = (lane & 7) + ((lane >> 3) & 1) * 8, vc = lane >> 4;
#pragma unroll
        for (int c = 0; c < D / 16; c += 2)
#pragma unroll
          for (int g = 0; g < KG; ++g) {
            // 16-byte chunks c and c + 1, read as pairs of columns: a register holds key 2q's and key
            // 2q + 1's codes of columns 2 * n8 and 2 * n8 + 1
            uint32_t w[4];
            ldsm4_t(w, sv + swz<ROWB>(g * 16 + vr, c + vc));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t a[4];
              e4m3x4_to_f16x4(__byte_perm(w[2 * h], 0u, 0x3120), a[0], a[1]);
              e4m3x4_to_f16x4(__byte_perm(w[2 * h + 1], 0u, 0x3120), a[2], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<true>(o[nt][c + h], a, pb[g][nt][0], pb[g][nt][1]);
            }
          }
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int g = 0; g < KG; ++g) {
            uint32_t a[4];
            ldsm4_t(a, sv + swz<ROWB>(g * 16 + (lane & 7) + (lane >> 4) * 8, 2 * c + ((lane >> 3) & 1)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[nt][c], a, pb[g][nt][0], pb[g][nt][1]);
          }
      }
    }
    stage = stage + 1 == NST ? 0 : stage + 1;

    // ---- the end of the item, or of this CTA's part of it: join the warps
    cc.left = cc.left_after(1);
    const bool done = cc.left <= 0;
    if (cc.last_tile() || done) {
      const bool whole = seg0 == 0 && cc.last_tile();
      const int slot = first_seg ? 0 : 1;
      if (tid == 0 && seg0 == 0 && !whole) {
        const int left = cc.r.tiles - (cc.t + 1);
        p.desc[blockIdx.x] = make_int4(cc.b, cc.g, cc.rt, slot | (1 + (left + quota - 1) / quota) << 1);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float sum = row_sum(l[nt][r]);
          if (n8 == 0) sml[warp * ROWS + nt * 8 + 2 * q4 + r] = make_float2(m[nt][r], sum);
        }
      const bool any_odd = __syncthreads_or(odd) != 0;
      const int64_t pbase = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * ROWS;
      float f[NT][2], unit2[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          // 2^(r - 127 - 15) as two factors, both normal numbers
          const uint32_t sp = FP8 ? span[nt][r] : 0u;
          const int u = FP8 && !wide_span(sp) ? static_cast<int>(sp & 0xffffu) - 142 : 0, u1 = u / 2;
          const float unit1 = __uint_as_float(static_cast<uint32_t>(127 + u1) << 23);
          unit2[nt][r] = __uint_as_float(static_cast<uint32_t>(127 + u - u1) << 23);
          float top = kNInf;
#pragma unroll
          for (int w = 0; w < W; ++w) top = fmaxf(top, sml[w * ROWS + nt * 8 + 2 * q4 + r].x);
          f[nt][r] = paged_ex2(m[nt][r] - (top == kNInf ? 0.f : top)) * unit1;
        }
      // columns of a row are exchanged by eights so that the four row pairs of a store differ in bank
      constexpr int COLS = L::kCols, PC = COLS / 16;
#pragma unroll
      for (int pass = 0; pass < D / COLS; ++pass) {
        float* mw = merge + warp * ROWS * COLS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < PC; ++c) {
            const float* v = o[nt][pass * PC + c];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float* row = mw + (nt * 8 + 2 * q4 + r) * COLS;
              const float fa = f[nt][r];
              if (FP8) {
                *reinterpret_cast<float2*>(row + ((16 * c + 2 * n8) ^ (q4 << 3 & (COLS - 1)))) =
                    make_float2(v[r] * fa * unit2[nt][r], v[2 + r] * fa * unit2[nt][r]);
              } else {
                row[(16 * c + n8) ^ (q4 << 3 & (COLS - 1))] = v[r] * fa;
                row[(16 * c + 8 + n8) ^ (q4 << 3 & (COLS - 1))] = v[2 + r] * fa;
              }
            }
          }
        __syncthreads();
        for (int e = tid; e < ROWS * (COLS / 4); e += L::kThreads) {
          const int pr = e / (COLS / 4), col = e % (COLS / 4) * 4, pc = col ^ ((pr >> 1 & 3) << 3 & (COLS - 1));
          const int R = cc.rt * ROWS + pr, d0 = pass * COLS + col;
          if (R >= cc.s.nq * p.G) continue;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          float top = kNInf, sum = 0.f;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(merge + (w * ROWS + pr) * COLS + pc);
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
            top = fmaxf(top, sml[w * ROWS + pr].x);
          }
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float2 t = sml[w * ROWS + pr];
            sum += t.y * paged_ex2(t.x - (top == kNInf ? 0.f : top));
          }
          if (whole) {
            const int i = R / p.G, h = cc.g * p.G + R - i * p.G, t = cc.s.q0 + i;
            const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
            if (d0 < p.c.d)
              *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(t) * p.Hq + h) * p.c.d + d0) =
                  make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
            if (d0 == 0) p.lse[static_cast<int64_t>(h) * p.T + t] = sum == 0.f ? kNInf : (top + log2f(sum)) * kPLn2;
          } else {
            *reinterpret_cast<float4*>(p.part_o + (pbase + pr) * D + d0) = a;
            if (d0 == 0) p.part_ml[pbase + pr] = make_float2(top, sum);
          }
          if (any_odd) {
            const int i = R / p.G, h = cc.g * p.G + R - i * p.G, mid = min(full_lo, cc.r.hi);
            const RowKeys rk = row_keys(p, cc.s, cc.s.pos0 + i);
            const OddKeys k{cc.b,    cc.g, cc.r.lo, mid, max(max(full_hi, cc.r.lo), mid), cc.r.hi, cc.r.sink_tiles, cc.r.main0,
                            seg0, cc.t};
            add_odd_values<FP8, L::kKeys>(
                p, k, rk.lo, rk.hi, d0, 4,
                whole ? p.out + (static_cast<int64_t>(cc.s.q0 + i) * p.Hq + h) * p.c.d : nullptr,
                p.part_o + (pbase + pr) * D, 4);
          }
        }
        __syncthreads();
      }
      first_seg = false;
      begin = true;
    }
    if (done) break;
    cc.next(p);
  }
}

// Joins the pieces of the items that more than one CTA of the token kernel worked on.  blockIdx.x:
// the CTA in which the item begins; blockIdx.y: its row.  The block's eight warps share the row's
// pieces (one sequence spread over the machine has up to kPagedCtas of them).
template <int D, int ROWS>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p) {
  constexpr int V = D / 32;
  __shared__ float sacc[8][D];
  __shared__ float2 sml[8];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 ds = p.desc[blockIdx.x];
  const int pieces = ds.w >> 1;
  if (pieces == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pr = blockIdx.y;
  const Seq s = load_seq(p, ds.x, false);
  const int r = ds.z * ROWS + pr;
  if (r >= s.nq * p.G) return;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * 2 + (ds.w & 1)) * ROWS + pr;
  const int64_t rest = static_cast<int64_t>(blockIdx.x) * 2 * ROWS + pr;  // piece i > 0: + i * 2 * ROWS
  float m = kNInf, l = 0.f, a[V];
#pragma unroll
  for (int e = 0; e < V; ++e) a[e] = 0.f;
#pragma unroll 4
  for (int i = warp; i < pieces; i += 8) {
    const int64_t at = i == 0 ? first : rest + static_cast<int64_t>(i) * 2 * ROWS;
    const float2 ml = p.part_ml[at];
    float x[V];
    if (V == 4) {
      const float4 f = *reinterpret_cast<const float4*>(p.part_o + at * D + lane * 4);
      x[0] = f.x, x[1] = f.y, x[V - 2] = f.z, x[V - 1] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(p.part_o + at * D + lane * 2);
      x[0] = f.x, x[1] = f.y;
    }
    const float mn = fmaxf(m, ml.x), base = mn == kNInf ? 0.f : mn;
    const float fa = paged_ex2(m - base), fb = paged_ex2(ml.x - base);
    l = l * fa + ml.y * fb;
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] = a[e] * fa + x[e] * fb;
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) sacc[warp][lane * V + e] = a[e];
  if (lane == 0) sml[warp] = make_float2(m, l);
  __syncthreads();
  if (warp > 0) return;
  m = kNInf;
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, sml[w].x);
  const float base = m == kNInf ? 0.f : m;
  l = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) a[e] = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float f = paged_ex2(sml[w].x - base);
    l += sml[w].y * f;
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] += sacc[w][lane * V + e] * f;
  }
  const int i = r / p.G, h = ds.y * p.G + r - i * p.G, t = s.q0 + i;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  if (lane * V < p.c.d) {
    uint16_t* dst = p.out + (static_cast<int64_t>(t) * p.Hq + h) * p.c.d + lane * V;
    if (V == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[V - 2] * inv, a[V - 1] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(a[0] * inv, a[1] * inv);
  }
  if (lane == 0) p.lse[static_cast<int64_t>(h) * p.T + t] = l == 0.f ? kNInf : (m + log2f(l)) * kPLn2;
}

// Joins the chunk kernel's pieces, which are [column / 4][row] float4: a block takes eight rows, so
// that eight threads next to each other read 128 contiguous bytes.
template <int D>
__global__ void __launch_bounds__(D * 2) paged_chunk_join_kernel(const PagedParams p) {
  constexpr int ROWS = kChunkItemRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 ds = p.desc[blockIdx.x];
  const int pieces = ds.w >> 1;
  if (pieces == 0) return;
  const int pr = blockIdx.y * 8 + (threadIdx.x & 7), col = threadIdx.x >> 3;
  const Seq s = load_seq(p, ds.x, false);
  const int r = ds.z * ROWS + pr;
  if (r >= s.nq * p.G) return;
  const float4* o = reinterpret_cast<const float4*>(p.part_o);
  float m = kNInf, l = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < pieces; ++i) {
    const int64_t pb = ((static_cast<int64_t>(blockIdx.x) + i) * 2 + (i == 0 ? ds.w & 1 : 0)) * ROWS;
    const float2 ml = p.part_ml[pb + pr];
    const float4 x = o[pb * (D / 4) + col * ROWS + pr];
    const float mn = fmaxf(m, ml.x), base = mn == kNInf ? 0.f : mn;
    const float fa = paged_ex2(m - base), fb = paged_ex2(ml.x - base);
    l = l * fa + ml.y * fb;
    a.x = a.x * fa + x.x * fb;
    a.y = a.y * fa + x.y * fb;
    a.z = a.z * fa + x.z * fb;
    a.w = a.w * fa + x.w * fb;
    m = mn;
  }
  const int i = r / p.G, h = ds.y * p.G + r - i * p.G, t = s.q0 + i;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  if (col * 4 < p.c.d)
    *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(t) * p.Hq + h) * p.c.d + col * 4) =
        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  if (col == 0) p.lse[static_cast<int64_t>(h) * p.T + t] = l == 0.f ? kNInf : (m + log2f(l)) * kPLn2;
}

// A join starts while the main kernel's last CTAs still run and waits for them on the device.
cudaError_t launch_join(void (*kern)(PagedParams), const PagedParams& p, int blocks_y, int threads,
                        cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kPagedCtas, blocks_y);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D, bool FP8, int NT>
cudaError_t launch_token(const PagedParams& p, cudaStream_t stream) {
  using L = TokCfg<D, FP8, NT>;
  auto kern = paged_token_kernel<D, FP8, NT>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = set_up_once(ready, kern, L::kTotal, 0);
  if (e != cudaSuccess) return e;
  kern<<<kPagedCtas, L::kThreads, L::kTotal, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.G;
  return launch_join(paged_join_kernel<D, 8 * NT>, p, static_cast<int>(rows < 8 * NT ? rows : 8 * NT), 256, stream);
}

template <int D, bool FP8>
cudaError_t launch_token_rows(const PagedParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.G;
  if (rows <= 8) return launch_token<D, FP8, 1>(p, stream);
  return launch_token<D, FP8, 2>(p, stream);
}

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct PagedLayout {
  size_t desc, ml, o, total;
};

// Rows of an item: the next multiple of eight on the token kernel, else the chunk kernel's.
int item_rows(const fdma_paged_args* a) {
  const int64_t rows = static_cast<int64_t>(a->max_q) * (a->Hq / a->cache.Hkv);
  return rows <= 8 ? 8 : rows <= kTokenRows ? kTokenRows : kChunkItemRows;
}

PagedLayout paged_layout(const fdma_paged_args* a) {
  const size_t rows = static_cast<size_t>(item_rows(a)), width = a->cache.d <= 64 ? 64 : 128;
  PagedLayout w{};
  w.desc = 0;
  w.ml = align256(kPagedCtas * sizeof(int4));
  w.o = align256(w.ml + kPagedCtas * 2 * rows * sizeof(float2));
  w.total = align256(w.o + kPagedCtas * 2 * rows * width * sizeof(float));
  return w;
}

int validate_paged(const fdma_paged_args* a) {
  if (a == nullptr) return FDMA_ERR_INVALID;
  const int st = validate_cache(&a->cache);
  if (st != FDMA_OK) return st;
  if (a->T < 0 || a->Hq <= 0 || a->max_q < 0 || a->Hq % a->cache.Hkv != 0) return FDMA_ERR_INVALID;
  if (static_cast<int64_t>(a->T) * a->Hq > 0x7fffff00 || a->max_q > (1 << 30) / a->Hq) return FDMA_ERR_UNSUPPORTED;
  if (a->causal != 0 && a->causal != 1) return FDMA_ERR_INVALID;
  if (a->window < 0 || a->sinks < 0 || (a->window > 0 && a->causal == 0)) return FDMA_ERR_INVALID;
  if (!(std::isfinite(a->scale * kPLog2e) && a->scale > 0.f)) return FDMA_ERR_INVALID;
  return FDMA_OK;
}

}  // namespace

cudaError_t launch_paged_token(bool fp8, const PagedParams& p, cudaStream_t stream) {
  if (p.c.d <= 64) return fp8 ? launch_token_rows<64, true>(p, stream) : launch_token_rows<64, false>(p, stream);
  return fp8 ? launch_token_rows<128, true>(p, stream) : launch_token_rows<128, false>(p, stream);
}

}  // namespace fdma

using namespace fdma;

extern "C" {

size_t fdma_paged_workspace_size(const fdma_paged_args* a) {
  return validate_paged(a) == FDMA_OK ? paged_layout(a).total : 0;
}

int fdma_paged_fwd(const fdma_paged_args* a, void* out, float* lse, void* stream) {
  const int st = validate_paged(a);
  if (st != FDMA_OK) return st;
  if (a->T == 0 || a->cache.B == 0 || a->max_q == 0) return FDMA_OK;
  if (a->q == nullptr || a->cu_q == nullptr || out == nullptr || lse == nullptr) return FDMA_ERR_INVALID;
  if (!aligned16(a->q) || !aligned16(out)) return FDMA_ERR_UNSUPPORTED;
  for (int i = 0; i < 2; ++i) {
    if (a->q_stride[i] < 0) return FDMA_ERR_INVALID;
    if (a->q_stride[i] % 8 != 0) return FDMA_ERR_UNSUPPORTED;
  }
  const PagedLayout w = paged_layout(a);
  if (a->workspace == nullptr || (reinterpret_cast<uintptr_t>(a->workspace) & 255u) != 0 ||
      a->workspace_bytes < w.total)
    return FDMA_ERR_WORKSPACE;
  PagedParams p{};
  p.c = cache_view(a->cache);
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_t = a->q_stride[0];
  p.q_h = a->q_stride[1];
  p.cu = a->cu_q;
  p.T = a->T;
  p.max_q = a->max_q;
  p.Hq = a->Hq;
  p.G = a->Hq / a->cache.Hkv;
  p.causal = a->causal;
  p.window = a->window;
  p.sinks = a->window > 0 ? a->sinks : 0;
  p.scale_log2 = a->scale * kPLog2e;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  p.desc = reinterpret_cast<int4*>(ws + w.desc);
  p.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  p.min_run = 1;
  const int64_t blocks = (static_cast<int64_t>(a->max_q) * p.G + item_rows(a) - 1) / item_rows(a);
  for (p.plan_lanes = 1; p.plan_lanes < 32 && p.plan_lanes < blocks;) p.plan_lanes *= 2;
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  const bool fp8 = a->cache.cache_type == FDMA_CACHE_E4M3;
  cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  if (item_rows(a) < kChunkItemRows) return launch_paged_token(fp8, p, st_) == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
  p.min_run = 2;
  if (launch_paged_chunk(fp8, p, st_) != cudaSuccess) return FDMA_ERR_CUDA;
  const int64_t rows = static_cast<int64_t>(a->max_q) * p.G;
  const int by = static_cast<int>(((rows < kChunkItemRows ? rows : kChunkItemRows) + 7) / 8);
  const cudaError_t e = p.c.d <= 64 ? launch_join(paged_chunk_join_kernel<64>, p, by, 128, st_)
                                    : launch_join(paged_chunk_join_kernel<128>, p, by, 256, st_);
  return e == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

}  // extern "C"
