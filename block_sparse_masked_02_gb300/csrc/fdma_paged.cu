// Attention of few new tokens a sequence (decoding, a handful of drafted tokens) over a
// paged cache, and the host side of fdma_paged_fwd.
//
// An item is a kv head's query rows of one sequence, at most 16 * MT of them.  Every key
// and value is read from HBM once and takes part in 4 * d flops a row, so with few rows the
// kernel is bound by memory, and its work is to keep enough loads in flight: each of the
// eight warps of a CTA runs its own ring of kStages cp.async stages of 16 keys' K and V rows
// (192 or 160 KB in flight on an SM at d = 128), with no barrier between warps inside the loop, and
// the ring runs on across items, so that a batch of short sequences streams like one long one.
// A tile of 128 keys is 16 keys a warp; page_size is a multiple of 16, so a warp's keys lie in
// one page.
//
// Each warp keeps its own running maximum, weight sum and output for its keys (online
// softmax), and the eight are joined at the end of the item.  The products are
// mma.sync.m16n8k16: at 16 rows the tensor pipe is idle most of the time whichever
// instruction feeds it, and this one takes the keys as they lie in shared memory and P straight
// from registers.
//
// e4m3 caches: codes become f16 exactly (one conversion for two), so the products run in f16.
// q is scaled by a power of two per row to [2^14, 2^15), which is exact but for parts below
// 2^-38 of the row's largest.  The key's scale multiplies S; the value's scale multiplies P,
// as 2^(e - r + 15) with r the largest e so far (the output is kept in units of 2^(r - 15)), so
// that P stays in f16's range and a weight keeps all 11 bits down to 2^-29 of the largest.
#include <cmath>

#include "fdma_paged.cuh"

namespace fdma {

namespace {

constexpr int kTokWarps = 8;
constexpr int kTokThreads = kTokWarps * 32;
constexpr int kTokenRows = 32;  // packed rows up to which the token kernel runs
constexpr float kNInf = -__builtin_huge_valf();

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
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// D: 64 or 128, the head dim's padded width (columns past d are read as zeros).
template <int D, bool FP8, int MT>
struct TokSmem {
  static constexpr int kRowB = FP8 ? D : 2 * D;        // bytes of a row in shared memory
  static constexpr int kHalfB = 16 * kRowB;            // 16 keys of K (or V)
  static constexpr int kStages = kRowB == 256 ? 3 : FP8 ? 5 : 6;
  static constexpr int kWarpB = kStages * 2 * kHalfB;
  static constexpr int kOffMerge = kTokWarps * kWarpB;     // [8][16][64] fp32
  static constexpr int kOffMl = kOffMerge + 8 * 16 * 64 * 4;  // [8][16 * MT] (maximum, sum)
  static constexpr int kOffExp = kOffMl + 8 * 16 * MT * 8;    // [8][kStages][32] scale bytes (e4m3)
  static constexpr int kOffPlan = kOffExp + (FP8 ? 8 * kStages * 32 : 0);
  static constexpr int kTotal = kOffPlan + static_cast<int>(sizeof(PlanSmem));
  static_assert(kTotal <= 232448, "shared memory of one CTA");
};

// Byte offset of 16-byte chunk c of key row r: the chunks of a row are exchanged so that the
// eight rows of an ldmatrix (and the 32 lanes of the e4m3 key reads) touch different banks.
template <int ROWB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return r * ROWB + ((ROWB == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7)) << 4);
}

template <int D, bool FP8, int MT>
__global__ void __launch_bounds__(kTokThreads, 1) paged_token_kernel(const PagedParams p) {
  using L = TokSmem<D, FP8, MT>;
  constexpr int ROWS = 16 * MT, NST = L::kStages, ROWB = L::kRowB;
  constexpr int CPR = ROWB / 16;           // 16-byte chunks of a row
  constexpr int RPP = 32 / CPR;            // rows that a warp copies at a time
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q4 = lane & 3, n8 = lane >> 2;
  PlanSmem* plan = reinterpret_cast<PlanSmem*>(smem + L::kOffPlan);
  float* merge = reinterpret_cast<float*>(smem + L::kOffMerge);
  float2* sml = reinterpret_cast<float2*>(smem + L::kOffMl);
  uint8_t* sexp = smem + L::kOffExp + warp * NST * 32;
  const uint32_t ring = smem_u32(smem) + warp * L::kWarpB;

  Cursor<ROWS> lc;  // the tile that is loaded next
  int quota;
  const int run = plan_run<ROWS, kTokThreads>(p, plan, lc, quota);
  if (tid == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  write_empty_blocks<ROWS>(p);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up; it waits for the end
  if (run == 0) return;
  Cursor<ROWS> cc = lc;  // the tile that is computed next

  // ---- loads: stage (x mod NST) of this warp's ring takes its 16 keys of tile x
  const int chunk = lane % CPR, crow = lane / CPR;
  const uint32_t cbytes = chunk * 16 < p.c.d * (FP8 ? 1 : 2) ? 16u : 0u;
  const int pmask = (1 << p.c.page_shift) - 1;
  uint32_t exp_pend = 127;
  auto page_of = [&](const Cursor<ROWS>& c) {
    const int j0 = c.key0() + warp * 16;
    // a warp's keys are looked up only where some row sees one of them
    return j0 < c.r.sink_hi || (j0 < c.r.hi && j0 + 16 > c.r.lo) ? key_page(p, c.b, j0) : -1;
  };
  int lpage = page_of(lc);
  auto issue = [&](int x) {
    const int st = x % NST;
    const uint32_t dst = ring + st * 2 * L::kHalfB;
    const int j0 = lc.key0() + warp * 16;
    if (FP8 && x > 0) sexp[((x - 1) % NST) * 32 + lane] = static_cast<uint8_t>(exp_pend);
    const int64_t pg = lpage < 0 ? 0 : lpage;
    const uint8_t* kb = p.c.k + pg * p.c.ks[0] + (j0 & pmask) * p.c.ks[1] + lc.g * p.c.ks[2] + chunk * 16;
    const uint8_t* vb = p.c.v + pg * p.c.vs[0] + (j0 & pmask) * p.c.vs[1] + lc.g * p.c.vs[2] + chunk * 16;
#pragma unroll
    for (int i = 0; i < 16 / RPP; ++i) {
      const int r = i * RPP + crow, j = j0 + r;
      const bool ok = lpage >= 0 && (j < lc.r.sink_hi || (j >= lc.r.lo && j < lc.r.hi));
      const uint32_t nb = ok ? cbytes : 0u;
      cp_async16(dst + swz<ROWB>(r, chunk), nb ? kb + r * p.c.ks[1] : p.c.k, nb);
      cp_async16(dst + L::kHalfB + swz<ROWB>(r, chunk), nb ? vb + r * p.c.vs[1] : p.c.v, nb);
    }
    if (FP8) {
      const int r = lane & 15, j = j0 + r;
      exp_pend = 0;
      if (lpage >= 0 && (j < lc.r.sink_hi || (j >= lc.r.lo && j < lc.r.hi))) {
        const int64_t* es = lane < 16 ? p.c.kes : p.c.ves;
        exp_pend = (lane < 16 ? p.c.ke : p.c.ve)[pg * es[0] + (j & pmask) * es[1] + lc.g * es[2]];
      }
    }
  };
  int loaded = 0;
  auto load_next = [&]() {
    if (loaded < run) {
      issue(loaded);
      if (++loaded < run) {
        lc.next(p);
        lpage = page_of(lc);
      }
    } else if (FP8 && loaded == run) {
      sexp[((run - 1) % NST) * 32 + lane] = static_cast<uint8_t>(exp_pend);
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < NST - 1; ++i) load_next();

  uint32_t qf[MT][D / 16][4];  // Q as A fragments
  float rowfac[MT][2];         // log2(e) * scale (and the row's power of two) of rows n8, n8 + 8
  RowKeys rk[MT][2];
  float o[MT][D / 8][4];
  float m[MT][2], l[MT][2];
  int ref = 0;  // e4m3: the largest value scale byte so far
  int seg0 = 0;             // tile of the item at which this CTA began
  bool first_seg = true;
  bool begin = true;

#pragma unroll 1
  for (int x = 0; x < run; ++x) {
    if (begin) {
      // ---- a new item: its query rows, and an empty softmax
      begin = false;
      seg0 = cc.t;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = cc.rt * ROWS + mt * 16 + h * 8 + n8;
          const bool in = r < cc.s.nq * p.G;
          const int i = in ? r / p.G : 0;
          const uint16_t* src = p.q + (cc.s.q0 + i) * p.q_t + (cc.g * p.G + (in ? r - i * p.G : 0)) * p.q_h;
          rk[mt][h] = row_keys(p, cc.s, cc.s.pos0 + i);
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // the pair's columns: with e4m3 a lane's key bytes are D / 4 adjacent ones, so the
              // order of the columns inside the product is that of those bytes
              const int col = FP8 ? q4 * (D / 4) + s * 4 + e * 2 : s * 16 + e * 8 + q4 * 2;
              qf[mt][s][h + 2 * e] =
                  in && col < p.c.d ? __ldg(reinterpret_cast<const uint32_t*>(src + col)) : 0u;
            }
          rowfac[mt][h] = p.scale_log2;
          if (FP8) {
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t w = qf[mt][s][h + 2 * e];
                top = max(top, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
              }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // q * 2^up has its largest part in [2^14, 2^15)
            const int E = static_cast<int>(top >> 7);
            const int up = E == 0 || E == 255 ? 0 : 14 + 127 - E;
            const float f1 = __uint_as_float(static_cast<uint32_t>(127 + up / 2) << 23);
            const float f2 = __uint_as_float(static_cast<uint32_t>(127 + up - up / 2) << 23);
            rowfac[mt][h] = p.scale_log2 / f1 / f2;
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t w = qf[mt][s][h + 2 * e];
                qf[mt][s][h + 2 * e] = pack_f16x2(__uint_as_float(w << 16) * f1 * f2,
                                                  __uint_as_float(w & 0xffff0000u) * f1 * f2);
              }
          }
          m[mt][h] = kNInf;
          l[mt][h] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][c][e] = 0.f;
      }
      ref = 0;
    }
    cp_async_wait<NST - 2>();
    __syncwarp();
    load_next();

    const int j0 = cc.key0() + warp * 16;
    if (j0 < cc.r.sink_hi || (j0 < cc.r.hi && j0 + 16 > cc.r.lo)) {
      const int st = x % NST;
      const uint32_t sk = ring + st * 2 * L::kHalfB, sv = sk + L::kHalfB;
      // ---- S = Q K^T: rows n8 (+8), keys j0 + 8 * nt + 2 * q4 + {0, 1}
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
      if (FP8) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 w = lds128(sk + swz<ROWB>(nt * 8 + n8, q4 * (D / 64) + c));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t b0 = e4m3x2_to_f16x2(ww[e]), b1 = e4m3x2_to_f16x2(ww[e] >> 16);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma16816<true>(s[mt][nt], qf[mt][c * 4 + e], b0, b1);
            }
          }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t b[4];
          ldsm4(b, sk + swz<ROWB>((lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816<false>(s[mt][0], qf[mt][ks], b[0], b[1]);
            mma16816<false>(s[mt][1], qf[mt][ks], b[2], b[3]);
          }
        }
      }
      float kf[2][2], vf[2][2];  // scales of the lane's four keys
      float oscale = 1.f;
      if (FP8) {
        const uint8_t* ex = sexp + st * 32;
        const int mx = __reduce_max_sync(0xffffffffu, lane >= 16 ? static_cast<int>(ex[lane]) : 0);
        if (mx > ref) {  // the output's unit grows
          oscale = ref == 0 ? 0.f : __uint_as_float(static_cast<uint32_t>(max(127 - (mx - ref), 0)) << 23);
          ref = mx;
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = nt * 8 + q4 * 2 + e;
            kf[nt][e] = exp_scale(ex[k]);
            const int ve = ex[16 + k];
            vf[nt][e] = __uint_as_float(static_cast<uint32_t>(max(127 + 15 - (ref - ve), 0)) << 23);
          }
      }
      // ---- softmax of these 16 keys
      uint32_t pa[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float alpha[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = kNInf;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = j0 + nt * 8 + q4 * 2 + e;
              float u = s[mt][nt][2 * h + e] * rowfac[mt][h];
              if (FP8) u *= kf[nt][e];
              if (!(j < rk[mt][h].hi && (j >= rk[mt][h].lo || j < p.sinks))) u = kNInf;
              s[mt][nt][2 * h + e] = u;
              mx = fmaxf(mx, u);
            }
          mx = fmaxf(m[mt][h], quad_max(mx));
          const float base = mx == kNInf ? 0.f : mx;
          alpha[h] = paged_ex2(m[mt][h] - base);
          m[mt][h] = mx;
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float w = paged_ex2(s[mt][nt][2 * h + e] - base);
              sum += w;
              s[mt][nt][2 * h + e] = FP8 ? w * vf[nt][e] : w;
            }
          l[mt][h] = l[mt][h] * alpha[h] + sum;
          alpha[h] *= oscale;
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            o[mt][c][0] *= alpha[0];
            o[mt][c][1] *= alpha[0];
            o[mt][c][2] *= alpha[1];
            o[mt][c][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            pa[mt][nt * 2 + h] = FP8 ? pack_f16x2(s[mt][nt][2 * h], s[mt][nt][2 * h + 1])
                                     : pack_bf16x2(s[mt][nt][2 * h], s[mt][nt][2 * h + 1]);
      }
      // ---- O += P V
      const int vr = (lane & 7) + ((lane >> 3) & 1) * 8, vc = lane >> 4;
      if (FP8) {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          // 16-byte chunks c and c + 1, read as pairs of columns: a register holds key 2q's and key
          // 2q + 1's codes of columns 2 * n8 and 2 * n8 + 1
          uint32_t w[4];
          ldsm4_t(w, sv + swz<ROWB>(vr, c + vc));
#pragma unroll
          for (int cc2 = 0; cc2 < 2; ++cc2)
#pragma unroll
            for (int par = 0; par < 2; ++par) {
              const uint32_t sel = par ? 0x0031u : 0x0020u;
              const uint32_t b0 = e4m3x2_to_f16x2(__byte_perm(w[2 * cc2], 0u, sel));
              const uint32_t b1 = e4m3x2_to_f16x2(__byte_perm(w[2 * cc2 + 1], 0u, sel));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma16816<true>(o[mt][2 * (c + cc2) + par], pa[mt], b0, b1);
            }
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 8; c += 2) {
          uint32_t b[4];
          ldsm4_t(b, sv + swz<ROWB>(vr, c + vc));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816<false>(o[mt][c], pa[mt], b[0], b[1]);
            mma16816<false>(o[mt][c + 1], pa[mt], b[2], b[3]);
          }
        }
      }
    }

    // ---- the end of the item, or of this CTA's part of it: join the eight warps
    if (cc.last_tile() || x + 1 == run) {
      const bool whole = seg0 == 0 && cc.last_tile();
      const int slot = first_seg ? 0 : 1;
      if (tid == 0 && seg0 == 0 && !whole) {
        const int left = cc.r.tiles - (cc.t + 1);
        p.desc[blockIdx.x] = make_int4(cc.b, cc.g, cc.rt, slot | (1 + (left + quota - 1) / quota) << 1);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float sum = quad_sum(l[mt][h]);
          if (q4 == 0) sml[warp * ROWS + mt * 16 + h * 8 + n8] = make_float2(m[mt][h], sum);
        }
      // 2^(ref - 127 - 15) as two factors, both normal numbers
      const int u = ref - 142, u1 = u / 2;
      const float unit1 = FP8 ? __uint_as_float(static_cast<uint32_t>(127 + u1) << 23) : 1.f;
      const float unit2 = FP8 ? __uint_as_float(static_cast<uint32_t>(127 + u - u1) << 23) : 1.f;
      __syncthreads();
      const int64_t pbase = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * ROWS;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float top = kNInf;
#pragma unroll
          for (int w = 0; w < kTokWarps; ++w) top = fmaxf(top, sml[w * ROWS + mt * 16 + h * 8 + n8].x);
          f[h] = paged_ex2(m[mt][h] - (top == kNInf ? 0.f : top));
          if (FP8) f[h] *= unit1;
        }
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          float* mw = merge + warp * 1024;
          if (FP8) {
            // columns 16c + 4 * q4 + {0, 1, 2, 3} of rows n8, n8 + 8
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float* a = o[mt][2 * (half * 4 + c)];
                const float* b = o[mt][2 * (half * 4 + c) + 1];
                *reinterpret_cast<float4*>(mw + (n8 + 8 * h) * 64 + ((16 * c + 4 * q4) ^ ((n8 & 1) << 4))) =
                    make_float4(a[2 * h] * f[h] * unit2, b[2 * h] * f[h] * unit2, a[2 * h + 1] * f[h] * unit2,
                                b[2 * h + 1] * f[h] * unit2);
              }
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2*>(mw + (n8 + 8 * h) * 64 + ((8 * c + 2 * q4) ^ ((n8 & 3) << 3))) =
                    make_float2(o[mt][half * 8 + c][2 * h] * f[h], o[mt][half * 8 + c][2 * h + 1] * f[h]);
          }
          __syncthreads();
          {
            const int row = tid >> 4, col = (tid & 15) * 4;
            const int pc = FP8 ? col ^ ((row & 1) << 4) : col ^ ((row & 3) << 3);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = kNInf, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kTokWarps; ++w) {
              const float4 v = *reinterpret_cast<const float4*>(merge + w * 1024 + row * 64 + pc);
              a.x += v.x;
              a.y += v.y;
              a.z += v.z;
              a.w += v.w;
              top = fmaxf(top, sml[w * ROWS + mt * 16 + row].x);
            }
#pragma unroll
            for (int w = 0; w < kTokWarps; ++w) {
              const float2 t = sml[w * ROWS + mt * 16 + row];
              sum += t.y * paged_ex2(t.x - (top == kNInf ? 0.f : top));
            }
            const int pr = mt * 16 + row, r = cc.rt * ROWS + pr, d0 = half * 64 + col;
            if (r < cc.s.nq * p.G) {
              if (whole) {
                const int i = r / p.G, h = cc.g * p.G + r - i * p.G, t = cc.s.q0 + i;
                const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
                if (d0 < p.c.d)
                  *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(t) * p.Hq + h) * p.c.d + d0) =
                      make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
                if (half == 0 && (tid & 15) == 0)
                  p.lse[static_cast<int64_t>(h) * p.T + t] = sum == 0.f ? kNInf : (top + log2f(sum)) * kPLn2;
              } else {
                *reinterpret_cast<float4*>(p.part_o + (pbase + pr) * D + d0) = a;
                if (half == 0 && (tid & 15) == 0) p.part_ml[pbase + pr] = make_float2(top, sum);
              }
            }
          }
          __syncthreads();
        }
      }
      first_seg = false;
      begin = true;
    }
    if (x + 1 < run) cc.next(p);
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

template <int D, bool FP8, int MT>
cudaError_t launch_token(const PagedParams& p, cudaStream_t stream) {
  using L = TokSmem<D, FP8, MT>;
  auto kern = paged_token_kernel<D, FP8, MT>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = set_up_once(ready, kern, L::kTotal, 0);
  if (e != cudaSuccess) return e;
  kern<<<kPagedCtas, kTokThreads, L::kTotal, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.G;
  return launch_join(paged_join_kernel<D, 16 * MT>, p, static_cast<int>(rows < 16 * MT ? rows : 16 * MT), 256, stream);
}

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct PagedLayout {
  size_t desc, ml, o, total;
};

// Rows of an item: 16 or 32 on the token kernel, else the chunk kernel's.
int item_rows(const fdma_paged_args* a) {
  const int64_t rows = static_cast<int64_t>(a->max_q) * (a->Hq / a->cache.Hkv);
  return rows <= 16 ? 16 : rows <= kTokenRows ? 32 : kChunkItemRows;
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
  if (!(std::isfinite(a->scale) && a->scale > 0.f)) return FDMA_ERR_INVALID;
  return FDMA_OK;
}

}  // namespace

cudaError_t launch_paged_token(bool fp8, const PagedParams& p, cudaStream_t stream) {
  const bool two = static_cast<int64_t>(p.max_q) * p.G > 16;
  if (p.c.d <= 64) {
    if (fp8) return two ? launch_token<64, true, 2>(p, stream) : launch_token<64, true, 1>(p, stream);
    return two ? launch_token<64, false, 2>(p, stream) : launch_token<64, false, 1>(p, stream);
  }
  if (fp8) return two ? launch_token<128, true, 2>(p, stream) : launch_token<128, true, 1>(p, stream);
  return two ? launch_token<128, false, 2>(p, stream) : launch_token<128, false, 1>(p, stream);
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
