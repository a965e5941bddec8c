// Norms of queries and keys for each head and the rotation of their positions, forward and
// backward (include/fdma_inputs.h).
//
// With x a row, r = 1 / sqrt(mean(x^2) + eps) and g the gradient of the output turned back:
//   forward   y = turned(x r w)
//   backward  e = g r,  dx = e w - x r^2 mean(e w x),  dw = sum over tokens (and heads that share it) of e x.
// (Both sums of a row can run together, as r may be taken into account last; that took more instructions and 3 % longer.)
//
// One kernel does either.  Bound by memory traffic, it keeps it going: a CTA has a chunk of one tensor's
// heads (one pass where every head has a weight of its own) and its warps walk over tokens, a pass a step, with
// the rows of the next steps and the angles of the next tokens on their way into shared memory; a lane's
// weight lies there too, which leaves registers for three CTAs an SM.  The backward sums a weight's gradient in
// registers; at the end the CTA adds its warps' sums in a fixed order and writes one part, and a second kernel
// adds the parts of a weight.
//
// 16384 tokens of 16 + 4 heads of 128, one weight a tensor, inputs not in L2: forward 31 us (176 MB, 5.6 TB/s; a copy of
// as much 26), backward 46 us (260 MB, 5.6 TB/s; 38), of which the sum of the weights' parts 2.  Two sequences of 4096 tokens of 32 + 8
// heads with a weight each, half of the columns turned, backward: 49 us (253 MB, 5.2 TB/s; 37), as every pass is then a new token's
// (54 us where such a walk went through the loop over a token's passes, and found every row's address from its token's number).  What bounds both is
// issue and latency (issue slots 63 and 52 % busy at 24 and 16 warps an SM), no longer the wait for memory (stalls on it: 0.3 of 8
// cycles an instruction).  Few heads cost more: 32768 tokens of 8 + 1 take 33 us for 168 MB and 55 for 243 (25 and 36 at a copy's
// rate), as a key's row then has a pass to itself.
//
// Steps that led here (the first case forward / backward, us): a row a lane group, addresses for each 52 / 102; a warp a token,
// arithmetic on pairs, pieces of 16 bytes 39 / 80; rows on their way in shared memory 36 / 70; angles and weights there too 34
// / 53; CTAs by what a token costs 31 / 46.
#include <algorithm>
#include <cmath>

#include "fdma_norm_rope.cuh"

namespace fdma {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSmemPerSm = 227 * 1024;
// CTAs of an SM that registers allow.  (Forward with two and all the registers: the same; backward with three and 80
// registers: 109 against 53 us, for spills.)
constexpr int ctas_per_sm(int piece, bool back) { return back && piece == 8 ? 2 : 3; }

struct TokenLine {
  int N, batches;  // batches 1: tokens are one line
  uint32_t tokens;
};

// A token of a warp's walk.
struct Token {
  uint32_t n;
  int b;
};
__device__ __forceinline__ bool wrap(const TokenLine& t, Token& k) {
  if (t.batches == 1 || k.n < static_cast<uint32_t>(t.N)) return false;
  const uint32_t more = k.n / t.N;
  k.b += more;
  k.n -= more * t.N;
  return true;
}
__device__ __forceinline__ uint16_t* row_of(const RowsView& r, const Token& k, int64_t first) {
  return r.p + k.b * r.st[0] + k.n * r.st[1] + first;
}

// Position of a token before it is checked.
__device__ __forceinline__ int position_of(const NormRopeView& v, int b, int n) {
  return v.pos != nullptr ? v.pos[b * v.pos_st[0] + n * v.pos_st[1]] : v.first + n;
}

constexpr int kMostChunks = 16;

// Where the input's rows, of q and k together, are more than 134 MB, the forward reads and writes rows as what L2 (129 MB) drops first:
// there are as many bytes of output, and the first of them would be gone before a next kernel reads them, while the angles stay.
// (MB of rows, of heads of 16 + 4: us usual / so.  84: 30.2 / 28.3, 105: 37.6 / 37.2, 126: 43.5 / 42.6, 147: 50.6 / 49.8, 168: 56.6 / 55.6, 252:
// 87.7 / 83.5, 336: 118 / 111.  So alone it would pay from 84 MB on, but the attention that follows then does not find the outputs in L2.)
// The backward has no registers for it (51 against 46 us, 170 against 175).  It takes one pass a chunk there instead: 84 MB 45.0 / 48.4,
// 105: 56.0 / 57.2, 126: 65.4 / 66.8, 147: 75.0 / 76.2, 168: 85.4 / 85.6, 252: 127 / 124, 336: 173 / 163, 671: 355 / 314.  (That crosses at about
// 180 MB: from 134 MB to there the common limit costs up to 1.6 %.)
constexpr int64_t kMostInL2 = 128 << 20;
bool beyond_l2(const fdma_norm_rope_args& a) {
  return static_cast<int64_t>(a.B) * a.N * (static_cast<int64_t>(a.Hq) + a.Hk) > kMostInL2 / (2 * a.d);
}

// How the work is dealt out: tensor s (q, k) has chunks[s] chunks of `per` passes (the last of fewer), each with ctas[s]
// CTAs.
struct WalkPlan {
  int per, chunks[2], ctas[2], grid;
  int rows;  // weight rows of a CTA's part
  size_t part_bytes;
  int smem, table;  // of a CTA; of a warp's row of angles
};

struct WalkView {
  NormRopeView v;
  TokenLine line;
  int H[2], passes[2];
  WalkPlan plan;
  RowsView x[2], g[2], out[2];  // g: backward
  float* part;  // backward: [cta][plan.rows][d]; nullptr: no weight's gradient
  int* err;
  bool heads;    // every head has a weight of its own
  bool pass_l2;  // forward: the rows do not displace what is in L2
};

template <int P, bool ADJ>
__device__ __forceinline__ void put_columns(float* s, const Pairs<P>& x, const Lane& at) {
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    float a0, a1, b0, b1;
    f2split(x.a[i], a0, a1);
    f2split(x.b[i], b0, b1);
    if (ADJ) {
      float* p = s + (i < P / 4 ? at.ca + 4 * i : at.cb + 4 * (i - P / 4));
      p[0] = a0, p[1] = b0, p[2] = a1, p[3] = b1;
    } else {
      s[at.ca + 2 * i] = a0, s[at.ca + 2 * i + 1] = a1;
      s[at.cb + 2 * i] = b0, s[at.cb + 2 * i + 1] = b1;
    }
  }
}

// Steps of a warp that are on their way at once: 2 KB of rows, backward 6 KB.  (Forward with 3, 4 and 6 KB: 31.1, 31.3 and 32.4 us
// against 31.3, and 119, 119 to 124 against 112 to 114 for 65536 tokens: DRAM does better with less in flight; 1 KB with four CTAs an SM
// 37 and 126.  Backward with 4 and 8: 48.2 and 46.7 against 46.0.)  There are angles of a token more than steps, where a token
// has several (the last of one token and the first of the next share a slot's turn), else as many.
template <int P, bool BACK>
constexpr int kSlots = BACK ? 24 / P : 16 / P;
template <int P, bool BACK>
constexpr int kRingBytes = kSlots<P, BACK> * (BACK ? 2 : 1) * Ring<P>::kSlot;

// ONE: a chunk is one pass.
template <int P, int LPR, bool ADJ, bool ONE, bool BACK>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(P, BACK)) norm_rope_kernel(const __grid_constant__ WalkView p) {
  constexpr int RPW = 32 / LPR, COLS = 2 * P * LPR, SLOTS = kSlots<P, BACK>, STEP = BACK ? 2 : 1, WEIGHT = 256 * P,
                TURNS = ONE ? SLOTS : SLOTS + 1;
  static_assert(kRingBytes<P, BACK> >= RPW * COLS * sizeof(float) || !BACK, "the sums take the rings' place");
  extern __shared__ __align__(16) uint8_t smem[];  // weight | rings | angles
  if (BACK) launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % LPR, g = lane / LPR, warp = threadIdx.x >> 5;
  int cta = blockIdx.x;
  const int side = cta >= p.plan.chunks[0] * p.plan.ctas[0];
  if (side) cta -= p.plan.chunks[0] * p.plan.ctas[0];
  const int chunk = cta / p.plan.ctas[side];
  const int q_first = chunk * p.plan.per, q_last = min(q_first + p.plan.per, p.passes[side]), H = p.H[side];
  const Lane at = lane_of<P, LPR, ADJ>(p.v, l, g);
  const RowsView &x = p.x[side], &gr = p.g[side], &out = p.out[side];
  const uint32_t step = p.plan.ctas[side] * kWarps, tok0 = (cta - chunk * p.plan.ctas[side]) * kWarps + warp;
  const uint32_t base = smem_u32(smem), weight = base + lane * 16;
  const Ring<P> ring(base + WEIGHT + warp * kRingBytes<P, BACK>, lane);
  const uint32_t table = base + WEIGHT + kWarps * kRingBytes<P, BACK> + warp * TURNS * p.plan.table;
  const int64_t by_x = RPW * x.st[2], by_g = BACK ? RPW * gr.st[2] : 0, by_out = RPW * out.st[2];
  const int h_first = q_first * RPW + g, h_end = at.in ? H : 0;
  const int64_t x_first = h_first * x.st[2] + at.ca, g_first = BACK ? h_first * gr.st[2] + at.ca : 0,
                out_first = h_first * out.st[2] + at.ca;

  uint64_t policy = 0;  // of the rows (forward), as they are read and as they are written
  if (!BACK) {
    if (p.pass_l2) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
  }
  // what is fetched next (ONE: a token's one pass, `hop` values behind the last one's)
  Token next{tok0, 0};
  wrap(p.line, next);
  uint32_t tok_next = tok0;
  int pos_next = tok_next < p.line.tokens ? position_of(p.v, next.b, next.n) : 0;
  int q_next = q_last, h_next = 0, row_next = 0;
  uint32_t left_out = 0, begun = 0;  // bit t % 32: token t of the walk is left out; tokens begun
  const uint16_t *x_next = nullptr, *g_next = nullptr;
  if (ONE) {
    x_next = row_of(x, next, x_first);
    if (BACK) g_next = row_of(gr, next, g_first);
  }
  const int64_t hop_x = static_cast<int64_t>(step) * x.st[1], hop_g = BACK ? static_cast<int64_t>(step) * gr.st[1] : 0,
                hop_out = static_cast<int64_t>(step) * out.st[1];
  auto copy = [&](int slot, bool real) {
    if (!BACK) {
      ring.copy(slot, x_next, at.apart, real, policy);
    } else {
      if (p.v.norm) ring.copy(2 * slot, x_next, at.apart, real);
      ring.copy(2 * slot + 1, g_next, at.apart, real);
    }
  };
  auto start = [&](int slot) {
    if ((ONE || q_next == q_last) && tok_next < p.line.tokens) {
      int pos = pos_next;
      if (p.v.pos != nullptr) {  // (else they are inside the table)
        pos = checked_position(p.v, pos, p.err);
        const uint32_t bit = 1u << (begun & 31u);
        left_out = pos < 0 ? left_out | bit : left_out & ~bit;
        ++begun;
      }
      __syncwarp();  // (these angles may take the place of those that were read last)
      if (pos >= 0) {
        const float* angles = p.v.rope + static_cast<int64_t>(pos) * p.v.rot;
        const uint32_t to = table + (ONE ? slot : row_next) * p.plan.table;
        for (int i = 4 * lane; i < p.v.rot; i += 128) cp_async16(to + 4 * i, angles + i, 16);
      }
      if (ONE) {
        copy(slot, pos >= 0 && h_first < h_end);
      } else {
        row_next = row_next + 1 == TURNS ? 0 : row_next + 1;
        x_next = row_of(x, next, x_first);
        if (BACK) g_next = row_of(gr, next, g_first);
        h_next = pos < 0 ? h_end : h_first;
        q_next = q_first;
      }
      tok_next += step;
      next.n += step;
      if (ONE) {
        x_next += hop_x;
        if (BACK) g_next += hop_g;
        if (wrap(p.line, next)) {
          x_next = row_of(x, next, x_first);
          if (BACK) g_next = row_of(gr, next, g_first);
        }
      } else {
        wrap(p.line, next);
      }
      if (tok_next < p.line.tokens) pos_next = position_of(p.v, next.b, next.n);
    }
    if (!ONE && q_next < q_last) {
      copy(slot, h_next < h_end);
      x_next += by_x;
      if (BACK) g_next += by_g;
      h_next += RPW;
      ++q_next;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < SLOTS; ++i) start(i);
  if (warp == 0) put_weight<P>(weight, load_weight<P, ADJ>(p.v, side, min(h_first, H - 1), at));
  __syncthreads();

  Pairs<P> acc;
#pragma unroll
  for (int e = 0; e < P / 2; ++e) acc.a[e] = acc.b[e] = 0;
  Token now{tok0, 0};
  wrap(p.line, now);
  int slot = 0, row = 0;
  uint32_t done = 0;
  // a pass of a token: this lane's row is head h, and goes to `to`
  auto pass = [&](uint16_t* to, int h, uint32_t angles, bool left) {
    const uint32_t half = 2 * p.v.rot;
    if (left) {
      if (BACK && h < h_end) store_raw<P>(to, at.apart, no_raw<P>());
    } else {
      Pairs<P> d = widen<P, ADJ>(ring.get(STEP * slot + STEP - 1));
      if constexpr (BACK) {
        if (p.v.norm) {
          Pairs<P> xs = widen<P, ADJ>(ring.get(STEP * slot));
          float by;
          const float r = row_rsqrt<LPR>(p.v, xs, by);
          turn_shared<true, ADJ>(d, angles, half, at);
          scale(d, r);
#pragma unroll
          for (int e = 0; e < P / 2; ++e) {
            acc.a[e] = fma2(d.a[e], xs.a[e], acc.a[e]);
            acc.b[e] = fma2(d.b[e], xs.b[e], acc.b[e]);
          }
          multiply_shared(d, weight);
          const float m = row_sum<LPR>(dot(d, xs)) * p.v.inv_d * (-r * r);
          const uint64_t m2 = f2(m, m);
#pragma unroll
          for (int e = 0; e < P / 2; ++e) {
            d.a[e] = fma2(xs.a[e], m2, d.a[e]);
            d.b[e] = fma2(xs.b[e], m2, d.b[e]);
          }
          if (__any_sync(0xffffffffu, by != 1.f)) scale(d, by);
        } else {
          turn_shared<true, ADJ>(d, angles, half, at);
        }
      } else {
        if (p.v.norm) {
          float by;
          scale(d, row_rsqrt<LPR>(p.v, d, by));
          multiply_shared(d, weight);
        }
        turn_shared<false, ADJ>(d, angles, half, at);
      }
      if (h < h_end) {
        if (BACK) store_raw<P>(to, at.apart, narrow<P, ADJ>(d));
        else store_raw<P>(to, at.apart, narrow<P, ADJ>(d), policy);
      }
    }
  };
  uint16_t* to = ONE ? row_of(out, now, out_first) : nullptr;
  for (uint32_t tok = tok0; tok < p.line.tokens; tok += step) {
    const bool left = (left_out >> (done & 31u)) & 1u;
    if (!ONE) to = row_of(out, now, out_first);
    cp_async_wait<SLOTS - 1>();
    __syncwarp();  // the angles, which other lanes fetched
    if (ONE) {
      pass(to, h_first, table + slot * p.plan.table, left);
      start(slot);
      slot = slot + 1 == SLOTS ? 0 : slot + 1;
    } else {
      const uint32_t angles = table + row * p.plan.table;
      int h = h_first;
#pragma unroll 1
      for (int q = q_first; q < q_last; ++q, h += RPW, to += by_out) {
        cp_async_wait<SLOTS - 1>();
        pass(to, h, angles, left);
        start(slot);
        slot = slot + 1 == SLOTS ? 0 : slot + 1;
      }
      row = row + 1 == TURNS ? 0 : row + 1;
    }
    if (p.v.pos != nullptr) ++done;
    now.n += step;
    to += hop_out;
    if (wrap(p.line, now)) to = row_of(out, now, out_first);
  }
  cp_async_wait_all();
  if (!BACK || p.part == nullptr) return;
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem + WEIGHT);  // [warp][row of a pass][column]
  if (at.in) put_columns<P, ADJ>(sums + (warp * RPW + g) * COLS, acc, at);
  __syncthreads();
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.plan.rows * p.v.d;
  for (int i = threadIdx.x; i < p.plan.rows * p.v.d; i += kThreads) {
    const int r = i / p.v.d, c = i - r * p.v.d;
    float sum = 0.f;
    for (int j = 0; j < kWarps; ++j) {
      if (p.heads) {
        sum += sums[(j * RPW + r) * COLS + c];
      } else {
#pragma unroll
        for (int k = 0; k < RPW; ++k) sum += sums[(j * RPW + k) * COLS + c];
      }
    }
    part[i] = sum;
  }
}

struct WeightSumView {
  const float* part;
  float* dw[2];
  WalkPlan plan;
  int d, H[2], heads, rpw;
};

// Adds the CTAs' parts: block (row of the weights, 32 columns) of 32 x 32 threads.
__global__ void __launch_bounds__(1024) weight_sum_kernel(const __grid_constant__ WeightSumView p) {
  __shared__ float s[32][33];
  wait_for_primary();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.y * 32 + tx;
  int side, h = 0;
  if (p.heads) {
    side = static_cast<int>(blockIdx.x) >= p.H[0];
    h = blockIdx.x - (side ? p.H[0] : 0);
  } else {
    side = blockIdx.x;
  }
  float* dw = side ? p.dw[1] : p.dw[0];
  if (dw == nullptr) return;
  const int heads = p.plan.per * p.rpw, chunk = p.heads ? h / heads : 0, row = p.heads ? h - chunk * heads : 0;
  const int ctas = p.plan.ctas[side];
  const int first = (side ? p.plan.chunks[0] * p.plan.ctas[0] : 0) + chunk * ctas, count = p.heads ? ctas : p.plan.chunks[side] * ctas;
  float sum = 0.f;
  if (c < p.d)
    for (int j = ty; j < count; j += 32) sum += p.part[(static_cast<int64_t>(first + j) * p.plan.rows + row) * p.d + c];
  s[ty][tx] = sum;
  __syncthreads();
  sum = s[tx][ty];  // column ty of the 32
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (tx == 0 && blockIdx.y * 32 + ty < p.d) dw[static_cast<int64_t>(h) * p.d + blockIdx.y * 32 + ty] = sum;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int passes_of(int H, int rows) { return (H + rows - 1) / rows; }

bool by_head(const fdma_norm_rope_args& a) { return a.q_weight_head != 0 || a.k_weight_head != 0; }

// The chunks of `per` passes with their CTAs, and what it costs the last warp (passes, times 3).
int64_t deal(WalkPlan& r, const int (&q)[2], int per, int64_t tokens, int64_t ctas) {
  r.per = per;
  // A token costs a chunk its passes and two thirds of one for what is done once (190 of 284 instructions, backward; the last
  // chunk counts as a whole one).  CTAs go by that, and, as a warp has whole tokens, by which of the two whole numbers
  // next to the even share of q's leaves less to the last warp of either.  (By passes alone: 34 and 53 us; with as much as a pass
  // for what is done once 33.6 and 48.9, against 31.2 and 46.)
  int64_t cost[2], all = 0;
  for (int s = 0; s < 2; ++s) {
    r.chunks[s] = (q[s] + per - 1) / per;
    cost[s] = 3 * (q[s] < per ? q[s] : per) + 2;
    all += r.chunks[s] * cost[s];
  }
  // tokens of a warp of n CTAs, and as well the CTAs whose warps have at most n
  auto share = [&](int64_t n) { return (tokens + n * kWarps - 1) / (n * kWarps); };
  const int64_t even = ctas * cost[0] / all, up = share(even < 1 ? 1 : even);
  int64_t best = -1;
  for (int64_t t = up; t >= 1 && t >= up - 1; --t) {
    const int64_t n = share(t), rest = r.chunks[1] > 0 ? (ctas - n * r.chunks[0]) / r.chunks[1] : 1;
    if (t < up && (rest < 1 || n * r.chunks[0] > ctas)) continue;  // (the first one is taken whatever there is)
    const int64_t m = r.chunks[1] > 0 ? share(share(rest < 1 ? 1 : rest)) : 0;
    const int64_t last = r.chunks[1] > 0 && share(m) * cost[1] > t * cost[0] ? share(m) * cost[1] : t * cost[0];
    if (best >= 0 && last >= best) continue;
    best = last;
    r.ctas[0] = static_cast<int>(n);
    r.ctas[1] = static_cast<int>(m);
  }
  r.grid = r.chunks[0] * r.ctas[0] + r.chunks[1] * r.ctas[1];
  return best;
}

WalkPlan walk_plan(const fdma_norm_rope_args& a, bool back) {
  WalkPlan r{};
  const int rot = a.rope != nullptr ? a.rot : 0, piece = piece_of(a.d, rot, a.interleaved != 0),
            rpw = pass_rows(a.d, rot, a.interleaved != 0);
  const int slots = back ? 24 / piece : 16 / piece;
  r.table = 4 * rot;
  r.smem = 256 * piece + kWarps * (slots * (back ? 2 : 1) * 128 * piece + (slots + 1) * r.table);
  int per_sm = kSmemPerSm / (r.smem + 1024);
  if (per_sm > ctas_per_sm(piece, back)) per_sm = ctas_per_sm(piece, back);
  const int64_t ctas = 152 * per_sm;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  const int q[2] = {passes_of(a.Hq, rpw), passes_of(a.Hk, rpw)};
  const bool one = by_head(a) || (back && beyond_l2(a));
  const int per = one ? 1 : plan_passes(q[0] + q[1], tokens, ctas * kWarps).per;
  int64_t best = deal(r, q, per, tokens, ctas);
  // A warp has whole tokens of a chunk: where that is few, the last one can have twice the even share, and other chunks
  // leave it less.  (1000 tokens of 64 + 8 heads of 128, forward / backward: 8.9 / 15.9 us, 9.6 / 18.4 without; 2500:
  // 20.5 / 29.1, 22.9 / 37.6.  What is less than a sixteenth by this count is no gain: up to 5 % slower.)
  const int64_t even = tokens * (3 * (q[0] + q[1]) + 4) / (ctas * kWarps);
  if (per > 1 && best > even + even / 16) {
    const int most = std::max(q[0], q[1]);
    for (int c = 1; c <= kMostChunks && c <= most; ++c) {
      WalkPlan other = r;
      const int64_t last = deal(other, q, (most + c - 1) / c, tokens, ctas);
      if (last + last / 16 >= best) continue;
      best = last;
      r = other;
    }
  }
  if (r.per == 1) r.smem -= kWarps * r.table;  // (as many rows of angles as steps)
  r.rows = by_head(a) ? r.per * rpw : 1;
  r.part_bytes = static_cast<size_t>(r.grid) * r.rows * a.d * sizeof(float);
  return r;
}

template <bool BACK>
cudaError_t launch_walk(const fdma_norm_rope_args& a, const WalkView& p, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  with_layout(a.d, p.v.rot, a.interleaved != 0, [&](auto P, auto L, auto A) {
    constexpr int kP = decltype(P)::value, kL = decltype(L)::value;
    auto run = [&](auto* kern, std::atomic<uint64_t>& ready) {
      e = set_up_once(ready, kern, kSmemPerSm / 2, 0);
      if (e == cudaSuccess) kern<<<p.plan.grid, kThreads, p.plan.smem, stream>>>(p);
    };
    static std::atomic<uint64_t> ready[2];
    if (p.plan.per == 1) run(norm_rope_kernel<kP, kL, decltype(A)::value, true, BACK>, ready[1]);
    else run(norm_rope_kernel<kP, kL, decltype(A)::value, false, BACK>, ready[0]);
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int validate_norm_rope(const fdma_norm_rope_args* a) {
  if (a == nullptr) return FDMA_ERR_INVALID;
  if (a->B < 0 || a->N < 0 || a->Hq <= 0 || a->Hk < 0 || a->d <= 0) return FDMA_ERR_INVALID;
  if (a->d > 256 || a->d % 8 != 0) return FDMA_ERR_UNSUPPORTED;
  if (a->Hq > (1 << 20) || a->Hk > (1 << 20) || static_cast<int64_t>(a->B) * a->N > 0x7fffffff) return FDMA_ERR_UNSUPPORTED;
  if (a->norm != 0 && a->norm != 1) return FDMA_ERR_INVALID;
  if (a->norm && !(std::isfinite(a->eps) && a->eps > 0.f)) return FDMA_ERR_INVALID;
  if (!a->norm && (a->rope == nullptr || a->q_weight != nullptr || a->k_weight != nullptr)) return FDMA_ERR_INVALID;
  if (a->weight_type != FDMA_FP32 && a->weight_type != FDMA_BF16) return FDMA_ERR_INVALID;
  if (a->Hk == 0 && a->k_weight != nullptr) return FDMA_ERR_INVALID;
  for (int i = 0; i < 2; ++i) {
    const void* w = i == 0 ? a->q_weight : a->k_weight;
    const int64_t head = i == 0 ? a->q_weight_head : a->k_weight_head;
    if (head < 0 || (head > 0 && head < a->d) || (w == nullptr && head != 0)) return FDMA_ERR_INVALID;
    if (!aligned16(w) || head % 8 != 0) return FDMA_ERR_UNSUPPORTED;
  }
  // one form for both weights: the parts of their gradients are laid out by it
  if (a->q_weight != nullptr && a->k_weight != nullptr && (a->q_weight_head == 0) != (a->k_weight_head == 0))
    return FDMA_ERR_UNSUPPORTED;
  if (a->interleaved != 0 && a->interleaved != 1) return FDMA_ERR_INVALID;
  if (a->rope != nullptr) {
    if (a->rot <= 0 || a->rot > a->d || a->rope_len < 0) return FDMA_ERR_INVALID;
    if (a->rot % 8 != 0 || !aligned16(a->rope)) return FDMA_ERR_UNSUPPORTED;
  } else if (a->rot != 0 || a->rope_len != 0) {
    return FDMA_ERR_INVALID;
  }
  return FDMA_OK;
}

NormRopeView norm_rope_view(const fdma_norm_rope_args& a) {
  NormRopeView v{};
  v.d = a.d;
  v.rot = a.rope != nullptr ? a.rot : 0;
  v.norm = a.norm;
  v.weight_bf16 = a.weight_type == FDMA_BF16;
  v.eps = a.eps;
  v.inv_d = 1.f / static_cast<float>(a.d);
  v.w[0] = {a.q_weight, a.q_weight_head};
  v.w[1] = {a.k_weight, a.k_weight_head};
  v.rope = a.rope;
  v.rope_len = a.rope_len;
  v.first = a.first;
  v.pos = a.positions;
  v.pos_st[0] = a.pos_stride[0];
  v.pos_st[1] = a.pos_stride[1];
  return v;
}

int validate_rows(const fdma_rows* r, const int64_t n[3], int d, bool written) {
  if (r == nullptr || r->p == nullptr) return FDMA_ERR_INVALID;
  if (!aligned16(r->p)) return FDMA_ERR_UNSUPPORTED;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (r->stride[i] < 0) return FDMA_ERR_INVALID;
    if (r->stride[i] % 8 != 0) return FDMA_ERR_UNSUPPORTED;
  }
  if (!written) return FDMA_OK;
  // from the smallest stride to the largest, each steps over all that the ones before reach
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int i, int j) { return r->stride[i] < r->stride[j]; });
  int64_t extent = d;
  for (int i : order) {
    if (n[i] <= 1) continue;
    if (r->stride[i] < extent) return FDMA_ERR_INVALID;
    extent += (n[i] - 1) * r->stride[i];
  }
  return FDMA_OK;
}

RowsView rows_view(const fdma_rows& r, const int64_t n[3]) {
  RowsView v{static_cast<uint16_t*>(r.p), {}};
  for (int i = 0; i < 3; ++i) v.st[i] = n[i] > 1 ? r.stride[i] : 0;
  return v;
}

namespace {

// Positions and the tokens' limits, where token n of a batch is at first + n.
int validate_positions(const fdma_norm_rope_args& a) {
  if (a.positions != nullptr) return a.pos_stride[0] < 0 || a.pos_stride[1] < 0 ? FDMA_ERR_INVALID : FDMA_OK;
  if (a.rope == nullptr) return FDMA_OK;
  return a.first < 0 || static_cast<int64_t>(a.first) + a.N > a.rope_len ? FDMA_ERR_INVALID : FDMA_OK;
}

void set_sides(const fdma_norm_rope_args& a, WalkView& p) {
  p.v = norm_rope_view(a);
  if (a.positions == nullptr && a.rope == nullptr) p.v.first = 0;
  p.line = {a.N, a.B, static_cast<uint32_t>(a.B) * static_cast<uint32_t>(a.N)};
  p.H[0] = a.Hq;
  p.H[1] = a.Hk;
  p.heads = by_head(a);
  p.pass_l2 = beyond_l2(a);
  for (int s = 0; s < 2; ++s) p.passes[s] = passes_of(p.H[s], pass_rows(a.d, p.v.rot, a.interleaved != 0));
}

int check_sides(const fdma_norm_rope_args& a, const fdma_rows* q, const fdma_rows* k, bool written) {
  const int64_t nq[3] = {a.B, a.N, a.Hq}, nk[3] = {a.B, a.N, a.Hk};
  const int st = validate_rows(q, nq, a.d, written);
  if (st != FDMA_OK || a.Hk == 0) return st;
  return validate_rows(k, nk, a.d, written);
}

void set_rows(const fdma_norm_rope_args& a, RowsView (&to)[2], const fdma_rows* q, const fdma_rows* k) {
  const int64_t nq[3] = {a.B, a.N, a.Hq}, nk[3] = {a.B, a.N, a.Hk};
  to[0] = rows_view(*q, nq);
  if (a.Hk > 0) to[1] = rows_view(*k, nk);
}

}  // namespace
}  // namespace fdma

using namespace fdma;

extern "C" {

int fdma_norm_rope(const fdma_norm_rope_args* a, const fdma_rows* q, const fdma_rows* k, const fdma_rows* q_out,
                   const fdma_rows* k_out, void* stream) {
  int st = validate_norm_rope(a);
  if (st == FDMA_OK) st = validate_positions(*a);
  if (st != FDMA_OK) return st;
  const int64_t tokens = static_cast<int64_t>(a->B) * a->N;
  if (tokens == 0) return FDMA_OK;
  st = check_sides(*a, q, k, false);
  if (st == FDMA_OK) st = check_sides(*a, q_out, k_out, true);
  if (st != FDMA_OK) return st;
  WalkView p{};
  p.plan = walk_plan(*a, false);
  set_sides(*a, p);
  set_rows(*a, p.x, q, k);
  set_rows(*a, p.out, q_out, k_out);
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  return launch_walk<false>(*a, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

size_t fdma_norm_rope_bwd_workspace_size(const fdma_norm_rope_args* a) {
  if (validate_norm_rope(a) != FDMA_OK || static_cast<int64_t>(a->B) * a->N == 0) return 0;
  return walk_plan(*a, true).part_bytes;
}

int fdma_norm_rope_bwd(const fdma_norm_rope_args* a, const fdma_rows* q, const fdma_rows* k, const fdma_rows* dq_out,
                       const fdma_rows* dk_out, const fdma_rows* dq, const fdma_rows* dk, float* dq_weight,
                       float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
  int st = validate_norm_rope(a);
  if (st == FDMA_OK) st = validate_positions(*a);
  if (st != FDMA_OK) return st;
  if ((dq_weight != nullptr && a->q_weight == nullptr) || (dk_weight != nullptr && a->k_weight == nullptr))
    return FDMA_ERR_INVALID;
  const int64_t tokens = static_cast<int64_t>(a->B) * a->N;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {  // no rows: the weights' gradients are zero
    for (int i = 0; i < 2; ++i) {
      float* dw = i == 0 ? dq_weight : dk_weight;
      const int64_t rows = (i == 0 ? a->q_weight_head : a->k_weight_head) != 0 ? (i == 0 ? a->Hq : a->Hk) : 1;
      if (dw != nullptr && cudaMemsetAsync(dw, 0, rows * a->d * sizeof(float), cs) != cudaSuccess) return FDMA_ERR_CUDA;
    }
    return FDMA_OK;
  }
  if (a->norm) st = check_sides(*a, q, k, false);
  if (st == FDMA_OK) st = check_sides(*a, dq_out, dk_out, false);
  if (st == FDMA_OK) st = check_sides(*a, dq, dk, true);
  if (st != FDMA_OK) return st;
  const bool want = dq_weight != nullptr || dk_weight != nullptr;
  const WalkPlan plan = walk_plan(*a, true);
  if (want && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < plan.part_bytes))
    return FDMA_ERR_WORKSPACE;
  WalkView p{};
  p.plan = plan;
  set_sides(*a, p);
  if (a->norm) set_rows(*a, p.x, q, k);
  set_rows(*a, p.g, dq_out, dk_out);
  set_rows(*a, p.out, dq, dk);
  p.part = want ? static_cast<float*>(workspace) : nullptr;
  p.err = paged_error_word();
  if (p.err == nullptr || launch_walk<true>(*a, p, cs) != cudaSuccess) return FDMA_ERR_CUDA;
  if (!want) return FDMA_OK;
  WeightSumView w{};
  w.part = p.part;
  w.dw[0] = dq_weight;
  w.dw[1] = dk_weight;
  w.plan = plan;
  w.d = a->d;
  w.H[0] = a->Hq;
  w.H[1] = a->Hk;
  w.heads = by_head(*a);
  w.rpw = pass_rows(a->d, p.v.rot, a->interleaved != 0);
  const dim3 grid(w.heads ? a->Hq + a->Hk : 2, (a->d + 31) / 32);
  // (launched behind: 8.4 instead of 9.1 us for 771 tokens of 5 + 5 heads)
  return launch_behind(weight_sum_kernel, grid, 1024, cs, w) == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

}  // extern "C"
