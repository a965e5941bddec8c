// Norms of queries and keys for each head and the rotation of their positions, forward and
// backward (include/fdma_inputs.h).
//
// Forward.  A warp takes a token, or a run of its passes where there are few tokens; position,
// angles and weights are looked up once for all of its rows, and each row is read once and written once.
//
// Backward.  With g the gradient of the output turned back, r = 1 / sqrt(mean(x^2) + eps), xn = x r:
//   dx = r (g w - xn mean(g w xn)),  dw = sum over tokens (and heads that share it) of g xn.
// A CTA keeps a chunk of one tensor's heads (one pass where every head has a weight of its own) and its warps walk
// over tokens, so that a lane has one weight and sums one gradient, in registers; the CTA adds its warps' sums in a
// fixed order and writes one part, and a second kernel adds the parts of a weight.
#include <cmath>

#include "fdma_norm_rope.cuh"

namespace fdma {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBwdCtas = 304;

struct TokenLine {
  int N, batches;  // batches 1: tokens are one line
  int64_t tokens;
};

__device__ __forceinline__ void split_token(const TokenLine& t, int64_t tok, int& b, int& n) {
  b = 0;
  n = static_cast<int>(tok);
  if (t.batches > 1) {
    b = static_cast<int>(static_cast<uint32_t>(tok) / static_cast<uint32_t>(t.N));
    n = static_cast<int>(tok) - b * t.N;
  }
}

// Position of a token before it is checked.
__device__ __forceinline__ int position_of(const NormRopeView& v, int b, int n) {
  return v.pos != nullptr ? v.pos[b * v.pos_st[0] + n * v.pos_st[1]] : v.first + n;
}

__device__ __forceinline__ uint16_t* token_rows(const RowsView& r, int b, int n) { return r.p + b * r.st[0] + n * r.st[1]; }

struct FwdView {
  NormRopeView v;
  TokenLine line;
  int H[2], passes_q;
  PassPlan plan;
  RowsView in[2], out[2];
  int* err;
};

// Passes of a warp that are on their way at once: 6 KB.
template <int P>
constexpr int kFwdSlots = 48 / P;

template <int P, int LPR, bool ADJ>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(const __grid_constant__ FwdView p) {
  constexpr int RPW = 32 / LPR, SLOTS = kFwdSlots<P>;
  __shared__ __align__(16) uint8_t rings[kWarps][SLOTS * Ring<P>::kSlot];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, g = lane / LPR;
  const uint32_t w = blockIdx.x * kWarps + warp;
  uint32_t tok = w, c = 0;
  if (p.plan.chunks > 1) {
    tok = w / p.plan.chunks;
    c = w - tok * p.plan.chunks;
  }
  if (tok >= p.line.tokens) return;
  int b, n;
  split_token(p.line, tok, b, n);
  const Lane at = lane_of<P, ADJ>(p.v, l);
  const Ring<P> ring(smem_u32(rings[warp]), lane);
  const int q0 = static_cast<int>(c) * p.plan.per, q1 = min(q0 + p.plan.per, p.plan.passes);
  auto start = [&](int q, int slot) {
    if (q < q1) {
      const int side = q >= p.passes_q, h = (q - (side ? p.passes_q : 0)) * RPW + g;
      const bool real = at.in && h < p.H[side];
      ring.copy(slot, token_rows(p.in[side], b, n) + (real ? h * p.in[side].st[2] : 0), at, real);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) start(q0 + i, i);
  const int pos = checked_position(p.v, position_of(p.v, b, n), p.err);
  if (pos < 0) {
    cp_async_wait_all();
    return;
  }
  const Turn<P> t = load_turn<P>(p.v, pos, l, at);
  Pairs<P> wt;
  int have = -1;  // the tensor whose weight wt holds
  int slot = 0;
  for (int q = q0; q < q1; ++q) {
    const int side = q >= p.passes_q, h = (q - (side ? p.passes_q : 0)) * RPW + g;
    const bool real = at.in && h < p.H[side];
    if (side != have || p.v.w[side].head != 0) {
      wt = load_weight<P, ADJ>(p.v, side, real ? h : 0, at);
      have = side;
    }
    cp_async_wait<SLOTS - 1>();
    Pairs<P> x = widen<P, ADJ>(ring.get(slot));
    norm_and_turn<LPR>(p.v, x, wt, t, at);
    if (real) store_raw<P>(token_rows(p.out[side], b, n) + h * p.out[side].st[2], at, narrow<P, ADJ>(x));
    start(q + SLOTS, slot);
    slot = slot + 1 == SLOTS ? 0 : slot + 1;
  }
}

// How the backward deals out its work: tensor s (q, k) has chunks[s] chunks of `per` passes (the last of fewer), each
// with ctas[s] CTAs.
struct BwdPlan {
  int per, chunks[2], ctas[2], grid;
  int rows;  // weight rows of a CTA's part
  size_t bytes;
};

struct BwdView {
  NormRopeView v;
  TokenLine line;
  int H[2], passes[2];
  BwdPlan plan;
  RowsView in[2], dout[2], din[2];
  float* part;  // [cta][plan.rows][d]; nullptr: no weight's gradient
  int* err;
};

template <int P>
__device__ __forceinline__ void put_columns(float* s, const Pairs<P>& x, const Lane& at, bool adj) {
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    float a0, a1, b0, b1;
    f2split(x.a[i], a0, a1);
    f2split(x.b[i], b0, b1);
    s[adj ? at.ca + 4 * i : at.ca + 2 * i] = a0;
    s[adj ? at.ca + 4 * i + 2 : at.ca + 2 * i + 1] = a1;
    s[adj ? at.ca + 4 * i + 1 : at.cb + 2 * i] = b0;
    s[adj ? at.ca + 4 * i + 3 : at.cb + 2 * i + 1] = b1;
  }
}

// Steps of a warp (a pass of the gradients and of the rows) that are on their way at once: 6 KB.
template <int P>
constexpr int kBwdSlots = 24 / P;

// HEADS: every head has a weight of its own.
template <int P, int LPR, bool ADJ, bool HEADS>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_bwd_kernel(const __grid_constant__ BwdView p) {
  constexpr int RPW = 32 / LPR, COLS = 2 * P * LPR, SLOTS = kBwdSlots<P>;
  __shared__ __align__(16) uint8_t rings[kWarps][2 * SLOTS * Ring<P>::kSlot];
  static_assert(sizeof(rings) >= kWarps * RPW * COLS * sizeof(float), "the sums take the rings' place");
  const int lane = threadIdx.x & 31, l = lane % LPR, g = lane / LPR, warp = threadIdx.x >> 5;
  int cta = blockIdx.x;
  const int side = cta >= p.plan.chunks[0] * p.plan.ctas[0];
  if (side) cta -= p.plan.chunks[0] * p.plan.ctas[0];
  const int chunk = cta / p.plan.ctas[side];
  const int q_first = chunk * p.plan.per, q_last = min(q_first + p.plan.per, p.passes[side]), H = p.H[side];
  const Lane at = lane_of<P, ADJ>(p.v, l);
  const RowsView in = p.in[side], dout = p.dout[side], din = p.din[side];
  const int64_t step = static_cast<int64_t>(p.plan.ctas[side]) * kWarps;
  const int64_t tok0 = (cta - chunk * p.plan.ctas[side]) * kWarps + warp;
  const Ring<P> ring(smem_u32(rings[warp]), lane);
  // what is fetched next
  int64_t tok_next = tok0;
  int q_next = q_first;
  const uint16_t *x_next = nullptr, *g_next = nullptr;
  auto start = [&](int slot) {
    if (tok_next < p.line.tokens) {
      if (q_next == q_first) {
        int b, n;
        split_token(p.line, tok_next, b, n);
        x_next = token_rows(in, b, n);
        g_next = token_rows(dout, b, n);
      }
      const int h = q_next * RPW + g;
      const bool real = at.in && h < H;
      if (p.v.norm) ring.copy(2 * slot, x_next + (real ? h * in.st[2] : 0), at, real);
      ring.copy(2 * slot + 1, g_next + (real ? h * dout.st[2] : 0), at, real);
      if (++q_next == q_last) {
        q_next = q_first;
        tok_next += step;
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) start(i);
  Pairs<P> acc;
#pragma unroll
  for (int e = 0; e < P / 2; ++e) acc.a[e] = acc.b[e] = 0;
  const Pairs<P> wt = load_weight<P, ADJ>(p.v, side, HEADS ? min(q_first * RPW + g, H - 1) : 0, at);
  int slot = 0;
  for (int64_t tok = tok0; tok < p.line.tokens; tok += step) {
    int b, n;
    split_token(p.line, tok, b, n);
    const int pos = checked_position(p.v, position_of(p.v, b, n), p.err);
    const Turn<P> t = load_turn<P>(p.v, max(pos, 0), l, at);
    uint16_t* o_at = token_rows(din, b, n);
    for (int q = q_first; q < q_last; ++q) {
      const int h = q * RPW + g;
      const bool real = at.in && h < H;
      cp_async_wait<SLOTS - 1>();
      // a token that is left out has no gradient, whatever it holds
      Pairs<P> d = widen<P, ADJ>(pos >= 0 ? ring.get(2 * slot + 1) : no_raw<P>());
      if (p.v.norm) {
        Pairs<P> x = widen<P, ADJ>(pos >= 0 ? ring.get(2 * slot) : no_raw<P>());
        float by;
        const float r = row_rsqrt<LPR>(p.v, x, by);
        turn<true>(d, t, at);
        // e = g r:  dw += e x,  dx = e w - x r^2 mean(e w x)   (of a scaled row: times `by`)
        scale(d, r);
#pragma unroll
        for (int e = 0; e < P / 2; ++e) {
          acc.a[e] = fma2(d.a[e], x.a[e], acc.a[e]);
          acc.b[e] = fma2(d.b[e], x.b[e], acc.b[e]);
        }
        multiply(d, wt);
        const float m = row_sum<LPR>(dot(d, x)) * p.v.inv_d * (-r * r);
        const uint64_t m2 = f2(m, m);
#pragma unroll
        for (int e = 0; e < P / 2; ++e) {
          d.a[e] = fma2(x.a[e], m2, d.a[e]);
          d.b[e] = fma2(x.b[e], m2, d.b[e]);
        }
        if (__any_sync(0xffffffffu, by != 1.f)) scale(d, by);
      } else {
        turn<true>(d, t, at);
      }
      if (real) store_raw<P>(o_at + h * din.st[2], at, pos < 0 ? no_raw<P>() : narrow<P, ADJ>(d));
      start(slot);
      slot = slot + 1 == SLOTS ? 0 : slot + 1;
    }
  }
  cp_async_wait_all();
  if (p.part == nullptr) return;
  __syncthreads();
  float* sums = reinterpret_cast<float*>(rings);  // [warp][row of a pass][column]
  if (at.in) put_columns(sums + (warp * RPW + g) * COLS, acc, at, ADJ);
  __syncthreads();
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.plan.rows * p.v.d;
  for (int x = threadIdx.x; x < p.plan.rows * p.v.d; x += kThreads) {
    const int row = x / p.v.d, c = x - row * p.v.d;
    float sum = 0.f;
    for (int j = 0; j < kWarps; ++j) {
      if (HEADS) {
        sum += sums[(j * RPW + row) * COLS + c];
      } else {
#pragma unroll
        for (int k = 0; k < RPW; ++k) sum += sums[(j * RPW + k) * COLS + c];
      }
    }
    out[x] = sum;
  }
}

struct WeightSumView {
  const float* part;
  float* dw[2];
  BwdPlan plan;
  int d, H[2], heads, rpw;
};

// Adds the CTAs' parts: block (row of the weights, 32 columns) of 32 x 32 threads.
__global__ void __launch_bounds__(1024) weight_sum_kernel(const __grid_constant__ WeightSumView p) {
  __shared__ float s[32][33];
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

BwdPlan bwd_plan(const fdma_norm_rope_args& a) {
  BwdPlan r{};
  const int rot = a.rope != nullptr ? a.rot : 0, rpw = pass_rows(a.d, rot);
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  const int q[2] = {passes_of(a.Hq, rpw), passes_of(a.Hk, rpw)};
  r.per = by_head(a) ? 1 : plan_passes(q[0] + q[1], tokens, kBwdCtas * kWarps).per;
  int64_t cost = 0;  // of a token, the last chunks counted as whole ones
  for (int s = 0; s < 2; ++s) {
    r.chunks[s] = (q[s] + r.per - 1) / r.per;
    cost += static_cast<int64_t>(r.chunks[s]) * (q[s] < r.per ? q[s] : r.per);
  }
  const int64_t most_ctas = (tokens + kWarps - 1) / kWarps;
  for (int s = 0; s < 2; ++s) {
    const int64_t n = kBwdCtas * static_cast<int64_t>(q[s] < r.per ? q[s] : r.per) / cost;
    r.ctas[s] = static_cast<int>(n < 1 ? 1 : n > most_ctas ? most_ctas : n);
    r.grid += r.chunks[s] * r.ctas[s];
  }
  r.rows = by_head(a) ? r.per * rpw : 1;
  r.bytes = static_cast<size_t>(r.grid) * r.rows * a.d * sizeof(float);
  return r;
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

int validate_rows(const fdma_rows* r, const int64_t n[3], bool written) {
  if (r == nullptr || r->p == nullptr) return FDMA_ERR_INVALID;
  if (!aligned16(r->p)) return FDMA_ERR_UNSUPPORTED;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (r->stride[i] < 0 || (written && r->stride[i] == 0)) return FDMA_ERR_INVALID;
    if (r->stride[i] % 8 != 0) return FDMA_ERR_UNSUPPORTED;
  }
  return FDMA_OK;
}

RowsView rows_view(const fdma_rows& r) {
  return {static_cast<uint16_t*>(r.p), {r.stride[0], r.stride[1], r.stride[2]}};
}

namespace {

// Positions and the tokens' limits, where token n of a batch is at first + n.
int validate_positions(const fdma_norm_rope_args& a) {
  if (a.positions != nullptr) return a.pos_stride[0] < 0 || a.pos_stride[1] < 0 ? FDMA_ERR_INVALID : FDMA_OK;
  if (a.rope == nullptr) return FDMA_OK;
  return a.first < 0 || static_cast<int64_t>(a.first) + a.N > a.rope_len ? FDMA_ERR_INVALID : FDMA_OK;
}

int check_sides(const fdma_norm_rope_args& a, const fdma_rows* q, const fdma_rows* k, bool written) {
  const int64_t nq[3] = {a.B, a.N, a.Hq}, nk[3] = {a.B, a.N, a.Hk};
  const int st = validate_rows(q, nq, written);
  if (st != FDMA_OK || a.Hk == 0) return st;
  return validate_rows(k, nk, written);
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
  FwdView p{};
  p.v = norm_rope_view(*a);
  if (a->positions == nullptr && a->rope == nullptr) p.v.first = 0;
  p.line = {a->N, a->B, tokens};
  p.H[0] = a->Hq;
  p.H[1] = a->Hk;
  p.in[0] = rows_view(*q);
  p.out[0] = rows_view(*q_out);
  if (a->Hk > 0) {
    p.in[1] = rows_view(*k);
    p.out[1] = rows_view(*k_out);
  }
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  const int rpw = pass_rows(a->d, p.v.rot);
  p.passes_q = passes_of(a->Hq, rpw);
  p.plan = plan_passes(p.passes_q + passes_of(a->Hk, rpw), tokens, 152 * 32);
  const int64_t blocks = (tokens * p.plan.chunks + kWarps - 1) / kWarps;
  if (blocks * kWarps > 0xffffffffll) return FDMA_ERR_UNSUPPORTED;
  with_layout(a->d, p.v.rot, a->interleaved != 0, [&](auto P, auto L, auto A) {
    norm_rope_kernel<decltype(P)::value, decltype(L)::value, decltype(A)::value>
        <<<static_cast<unsigned>(blocks), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  });
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

size_t fdma_norm_rope_bwd_workspace_size(const fdma_norm_rope_args* a) {
  if (validate_norm_rope(a) != FDMA_OK || static_cast<int64_t>(a->B) * a->N == 0) return 0;
  return bwd_plan(*a).bytes;
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
  const BwdPlan plan = bwd_plan(*a);
  if (want && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < plan.bytes))
    return FDMA_ERR_WORKSPACE;
  BwdView p{};
  p.v = norm_rope_view(*a);
  if (a->positions == nullptr && a->rope == nullptr) p.v.first = 0;
  p.line = {a->N, a->B, tokens};
  p.plan = plan;
  const int rpw = pass_rows(a->d, p.v.rot);
  p.H[0] = a->Hq;
  p.H[1] = a->Hk;
  for (int s = 0; s < 2; ++s) p.passes[s] = passes_of(p.H[s], rpw);
  p.dout[0] = rows_view(*dq_out);
  p.din[0] = rows_view(*dq);
  if (a->norm) p.in[0] = rows_view(*q);
  if (a->Hk > 0) {
    p.dout[1] = rows_view(*dk_out);
    p.din[1] = rows_view(*dk);
    if (a->norm) p.in[1] = rows_view(*k);
  }
  p.part = want ? static_cast<float*>(workspace) : nullptr;
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  const bool heads = by_head(*a);
  with_layout(a->d, p.v.rot, a->interleaved != 0, [&](auto P, auto L, auto A) {
    if (heads) norm_rope_bwd_kernel<decltype(P)::value, decltype(L)::value, decltype(A)::value, true><<<plan.grid, kThreads, 0, cs>>>(p);
    else norm_rope_bwd_kernel<decltype(P)::value, decltype(L)::value, decltype(A)::value, false><<<plan.grid, kThreads, 0, cs>>>(p);
  });
  if (cudaGetLastError() != cudaSuccess) return FDMA_ERR_CUDA;
  if (!want) return FDMA_OK;
  WeightSumView w{};
  w.part = p.part;
  w.dw[0] = dq_weight;
  w.dw[1] = dk_weight;
  w.plan = plan;
  w.d = a->d;
  w.H[0] = a->Hq;
  w.H[1] = a->Hk;
  w.heads = heads;
  w.rpw = rpw;
  const dim3 grid(heads ? a->Hq + a->Hk : 2, (a->d + 31) / 32);
  weight_sum_kernel<<<grid, 1024, 0, cs>>>(w);
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

}  // extern "C"
