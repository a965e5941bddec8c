// Norms of queries and keys for each head and the rotation of their positions, forward and
// backward (include/fdma_inputs.h).
//
// Forward.  All rows of a call (token, head of q or k) form one line of which a warp takes
// ROWS times those that its lanes hold at once; each row is read once and written once.
//
// Backward.  With g the gradient of the output turned back, r = 1 / sqrt(mean(x^2) + eps) and
// S = sum(g w x):  dx = r g w - x r^3 S / d,  dw = sum over tokens of g x r.
// The rows are dealt to slots, each of which keeps one head and walks over tokens, so
// that a weight's gradient is summed in registers; a CTA adds its slots in a fixed order and
// writes one part for each weight row that it has, and a second kernel adds the parts.
#include <cmath>

#include "fdma_norm_rope.cuh"

namespace fdma {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 4;     // rows of a lane
constexpr int kBwdCtas = 304;

struct FwdView {
  NormRopeView v;
  int H, Hq, N;  // heads of q and k together
  int batches;   // 1: tokens are one line
  int64_t tokens;
  RowsView in[2], out[2];
  int* err;
};

__device__ __forceinline__ int64_t row_at(const RowsView& r, int b, int n, int h) {
  return b * r.st[0] + n * r.st[1] + h * r.st[2];
}

// One row of the line.
struct RowId {
  int b, n, h, side;
  bool real;
};

__device__ __forceinline__ void split_token(int64_t tok, int N, int batches, int& b, int& n) {
  b = 0;
  n = static_cast<int>(tok);
  if (batches > 1) {
    b = static_cast<int>(static_cast<uint32_t>(tok) / static_cast<uint32_t>(N));
    n = static_cast<int>(tok) - b * N;
  }
}

// Position of a token before it is checked.
__device__ __forceinline__ int position_of(const NormRopeView& v, int b, int n) {
  return v.pos != nullptr ? v.pos[b * v.pos_st[0] + n * v.pos_st[1]] : v.first + n;
}

template <int LPR, bool ADJ>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ FwdView p) {
  constexpr int RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * (RPW * kRows);
  const int64_t tok0 = first / p.H;
  if (tok0 >= p.tokens) return;
  const int rem = static_cast<int>(first - tok0 * p.H);
  const Lane at = lane_of<ADJ>(p.v, l);
  RowId id[kRows];
  Raw raw[kRows];
  int pos[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    RowId& r = id[i];
    const int x = rem + i * RPW + lane / LPR, t = x / p.H;
    r.h = x - t * p.H;
    r.side = r.h >= p.Hq ? 1 : 0;
    if (r.side) r.h -= p.Hq;
    r.real = tok0 + t < p.tokens;
    split_token(tok0 + t, p.N, p.batches, r.b, r.n);
    raw[i] = Raw{};
    pos[i] = -1;
    if (!r.real) continue;
    const RowsView& s = p.in[r.side];
    if (at.in) raw[i] = load_raw<ADJ>(s.p + row_at(s, r.b, r.n, r.h), at);
    pos[i] = position_of(p.v, r.b, r.n);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const RowId& r = id[i];
    const int q = r.real ? checked_position(p.v, pos[i], p.err) : -1;
    const Turn t = load_turn(p.v, max(q, 0), l, at);
    const Pairs w = load_weight<ADJ>(p.v, r.side, r.h, at);
    Pairs x = widen<ADJ>(raw[i]);
    norm_and_turn<LPR>(p.v, x, w, t, at);
    const RowsView& o = p.out[r.side];
    if (q >= 0 && at.in) store_raw<ADJ>(o.p + row_at(o, r.b, r.n, r.h), at, narrow<ADJ>(x));
  }
}

struct BwdView {
  NormRopeView v;
  int H, Hq, N, batches;
  int64_t tokens;
  int par, steps;  // tokens side by side; tokens of a slot
  RowsView in[2], dout[2], din[2];
  float* part;  // [cta][rows of a CTA][d]; nullptr: no weight's gradient
  int part_rows;
  int by_head;
  int* err;
};

// Slots of a CTA: they keep heads (first slot of the CTA + j) % H.
template <int LPR>
constexpr int kCtaSlots = kWarps * (32 / LPR) * kRows;

template <int LPR, bool ADJ>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_bwd_kernel(const __grid_constant__ BwdView p) {
  constexpr int RPW = 32 / LPR, SLOTS = kCtaSlots<LPR>, COLS = LPR * 8;
  __shared__ float sums[SLOTS * COLS];
  const int lane = threadIdx.x & 31, l = lane % LPR, warp = threadIdx.x >> 5;
  const Lane at = lane_of<ADJ>(p.v, l);
  const int slot0 = blockIdx.x * SLOTS;
  Pairs acc[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i].a[e] = acc[i].b[e] = 0.f;
  for (int k = 0; k < p.steps; ++k) {
    RowId id[kRows];
    Raw xr[kRows], gr[kRows];
    int pos[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      RowId& r = id[i];
      const int s = slot0 + (warp * kRows + i) * RPW + lane / LPR, t = s / p.H;
      const int64_t tok = t + static_cast<int64_t>(k) * p.par;
      r.h = s - t * p.H;
      r.side = r.h >= p.Hq ? 1 : 0;
      if (r.side) r.h -= p.Hq;
      r.real = t < p.par && tok < p.tokens;
      split_token(tok, p.N, p.batches, r.b, r.n);
      xr[i] = gr[i] = Raw{};
      pos[i] = -1;
      if (!r.real) continue;
      const RowsView &sx = p.in[r.side], &sg = p.dout[r.side];
      if (at.in) {
        if (p.v.norm) xr[i] = load_raw<ADJ>(sx.p + row_at(sx, r.b, r.n, r.h), at);
        gr[i] = load_raw<ADJ>(sg.p + row_at(sg, r.b, r.n, r.h), at);
      }
      pos[i] = position_of(p.v, r.b, r.n);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const RowId& r = id[i];
      const int q = r.real ? checked_position(p.v, pos[i], p.err) : -1;
      if (q < 0) gr[i] = xr[i] = Raw{};  // left out: no gradient (not even from values that are not finite)
      const Turn t = load_turn(p.v, max(q, 0), l, at);
      Pairs g = widen<ADJ>(gr[i]);
      turn<true>(g, t, at);
      if (p.v.norm) {
        const Pairs w = load_weight<ADJ>(p.v, r.side, r.h, at);
        Pairs x = widen<ADJ>(xr[i]);
        float scale;
        const float rs = row_rsqrt<LPR>(p.v, x, scale);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x.a[e] *= rs;
          x.b[e] *= rs;
          acc[i].a[e] += g.a[e] * x.a[e];
          acc[i].b[e] += g.b[e] * x.b[e];
          g.a[e] *= w.a[e];
          g.b[e] *= w.b[e];
          dot += g.a[e] * x.a[e] + g.b[e] * x.b[e];
        }
        // with xn = x r:  dx = r (g w - xn mean(g w xn))
        dot = row_sum<LPR>(dot) * p.v.inv_d;
        const float f = rs * scale;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g.a[e] = f * (g.a[e] - x.a[e] * dot);
          g.b[e] = f * (g.b[e] - x.b[e] * dot);
        }
      }
      const RowsView& o = p.din[r.side];
      if (r.real && at.in) store_raw<ADJ>(o.p + row_at(o, r.b, r.n, r.h), at, q < 0 ? Raw{} : narrow<ADJ>(g));
    }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float* s = sums + ((warp * kRows + i) * RPW + lane / LPR) * COLS;
    if (!at.in) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[ADJ ? at.ca + 2 * e : at.ca + e] = acc[i].a[e];
      s[ADJ ? at.ca + 2 * e + 1 : at.cb + e] = acc[i].b[e];
    }
  }
  __syncthreads();
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.part_rows * p.v.d;
  for (int x = threadIdx.x; x < p.part_rows * p.v.d; x += kThreads) {
    const int row = x / p.v.d, c = x - row * p.v.d;
    float sum = 0.f;
    if (p.by_head) {  // the slots of one head
      for (int j = row; j < SLOTS; j += p.H) sum += sums[j * COLS + c];
    } else {  // those of q (row 0) or k
      int h = slot0 % p.H;
      for (int j = 0; j < SLOTS; ++j) {
        if ((h >= p.Hq) == (row == 1)) sum += sums[j * COLS + c];
        if (++h == p.H) h = 0;
      }
    }
    out[x] = sum;
  }
}

struct WeightSumView {
  const float* part;
  float* dw[2];
  int ctas, part_rows, slots, d, H, Hq, by_head;
};

// Adds the CTAs' parts: block (row of the weights, 32 columns) of 32 x 8 threads.
__global__ void __launch_bounds__(256) weight_sum_kernel(const WeightSumView p) {
  __shared__ float s[8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.y * 32 + tx, row = blockIdx.x;
  const int side = p.by_head ? row >= p.Hq : row, h = p.by_head ? row - side * p.Hq : 0;
  if (p.dw[side] == nullptr) return;
  float sum = 0.f;
  if (c < p.d) {
    for (int b = ty; b < p.ctas; b += 8) {
      int at = row;
      if (p.by_head) {  // where this CTA has the head
        at = row - static_cast<int>(static_cast<int64_t>(b) * p.slots % p.H);
        if (at < 0) at += p.H;
        if (at >= p.part_rows) continue;
      }
      sum += p.part[(static_cast<int64_t>(b) * p.part_rows + at) * p.d + c];
    }
  }
  s[ty][tx] = sum;
  __syncthreads();
  if (ty != 0 || c >= p.d) return;
  for (int j = 1; j < 8; ++j) sum += s[j][tx];
  p.dw[side][static_cast<int64_t>(h) * p.d + c] = sum;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int lanes_of(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }

struct BwdPlan {
  int par, steps, ctas, slots, part_rows;
  size_t bytes;
};

BwdPlan bwd_plan(const fdma_norm_rope_args& a) {
  BwdPlan r{};
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N, H = a.Hq + a.Hk;
  r.slots = kWarps * (32 / lanes_of(a.d)) * kRows;
  int64_t par = kBwdCtas * r.slots / H;
  par = par < 1 ? 1 : par > tokens ? tokens : par;
  r.steps = static_cast<int>((tokens + par - 1) / par);
  r.par = static_cast<int>((tokens + r.steps - 1) / r.steps);
  r.ctas = static_cast<int>((r.par * H + r.slots - 1) / r.slots);
  const bool by_head = a.q_weight_head != 0 || a.k_weight_head != 0;
  r.part_rows = !by_head ? 2 : H < r.slots ? static_cast<int>(H) : r.slots;
  r.bytes = static_cast<size_t>(r.ctas) * r.part_rows * a.d * sizeof(float);
  return r;
}

template <typename F>
void with_lanes(int d, bool adj, F&& f) {
  using std::integral_constant;
  using T = integral_constant<bool, true>;
  using N = integral_constant<bool, false>;
  if (d <= 64) adj ? f(integral_constant<int, 8>{}, T{}) : f(integral_constant<int, 8>{}, N{});
  else if (d <= 128) adj ? f(integral_constant<int, 16>{}, T{}) : f(integral_constant<int, 16>{}, N{});
  else adj ? f(integral_constant<int, 32>{}, T{}) : f(integral_constant<int, 32>{}, N{});
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
  p.H = a->Hq + a->Hk;
  p.Hq = a->Hq;
  p.N = a->N;
  p.tokens = tokens;
  p.in[0] = rows_view(*q);
  p.out[0] = rows_view(*q_out);
  if (a->Hk > 0) {
    p.in[1] = rows_view(*k);
    p.out[1] = rows_view(*k_out);
  }
  p.batches = a->B;
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  const int per = kWarps * (32 / lanes_of(a->d)) * kRows;
  const int64_t blocks = (tokens * p.H + per - 1) / per;
  if (blocks > 0x7fffffff) return FDMA_ERR_UNSUPPORTED;
  with_lanes(a->d, a->interleaved != 0, [&](auto L, auto A) {
    norm_rope_kernel<decltype(L)::value, decltype(A)::value>
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
  p.H = a->Hq + a->Hk;
  p.Hq = a->Hq;
  p.N = a->N;
  p.tokens = tokens;
  p.batches = a->B;
  p.par = plan.par;
  p.steps = plan.steps;
  p.dout[0] = rows_view(*dq_out);
  p.din[0] = rows_view(*dq);
  if (a->norm) p.in[0] = rows_view(*q);
  if (a->Hk > 0) {
    p.dout[1] = rows_view(*dk_out);
    p.din[1] = rows_view(*dk);
    if (a->norm) p.in[1] = rows_view(*k);
  }
  p.part = want ? static_cast<float*>(workspace) : nullptr;
  p.part_rows = plan.part_rows;
  p.by_head = a->q_weight_head != 0 || a->k_weight_head != 0;
  p.err = paged_error_word();
  if (p.err == nullptr) return FDMA_ERR_CUDA;
  with_lanes(a->d, a->interleaved != 0, [&](auto L, auto A) {
    norm_rope_bwd_kernel<decltype(L)::value, decltype(A)::value><<<plan.ctas, kThreads, 0, cs>>>(p);
  });
  if (cudaGetLastError() != cudaSuccess) return FDMA_ERR_CUDA;
  if (!want) return FDMA_OK;
  WeightSumView w{};
  w.part = p.part;
  w.dw[0] = dq_weight;
  w.dw[1] = dk_weight;
  w.ctas = plan.ctas;
  w.part_rows = plan.part_rows;
  w.slots = plan.slots;
  w.d = a->d;
  w.H = p.H;
  w.Hq = p.Hq;
  w.by_head = p.by_head;
  const dim3 grid(p.by_head ? p.H : 2, (a->d + 31) / 32);
  weight_sum_kernel<<<grid, 256, 0, cs>>>(w);
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

}  // extern "C"
