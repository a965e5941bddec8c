// A learned bias by buckets of the distance between query and key, and the gradient of
// its table (include/fdma_inputs.h).
//
// Both use that the bias depends on j - i alone.  The matrix is cut into blocks of 8 rows by 8
// columns; a block holds 15 diagonals, and the block one further down and to the right holds the
// same ones.  So a lane that walks down its diagonal of blocks needs 15 values for all of them: the
// forward looks them up once and then only stores (16 bytes a row), the backward adds every element to one
// of 15 sums in registers (one add an element, no atomics) and is done with buckets at the end of its walk.
// The 32 lanes of a warp hold neighbouring blocks, 512 contiguous bytes a row.  A unit of work is
// such a walk of a warp over `walk` block rows; units begin walk - 1 block columns to the left of
// the matrix, so that all of it is covered.
#include "../../include/fdma_inputs.h"
#include "fdma_internal.h"
#include "fdma_ptx.cuh"

namespace fdma {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxLen = 131072;  // as fdma_fwd's
constexpr int kSpan = 32 * 8 + 7;  // diagonals of a warp

struct RelView {
  int H, Nq, Nk, off;
  int n, two_sided;     // buckets of a side
  int walk, nrc, ncc;   // block rows of a unit; units along the rows and the columns
  int starts[FDMA_MAX_BUCKETS];

  __host__ __device__ int buckets() const { return two_sided ? 2 * n : n; }
  // The bucket of a distance.
  __device__ __forceinline__ int side(int a) const {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (starts[mid] <= a) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
  // ... of a difference key - query.  It falls as delta rises to 0, and rises (from n, two-sided) or stays behind
  // it: where both ends of an interval have the same bucket, all of it has.
  __device__ __forceinline__ int bucket(int delta) const {
    if (delta <= 0) return side(-delta);
    return two_sided ? n + side(delta) : side(0);
  }
  // The first diagonal of a unit's first lane.
  __device__ __forceinline__ int first_delta(int rc, int cc) const {
    return 8 * (32 * cc - (walk - 1)) - 8 * walk * rc - off - 7;
  }
};

// ---- forward

struct FwdView {
  RelView r;
  const void* table;
  int table_bf16;
  int64_t ts[2];
  uint16_t* out;
  int64_t os[2];
  int64_t units;
};

__device__ __forceinline__ uint32_t table_value(const FwdView& p, int bucket, int h) {
  const int64_t at = bucket * p.ts[0] + h * p.ts[1];
  if (p.table_bf16) return static_cast<const uint16_t*>(p.table)[at];
  return pack_bf16x2(static_cast<const float*>(p.table)[at], 0.f) & 0xffffu;
}

__global__ void __launch_bounds__(kThreads) rel_bias_kernel(const __grid_constant__ FwdView p) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  const int64_t hr = unit / p.r.ncc;
  const int cc = static_cast<int>(unit - hr * p.r.ncc), h = static_cast<int>(hr / p.r.nrc),
            rc = static_cast<int>(hr - static_cast<int64_t>(h) * p.r.nrc);
  const int lo = p.r.first_delta(rc, cc);
  uint32_t w[14];  // neighbouring diagonals in pairs
  const int b0 = p.r.bucket(lo);
  if (b0 == p.r.bucket(lo + kSpan - 1)) {
    const uint32_t v = table_value(p, b0, h) * 0x10001u;
#pragma unroll
    for (int i = 0; i < 14; ++i) w[i] = v;
  } else {
    uint32_t before = 0;
#pragma unroll
    for (int i = 0; i < 15; ++i) {
      const uint32_t v = table_value(p, p.r.bucket(lo + 8 * lane + i), h);
      if (i > 0) w[i - 1] = before | (v << 16);
      before = v;
    }
  }
  const int rb0 = rc * p.r.walk, nkb = p.r.Nk >> 3;
  int cb = 32 * cc - (p.r.walk - 1) + lane;
  const int rows = min(p.r.Nq - rb0 * 8, p.r.walk * 8);
  uint16_t* at = p.out + h * p.os[0] + static_cast<int64_t>(rb0) * 8 * p.os[1] + static_cast<int64_t>(cb) * 8;
  const int64_t row = p.os[1];
  for (int i = 0; i < rows; i += 8, ++cb, at += 8 * row + 8) {
    if (cb < 0 || cb >= nkb) continue;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (i + r < rows) *reinterpret_cast<uint4*>(at + r * row) = make_uint4(w[7 - r], w[9 - r], w[11 - r], w[13 - r]);
  }
}

// ---- backward

struct BwdView {
  RelView r;
  int B, causal;
  const uint16_t* db;
  int64_t ds[3];
  float* part;  // [unit][bucket]: the sums of the buckets that the unit has
  float* dtable;
  int64_t units;
};

// Of a unit, or a bucket: the diagonals lo .. hi.
struct Deltas {
  int lo, hi;
};
__device__ __forceinline__ Deltas unit_deltas(const BwdView& p, int rc, int cc) {
  Deltas d;
  d.lo = p.r.first_delta(rc, cc);
  d.hi = d.lo + kSpan - 1;
  if (p.causal) d.hi = min(d.hi, 0);
  return d;
}
__device__ __forceinline__ Deltas bucket_deltas(const RelView& r, int bucket) {
  constexpr int kFar = 0x7fffffff;
  const bool right = bucket >= r.n;
  const int s = right ? bucket - r.n : bucket, a0 = r.starts[s], a1 = s + 1 < r.n ? r.starts[s + 1] - 1 : kFar;
  Deltas d;
  if (right) {
    d.lo = max(a0, 1);
    d.hi = a1;
  } else {
    d.lo = -a1;
    d.hi = a0 == 0 && a1 >= 0 && !r.two_sided ? kFar : -a0;
  }
  return d;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__global__ void __launch_bounds__(kThreads) rel_bias_bwd_kernel(const __grid_constant__ BwdView p) {
  __shared__ float diag[kWarps][kSpan + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (unit >= p.units) return;
  const int64_t hr = unit / p.r.ncc, hb = hr / p.r.nrc;
  const int cc = static_cast<int>(unit - hr * p.r.ncc), rc = static_cast<int>(hr - hb * p.r.nrc);
  const int h = static_cast<int>(hb / p.B), b = static_cast<int>(hb - static_cast<int64_t>(h) * p.B);
  const Deltas d = unit_deltas(p, rc, cc);
  if (d.lo > d.hi) return;
  float acc[15];
#pragma unroll
  for (int i = 0; i < 15; ++i) acc[i] = 0.f;
  const int rb0 = rc * p.r.walk, nkb = p.r.Nk >> 3;
  int cb = 32 * cc - (p.r.walk - 1) + lane;
  const int rows = min(p.r.Nq - rb0 * 8, p.r.walk * 8);
  const int64_t row = p.ds[2];
  const uint16_t* at = p.db + b * p.ds[0] + h * p.ds[1] + static_cast<int64_t>(rb0) * 8 * row + static_cast<int64_t>(cb) * 8;
  const bool any = d.lo + 8 * lane <= d.hi;
  for (int i = 0; i < rows; i += 8, ++cb, at += 8 * row + 8) {
    if (!any || cb < 0 || cb >= nkb) continue;
    uint4 v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = i + r < rows ? __ldg(reinterpret_cast<const uint4*>(at + r * row)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[2 * e - r + 7] = add_bf16lo(w[e], acc[2 * e - r + 7]);
        acc[2 * e - r + 8] = add_bf16hi(w[e], acc[2 * e - r + 8]);
      }
    }
  }
  // (a diagonal behind the causal one is dropped, not multiplied: it may hold anything)
#pragma unroll
  for (int i = 0; i < 15; ++i)
    if (d.lo + 8 * lane + i > d.hi) acc[i] = 0.f;
  float* part = p.part + unit * p.r.buckets();
  const int b_lo = p.r.bucket(d.lo);
  if (b_lo == p.r.bucket(d.hi)) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 15; ++i) s += acc[i];
    s = warp_sum(s);
    if (lane == 0) part[b_lo] = s;
    return;
  }
  // diagonal 8 lane + i of the warp: i >= 7 is this lane's, the others are the lane's before, too
  float* x = diag[warp];
  if (lane == 0)
    for (int i = 0; i < 7; ++i) x[i] = 0.f;
#pragma unroll
  for (int i = 7; i < 15; ++i) x[8 * lane + i] = acc[i];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 7; ++i) x[8 * lane + i] += acc[i];
  __syncwarp();
  auto add_bucket = [&](int k) {
    const Deltas q = bucket_deltas(p.r, k);
    const int from = max(q.lo, d.lo) - d.lo, to = min(q.hi, d.hi) - d.lo;
    if (from > to) return;
    float s = 0.f;
    for (int i = from + lane; i <= to; i += 32) s += x[i];
    s = warp_sum(s);
    if (lane == 0) part[k] = s;
  };
  if (d.lo <= 0)
    for (int k = p.r.side(max(-d.hi, 0)); k <= b_lo; ++k) add_bucket(k);
  if (d.hi > 0 && p.r.two_sided) {
    const int last = p.r.side(d.hi);
    for (int k = p.r.side(max(d.lo, 1)); k <= last; ++k) add_bucket(p.r.n + k);
  }
}

// Adds the units' sums of one bucket and head.
__global__ void __launch_bounds__(kThreads) rel_bias_join_kernel(const __grid_constant__ BwdView p) {
  __shared__ double s[kThreads];
  const int k = blockIdx.x % p.r.buckets(), h = blockIdx.x / p.r.buckets();
  const Deltas q = bucket_deltas(p.r, k);
  const int64_t per = static_cast<int64_t>(p.B) * p.r.nrc * p.r.ncc;
  const float* part = p.part + h * per * p.r.buckets() + k;
  double sum = 0.;
  for (int64_t u = threadIdx.x; u < per; u += kThreads) {
    const int64_t r = u / p.r.ncc;
    const Deltas d = unit_deltas(p, static_cast<int>(r % p.r.nrc), static_cast<int>(u - r * p.r.ncc));
    if (max(d.lo, q.lo) <= min(d.hi, q.hi)) sum += part[u * p.r.buckets()];
  }
  s[threadIdx.x] = sum;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) s[threadIdx.x] += s[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) p.dtable[static_cast<int64_t>(k) * p.r.H + h] = static_cast<float>(s[0]);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int validate(const fdma_rel_args* a) {
  if (a == nullptr) return FDMA_ERR_INVALID;
  if (a->H <= 0 || a->Nq < 0 || a->Nk < 0 || a->num_starts <= 0 || a->starts == nullptr) return FDMA_ERR_INVALID;
  if (a->two_sided != 0 && a->two_sided != 1) return FDMA_ERR_INVALID;
  if (a->offset > (1 << 30) || a->offset < -(1 << 30)) return FDMA_ERR_INVALID;
  if (a->num_starts > FDMA_MAX_BUCKETS || a->H > (1 << 20) || a->Nq > kMaxLen || a->Nk > kMaxLen || a->Nk % 8 != 0)
    return FDMA_ERR_UNSUPPORTED;
  if (a->starts[0] != 0) return FDMA_ERR_INVALID;
  for (int i = 1; i < a->num_starts; ++i)
    if (a->starts[i] < a->starts[i - 1]) return FDMA_ERR_INVALID;
  return FDMA_OK;
}

// Units of `most` block rows, fewer where that leaves too few warps for the machine.
RelView view(const fdma_rel_args& a, int64_t batches, int most) {
  RelView r{};
  r.H = a.H;
  r.Nq = a.Nq;
  r.Nk = a.Nk;
  r.off = a.offset;
  r.n = a.num_starts;
  r.two_sided = a.two_sided;
  for (int i = 0; i < r.n; ++i) r.starts[i] = a.starts[i];
  const int nqb = (a.Nq + 7) / 8, nkb = a.Nk / 8;
  for (r.walk = most;; r.walk /= 2) {
    r.nrc = (nqb + r.walk - 1) / r.walk;
    r.ncc = (nkb + r.walk - 1 + 31) / 32;
    if (r.walk == 1 || batches * a.H * r.nrc * r.ncc >= 152 * 16) break;
  }
  return r;
}
constexpr int kFwdWalk = 4, kBwdWalk = 32;

int64_t units_of(const RelView& r, int64_t batches) { return batches * r.H * r.nrc * r.ncc; }

}  // namespace
}  // namespace fdma

using namespace fdma;

extern "C" {

int fdma_rel_bias(const fdma_rel_args* a, const void* table, int table_type, const int64_t ts[2], void* out,
                  const int64_t os[2], void* stream) {
  const int st = validate(a);
  if (st != FDMA_OK) return st;
  if (table == nullptr || ts == nullptr || os == nullptr) return FDMA_ERR_INVALID;
  if (table_type != FDMA_FP32 && table_type != FDMA_BF16) return FDMA_ERR_INVALID;
  if (ts[0] < 0 || ts[1] < 0) return FDMA_ERR_INVALID;
  if (a->Nq == 0 || a->Nk == 0) return FDMA_OK;
  if (out == nullptr || (a->H > 1 && os[0] <= 0) || (a->Nq > 1 && os[1] < a->Nk)) return FDMA_ERR_INVALID;
  if (a->H > 1 && os[0] < (a->Nq - 1) * os[1] + a->Nk && a->Nq > 1 && os[1] < (a->H - 1) * os[0] + a->Nk)
    return FDMA_ERR_INVALID;  // rows that overlap
  if (a->H > 1 && a->Nq == 1 && os[0] < a->Nk) return FDMA_ERR_INVALID;
  if (!aligned16(out) || (a->H > 1 && os[0] % 8 != 0) || (a->Nq > 1 && os[1] % 8 != 0)) return FDMA_ERR_UNSUPPORTED;
  FwdView p{};
  p.r = view(*a, 1, kFwdWalk);
  p.table = table;
  p.table_bf16 = table_type == FDMA_BF16;
  p.out = static_cast<uint16_t*>(out);
  for (int i = 0; i < 2; ++i) {
    p.ts[i] = ts[i];
    p.os[i] = os[i];
  }
  p.units = units_of(p.r, 1);
  const int64_t blocks = (p.units + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return FDMA_ERR_UNSUPPORTED;
  rel_bias_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

size_t fdma_rel_bias_bwd_workspace_size(const fdma_rel_args* a, int B) {
  if (validate(a) != FDMA_OK || B <= 0 || B > (1 << 20) || a->Nq == 0 || a->Nk == 0) return 0;
  const RelView r = view(*a, B, kBwdWalk);
  return static_cast<size_t>(units_of(r, B)) * r.buckets() * sizeof(float);
}

int fdma_rel_bias_bwd(const fdma_rel_args* a, int B, const void* dbias, const int64_t ds[3], int causal, float* dtable,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const int st = validate(a);
  if (st != FDMA_OK) return st;
  if (B < 0 || (causal != 0 && causal != 1) || dtable == nullptr) return FDMA_ERR_INVALID;
  if (B > (1 << 20)) return FDMA_ERR_UNSUPPORTED;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int64_t buckets = static_cast<int64_t>(a->two_sided ? 2 : 1) * a->num_starts;
  if (buckets * a->H > 0x7fffffff) return FDMA_ERR_UNSUPPORTED;
  if (B == 0 || a->Nq == 0 || a->Nk == 0)
    return cudaMemsetAsync(dtable, 0, buckets * a->H * sizeof(float), cs) == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
  if (dbias == nullptr || ds == nullptr) return FDMA_ERR_INVALID;
  const int n[3] = {B, a->H, a->Nq};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (ds[i] < 0) return FDMA_ERR_INVALID;
    if (ds[i] % 8 != 0) return FDMA_ERR_UNSUPPORTED;
  }
  if (!aligned16(dbias)) return FDMA_ERR_UNSUPPORTED;
  BwdView p{};
  p.r = view(*a, B, kBwdWalk);
  p.units = units_of(p.r, B);
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < static_cast<size_t>(p.units) * buckets * sizeof(float))
    return FDMA_ERR_WORKSPACE;
  p.B = B;
  p.causal = causal;
  p.db = static_cast<const uint16_t*>(dbias);
  for (int i = 0; i < 3; ++i) p.ds[i] = ds[i];
  p.part = static_cast<float*>(workspace);
  p.dtable = dtable;
  const int64_t blocks = (p.units + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return FDMA_ERR_UNSUPPORTED;
  rel_bias_bwd_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, cs>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FDMA_ERR_CUDA;
  rel_bias_join_kernel<<<static_cast<unsigned>(buckets * a->H), kThreads, 0, cs>>>(p);
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

}  // extern "C"
