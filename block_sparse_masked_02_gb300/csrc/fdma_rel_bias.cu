// A learned bias by buckets of the distance between query and key, and the gradient of
// its table (include/fdma_inputs.h).
//
// Both use that the bias depends on j - i alone.  The matrix is cut into blocks of 8 rows by 8
// columns, one a lane: a block holds 15 diagonals, and the 32 neighbouring blocks of a warp 263 (512
// contiguous bytes a row).  The forward looks up a block's 15 values and stores 16 bytes a row.
//
// Backward.  The block one further down and to the right holds the same diagonals, so a lane that walks down
// its diagonal of blocks adds every element to one of 15 sums in registers: one add an element, no atomics, and buckets
// only at the end of the walk.  A band is the 32 neighbouring diagonals of blocks that a warp walks along; its block rows
// are dealt out to `parts` warps in turn (warp p takes p, p + parts, ...), so that all warps sweep
// over the matrix together and DRAM sees neighbouring rows.  A CTA's warps have eight parts of a band; it
// joins their sums and writes one number where the whole band is in one bucket, as far from the diagonal nearly all are,
// else the sums of the band's diagonals.  A second kernel adds what each bucket has of those, in a fixed order.
// Bound by reading: the causal half of four heads of 16384 x 16384 (1.07 GB) takes 170 us, 6.3 TB/s, 5 us of it the second kernel;
// 55 MB in 3 x 6 heads 16 us, of which that is 3 and start and end of 540 CTAs of five block rows a warp most of the rest.
// (Block rows of a unit one after the other, 512 rows of a matrix apart from the next unit's: 376 us.)
#include "../../include/fdma_inputs.h"
#include "fdma_internal.h"
#include "fdma_ptx.cuh"

namespace fdma {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxLen = 131072;  // as fdma_fwd's
constexpr int kSpan = 32 * 8 + 7;  // diagonals of a warp
constexpr int kPart = 264;
constexpr int64_t kMostCtas = 1 << 28;  // of a backward (their parts take 283 GB)
// Block rows of a backward walk, and the CTAs that a call should have if its walks get shorter for it.  (Four causal heads of
// 16384 x 16384 / 3 x 6 of 1001 x 1528, us: 8 steps 175 / 15.9, 16: 171 / 15.9, 24: 175 / 16.3; 600 CTAs 172 / 18.3, 150: 172 / 22.)
constexpr int kBwdSteps = 16, kBwdCtas = 456;

struct RelView {
  int H, Nq, Nk, off;
  int n, two_sided;  // buckets of a side
  int top;           // the power of two that a search over them begins with
  int starts[FDMA_MAX_BUCKETS];

  __host__ __device__ int buckets() const { return two_sided ? 2 * n : n; }
  __host__ __device__ int row_blocks() const { return (Nq + 7) >> 3; }
  // The bucket of a distance on its side.
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
};

// ---- forward

struct FwdView {
  RelView r;
  const void* table;
  int table_bf16;
  int64_t ts[2];
  uint16_t* out;
  int64_t os[2];
  uint32_t ncc, units;  // warps along the columns; of all rows and heads
};

__device__ __forceinline__ uint32_t table_value(const FwdView& p, int bucket, int h) {
  const int64_t at = bucket * p.ts[0] + h * p.ts[1];
  if (p.table_bf16) return static_cast<const uint16_t*>(p.table)[at];
  return pack_bf16x2(static_cast<const float*>(p.table)[at], 0.f) & 0xffffu;
}

// A warp writes 8 rows of 256 columns.  Bound by writing: four heads of 16384 x 16384 (2.1 GB) take 278 us, 7.7 TB/s, 94 % of
// what DRAM has (a copy moves 6.8).  (Walks of 2, 4, 8 or 16 blocks down the diagonal, which look up their values once for all
// of them, took 310, 319, 330 or 353 us: rows that are written at the same time should be neighbours.)  A few rows take 3 us,
// most of it the launch and the searches near the diagonal.
__global__ void __launch_bounds__(kThreads) rel_bias_kernel(const __grid_constant__ FwdView p) {
  __shared__ int first[FDMA_MAX_BUCKETS];  // (lanes look at different ones, which constant memory serves in turn)
  __shared__ __align__(16) uint16_t values[kWarps][272];  // of a warp's diagonals
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = blockIdx.x * kWarps + warp;
  const uint32_t hr = unit / p.ncc, nrb = p.r.row_blocks();
  const int cc = static_cast<int>(unit - hr * p.ncc), h = static_cast<int>(hr / nrb), rb = static_cast<int>(hr - h * nrb);
  const int lo = 256 * cc - 8 * rb - p.r.off - 7;
  const int b0 = p.r.bucket(lo);
  const bool one = b0 == p.r.bucket(lo + kSpan - 1) || unit >= p.units;
  if (__syncthreads_or(!one)) {
    for (int i = threadIdx.x; i < FDMA_MAX_BUCKETS; i += kThreads) first[i] = i < p.r.n ? p.r.starts[i] : 0x7fffffff;
    __syncthreads();
  }
  if (unit >= p.units) return;
  uint32_t w[14];  // neighbouring diagonals in pairs
  if (one) {
    const uint32_t v = table_value(p, b0, h) * 0x10001u;
#pragma unroll
    for (int i = 0; i < 14; ++i) w[i] = v;
  } else {
    // nine diagonals a lane, looked up side by side (one after the other, 5 rows of 4096 keys took 8.7 instead of 3.1 us)
    int a[9], s[9];
#pragma unroll
    for (int k = 0; k < 9; ++k) {
      const int delta = lo + 32 * k + lane;
      a[k] = p.r.two_sided ? abs(delta) : max(-delta, 0);
      s[k] = 0;
    }
    for (int step = p.r.top; step > 0; step >>= 1)
#pragma unroll
      for (int k = 0; k < 9; ++k)
        if (first[s[k] + step] <= a[k]) s[k] += step;
#pragma unroll
    for (int k = 0; k < 9; ++k) {
      const int i = 32 * k + lane;
      if (i < 272) values[warp][i] = table_value(p, s[k] + (p.r.two_sided && lo + i > 0 ? p.r.n : 0), h);
    }
    __syncwarp();
    const uint4 x = *reinterpret_cast<const uint4*>(&values[warp][8 * lane]), y = *reinterpret_cast<const uint4*>(&values[warp][8 * lane + 8]);
    const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 14; ++i) w[i] = i % 2 == 0 ? v[i / 2] : __byte_perm(v[i / 2], v[i / 2 + 1], 0x5432);
  }
  const int cb = 32 * cc + lane, rows = min(p.r.Nq - 8 * rb, 8);
  if (cb >= p.r.Nk >> 3) return;
  uint16_t* at = p.out + h * p.os[0] + static_cast<int64_t>(8 * rb) * p.os[1] + 8 * cb;
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (r < rows) *reinterpret_cast<uint4*>(at + r * p.os[1]) = make_uint4(w[7 - r], w[9 - r], w[11 - r], w[13 - r]);
}

// ---- backward

struct BwdView {
  RelView r;
  int B, causal;
  int bands, parts;  // bands with anything in them; parts is a multiple of 8
  const uint16_t* db;
  int64_t ds[3];
  float* part;  // [cta][kPart]: the sums of the band's diagonals, or the sum of all of them where they are in one bucket
  float* dtable;
};

// Of a band, or a bucket: the diagonals lo .. hi.
struct Deltas {
  int lo, hi;
};
// Band 0 begins with the block in the matrix's lower left corner.
__device__ __forceinline__ int first_delta(const RelView& r) { return -8 * (r.row_blocks() - 1) - r.off - 7; }
__device__ __forceinline__ Deltas band_deltas(const BwdView& p, int band) {
  Deltas d;
  d.lo = first_delta(p.r) + 256 * band;
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

__global__ void __launch_bounds__(kThreads, 4) rel_bias_bwd_kernel(const __grid_constant__ BwdView p) {
  __shared__ float diag[kWarps][kSpan + 1];
  __shared__ float sums[kWarps];
  __shared__ int one_bucket;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the bands from right to left: a causal matrix's longest ones come first
  const uint32_t u = blockIdx.x / p.bands, groups = p.parts / kWarps;
  const int band = p.bands - 1 - static_cast<int>(blockIdx.x - u * p.bands);
  const uint32_t hb = u / groups;
  const int part = static_cast<int>(u - hb * groups) * kWarps + warp;
  const int h = static_cast<int>(hb / p.B), b = static_cast<int>(hb - h * p.B);
  const Deltas d = band_deltas(p, band);
  const int nrb = p.r.row_blocks(), ncb = p.r.Nk >> 3, db0 = 32 * band - (nrb - 1), db = db0 + lane;
  if (threadIdx.x == 0) one_bucket = p.r.bucket(d.lo) == p.r.bucket(d.hi);
  float acc[15];
#pragma unroll
  for (int i = 0; i < 15; ++i) acc[i] = 0.f;
  const int64_t row = p.ds[2];
  // block rows in which some lane has a block
  int rb = max(0, -(db0 + 31));
  const int end = min(nrb, ncb - db0);
  rb += (part - rb % p.parts + p.parts) % p.parts;
  const bool any = d.lo + 8 * lane <= d.hi;
  const uint16_t* at = p.db + b * p.ds[0] + h * p.ds[1] + static_cast<int64_t>(8 * rb) * row + 8 * (db + rb);
  const int64_t step = static_cast<int64_t>(8 * p.parts) * row + 8 * p.parts;
  for (; rb < end; rb += p.parts, at += step) {
    if (!any || db + rb < 0 || db + rb >= ncb) continue;
    uint4 v[8];
    if (8 * rb + 8 <= p.r.Nq) {
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = __ldg(reinterpret_cast<const uint4*>(at + r * row));
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        v[r] = 8 * rb + r < p.r.Nq ? __ldg(reinterpret_cast<const uint4*>(at + r * row)) : make_uint4(0u, 0u, 0u, 0u);
    }
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
  // diagonal 8 lane + i of the warp: i >= 7 is this lane's, the others are the lane's before, too
  float* x = diag[warp];
  if (lane == 0)
    for (int i = 0; i < 7; ++i) x[i] = 0.f;
#pragma unroll
  for (int i = 7; i < 15; ++i) x[8 * lane + i] = acc[i];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 7; ++i) x[8 * lane + i] += acc[i];
  __syncthreads();
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * kPart;
  const bool one = one_bucket;
  float total = 0.f;
  for (int i = threadIdx.x; i <= d.hi - d.lo; i += kThreads) {  // (diagonals behind d.hi may hold anything)
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) s += diag[j][i];
    total += s;
    if (!one) out[i] = s;
  }
  if (!one) return;
  total = warp_sum(total);
  if (lane == 0) sums[warp] = total;
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int j = 1; j < kWarps; ++j) total += sums[j];
  out[0] = total;
}

// Adds the CTAs' sums of one bucket and head.
__global__ void __launch_bounds__(kThreads) rel_bias_join_kernel(const __grid_constant__ BwdView p) {
  __shared__ float s[kWarps];
  const int k = blockIdx.x % p.r.buckets(), h = blockIdx.x / p.r.buckets();
  const Deltas q = bucket_deltas(p.r, k);
  // the bands that have some of it
  const int64_t base = first_delta(p.r), hi = p.causal ? min(q.hi, 0) : q.hi;
  const int lo_band = static_cast<int>(max(int64_t{0}, (max(static_cast<int64_t>(q.lo), base) - base - (kSpan - 1) + 255) / 256));
  const int hi_band = hi < base ? -1 : static_cast<int>(min(static_cast<int64_t>(p.bands - 1), (hi - base) / 256));
  float sum = 0.f;
  if (q.lo <= hi && lo_band <= hi_band) {
    const uint32_t shares = static_cast<uint32_t>(p.B) * (p.parts / kWarps);  // CTAs of a band
    const float* part = p.part + static_cast<int64_t>(h) * shares * p.bands * kPart;
    auto of = [&](uint32_t u, int band) { return part + (static_cast<int64_t>(u) * p.bands + (p.bands - 1 - band)) * kPart; };
    // those that it has whole, all but one or two at either end, give a number each, the others the diagonals that it has;
    // all in one line, so that a thread's loads run together
    int first = lo_band, last = hi_band;
    auto whole = [&](int band) {
      const Deltas d = band_deltas(p, band);
      return d.lo >= q.lo && d.hi <= q.hi;
    };
    while (first <= last && !whole(first)) ++first;
    while (last >= first && !whole(last)) --last;
    const int left = first - lo_band, edges = left + (hi_band - last);
    uint32_t n[5] = {static_cast<uint32_t>(last - first + 1), 0, 0, 0, 0}, end[5];
    int band[5] = {first, 0, 0, 0, 0}, from[5] = {0, 0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 5; ++e) {
      if (e > 0 && e <= edges) {
        band[e] = e <= left ? lo_band + e - 1 : last + e - left;
        const Deltas d = band_deltas(p, band[e]);
        from[e] = max(q.lo, d.lo) - d.lo;
        n[e] = static_cast<uint32_t>(min(q.hi, d.hi) - d.lo - from[e] + 1);
      }
      end[e] = (e > 0 ? end[e - 1] : 0u) + n[e] * shares;
    }
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < end[4]; i += kThreads) {
      uint32_t begin = 0, m = n[0];
      int at = band[0], off = -1;
#pragma unroll
      for (int e = 1; e < 5; ++e) {
        if (i >= end[e - 1]) {
          begin = end[e - 1];
          m = n[e];
          at = band[e];
          off = from[e];
        }
      }
      const uint32_t u = (i - begin) / m;
      const int x = static_cast<int>(i - begin - u * m);
      sum += off < 0 ? *of(u, at + x) : of(u, at)[off + x];
    }
  }
  sum = warp_sum(sum);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int j = 1; j < kWarps; ++j) sum += s[j];
  p.dtable[static_cast<int64_t>(k) * p.r.H + h] = sum;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int validate(const fdma_rel_args* a) {
  if (a == nullptr) return FDMA_ERR_INVALID;
  if (a->H <= 0 || a->Nq < 0 || a->Nk < 0 || a->num_starts <= 0) return FDMA_ERR_INVALID;
  if (a->two_sided != 0 && a->two_sided != 1) return FDMA_ERR_INVALID;
  if (a->offset > (1 << 30) || a->offset < -(1 << 30)) return FDMA_ERR_INVALID;
  if (a->num_starts > FDMA_MAX_BUCKETS || a->H > (1 << 20) || a->Nq > kMaxLen || a->Nk > kMaxLen || a->Nk % 8 != 0)
    return FDMA_ERR_UNSUPPORTED;
  return FDMA_OK;
}

int validate_starts(const fdma_rel_args& a, const int32_t* starts) {
  if (starts == nullptr || starts[0] != 0) return FDMA_ERR_INVALID;
  for (int i = 1; i < a.num_starts; ++i)
    if (starts[i] < starts[i - 1]) return FDMA_ERR_INVALID;
  return FDMA_OK;
}

void set_view(RelView& r, const fdma_rel_args& a, const int32_t* starts) {
  r.H = a.H;
  r.Nq = a.Nq;
  r.Nk = a.Nk;
  r.off = a.offset;
  r.n = a.num_starts;
  r.two_sided = a.two_sided;
  r.top = 0;
  while (2 * r.top < r.n && r.n > 1) r.top = r.top == 0 ? 1 : 2 * r.top;
  for (int i = 0; i < r.n; ++i) r.starts[i] = starts[i];
}

int row_blocks(const fdma_rel_args& a) { return (a.Nq + 7) / 8; }

struct BwdPlan {
  int bands, parts;
  int64_t ctas;
};
// Bands and parts of a call; what it needs of the workspace does not depend on `causal`.
BwdPlan bwd_plan(const fdma_rel_args& r, int64_t B, bool causal) {
  BwdPlan p;
  const int nrb = row_blocks(r), ncb = r.Nk / 8, bands = (nrb + ncb - 1 + 31) / 32;
  // groups of eight warps that share a band, which runs through `rows` block rows at most: walks of about kBwdSteps of them,
  // shorter ones where that is too few CTAs for the machine
  const int rows = nrb < ncb + 31 ? nrb : ncb + 31;
  const int64_t fill = (kBwdCtas + B * r.H * bands - 1) / (B * r.H * bands), most = (rows + kWarps - 1) / kWarps;
  int64_t groups = (rows + kWarps * kBwdSteps - 1) / (kWarps * kBwdSteps);
  if (groups < fill) groups = fill < most ? fill : most;
  p.parts = kWarps * static_cast<int>(groups);
  p.bands = bands;
  if (causal) {  // those that begin at a key that some query sees
    const int64_t lo = -8ll * (nrb - 1) - r.offset - 7;
    const int64_t n = lo > 0 ? 0 : -lo / 256 + 1;
    if (n < bands) p.bands = static_cast<int>(n);
  }
  p.ctas = B * r.H * (p.parts / kWarps) * p.bands;
  return p;
}

}  // namespace
}  // namespace fdma

using namespace fdma;

extern "C" {

int fdma_rel_bias(const fdma_rel_args* a, const int32_t* starts, const void* table, int table_type, const int64_t ts[2],
                  void* out, const int64_t os[2], void* stream) {
  int st = validate(a);
  if (st == FDMA_OK) st = validate_starts(*a, starts);
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
  const int64_t ncc = (a->Nk / 8 + 31) / 32, units = ncc * row_blocks(*a) * a->H;
  if (units > 0x7fffffff) return FDMA_ERR_UNSUPPORTED;
  FwdView p;
  set_view(p.r, *a, starts);
  p.table = table;
  p.table_bf16 = table_type == FDMA_BF16;
  p.out = static_cast<uint16_t*>(out);
  for (int i = 0; i < 2; ++i) {
    p.ts[i] = ts[i];
    p.os[i] = os[i];
  }
  p.ncc = static_cast<uint32_t>(ncc);
  p.units = static_cast<uint32_t>(units);
  rel_bias_kernel<<<static_cast<unsigned>((units + kWarps - 1) / kWarps), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

size_t fdma_rel_bias_bwd_workspace_size(const fdma_rel_args* a, int B) {
  if (validate(a) != FDMA_OK || B <= 0 || B > (1 << 20) || a->Nq == 0 || a->Nk == 0) return 0;
  const BwdPlan plan = bwd_plan(*a, B, false);
  return plan.ctas > kMostCtas ? 0 : static_cast<size_t>(plan.ctas) * kPart * sizeof(float);
}

int fdma_rel_bias_bwd(const fdma_rel_args* a, const int32_t* starts, int B, const void* dbias, const int64_t ds[3], int causal,
                      float* dtable, void* workspace, size_t workspace_bytes, void* stream) {
  int st = validate(a);
  if (st == FDMA_OK) st = validate_starts(*a, starts);
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
  const BwdPlan whole = bwd_plan(*a, B, false), plan = bwd_plan(*a, B, causal != 0);
  if (whole.ctas > kMostCtas) return FDMA_ERR_UNSUPPORTED;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < static_cast<size_t>(whole.ctas) * kPart * sizeof(float))
    return FDMA_ERR_WORKSPACE;
  BwdView p;
  set_view(p.r, *a, starts);
  p.B = B;
  p.causal = causal;
  p.bands = plan.bands;
  p.parts = plan.parts;
  p.db = static_cast<const uint16_t*>(dbias);
  for (int i = 0; i < 3; ++i) p.ds[i] = ds[i];
  p.part = static_cast<float*>(workspace);
  p.dtable = dtable;
  if (plan.ctas > 0) {
    rel_bias_bwd_kernel<<<static_cast<unsigned>(plan.ctas), kThreads, 0, cs>>>(p);
    if (cudaGetLastError() != cudaSuccess) return FDMA_ERR_CUDA;
  }
  rel_bias_join_kernel<<<static_cast<unsigned>(buckets * a->H), kThreads, 0, cs>>>(p);
  return cudaGetLastError() == cudaSuccess ? FDMA_OK : FDMA_ERR_CUDA;
}

}  // extern "C"
