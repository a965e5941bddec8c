// The norm of a row (one token's values of one head) and the rotation of its pairs, as the
// kernels of fdma_norm_rope.cu and the cache write in fdma_cache.cu share them.
//
// A row is held by LPR lanes (powers of two, five, six or ten), two pieces of P values a lane, P pairs (a[i], b[i]) in all.  The pieces a of a row's
// lanes follow each other, and so do the pieces b (16 bytes of a lane beside those of the next: with both pieces of a lane side
// by side, every store wrote half a sector, and adjacent pairs took 42 instead of 31 us forward, 68 instead of 46 backward):
//   halves    lane l of the first rot / (2 P) holds columns P l + i and rot / 2 + P l + i, so both values
//             of a pair are in one lane; the m lanes behind hold, by their number u from 0 on, columns rot + P u + i and
//             rot + P m + P u + i;
//   adjacent  lane l holds columns P l + i and d / 2 + P l + i, P / 2 whole pairs each.
// Lanes with 2 P l >= d hold zeros, as do the last two of a warp where LPR is no power of two.  A warp holds 32 / LPR rows at
// once, all of one tensor: a pass.  Arithmetic is on
// pairs of fp32 values, one instruction for two.
//
// P is 8, pieces of 16 bytes, where d and (halves) rot are multiples of 16, else 4, which other sizes need.  (With pieces of 4
// for all, the long cases of rows of 128 take 37 instead of 31 us forward, 60 instead of 46 backward and 85 instead of 79 into
// the cache.)
#pragma once

#include <type_traits>

#include "../../include/fdma_inputs.h"
#include "fdma_internal.h"
#include "fdma_paged.cuh"
#include "fdma_ptx.cuh"

namespace fdma {

struct RowsView {
  uint16_t* p;
  int64_t st[3];  // elements: batch, token, head
};

struct WeightView {
  const void* p;  // nullptr: ones
  int64_t head;   // elements
};

struct NormRopeView {
  int d, rot;  // rot 0: no rotation
  int norm, weight_bf16;
  float eps, inv_d;
  WeightView w[2];  // q, k
  const float* rope;
  int rope_len;
  int first;
  const int32_t* pos;
  int64_t pos_st[2];
};

int validate_norm_rope(const fdma_norm_rope_args* a);
NormRopeView norm_rope_view(const fdma_norm_rope_args& a);
// Rows of n[0] batches, n[1] tokens and n[2] heads; those that are written must not overlap.
int validate_rows(const fdma_rows* r, const int64_t n[3], int d, bool written);
// ... as the kernels take them: the stride of a dimension of one is 0, whatever the caller has there.  Lanes without a row form
// addresses too (copies of 0 bytes), and those have to be aligned like all others.
RowsView rows_view(const fdma_rows& r, const int64_t n[3]);

// Pairs of a lane.
inline int piece_of(int d, int rot, bool adj) { return d % 16 == 0 && (adj || rot % 16 == 0) ? 8 : 4; }

// Lanes of a row.  (16384 tokens of 20 + 5 heads, forward / backward, us: rows of 96 in six lanes 31 / 47, in eight 40 / 59; of 80
// in five 32 / 51, in eight 39 / 60; of 72 in ten (pieces of 4) 35 / 63, in sixteen 41 / 68.  64 + 8 rows of 32 in two 32 / 54, in
// four 42 / 62.)
inline int lanes_of(int d, int rot, bool adj) {
  if (piece_of(d, rot, adj) == 8) return d <= 32 ? 2 : d <= 64 ? 4 : d <= 80 ? 5 : d <= 96 ? 6 : d <= 128 ? 8 : 16;
  return d <= 64 ? 8 : d <= 80 ? 10 : d <= 128 ? 16 : 32;
}
// Calls f(P, LPR, ADJ) with the constants that a row of d values with rot turned ones takes.
template <typename F>
void with_layout(int d, int rot, bool adj, F&& f) {
  auto with = [&](auto P, auto L) {
    if (lanes_of(d, rot, adj) != decltype(L)::value || piece_of(d, rot, adj) != decltype(P)::value) return;
    if (adj) f(P, L, std::true_type{});
    else f(P, L, std::false_type{});
  };
  using Eight = std::integral_constant<int, 8>;
  using Four = std::integral_constant<int, 4>;
  with(Eight{}, std::integral_constant<int, 2>{});
  with(Eight{}, std::integral_constant<int, 4>{});
  with(Eight{}, std::integral_constant<int, 5>{});
  with(Eight{}, std::integral_constant<int, 6>{});
  with(Eight{}, std::integral_constant<int, 8>{});
  with(Eight{}, std::integral_constant<int, 16>{});
  with(Four{}, std::integral_constant<int, 8>{});
  with(Four{}, std::integral_constant<int, 10>{});
  with(Four{}, std::integral_constant<int, 16>{});
  with(Four{}, std::integral_constant<int, 32>{});
}
// Rows of a pass.
inline int pass_rows(int d, int rot, bool adj) { return 32 / lanes_of(d, rot, adj); }

// Where a lane's values lie in a row.
struct Lane {
  int ca, cb;  // columns of its two pieces of P values
  int apart;   // cb - ca
  bool in;     // 2 P l < d, and the row is one
  // whether the pairs of piece a (halves: all of them) and of piece b (adjacent) are turned, and where their angles begin
  bool turned, turned_b;
  int ta, tb;
};

// Lane l of row g of a pass.
template <int P, int LPR, bool ADJ>
__device__ __forceinline__ Lane lane_of(const NormRopeView& v, int l, int g) {
  Lane r;
  r.in = 2 * P * l < v.d && g < 32 / LPR;
  if (ADJ) {
    r.ca = P * l;
    r.cb = (v.d >> 1) + P * l;
    r.turned = r.ca < v.rot;
    r.turned_b = r.cb < v.rot;
    r.ta = r.ca >> 1;
    r.tb = r.cb >> 1;
  } else {
    r.turned = r.turned_b = 2 * P * l < v.rot;
    const int first = r.turned ? 0 : v.rot, u = l - (r.turned ? 0 : v.rot / (2 * P));
    r.ca = first + P * u;
    r.cb = first + (((r.turned ? v.rot : v.d) - first) >> 1) + P * u;
    r.ta = r.tb = P * l;
  }
  r.apart = r.cb - r.ca;
  return r;
}

// A lane's values as they are stored: word i holds two neighbouring columns, the first P / 2 those of piece a.
template <int P>
struct Raw {
  uint32_t w[P];
};

template <int P>
__device__ __forceinline__ Raw<P> no_raw() {
  Raw<P> r;
#pragma unroll
  for (int i = 0; i < P; ++i) r.w[i] = 0u;
  return r;
}

template <int P>
__device__ __forceinline__ Raw<P> load_raw(const uint16_t* row, const Lane& n) {
  Raw<P> r;
  if constexpr (P == 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + n.ca), y = *reinterpret_cast<const uint4*>(row + n.cb);
    r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w, r.w[4] = y.x, r.w[5] = y.y, r.w[6] = y.z, r.w[7] = y.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(row + n.ca), y = *reinterpret_cast<const uint2*>(row + n.cb);
    r.w[0] = x.x, r.w[1] = x.y, r.w[2] = y.x, r.w[3] = y.y;
  }
  return r;
}
// (piece: where the first one lies, the second `apart` values behind it)
template <int P>
__device__ __forceinline__ void store_raw(uint16_t* piece, int apart, const Raw<P>& r) {
  if constexpr (P == 8) {
    *reinterpret_cast<uint4*>(piece) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    *reinterpret_cast<uint4*>(piece + apart) = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
  } else {
    *reinterpret_cast<uint2*>(piece) = make_uint2(r.w[0], r.w[1]);
    *reinterpret_cast<uint2*>(piece + apart) = make_uint2(r.w[2], r.w[3]);
  }
}
// ... with a policy for L2.
template <int P>
__device__ __forceinline__ void store_raw(uint16_t* piece, int apart, const Raw<P>& r, uint64_t policy) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint16_t* to = piece + k * apart;
    const uint32_t* w = r.w + k * P / 2;
    if constexpr (P == 8)
      asm volatile("st.global.L2::cache_hint.v4.b32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "l"(policy) : "memory");
    else
      asm volatile("st.global.L2::cache_hint.v2.b32 [%0], {%1, %2}, %3;" ::"l"(to), "r"(w[0]), "r"(w[1]), "l"(policy) : "memory");
  }
}

// Rows on their way, in shared memory: a slot holds a lane's two pieces of a pass, where only this lane writes and reads
// them, so that a warp has many passes in flight without registers for them and without a barrier.
template <int P>
struct Ring {
  static constexpr int kSlot = 128 * P;  // bytes of a warp's slot
  uint32_t at;                           // this lane's piece a of slot 0

  __device__ __forceinline__ Ring(uint32_t warp_base, int lane) : at(warp_base + lane * 2 * P) {}
  // Starts a copy of a lane's pieces, `apart` values from each other; with real false nothing is read and zeros are written.
  __device__ __forceinline__ void copy(int slot, const uint16_t* piece, int apart, bool real) const {
    const uint32_t to = at + slot * kSlot, bytes = real ? 2 * P : 0;
    if constexpr (P == 8) {
      cp_async16(to, piece, bytes);
      cp_async16(to + 64 * P, piece + apart, bytes);
    } else {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(piece), "r"(bytes) : "memory");
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to + 64 * P), "l"(piece + apart), "r"(bytes) : "memory");
    }
  }
  // ... with a policy for L2.
  __device__ __forceinline__ void copy(int slot, const uint16_t* piece, int apart, bool real, uint64_t policy) const {
    const uint32_t to = at + slot * kSlot, bytes = real ? 2 * P : 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (P == 8)
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(to + k * 64 * P), "l"(piece + k * apart), "r"(bytes), "l"(policy) : "memory");
      else
        asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], 8, %2, %3;" ::"r"(to + k * 64 * P), "l"(piece + k * apart), "r"(bytes), "l"(policy) : "memory");
    }
  }
  __device__ __forceinline__ Raw<P> get(int slot) const {
    Raw<P> r;
    const uint32_t from = at + slot * kSlot;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (P == 8)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r.w[4 * k]), "=r"(r.w[4 * k + 1]), "=r"(r.w[4 * k + 2]), "=r"(r.w[4 * k + 3])
                     : "r"(from + k * 64 * P)
                     : "memory");
      else
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                     : "=r"(r.w[2 * k]), "=r"(r.w[2 * k + 1])
                     : "r"(from + k * 64 * P)
                     : "memory");
    }
    return r;
  }
};

// Values in the order of the pairs: a[i] holds those of pairs 2 i and 2 i + 1.
template <int P>
struct Pairs {
  uint64_t a[P / 2], b[P / 2];
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <int P, bool ADJ>
__device__ __forceinline__ Pairs<P> widen(const Raw<P>& r) {
  Pairs<P> x;
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    if constexpr (ADJ) {
      x.a[i] = f2(bf16_lo(r.w[2 * i]), bf16_lo(r.w[2 * i + 1]));
      x.b[i] = f2(bf16_hi(r.w[2 * i]), bf16_hi(r.w[2 * i + 1]));
    } else {
      x.a[i] = bf16x2_to_f2(r.w[i]);
      x.b[i] = bf16x2_to_f2(r.w[P / 2 + i]);
    }
  }
  return x;
}
template <int P, bool ADJ>
__device__ __forceinline__ Raw<P> narrow(const Pairs<P>& x) {
  Raw<P> r;
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    float a0, a1, b0, b1;
    f2split(x.a[i], a0, a1);
    f2split(x.b[i], b0, b1);
    if constexpr (ADJ) {
      r.w[2 * i] = pack_bf16x2(a0, b0);
      r.w[2 * i + 1] = pack_bf16x2(a1, b1);
    } else {
      r.w[i] = pack_bf16x2(a0, a1);
      r.w[P / 2 + i] = pack_bf16x2(b0, b1);
    }
  }
  return r;
}

// The weight of a head in the order of the pairs (ones without a weight).
template <int P, bool ADJ>
__device__ __forceinline__ Pairs<P> load_weight(const NormRopeView& v, int side, int head, const Lane& n) {
  Pairs<P> w;
  const WeightView& f = v.w[side];
  if (f.p == nullptr || !n.in) {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) w.a[i] = w.b[i] = f2(1.f, 1.f);
    return w;
  }
  const int64_t at = head * f.head;
  if (v.weight_bf16) return widen<P, ADJ>(load_raw<P>(static_cast<const uint16_t*>(f.p) + at, n));
  const float* p = static_cast<const float*>(f.p) + at;
  float x[2 * P];
#pragma unroll
  for (int i = 0; i < P; i += 4) {
    const float4 y = *reinterpret_cast<const float4*>(p + n.ca + i), z = *reinterpret_cast<const float4*>(p + n.cb + i);
    x[i] = y.x, x[i + 1] = y.y, x[i + 2] = y.z, x[i + 3] = y.w;
    x[P + i] = z.x, x[P + i + 1] = z.y, x[P + i + 2] = z.z, x[P + i + 3] = z.w;
  }
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    w.a[i] = ADJ ? f2(x[4 * i], x[4 * i + 2]) : f2(x[2 * i], x[2 * i + 1]);
    w.b[i] = ADJ ? f2(x[4 * i + 1], x[4 * i + 3]) : f2(x[P + 2 * i], x[P + 2 * i + 1]);
  }
  return w;
}

// Cosines and sines.
template <int P>
struct Turn {
  uint64_t c[P / 2], s[P / 2];
};
// Turns a lane's pairs 2 i and 2 i + 1 (BACK: the other way).
template <bool BACK, int P>
__device__ __forceinline__ void turn_pair(Pairs<P>& x, int i, uint64_t c, uint64_t s) {
  const uint64_t a = x.a[i], b = x.b[i];
  // (negative sines would take registers that are not there)
  x.a[i] = BACK ? fma2(b, s, mul2(a, c)) : sub2(mul2(a, c), mul2(b, s));
  x.b[i] = BACK ? sub2(mul2(b, c), mul2(a, s)) : fma2(a, s, mul2(b, c));
}

// The angles of a lane's pairs at a position inside the table.
template <int P, bool ADJ>
__device__ __forceinline__ Turn<P> load_turn(const NormRopeView& v, int pos, const Lane& n) {
  Turn<P> t;
#pragma unroll
  for (int i = 0; i < P / 2; ++i) t.c[i] = t.s[i] = 0;
  if (!n.turned) return t;
  const float* row = v.rope + static_cast<int64_t>(pos) * v.rot;
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    const bool b = ADJ && i >= P / 4;
    if (b && !n.turned_b) continue;
    const float* p = row + (b ? n.tb + 2 * (i - P / 4) : n.ta + 2 * i);
    const float2 c = __ldg(reinterpret_cast<const float2*>(p)), s = __ldg(reinterpret_cast<const float2*>(p + (v.rot >> 1)));
    t.c[i] = f2(c.x, c.y);
    t.s[i] = f2(s.x, s.y);
  }
  return t;
}

// Turns a lane's pairs.  Those that are not turned keep their values: a product with a sine of 0 would carry an
// infinity of one column into another.
template <bool BACK, bool ADJ, int P>
__device__ __forceinline__ void turn(Pairs<P>& x, const Turn<P>& t, const Lane& n) {
  if (!n.turned) return;
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    if (ADJ && i >= P / 4 && !n.turned_b) continue;
    turn_pair<BACK>(x, i, t.c[i], t.s[i]);
  }
}

// Two pairs of fp32 values from 16 bytes of shared memory.
__device__ __forceinline__ void shared_pairs(uint32_t at, uint64_t& x, uint64_t& y) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(at) : "memory");
}

// ... by a row of the table in shared memory (half: from the cosines to the sines, in bytes).
template <bool BACK, bool ADJ, int P>
__device__ __forceinline__ void turn_shared(Pairs<P>& x, uint32_t row, uint32_t half, const Lane& n) {
  if (!n.turned) return;
  auto some = [&](int from, int count, uint32_t at) {  // count pairs of pairs
#pragma unroll
    for (int i = 0; i < count; i += 2) {
      uint64_t c0, c1, s0, s1;
      if (count > 1) {
        shared_pairs(at + 8 * i, c0, c1);
        shared_pairs(at + half + 8 * i, s0, s1);
        turn_pair<BACK>(x, from + i, c0, s0);
        turn_pair<BACK>(x, from + i + 1, c1, s1);
      } else {
        asm volatile("ld.shared.b64 %0, [%1];" : "=l"(c0) : "r"(at) : "memory");
        asm volatile("ld.shared.b64 %0, [%1];" : "=l"(s0) : "r"(at + half) : "memory");
        turn_pair<BACK>(x, from, c0, s0);
      }
    }
  };
  some(0, ADJ ? P / 4 : P / 2, row + 4 * n.ta);
  if (ADJ && n.turned_b) some(P / 4, P / 4, row + 4 * n.tb);
}

// op over a row's lanes, the same in all of them.  Every lane of the warp calls it.
template <int LPR, typename T, typename F>
__device__ __forceinline__ T row_all(T x, F&& op) {
  if constexpr ((LPR & (LPR - 1)) == 0) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  } else {
    static_assert(LPR == 5 || LPR == 6 || LPR == 10, "lanes of a row");
    const int lane = threadIdx.x & 31, l = lane % LPR, first = lane - l;
    auto behind = [&](T y, int k) { return __shfl_sync(0xffffffffu, y, first + (l + k < LPR ? l + k : l + k - LPR)); };
    if (LPR == 6) {
      const T y = op(x, behind(x, 3));
      x = op(op(y, behind(y, 1)), behind(y, 2));
    } else {
      if (LPR == 10) x = op(x, behind(x, 5));
      const T y = op(x, behind(x, 1));
      x = op(op(y, behind(y, 2)), behind(x, 4));
    }
    return __shfl_sync(0xffffffffu, x, first);  // (each lane has added in an order of its own)
  }
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
  return row_all<LPR>(x, [](float a, float b) { return a + b; });
}

// The sum of a lane's products.
template <int P>
__device__ __forceinline__ float dot(const Pairs<P>& x, const Pairs<P>& y) {
  uint64_t s = mul2(x.a[0], y.a[0]), u = mul2(x.b[0], y.b[0]);
#pragma unroll
  for (int i = 1; i < P / 2; ++i) {
    s = fma2(x.a[i], y.a[i], s);
    u = fma2(x.b[i], y.b[i], u);
  }
  float lo, hi;
  f2split(add2(s, u), lo, hi);
  return lo + hi;
}

template <int P>
__device__ __forceinline__ void scale(Pairs<P>& x, float f) {
  const uint64_t g = f2(f, f);
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    x.a[i] = mul2(x.a[i], g);
    x.b[i] = mul2(x.b[i], g);
  }
}
template <int P>
__device__ __forceinline__ void multiply(Pairs<P>& x, const Pairs<P>& w) {
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    x.a[i] = mul2(x.a[i], w.a[i]);
    x.b[i] = mul2(x.b[i], w.b[i]);
  }
}

// ... with a weight in shared memory, 16 bytes of it for every lane in turn.
template <int P>
__device__ __forceinline__ void multiply_shared(Pairs<P>& x, uint32_t at) {
#pragma unroll
  for (int i = 0; i < P / 2; i += 2) {
    uint64_t w0, w1;
    shared_pairs(at + 256 * i, w0, w1);
    x.a[i] = mul2(x.a[i], w0);
    x.a[i + 1] = mul2(x.a[i + 1], w1);
    shared_pairs(at + 128 * P + 256 * i, w0, w1);
    x.b[i] = mul2(x.b[i], w0);
    x.b[i + 1] = mul2(x.b[i + 1], w1);
  }
}
template <int P>
__device__ __forceinline__ void put_weight(uint32_t at, const Pairs<P>& w) {
#pragma unroll
  for (int i = 0; i < P / 2; i += 2) {
    asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(at + 256 * i), "l"(w.a[i]), "l"(w.a[i + 1]) : "memory");
    asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(at + 128 * P + 256 * i), "l"(w.b[i]), "l"(w.b[i + 1]) : "memory");
  }
}

// 1 / sqrt(z) of the row, z = mean(x^2) + eps.  fp32 does not hold all squares, and the backward multiplies with 1 / z: a row
// whose z is not in [2^-64, 2^48) is multiplied by a power of two first, `by` says which, and what is returned belongs to the
// scaled row (sqrt(z) times `by`).  2^40 leaves z below 2^16 and, as eps is at least 2^-149, above 2^-70; 2^-32 leaves what is
// finite between 2^-16 and 2^64; 2^-70, where it is not, sums below 2^125.  What a scaled row loses of its smallest values is less
// than bf16's least step in the output.  Ordinary rows are not touched, rows of zeros with an ordinary eps among them.  (Squares
// that overflow alone: with rows of 2^60 and gradients of 2^-30, 1 / z times the mean was a subnormal and two thirds of the
// gradient's projection were lost; with eps below 2^-128, 1 / z was infinite.)  Every lane of the warp calls it.
template <int LPR, int P>
__device__ __forceinline__ float row_rsqrt(const NormRopeView& v, Pairs<P>& x, float& by) {
  constexpr uint32_t kLeast = (127 - 64) << 23, kMost = (127 + 48) << 23;  // (as bits; NaN is above them)
  float z = row_sum<LPR>(dot(x, x)) * v.inv_d + v.eps;
  by = 1.f;
  const uint32_t bits = __float_as_uint(z);
  const bool out = bits - kLeast >= kMost - kLeast;
  if (__any_sync(0xffffffffu, out)) {
    if (out) {
      by = bits < kLeast ? 0x1p40f : z == __int_as_float(0x7f800000) ? 0x1p-70f : 0x1p-32f;
      scale(x, by);
    }
    z = row_sum<LPR>(dot(x, x)) * v.inv_d + v.eps * by * by;
  }
  return rsqrtf(z);
}

// Position of a token, checked: -1 where it is left out.
__device__ __forceinline__ int checked_position(const NormRopeView& v, int pos, int* err) {
  if (v.rot > 0 && pos >= v.rope_len) {
    atomicCAS(err, 0, FDMA_ERR_INVALID);
    return -1;
  }
  return max(pos, -1);
}

// The line of a token's passes, cut into `chunks` runs of `per` for as many warps.
struct PassPlan {
  int passes, per, chunks;
};
// Whole tokens a warp where that leaves `warps` of them, else shorter runs: a warp's lookups (position, angles,
// weights) are then paid for by fewer rows.
inline PassPlan plan_passes(int passes, int64_t tokens, int64_t warps) {
  PassPlan r{passes, 1, 1};
  const int64_t per = passes * tokens / warps;
  r.per = per < 1 ? 1 : per > passes ? passes : static_cast<int>(per);
  r.chunks = (passes + r.per - 1) / r.per;
  return r;
}

}  // namespace fdma
