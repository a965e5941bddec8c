// The norm of a row (one token's values of one head) and the rotation of its pairs, as the
// kernels of fdma_norm_rope.cu and the cache write in fdma_cache.cu share them.
//
// A row is held by LPR lanes (a power of two), eight values a lane as four pairs (a[i], b[i]):
//   halves    lane l of the first rot / 8 holds columns 4 l + i and rot / 2 + 4 l + i, so both values
//             of a pair are in one lane whatever rot is; the lanes behind hold columns 8 l + i and 8 l + 4 + i;
//   adjacent  lane l holds columns 8 l + 2 i and 8 l + 2 i + 1.
// Either way lane l turns its pairs by the angles 4 l + i.  Lanes with 8 l >= d hold zeros.
#pragma once

#include "../../include/fdma_inputs.h"
#include "fdma_internal.h"
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
// Rows of n[0] batches, n[1] tokens and n[2] heads; those that are written have to be distinct.
int validate_rows(const fdma_rows* r, const int64_t n[3], bool written);
RowsView rows_view(const fdma_rows& r);

// Where a lane's values lie in a row.
struct Lane {
  int ca, cb;   // columns of the two 4-value pieces
  bool in;      // 8 l < d
  bool turned;  // its pairs are rotated
};

template <bool ADJ>
__device__ __forceinline__ Lane lane_of(const NormRopeView& v, int l) {
  Lane r;
  r.in = 8 * l < v.d;
  r.turned = 8 * l < v.rot;
  r.ca = !ADJ && r.turned ? 4 * l : 8 * l;
  r.cb = !ADJ && r.turned ? (v.rot >> 1) + 4 * l : 8 * l + 4;
  return r;
}

struct Raw {
  uint2 a, b;
};

template <bool ADJ>
__device__ __forceinline__ Raw load_raw(const uint16_t* row, const Lane& n) {
  Raw r;
  if (ADJ) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + n.ca);
    r.a = make_uint2(v.x, v.y);
    r.b = make_uint2(v.z, v.w);
  } else {
    r.a = *reinterpret_cast<const uint2*>(row + n.ca);
    r.b = *reinterpret_cast<const uint2*>(row + n.cb);
  }
  return r;
}
template <bool ADJ>
__device__ __forceinline__ void store_raw(uint16_t* row, const Lane& n, const Raw& r) {
  if (ADJ) {
    *reinterpret_cast<uint4*>(row + n.ca) = make_uint4(r.a.x, r.a.y, r.b.x, r.b.y);
  } else {
    *reinterpret_cast<uint2*>(row + n.ca) = r.a;
    *reinterpret_cast<uint2*>(row + n.cb) = r.b;
  }
}

// Values in the order of the pairs.
struct Pairs {
  float a[4], b[4];
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool ADJ>
__device__ __forceinline__ Pairs widen(const Raw& r) {
  Pairs x;
  if (ADJ) {
    x.a[0] = bf16_lo(r.a.x), x.b[0] = bf16_hi(r.a.x), x.a[1] = bf16_lo(r.a.y), x.b[1] = bf16_hi(r.a.y);
    x.a[2] = bf16_lo(r.b.x), x.b[2] = bf16_hi(r.b.x), x.a[3] = bf16_lo(r.b.y), x.b[3] = bf16_hi(r.b.y);
  } else {
    x.a[0] = bf16_lo(r.a.x), x.a[1] = bf16_hi(r.a.x), x.a[2] = bf16_lo(r.a.y), x.a[3] = bf16_hi(r.a.y);
    x.b[0] = bf16_lo(r.b.x), x.b[1] = bf16_hi(r.b.x), x.b[2] = bf16_lo(r.b.y), x.b[3] = bf16_hi(r.b.y);
  }
  return x;
}
template <bool ADJ>
__device__ __forceinline__ Raw narrow(const Pairs& x) {
  Raw r;
  if (ADJ) {
    r.a = make_uint2(pack_bf16x2(x.a[0], x.b[0]), pack_bf16x2(x.a[1], x.b[1]));
    r.b = make_uint2(pack_bf16x2(x.a[2], x.b[2]), pack_bf16x2(x.a[3], x.b[3]));
  } else {
    r.a = make_uint2(pack_bf16x2(x.a[0], x.a[1]), pack_bf16x2(x.a[2], x.a[3]));
    r.b = make_uint2(pack_bf16x2(x.b[0], x.b[1]), pack_bf16x2(x.b[2], x.b[3]));
  }
  return r;
}

// The weight of a head in the order of the pairs (ones without a weight).
template <bool ADJ>
__device__ __forceinline__ Pairs load_weight(const NormRopeView& v, int side, int head, const Lane& n) {
  Pairs w;
  const WeightView& f = v.w[side];
  if (f.p == nullptr || !n.in) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w.a[i] = w.b[i] = 1.f;
    return w;
  }
  const int64_t at = head * f.head;
  if (v.weight_bf16) return widen<ADJ>(load_raw<ADJ>(static_cast<const uint16_t*>(f.p) + at, n));
  const float* p = static_cast<const float*>(f.p) + at;
  const float4 x = *reinterpret_cast<const float4*>(p + n.ca), y = *reinterpret_cast<const float4*>(p + n.cb);
  if (ADJ) {
    w.a[0] = x.x, w.b[0] = x.y, w.a[1] = x.z, w.b[1] = x.w;
    w.a[2] = y.x, w.b[2] = y.y, w.a[3] = y.z, w.b[3] = y.w;
  } else {
    w.a[0] = x.x, w.a[1] = x.y, w.a[2] = x.z, w.a[3] = x.w;
    w.b[0] = y.x, w.b[1] = y.y, w.b[2] = y.z, w.b[3] = y.w;
  }
  return w;
}

struct Turn {
  float4 c, s;
};
// Cosines and sines of a lane's pairs at a position inside the table.
__device__ __forceinline__ Turn load_turn(const NormRopeView& v, int pos, int l, const Lane& n) {
  Turn t{};
  if (n.turned) {
    const float* p = v.rope + static_cast<int64_t>(pos) * v.rot + 4 * l;
    t.c = __ldg(reinterpret_cast<const float4*>(p));
    t.s = __ldg(reinterpret_cast<const float4*>(p + (v.rot >> 1)));
  }
  return t;
}

// Turns a lane's pairs (BACK: the other way).  Lanes that are not turned keep their values: a product with
// a sine of 0 would carry an infinity of one column into another.
template <bool BACK>
__device__ __forceinline__ void turn(Pairs& x, const Turn& t, const Lane& n) {
  if (!n.turned) return;
  const float c[4] = {t.c.x, t.c.y, t.c.z, t.c.w}, s[4] = {t.s.x, t.s.y, t.s.z, t.s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x.a[i], b = x.b[i], z = BACK ? -s[i] : s[i];
    x.a[i] = a * c[i] - b * z;
    x.b[i] = b * c[i] + a * z;
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float square_sum(const Pairs& x) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) s += x.a[i] * x.a[i] + x.b[i] * x.b[i];
  return s;
}

// 1 / sqrt(mean(x^2) + eps) of the row.  Values above 2^64 have squares that fp32 does not hold: such a row is
// multiplied by 2^-70 first (its squares then sum to less than 2^125), `scale` says so, and what is returned belongs to
// the scaled row.  Every lane of the warp calls it.
template <int LPR>
__device__ __forceinline__ float row_rsqrt(const NormRopeView& v, Pairs& x, float& scale) {
  constexpr float kDown = 0x1p-70f;
  float s = row_sum<LPR>(square_sum(x));
  scale = 1.f;
  const bool over = s == __int_as_float(0x7f800000);
  if (__any_sync(0xffffffffu, over)) {
    if (over) {
      scale = kDown;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x.a[i] *= kDown;
        x.b[i] *= kDown;
      }
    }
    s = row_sum<LPR>(square_sum(x));
  }
  return rsqrtf(s * v.inv_d + v.eps * scale * scale);
}

// The forward of a row: x becomes what is stored.  Every lane of the warp calls it.
template <int LPR>
__device__ __forceinline__ void norm_and_turn(const NormRopeView& v, Pairs& x, const Pairs& w, const Turn& t, const Lane& n) {
  if (v.norm) {
    float scale;
    const float r = row_rsqrt<LPR>(v, x, scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x.a[i] = x.a[i] * r * w.a[i];
      x.b[i] = x.b[i] * r * w.b[i];
    }
  }
  turn<false>(x, t, n);
}

// Position of a token, checked: -1 where it is left out.
__device__ __forceinline__ int checked_position(const NormRopeView& v, int pos, int* err) {
  if (v.rot > 0 && pos >= v.rope_len) {
    atomicCAS(err, 0, FDMA_ERR_INVALID);
    return -1;
  }
  return max(pos, -1);
}

}  // namespace fdma
