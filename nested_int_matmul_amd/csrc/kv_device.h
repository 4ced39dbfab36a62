// Device-side helpers of the 8-bit key/value cache and the rotary positions.
#pragma once

#include "mq_device.h"
#include "mq_internal.h"

namespace mq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Smallest scale of a page with codes other than 0: multiples of the scale by
// half codes, and what is left of a value beside them, are fp32 numbers.
constexpr float kMinScale = 0x1p-100f;

// 1 / (largest code) as fp32
__device__ __forceinline__ float kv_inv_qmax(bool e4m3) { return e4m3 ? 1.f / 448.f : 1.f / 127.f; }

// One sequence's tokens of a call: rows [row0, row0 + n), positions
// [start, start + n), cut to what the batch's sizes allow.
struct SeqSpan {
  int row0, n;
  int64_t start;
};
__device__ __forceinline__ SeqSpan seq_span(const KvBatch& b, int s) {
  SeqSpan r;
  const int64_t a = b.q_start[s], e = b.q_start[s + 1];
  const int64_t lo = a < 0 ? 0 : (a > b.rows ? b.rows : a);
  const int64_t hi = e < lo ? lo : (e > b.rows ? b.rows : e);
  r.row0 = (int)lo;
  r.n = (int)(hi - lo);
  r.start = (int64_t)b.kv_len[s] - r.n;
  if (r.n > b.max_new) r.n = b.max_new;
  return r;
}

// Physical page of a position's page index, or -1 where none is held.
__device__ __forceinline__ int page_of(const KvBatch& b, int s, int64_t pi, int pages) {
  if (pi < 0 || pi >= b.table_pages) return -1;
  const int p = b.page_table[(int64_t)s * b.table_pages + pi];
  return (p < 0 || p >= pages) ? -1 : p;
}

// ---- rounding to codes
// fp64 -> fp32 rounded to odd
__device__ __forceinline__ float f64_to_f32_odd(double q) {
  const float f = (float)q;
  int bits = __float_as_int(f);
  if ((double)f != q) {
    if (fabs((double)f) > fabs(q)) bits -= 1;
    bits |= 1;
  }
  return __int_as_float(bits);
}

// Eight values x to the codes nearest to the exact quotients x / s, ties to
// even; rs = 1 / s.  |x| rs, good to 2^-23 of itself, names the interval
// between two codes, whose one border b (half way) has so few bits that the
// sign of |x| - b s is exact in one fma (s >= 2^-100: nothing underflows).  The
// border, moved by that sign in its last bit, then rounds the way the exact
// quotient does, and to even if the quotient is the border; an estimate next to
// a code may name the interval on the other side of it, whose border sends it
// back to the same code.  bf16 values meet borders all the time (one in a
// hundred where 1 / s has few bits), so this is done for all of them, without
// branches.
__device__ __forceinline__ void codes_of_values(const float* x, float s, float rs, bool e4m3,
                                                uint32_t* out) {
  auto beside = [&](float b, float ax) {  // b moved towards the quotient
    const int e = __float_as_int(fmaf(-b, s, ax));
    return __int_as_float(__float_as_int(b) + (e > 1 ? 1 : e < -1 ? -1 : e));
  };
  if (e4m3) {
    // three mantissa bits; below 2^-6 the spacing of [2^-6, 2^-5)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = x[4 * h + i], ax = fabsf(v), m = ax * rs;
        const float low = m < 0x1p-6f ? 0x1p-6f : 0.f;
        const uint32_t z = (__float_as_uint(m + low) & 0xfff00000u) | 0x00080000u;
        y[i] = copysignf(beside(__uint_as_float(z) - low, ax), v);
      }
      const int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
      out[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
    }
    return;
  }
  // 1.5 * 2^23 added rounds to the nearest integer, ties to even, and leaves it
  // in the low byte
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = x[4 * h + i], ax = fabsf(v);
      const float b = __builtin_floorf(ax * rs) + 0.5f;
      z[i] = __float_as_uint(copysignf(beside(b, ax), v) + 12582912.f);
    }
    const uint32_t lo = __builtin_amdgcn_perm(z[1], z[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(z[3], z[2], 0x04000c0cu);
    out[h] = lo | hi;
  }
}

// Four quotients (rounded to odd) to four code bytes.
__device__ __forceinline__ uint32_t codes_of(const float* y, bool e4m3) {
  if (e4m3) {
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = fminf(fmaxf(y[i], -448.f), 448.f);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
  }
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = (int)__builtin_rintf(fminf(fmaxf(y[i], -127.f), 127.f));
    w |= ((uint32_t)c & 0xffu) << (8 * i);
  }
  return w;
}

// The number a code byte stands for (without the scale).
__device__ __forceinline__ void numbers_of(uint32_t w, bool e4m3, float* y) {
  if (e4m3) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    y[0] = a[0]; y[1] = a[1]; y[2] = b[0]; y[3] = b[1];
  } else {
    y[0] = (float)(int8_t)(w & 0xffu);
    y[1] = (float)(int8_t)((w >> 8) & 0xffu);
    y[2] = (float)(int8_t)((w >> 16) & 0xffu);
    y[3] = (float)(int8_t)(w >> 24);
  }
}

// Four code bytes whose page's scale grows, by ratio = was / now in float64.
// A product with it is off by 2^-52 of itself at most; a quotient that is not
// on a border between codes is at least 2^-34 of itself away from one (both
// scales have 24 bits, codes and borders 8), so rounding the product to 41
// bits first puts the quotients that are on one exactly there.
__device__ __forceinline__ uint32_t recode(uint32_t w, bool e4m3, double ratio) {
  float y[4];
  numbers_of(w, e4m3, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double q = (double)y[i] * ratio;
    const double wide = q * 4097.0;  // 2^12 + 1
    const float f = f64_to_f32_odd(wide - (wide - q));
    y[i] = f == f ? f : 0.f;
  }
  return codes_of(y, e4m3);
}

// ---- rotary positions
// sin and cos of a in float64.  a is reduced by the nearest multiple k of
// pi/2, with pi/2 as a sum of two float64 (k * hi is exact within the fma, and
// k * lo is below 2^-22 for |k| < 2^32, so the reduction adds less than half
// an ulp of 1); on |r| <= pi/4 the Taylor series to r^17 and r^16 are cut
// below 2^-60.
__device__ __forceinline__ void sincos64(double a, double* s, double* c) {
  const double k = rint(a * 0.63661977236758134308);  // 2 / pi
  double r = fma(-k, 1.57079632679489655800, a);      // pi/2, upper 53 bits
  r = fma(-k, 6.12323399573676603587e-17, r);         // pi/2, the rest
  const double z = r * r;
  double p = 1.0 / 355687428096000.0;                 // 1 / 17!
  p = fma(p, z, -1.0 / 1307674368000.0);
  p = fma(p, z, 1.0 / 6227020800.0);
  p = fma(p, z, -1.0 / 39916800.0);
  p = fma(p, z, 1.0 / 362880.0);
  p = fma(p, z, -1.0 / 5040.0);
  p = fma(p, z, 1.0 / 120.0);
  p = fma(p, z, -1.0 / 6.0);
  const double sn = fma(p * z, r, r);
  double q = 1.0 / 20922789888000.0;                  // 1 / 16!
  q = fma(q, z, -1.0 / 87178291200.0);
  q = fma(q, z, 1.0 / 479001600.0);
  q = fma(q, z, -1.0 / 3628800.0);
  q = fma(q, z, 1.0 / 40320.0);
  q = fma(q, z, -1.0 / 720.0);
  q = fma(q, z, 1.0 / 24.0);
  q = fma(q, z, -0.5);
  const double cs = fma(q, z, 1.0);
  const long long m = (long long)k;
  const double s0 = (m & 1) ? cs : sn, c0 = (m & 1) ? sn : cs;
  *s = (m & 2) ? -s0 : s0;
  *c = ((m + 1) & 2) ? -c0 : c0;
}

// A thread's unit of a head: eight entries as two runs of four, [lo, lo + 4)
// and [hi, hi + 4).  In the rotated part the unit holds four pairs; pairs()
// gives the first pair's index.
struct Unit {
  int lo, hi, pair0;
  bool turns;
};
__device__ __forceinline__ Unit unit_of(int u, int rot, bool interleaved) {
  Unit r;
  r.turns = u * 8 < rot;
  r.pair0 = 4 * u;
  if (r.turns && !interleaved) {
    r.lo = 4 * u;
    r.hi = rot / 2 + 4 * u;
  } else {
    r.lo = 8 * u;
    r.hi = 8 * u + 4;
  }
  return r;
}

// The unit's eight entries as loaded (bf16: four dwords, fp32: eight), so that
// several units can be in flight before the first is used, and as numbers.
template <bool F32>
struct RawUnit {
  u32x4 lo, hi;  // bf16: the first two dwords of each
};
template <bool F32>
__device__ __forceinline__ RawUnit<F32> load_unit(const void* x, int64_t at, const Unit& u) {
  RawUnit<F32> r;
  if (F32) {
    const float* p = static_cast<const float*>(x) + at;
    r.lo = *reinterpret_cast<const u32x4*>(p + u.lo);
    r.hi = *reinterpret_cast<const u32x4*>(p + u.hi);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(x) + at;
    const u32x2 a = *reinterpret_cast<const u32x2*>(p + u.lo);
    const u32x2 b = *reinterpret_cast<const u32x2*>(p + u.hi);
    r.lo = u32x4{a[0], a[1], 0, 0};
    r.hi = u32x4{b[0], b[1], 0, 0};
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void numbers_of_unit(const RawUnit<F32>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F32) {
      v[i] = __uint_as_float(r.lo[i]);
      v[4 + i] = __uint_as_float(r.hi[i]);
    } else {
      const uint32_t a = r.lo[i >> 1], b = r.hi[i >> 1];
      v[i] = __uint_as_float((i & 1) ? a & 0xffff0000u : a << 16);
      v[4 + i] = __uint_as_float((i & 1) ? b & 0xffff0000u : b << 16);
    }
  }
}

// Turn the unit's four pairs by (c, s) in float64, each result rounded once
// to fp32.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_pairs(float* v, const double* c, const double* s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr int A = INTERLEAVED ? 2 : 1, B = INTERLEAVED ? 1 : 4;
    const double x1 = v[A * i], x2 = v[A * i + B];
    v[A * i] = (float)(x1 * c[i] - x2 * s[i]);
    v[A * i + B] = (float)(x2 * c[i] + x1 * s[i]);
  }
}
__device__ __forceinline__ void turn_unit(float* v, const double* c, const double* s,
                                          bool interleaved) {
  if (interleaved)
    turn_pairs<true>(v, c, s);
  else
    turn_pairs<false>(v, c, s);
}

// Sines and cosines of a unit's four pairs at one position, times the factor;
// and of a step of positions, by which advance() moves them on (one complex
// product in float64, so a few of them in a row stay below 2^-48).
struct Turn {
  double c[4], s[4];
  __device__ __forceinline__ void at(const RopeSpec& r, const Unit& u, double pos, double factor) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sincos64(pos * r.freq[u.pair0 + i], &s[i], &c[i]);
      s[i] *= factor;
      c[i] *= factor;
    }
  }
  // one after the other
  __device__ __forceinline__ void advance(const Turn& d) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double n = c[i] * d.c[i] - s[i] * d.s[i];
      s[i] = s[i] * d.c[i] + c[i] * d.s[i];
      c[i] = n;
    }
  }
  __device__ __forceinline__ void advance_if(bool yes, const Turn& d) {
    Turn t = *this;
    t.advance(d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = yes ? t.c[i] : c[i];
      s[i] = yes ? t.s[i] : s[i];
    }
  }
  __device__ __forceinline__ void from_table(const double* table, const Unit& u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = table[2 * (u.pair0 + i)];
      s[i] = table[2 * (u.pair0 + i) + 1];
    }
  }
};

// A workgroup's table (in LDS) of the turns of all pairs at position `pos`
// (times the factor), then of one position: one evaluation a thread for both,
// where every thread by itself would make eight.  Ends with a barrier.
__device__ __forceinline__ void turn_table(double* table, const RopeSpec& r, double pos) {
  const int pairs = r.rot >> 1;
  for (int i = threadIdx.x; i < 2 * pairs; i += blockDim.x) {
    const bool one = i >= pairs;
    double sn, cs;
    sincos64((one ? 1.0 : pos) * r.freq[one ? i - pairs : i], &sn, &cs);
    const double f = one ? 1.0 : r.factor;
    table[2 * i] = cs * f;
    table[2 * i + 1] = sn * f;
  }
  __syncthreads();
}

// A pair of fp32 -> bf16 bits, nearest even; NaN stays a NaN.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
// Four dwords of bf16 pairs: the unit's lo run in w[0..1], its hi run in w[2..3].
__device__ __forceinline__ void pack_unit(const float* v, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
}

}  // namespace mq
