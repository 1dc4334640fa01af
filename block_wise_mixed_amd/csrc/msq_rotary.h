// Rotary positions on the device (msq_rotary.hip, msq_kv_append.hip): formulas and
// roundings in msq.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "msq.h"

namespace msq {

struct RotaryView {
  const double* freq;
  double amplitude;
  int half;         // pairs of a head
  int interleaved;
};

// Cosine (x) and sine (y) of position * freq, times the amplitude, as fp32.  The angle is
// brought to -pi/4 .. pi/4 by two steps (pi/2 as a sum of two fp64 numbers: 2^-106 of
// it is left, so up to 2^32 the error stays far below a unit), then the Taylor series of
// both, whose first terms left out are below 5e-17.  Some 30 fp64 operations: fp32 would
// give other roundings of some hundredth of all cosines, and with them other codes.
__device__ inline float2 turn_of(int position, double freq, double amplitude) {
#pragma clang fp contract(off)
  const double angle = (double)position * freq;
  const double n = rint(angle * 0.63661977236758134308);
  double x = fma(-n, 1.57079632679489661923, angle);
  x = fma(-n, 6.12323399573676603587e-17, x);
  const double z = x * x;
  double s = -7.64716373181981647590e-13;  // -1 / 15!
  s = fma(s, z, 1.60590438368216145994e-10);
  s = fma(s, z, -2.50521083854417187751e-8);
  s = fma(s, z, 2.75573192239858906526e-6);
  s = fma(s, z, -1.98412698412698412698e-4);
  s = fma(s, z, 8.33333333333333333333e-3);
  s = fma(s, z, -1.66666666666666666667e-1);
  s = fma(s * z, x, x);
  double c = 4.77947733238738529744e-14;  // 1 / 16!
  c = fma(c, z, -1.14707455977297247139e-11);
  c = fma(c, z, 2.08767569878680989792e-9);
  c = fma(c, z, -2.75573192239858906526e-7);
  c = fma(c, z, 2.48015873015873015873e-5);
  c = fma(c, z, -1.38888888888888888889e-3);
  c = fma(c, z, 4.16666666666666666667e-2);
  c = fma(c, z, -0.5);
  c = fma(c, z, 1.0);
  const int quarter = (int)((long long)n & 3);
  const double co = quarter & 1 ? s : c, si = quarter & 1 ? c : s;
  return make_float2((float)(amplitude * (quarter == 1 || quarter == 2 ? -co : co)),
                     (float)(amplitude * (quarter & 2 ? -si : si)));
}

// a cos - b sin, and b cos + a sin, with one rounding an operation.
__device__ inline void turn(float& a, float& b, float2 t) {
#pragma clang fp contract(off)
  const float p = a * t.x, q = b * t.y, r = b * t.x, s = a * t.y;
  a = p - q;
  b = r + s;
}
__device__ inline float turned_low(float a, float b, float2 t) {
#pragma clang fp contract(off)
  const float p = a * t.x, q = b * t.y;
  return p - q;
}
__device__ inline float turned_high(float b, float a, float2 t) {
#pragma clang fp contract(off)
  const float p = b * t.x, q = a * t.y;
  return p + q;
}

// Rows as the kernels take them.
struct RotaryRowsView {
  const void* x;
  void* out;
  int64_t xts, xhs, ots, ohs;
  int heads, units;  // units of 16 values a head
  int x_f32, out_f32;
};

// A unit: 16 values of a head as two groups of 8, pairs 8 u .. 8 u + 7 for u < half / 8
// (in halves, groups at 8 u and half + 8 u), else values that stay.
struct Unit {
  uint4 w[4];  // bf16: w[0], w[2]
};
__device__ inline void unit_at(const RotaryView& r, int u, int& lo, int& hi) {
  const bool split = !r.interleaved && 8 * u < r.half;
  lo = split ? 8 * u : 16 * u;
  hi = split ? r.half + 8 * u : 16 * u + 8;
}
__device__ inline void load_unit(const RotaryRowsView& v, const RotaryView& r, int64_t row, int h, int u, Unit& t) {
  int lo, hi;
  unit_at(r, u, lo, hi);
  const int64_t at = row * v.xts + (int64_t)h * v.xhs;
  if (v.x_f32) {
    const float* p = reinterpret_cast<const float*>(v.x) + at;
    const uint4 *a = reinterpret_cast<const uint4*>(p + lo), *b = reinterpret_cast<const uint4*>(p + hi);
    t.w[0] = a[0], t.w[1] = a[1], t.w[2] = b[0], t.w[3] = b[1];
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(v.x) + at;
    t.w[0] = *reinterpret_cast<const uint4*>(p + lo);
    t.w[2] = *reinterpret_cast<const uint4*>(p + hi);
  }
}
__device__ inline void eight(const uint4* w, int f32, float* x) {
  const uint32_t a[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
  if (f32) {
    const uint32_t b[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(a[i]), x[4 + i] = __uint_as_float(b[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(a[i] << 16);
      x[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}
__device__ inline void put_eight(void* out, int f32, int64_t at, const float* x) {
  if (f32) {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    union {
      __bf16 b[8];
      uint4 u;
    } o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.b[i] = (__bf16)x[i];
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + at) = o.u;
  }
}
// turns: of this row, [half]
__device__ inline void finish_unit(const RotaryRowsView& v, const RotaryView& r, int64_t row, int h, int u,
                                   const Unit& t, const float2* turns) {
  float a[8], b[8];
  eight(t.w, v.x_f32, a);
  eight(t.w + 2, v.x_f32, b);
  if (8 * u < r.half) {
    float2 c[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(c)[i] = reinterpret_cast<const float4*>(turns + 8 * u)[i];
    if (r.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn(a[2 * i], a[2 * i + 1], c[i]), turn(b[2 * i], b[2 * i + 1], c[4 + i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(a[i], b[i], c[i]);
    }
  }
  int lo, hi;
  unit_at(r, u, lo, hi);
  const int64_t at = row * v.ots + (int64_t)h * v.ohs;
  put_eight(v.out, v.out_f32, at + lo, a);
  put_eight(v.out, v.out_f32, at + hi, b);
}

// Rows row0 .. row0 + rows - 1 of all heads by one workgroup; position(i) that of row
// row0 + i, turns: LDS, [rows][half].  Units are read four at a time; the first ones
// are on their way while the turns are made.
template <typename Position>
__device__ inline void rotate_rows(const RotaryRowsView& v, const RotaryView& r, int64_t row0, int rows, int h0,
                                   int heads, float2* turns, Position&& position) {
  constexpr int kAtOnce = 4;
  const unsigned threads = blockDim.x, units = v.units, row_units = units * heads, all = row_units * rows;
  Unit t[kAtOnce];
  auto place = [&](unsigned n, int& i, int& h, int& u) {
    i = (int)(n / row_units);
    const unsigned m = n - i * row_units;
    h = (int)(m / units);
    u = (int)(m - h * units);
    h += h0;
  };
  auto load = [&](unsigned n0) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const unsigned n = n0 + k * threads;
      if (n >= all) break;
      int i, h, u;
      place(n, i, h, u);
      load_unit(v, r, row0 + i, h, u, t[k]);
    }
  };
  load(threadIdx.x);
  for (unsigned n = threadIdx.x; n < (unsigned)(rows * r.half); n += threads) {
    const int i = (int)(n / (unsigned)r.half), pair = (int)(n - i * (unsigned)r.half);
    turns[n] = turn_of(position(i), r.freq[pair], r.amplitude);
  }
  __syncthreads();
  for (unsigned n0 = threadIdx.x; n0 < all; n0 += kAtOnce * threads) {
    if (n0 != threadIdx.x) load(n0);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const unsigned n = n0 + k * threads;
      if (n >= all) break;
      int i, h, u;
      place(n, i, h, u);
      finish_unit(v, r, row0 + i, h, u, t[k], turns + (int64_t)i * r.half);
    }
  }
}

// Host checks of a rotation (dims 0 allowed where none) and of its rows; fills the views.
msq_status rotary_view(const msq_rotary* rot, int head_dim, bool none, RotaryView& r);
msq_status rotary_rows_view(const msq_rotary_rows* x, RotaryRowsView& v);
msq_status rotary_rows_pointers(const msq_rotary_rows* x);

}  // namespace msq
