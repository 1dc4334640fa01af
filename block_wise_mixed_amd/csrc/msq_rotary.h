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
// both, whose first terms left out are below 5e-17.  Some 30 fp64 operations for all heads
// of a row; in fp32 an angle of 10^6 alone would be rounded by up to 0.03 radians.
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

// A unit: two groups of 8 values of a head, half of the rotated dims apart (which are the
// pairs of a rotation in halves), or half of the others: either way neighbouring
// units are contiguous in memory.  (Nontemporal reads and writes where these runs are whole
// lines: 470 MB 81 -> 78 us alone, but in an append the read of the cache that followed
// 125 -> 149 us.)
typedef uint32_t words4 __attribute__((ext_vector_type(4)));
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  words4 w;
  __device__ void load(const uint16_t* p) { w = *reinterpret_cast<const words4*>(p); }
  __device__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static void put(uint16_t* p, const float (&x)[8]) {
    union {
      __bf16 b[8];
      words4 w;
    } o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.b[i] = (__bf16)x[i];
    *reinterpret_cast<words4*>(p) = o.w;
  }
};
template <>
struct Eight<float> {
  words4 a, b;
  __device__ void load(const float* p) { a = reinterpret_cast<const words4*>(p)[0], b = reinterpret_cast<const words4*>(p)[1]; }
  __device__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(a[i]), x[4 + i] = __uint_as_float(b[i]);
  }
  __device__ static void put(float* p, const float (&x)[8]) {
    words4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(x[i]), b[i] = __float_as_uint(x[4 + i]);
    reinterpret_cast<words4*>(p)[0] = a;
    reinterpret_cast<words4*>(p)[1] = b;
  }
};

// Where a thread's unit is: of row `row`, from dim lo on.
struct UnitPlace {
  bool on;
  int row, lo, apart;
  int64_t from, to;
};

template <typename TX, typename TO, bool kPairs, typename Turns>
__device__ __forceinline__ void rotate_unit(const RotaryRowsView& v, const RotaryView& r, const UnitPlace& p,
                                            const float2* turns, Turns&& make_turns) {
  Eight<TX> ra, rb;
  if (p.on) {
    const TX* x = reinterpret_cast<const TX*>(v.x) + p.from;
    ra.load(x);
    rb.load(x + p.apart);
  }
  make_turns();
  if (!p.on) return;
  float a[8], b[8];
  ra.get(a);
  rb.get(b);
  if (p.lo < r.half) {
    const float2* t = turns + p.row * r.half;
    float2 c[8];
    if (kPairs) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        reinterpret_cast<float4*>(c)[i] = reinterpret_cast<const float4*>(t + p.lo / 2)[i];
        reinterpret_cast<float4*>(c)[2 + i] = reinterpret_cast<const float4*>(t + (p.lo + r.half) / 2)[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) turn(a[2 * i], a[2 * i + 1], c[i]), turn(b[2 * i], b[2 * i + 1], c[4 + i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(c)[i] = reinterpret_cast<const float4*>(t + p.lo)[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(a[i], b[i], c[i]);
    }
  }
  TO* y = reinterpret_cast<TO*>(v.out) + p.to;
  Eight<TO>::put(y, a);
  Eight<TO>::put(y + p.apart, b);
}

// Rows row0 .. row0 + rows - 1 of the heads h0 .. by one workgroup, a unit a thread (rows *
// heads * units are at most its threads); position(i) that of row row0 + i, turns: LDS,
// [rows][half].  The values are on their way while the turns are made, whose positions
// and frequencies are read before them, for loads return in order.
template <typename Position>
__device__ inline void rotate_rows(const RotaryRowsView& v, const RotaryView& r, int64_t row0, int rows, int h0,
                                   int heads, float2* turns, Position&& position) {
  const unsigned tid = threadIdx.x, units = v.units, all = (unsigned)(rows * r.half);
  int at = 0;
  double f = 0.0;
  if (tid < all) {
    const unsigned i = tid / (unsigned)r.half;
    at = position((int)i);
    f = r.freq[tid - i * (unsigned)r.half];
  }
  const unsigned slot = tid / units, row = slot / (unsigned)heads;
  const int u = (int)(tid - slot * units), h = h0 + (int)(slot - row * heads), turned = r.half >> 3;
  UnitPlace p;
  p.on = row < (unsigned)rows;
  p.row = (int)row;
  p.lo = u < turned ? 8 * u : 2 * r.half + 8 * (u - turned);
  p.apart = u < turned ? r.half : 8 * (int)units - r.half;
  p.from = (row0 + row) * v.xts + h * v.xhs + p.lo;
  p.to = (row0 + row) * v.ots + h * v.ohs + p.lo;
  auto make_turns = [&] {
    if (tid < all) turns[tid] = turn_of(at, f, r.amplitude);
    for (unsigned n = tid + blockDim.x; n < all; n += blockDim.x) {
      const unsigned i = n / (unsigned)r.half;
      turns[n] = turn_of(position((int)i), r.freq[n - i * (unsigned)r.half], r.amplitude);
    }
    __syncthreads();
  };
  auto go = [&](auto x, auto y) {
    using X = decltype(x);
    using Y = decltype(y);
    r.interleaved ? rotate_unit<X, Y, true>(v, r, p, turns, make_turns)
                  : rotate_unit<X, Y, false>(v, r, p, turns, make_turns);
  };
  if (v.x_f32)
    v.out_f32 ? go(float{}, float{}) : go(float{}, uint16_t{});
  else
    v.out_f32 ? go(uint16_t{}, float{}) : go(uint16_t{}, uint16_t{});
}

// Rows and heads of a workgroup of `threads`, workgroups that share its rows' heads.
struct RotaryShare {
  int rows, heads, parts;
};
inline RotaryShare rotary_share(const RotaryRowsView& v, int threads, int64_t rows) {
  RotaryShare s;
  s.heads = v.heads < threads / v.units ? v.heads : threads / v.units;
  s.parts = (v.heads + s.heads - 1) / s.heads;
  const int most = threads / (v.units * s.heads);
  s.rows = (int)(rows < most ? (rows < 1 ? 1 : rows) : most);
  return s;
}

// Host checks of a rotation (dims 0 allowed where none) and of its rows; fills the views.
msq_status rotary_view(const msq_rotary* rot, int head_dim, bool none, RotaryView& r);
msq_status rotary_rows_view(const msq_rotary_rows* x, RotaryRowsView& v);
msq_status rotary_rows_pointers(const msq_rotary_rows* x);

}  // namespace msq
