// Attention over the 8-bit key/value cache (msq_kv_attention).
//
// For a query row with scores x_t = c q.k_t (base-2 logarithms, c = scale *
// log2 e) over the tokens it sees, o = sum 2^x_t v_t / sum 2^x_t.  One pass
// keeps a reference exponent M, the weighted sum O = sum w_t code(v_t) and
// the denominator L.  The scale s of a block's values is a factor of its
// tokens' weights, w_t = 2^(x_t + log2 s - M), so no product with s is left
// for O, and L = sum w_t / s.  M follows the largest weighted exponent: w is
// rounded to f16, and this way its error is relative to the largest
// contribution to O whatever the blocks' scales are.
//
// A block whose values are all 0 (or below 2^-93, which count as 0) adds to the
// denominator only.  Whatever its scores, they say nothing of the size of O, so
// its tokens have a reference Mz and a sum Lz of their own, joined to M and L at
// the end.  The same goes for the denominator of a block whose scale is more than
// 2^64 below the largest that its wavefront has met: at weights that its values
// no longer reach, its scores can still be the ones that count.
//
// M is only moved when some weight would pass 2^14 (f16 ends at 2^16), and
// then to 6 below the maximum: most tiles need neither the cross-lane maximum
// nor a rescale, and weights down to 2^-20 of the largest stay normal f16
// numbers.
//
// Scores may have any finite size.  Fp32 numbers of 2^28 lie 32 apart: log2 s - 6
// is lost in an M of that size, and an exact product less a rounded M can be as far
// from 0 at the top itself.  For a row whose top score passes 2^11 (where numbers lie
// 2^-12 apart, a weight's rounding) the reference is therefore M + off, a score
// rounded like all others and the small rest, and the exponents are
// (x_t - M) + (log2 s - off), whose difference is exact near the top.  Such a row
// takes this way in every tile.
//
// Codes become f16 exactly: the bytes code + 128 under the exponent byte 0x64
// are the f16 numbers 1024 + byte, and one packed subtraction of 1152 leaves
// the code.  A query row is scaled by the power of two that puts its largest
// value in [2^14, 2^15), so bf16 queries are exact down to 2^-28 of it.  fp32 ones are
// rounded to 11 bits where the results are bf16; for fp32 results (kFine) what is left
// of them goes through the products as a second f16 term, 22 bits in all.  The
// weights are rounded to f16 either way, and L is the sum of the unrounded ones.
// Against 64 bits (128 dims, 700 tokens, score spreads of 0.3 to 4) fp32 results are
// 2e-4 or less away (rms), with fp32 queries in one term 1.6e-4 to 4.4e-4; rounding to
// bf16 alone is 1.7e-3.  The second term costs 2 to 4% in k_kv_decode and 18 to 29%
// in k_kv_prefill (2048 rows of 64 heads on 16000 tokens 941 -> 1215 us).  L of the
// rounded weights, which cancels some of their rounding: 1.9e-4 -> 1.7e-4 and 1.2e-4 ->
// 0.7e-4, at 4% of the time of many rows; not taken.
#include <hip/hip_runtime.h>
#include <unistd.h>

#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "msq.h"
#include "msq_kv.h"

namespace msq {
namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kNone = -3.402823466e38f;  // M before any token: no score is below it
constexpr float kTop = 14.f;       // weights stay below 2^kTop
constexpr float kTopWeight = 16384.f;  // 2^kTop
constexpr float kPlace = 6.f;      // a moved M puts the largest weight at 2^kPlace
constexpr float kNear = 2048.f;    // up to here M holds a score and log2 s in one number
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kTinyBits = 27u << 23;  // 2^-100: value scales below it count as 0
constexpr int kSpan = 32;          // tokens of a tile of k_kv_decode
constexpr int kRowTile = 16;       // and its query rows
constexpr int kMostParts = 64;     // parts of a row tile's tokens
constexpr uint32_t kNoScale = 0x72000000;  // 2^101, inverse of less than any scale
constexpr uint32_t kFaint = 64u << 23;  // 2^64, between the bit patterns of two scales' inverses
constexpr float kTinyStep = 1e-37f;  // keeps -inf * step from being NaN where a step is 0

struct AttnArgs {
  KvCacheView c;
  KvSeqsView s;
  const void* q;
  int64_t qts, qhs;
  const int32_t* kv_len;
  void* out;
  float* lse;
  float* part_o;   // [nsplit][total * Hq][D], null for one split
  float2* part_ml; // [nsplit][total * Hq]: M, L
  uint64_t* tags;  // [item][kMostParts]: which parts of this call are there; null: a join launch
  uint64_t call;
  int Hq, G, q_f32, out_f32, causal, window;
  int nsplit;      // workgroups along a row tile's tokens
  int span_tiles;  // tiles of one such part (more where nsplit parts cannot cover the range)
  int row_tiles, tile_rows, tile_shift;  // tiles of tile_rows x 2^tile_shift tokens
  float c2;        // scale * log2 e
};

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ inline float log2_fast(float x) { return __builtin_amdgcn_logf(x); }

// Four bytes code + 128 -> four f16 codes.
__device__ inline void codes_f16(uint32_t w, half2v& a, half2v& b) {
  const half2v off = {(_Float16)(-1152.f), (_Float16)(-1152.f)};
  a = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off;
  b = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off;
}
__device__ inline half8 codes_f16x8(uint32_t w0, uint32_t w1) {
  union {
    half2v p[4];
    half8 h;
  } r;
  codes_f16(w0, r.p[0], r.p[1]);
  codes_f16(w1, r.p[2], r.p[3]);
  return r.h;
}

// Eight query values as loaded.
struct Raw8 {
  uint4 a, b;  // bf16: a only
};
__device__ inline Raw8 load8(const void* q, int f32, int64_t at) {
  Raw8 r{};
  if (f32) {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(q) + at);
    r.a = p[0];
    r.b = p[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(q) + at);
  }
  return r;
}
// The power of two 2^e that the row is multiplied by, from its largest
// magnitude (NaN if the row has a non-finite value), and its inverse.
__device__ inline void row_scale(float amax, bool bad, float& up, float& down) {
  int e = 0;
  if (amax > 0.f && !bad) {
    (void)frexpf(amax, &e);  // amax = m 2^e, 1/2 <= m < 1
    e = 15 - e;
  }
  e = min(max(e, -126), 126);
  up = bad ? __uint_as_float(0x7FC00000u) : ldexpf(1.f, e);
  down = ldexpf(1.f, -e);
}

// The f16 fragments of a query row, whose values the lanes lane ^ kFirst * m
// hold between them, and the inverse of their scale; of an fp32 row with kFine also
// what f16 leaves of it, as f16 fragments rest.
template <bool kFine, int N, int kFirst>
__device__ inline void query_fragments(const Raw8 (&raw)[N], int f32, half8 (&q)[N],
                                       half8 (&rest)[kFine ? N : 1], float& down) {
  typedef uint16_t pair __attribute__((ext_vector_type(2)));
  uint32_t most = 0;  // the largest magnitude, as an fp32 bit pattern
  if (f32) {
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint32_t w[8] = {raw[s].a.x, raw[s].a.y, raw[s].a.z, raw[s].a.w,
                             raw[s].b.x, raw[s].b.y, raw[s].b.z, raw[s].b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) most = max(most, w[e] & 0x7FFFFFFFu);
    }
  } else {
    pair m = {0, 0};
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint32_t w[4] = {raw[s].a.x, raw[s].a.y, raw[s].a.z, raw[s].a.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(pair, w[e] & 0x7FFF7FFFu));
    }
    most = (uint32_t)max(m[0], m[1]) << 16;
  }
#pragma unroll
  for (int x = kFirst; x < 64; x <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, x));
  float up;
  row_scale(__uint_as_float(most), most >= 0x7F800000u, up, down);
  if (f32) {
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint32_t w[8] = {raw[s].a.x, raw[s].a.y, raw[s].a.z, raw[s].a.w,
                             raw[s].b.x, raw[s].b.y, raw[s].b.z, raw[s].b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = __uint_as_float(w[e]) * up;
        q[s][e] = (_Float16)x;
        if constexpr (kFine) rest[s][e] = (_Float16)(x - (float)q[s][e]);
      }
    }
  } else {
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint32_t w[4] = {raw[s].a.x, raw[s].a.y, raw[s].a.z, raw[s].a.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[s][2 * e] = (_Float16)(__uint_as_float(w[e] << 16) * up);
        q[s][2 * e + 1] = (_Float16)(__uint_as_float(w[e] & 0xFFFF0000u) * up);
      }
    }
  }
}

// Log2 and inverse of a value scale; -inf and 0 for a block of zeros, whose
// weights then come out 0.  A block before a window may never have been written:
// all its weights are of masked tokens, and no scale that it holds, an infinite
// one among them, may make more of them than 0 (a written scale is at most 2^121).
// One comparison of bit patterns, for the chain of loads goes on behind it (two of
// numbers: one token on 777 cached 7.8 -> 8.1 us).
__device__ inline void value_scale(float s, float& lam, float& inv) {
  const bool some = __float_as_uint(s) - kTinyBits < 0x7F800000u - kTinyBits;  // finite, 2^-100 or more
  lam = some ? log2_fast(s) : -INFINITY;
  inv = some ? __builtin_amdgcn_rcpf(s) : 0.f;
}

// A score s * f, rounded (and no part of an fma).
__device__ inline float score_of(float s, float f) {
#pragma clang fp contract(off)
  return s * f;
}

// 2^(x / 2), a factor of L twice over: L may be as large as 2^x is small.
__device__ inline float half_exp2(float x) { return exp2_fast(0.5f * x); }

// Moves the reference of a row to the score `most` of a block whose values have
// scale 2^lam, and its sum L with it; returns the factor of O.
__device__ inline float move_reference(float most, float lam, float& M, float& off, float& L,
                                       bool& far) {
  far = fabsf(most) > kNear;
  const float m = far ? most : most + lam - kPlace, rest = far ? lam - kPlace : 0.f;
  const float g = half_exp2((M - m) + (off - rest));
  L = L * g * g;
  M = m;
  off = rest;
  return g * g;
}

// M + off as one number, M; what rounding takes from it goes to L and, as the
// factor that it returns, to O.
__device__ inline float one_reference(float& M, float off, float& L) {
  const float m = M + off, g = exp2_fast((M - m) + off);
  M = m;
  L *= g;
  return g;
}

// Scores s (times f; -inf where masked) of a block of zeros, or a faint one, into Mz
// and Lz; the lanes lane ^ kFirst * m have the same row.
template <int kFirst, int N>
__device__ inline void add_zeros(const float (&s)[N], float f, float& Mz, float& Lz) {
  float most = s[0];
#pragma unroll
  for (int e = 1; e < N; ++e) most = fmaxf(most, s[e]);
#pragma unroll
  for (int x = kFirst; x < 64; x <<= 1) most = fmaxf(most, __shfl_xor(most, x));
  const float m = fmaxf(Mz, score_of(most, f));
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) sum += exp2_fast(score_of(s[e], f) - m);
  Lz = fmaf(Lz, exp2_fast(Mz - m), sum);
  Mz = m;
}

// Blocks by the bits of their values' inverse scale, `in` (0: zeros), beside the least
// so far, of the largest scale; all the same in a wavefront.  One comparison tells
// a block of zeros, a faint one or a new least from all others; of these,
// meet_scale returns true for the first two.
__device__ inline bool is_special(uint32_t in, uint32_t least) { return in - least > kFaint; }
__device__ inline bool meet_scale(uint32_t in, uint32_t& least) {
  if (in == 0 || in > least) return true;
  least = in;
  return false;
}

// The sums of a row's lanes joined, and Mz and Lz joined to M and L; O is to be
// multiplied by what it returns.  M ends at least 2^64 below Mz (level with it where
// numbers of its size lie further apart), so that L stays finite; where that
// takes bits of O, the result ends below 2^-126.
template <int kFirst>
__device__ inline float join_zeros(float& M, float& L, float Mz, float Lz) {
#pragma unroll
  for (int x = kFirst; x < 64; x <<= 1) {
    L += __shfl_xor(L, x);
    Lz += __shfl_xor(Lz, x);
  }
  const float m = fmaxf(M, fabsf(Mz) < 0x1p28f ? Mz - 64.f : Mz), g = exp2_fast(M - m);
  if (Lz != 0.f) L = fmaf(L, g, Lz * exp2_fast(Mz - m));
  M = m;
  return g;
}

// The positions lo <= t < hi of the table that row i of n of a sequence with len
// tokens sees: a length past the table still says where its rows stand (32-bit
// numbers and unsigned divisions here and below: the kernels start with a chain
// of them).
__device__ inline void row_range(const AttnArgs& a, int len, int n, int i, int& lo, int& hi) {
  lo = 0;
  hi = len;
  if (a.causal) {
    const int pos = len - n + i;
    hi = max(pos + 1, 0);
    if (a.window > 0 && pos >= a.window) lo = pos - a.window + 1;
  }
  hi = min(hi, a.s.width << a.c.shift);
}

__device__ inline int length_of(const AttnArgs& a, int b) { return max(a.kv_len[b], 0); }

__device__ inline void write_row(const AttnArgs& a, int64_t at, int n, const float* x) {
  if (a.out_f32) {
    float* p = reinterpret_cast<float*>(a.out) + at;
    for (int i = 0; i < n; ++i) p[i] = x[i];
  } else {
    __bf16* p = reinterpret_cast<__bf16*>(a.out) + at;
    for (int i = 0; i < n; ++i) p[i] = (__bf16)x[i];
  }
}

// Two floats at a time past the caches that the XCDs do not share.
__device__ inline void put2(uint64_t* p, float x, float y, bool on) {
  if (on)
    __hip_atomic_store(p, (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline float2 get2(const uint64_t* p) {
  const uint64_t v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

// The tiles of a part: query rows r0 .. of a sequence with n * G rows see the
// tokens lo .. hi - 1 between them, cut into tiles and those
// into parts of the same number of tiles.
struct Parts {
  int lo, hi;          // of all rows together
  int lo_last, hi_first;  // tokens from lo_last to hi_first are seen by every row
  int first, end;      // tiles
  int span, parts;     // tiles per part, parts that have tiles
};
__device__ inline int over(int x, int y) { return (int)((unsigned)x / (unsigned)y); }
__device__ inline Parts parts_of(const AttnArgs& a, int len, int n, int r0) {
  Parts p;
  const int last = min(r0 + a.tile_rows, n * a.G) - 1;
  row_range(a, len, n, over(r0, a.G), p.lo, p.hi_first);
  row_range(a, len, n, over(last, a.G), p.lo_last, p.hi);
  p.first = p.lo >> a.tile_shift;
  p.end = max(p.first, (p.hi + (1 << a.tile_shift) - 1) >> a.tile_shift);
  p.span = max(a.span_tiles, p.end - p.first);
  p.parts = p.end > p.first ? 1 : 0;
  if (a.nsplit > 1) {
    p.span = max(a.span_tiles, over(p.end - p.first + a.nsplit - 1, a.nsplit));
    p.parts = over(p.end - p.first + p.span - 1, p.span);
  }
  return p;
}

// Workgroup n = ((high * lows + low) * parts + part) * H + h.
struct Place {
  int h, part, low, high;
};
__device__ inline Place place_of(int H, int parts, int lows) {
  Place p;
  int n = blockIdx.x, m = over(n, H);
  p.h = n - m * H;
  p.part = 0;
  if (parts > 1) {
    n = m;
    m = over(n, parts);
    p.part = n - m * parts;
  }
  p.high = over(m, lows);
  p.low = m - p.high * lows;
  return p;
}

// Workgroup barrier that waits for the wavefront's LDS operations only (global
// loads stay in flight).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

extern __shared__ __align__(16) unsigned char smem_kv[];

// ---- few query rows --------------------------------------------------------
// Workgroup: 16 query rows (new tokens x the heads of one kv head) and one
// part of their tokens; its four wavefronts take the part's tiles of 32
// tokens in turn, straight from HBM into registers (the cache order is the
// operand order), the next tile's loads in flight during the current one's
// products.  S^T = K Q^T (16 x 16 x 32, tokens down, rows across), whose
// result registers are the B operand of O^T = V^T P^T: no LDS in the loop, but for
// the second term of fp32 queries.
//
// Bound by HBM, 2 D bytes a token and kv head: 4 sequences of 131072 tokens, 64
// query heads on 8 of 128, 1.07 GB in 191 us, 5.6 TB/s; 32 of up to 4097, 179 MB in
// 44 us, 4.1 TB/s (their lengths differ, and each workgroup starts with a chain
// of loads: lengths, table, codes); heads of 256, 32 of 4096 tokens, 537 MB in 102
// us.  Few tokens: that chain, 5.3 us from launch to launch for a prompt of 16, 7.9
// for one token on 777; heads of 256, one wavefront a SIMD, 8 sequences of 2000
// tokens, 33 MB, 15.8.  More than 16 rows read a sequence once for every 16: 20 rows
// of heads of 64 on 1024 tokens of 8 sequences 9.1 us, 512 workgroups of some nine
// tiles each.  Tiles of 32 rows halve that but leave two wavefronts a SIMD instead
// of three (128 rows on 4096 tokens of 128 heads: 45 -> 54 us).
template <int D>
struct Tile {
  uint4 k[D / 32];  // [16-token half][64-dim chunk]
  uint4 v[D / 32];  // [32-dim chunk]
};

template <int D>
__device__ inline void load_tile(Tile<D>& t, const KvCacheView& c, int id, int h, int tile,
                                 int lane) {
  const int P = 1 << c.shift;
  const int64_t at = ((int64_t)max(id, 0) * c.H + h) * P * D +
                     (int64_t)((tile * kSpan) & (P - 1)) * D;
  const uint4* k = reinterpret_cast<const uint4*>(c.kc + at) + lane;
  const uint4* v = reinterpret_cast<const uint4*>(c.vc + at) + lane;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) t.k[i] = k[64 * i];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) t.v[i] = v[64 * i];
}

template <int D, bool kFine>
__global__ __launch_bounds__(256, D == 256 ? 1 : D == 128 ? 3 : 4) void k_kv_decode(AttnArgs a) {
  constexpr int kSteps = D / 32, kTiles = D / 16, kWaves = 4;
  constexpr int kStride = D + 4;
  const Place at_wg = place_of(a.c.H, a.nsplit, a.row_tiles);
  const int h = at_wg.h, sp = at_wg.part, tile_row = at_wg.low, b = at_wg.high;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int len = length_of(a, b);
  int row0, n;
  kv_rows(a.s, b, row0, n);
  const int rows = n * a.G, r0 = tile_row * kRowTile;
  if (r0 >= rows) return;
  const Parts pt = parts_of(a, len, n, r0);
  const int lo1 = pt.lo_last, hi0 = pt.hi_first;
  const int t0 = pt.first + sp * pt.span, t1 = min(t0 + pt.span, pt.end);
  const int parts = pt.parts;
  // rows that see nothing are left to the first part, or to the join launch
  if (t0 >= t1 && a.nsplit > 1 && !(a.tags && parts == 0 && sp == 0)) return;

  const int r = min(r0 + col, rows - 1);
  const int i = over(r, a.G), hq = h * a.G + r - i * a.G;
  int my_lo, my_hi;
  row_range(a, len, n, i, my_lo, my_hi);

  // query fragments: slots (g, e) of step 2c + u are dims 64c + 16g + 8u + e
  half8 q[kSteps];
  float down;
  {
    Raw8 raw[kSteps];
    const int64_t at = (int64_t)(row0 + i) * a.qts + (int64_t)hq * a.qhs + 16 * g;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      raw[s] = load8(a.q, a.q_f32, at + 64 * (s >> 1) + 8 * (s & 1));
    half8 rest[kFine ? kSteps : 1];
    query_fragments<kFine, kSteps, 16>(raw, a.q_f32, q, rest, down);
    if constexpr (kFine) {
      // into the wavefront's part of what holds its results in the end, read again in
      // every tile: in registers they would take a wavefront a SIMD
      half8* to = reinterpret_cast<half8*>(reinterpret_cast<float*>(smem_kv) + wave * 16 * kStride) + lane;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) to[64 * s] = rest[s];
    }
  }
  const float cq = a.c2 * down;

  f32x4 o[kTiles];
#pragma unroll
  for (int d = 0; d < kTiles; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  // limit: of the exponents x + log2 s, M + kTop; -inf for a row whose off is in use
  float M = kNone, off = 0.f, limit = kNone, L = 0.f, Mz = kNone, Lz = 0.f;
  uint32_t least = kNoScale;

  // Lane j holds the block and the scales of this wavefront's j-th tile (of a
  // batch of 64), so that a tile's loads wait for no chain of their own.
  int id = 0;
  float sk = 0.f, lam = 0.f, inv = 1.f;
  auto batch_at = [&](int t) {
    const int64_t mine = (int64_t)t + kWaves * lane;
    id = mine < t1 ? kv_block(a.c, a.s, b, mine >> (a.c.shift - 5)) : -1;
    const int64_t hb = (int64_t)max(id, 0) * a.c.H + h;
    sk = a.c.ks[hb];
    value_scale(a.c.vs[hb], lam, inv);
  };
  auto work = [&](const Tile<D>& tl, int t, int j) {
    if (__builtin_amdgcn_readlane(id, j) < 0) return;  // an absent block
    f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
    const half8* rest = nullptr;
    if constexpr (kFine) {
      int at = wave * 16 * kStride * 4 + 16 * lane;
      asm volatile("" : "+v"(at));  // not to be read ahead of the loop
      rest = reinterpret_cast<const half8*>(smem_kv + at);
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const uint4 k0 = tl.k[c], k1 = tl.k[D / 64 + c];
      auto add = [&](f32x4& to, uint32_t w0, uint32_t w1, int step) {
        const half8 k = codes_f16x8(w0, w1);
        to = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[step], to, 0, 0, 0);
        if constexpr (kFine)
          to = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, rest[64 * step], to, 0, 0, 0);
      };
      add(s0, k0.x, k0.y, 2 * c);
      add(s1, k1.x, k1.y, 2 * c);
      add(s0, k0.z, k0.w, 2 * c + 1);
      add(s1, k1.z, k1.w, 2 * c + 1);
    }
    // lane (col, g): scores of row col at tokens 4g + 0..3 and 16 + 4g + 0..3
    const float f = fmaxf(cq * __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sk), j)), kTinyStep);
    const float lm = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lam), j));
    const uint32_t in = __builtin_amdgcn_readlane(__float_as_int(inv), j);
    const int tok = t * kSpan;
    if (tok < lo1 || tok + kSpan > hi0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = tok + 4 * g + e;
        if (p < my_lo || p >= my_hi) s0[e] = -INFINITY;
        if (p + 16 < my_lo || p + 16 >= my_hi) s1[e] = -INFINITY;
      }
    }
    uint32_t in_l = in;  // what its weights have in L
    if (is_special(in, least) && meet_scale(in, least)) {
      const float z[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
      add_zeros<16>(z, f, Mz, Lz);
      in_l = 0;
    }
    float most = fmaxf(fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s0[2], s0[3])),
                       fmaxf(fmaxf(s1[0], s1[1]), fmaxf(s1[2], s1[3])));
    float ff = f, add = lm - M;
    if (__any(fmaf(most, f, lm) > limit)) {
      most = fmaxf(most, __shfl_xor(most, 16));
      most = score_of(fmaxf(most, __shfl_xor(most, 32)), f);
      if ((most - M) + (lm - off) > kTop) {
        bool far;
        const float al = move_reference(most, lm, M, off, L, far);
        limit = far ? -INFINITY : M + kTop;
#pragma unroll
        for (int d = 0; d < kTiles; ++d) o[d] *= al;
      }
      add = lm - M;
      if (limit == -INFINITY) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s0[e] = (score_of(s0[e], f) - M) + (lm - off);
          s1[e] = (score_of(s1[e], f) - M) + (lm - off);
        }
        ff = 1.f;
        add = 0.f;
      }
    }
    float sum = 0.f;
    half8 p;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float w = exp2_fast(fmaf(e < 4 ? s0[e & 3] : s1[e & 3], ff, add));
      sum += w;
      p[e] = (_Float16)w;
    }
    L = fmaf(sum, __uint_as_float(in_l), L);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const uint4 v = tl.v[c];
      o[2 * c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16x8(v.x, v.y), p, o[2 * c], 0, 0, 0);
      o[2 * c + 1] =
          __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16x8(v.z, v.w), p, o[2 * c + 1], 0, 0, 0);
    }
  };
  for (int tb = t0 + wave; tb < t1; tb += 64 * kWaves) {
    batch_at(tb);
    const int tiles = min(64, (t1 - tb + kWaves - 1) / kWaves);
    Tile<D> ta, tc;
    auto fetch = [&](Tile<D>& tl, int j) {
      load_tile<D>(tl, a.c, __builtin_amdgcn_readlane(id, j), h, tb + kWaves * j, lane);
    };
    fetch(ta, 0);
    for (int j = 0; j < tiles; j += 2) {
      if (j + 1 < tiles) fetch(tc, j + 1);
      work(ta, tb + kWaves * j, j);
      if (j + 1 >= tiles) break;
      if (j + 2 < tiles) fetch(ta, j + 2);
      work(tc, tb + kWaves * (j + 1), j + 1);
    }
  }

  // join the wavefronts: M and L per row, then the weighted sum of O
  float grown = one_reference(M, off, L);
  grown *= join_zeros<16>(M, L, Mz, Lz);
  float* lo_o = reinterpret_cast<float*>(smem_kv);           // [wave][16][kStride]
  float* lo_m = lo_o + kWaves * 16 * kStride;                 // [wave][16]
  float* lo_l = lo_m + kWaves * 16;
  float* lo_g = lo_l + kWaves * 16;  // O's factor
#pragma unroll
  for (int d = 0; d < kTiles; ++d)
    *reinterpret_cast<f32x4*>(lo_o + (wave * 16 + col) * kStride + 16 * d + 4 * g) = o[d];
  if (g == 0) {
    lo_m[wave * 16 + col] = M;
    lo_l[wave * 16 + col] = L;
    lo_g[wave * 16 + col] = grown;
  }
  __syncthreads();
  constexpr int kPer = D / 4 / kWaves;  // outputs per thread, 4 kWaves threads a row
  const int rr = threadIdx.x / (4 * kWaves), d0 = threadIdx.x % (4 * kWaves) * kPer;
  float m = kNone;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = fmaxf(m, lo_m[w * 16 + rr]);
  float x[kPer], l = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float f = half_exp2(lo_m[w * 16 + rr] - m);
    l += f * lo_l[w * 16 + rr] * f;
    const float fo = f * f * lo_g[w * 16 + rr];
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] += fo * lo_o[(w * 16 + rr) * kStride + d0 + e];
  }
  const int ro = min(r0 + rr, rows - 1);
  const int io = over(ro, a.G);
  const int64_t orow = (int64_t)(row0 + io) * a.Hq + h * a.G + ro - io * a.G;
  const int64_t step = (int64_t)a.s.total * a.Hq;
  const bool mine = r0 + rr < rows;
  if (a.tags ? parts > 1 : a.nsplit > 1) {
    if (mine) {
      put2(reinterpret_cast<uint64_t*>(a.part_ml + sp * step + orow), m, l, d0 == 0);
      uint64_t* po = reinterpret_cast<uint64_t*>(a.part_o + (sp * step + orow) * D + d0);
#pragma unroll
      for (int e = 0; e < kPer; e += 2) put2(po + e / 2, x[e], x[e + 1], true);
    }
    if (!a.tags) return;
    // Join here if this part is the last to come.  The device-scope stores above
    // have reached the level that all XCDs share once vmcnt is 0; only then is
    // the part's tag stored, and the tags are looked at after that, so the part
    // whose tag comes last sees all of them.  (Two parts may both see all: they
    // write the same results.)  A tag is this call's number, so whatever the
    // workspace held before counts as not there; whoever joins clears the tags,
    // for a graph replays the same number.
    __shared__ int complete;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (wave == 0) {
      uint64_t* tags = a.tags + (((int64_t)b * a.row_tiles + tile_row) * a.c.H + h) * kMostParts;
      if (lane == 0)
        __hip_atomic_store(tags + sp, a.call, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const bool there =
          lane >= parts ||
          __hip_atomic_load(tags + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.call;
      const bool all = __all(there);
      if (all && lane < parts)
        __hip_atomic_store(tags + lane, (uint64_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (lane == 0) complete = all;
    }
    __syncthreads();
    if (!complete || !mine) return;
    // four parts' loads in flight at a time, the sums rescaled as M moves
    m = kNone;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = 0.f;
    for (int p0 = 0; p0 < parts; p0 += 4) {
      float2 ml[4], v[4][kPer / 2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = min(p0 + j, parts - 1) * step + orow;
        ml[j] = get2(reinterpret_cast<const uint64_t*>(a.part_ml + at));
        const uint64_t* po = reinterpret_cast<const uint64_t*>(a.part_o + at * D + d0);
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) v[j][e] = get2(po + e);
        if (p0 + j >= parts) ml[j] = make_float2(kNone, 0.f);
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, ml[j].x);
      const float al = half_exp2(m - top);
      l = l * al * al;
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[e] *= al * al;
      m = top;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p0 + j >= parts) break;
        const float f = half_exp2(ml[j].x - m), w = f * f;
        l = fmaf(f * ml[j].y, f, l);
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) {
          x[2 * e] = fmaf(w, v[j][e].x, x[2 * e]);
          x[2 * e + 1] = fmaf(w, v[j][e].y, x[2 * e + 1]);
        }
      }
    }
  }
  if (!mine) return;
  const float f = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = l == 0.f ? 0.f : x[e] * f;
  write_row(a, orow * D + d0, kPer, x);
  if (a.lse && d0 == 0) a.lse[orow] = l == 0.f ? -INFINITY : kLn2 * (m + log2_fast(l));
}

// ---- many query rows -------------------------------------------------------
// Workgroup: wavefronts of 32 query rows of one kv head, over one part of their
// tokens, a stage of 64 tokens at a time.  S^T = K Q^T (32 x 32 x 16), softmax in
// registers, O^T += V^T P^T with the score registers as operand: inside 32
// tokens the key rows are placed so that those registers hold the weights in
// the order of the value codes (token t is row t with bits 3 and 4 swapped).
//
// The workgroup turns each stage's codes into f16 once, in LDS, in operand
// order, from registers loaded a stage before.  Half a stage (32 tokens, a
// strip) at a time, a wavefront multiplies the values of strip i - 1 and the
// keys of strip i + 1 while it turns the scores of strip i into weights: the
// three do not depend on each other, so its vector instructions run between its
// matrix instructions.  LDS holds four strips of keys and four of values, in
// turn; one barrier a stage.
//
// Bound by the matrix and the vector instructions together, and by the clock
// that the card holds under them (1.9 to 2.0 GHz): 2048 tokens, 64 query heads on
// 8 of 128, on 32049 tokens, 2.08 Tflop in 1.84 to 1.91 ms over cards, 1.1
// Pflop/s; matrix units busy 56% of the time, vector units 58% (16 exponentials, at a
// quarter of the rate, and some 60 other instructions a strip and 16 products), the
// LDS 35%, no bank conflicts.  2048 on 16000, heads of 64 (128 of them) 1220 us,
// matrix 35%, vector 62%; of 256 (32) 1084 us, 40% and 38%, LDS 30%, one wavefront a
// SIMD.  A prompt from its start: 2048 tokens, 32 heads on 8 of 128, 63 us, 26 at the
// matrix rate: its 256 workgroups, one a compute unit, have 1 to 32 stages, so the
// units are at work half of the time.  Tried and slower: stages of 128 tokens (1900 ->
// 1925 us), 4 or 8 operands read ahead instead of 2 (1%), two groups of wavefronts
// that alternate between products and softmax (1972 -> 2090), 64 rows a
// wavefront (1850 -> 2430: past 256 registers every operand is copied between the
// two files), the row sums as dot products of the rounded weights (1846 ->
// 1855).
template <int D, int W>
struct Prefill {
  static constexpr int kStrips = 2;                // a stage
  static constexpr int kStage = 32 * kStrips;      // tokens
  static constexpr int kSteps = D / 16, kTiles = D / 32;
  static constexpr int kWaves = W;
  static constexpr int kThreads = 64 * kWaves, kRows = 32 * kWaves;
  static constexpr int kUnits = 4 * kStrips * D / kThreads;  // 16-byte pieces of keys and values a thread
  static constexpr int kStrip = 4 * D;             // 16-byte pieces of a strip in LDS
  static constexpr int kProducts = kSteps + 2 * kTiles;  // of a strip: keys, then values
  static constexpr int kPage = 32 * 16;            // 16-byte pieces of a wavefront's 32 rows x 64 results
  static constexpr int kRingPieces = 4 * kStrips * kStrip;
  static constexpr int kLds =                      // bytes: the strips, and then the results
      16 * (kRingPieces > kWaves * kPage ? kRingPieces : kWaves * kPage);
  static constexpr int kAhead = 2;                 // operands read from LDS before their product
  // which of the stage's strips a thread's piece u is of (the same in a wavefront,
  // and known here or the same for all its pieces, which then share its address)
  __device__ static int strip_of(int u) {
    static_assert(2 * D % kThreads == 0 || kThreads % (2 * D * kStrips) == 0);
    if constexpr (2 * D % kThreads == 0)
      return kThreads * u / (2 * D) & (kStrips - 1);
    else
      return __builtin_amdgcn_readfirstlane(threadIdx.x) / (2 * D) & (kStrips - 1);
  }
  // whether a thread's piece u is one of the values' (the same in a wavefront)
  __device__ static int kind(int u) {
    if constexpr (kThreads > 2 * kStrips * D)
      return __builtin_amdgcn_readfirstlane(threadIdx.x) / (2 * kStrips * D);
    else
      return kThreads * u / (2 * kStrips * D);
  }
};

template <int D, int W, bool kFine>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void k_kv_prefill(AttnArgs a) {
  using C = Prefill<D, W>;
  constexpr int kStage = C::kStage, kSteps = C::kSteps, kTiles = C::kTiles;
  constexpr int kProducts = C::kProducts, kAhead = C::kAhead, kStrips = C::kStrips;
  constexpr int kRing = 2 * kStrips, kBatch = 64 / kStrips;
  const Place at_wg = place_of(a.c.H, a.nsplit, a.s.batch);
  const int h = at_wg.h, sp = at_wg.part, b = at_wg.low;
  const int tile_row = a.row_tiles - 1 - at_wg.high;  // the longest rows first
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, half = lane >> 5;
  // Blocks of the strips: lane j holds that of the j-th strip of a batch of 64,
  // read with vector loads two batches ahead (scalar loads would share their
  // counter with the LDS reads, so that every stage waited for them).  The first
  // ones are read from where the part begins unless it has a window or more
  // tokens than the plan knew of, beside the lengths and not after them.
  auto blocks_at = [&](int t) {  // of the batch that begins at stage t
    return kv_block(a.c, a.s, b, ((int64_t)t * kStage + 32 * lane) >> a.c.shift);
  };
  const int guess = sp * a.span_tiles;
  int id0 = blocks_at(guess), id1 = blocks_at(guess + kBatch), id2 = blocks_at(guess + 2 * kBatch);
  const int len = length_of(a, b);
  int row0, n;
  kv_rows(a.s, b, row0, n);
  const int rows = n * a.G, r0 = tile_row * C::kRows;
  if (r0 >= rows) return;
  const Parts pt = parts_of(a, len, n, r0);
  const int t0 = pt.first + sp * pt.span, t1 = min(t0 + pt.span, pt.end);
  if (t0 >= t1 && a.nsplit > 1) return;
  if (t0 != guess) id0 = blocks_at(t0), id1 = blocks_at(t0 + kBatch), id2 = blocks_at(t0 + 2 * kBatch);

  // this wavefront's rows (past the end: the last row again, never written)
  const int w0 = r0 + 32 * wave;
  const int r = min(w0 + col, rows - 1);
  const int i = over(r, a.G), hq = h * a.G + r - i * a.G;
  Raw8 qraw[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    qraw[s] = load8(a.q, a.q_f32, (int64_t)(row0 + i) * a.qts + (int64_t)hq * a.qhs + 8 * half + 16 * s);
  int my_lo, my_hi;
  row_range(a, len, n, i, my_lo, my_hi);
  int w_lo, w_hi, w_lo_last, w_hi_first;
  row_range(a, len, n, over(min(w0, rows - 1), a.G), w_lo, w_hi_first);
  row_range(a, len, n, over(min(w0 + 31, rows - 1), a.G), w_lo_last, w_hi);
  if (w0 >= rows) w_hi = 0;
  // its stages: a0 .. a1 - 1 (none: a0 == a1)
  const int a0 = min(max(t0, w_lo / kStage), t1);
  const int a1 = max(a0, min(t1, (w_hi + kStage - 1) / kStage));

  f32x16 o[kTiles];
#pragma unroll
  for (int d = 0; d < kTiles; ++d) o[d] = f32x16{};
  // limit: of the sums of weights; below all of them for a row whose off is in use
  float M = kNone, off = 0.f, limit = kTopWeight, L = 0.f, Mz = kNone, Lz = 0.f;
  uint32_t least = kNoScale;

  // The strips' scales, held like their blocks and read a batch ahead.
  const int P = 1 << a.c.shift;
  struct Scales {
    float sk, lam, inv;  // keys' scale; values': log2 and inverse
  };
  auto scales_at = [&](int t, int id) {
    // a strip past the end: its block may be absent or never written, whose
    // scales may be anything
    const bool none = id < 0 || (int64_t)t * kStage + 32 * lane >= len;
    const int64_t hb = (int64_t)max(id, 0) * a.c.H + h;
    Scales s;
    s.sk = none ? 0.f : a.c.ks[hb];
    value_scale(none ? 1.f : a.c.vs[hb], s.lam, s.inv);
    return s;
  };
  int batch = kStrips * t0;  // its first strip
  auto id_of = [&](int i) {  // a strip of this batch, the next one, or just before
    const int j = i - batch;
    return __builtin_amdgcn_readlane(j < 64 ? id0 : id1, j & 63);
  };

  // this thread's pieces of the keys of strips ik, ik + 1 and of the values of
  // strips iv, iv + 1, into registers
  const int64_t block_bytes = (int64_t)a.c.H * P * D;
  const uint8_t* const kc = a.c.kc + (int64_t)h * P * D;
  const uint8_t* const vc = a.c.vc + (int64_t)h * P * D;
  typedef uint4 Codes[C::kUnits];
  auto load_one = [&](Codes& st, int ik, int iv, int u) {
    const int n = C::kThreads * u + (int)threadIdx.x, kind = C::kind(u);
    const int i = (kind ? iv : ik) + C::strip_of(u);
    const int64_t blk = max(id_of(i), 0) * block_bytes;
    const uint32_t at = (uint32_t)(((32 * i) & (P - 1)) * D + 16 * (n & (2 * D - 1)));
    st[u] = *reinterpret_cast<const uint4*>((kind ? vc : kc) + blk + at);
  };
  auto load = [&](Codes& st, int ik, int iv) {
#pragma unroll
    for (int u = 0; u < C::kUnits; ++u) load_one(st, ik, iv, u);
  };
  // The keys of the first three strips and the values of the first; the strip of
  // values before it is multiplied by weights of 0, so it gets finite numbers.
  Codes st, st0, st1;
  const int i0 = kStrips * t0;
  load(st0, i0 - kStrips + 1, i0 - 1);
  load(st1, i0 + 1, i0 + kStrips - 1);
  load(st, i0 + kStrips + 1, i0 + kStrips - 1);
  Scales sc0 = scales_at(t0, id0), sc1 = scales_at(t0 + kBatch, id1);
  auto lane_of = [&](float x, int i) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), i - batch));
  };

  half8 q[kSteps];  // slots (half, e) of step s are dims 16 s + 8 half + e
  float down;
  half8 rest[kFine ? kSteps : 1];
  query_fragments<kFine, kSteps, 32>(qraw, a.q_f32, q, rest, down);
#ifdef __HIP_DEVICE_COMPILE__
  // Head dim 256: into the accumulation registers, from which the products read
  // them too (left to itself the compiler moves them there and back in every
  // strip: 1097 -> 1055 us for 2048 rows of 32 heads on 16000 tokens).
  if constexpr (D == 256) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) asm volatile("" : "+a"(q[k]));
  }
#endif
  const float cq = a.c2 * down;

  // and from there as f16 into LDS: keys [strip][step][half][row], values
  // [strip][d tile][step][half][d], 16 bytes each
  half8* const lds = reinterpret_cast<half8*>(smem_kv);
  auto convert_half = [&](const Codes& st, int ik, int iv, int u, int second) {
    const int n = C::kThreads * u + (int)threadIdx.x, kind = C::kind(u);
    const int m = n & (2 * D - 1), g = m % 64 / 16;
    const int i = (kind ? iv : ik) + C::strip_of(u);
    const int tok = 16 * (m / D) + (m & 15);
    half8* p = lds + (kRing * kind + (i & (kRing - 1))) * C::kStrip +
               (kind ? (4 * (m / 64) + g) * 32 + (m & 15)
                     : (4 * (m % D / 64) + g) * 64 + ((tok & 7) | (tok & 8) << 1 | (tok & 16) >> 1));
    p[second * (kind ? 16 : 32)] =
        second ? codes_f16x8(st[u].z, st[u].w) : codes_f16x8(st[u].x, st[u].y);
  };
  auto convert = [&](const Codes& st, int ik, int iv) {
#pragma unroll
    for (int j = 0; j < 2 * C::kUnits; ++j) convert_half(st, ik, iv, j >> 1, j & 1);
  };
  // operand m of strip i's products: the keys of strip i + 1, then the values
  // of strip i - 1
  auto operand = [&](int i, int m) {
    const half8* kl = lds + ((i + 1) & (kRing - 1)) * C::kStrip + lane;
    const half8* vl = lds + (kRing + ((i - 1) & (kRing - 1))) * C::kStrip + lane;
    const int v = m - kSteps;
    return m < kSteps ? kl[m * 64] : vl[(2 * (v % kTiles) + v / kTiles) * 64];
  };
  half8 fr[kAhead];
  auto values = [&](int i, const half8 (&p)[2]) {
#pragma unroll
    for (int v = 0; v < 2 * kTiles; ++v)
      o[v % kTiles] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
          operand(i + 1, kSteps + v), p[v / kTiles], o[v % kTiles], 0, 0, 0);
  };
  // Strip i: its scores s -> weights p; scores sn of strip i + 1; values of strip
  // i - 1 by their weights pp.  Lane (col, half), register e: row col, token
  // 8 (e / 8) + 4 half + e % 4 + 16 (e / 4 % 2).
  auto strip = [&](int i, f32x16& s, f32x16& sn, half8 (&p)[2], const half8 (&pp)[2], auto which) {
    constexpr int kWhich = decltype(which)::value;  // of its stage
    const int tok = 32 * i;
    const bool gone = __builtin_amdgcn_readlane(id0, i - batch) < 0;
    const float f = fmaxf(cq * lane_of(sc0.sk, i), kTinyStep);
    const float lam = lane_of(sc0.lam, i), inv = lane_of(sc0.inv, i);
    if (tok < w_lo_last || tok + 32 > w_hi_first || gone) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int at = tok + 8 * (e >> 3) + 4 * half + (e & 3) + 16 * ((e >> 2) & 1);
        if (at < my_lo || at >= my_hi || gone) s[e] = -INFINITY;
      }
    }
    const float add = lam - M;
    float w[16], sum = 0.f;
    half2v pairs[8];
    sn = f32x16{};
    // (the empty asm statements keep each result at its place in this order)
    auto use = [&](int e) {
      sum += w[e];
      asm volatile("" : "+v"(sum));
      if (e & 1) {
        pairs[e >> 1] = half2v{(_Float16)w[e - 1], (_Float16)w[e]};
        asm volatile("" : "+v"(pairs[e >> 1]));
      }
    };
    // A product, the read of a later one's operand, and a share of the vector
    // work at a time, in this order: the scheduler left to itself reads operands
    // right before their products and gathers the vector work at the end.
#pragma unroll
    for (int m = 0; m < kProducts; ++m) {
      const int v = m - kSteps;
      if (m < kSteps) {
        sn = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr[m % kAhead], q[m], sn, 0, 0, 0);
        if constexpr (kFine)
          sn = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr[m % kAhead], rest[m], sn, 0, 0, 0);
      } else
        o[v % kTiles] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr[m % kAhead], pp[v / kTiles],
                                                               o[v % kTiles], 0, 0, 0);
      if (m + kAhead < kProducts)
        fr[m % kAhead] = operand(i, m + kAhead);
      else if (kWhich < kStrips - 1)
        fr[m % kAhead] = operand(i + 1, m + kAhead - kProducts);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e * kProducts / 16 != m) continue;
        w[e] = exp2_fast(fmaf(s[e], f, add));
        if (e >= 2) use(e - 2);
      }
      // a stage's first strip converts, its second one loads
      if constexpr (kWhich == 0) {
#pragma unroll
        for (int j = 0; j < 2 * C::kUnits; ++j)
          if (j * kProducts / (2 * C::kUnits) == m)
            convert_half(st, i + kStrips + 1, i + kStrips - 1, j >> 1, j & 1);
      } else {
#pragma unroll
        for (int u = 0; u < C::kUnits; ++u)
          if (u * kProducts / C::kUnits == m)
            load_one(st, i - 1 + 2 * kStrips + 1, i - 1 + 2 * kStrips - 1, u);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    use(14);
    use(15);
    // Every weight is below 2^kTop unless some lane's sum is not (a sum of NaN is
    // a row of NaN); only then is M moved and are the weights made again.
    const uint32_t in = __float_as_uint(inv);
    if (in != 0 && __any(sum > limit)) {
      float most = s[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) most = fmaxf(most, s[e]);
      most = score_of(fmaxf(most, __shfl_xor(most, 32)), f);
      if ((most - M) + (lam - off) > kPlace) {
        bool far;
        const float al = move_reference(most, lam, M, off, L, far);
        limit = far ? -1.f : kTopWeight;
#pragma unroll
        for (int d = 0; d < kTiles; ++d) o[d] *= al;
      }
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = limit < 0.f ? (score_of(s[e], f) - M) + (lam - off) : fmaf(s[e], f, lam - M);
        const float y = exp2_fast(x);
        sum += y;
        pairs[e >> 1][e & 1] = (_Float16)y;
      }
    }
    uint32_t in_l = in;  // what its weights have in L
    if (is_special(in, least) && meet_scale(in, least)) {
      float z[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) z[e] = s[e];
      add_zeros<32>(z, f, Mz, Lz);
      in_l = 0;
    }
    L = fmaf(sum, __uint_as_float(in_l), L);
    asm volatile("" : "+v"(L));
#pragma unroll
    for (int e = 0; e < 16; ++e) p[e >> 3][e & 7] = pairs[e >> 1][e & 1];
  };

  if (t0 < t1) {
    f32x16 sa, sb;
    half8 pa[2], pb[2];
    pa[0] = pa[1] = pb[0] = pb[1] = half8{};
    convert(st0, i0 - kStrips + 1, i0 - 1);
#pragma unroll
    for (int u = 0; u < C::kUnits; ++u)
      if (C::kind(u) == 0) {  // its values have no place yet
        convert_half(st1, i0 + 1, 0, u, 0);
        convert_half(st1, i0 + 1, 0, u, 1);
      }
    lds_barrier();
    sa = f32x16{};
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      sa = __builtin_amdgcn_mfma_f32_32x32x16_f16(operand(i0 - 1, k), q[k], sa, 0, 0, 0);
      if constexpr (kFine)
        sa = __builtin_amdgcn_mfma_f32_32x32x16_f16(operand(i0 - 1, k), rest[k], sa, 0, 0, 0);
    }
    lds_barrier();  // the first stage's conversion takes the place of these keys
    auto next_batch = [&](int t) {
      if (kStrips * t - batch == 64) {
        batch = kStrips * t;
        id0 = id1, sc0 = sc1, id1 = id2;
        sc1 = scales_at(t + kBatch, id1);
        id2 = blocks_at(t + 2 * kBatch);
      }
    };
    auto convert_only = [&](int t) {
      next_batch(t);
      convert(st, kStrips * (t + 1) + 1, kStrips * (t + 1) - 1);
      load(st, kStrips * (t + 2) + 1, kStrips * (t + 2) - 1);
      lds_barrier();
    };
    // outside its own stages a wavefront only converts; the stage before them
    // and the one after are worked through as masked ones
    int t = t0;
    for (; t < a0 - 1; ++t) convert_only(t);
    for (const int end = min(a1 + 1, t1); t < end; ++t) {
      next_batch(t);
      const int i = kStrips * t;
#pragma unroll
      for (int m = 0; m < kAhead; ++m) fr[m] = operand(i, m);
      strip(i, sa, sb, pa, pb, std::integral_constant<int, 0>{});
      strip(i + 1, sb, sa, pb, pa, std::integral_constant<int, 1>{});
      lds_barrier();
    }
    if (a1 >= t1) values(kStrips * t1 - 1, pb);
    for (; t < t1; ++t) convert_only(t);
  }

  // Out through LDS, 64 dims at a time, so that a store instruction writes whole
  // lines (from the registers it would write 16 bytes of each of 32 rows; with
  // the early table loads, two sequences of 2048 tokens 78.5 -> 73.6 us).
  // Register e of tile d: dim 32 d + 8 (e / 4) + 4 half + e % 4.
  float grown = one_reference(M, off, L);
  grown *= join_zeros<32>(M, L, Mz, Lz);
  const int orow = (row0 + i) * a.Hq + hq;  // total * q_heads < 2^31
  const int64_t first = a.nsplit > 1 ? (int64_t)sp * a.s.total * a.Hq : 0;  // part's first row
  const float f = grown * (a.nsplit > 1 ? 1.f : L == 0.f ? 0.f : 1.f / L);
  float4* const page = reinterpret_cast<float4*>(smem_kv) + wave * C::kPage;  // [row][4 dims]
  lds_barrier();
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = L == 0.f ? 0.f : o[2 * c + d][e + k] * f;
        page[col * 16 + ((8 * d + e / 2 + half) ^ (col & 15))] = make_float4(x[0], x[1], x[2], x[3]);
      }
    __builtin_amdgcn_wave_barrier();  // the page is this wavefront's own
    if (a.nsplit > 1 || a.out_f32) {
      float* to = a.nsplit > 1 ? a.part_o : reinterpret_cast<float*>(a.out);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int rr = 4 * k + (lane >> 4), v = lane & 15;
        const int64_t at = (first + __shfl(orow, rr)) * D + 64 * c + 4 * v;
        const float4 x = page[rr * 16 + (v ^ (rr & 15))];
        if (w0 + rr < rows) *reinterpret_cast<float4*>(to + at) = x;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int rr = 8 * k + (lane >> 3), v = lane & 7;
        const int64_t at = (int64_t)__shfl(orow, rr) * D + 64 * c + 8 * v;
        const float4 x = page[rr * 16 + (2 * v ^ (rr & 15))], y = page[rr * 16 + ((2 * v + 1) ^ (rr & 15))];
        union {
          __bf16 b[8];
          uint4 u;
        } w;
        w.b[0] = (__bf16)x.x, w.b[1] = (__bf16)x.y, w.b[2] = (__bf16)x.z, w.b[3] = (__bf16)x.w;
        w.b[4] = (__bf16)y.x, w.b[5] = (__bf16)y.y, w.b[6] = (__bf16)y.z, w.b[7] = (__bf16)y.w;
        if (w0 + rr < rows)
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at) = w.u;
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  if (half == 0 && w0 + col < rows) {
    if (a.nsplit > 1)
      a.part_ml[first + orow] = make_float2(M, L);
    else if (a.lse)
      a.lse[orow] = L == 0.f ? -INFINITY : kLn2 * (M + log2_fast(L));
  }
}

// ---- the join of a split call ----------------------------------------------
// kWaves wavefronts (1 or 4) take one query row and head.  Lane j of each holds
// part j's M and L (at most 64 parts); each wavefront adds up its share of the
// parts, in order, and with four of them one another's sums.  Bound by its
// chain of loads (lengths, M and L, partial sums), 2 to 3 us, or for many rows by
// the partials' traffic, 4 D bytes a row and part.
template <int D, int kWaves>
__global__ __launch_bounds__(256) void k_kv_join(AttnArgs a, int rows) {
  constexpr int kPer = D / 64;
  __shared__ float sums[kWaves == 4 ? 4 : 1][D];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mine = kWaves == 4 ? wave : 0;
  const int id = kWaves == 4 ? blockIdx.x : 4 * blockIdx.x + wave;
  if (id >= rows) return;
  const int row = over(id, a.Hq), hq = id - row * a.Hq, b = over(row, a.s.max_count);
  const int i = row - b * a.s.max_count;
  int row0, n;
  kv_rows(a.s, b, row0, n);
  if (i >= n) return;
  const int len = length_of(a, b);
  // the row tile this row was in, as the split kernel saw it
  const int r = i * a.G + hq - over(hq, a.G) * a.G;
  const Parts pt = parts_of(a, len, n, over(r, a.tile_rows) * a.tile_rows);
  const int parts = pt.parts;
  const int64_t orow = (int64_t)(row0 + i) * a.Hq + hq, step = (int64_t)a.s.total * a.Hq;
  const float2 ml = lane < parts ? a.part_ml[lane * step + orow] : make_float2(kNone, 0.f);
  const int each = (parts + kWaves - 1) / kWaves, p1 = min(parts, (mine + 1) * each);
  const float* po = a.part_o + orow * D + lane * kPer;
  float v[4][kPer], sum[kPer];
  auto fetch = [&](int p) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[j][e] = po[min(p + j, p1 - 1) * step * D + e];
  };
  int p = mine * each;
  if (p < p1) fetch(p);
  float m = ml.x;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
  const float h = half_exp2(ml.x - m), f = h * h;
  float l = h * ml.y * h;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);
#pragma unroll
  for (int e = 0; e < kPer; ++e) sum[e] = 0.f;
  for (; p < p1; p += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), (p + j) & 63));
#pragma unroll
      for (int e = 0; e < kPer; ++e) sum[e] = p + j < p1 ? fmaf(w, v[j][e], sum[e]) : sum[e];
    }
    if (p + 4 < p1) fetch(p + 4);
  }
  if constexpr (kWaves == 4) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) sums[wave][lane * kPer + e] = sum[e];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int d = lane * kPer + e;
      sum[e] = sums[0][d] + sums[1][d] + (sums[2][d] + sums[3][d]);
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) sum[e] = l == 0.f ? 0.f : sum[e] / l;
  write_row(a, orow * D + lane * kPer, kPer, sum);
  if (a.lse && lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : kLn2 * (m + log2_fast(l));
}

// ---- host ------------------------------------------------------------------
struct AttnPlan {
  int waves;  // of k_kv_prefill; 0: k_kv_decode
  int tile_rows, tile_tokens, row_tiles, nsplit, span_tiles;
  int64_t blocks;     // workgroups of the attention launch
  size_t workspace, ml_at, tags_at;  // tags_at 0: the parts are joined by a launch of their own
};

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Most parts, and most floats of them, that the last workgroup of a row tile joins
// itself: a second launch costs the host 3 us (one token on 776 cached, 4 query
// heads on each of 8: 9.3 us a call joined inside, 12.4 with a launch), but spreads the
// reads over the GPU.  Timed on the GPU alone, inside and by a launch:
// 7 parts of 4 rows of 128 7.7, 8.7 us; 16 of 4 9.5, 9.9; 16 of 8 13.0, 10.3; 32 of
// one 12.2, 9.0; 16 of 16 rows of 256 58.4, 32.7.
constexpr int kJoinInside = 16, kJoinFloats = 8192;
// Bytes that k_kv_decode reads in all (the cache once for every 16 query rows,
// mostly from the L2s) from which more than kFewRows rows take k_kv_prefill.
// k_kv_decode and k_kv_prefill (the better of its ways), us: head dim 128, 102 MB
// 18.6, 20.5; 262 22.0, 27.2; 393 38.5, 35.6; 410 43.0, 32.8 and 39.3, 37.5; 537 30.1,
// 29.7; 1208 53, 43; 64, 131 MB 19.2, 21.1; 205 29.9, 24.6 and 24.8, 27.4; 262 30.1,
// 31.1; 256, 131 MB 27.6, 28.5; 164 36.0, 32.9 and 205 28.0, 31.4; 262 32.5, 38.8 and
// 30.4, 40.3; 268 34.9, 30.2; 328 57, 42; 524 58, 48.  Around the limits the bytes alone
// do not tell which is faster (how the tiles fill the GPU does too): the one
// taken was up to 10% slower than the other at 128, 22% at 64, a third at 256.  Up
// to kFewRows rows k_kv_decode keeps ahead or level at any size (64 rows, 537 MB 49.6,
// 55.7; 2147 MB 180, 173).
constexpr int64_t decode_bytes(int D) { return D == 256 ? 240000000 : 400000000; }
constexpr int kFewRows = 64;

// A workgroup size of k_kv_prefill: wavefronts, workgroups that the GPU runs at once,
// time of a stage, stages that its start and end take the time of, and the
// stages of a sequence for which it is considered.
//
// With 8 wavefronts a strip is converted for twice the rows.  Head dim 128: two
// wavefronts a SIMD either way, and workgroups of 4 only fill the GPU better
// where sequences are short.  4 and 8 wavefronts, 32 heads on 8, us: prompts from
// their start, 1024 tokens 29.9, 34.5; 1536 43.3, 47.3; 2048 58.3, 61.9; 3000 96.9, 94.9;
// 4096 172, 150; two of 1024 34.5, 36.9, of 1536 60.7, 54.5; four of 1024 57.4, 52.4;
// on longer sequences, 8 x 512 on 1000 73, 70, on 1500 106, 101; 64 heads, 1024 on 8192
// 284, 262.  (The limit of 1024 tokens takes the slower one, by up to 10%, for single
// prompts above it and batches below.)  64: three workgroups of 4 a compute unit or
// one of 8, a tile 1.73 to 1 in time (2048 rows of 128 heads on 16000 tokens 1337,
// 1180 us; 8 x 512 of 64 on 2000 158, 164).
struct Way {
  int waves;
  int64_t slots;
  double tile;
  int64_t start, from, to;
};
constexpr int64_t kAny = (int64_t)1 << 40;
constexpr Way kWays64[2] = {{4, 768, 1.73, 4, 1, kAny}, {8, 256, 1, 10, 1, kAny}};
constexpr Way kWays128[2] = {{4, 512, 1, 4, 1, 16}, {8, 256, 1, 4, 17, kAny}};
constexpr Way kWays256[2] = {{4, 256, 1, 4, 1, kAny}, {4, 256, 1, 4, kAny, 0}};
const Way* ways_of(int D) { return D == 64 ? kWays64 : D == 128 ? kWays128 : kWays256; }

// What the plans of a call's sizes have in common, for any length of its sequences.
struct Shape {
  int D;
  int64_t rows, lists;  // query rows of a head, (sequence, kv head) pairs
  int64_t outputs;      // (query row, head) pairs of all sequences
  bool join;            // the join's grid of (sequence, row, head) fits one launch

  int64_t all(int tile_rows) const { return lists * ((rows + tile_rows - 1) / tile_rows); }
  // A tile's tokens may be in several parts where the most parts of all tiles fit one launch.
  int64_t most_parts(int64_t items) const {
    return join && items <= kMostThreads / 512 / kMostParts ? kMostParts : 1;
  }
  // k_kv_decode's tiles of 32 tokens of `tiles` in a part
  int64_t decode_span(int64_t tiles) const {
    const int64_t want = decode_parts();
    return std::min<int64_t>(std::max<int64_t>(tiles <= 12 ? 12 : 4, (tiles + want - 1) / want), 256);
  }
  int64_t decode_fill() const { return D == 256 ? 256 : 512; }
  int64_t decode_parts() const { return std::max<int64_t>(1, decode_fill() / all(kRowTile)); }
  int64_t decode_tiles() const { return decode_bytes(D) / (2 * D * kSpan); }
  // k_kv_prefill's cost of n parts: rounds of workgroups over the GPU (in fractions where three
  // share a compute unit), each its stages and some more to start and end; where there are
  // several parts, 3 for the join's launch and their traffic (8 MB in the time of a stage).
  double rounds(const Way& w, int64_t n) const {
    const int64_t work = all(32 * w.waves) * n;
    return w.slots == 768 ? std::max(1., (double)work / 768) : (double)((work + w.slots - 1) / w.slots);
  }
  double joining(int64_t n) const { return n > 1 ? 3 + (double)outputs * D * 8 / 8e6 * (double)n : 0; }

  size_t partials(int64_t parts) const {  // bytes of the parts' sums
    return parts > 1 ? ((size_t)(outputs * parts) * D * 4 + 255) / 256 * 256 : 0;
  }
  size_t workspace(int64_t parts) const {  // and of M and L
    return parts > 1 ? partials(parts) + (size_t)(outputs * parts) * 8 : 0;
  }
  int64_t tagged_parts() const {  // the most that the launch itself joins
    return std::min<int64_t>(kJoinInside, kJoinFloats / (std::min<int64_t>(rows, kRowTile) * D));
  }
  size_t tags_at(int64_t parts) const { return (workspace(parts) + 255) / 256 * 256; }
  size_t tags_end(int64_t parts) const {
    return tags_at(parts) + (size_t)all(kRowTile) * kMostParts * 8;
  }
};

// The most workspace that any plan for sequences of up to `longest` tokens needs: more
// tokens can mean fewer parts, since a part's tokens are a whole number of tiles.
size_t most_workspace(const Shape& z, int64_t longest) {
  // k_kv_decode: as many parts as wanted or of 4 tiles, or those of 256 tiles
  int64_t tiles = std::max<int64_t>(1, (longest + kSpan - 1) / kSpan);
  if (z.rows > kFewRows) tiles = std::min(tiles, z.decode_tiles() / z.all(kRowTile));
  int64_t parts = 1;
  if (tiles > 12)
    parts = std::max(std::min(z.decode_parts(), (tiles + 3) / 4), (tiles + 255) / 256);
  parts = std::min(parts, z.most_parts(z.all(kRowTile)));
  size_t most = z.workspace(parts);
  if (const int64_t tagged = std::min(parts, z.tagged_parts()); tagged > 1)
    most = std::max(most, z.tags_end(tagged));
  if (z.rows <= kFewRows) return most;
  // k_kv_prefill: the largest n whose cost is, for some number of stages x that is not
  // beyond `longest`, not above that of any smaller m, with x / n for n's stages a part
  // and (x + m - 1) / m for m's, the least and the most that they can be: each m
  // leaves an interval of x.
  const int64_t stages = std::max<int64_t>(1, (longest + 63) / 64);
  const Way* ways = ways_of(z.D);
  for (int i = 0; i < 2; ++i) {
    const Way& w = ways[i];
    const int64_t end = std::min(stages, w.to);
    for (int64_t n = std::min(end, z.most_parts(z.all(32 * w.waves))); n > 1; --n) {
      if (z.workspace(n) <= most) break;
      double lo = (double)std::max(n, w.from), hi = (double)end;
      const double slope = z.rounds(w, n) * w.tile / (double)n;
      const double fixed = z.rounds(w, n) * (double)w.start * w.tile + z.joining(n);
      for (int j = 0; j < 2 && lo <= hi; ++j) {
        const Way& v = ways[j];
        if ((double)v.from > lo || (double)v.to < hi) continue;
        for (int64_t m = 1; m <= n && lo <= hi; ++m) {
          if (i == j && m == n) continue;
          const double a = slope - z.rounds(v, m) * v.tile / (double)m;
          const double b = z.rounds(v, m) * ((double)(m - 1) / (double)m + (double)v.start) * v.tile +
                           z.joining(m) - fixed + 1e-9 * fixed;
          if (a > 0) hi = std::min(hi, b / a);
          else if (a < 0) lo = std::max(lo, b / a);
          else if (b < 0) hi = lo - 1;
        }
      }
      if (lo <= hi) {
        most = z.workspace(n);
        break;
      }
    }
  }
  return most;
}

// Sizes only; MSQ_OK with blocks == 0 for an empty call.  most: also the most
// workspace of calls with shorter sequences.
msq_status plan_attn(const KvCacheView& c, const KvSeqsView& s, const msq_kv_attn& t, int D,
                     AttnPlan& p, size_t* most = nullptr) {
  p = AttnPlan{};
  if (t.q_heads < 1 || t.q_heads % c.H != 0 || t.window < 0 || t.max_kv_len < 0)
    return MSQ_ERR_SHAPE;
  if (t.window > 0 && !t.causal) return MSQ_ERR_INVALID_ARG;
  if (s.batch == 0 || s.total == 0) return MSQ_OK;
  const int64_t G = t.q_heads / c.H;
  if ((int64_t)s.total * t.q_heads > (int64_t)0x7FFFFFFF ||
      (int64_t)s.max_count * G > (int64_t)0x7FFFFFFF - 256)
    return MSQ_ERR_SHAPE;
  int64_t longest = (int64_t)s.width << c.shift;
  if (t.max_kv_len > 0) longest = std::min(longest, t.max_kv_len);
  if (t.window > 0) longest = std::min<int64_t>(longest, (int64_t)t.window + s.max_count + kSpan);
  const Shape z{D, s.max_count * G, (int64_t)s.batch * c.H, (int64_t)s.total * t.q_heads,
                (int64_t)s.batch * s.max_count * G <= kMostThreads / 256 / c.H};
  const int64_t most_blocks = kMostThreads / 512;
  if (z.lists > most_blocks) return MSQ_ERR_SHAPE;
  int64_t items = 0, tiles = 0, span = 0;
  auto cut = [&](int tile_rows, int tile_tokens) {
    p.tile_rows = tile_rows;
    p.tile_tokens = tile_tokens;
    p.row_tiles = (int)((z.rows + tile_rows - 1) / tile_rows);
    items = z.all(tile_rows);
    tiles = std::max<int64_t>(1, (longest + tile_tokens - 1) / tile_tokens);
  };
  // k_kv_decode.  Parts: about two workgroups a compute unit (one at D = 256, whose
  // registers leave room for one), each 4 to 256 tiles, unsplit up to 12.  More and
  // smaller parts spend longer in their starts and joins (32 sequences of up to
  // 4097 tokens on 8 heads: 2, 3, 4, 8 parts 44, 47, 54, 61 us; 4 of 131072: 16, 32, 64
  // parts 191, 205, 206 us; one of 384 in 1 and 3 parts 6.3, 7.1 us), one a compute
  // unit leaves it idle behind the short sequences (46 us).  D = 256, 8
  // sequences of 2000 on 4 heads: 8 and 16 parts 15.5, 20.3 us.
  cut(kRowTile, kSpan);
  if (items > 16 * most_blocks) return MSQ_ERR_SHAPE;  // a sixteenth as many of k_kv_prefill are too
  span = z.decode_span(tiles);
  const int64_t at_work = std::max(z.decode_fill(), items * ((tiles + span - 1) / span));
  if (z.rows > kFewRows && at_work * std::min(span, tiles) > z.decode_tiles()) {
    // k_kv_prefill, with the parts that cost least
    const int64_t stages = (longest + Prefill<128, 8>::kStage - 1) / Prefill<128, 8>::kStage;
    double least = 1e300;
    for (int i = 0; i < 2; ++i) {
      const Way& w = ways_of(D)[i];
      if (stages < w.from || stages > w.to) continue;
      for (int64_t n = 1; n <= std::min(z.most_parts(z.all(32 * w.waves)), stages); ++n) {
        const int64_t each = (stages + n - 1) / n;
        const double cost = z.rounds(w, n) * (double)(each + w.start) * w.tile + z.joining(n);
        if (cost < least) least = cost, p.waves = w.waves, span = each;
      }
    }
    cut(32 * p.waves, Prefill<128, 8>::kStage);
  }
  p.nsplit = (int)std::min<int64_t>((tiles + span - 1) / span, z.most_parts(items));
  p.span_tiles = (int)((tiles + p.nsplit - 1) / p.nsplit);
  p.blocks = items * p.nsplit;
  if (p.blocks > most_blocks) return MSQ_ERR_SHAPE;
  p.ml_at = z.partials(p.nsplit);
  p.workspace = z.workspace(p.nsplit);
  if (!p.waves && p.nsplit > 1 && p.nsplit <= z.tagged_parts()) {
    p.tags_at = z.tags_at(p.nsplit);
    p.workspace = z.tags_end(p.nsplit);
  }
  if (most) *most = std::max(p.workspace, most_workspace(z, longest));
  return MSQ_OK;
}

// A number for one call: never 0, and from a start that depends on the time, the
// process and where it was loaded, so that no call finds its number in what a
// workspace held before.
uint64_t next_call() {
  static std::atomic<uint64_t> count{0};
  static const uint64_t start = [] {
    uint64_t z = (uint64_t)std::chrono::steady_clock::now().time_since_epoch().count() ^
                 (uint64_t)getpid() << 40 ^ (uint64_t)reinterpret_cast<uintptr_t>(&count);
    z = (z ^ z >> 30) * 0xBF58476D1CE4E5B9u;  // a mix of all bits (splitmix64)
    z = (z ^ z >> 27) * 0x94D049BB133111EBu;
    return z ^ z >> 31;
  }();
  const uint64_t n = start + count.fetch_add(1, std::memory_order_relaxed);
  return n ? n : start + count.fetch_add(1, std::memory_order_relaxed);
}

template <int D, bool kFine>
hipError_t launch_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if (p.waves) {
    auto prefill = [&](auto w) {
      using C = Prefill<D, decltype(w)::value>;
      hipLaunchKernelGGL((k_kv_prefill<D, C::kWaves, kFine>), dim3((unsigned)p.blocks), dim3(C::kThreads),
                         C::kLds, stream, a);
    };
    if constexpr (D != 256)
      if (p.waves == 8) prefill(std::integral_constant<int, 8>{});
    if (p.waves == 4) prefill(std::integral_constant<int, 4>{});
  } else {
    const size_t lds = 4 * kRowTile * (D + 4 + 3) * 4;
    hipLaunchKernelGGL((k_kv_decode<D, kFine>), dim3((unsigned)p.blocks), dim3(256), lds, stream, a);
  }
  if (p.nsplit > 1 && !p.tags_at) {
    const int rows = a.s.batch * a.s.max_count * a.Hq;
    // few rows: four wavefronts each (64 rows of 60 parts: 12.1 -> 9.6 us; 4800 rows of 17
    // parts: 34.7 -> 43.1)
    if (rows <= 1024)
      hipLaunchKernelGGL((k_kv_join<D, 4>), dim3((unsigned)rows), dim3(256), 0, stream, a, rows);
    else
      hipLaunchKernelGGL((k_kv_join<D, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a, rows);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace msq

using namespace msq;

extern "C" msq_status msq_kv_attention_plan(const msq_kv_cache* cache, const msq_kv_seqs* seqs,
                                            const msq_kv_attn* attn, msq_kv_plan* plan) {
  if (!attn || !plan) return MSQ_ERR_INVALID_ARG;
  KvCacheView c;
  KvSeqsView s;
  AttnPlan p;
  msq_status st = kv_views(cache, seqs, c, s);
  if (st == MSQ_OK) st = plan_attn(c, s, *attn, cache->head_dim, p);
  if (st != MSQ_OK) return st;
  *plan = msq_kv_plan{};
  if (p.blocks == 0) return MSQ_OK;
  plan->tile_rows = p.tile_rows;
  plan->wavefronts = p.waves ? p.waves : 4;
  plan->parts = p.nsplit;
  plan->join = p.nsplit == 1 ? 0 : p.tags_at ? 1 : 2;
  plan->workspace_bytes = p.workspace;
  return MSQ_OK;
}

extern "C" size_t msq_kv_attention_workspace_bytes(const msq_kv_cache* cache,
                                                   const msq_kv_seqs* seqs,
                                                   const msq_kv_attn* attn) {
  KvCacheView c;
  KvSeqsView s;
  AttnPlan p;
  if (!attn || kv_views(cache, seqs, c, s) != MSQ_OK) return 0;
  size_t most = 0;
  if (plan_attn(c, s, *attn, cache->head_dim, p, &most) != MSQ_OK) return 0;
  return most;
}

extern "C" msq_status msq_kv_attention(const msq_kv_cache* cache, const msq_kv_seqs* seqs,
                                       const msq_kv_attn* attn, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
  if (!attn) return MSQ_ERR_INVALID_ARG;
  AttnArgs a{};
  msq_status st = kv_views(cache, seqs, a.c, a.s);
  if (st != MSQ_OK) return st;
  const msq_kv_attn& t = *attn;
  const int D = cache->head_dim;
  if ((t.q_dtype != MSQ_DTYPE_BF16 && t.q_dtype != MSQ_DTYPE_F32) ||
      (t.out_dtype != MSQ_DTYPE_BF16 && t.out_dtype != MSQ_DTYPE_F32) ||
      !(t.scale >= 0.f) || !std::isfinite(t.scale))
    return MSQ_ERR_INVALID_ARG;
  AttnPlan p;
  st = plan_attn(a.c, a.s, t, D, p);
  if (st != MSQ_OK || p.blocks == 0) return st;
  st = kv_pointers(cache, seqs);
  if (st != MSQ_OK) return st;
  const int64_t per16 = t.q_dtype == MSQ_DTYPE_F32 ? 4 : 8;
  if (!t.q || !t.kv_len || !t.out || !aligned_to(t.q, 16) || !aligned_to(t.out, 16) ||
      !aligned_to(t.kv_len, 4) || !aligned_to(t.lse, 4) || t.q_token_stride % per16 ||
      t.q_head_stride % per16)
    return MSQ_ERR_INVALID_ARG;
  if (p.workspace > 0) {
    if (workspace_bytes < p.workspace) return MSQ_ERR_BUFFER_TOO_SMALL;
    if (!workspace || !aligned_to(workspace, 256)) return MSQ_ERR_INVALID_ARG;
    a.part_o = reinterpret_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(workspace) + p.ml_at);
    if (p.tags_at) {
      a.tags = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(workspace) + p.tags_at);
      a.call = next_call();
    }
  }
  a.q = t.q;
  a.qts = t.q_token_stride;
  a.qhs = t.q_head_stride;
  a.kv_len = t.kv_len;
  a.out = t.out;
  a.lse = t.lse;
  a.Hq = t.q_heads;
  a.G = t.q_heads / a.c.H;
  a.q_f32 = t.q_dtype == MSQ_DTYPE_F32;
  a.out_f32 = t.out_dtype == MSQ_DTYPE_F32;
  a.causal = t.causal != 0;
  a.window = t.window;
  a.nsplit = p.nsplit;
  a.span_tiles = p.span_tiles;
  a.row_tiles = p.row_tiles;
  a.tile_rows = p.tile_rows;
  a.tile_shift = p.tile_tokens == 64 ? 6 : 5;
  a.c2 = (t.scale > 0.f ? t.scale : 1.f / std::sqrt((float)D)) * kLog2e;
  const bool fine = a.q_f32 && a.out_f32;
  hipError_t e;
  switch (D) {
    case 64: e = fine ? launch_attn<64, true>(a, p, stream) : launch_attn<64, false>(a, p, stream); break;
    case 128: e = fine ? launch_attn<128, true>(a, p, stream) : launch_attn<128, false>(a, p, stream); break;
    default: e = fine ? launch_attn<256, true>(a, p, stream) : launch_attn<256, false>(a, p, stream); break;
  }
  return e == hipSuccess ? MSQ_OK : MSQ_ERR_HIP;
}
