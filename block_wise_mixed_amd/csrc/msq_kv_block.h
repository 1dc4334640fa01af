// What the kernels that write and read a block of the 8-bit key/value cache share
// (msq_kv.hip, msq_kv_append.hip): the quantiser, a wavefront's pieces of a block,
// the checks and launches of their calls.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "msq.h"
#include "msq_kv.h"

namespace msq {
namespace {

constexpr float kFinite = 3.402823466e38f;

// Eight consecutive values as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint4 v;
  __device__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  // the larger of m and the magnitudes, as bit patterns: two in the halves of a word
  __device__ uint32_t most(uint32_t m) const {
    typedef uint16_t pair __attribute__((ext_vector_type(2)));
    pair r = __builtin_bit_cast(pair, m);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r = __builtin_elementwise_max(r, __builtin_bit_cast(pair, w[i] & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, r);
  }
  __device__ static float widen(uint32_t m) { return __uint_as_float(max(m << 16, m & 0xFFFF0000u)); }
  __device__ void get(float* x) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ uint32_t most(uint32_t m) const {
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ static float widen(uint32_t m) { return __uint_as_float(m); }
  __device__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

__device__ inline float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= kFinite ? a : 0.f;  // NaN and infinities do not set the scale
}

// code + 128 of x at scale s (correctly rounded division, ties to even).
__device__ inline uint32_t kv_code(float x, float s) {
  float t = rintf(x / s);
  t = fminf(fmaxf(t, -127.f), 127.f);
  if (!(s > 0.f) || x != x) t = 0.f;
  return (uint32_t)((int)t + 128);
}

// An earlier code (+128) at a scale that grew from `old` to s.
__device__ inline uint32_t kv_recode(uint32_t u, float old, float s) {
  const float v = (float)((int)u - 128) * old;
  return kv_code(v, s);
}

// Codes of eight values.  inv > 0: a reciprocal of s (v_rcp_f32, 1 ulp) that
// may stand in for the division: t = x * inv and fl(x / s) are within 127 *
// (1.5 * 2^-23 + 2^-24) < 2^-15 of each other, so they round to the same code
// unless t is within 2^-14 of a half-integer; then the lane divides.  (inv is 0
// where s is out of range or the lane has a NaN.)  The rounding is an addition
// of 1.5 * 2^23, which leaves code + 128 in the low byte.
__device__ inline uint2 kv_codes8(const float* x, float s, float inv) {
  constexpr float kMagic = 12582912.f + 128.f;
  uint32_t m[8], w[2];
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __builtin_amdgcn_fmed3f(x[i] * inv, -127.f, 127.f);
    const float r = t + kMagic;
    off = fmaxf(off, fabsf(t - (r - kMagic)));
    m[i] = __float_as_uint(r);
  }
  if (!(inv > 0.f) || off > 0.5f - 0x1p-14f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = kv_code(x[i], s);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(m[4 * i + 1], m[4 * i], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(m[4 * i + 3], m[4 * i + 2], 0x04000C0Cu);
    w[i] = lo | hi;
  }
  return make_uint2(w[0], w[1]);
}

__device__ inline uint32_t kv_recode4(uint32_t w, float old, float s) {
  uint32_t r = 0;
#pragma unroll
  for (int n = 0; n < 4; ++n) r |= kv_recode((w >> (8 * n)) & 255u, old, s) << (8 * n);
  return r;
}

// 4 x 4 bytes: byte j of out[i] is byte i of in[j].
__device__ inline void transpose4(const uint32_t* in, uint32_t* out) {
  const uint32_t ab0 = __builtin_amdgcn_perm(in[1], in[0], 0x05010400u);
  const uint32_t ab1 = __builtin_amdgcn_perm(in[1], in[0], 0x07030602u);
  const uint32_t cd0 = __builtin_amdgcn_perm(in[3], in[2], 0x05010400u);
  const uint32_t cd1 = __builtin_amdgcn_perm(in[3], in[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302u);
}

__device__ inline float wave_max(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// What one workgroup of either kernel works on.
struct Task {
  int b, j, h, values;
};
__device__ inline Task task_of(unsigned id, unsigned H, unsigned reach) {
  Task t;
  const unsigned list = id / H, seq = list / 2 / reach;
  t.h = (int)(id - list * H);
  t.values = (int)(list & 1);
  t.j = (int)(list / 2 - seq * reach);
  t.b = (int)seq;
  return t;
}

// Pieces of a wavefront's 32 slots x D dims.
template <int D>
struct Map {
  // rows: a lane holds dims 8 * part .. of slots row(lane, u), u < kRows
  static constexpr int kParts = D / 8, kRows = D / 16;
  __device__ static int part(int lane) { return lane % kParts; }
  __device__ static int row(int lane, int u) { return lane / kParts + 64 / kParts * u; }
  // byte of that piece in the keys' order, from the first of the 32 slots
  __device__ static int key_byte(int slot, int part) {
    return 16 * D * (slot >> 4) + 1024 * (part >> 3) +
           16 * ((slot & 15) + 16 * ((part >> 1) & 3)) + 8 * (part & 1);
  }
  // values' order: a lane holds 8 tokens (group g) x dims 4 q .. and 16 + 4 q
  // .. of chunk c, cq = 4 c + q; kUnits of them (half the lanes idle at D = 64)
  static constexpr int kLanes = D / 8 < 16 ? D / 8 : 16, kUnits = D / 8 / kLanes;
  __device__ static bool active(int lane) { return lane < 4 * kLanes; }
  __device__ static int g(int lane) { return lane / kLanes; }
  __device__ static int cq(int lane, int u) { return lane % kLanes + kLanes * u; }
  // LDS image of the codes, [slot][dim]
  static constexpr int kStride = D + 8, kImage = 32 * kStride;
};
__device__ inline int value_slot(int g, int j) { return j < 4 ? 4 * g + j : 12 + 4 * g + j; }

extern __shared__ __align__(16) unsigned char smem_codes[];

// The slots lo .. hi - 1 that a call writes of one block and head: fill(raw) gives a
// lane its kRows pieces of the new tokens (slots in that range only), which are
// coded here, with the block's scale.  values: of the values, else of the keys.
// part_max: of the workgroup, one for each wavefront; lane: threadIdx.x & 63.
template <int D, int E, typename Held, typename Fill>
__device__ __forceinline__ void write_block(const KvCacheView& c, bool values, int64_t hb, int lo, int hi,
                                            float* part_max, int lane, Fill&& fill) {
  using Mp = Map<E>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int P = 1 << c.shift;
  float* scale = (values ? c.vs : c.ks) + hb;
  const int s0 = 32 * (wave / (D / E)), first_part = wave % (D / E) * (E / 8);
  uint8_t* codes = (values ? c.vc : c.kc) + (hb * P + s0) * D;
  const float old = lo > 0 ? *scale : 0.f;

  const int here = Mp::part(lane), part = first_part + here;
  Held raw[Mp::kRows];
  fill(raw);
  uint32_t most = 0;
#pragma unroll
  for (int u = 0; u < Mp::kRows; ++u) {
    const int slot = s0 + Mp::row(lane, u);
    if (slot >= lo && slot < hi) most = raw[u].most(most);
  }
  float amax = Held::widen(most);
  const bool finite = amax <= kFinite;  // all of this lane's values
  if (!finite) {
    amax = 0.f;
#pragma unroll
    for (int u = 0; u < Mp::kRows; ++u) {
      const int slot = s0 + Mp::row(lane, u);
      if (slot >= lo && slot < hi) {
        float x[8];
        raw[u].get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite_abs(x[i]));
      }
    }
  }
  amax = wave_max(amax);
  if (waves > 1) {
    if (lane == 0) part_max[wave] = amax;
    __syncthreads();
    for (int w = 0; w < waves; ++w) amax = fmaxf(amax, part_max[w]);
  }
  float s = amax / 127.0f;
  const bool grown = lo > 0 && s > old;
  if (lo > 0 && !grown) s = old;
  if (threadIdx.x == 0 && (lo == 0 || grown)) *scale = s;
  const float inv = finite && s > 1e-30f && s < 1e30f ? __builtin_amdgcn_rcpf(s) : 0.f;

  uint8_t* image = smem_codes + wave * Mp::kImage;
#pragma unroll
  for (int u = 0; u < Mp::kRows; ++u) {
    const int in = Mp::row(lane, u), slot = s0 + in;
    uint2* at = reinterpret_cast<uint2*>(codes + Map<D>::key_byte(in, part));
    if (slot >= lo && slot < hi) {
      float x[8];
      raw[u].get(x);
      const uint2 q = kv_codes8(x, s, inv);
      if (values)
        *reinterpret_cast<uint2*>(image + in * Mp::kStride + 8 * here) = q;
      else
        *at = q;
    } else if (grown && slot < lo && !values) {
      const uint2 q = *at;
      *at = make_uint2(kv_recode4(q.x, old, s), kv_recode4(q.y, old, s));
    }
  }
  if (!values || !Mp::active(lane)) return;
  __builtin_amdgcn_wave_barrier();  // the image is this wavefront's own

  const int g = Mp::g(lane);
  uint32_t fresh[2] = {0, 0}, keep[2] = {0, 0};  // bytes of new and of moved earlier codes
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int slot = s0 + value_slot(g, j);
    if (slot >= lo && slot < hi) fresh[j >> 2] |= 255u << (8 * (j & 3));
    if (grown && slot < lo) keep[j >> 2] |= 255u << (8 * (j & 3));
  }
  if (!(fresh[0] | fresh[1] | keep[0] | keep[1])) return;
  const bool all = (fresh[0] & fresh[1]) == 0xFFFFFFFFu;
#pragma unroll
  for (int u = 0; u < Mp::kUnits; ++u) {
    const int cq = Mp::cq(lane, u);
    const uint8_t* from = image + 32 * (cq >> 2) + 4 * (cq & 3);
    uint32_t w[4][4];  // [dim][word]: word i holds dims d + 16 (i / 2), tokens 4 (i % 2) ..
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t in[4], out[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
        in[n] = *reinterpret_cast<const uint32_t*>(
            from + value_slot(g, 4 * (i & 1) + n) * Mp::kStride + 16 * (i >> 1));
      transpose4(in, out);
#pragma unroll
      for (int d = 0; d < 4; ++d) w[d][i] = out[d];
    }
    uint4* at = reinterpret_cast<uint4*>(codes + 1024 * ((first_part + cq) >> 2)) + 4 * (cq & 3) + 16 * g;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (!all) {
        const uint4 q = at[d];
        const uint32_t was[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t r = (w[d][i] & fresh[i & 1]) | (was[i] & ~fresh[i & 1]);
          if (keep[i & 1]) r = (r & ~keep[i & 1]) | (kv_recode4(was[i], old, s) & keep[i & 1]);
          w[d][i] = r;
        }
      }
      at[d] = make_uint4(w[d][0], w[d][1], w[d][2], w[d][3]);
    }
  }
}

// What a call writes into the block of table entry first / P + j of a sequence with
// count rows from row0 on: slots lo .. hi - 1 of block id; row: that of slot 0.
struct Span {
  int id, lo, hi;
  int64_t base, row;
};
__device__ inline bool span_of(const KvCacheView& c, const KvSeqsView& s, int b, int j, int64_t f, int row0,
                               int count, Span& sp) {
  if (f < 0 || count <= 0) return false;
  const int64_t e = (f >> c.shift) + j;
  sp.base = e << c.shift;
  if (sp.base >= f + count) return false;
  sp.id = kv_block(c, s, b, e);
  if (sp.id < 0) return false;
  sp.lo = (int)max(f - sp.base, (int64_t)0);
  sp.hi = (int)min(f + count - sp.base, (int64_t)(1 << c.shift));
  sp.row = (int64_t)row0 + sp.base - f;
  return true;
}

__device__ inline void store8(uint16_t* p, const float* x) {
  union {
    __bf16 b[8];
    uint4 u;
  } o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.b[i] = (__bf16)x[i];
  *reinterpret_cast<uint4*>(p) = o.u;
}
__device__ inline void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Blocks a run of max_count positions can touch.
inline int64_t reach_of(const KvSeqsView& s, int shift) {
  const int64_t n = s.offset ? s.max_count : s.per_seq, P = (int64_t)1 << shift;
  return (n + P - 2) / P + 1;
}

// One launch, or as many as it takes at fewer than 2^32 threads each.
template <typename Args, typename Go>
msq_status launch_all(Args& a, unsigned blocks, int threads, Go&& go) {
  const unsigned most = (unsigned)(kMostThreads / threads);
  for (unsigned done = 0; done < blocks; done += most) {
    a.begin = done;
    go(dim3(std::min(blocks - done, most)), dim3(threads));
    if (hipGetLastError() != hipSuccess) return MSQ_ERR_HIP;
    if (blocks - done <= most) break;
  }
  return MSQ_OK;
}

// Checks that write and read share; *reach: the most blocks of a sequence that the call works
// on (table_only: those that the table has), *blocks: its workgroups.
inline msq_status kv_common(const msq_kv_cache* cache, const msq_kv_seqs* seqs, const int32_t* first,
                     const void* k, const void* v, int32_t dtype, bool table_only, KvCacheView& c,
                     KvSeqsView& s, int64_t* reach, int64_t* blocks) {
  msq_status st = kv_views(cache, seqs, c, s);
  if (st != MSQ_OK) return st;
  if (dtype != MSQ_DTYPE_BF16 && dtype != MSQ_DTYPE_F32) return MSQ_ERR_INVALID_ARG;
  *blocks = 0;
  if (s.batch == 0 || s.total == 0) return MSQ_OK;
  st = kv_pointers(cache, seqs);
  if (st != MSQ_OK) return st;
  if (!first || !k || !v || !aligned_to(first, 4) || !aligned_to(k, 16) || !aligned_to(v, 16))
    return MSQ_ERR_INVALID_ARG;
  *reach = reach_of(s, c.shift);
  if (table_only) *reach = std::min<int64_t>(*reach, s.width);
  const int64_t lists = (int64_t)s.batch * *reach;  // < 2^31 * 2^27
  if (lists > 0x7FFFFFFF / 2 / c.H) return MSQ_ERR_SHAPE;
  *blocks = lists * 2 * c.H;
  return MSQ_OK;
}

}  // namespace
}  // namespace msq
