// 8-bit key/value cache: quantising new tokens into it (msq_kv_write) and
// reading positions back (msq_kv_read).  The quantiser and the code order are
// stated in msq.h.
//
// Both kernels give one workgroup to (sequence, block its rows reach, keys or
// values, head): it owns everything the call changes in that block and head,
// so a scale that grows and the earlier codes it moves need no second launch
// and no atomics.  A wavefront takes 32 slots.  On the tensors' side a lane
// holds 8 dims of a token (whole rows per instruction).  In the keys' order
// these are 8 contiguous code bytes; the values' order puts 8 tokens of a dim
// together, so values pass through LDS and 4 x 4 byte transpositions in
// registers: a lane there holds 8 tokens x (4 + 4) dims, 64 contiguous code
// bytes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

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

struct WriteArgs {
  KvCacheView c;
  KvSeqsView s;
  const int32_t* first;
  const void *k, *v;
  int64_t kts, khs, vts, vhs;
  int reach;
  unsigned begin;  // task of the launch's first workgroup
};

// A wavefront takes 32 slots x E dims (64 where the workgroup's 16 wavefronts
// allow it).  HBM bound on long runs (each value is read once and kept in
// registers between the maximum and the coding): 16 sequences of 4097 to 8192
// bf16 tokens, 8 heads of 128, 625 MB in 153 us, 4.1 TB/s, fp32 1.04 GB in 209 to 228, 4.6
// to 5.0.  A call of single tokens is a chain of four dependent loads, 4.8 us from
// launch to launch for one token.
template <int D, int E, typename T>
__global__ __launch_bounds__(1024) void k_kv_write(WriteArgs a) {
  using Mp = Map<E>;
  __shared__ float part_max[16];
  const Task tk = task_of(a.begin + blockIdx.x, a.c.H, a.reach);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int P = 1 << a.c.shift;
  const int64_t f = a.first[tk.b];
  int row0, count;
  kv_rows(a.s, tk.b, row0, count);
  if (f < 0 || count <= 0) return;
  const int64_t e = (f >> a.c.shift) + tk.j;
  const int64_t base = e << a.c.shift;
  if (base >= f + count) return;
  const int id = kv_block(a.c, a.s, tk.b, e);
  if (id < 0) return;
  const int lo = (int)max(f - base, (int64_t)0);
  const int hi = (int)min(f + count - base, (int64_t)P);
  const int64_t row = (int64_t)row0 + base - f;  // row of slot 0
  const int64_t hb = (int64_t)id * a.c.H + tk.h;
  float* scale = (tk.values ? a.c.vs : a.c.ks) + hb;
  const int s0 = 32 * (wave / (D / E)), first_part = wave % (D / E) * (E / 8);
  uint8_t* codes = (tk.values ? a.c.vc : a.c.kc) + (hb * P + s0) * D;
  const T* src = reinterpret_cast<const T*>(tk.values ? a.v : a.k) +
                 tk.h * (tk.values ? a.vhs : a.khs);
  const int64_t ts = tk.values ? a.vts : a.kts;
  const float old = lo > 0 ? *scale : 0.f;

  const int here = Mp::part(lane), part = first_part + here;
  Raw8<T> raw[Mp::kRows];
#pragma unroll
  for (int u = 0; u < Mp::kRows; ++u) {
    const int slot = s0 + Mp::row(lane, u);
    if (slot >= lo && slot < hi) raw[u].load(src + (row + slot) * ts + 8 * part);
  }
  uint32_t most = 0;
#pragma unroll
  for (int u = 0; u < Mp::kRows; ++u) {
    const int slot = s0 + Mp::row(lane, u);
    if (slot >= lo && slot < hi) most = raw[u].most(most);
  }
  float amax = Raw8<T>::widen(most);
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
      if (tk.values)
        *reinterpret_cast<uint2*>(image + in * Mp::kStride + 8 * here) = q;
      else
        *at = q;
    } else if (grown && slot < lo && !tk.values) {
      const uint2 q = *at;
      *at = make_uint2(kv_recode4(q.x, old, s), kv_recode4(q.y, old, s));
    }
  }
  if (!tk.values || !Mp::active(lane)) return;
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

struct ReadArgs {
  KvCacheView c;
  KvSeqsView s;
  const int32_t* first;
  void *k, *v;
  int reach;
  unsigned begin;
};

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

// HBM bound: codes in, values out, once each: 101700 tokens of 8 heads of 128 to
// bf16, 625 MB in 118 to 133 us, 4.7 to 5.3 TB/s; to fp32, 1.04 GB in 254 to 263, 4.0 to
// 4.1 (mostly writes).
template <int D, typename T>
__global__ __launch_bounds__(512) void k_kv_read(ReadArgs a) {
  using Mp = Map<D>;
  const Task tk = task_of(a.begin + blockIdx.x, a.c.H, a.reach);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int P = 1 << a.c.shift;
  const int64_t f = a.first[tk.b];
  int row0, count;
  kv_rows(a.s, tk.b, row0, count);
  if (count <= 0) return;
  const int64_t e = (f >> a.c.shift) + tk.j;  // arithmetic shift: floor, also below 0
  const int64_t base = e << a.c.shift;
  if (base >= f + count) return;
  const int id = kv_block(a.c, a.s, tk.b, e);
  const int lo = (int)max(f - base, (int64_t)0);
  const int hi = (int)min(f + count - base, (int64_t)P);
  const int s0 = 32 * wave;
  if (s0 >= hi || s0 + 32 <= lo) return;
  const int64_t row = (int64_t)row0 + base - f;
  const int64_t hb = (int64_t)max(id, 0) * a.c.H + tk.h;
  const float s = id < 0 ? 0.f : (tk.values ? a.c.vs : a.c.ks)[hb];
  const uint8_t* codes = (tk.values ? a.c.vc : a.c.kc) + (hb * P + s0) * D;
  T* dst = reinterpret_cast<T*>(tk.values ? a.v : a.k) + (int64_t)tk.h * D;
  const int64_t ts = (int64_t)a.c.H * D;
  const int part = Mp::part(lane);
  uint8_t* image = smem_codes + wave * Mp::kImage;
  uint2 q[Mp::kRows];
  if (!tk.values) {
#pragma unroll
    for (int u = 0; u < Mp::kRows; ++u)
      q[u] = *reinterpret_cast<const uint2*>(codes + Mp::key_byte(Mp::row(lane, u), part));
  } else {
    if (Mp::active(lane)) {
      const int g = Mp::g(lane);
#pragma unroll
      for (int u = 0; u < Mp::kUnits; ++u) {
        const int cq = Mp::cq(lane, u);
        const uint4* at = reinterpret_cast<const uint4*>(codes + 1024 * (cq >> 2)) + 4 * (cq & 3) + 16 * g;
        uint8_t* to = image + 32 * (cq >> 2) + 4 * (cq & 3);
        uint32_t w[4][4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const uint4 v = at[d];
          w[0][d] = v.x, w[1][d] = v.y, w[2][d] = v.z, w[3][d] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t out[4];
          transpose4(w[i], out);
#pragma unroll
          for (int n = 0; n < 4; ++n)
            *reinterpret_cast<uint32_t*>(to + value_slot(g, 4 * (i & 1) + n) * Mp::kStride +
                                         16 * (i >> 1)) = out[n];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();  // the image is this wavefront's own
#pragma unroll
    for (int u = 0; u < Mp::kRows; ++u)
      q[u] = *reinterpret_cast<const uint2*>(image + Mp::row(lane, u) * Mp::kStride + 8 * part);
  }
#pragma unroll
  for (int u = 0; u < Mp::kRows; ++u) {
    const int slot = s0 + Mp::row(lane, u);
    if (slot < lo || slot >= hi) continue;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = id < 0 ? 0.f : (float)((int)(((i < 4 ? q[u].x : q[u].y) >> (8 * (i & 3))) & 255u) - 128) * s;
    store8(dst + (row + slot) * ts + 8 * part, x);
  }
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Blocks a run of max_count positions can touch.
int64_t reach_of(const KvSeqsView& s, int shift) {
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

template <int D, typename T>
msq_status launch_write(unsigned blocks, WriteArgs& a, hipStream_t stream) {
  const int strips = 1 << (a.c.shift - 5);
  auto go = [&](auto dims) {
    constexpr int E = decltype(dims)::value;
    const int waves = strips * (D / E);
    return launch_all(a, blocks, 64 * waves, [&](dim3 grid, dim3 block) {
      hipLaunchKernelGGL((k_kv_write<D, E, T>), grid, block, waves * Map<E>::kImage, stream, a);
    });
  };
  // More wavefronts shorten the coding of a run (2011 tokens of 8 heads of 128:
  // 10.7 -> 7.9 us) and idle where a block gets a token or two (256 single
  // tokens: 10.9 -> 14.4 us).
  if (a.s.max_count >= 16 && strips * (D / 64) <= 16)
    return go(std::integral_constant<int, 64>{});
  return go(std::integral_constant<int, D < 128 ? 64 : 128>{});
}
template <int D, typename T>
msq_status launch_read(unsigned blocks, ReadArgs& a, hipStream_t stream) {
  const int waves = 1 << (a.c.shift - 5);
  return launch_all(a, blocks, 64 * waves, [&](dim3 grid, dim3 block) {
    hipLaunchKernelGGL((k_kv_read<D, T>), grid, block, waves * Map<D>::kImage, stream, a);
  });
}

}  // namespace

msq_status kv_views(const msq_kv_cache* cache, const msq_kv_seqs* seqs, KvCacheView& c,
                    KvSeqsView& s) {
  if (!cache || !seqs) return MSQ_ERR_INVALID_ARG;
  const int64_t most = 0x7FFFFFFF;
  if (cache->num_blocks < 1 || cache->num_blocks > most || cache->kv_heads < 1)
    return MSQ_ERR_SHAPE;
  if (cache->head_dim != 64 && cache->head_dim != 128 && cache->head_dim != 256)
    return MSQ_ERR_UNSUPPORTED;
  int shift = 5;
  while (shift < 8 && (1 << shift) != cache->block_tokens) ++shift;
  if ((1 << shift) != cache->block_tokens) return MSQ_ERR_UNSUPPORTED;
  if (seqs->batch < 0 || seqs->total < 0 || seqs->total > most || seqs->table_width < 1 ||
      (int64_t)seqs->table_width * cache->block_tokens > ((int64_t)1 << 30) ||
      seqs->max_count < 0)
    return MSQ_ERR_SHAPE;
  if (!seqs->offset && (seqs->batch == 0 ? seqs->total != 0 : seqs->total % seqs->batch != 0))
    return MSQ_ERR_SHAPE;
  c.kc = cache->k_codes;
  c.vc = cache->v_codes;
  c.ks = cache->k_scale;
  c.vs = cache->v_scale;
  c.nblocks = (int)cache->num_blocks;
  c.H = cache->kv_heads;
  c.shift = shift;
  s.table = seqs->block_table;
  s.offset = seqs->offset;
  s.batch = seqs->batch;
  s.width = seqs->table_width;
  s.total = (int)seqs->total;
  s.per_seq = seqs->batch > 0 ? (int)(seqs->total / seqs->batch) : 0;
  s.max_count = seqs->max_count > 0 ? (int)(seqs->max_count < seqs->total ? seqs->max_count
                                                                           : seqs->total)
                                    : (int)seqs->total;
  if (!seqs->offset) s.max_count = s.per_seq;
  return MSQ_OK;
}

msq_status kv_pointers(const msq_kv_cache* cache, const msq_kv_seqs* seqs) {
  if (!cache->k_codes || !cache->v_codes || !cache->k_scale || !cache->v_scale ||
      !seqs->block_table)
    return MSQ_ERR_INVALID_ARG;
  if (!aligned_to(cache->k_codes, 16) || !aligned_to(cache->v_codes, 16) ||
      !aligned_to(cache->k_scale, 4) || !aligned_to(cache->v_scale, 4) ||
      !aligned_to(seqs->block_table, 4) || !aligned_to(seqs->offset, 4))
    return MSQ_ERR_INVALID_ARG;
  return MSQ_OK;
}

namespace {

// Checks that write and read share; *reach: the most blocks of a sequence that the call works
// on (table_only: those that the table has), *blocks: its workgroups.
msq_status kv_common(const msq_kv_cache* cache, const msq_kv_seqs* seqs, const int32_t* first,
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

using namespace msq;

extern "C" msq_status msq_kv_write(const msq_kv_cache* cache, const msq_kv_seqs* seqs,
                                   const int32_t* first, const void* k, int64_t k_token_stride,
                                   int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                   int64_t v_head_stride, int32_t dtype, hipStream_t stream) {
  WriteArgs a{};
  int64_t reach = 0, blocks = 0;
  const msq_status st = kv_common(cache, seqs, first, k, v, dtype, true, a.c, a.s, &reach, &blocks);
  if (st != MSQ_OK || blocks == 0) return st;
  const int64_t per16 = dtype == MSQ_DTYPE_F32 ? 4 : 8;
  if (k_token_stride % per16 || k_head_stride % per16 || v_token_stride % per16 ||
      v_head_stride % per16)
    return MSQ_ERR_INVALID_ARG;
  a.first = first;
  a.k = k;
  a.v = v;
  a.kts = k_token_stride;
  a.khs = k_head_stride;
  a.vts = v_token_stride;
  a.vhs = v_head_stride;
  a.reach = (int)reach;
  const bool f32 = dtype == MSQ_DTYPE_F32;
  const unsigned n = (unsigned)blocks;
  switch (cache->head_dim) {
    case 64: return f32 ? launch_write<64, float>(n, a, stream) : launch_write<64, uint16_t>(n, a, stream);
    case 128: return f32 ? launch_write<128, float>(n, a, stream) : launch_write<128, uint16_t>(n, a, stream);
    default: return f32 ? launch_write<256, float>(n, a, stream) : launch_write<256, uint16_t>(n, a, stream);
  }
}

extern "C" msq_status msq_kv_read(const msq_kv_cache* cache, const msq_kv_seqs* seqs,
                                  const int32_t* first, void* k, void* v, int32_t dtype,
                                  hipStream_t stream) {
  ReadArgs a{};
  int64_t reach = 0, blocks = 0;
  const msq_status st = kv_common(cache, seqs, first, k, v, dtype, false, a.c, a.s, &reach, &blocks);
  if (st != MSQ_OK || blocks == 0) return st;
  a.first = first;
  a.k = k;
  a.v = v;
  a.reach = (int)reach;
  const bool f32 = dtype == MSQ_DTYPE_F32;
  const unsigned n = (unsigned)blocks;
  switch (cache->head_dim) {
    case 64: return f32 ? launch_read<64, float>(n, a, stream) : launch_read<64, uint16_t>(n, a, stream);
    case 128: return f32 ? launch_read<128, float>(n, a, stream) : launch_read<128, uint16_t>(n, a, stream);
    default: return f32 ? launch_read<256, float>(n, a, stream) : launch_read<256, uint16_t>(n, a, stream);
  }
}
