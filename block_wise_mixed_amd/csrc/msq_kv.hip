// 8-bit key/value cache: quantising new tokens into it (msq_kv_write) and
// reading positions back (msq_kv_read).  The quantiser and the code order are
// stated in msq.h.
//
// Both kernels give one workgroup to (sequence, block its rows reach, keys or
// values, head): it owns everything the call changes in that block and head,
// so a scale that grows and the earlier codes it moves need no second launch
// and no atomics.  A wavefront takes 32 slots.  Keys: a lane holds 16 dims of
// a token, which are 16 contiguous code bytes.  Values: a lane holds 8 tokens
// x (4 + 4) dims, which are 64 contiguous code bytes (the value order puts 8
// tokens of a dim together, so the transposition happens in registers).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "msq.h"
#include "msq_kv.h"

namespace msq {
namespace {

constexpr float kFinite = 3.402823466e38f;

__device__ inline float bf16_f32(uint32_t bits) { return __uint_as_float(bits << 16); }

// Four consecutive values as loaded: 8 bytes of bf16, 16 of fp32.
template <typename T>
struct Raw4;
template <>
struct Raw4<uint16_t> {
  uint2 v;
  __device__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return i & 1 ? __uint_as_float(w & 0xFFFF0000u) : bf16_f32(w & 0xFFFFu);
  }
};
template <>
struct Raw4<float> {
  float4 v;
  __device__ float get(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};

template <typename T>
__device__ inline Raw4<T> load4(const T* p) {
  Raw4<T> r;
  r.v = *reinterpret_cast<const decltype(r.v)*>(p);
  return r;
}

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

__device__ inline float wave_max(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// What one workgroup of either kernel works on.
struct Task {
  int b, j, h, values;
};
__device__ inline Task task_of(int64_t id, int H, int reach) {
  Task t;
  t.h = (int)(id % H);
  id /= H;
  t.values = (int)(id & 1);
  id >>= 1;
  t.j = (int)(id % reach);
  t.b = (int)(id / reach);
  return t;
}

// Value-order pieces of a wavefront's 32 slots x D dims: lane -> token group
// g, first dim; kUnits of them per lane (the upper half of the lanes has none
// at D = 64).
template <int D>
struct ValueMap {
  static constexpr int kPerG = D / 8;               // (dim chunk, quad) pairs: D/32 * 4
  static constexpr int kLanes = kPerG < 16 ? kPerG : 16;
  static constexpr int kUnits = kPerG / kLanes;
  __device__ static bool active(int lane) { return lane < 4 * kLanes; }
  __device__ static int g(int lane) { return lane / kLanes; }
  // index of unit u: 4 * chunk + quad
  __device__ static int cq(int lane, int u) { return lane % kLanes + kLanes * u; }
};
__device__ inline int value_slot(int g, int j) { return j < 4 ? 4 * g + j : 12 + 4 * g + j; }

struct WriteArgs {
  KvCacheView c;
  KvSeqsView s;
  const int32_t* first;
  const void *k, *v;
  int64_t kts, khs, vts, vhs;
  int reach;
};

// Workgroup of block_tokens / 32 wavefronts.  HBM bound on long runs (each
// value is read once and kept in registers between the maximum and the
// coding); a call of single tokens is a chain of four dependent loads.
template <int D, typename T>
__global__ __launch_bounds__(512) void k_kv_write(WriteArgs a) {
  __shared__ float part[8];
  const Task tk = task_of(blockIdx.x, a.c.H, a.reach);
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
  uint8_t* codes = (tk.values ? a.c.vc : a.c.kc) + hb * P * D;
  const T* src = reinterpret_cast<const T*>(tk.values ? a.v : a.k) +
                 tk.h * (tk.values ? a.vhs : a.khs);
  const int64_t ts = tk.values ? a.vts : a.kts;
  const float old = lo > 0 ? *scale : 0.f;

  const int s0 = 32 * wave;
  constexpr int kKeyUnits = 2 * (D / 64);
  using VM = ValueMap<D>;
  constexpr int kRaw = kKeyUnits * 4 > VM::kUnits * 16 ? kKeyUnits * 4 : VM::kUnits * 16;
  Raw4<T> raw[kRaw];
  float amax = 0.f;
  if (!tk.values) {
#pragma unroll
    for (int u = 0; u < kKeyUnits; ++u) {
      const int slot = s0 + 16 * (u & 1) + (lane & 15);
      if (slot >= lo && slot < hi) {
        const T* p = src + (row + slot) * ts + 64 * (u >> 1) + 16 * (lane >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[4 * u + i] = load4(p + 4 * i);
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(raw[4 * u + i / 4].get(i & 3)));
      }
    }
  } else if (VM::active(lane)) {
#pragma unroll
    for (int u = 0; u < VM::kUnits; ++u) {
      const int cq = VM::cq(lane, u), d = 32 * (cq >> 2) + 4 * (cq & 3);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int slot = s0 + value_slot(VM::g(lane), j);
        if (slot >= lo && slot < hi) {
          const T* p = src + (row + slot) * ts + d;
          raw[16 * u + 2 * j] = load4(p);
          raw[16 * u + 2 * j + 1] = load4(p + 16);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            amax = fmaxf(amax, finite_abs(raw[16 * u + 2 * j + i / 4].get(i & 3)));
        }
      }
    }
  }
  amax = wave_max(amax);
  if (waves > 1) {
    if (lane == 0) part[wave] = amax;
    __syncthreads();
    for (int w = 0; w < waves; ++w) amax = fmaxf(amax, part[w]);
  }
  float s = amax / 127.0f;
  const bool grown = lo > 0 && s > old;
  if (lo > 0 && !grown) s = old;
  if (threadIdx.x == 0 && (lo == 0 || grown)) *scale = s;

  if (!tk.values) {
#pragma unroll
    for (int u = 0; u < kKeyUnits; ++u) {
      const int slot = s0 + 16 * (u & 1) + (lane & 15);
      uint4* at = reinterpret_cast<uint4*>(codes + 16 * D * (slot >> 4) + 1024 * (u >> 1)) + lane;
      if (slot >= lo && slot < hi) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = 0;
#pragma unroll
          for (int n = 0; n < 4; ++n) w[i] |= kv_code(raw[4 * u + i].get(n), s) << (8 * n);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (grown && slot < lo) {
        const uint4 q = *at;
        uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t r = 0;
#pragma unroll
          for (int n = 0; n < 4; ++n) r |= kv_recode((w[i] >> (8 * n)) & 255u, old, s) << (8 * n);
          w[i] = r;
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  } else if (VM::active(lane)) {
    const int g = VM::g(lane);
    bool any = false, all = true;  // of this lane's 8 slots: some change, all are new
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int slot = s0 + value_slot(g, j);
      const bool isnew = slot >= lo && slot < hi;
      any |= isnew || (grown && slot < lo);
      all &= isnew;
    }
    if (!any) return;
#pragma unroll
    for (int u = 0; u < VM::kUnits; ++u) {
      const int cq = VM::cq(lane, u);
      uint4* at = reinterpret_cast<uint4*>(codes + 32 * D * wave + 1024 * (cq >> 2)) +
                  4 * (cq & 3) + 16 * g;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (!all) q = at[d];
        uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // word i: dims d + 16 * (i / 2), slots 4 * (i % 2) ..
          uint32_t r = 0;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const int j = 4 * (i & 1) + n;
            const int slot = s0 + value_slot(g, j);
            uint32_t code = (w[i] >> (8 * n)) & 255u;
            if (slot >= lo && slot < hi)
              code = kv_code(raw[16 * u + 2 * j + (i >> 1)].get(d), s);
            else if (grown && slot < lo)
              code = kv_recode(code, old, s);
            r |= code << (8 * n);
          }
          w[i] = r;
        }
        at[d] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

struct ReadArgs {
  KvCacheView c;
  KvSeqsView s;
  const int32_t* first;
  void *k, *v;
  int reach;
};

__device__ inline void store4(uint16_t* p, const float* x) {
  union {
    __bf16 b[4];
    uint2 u;
  } o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.b[i] = (__bf16)x[i];
  *reinterpret_cast<uint2*>(p) = o.u;
}
__device__ inline void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

__device__ inline float kv_value(uint32_t w, int n, float s) {
  return (float)((int)((w >> (8 * n)) & 255u) - 128) * s;
}

// HBM bound: codes in, values out, once each.
template <int D, typename T>
__global__ __launch_bounds__(512) void k_kv_read(ReadArgs a) {
  const Task tk = task_of(blockIdx.x, a.c.H, a.reach);
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
  const int64_t row = (int64_t)row0 + base - f;
  const int64_t hb = (int64_t)max(id, 0) * a.c.H + tk.h;
  const float s = id < 0 ? 0.f : (tk.values ? a.c.vs : a.c.ks)[hb];
  const uint8_t* codes = (tk.values ? a.c.vc : a.c.kc) + hb * P * D;
  T* dst = reinterpret_cast<T*>(tk.values ? a.v : a.k) + (int64_t)tk.h * D;
  const int64_t ts = (int64_t)a.c.H * D;
  const int s0 = 32 * wave;
  using VM = ValueMap<D>;
  if (!tk.values) {
#pragma unroll
    for (int u = 0; u < 2 * (D / 64); ++u) {
      const int slot = s0 + 16 * (u & 1) + (lane & 15);
      if (slot < lo || slot >= hi) continue;
      const uint4 q =
          *(reinterpret_cast<const uint4*>(codes + 16 * D * (slot >> 4) + 1024 * (u >> 1)) + lane);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      T* p = dst + (row + slot) * ts + 64 * (u >> 1) + 16 * (lane >> 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) x[n] = id < 0 ? 0.f : kv_value(w[i], n, s);
        store4(p + 4 * i, x);
      }
    }
  } else if (VM::active(lane)) {
    const int g = VM::g(lane);
#pragma unroll
    for (int u = 0; u < VM::kUnits; ++u) {
      const int cq = VM::cq(lane, u);
      const uint4* at =
          reinterpret_cast<const uint4*>(codes + 32 * D * wave + 1024 * (cq >> 2)) +
          4 * (cq & 3) + 16 * g;
      uint32_t w[4][4];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint4 q = at[d];
        w[d][0] = q.x, w[d][1] = q.y, w[d][2] = q.z, w[d][3] = q.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int slot = s0 + value_slot(g, j);
        if (slot < lo || slot >= hi) continue;
        T* p = dst + (row + slot) * ts + 32 * (cq >> 2) + 4 * (cq & 3);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[4];
#pragma unroll
          for (int d = 0; d < 4; ++d)
            x[d] = id < 0 ? 0.f : kv_value(w[d][2 * half + (j >> 2)], j & 3, s);
          store4(p + 16 * half, x);
        }
      }
    }
  }
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Blocks a run of max_count positions can touch.
int64_t reach_of(const KvSeqsView& s, int shift) {
  const int64_t n = s.offset ? s.max_count : s.per_seq, P = (int64_t)1 << shift;
  return (n + P - 2) / P + 1;
}

template <template <int, typename> class Launch, typename Args>
hipError_t dispatch(int D, int dtype, dim3 grid, dim3 block, hipStream_t stream, const Args& a) {
  const bool f32 = dtype == MSQ_DTYPE_F32;
  switch (D) {
    case 64: f32 ? Launch<64, float>::go(grid, block, stream, a) : Launch<64, uint16_t>::go(grid, block, stream, a); break;
    case 128: f32 ? Launch<128, float>::go(grid, block, stream, a) : Launch<128, uint16_t>::go(grid, block, stream, a); break;
    default: f32 ? Launch<256, float>::go(grid, block, stream, a) : Launch<256, uint16_t>::go(grid, block, stream, a); break;
  }
  return hipGetLastError();
}
template <int D, typename T>
struct LaunchWrite {
  static void go(dim3 grid, dim3 block, hipStream_t stream, const WriteArgs& a) {
    hipLaunchKernelGGL((k_kv_write<D, T>), grid, block, 0, stream, a);
  }
};
template <int D, typename T>
struct LaunchRead {
  static void go(dim3 grid, dim3 block, hipStream_t stream, const ReadArgs& a) {
    hipLaunchKernelGGL((k_kv_read<D, T>), grid, block, 0, stream, a);
  }
};

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
      (int64_t)seqs->table_width * cache->block_tokens > most || seqs->max_count < 0)
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

// Checks that write and read share; *blocks: the launch's workgroups.
msq_status kv_common(const msq_kv_cache* cache, const msq_kv_seqs* seqs, const int32_t* first,
                     const void* k, const void* v, int32_t dtype, KvCacheView& c, KvSeqsView& s,
                     int64_t* reach, int64_t* blocks) {
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
  const int64_t lists = (int64_t)s.batch * *reach;  // < 2^31 * 2^27
  if (lists > (int64_t)0x7FFFFFFF / 2 / c.H) return MSQ_ERR_SHAPE;
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
  const msq_status st = kv_common(cache, seqs, first, k, v, dtype, a.c, a.s, &reach, &blocks);
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
  const hipError_t e = dispatch<LaunchWrite>(cache->head_dim, dtype, dim3((unsigned)blocks),
                                             dim3(2u << a.c.shift), stream, a);
  return e == hipSuccess ? MSQ_OK : MSQ_ERR_HIP;
}

extern "C" msq_status msq_kv_read(const msq_kv_cache* cache, const msq_kv_seqs* seqs,
                                  const int32_t* first, void* k, void* v, int32_t dtype,
                                  hipStream_t stream) {
  ReadArgs a{};
  int64_t reach = 0, blocks = 0;
  const msq_status st = kv_common(cache, seqs, first, k, v, dtype, a.c, a.s, &reach, &blocks);
  if (st != MSQ_OK || blocks == 0) return st;
  a.first = first;
  a.k = k;
  a.v = v;
  a.reach = (int)reach;
  const hipError_t e = dispatch<LaunchRead>(cache->head_dim, dtype, dim3((unsigned)blocks),
                                            dim3(2u << a.c.shift), stream, a);
  return e == hipSuccess ? MSQ_OK : MSQ_ERR_HIP;
}
