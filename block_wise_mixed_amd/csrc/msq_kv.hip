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
#include "msq_kv_block.h"

namespace msq {
namespace {

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
  const int64_t f = a.first[tk.b];
  int row0, count;
  kv_rows(a.s, tk.b, row0, count);
  Span sp;
  if (!span_of(a.c, a.s, tk.b, tk.j, f, row0, count, sp)) return;
  const T* src = reinterpret_cast<const T*>(tk.values ? a.v : a.k) +
                 tk.h * (tk.values ? a.vhs : a.khs);
  const int64_t ts = tk.values ? a.vts : a.kts;
  const int lane = threadIdx.x & 63;
  write_block<D, E, Raw8<T>>(
      a.c, tk.values, (int64_t)sp.id * a.c.H + tk.h, sp.lo, sp.hi, part_max, lane, [&](Raw8<T>(&raw)[Mp::kRows]) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int s0 = 32 * (wave / (D / E)), part = wave % (D / E) * (E / 8) + Mp::part(lane);
#pragma unroll
        for (int u = 0; u < Mp::kRows; ++u) {
          const int slot = s0 + Mp::row(lane, u);
          if (slot >= sp.lo && slot < sp.hi) raw[u].load(src + (sp.row + slot) * ts + 8 * part);
        }
      });
}

struct ReadArgs {
  KvCacheView c;
  KvSeqsView s;
  const int32_t* first;
  void *k, *v;
  int reach;
  unsigned begin;
};

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
