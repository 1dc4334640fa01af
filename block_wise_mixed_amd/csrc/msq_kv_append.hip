// Rotated keys, values and the rotation of queries in one launch (msq_kv_append).
//
// Three kinds of workgroups, in this order: keys of a (sequence, block, some heads),
// values of a (sequence, block, head), queries of some rows of a sequence.  The first
// two own what the call changes in their block and heads, as in msq_kv.hip, and the
// quantiser is the same.  The turns (cosine and sine of a position) of a block's new
// tokens are made in LDS, in fp64, and used for all heads of the workgroup; a lane
// reads the 8 dims it holds and the 8 that these are paired with (from L1: HBM sees
// every value once, 1.00 of what the call has to move by the counters).
//
// HBM bound on long runs: 16 sequences of 4097 to 8192 bf16 tokens, 32 query heads on 8 of
// 128, 2.28 GB in 455 to 473 us, 4.8 to 5.0 TB/s.  A step of 64 fp32 tokens with 64
// query heads: 7.0 us, a chain of loads (first, table, positions, frequencies) and the fp64
// turns behind it.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "msq.h"
#include "msq_kv.h"
#include "msq_kv_block.h"
#include "msq_rotary.h"

namespace msq {
namespace {

struct AppendArgs {
  KvCacheView c;
  KvSeqsView s;
  const int32_t* first;
  const void *k, *v;
  int64_t kts, khs, vts, vhs;
  const int32_t *source, *count, *positions;
  int kv_rows, reach;
  int heads, groups;  // of a workgroup of keys; workgroups that share a block's heads
  unsigned keys, values;  // workgroups of these kinds
  RotaryView r;
  RotaryRowsView q;
  int q_rows, q_heads;   // query rows and heads of a workgroup
  int q_chunks, q_parts;  // such workgroups of a sequence, and of their heads
  unsigned begin;
};

// The rows of sequence b that the call takes.
__device__ inline void rows_of(const AppendArgs& a, int b, int& row0, int& count) {
  kv_rows(a.s, b, row0, count);
  if (a.count) count = min(count, max(a.count[b], 0));
}
// Row of k and v that row `row` of the call takes.
__device__ inline int64_t source_of(const AppendArgs& a, int64_t row) {
  return a.source ? min(max(a.source[row], 0), a.kv_rows - 1) : row;
}

// The keys of one block, some heads one after another.  A lane reads its pieces and,
// where they are rotated in halves, the ones that these are paired with.  kTable: the
// turns of all new slots fit the LDS; else each lane makes its own (slower: blocks of
// 256 tokens with more than 128 rotated dims of heads of 256 only).
template <int D, int E, typename T, bool kTable>
__device__ __forceinline__ void append_keys(const AppendArgs& a, const Span& sp, int h0, int heads,
                                            float (&part_max)[2][16]) {
  using Mp = Map<E>;
  constexpr int kAtOnce = Mp::kRows * (int)sizeof(T) > 16 ? 8 / (int)sizeof(T) : Mp::kRows;  // rows read before the first is rotated
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int s0 = 32 * (wave / (D / E)), half = a.r.half;
  auto position = [&](int slot) { return a.positions ? a.positions[sp.row + slot] : (int)(sp.base + slot); };
  float2* const turns = reinterpret_cast<float2*>(smem_codes);  // [slot - lo][half]
  if constexpr (kTable) {
    const unsigned all = (unsigned)((sp.hi - sp.lo) * half);
    for (unsigned n = threadIdx.x; n < all; n += blockDim.x) {
      const int slot = (int)(n / (unsigned)half), pair = (int)(n - slot * (unsigned)half);
      turns[n] = turn_of(position(sp.lo + slot), a.r.freq[pair], a.r.amplitude);
    }
    __syncthreads();
  }
  for (int j = 0; j < heads; ++j) {
    const int h = h0 + j;
    const T* src = reinterpret_cast<const T*>(a.k) + h * a.khs;
    // (what follows from the lane is not to be kept from head to head: the registers do not hold it)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    // dims 8 part .. : rotated in halves (mate: the paired dims), with their neighbours, or not
    const int part = wave % (D / E) * (E / 8) + Mp::part(lane);
    const bool turned = 8 * part < 2 * half, split = turned && !a.r.interleaved;
    const bool high = split && 8 * part >= half;
    const int mate = high ? 8 * part - half : 8 * part + half;
    const int pair0 = split ? (high ? mate : 8 * part) : 4 * part;
    write_block<D, E, Raw8<float>>(
        a.c, false, (int64_t)sp.id * a.c.H + h, sp.lo, sp.hi, part_max[j & 1], lane, [&](Raw8<float>(&out)[Mp::kRows]) {
#pragma unroll
          for (int u0 = 0; u0 < Mp::kRows; u0 += kAtOnce) {
            Raw8<T> own[kAtOnce], other[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
              const int slot = s0 + Mp::row(lane, u0 + u);
              if (slot < sp.lo || slot >= sp.hi) continue;
              const T* p = src + source_of(a, sp.row + slot) * a.kts;
              own[u].load(p + 8 * part);
              if (split) other[u].load(p + mate);
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
              const int slot = s0 + Mp::row(lane, u0 + u);
              if (slot < sp.lo || slot >= sp.hi) continue;
              float x[8];
              own[u].get(x);
              if (turned) {
                float2 t[8];
                if constexpr (kTable) {
                  const float4* at = reinterpret_cast<const float4*>(turns + (slot - sp.lo) * half + pair0);
                  reinterpret_cast<float4*>(t)[0] = at[0];
                  reinterpret_cast<float4*>(t)[1] = at[1];
                  if (split) {
                    reinterpret_cast<float4*>(t)[2] = at[2];
                    reinterpret_cast<float4*>(t)[3] = at[3];
                  }
                } else {
                  const int at = position(slot);
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    if (i < 4 || split) t[i] = turn_of(at, a.r.freq[pair0 + i], a.r.amplitude);
                }
                if (split) {
                  float y[8];
                  other[u].get(y);
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    x[i] = high ? turned_high(x[i], y[i], t[i]) : turned_low(x[i], y[i], t[i]);
                } else {
#pragma unroll
                  for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], t[i]);
                }
              }
              out[u0 + u].a = make_float4(x[0], x[1], x[2], x[3]);
              out[u0 + u].b = make_float4(x[4], x[5], x[6], x[7]);
            }
          }
        });
  }
}

template <int D, int E, typename T, bool kTable>
__global__ __launch_bounds__(1024) void k_kv_append(AppendArgs a) {
  using Mp = Map<E>;
  __shared__ float part_max[2][16];
  unsigned id = a.begin + blockIdx.x;
  if (id >= a.keys + a.values) {  // queries
    id -= a.keys + a.values;
    const unsigned list = id / (unsigned)a.q_parts;
    const int h0 = (int)(id - list * a.q_parts) * a.q_heads;
    const int b = (int)(list / (unsigned)a.q_chunks), i0 = (int)(list - b * (unsigned)a.q_chunks) * a.q_rows;
    const int f = a.first[b];
    int row0, count;
    rows_of(a, b, row0, count);
    if (f < 0 || i0 >= count) return;
    rotate_rows(a.q, a.r, row0 + i0, min(a.q_rows, count - i0), h0, min(a.q_heads, a.q.heads - h0),
                reinterpret_cast<float2*>(smem_codes),
                [&](int i) { return a.positions ? a.positions[row0 + i0 + i] : f + i0 + i; });
    return;
  }
  const bool values = id >= a.keys;
  if (values) id -= a.keys;
  const unsigned sets = values ? a.c.H : a.groups, list = id / sets;
  const int set = (int)(id - list * sets), b = (int)(list / (unsigned)a.reach);
  const int64_t f = a.first[b];
  int row0, count;
  rows_of(a, b, row0, count);
  Span sp;
  if (!span_of(a.c, a.s, b, (int)(list - b * (unsigned)a.reach), f, row0, count, sp)) return;
  if (!values) {
    append_keys<D, E, T, kTable>(a, sp, set * a.heads, min(a.heads, a.c.H - set * a.heads), part_max);
    return;
  }
  const T* src = reinterpret_cast<const T*>(a.v) + set * a.vhs;
  const int lane = threadIdx.x & 63;
  write_block<D, E, Raw8<T>>(
      a.c, true, (int64_t)sp.id * a.c.H + set, sp.lo, sp.hi, part_max[0], lane, [&](Raw8<T>(&raw)[Mp::kRows]) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int s0 = 32 * (wave / (D / E)), part = wave % (D / E) * (E / 8) + Mp::part(lane);
#pragma unroll
        for (int u = 0; u < Mp::kRows; ++u) {
          const int slot = s0 + Mp::row(lane, u);
          if (slot >= sp.lo && slot < sp.hi) raw[u].load(src + source_of(a, sp.row + slot) * a.vts + 8 * part);
        }
      });
}

// Most LDS for a table of turns (a compute unit has 160 KB).  A table of that size, of blocks of
// 256 tokens, leaves one workgroup a compute unit and is still ahead of turns made by each lane
// (16 sequences of 3000 tokens, 4 heads of 256, a head a workgroup: 117 and 154 us).
constexpr size_t kMostTable = 128 << 10;

template <int D, typename T>
msq_status launch_append(AppendArgs& a, int64_t lists, bool queries, hipStream_t stream) {
  const int strips = 1 << (a.c.shift - 5), P = 1 << a.c.shift;
  const bool wide = a.s.max_count >= 16 && strips * (D / 64) <= 16;
  const int waves = strips * (D / (wide || D == 64 ? 64 : 128)), threads = 64 * waves;
  const size_t table = (size_t)std::min(P, a.s.max_count) * a.r.half * sizeof(float2);
  const bool fits = table <= kMostTable;
  // Heads of a workgroup of keys: more share the turns, fewer fill the GPU; as many as leave
  // 12 wavefronts a compute unit.  Keys and values of 8 heads of 128 in blocks of 64, 1, 2, 4 and 8
  // heads a workgroup: 16 sequences of 6000 tokens 243, 189, 165, 153 us; one of 2000 11, 14, 20, 32;
  // 64 of 64 15.0, 15.5, 21.5, 33; 4 heads of 256 in blocks of 256, 16 of 3000, 1, 2, 4: 117, 98, 86.
  a.heads = fits ? (int)std::clamp<int64_t>(lists * a.c.H * waves / (12 * 256), 1, a.c.H) : 1;
  a.groups = (a.c.H + a.heads - 1) / a.heads;
  int64_t query_sets = 0;
  size_t lds = std::max(fits ? table : 0, (size_t)waves * (wide || D == 64 ? Map<64>::kImage : Map<128>::kImage));
  if (queries) {
    const RotaryShare share = rotary_share(a.q, threads, a.s.total);
    a.q_rows = std::min(share.rows, a.s.max_count);
    a.q_heads = share.heads;
    a.q_parts = share.parts;
    a.q_chunks = (a.s.max_count + a.q_rows - 1) / a.q_rows;
    query_sets = (int64_t)a.s.batch * a.q_chunks * a.q_parts;
    lds = std::max(lds, (size_t)a.q_rows * a.r.half * sizeof(float2));
  }
  const int64_t all = lists * (a.groups + a.c.H) + query_sets;
  if (all > 0x7FFFFFFF) return MSQ_ERR_SHAPE;
  a.keys = (unsigned)(lists * a.groups);
  a.values = (unsigned)(lists * a.c.H);
  auto go = [&](auto dims, auto in_table) {
    return launch_all(a, (unsigned)all, threads, [&](dim3 grid, dim3 block) {
      hipLaunchKernelGGL((k_kv_append<D, decltype(dims)::value, T, decltype(in_table)::value>), grid, block, lds,
                         stream, a);
    });
  };
  if constexpr (D == 256)
    if (!fits) return go(std::integral_constant<int, 128>{}, std::false_type{});  // blocks of 256: not wide
  if constexpr (D != 64)
    if (!wide) return go(std::integral_constant<int, 128>{}, std::true_type{});
  return go(std::integral_constant<int, 64>{}, std::true_type{});
}

}  // namespace
}  // namespace msq

using namespace msq;

extern "C" msq_status msq_kv_append(const msq_kv_cache* cache, const msq_kv_seqs* seqs, const int32_t* first,
                                    const msq_kv_new* rows, hipStream_t stream) {
  if (!rows) return MSQ_ERR_INVALID_ARG;
  AppendArgs a{};
  int64_t reach = 0, blocks = 0;
  msq_status st = kv_common(cache, seqs, first, rows->k, rows->v, rows->dtype, true, a.c, a.s, &reach, &blocks);
  if (st != MSQ_OK) return st;
  const bool queries = rows->q.x != nullptr;
  st = rotary_view(&rows->rot, cache->head_dim, true, a.r);
  if (st != MSQ_OK) return st;
  if (queries) {
    if (rows->source) return MSQ_ERR_INVALID_ARG;
    if (rows->q.head_dim != cache->head_dim) return MSQ_ERR_SHAPE;
    st = rotary_rows_view(&rows->q, a.q);
    if (st != MSQ_OK) return st;
  }
  if (blocks == 0) return MSQ_OK;
  const int64_t per16 = rows->dtype == MSQ_DTYPE_F32 ? 4 : 8;
  if (rows->k_token_stride % per16 || rows->k_head_stride % per16 || rows->v_token_stride % per16 ||
      rows->v_head_stride % per16)
    return MSQ_ERR_INVALID_ARG;
  if (rows->kv_rows < (rows->source ? 1 : a.s.total) || rows->kv_rows > 0x7FFFFFFF) return MSQ_ERR_SHAPE;
  if (!aligned_to(rows->source, 4) || !aligned_to(rows->count, 4) || !aligned_to(rows->positions, 4))
    return MSQ_ERR_INVALID_ARG;
  if (queries && (st = rotary_rows_pointers(&rows->q)) != MSQ_OK) return st;
  a.first = first;
  a.k = rows->k, a.kts = rows->k_token_stride, a.khs = rows->k_head_stride;
  a.v = rows->v, a.vts = rows->v_token_stride, a.vhs = rows->v_head_stride;
  a.source = rows->source;
  a.count = rows->count;
  a.positions = rows->positions;
  a.kv_rows = (int)rows->kv_rows;
  a.reach = (int)reach;
  const int64_t lists = (int64_t)a.s.batch * reach;
  const bool f32 = rows->dtype == MSQ_DTYPE_F32;
  switch (cache->head_dim) {
    case 64: return f32 ? launch_append<64, float>(a, lists, queries, stream) : launch_append<64, uint16_t>(a, lists, queries, stream);
    case 128: return f32 ? launch_append<128, float>(a, lists, queries, stream) : launch_append<128, uint16_t>(a, lists, queries, stream);
    default: return f32 ? launch_append<256, float>(a, lists, queries, stream) : launch_append<256, uint16_t>(a, lists, queries, stream);
  }
}
