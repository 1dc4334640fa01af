// Drafted tokens: the sets of a tree (msq_draft_tree) and which of them the target's
// probabilities keep (msq_verify_draft).  Formulas in msq.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "msq.h"
#include "msq_kv.h"

namespace msq {
namespace {

constexpr int kMostRows = MSQ_DRAFT_MAX_ROWS;
constexpr int kNobody = 0x7FFFFFFF;

// The rows of the sequences of a call; those of one: row0 .. row0 + count - 1, of which
// the first n are looked at.
struct Rows {
  const int32_t* offset;
  int batch, total, per_seq, most;  // most: rows of a sequence that are looked at
};
__device__ inline void rows_of(const Rows& r, int b, int& row0, int& count, int& n) {
  row0 = b * r.per_seq;
  count = r.per_seq;
  if (r.offset) {
    row0 = min(max(r.offset[b], 0), r.total);
    count = min(max(r.offset[b + 1], row0), r.total) - row0;
  }
  n = min(count, r.most);
}

// The parent of row i as the walk takes it: a smaller row, or -1.
__device__ inline int parent_of(const int32_t* parents, int row0, int i) {
  const int p = parents ? parents[row0 + i] : i - 1;
  return p >= 0 && p < i ? p : -1;
}

// ---- sets of a tree ----------------------------------------------------------
struct TreeArgs {
  Rows r;
  const int32_t *parents, *first;
  uint32_t* sets;
  int words;
  int32_t* positions;
};

// A workgroup takes a sequence: parents in LDS, and each thread walks up from its rows,
// down through the words of its set.
__global__ __launch_bounds__(256) void k_draft_tree(TreeArgs a) {
  __shared__ int parent[kMostRows];
  const int b = blockIdx.x;
  int row0, count, n;
  rows_of(a.r, b, row0, count, n);
  for (int i = threadIdx.x; i < n; i += blockDim.x) parent[i] = parent_of(a.parents, row0, i);
  __syncthreads();
  const int first = a.positions && a.first ? a.first[b] : 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    uint32_t* set = a.sets + (int64_t)(row0 + i) * a.words;
    int w = a.words - 1, depth = -1;
    uint32_t m = 0;
    for (int j = i; j >= 0; j = parent[j], ++depth) {
      for (; w > j >> 5; --w, m = 0) set[w] = m;
      m |= 1u << (j & 31);
    }
    for (; w >= 0; --w, m = 0) set[w] = m;
    if (a.positions) a.positions[row0 + i] = first + depth;
  }
}

// ---- verification ------------------------------------------------------------
struct VerifyArgs {
  Rows r;
  int V;
  const int32_t *tokens, *parents;
  const void *target, *draft;
  int64_t ts, ds;  // row strides
  const float* uniform;
  int32_t *token, *taken, *path;
  int parts;     // workgroups of a sequence (by chance), of a row (by the largest entries)
  int slice;     // entries of a wavefront's share, of a workgroup's
  int aligned;   // rows can be read four entries at a time
  double* sums;  // [batch][4 parts]
  uint64_t* tags;  // [batch][parts]
  uint64_t call;
  float* top;    // [total * parts], and beside it the entries' numbers
  int32_t* top_at;
};

__device__ inline float entry(const float* p) { return *p; }
__device__ inline float entry(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// Entries v .. v + 3 of a row, `none` past its end.
template <typename T>
__device__ inline void load4(const T* row, int v, int V, bool aligned, float none, float (&x)[4]) {
  if (aligned && v + 4 <= V) {
    if constexpr (sizeof(T) == 4) {
      const float4 f = *reinterpret_cast<const float4*>(row + v);
      x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(row + v);
      x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xFFFF0000u);
      x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xFFFF0000u);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = v + e < V ? entry(row + v + e) : none;
}

// A probability: what is negative, NaN or infinite counts as 0.
__device__ inline double mass(float x) { return x > 0.f && x < INFINITY ? (double)x : 0.0; }
// A random number in [0, 1].
__device__ inline double number(float u) { return u > 0.f ? (double)fminf(u, 1.f) : 0.0; }

__device__ inline double wave_sum(double x) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
  return x;
}
// The sum of the lanes up to this one.
__device__ inline double wave_scan(double x, int lane) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double y = __shfl_up(x, m);
    if (lane >= m) x += y;
  }
  return x;
}

// What is left of the target's distribution after row `at` once the rows in gone were not
// taken: with draft by the sums m of what was left before each of them, else without
// their tokens.
struct Left {
  const double* m;
  const int* gone;
  int count;
};
template <bool kDraft>
__device__ inline double left_of(const Left& l, double p, double q) {
  if constexpr (kDraft) {
    for (int k = 0; k < l.count; ++k) {
      const double m = l.m[k];
      p = fmax((k == 0 || m <= 0.0 ? p : p / m) - q, 0.0);
    }
  }
  return p;
}

// Four entries of what is left.
template <typename T, bool kDraft>
__device__ inline void left4(const VerifyArgs& a, const Left& l, const T* p, const T* q, int v, double (&r)[4]) {
  float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
  load4(p, v, a.V, a.aligned, 0.f, x);
  if (kDraft && l.count > 0) load4(q, v, a.V, a.aligned, 0.f, y);
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = left_of<kDraft>(l, mass(x[e]), mass(y[e]));
  if constexpr (!kDraft) {
    for (int k = 0; k < l.count; ++k) {
      const int t = l.gone[k] - v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t == e) r[e] = 0.0;
    }
  }
}

// Its sum over the entries lo .. hi - 1 by one wavefront.
template <typename T, bool kDraft>
__device__ inline double left_sum(const VerifyArgs& a, const Left& l, const T* p, const T* q, int lo, int hi, int lane) {
  double sum = 0.0;
  for (int v = lo + 4 * lane; v < hi; v += 256) {
    double r[4];
    left4<T, kDraft>(a, l, p, q, v, r);
    sum += (r[0] + r[1]) + (r[2] + r[3]);
  }
  return wave_sum(sum);
}

// By chance.  Every workgroup of a sequence walks through its tree: the probabilities of
// the drafted tokens come into LDS at once, so a step is no chain of loads; a sum
// over all entries is needed only between siblings drawn from q.  Then its wavefronts add
// up their slices of what is left at the row where the walk ends; the workgroup that
// comes last (tags as in the cache attention's join) finds the slice in which the
// running sum passes the number, and the entry in it.
template <typename T, bool kDraft>
__global__ __launch_bounds__(256) void k_verify_chance(VerifyArgs a) {
  constexpr int kWaves = 4;
  __shared__ int parent[kMostRows], token[kMostRows], path[kMostRows], gone[kMostRows];
  __shared__ float prob[kMostRows], drawn[kDraft ? kMostRows : 1], number_of[kMostRows];
  __shared__ double m_of[kDraft ? kMostRows : 1], shared_sum[kWaves];
  __shared__ int complete;
  const int part = blockIdx.x % (unsigned)a.parts, b = blockIdx.x / (unsigned)a.parts;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int row0, count, n;
  rows_of(a.r, b, row0, count, n);
  if (n == 0) {
    if (part == 0 && threadIdx.x == 0) a.token[b] = -1, a.taken[b] = 0;
    return;
  }
  const T* target = reinterpret_cast<const T*>(a.target);
  const T* draft = reinterpret_cast<const T*>(a.draft);
  for (int i = threadIdx.x; i < n; i += 256) {
    const int p = parent_of(a.parents, row0, i), t = a.tokens[row0 + i];
    const bool some = p >= 0 && t >= 0 && t < a.V;
    parent[i] = p;
    token[i] = t;
    number_of[i] = a.uniform[row0 + i];
    prob[i] = some ? entry(target + (row0 + p) * a.ts + t) : 0.f;
    if constexpr (kDraft) drawn[i] = some ? entry(draft + (row0 + p) * a.ds + t) : 0.f;
  }
  __syncthreads();

  // the walk, the same in all wavefronts
  int at = 0, taken = 1;
  double m = 1.0;
  Left l{m_of, gone, 0};
  if (threadIdx.x == 0) path[0] = 0;
  for (int c = 0; c < n; c += 64) {
    const int mine = c + lane < n ? parent[c + lane] : -1;
    uint64_t open = ~0ull;  // rows of these 64 that are still to come
    for (;;) {
      const uint64_t below = __ballot(mine == at && c + lane > 0) & open;
      if (!below) break;
      const int j = c + __builtin_ctzll(below);
      open = j - c == 63 ? 0 : ~0ull << (j - c + 1);
      const int x = __builtin_amdgcn_readfirstlane(token[j]);
      double r = mass(prob[j]), q = 1.0;
      if constexpr (kDraft) {
        q = mass(drawn[j]);
        if (l.count > 0) {  // m is that of what is left now
          const T* pr = target + (row0 + at) * a.ts;
          const T* qr = draft + (row0 + at) * a.ds;
          if (m < 0.0) {
            // the sum that the last row not taken leaves: by slices of the wavefronts
            const int each = ((a.V + kWaves - 1) / kWaves + 255) / 256 * 256;
            const double s = left_sum<T, true>(a, l, pr, qr, min(wave * each, a.V), min((wave + 1) * each, a.V), lane);
            __syncthreads();
            if (lane == 0) shared_sum[wave] = s;
            __syncthreads();
            m = (shared_sum[0] + shared_sum[1]) + (shared_sum[2] + shared_sum[3]);
          }
          r = left_of<true>(l, r, q);
        }
      } else {
        for (int k = 0; k < l.count; ++k)
          if (gone[k] == x) r = 0.0;
      }
      const bool take = x >= 0 && x < a.V && number(number_of[j]) * q * m < r;
      if (take) {
        if (threadIdx.x == 0) path[taken] = j;
        ++taken;
        at = j;
        m = 1.0;
        l.count = 0;
      } else {
        if constexpr (kDraft) {
          __syncthreads();  // every wavefront has read what was there
          if (threadIdx.x == 0) m_of[l.count] = m;
          __syncthreads();
          m = -1.0;  // not known yet
        } else {
          __syncthreads();
          if (threadIdx.x == 0) gone[l.count] = x;
          __syncthreads();
          m -= r;
        }
        ++l.count;
      }
    }
  }

  const T* pr = target + (row0 + at) * a.ts;
  const T* qr = kDraft ? draft + (row0 + at) * a.ds : pr;
  const int slices = kWaves * a.parts;
  double* sums = a.sums + (int64_t)b * slices;
  auto slice_sum = [&](int s) {
    const int lo = (int)min((int64_t)s * a.slice, (int64_t)a.V);
    return left_sum<T, kDraft>(a, l, pr, qr, lo, (int)min((int64_t)lo + a.slice, (int64_t)a.V), lane);
  };
  {
    const int s = part * kWaves + wave;
    const double sum = slice_sum(s);
    if (lane == 0)
      __hip_atomic_store(sums + s, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // device-scope stores have reached the level that all XCDs share once vmcnt is 0
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (a.parts > 1) {
    if (wave == 0) {
      uint64_t* tags = a.tags + (int64_t)b * a.parts;
      if (lane == 0) __hip_atomic_store(tags + part, a.call, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const bool there = lane >= a.parts ||
                         __hip_atomic_load(tags + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.call;
      const bool all = __all(there);
      if (all && lane < a.parts) __hip_atomic_store(tags + lane, (uint64_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (lane == 0) complete = all;
    }
    __syncthreads();
    if (!complete) return;
  }

  // slice s of the running sum that passes x, and what comes before it; if rounding
  // leaves none, the last one that has any
  const double u = number(number_of[0]);
  double x = 0.0, before = 0.0;
  int s = -1;
  for (int attempt = 0; attempt < 2; ++attempt) {
    double four[4], mine = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 4 * lane + e;
      four[e] = i < slices ? __hip_atomic_load(sums + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
      mine += four[e];
    }
    const double upto = wave_scan(mine, lane);
    const double all = __shfl(upto, 63);
    if (all > 0.0) {
      x = u * all;
      const uint64_t past = __ballot(upto > x), some = __ballot(mine > 0.0);
      const int from = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
      // in that lane's four
      double run = upto - mine, start = run;
      int e_hit = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool hit = past ? run + four[e] > x && e_hit < 0 : four[e] > 0.0;
        if (hit) e_hit = e, start = run;
        run += four[e];
      }
      if (e_hit < 0) {  // passed by the lanes' sums, not by these: the last one that has any
        double r = upto - mine;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (four[e] > 0.0) e_hit = e, start = r;
          r += four[e];
        }
      }
      s = 4 * from + __shfl(e_hit, from);
      before = __shfl(start, from);
      break;
    }
    // nothing left: the distribution as it was
    if (attempt == 1 || l.count == 0) break;
    l.count = 0;
    __syncthreads();
    for (int i = wave; i < slices; i += kWaves) {
      const double sum = slice_sum(i);
      if (lane == 0) __hip_atomic_store(sums + i, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }
  int found = -1;
  if (s >= 0) {
    // its quarter, then the entry
    const int lo = (int)min((int64_t)s * a.slice, (int64_t)a.V), hi = (int)min((int64_t)lo + a.slice, (int64_t)a.V);
    const int each = (a.slice / kWaves + 255) / 256 * 256;
    const double mine = left_sum<T, kDraft>(a, l, pr, qr, min(lo + wave * each, hi), min(lo + (wave + 1) * each, hi), lane);
    __syncthreads();
    if (lane == 0) shared_sum[wave] = mine;
    __syncthreads();
    int quarter = -1, last = 0;
    double run = before, start = before, last_start = before;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const double t = shared_sum[w];
      if (quarter < 0 && run + t > x) quarter = w, start = run;
      if (t > 0.0) last = w, last_start = run;
      run += t;
    }
    if (quarter < 0) quarter = last, start = last_start;
    if (wave == 0) {
      const int end = min(lo + (quarter + 1) * each, hi);
      int spare = -1;  // the last entry with any mass
      for (int v0 = lo + quarter * each; v0 < end; v0 += 256) {
        const int v = v0 + 4 * lane;
        double r[4] = {0.0, 0.0, 0.0, 0.0};
        if (v < end) left4<T, kDraft>(a, l, pr, qr, v, r);
        const double here = (r[0] + r[1]) + (r[2] + r[3]);
        const double upto = wave_scan(here, lane);
        const uint64_t past = __ballot(start + upto > x && here > 0.0), some = __ballot(here > 0.0);
        if (past) {
          const int from = __builtin_ctzll(past);
          double t = start + (upto - here);
          int hit = -1, any = -1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            t += r[e];
            if (r[e] > 0.0) any = v + e;
            if (hit < 0 && r[e] > 0.0 && t > x) hit = v + e;
          }
          found = __shfl(hit >= 0 ? hit : any, from);
          break;
        }
        if (some) {
          int any = -1;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (r[e] > 0.0) any = v + e;
          spare = __shfl(any, 63 - __builtin_clzll(some));
        }
        start += __shfl(upto, 63);
      }
      if (found < 0) found = spare;
    }
  }
  if (threadIdx.x == 0) a.token[b] = found, a.taken[b] = taken;
  for (int i = threadIdx.x; i < count; i += 256) a.path[row0 + i] = i < taken ? row0 + path[i] : -1;
}

// Entry x at v before y at w: larger, or as large and first.
__device__ inline bool before(float x, int v, float y, int w) { return x > y || (x == y && v < w); }

// The largest entry of a workgroup's slice of a row, the first of equal ones.
template <typename T>
__global__ __launch_bounds__(256) void k_row_largest(VerifyArgs a) {
  __shared__ float best_of[4];
  __shared__ int at_of[4];
  const int part = blockIdx.x % (unsigned)a.parts, row = blockIdx.x / (unsigned)a.parts;
  const T* p = reinterpret_cast<const T*>(a.target) + row * a.ts;
  const int lo = (int)min((int64_t)part * a.slice, (int64_t)a.V), hi = (int)min((int64_t)lo + a.slice, (int64_t)a.V);
  float best = -INFINITY;
  int at = kNobody;
  for (int v = lo + 4 * threadIdx.x; v < hi; v += 1024) {
    float x[4];
    load4(p, v, a.V, a.aligned, NAN, x);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (before(x[e], v + e, best, at)) best = x[e], at = v + e;
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const float x = __shfl_xor(best, m);
    const int v = __shfl_xor(at, m);
    if (before(x, v, best, at)) best = x, at = v;
  }
  if ((threadIdx.x & 63) == 0) best_of[threadIdx.x >> 6] = best, at_of[threadIdx.x >> 6] = at;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 4; ++w)
      if (before(best_of[w], at_of[w], best, at)) best = best_of[w], at = at_of[w];
    a.top[blockIdx.x] = best;
    a.top_at[blockIdx.x] = at;
  }
}

// By the largest entries: the walk of a sequence.
__global__ __launch_bounds__(256) void k_verify_largest(VerifyArgs a) {
  __shared__ int parent[kMostRows], token[kMostRows], best[kMostRows], path[kMostRows];
  const int b = blockIdx.x, lane = threadIdx.x & 63;
  int row0, count, n;
  rows_of(a.r, b, row0, count, n);
  for (int i = threadIdx.x; i < n; i += 256) {
    parent[i] = parent_of(a.parents, row0, i);
    token[i] = a.tokens[row0 + i];
    const int64_t t = (int64_t)(row0 + i) * a.parts;
    float x = a.top[t];
    int at = a.top_at[t];
    for (int k = 1; k < a.parts; ++k)
      if (before(a.top[t + k], a.top_at[t + k], x, at)) x = a.top[t + k], at = a.top_at[t + k];
    best[i] = at;
  }
  __syncthreads();
  int at = 0, taken = n > 0 ? 1 : 0;
  if (threadIdx.x == 0) path[0] = 0;
  for (int c = 0; c < n; c += 64) {
    const int i = c + lane, mine = i < n ? parent[i] : -1, x = i < n ? token[i] : -1;
    uint64_t open = ~0ull;
    for (;;) {
      const uint64_t fits = __ballot(i > 0 && mine == at && x == best[at]) & open;
      if (!fits) break;
      const int j = c + __builtin_ctzll(fits);
      open = j - c == 63 ? 0 : ~0ull << (j - c + 1);
      if (threadIdx.x == 0) path[taken] = j;
      ++taken;
      at = j;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.token[b] = n > 0 && best[at] != kNobody ? best[at] : -1;
    a.taken[b] = taken;
  }
  for (int i = threadIdx.x; i < count; i += 256) a.path[row0 + i] = i < taken ? row0 + path[i] : -1;
}

// ---- host --------------------------------------------------------------------
bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

msq_status rows_view(const int32_t* offset, int32_t batch, int64_t total, int32_t max_count, Rows& r) {
  if (batch < 0 || total < 0 || total > 0x7FFFFFFF || max_count < 0) return MSQ_ERR_SHAPE;
  if (!offset && (batch == 0 ? total != 0 : total % batch != 0)) return MSQ_ERR_SHAPE;
  r.offset = offset;
  r.batch = batch;
  r.total = (int)total;
  r.per_seq = batch > 0 ? (int)(total / batch) : 0;
  int64_t most = max_count > 0 ? max_count : total;
  if (!offset) most = r.per_seq;
  r.most = (int)std::min<int64_t>({most, total, (int64_t)kMostRows});
  return MSQ_OK;
}

// Workgroups that the calls aim at (by chance, by the largest entries), and the most
// parts of a sequence: its tags are looked at by one wavefront, its slices by four a lane.
constexpr int kChanceFill = 512, kLargestFill = 1024, kMostParts = 64;

struct VerifyPlan {
  int parts, slice;
  int64_t blocks;
  size_t workspace, at;  // at: of the tags, or of the entries' numbers
};
msq_status plan_verify(const msq_draft& d, VerifyArgs& a, VerifyPlan& p) {
  p = VerifyPlan{};
  const msq_status st = rows_view(d.offset, d.batch, d.total, d.max_count, a.r);
  if (st != MSQ_OK) return st;
  if (d.vocab < 1) return MSQ_ERR_SHAPE;
  if (d.batch == 0) return MSQ_OK;
  const int64_t items = d.uniform ? d.batch : d.total, fill = d.uniform ? kChanceFill : kLargestFill;
  const int64_t most = std::max(items, fill);  // parts of all items, at any size up to this one
  p.workspace = d.uniform ? (size_t)most * 40 : (size_t)most * 8;
  p.at = d.uniform ? (size_t)most * 32 : (size_t)most * 4;
  // parts of at least 1024 entries (a wavefront's slice: a multiple of 256)
  const int64_t parts = std::clamp<int64_t>(std::min(fill / std::max<int64_t>(items, 1), ((int64_t)d.vocab + 1023) / 1024), 1, kMostParts);
  const int64_t shares = d.uniform ? 4 * parts : parts, unit = d.uniform ? 256 : 1024;
  const int64_t slice = ((d.vocab + shares - 1) / shares + unit - 1) / unit * unit;
  p.parts = (int)parts;
  p.slice = (int)std::min<int64_t>(slice, 0x7FFFFF00);
  p.blocks = items * parts;
  if (p.blocks > kMostThreads / 256 || d.batch > kMostThreads / 256) return MSQ_ERR_SHAPE;
  return MSQ_OK;
}

}  // namespace
}  // namespace msq

using namespace msq;

extern "C" msq_status msq_draft_tree(const int32_t* parents, const int32_t* offset, int32_t batch, int64_t total,
                                     int32_t max_count, const int32_t* first, uint32_t* sets, int32_t words,
                                     int32_t* positions, hipStream_t stream) {
  TreeArgs a{};
  const msq_status st = rows_view(offset, batch, total, max_count, a.r);
  if (st != MSQ_OK) return st;
  if (batch == 0 || total == 0) return MSQ_OK;
  if (words < 1 || (int64_t)words * 32 < a.r.most || batch > (int)(kMostThreads / 256)) return MSQ_ERR_SHAPE;
  if (!parents || !sets || !aligned_to(parents, 4) || !aligned_to(offset, 4) || !aligned_to(first, 4) ||
      !aligned_to(sets, 4) || !aligned_to(positions, 4))
    return MSQ_ERR_INVALID_ARG;
  a.parents = parents;
  a.first = first;
  a.sets = sets;
  a.words = words;
  a.positions = positions;
  const int threads = std::min(256, (a.r.most + 63) / 64 * 64);
  hipLaunchKernelGGL(k_draft_tree, dim3((unsigned)batch), dim3(threads), 0, stream, a);
  return hipGetLastError() == hipSuccess ? MSQ_OK : MSQ_ERR_HIP;
}

extern "C" size_t msq_verify_draft_workspace_bytes(const msq_draft* d) {
  VerifyArgs a{};
  VerifyPlan p;
  return d && plan_verify(*d, a, p) == MSQ_OK ? p.workspace : 0;
}

extern "C" msq_status msq_verify_draft(const msq_draft* d, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
  if (!d) return MSQ_ERR_INVALID_ARG;
  VerifyArgs a{};
  VerifyPlan p;
  const msq_status st = plan_verify(*d, a, p);
  if (st != MSQ_OK) return st;
  if (d->dtype != MSQ_DTYPE_BF16 && d->dtype != MSQ_DTYPE_F32) return MSQ_ERR_INVALID_ARG;
  if (d->batch == 0) return MSQ_OK;
  const bool f32 = d->dtype == MSQ_DTYPE_F32, chance = d->uniform != nullptr, drawn = chance && d->draft;
  if (d->target_stride < d->vocab || (drawn && d->draft_stride < d->vocab)) return MSQ_ERR_SHAPE;
  const size_t size = f32 ? 4 : 2;
  const bool rows = d->total > 0;
  if (!d->token || !d->taken || (rows && (!d->tokens || !d->target || !d->path)) || !aligned_to(d->tokens, 4) ||
      !aligned_to(d->parents, 4) || !aligned_to(d->offset, 4) || !aligned_to(d->uniform, 4) ||
      !aligned_to(d->token, 4) || !aligned_to(d->taken, 4) || !aligned_to(d->path, 4) ||
      !aligned_to(d->target, size) || (drawn && !aligned_to(d->draft, size)))
    return MSQ_ERR_INVALID_ARG;
  if (workspace_bytes < p.workspace) return MSQ_ERR_BUFFER_TOO_SMALL;
  if (!workspace || !aligned_to(workspace, 256)) return MSQ_ERR_INVALID_ARG;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  a.V = d->vocab;
  a.tokens = d->tokens, a.parents = d->parents, a.uniform = d->uniform;
  a.target = d->target, a.ts = d->target_stride;
  a.draft = d->draft, a.ds = d->draft_stride;
  a.token = d->token, a.taken = d->taken, a.path = d->path;
  a.parts = p.parts;
  a.slice = p.slice;
  a.aligned = d->target_stride % 4 == 0 && aligned_to(d->target, 4 * size) &&
              (!drawn || (d->draft_stride % 4 == 0 && aligned_to(d->draft, 4 * size)));
  const dim3 threads(256);
  if (chance) {
    a.sums = reinterpret_cast<double*>(ws);
    a.tags = reinterpret_cast<uint64_t*>(ws + p.at);
    a.call = next_call();
    const dim3 grid((unsigned)p.blocks);
    if (f32 && drawn) hipLaunchKernelGGL((k_verify_chance<float, true>), grid, threads, 0, stream, a);
    else if (f32) hipLaunchKernelGGL((k_verify_chance<float, false>), grid, threads, 0, stream, a);
    else if (drawn) hipLaunchKernelGGL((k_verify_chance<uint16_t, true>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((k_verify_chance<uint16_t, false>), grid, threads, 0, stream, a);
    return hipGetLastError() == hipSuccess ? MSQ_OK : MSQ_ERR_HIP;
  }
  a.top = reinterpret_cast<float*>(ws);
  a.top_at = reinterpret_cast<int32_t*>(ws + p.at);
  if (p.blocks > 0) {
    const dim3 grid((unsigned)p.blocks);
    if (f32) hipLaunchKernelGGL((k_row_largest<float>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((k_row_largest<uint16_t>), grid, threads, 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MSQ_ERR_HIP;
  }
  hipLaunchKernelGGL(k_verify_largest, dim3((unsigned)d->batch), threads, 0, stream, a);
  return hipGetLastError() == hipSuccess ? MSQ_OK : MSQ_ERR_HIP;
}
