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
// Workgroups that the verifications aim at.  256, 512, 1024: 64 chains of 5 of 128000 entries
// 22.2, 17.9, 18.2 us; 128 trees of 8 of 32000 17.4, 14.9, 14.8.
constexpr int kFill = 1024;
static_assert(kMostRows <= kFill);

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
// down through the words of its set.  A chain of loads and a step of LDS latency for each
// level: one tree of 26 2.2 us, 256 of up to 64 3.4.
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
  int parts;       // workgroups of a sequence (by chance), of a row (by the largest entries)
  int slice;       // entries of a slice (by chance), of a workgroup's share
  int slices;      // of a row
  double* sums;    // [batch][slices]
  uint64_t* best;  // [batch][most][parts]: an entry (high word) and its number
  uint64_t* tags;  // [batch][parts] or [batch][most][parts]: which of this call are there
  uint64_t call;
};

__device__ inline float entry(const float* p) { return *p; }
__device__ inline float entry(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// Rows begin anywhere; groups of four entries begin at -lead, 4 - lead .. so that they can be
// read at once.
template <typename T>
__device__ inline int lead_of(const T* row) {
  return (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T) & 3);
}
// Entries v .. v + 3 of a row, v + lead a multiple of 4, all of them in it.
template <typename T>
__device__ inline void load4(const T* row, int v, float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 f = *reinterpret_cast<const float4*>(row + v);
    x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(row + v);
    x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xFFFF0000u);
    x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xFFFF0000u);
  }
}
// Those of a wavefront's tile of 256 from v on, `none` outside the row.
template <typename T>
__device__ inline void load_tile(const T* row, int v, int V, bool aligned, int lane, float none, float (&x)[4]) {
  if (aligned && v >= 0 && v + 256 <= V) {
    load4(row, v + 4 * lane, x);
  } else if (v >= V) {
    x[0] = x[1] = x[2] = x[3] = none;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = v + 4 * lane + e;
      const float t = entry(row + min(max(i, 0), V - 1));
      x[e] = i >= 0 && i < V ? t : none;
    }
  }
}

// A probability: what is negative, NaN or infinite counts as 0.
__device__ inline double mass(float x) {
  const float p = fmaxf(x, 0.f);  // 0 of a NaN
  return (double)(p < INFINITY ? p : 0.f);
}
// A random number in [0, 1].
__device__ inline double number(float u) { return (double)fminf(fmaxf(u, 0.f), 1.f); }

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

// How the children of a row came about: chosen; drawn, one of each row; drawn, siblings
// one after another.
enum Drafts { kChosen, kDrawnOne, kDrawn };

// The row that the walk has reached, and what it has not taken there.  Of chosen ones count
// rows from `first` on, each with its token and the next one.  Of drawn ones what is left
// is max(scale p - share q, 0): what max(r / m - q, 0) has brought to 0 stays 0, so the
// steps one after another, r / m - q each, come to one multiple of p and one of q
// (scale / m and share / m + 1), and no row is gone through more than once for a step.
// Both multiples are large where m is small, and what rounding leaves of their difference grows
// with them: past 2^53 it is more than q, and entries that have nothing left would get some.  So
// steps are put together up to a scale of kMostScale (1 / scale is the probability that none of
// these siblings is taken); a step past it begins multiples of its own, of what those before it
// (`steps` pairs in `step`) leave.
constexpr double kMostScale = 16.0;
template <typename T>
struct Row {
  const T *p, *q;
  int V, lead;
  bool aligned;
  int count, first;
  const int *next, *token;
  int steps;
  const double2* step;
  double scale, share;
};
// each(f): f(p, q) of all entries that a lane has, p becomes what is left.
template <typename T, Drafts kWay, typename Each>
__device__ inline void left_of(const Row<T>& row, Each&& each) {
#pragma unroll 1
  for (int k = 0;; ++k) {
    const bool last = kWay != kDrawn || k >= row.steps;
    const double2 by = last ? make_double2(row.scale, row.share) : row.step[k];
    each([&](double& p, double q) { p = fmax(fma(by.x, p, -by.y * q), 0.0); });
    if (last) break;
  }
}

// What is left there of N tiles from v on (v + lead a multiple of 4), all read at once.
template <typename T, Drafts kWay, int N>
__device__ inline void left_at(const Row<T>& row, int v, int lane, double (&r)[N][4]) {
  float x[N][4], y[N][4];
#pragma unroll
  for (int k = 0; k < N; ++k) load_tile(row.p, v + 256 * k, row.V, row.aligned, lane, 0.f, x[k]);
  if (kWay != kChosen && row.count > 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) load_tile(row.q, v + 256 * k, row.V, row.aligned, lane, 0.f, y[k]);
  }
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) r[k][e] = mass(x[k][e]);
  if (row.count == 0) return;
  auto each = [&](auto&& f) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) f(r[k][e], y[k][e], 256 * k + e);
  };
  if constexpr (kWay == kChosen) {
#pragma unroll 1
    for (int k = 0, j = row.first; k < row.count; ++k, j = row.next[j]) {
      const int t = __builtin_amdgcn_readfirstlane(row.token[j]) - v;
      if (t < 0 || t >= 256 * N) continue;
      each([&](double& p, float, int at) { p = t - 4 * lane == at ? 0.0 : p; });
    }
  } else {
    left_of<T, kWay>(row, [&](auto&& f) {
      each([&](double& p, float& q, int) {
        if constexpr (kWay == kDrawn) asm volatile("" : "+v"(q));  // widened anew in each turn: no registers for it
        f(p, mass(q));
      });
    });
  }
}

// A lane's part of the sum of what is left in the slice from lo on.  (A kernel's code is fetched
// as it goes: with tiles unrolled wherever they are looked at, 50 KB, a call took twice as
// long as with a tile at a time.)
constexpr int kSlice = 1024, kMostSlices = 256;
template <typename T, Drafts kWay>
__device__ inline double left_sum(const Row<T>& row, int64_t lo, int size, int lane) {
  double sum = 0.0;
  const int64_t hi = min(lo + size, (int64_t)row.V);
#pragma unroll 1
  for (; lo < hi; lo += kSlice) {
    double r[4][4];
    left_at<T, kWay>(row, (int)lo, lane, r);
#pragma unroll
    for (int k = 0; k < 4; ++k) sum += (r[k][0] + r[k][1]) + (r[k][2] + r[k][3]);
  }
  return sum;
}

// By chance.  Every workgroup of a sequence walks through its tree: the probabilities of
// the drafted tokens come into LDS at once, so a step is no chain of loads; a sum
// over all entries is needed only between siblings drawn from q.  Then its wavefronts add
// up their slices of what is left at the row where the walk ends; the workgroup that
// comes last (tags as in the cache attention's join) finds the slice in which the
// running sum passes the number, and the entry in it.
//
// One row of probabilities for each sequence has to be read (two if drawn): 64 chains of 5 of
// 128000 fp32 entries, 65 MB in 16 to 18 us (12.7 at the copy rate).  Fewer sequences are a
// chain of some ten loads, stores and waits: one chain of 32000 8.7 us, a chosen tree of 26
// of 128000 11, 16 of up to 32 16.  Between drawn siblings a compute unit reads both rows,
// 1 MB for 128000 entries, some 10 us a sibling: 16 trees of 32 153 us, one of 26 21 (with
// four wavefronts a workgroup and r / m - q for each sibling in turn 756 and 27).
constexpr int waves_of(Drafts way) { return way == kDrawn ? 16 : 4; }
template <typename T, Drafts kWay>
__global__ __launch_bounds__(64 * waves_of(kWay)) void k_verify_chance(VerifyArgs a) {
  constexpr int kWaves = waves_of(kWay), kThreads = 64 * kWaves;
  constexpr bool kDraft = kWay != kChosen;
  __shared__ int parent[kMostRows], token[kMostRows], path[kMostRows], next[kDraft ? 1 : kMostRows];
  __shared__ float prob[kMostRows], drawn[kDraft ? kMostRows : 1], number_of[kMostRows];
  __shared__ double shared_sum[kWaves];
  __shared__ double fresh[kMostSlices];  // sums of slices made by the workgroup that joins
  __shared__ double2 step[kWay == kDrawn ? kMostRows : 1];
  __shared__ int complete, last_of[kWaves], found;
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
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int p = parent_of(a.parents, row0, i), t = a.tokens[row0 + i];
    const bool some = p >= 0 && t >= 0 && t < a.V;
    parent[i] = p;
    token[i] = some ? t : -1;
    number_of[i] = a.uniform[row0 + i];
    prob[i] = some ? entry(target + (row0 + p) * a.ts + t) : 0.f;
    if constexpr (kDraft) drawn[i] = some ? entry(draft + (row0 + p) * a.ds + t) : 0.f;
  }
  if (threadIdx.x == 0) path[0] = 0;
  __syncthreads();

  Row<T> row;
  row.V = a.V;
  row.first = 0;
  row.next = next;
  row.token = token;
  row.step = step;
  auto reach = [&](int i) {
    row.p = target + (row0 + i) * a.ts;
    row.q = kDraft ? draft + (row0 + i) * a.ds : row.p;
    row.lead = lead_of(row.p);
    row.aligned = lead_of(row.q) == row.lead;
    row.count = 0;
    row.steps = 0;
    row.scale = 1.0;
    row.share = 0.0;
  };
  reach(0);
  // the walk, the same in all wavefronts
  int at = 0, taken = 1, last = 0;
  double m = 1.0;  // the sum of what is left; of drawn siblings -1 until it is needed
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
      if constexpr (kDraft) q = mass(drawn[j]);
      if constexpr (kWay == kChosen) {
        for (int k = 0, i = row.first; k < row.count; ++k, i = next[i])
          if (token[i] == x) r = 0.0;
      }
      if constexpr (kWay == kDrawn) {
        if (row.count > 0) {
          if (m < 0.0) {
            double s = 0.0;
            for (int i = wave; i < a.slices; i += kWaves)
              s += left_sum<T, kWay>(row, (int64_t)i * a.slice - row.lead, a.slice, lane);
            __syncthreads();
            s = wave_sum(s);
            if (lane == 0) shared_sum[wave] = s;
            __syncthreads();
            m = 0.0;
            for (int w = 0; w < kWaves; ++w) m += shared_sum[w];
          }
          left_of<T, kWay>(row, [&](auto&& f) { f(r, q); });
        }
      }
      if (x >= 0 && number(number_of[j]) * q * m < r) {
        if (threadIdx.x == 0) path[taken] = j;
        ++taken;
        at = j;
        m = 1.0;
        reach(j);
      } else {
        if constexpr (kDraft) {
          if constexpr (kWay == kDrawn) {
            if (m > 0.0 && row.count > 0 && !(row.scale <= kMostScale * m)) {
              // (as with `next`; the last wavefront that read an entry of another row's steps has since
              // come to the sum above)
              step[row.steps] = make_double2(row.scale, row.share);
              __builtin_amdgcn_wave_barrier();
              ++row.steps;
              row.scale = 1.0, row.share = 0.0;
            }
          }
          if (m > 0.0) row.scale /= m, row.share /= m;
          row.share += 1.0;
          m = -1.0;
        } else {
          // (every wavefront writes this, the same, and none reads it before it has)
          if (row.count == 0)
            row.first = j;
          else
            next[last] = j;
          last = j;
          __builtin_amdgcn_wave_barrier();
          m -= r;
        }
        ++row.count;
      }
    }
  }

  double* sums = a.sums + (int64_t)b * a.slices;
  const int each = (a.slices + a.parts - 1) / a.parts;
  int begin = part * each, end = min(begin + each, a.slices);
  const double u = number(number_of[0]);
  double x = 0.0, start = 0.0;
  int s = -1;
  for (bool joined = false;; joined = true) {
    for (int i = begin + wave; i < end; i += kWaves) {
      const double sum = wave_sum(left_sum<T, kWay>(row, (int64_t)i * a.slice - row.lead, a.slice, lane));
      if (lane == 0) {
        // (two workgroups may both see that all have come: what one makes after that is its own)
        if (joined)
          fresh[i] = sum;
        else
          __hip_atomic_store(sums + i, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    auto sum_of = [&](int i) {
      return joined ? fresh[i] : __hip_atomic_load(sums + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    // device-scope stores have reached the level that all XCDs share once vmcnt is 0
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (!joined && a.parts > 1) {
      if (wave == 0) {
        uint64_t* tags = a.tags + (int64_t)b * a.parts;
        if (lane == 0) __hip_atomic_store(tags + part, a.call, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const bool there = lane >= a.parts ||
                           __hip_atomic_load(tags + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.call;
        const bool all = __all(there);
        if (all && lane < a.parts)
          __hip_atomic_store(tags + lane, (uint64_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (lane == 0) complete = all;
      }
      __syncthreads();
      if (!complete) return;
    }
    // the slice in which the running sum passes x, and the sum before it; where rounding leaves
    // none, the last one that has any
    double four[4], mine = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) four[e] = 4 * lane + e < a.slices ? sum_of(4 * lane + e) : 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) mine += four[e];
    const double upto = wave_scan(mine, lane), all = __shfl(upto, 63);
    if (all > 0.0) {
      x = u * all;
      const uint64_t past = __ballot(upto > x && mine > 0.0), some = __ballot(mine > 0.0);
      const int from = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
      double run = upto - mine, run_at = run;
      int hit = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (four[e] > 0.0 && !(hit >= 0 && run > x)) hit = 4 * lane + e, run_at = run;
        run += four[e];
      }
      s = __shfl(hit, from);
      start = __shfl(run_at, from);
      break;
    }
    if (joined || row.count == 0) break;
    reach(at);  // nothing is left: the distribution as it was
    begin = 0, end = a.slices;
    __syncthreads();
  }
  if (threadIdx.x == 0) found = -1;
  if (s >= 0) {
    // a tile for each wavefront
    const int64_t lo = (int64_t)s * a.slice - row.lead, hi = min(lo + a.slice, (int64_t)a.V);
    int spare = -1;  // the last entry with any mass
    for (int64_t c = lo; c < hi; c += 256 * kWaves) {
      const int v = (int)c + 256 * wave + 4 * lane;
      double tile[1][4] = {{0.0, 0.0, 0.0, 0.0}};
      if (c + 256 * wave < hi) left_at<T, kWay>(row, (int)c + 256 * wave, lane, tile);
      const double(&r)[4] = tile[0];
      const double here = (r[0] + r[1]) + (r[2] + r[3]);
      const double upto = wave_scan(here, lane), sum = __shfl(upto, 63);
      int any = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r[e] > 0.0) any = v + e;
      const uint64_t some = __ballot(any >= 0);
      __syncthreads();
      if (lane == 0) shared_sum[wave] = sum;
      const int wave_last = some ? __shfl(any, 63 - __builtin_clzll(some)) : -1;
      if (lane == 0) last_of[wave] = wave_last;
      __syncthreads();
      int hit_wave = -1;
      double before = start;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const double t = shared_sum[w];
        if (last_of[w] >= 0) spare = last_of[w];
        if (hit_wave < 0 && t > 0.0 && start + t > x) hit_wave = w, before = start;
        start += t;
      }
      if (hit_wave < 0) continue;
      if (wave == hit_wave) {
        const uint64_t past = __ballot(any >= 0 && before + upto > x);
        const int from = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
        double t = before + (upto - here);
        int hit = any;
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          double run = t;
#pragma unroll
          for (int i = 0; i <= e; ++i) run += r[i];
          if (r[e] > 0.0 && run > x) hit = v + e;
        }
        hit = __shfl(hit, from);
        if (lane == 0) found = hit;
      }
      spare = -1;
      break;
    }
    __syncthreads();
    if (spare >= 0 && threadIdx.x == 0) found = spare;
  }
  if (threadIdx.x == 0) a.token[b] = found, a.taken[b] = taken;
  for (int i = threadIdx.x; i < count; i += kThreads) a.path[row0 + i] = i < taken ? row0 + path[i] : -1;
}

constexpr int kRowPart = 4096;  // least entries of a row's part: each thread reads 16 at once

// Entry x at v before y at w: larger, or as large and first.
__device__ inline bool before(float x, int v, float y, int w) { return x > y || (x == y && v < w); }

// By the largest entries.  A workgroup finds the largest of its slice of a row, the first
// of equal ones; the one that comes last of a sequence (tags again) walks through its tree.
// All rows are read, also those that the walk leaves out, for it would wait for each row
// in turn: one tree of 26 of 32000 fp32 entries 7.1 us (in two launches 10), 64 chains of
// 5 of 128000, 164 MB, 34 us, 4.8 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void k_verify_largest(VerifyArgs a) {
  __shared__ int parent[kMostRows], token[kMostRows], top[kMostRows], path[kMostRows];
  __shared__ uint64_t best_of[4], part_best[kFill];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned item = blockIdx.x / (unsigned)a.parts, b = item / (unsigned)a.r.most;
  const int part = (int)(blockIdx.x - item * a.parts), mine = (int)(item - b * a.r.most);
  int row0, count, n;
  rows_of(a.r, b, row0, count, n);
  if (mine >= n) {
    if (mine == 0 && part == 0 && threadIdx.x == 0) a.token[b] = -1, a.taken[b] = 0;
    return;
  }
  const T* p = reinterpret_cast<const T*>(a.target) + (row0 + mine) * a.ts;
  const int64_t first = (int64_t)part * a.slice - lead_of(p);
  const int lo = (int)min(first, (int64_t)a.V), hi = (int)min(first + a.slice, (int64_t)a.V);
  float best = -INFINITY;
  int at = kNobody;
  auto meet = [&](const float (&x)[4], int v) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (before(x[e], v + e, best, at)) best = x[e], at = v + e;
  };
#pragma unroll 1
  for (int v0 = lo + 256 * wave; v0 < hi; v0 += kRowPart) {
    float x[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) load_tile(p, v0 + 1024 * k, a.V, true, lane, NAN, x[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) meet(x[k], v0 + 1024 * k + 4 * lane);
  }
  auto join = [&](float x, int v) {
    if (before(x, v, best, at)) best = x, at = v;
  };
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) join(__shfl_xor(best, m), __shfl_xor(at, m));
  if (lane == 0) best_of[wave] = (uint64_t)__float_as_uint(best) << 32 | (uint32_t)at;
  __syncthreads();
  const int64_t seq = (int64_t)b * a.r.most * a.parts;
  uint64_t *bests = a.best + seq, *tags = a.tags + seq;
  const int place = mine * a.parts + part, all = n * a.parts;
  if (threadIdx.x == 0) {
    for (int w = 1; w < 4; ++w) join(__uint_as_float((uint32_t)(best_of[w] >> 32)), (int)(uint32_t)best_of[w]);
    __hip_atomic_store(bests + place, (uint64_t)__float_as_uint(best) << 32 | (uint32_t)at, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
    // it has reached the level that all XCDs share once vmcnt is 0; then the tag, then the look
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __hip_atomic_store(tags + place, a.call, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  __syncthreads();
  bool there = true;  // four at once: all <= kFill, or one part of each of at most kMostRows rows
#pragma unroll
  for (int k = 0; k < kFill / 256; ++k) {
    const int i = 256 * k + threadIdx.x;
    there &= i >= all || __hip_atomic_load(tags + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.call;
  }
  if (!__syncthreads_and(there)) return;
#pragma unroll
  for (int k = 0; k < kFill / 256; ++k) {
    const int i = 256 * k + threadIdx.x;
    if (i < all) {
      part_best[i] = __hip_atomic_load(bests + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(tags + i, (uint64_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (i < n) {
      parent[i] = parent_of(a.parents, row0, i);
      // (kNobody, the largest of a row of NaN, is no token either)
      const int t = a.tokens[row0 + i];
      token[i] = t >= 0 && t < a.V ? t : -1;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 256) {
    best = -INFINITY;
    at = kNobody;
    for (int k = 0; k < a.parts; ++k) {
      const uint64_t w = part_best[i * a.parts + k];
      join(__uint_as_float((uint32_t)(w >> 32)), (int)(uint32_t)w);
    }
    top[i] = at;
  }
  __syncthreads();
  int node = 0, taken = 1;
  if (threadIdx.x == 0) path[0] = 0;
  for (int c = 0; c < n; c += 64) {
    const int i = c + lane, above = i < n ? parent[i] : -1, x = i < n ? token[i] : -1;
    uint64_t open = ~0ull;
    for (;;) {
      const uint64_t fits = __ballot(i > 0 && above == node && x == top[node]) & open;
      if (!fits) break;
      const int j = c + __builtin_ctzll(fits);
      open = j - c == 63 ? 0 : ~0ull << (j - c + 1);
      if (threadIdx.x == 0) path[taken] = j;
      ++taken;
      node = j;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.token[b] = top[node] != kNobody ? top[node] : -1;
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

constexpr int kMostParts = 64;  // of a sequence or row: one wavefront looks at a sequence's tags

struct VerifyPlan {
  int parts, slice, slices;
  int64_t blocks;
  size_t workspace, at;  // at: of the tags
};
msq_status plan_verify(const msq_draft& d, Rows& r, VerifyPlan& p) {
  p = VerifyPlan{};
  const msq_status st = rows_view(d.offset, d.batch, d.total, d.max_count, r);
  if (st != MSQ_OK) return st;
  if (d.vocab < 1 || d.vocab > 1 << 30) return MSQ_ERR_SHAPE;
  if (d.batch == 0) return MSQ_OK;
  r.most = std::max(r.most, 1);
  const int64_t items = d.uniform ? d.batch : (int64_t)d.batch * r.most;
  // all parts of calls of any size up to this one are at most `most` (a row may begin three
  // entries before its first group of four)
  const int64_t unit = d.uniform ? kSlice : kRowPart;
  const int64_t most = std::max<int64_t>(items, kFill), groups = ((int64_t)d.vocab + 3 + unit - 1) / unit;
  const int64_t waves = waves_of(!d.draft ? kChosen : d.parents ? kDrawn : kDrawnOne);
  const int64_t fill = d.uniform ? 4 * kFill / waves : kFill;           // workgroups
  const int64_t split = d.uniform ? (groups + waves - 1) / waves : groups;  // a slice a wavefront at least
  p.parts = (int)std::clamp<int64_t>(std::min(fill / items, split), 1, kMostParts);
  if (d.uniform) {
    p.slice = (int)((groups + kMostSlices - 1) / kMostSlices * kSlice);
    p.slices = (int)(((int64_t)d.vocab + 3 + p.slice - 1) / p.slice);
    p.at = (size_t)d.batch * std::min<int64_t>(groups, kMostSlices) * 8;
  } else {
    p.slice = (int)((groups + p.parts - 1) / p.parts * unit);
    p.at = (size_t)most * 8;
  }
  p.workspace = p.at + (size_t)most * 8;
  p.blocks = items * p.parts;
  if (p.blocks > kMostThreads / (64 * (d.uniform ? waves : 4))) return MSQ_ERR_SHAPE;
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
  Rows r;
  VerifyPlan p;
  return d && plan_verify(*d, r, p) == MSQ_OK ? p.workspace : 0;
}

extern "C" msq_status msq_verify_draft(const msq_draft* d, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
  if (!d) return MSQ_ERR_INVALID_ARG;
  VerifyArgs a{};
  VerifyPlan p;
  const msq_status st = plan_verify(*d, a.r, p);
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
  // (without rows no workgroup gets as far as the workspace, and `uniform`, an array of as many numbers
  // as rows, may be null in either way)
  if (rows && workspace_bytes < p.workspace) return MSQ_ERR_BUFFER_TOO_SMALL;
  if (rows && (!workspace || !aligned_to(workspace, 256))) return MSQ_ERR_INVALID_ARG;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  a.V = d->vocab;
  a.tokens = d->tokens, a.parents = d->parents, a.uniform = d->uniform;
  a.target = d->target, a.ts = d->target_stride;
  a.draft = d->draft, a.ds = d->draft_stride;
  a.token = d->token, a.taken = d->taken, a.path = d->path;
  a.parts = p.parts;
  a.slice = p.slice;
  a.slices = p.slices;
  const dim3 threads(256);
  if (chance) {
    a.sums = reinterpret_cast<double*>(ws);
    a.tags = reinterpret_cast<uint64_t*>(ws + p.at);
    a.call = next_call();
    const dim3 grid((unsigned)p.blocks);
    auto go = [&](auto t) {
      using T = decltype(t);
      if (!drawn) hipLaunchKernelGGL((k_verify_chance<T, kChosen>), grid, threads, 0, stream, a);
      else if (!d->parents) hipLaunchKernelGGL((k_verify_chance<T, kDrawnOne>), grid, threads, 0, stream, a);
      else hipLaunchKernelGGL((k_verify_chance<T, kDrawn>), grid, dim3(64 * waves_of(kDrawn)), 0, stream, a);
    };
    f32 ? go(float{}) : go(uint16_t{});
    return hipGetLastError() == hipSuccess ? MSQ_OK : MSQ_ERR_HIP;
  }
  a.best = reinterpret_cast<uint64_t*>(ws);
  a.tags = reinterpret_cast<uint64_t*>(ws + p.at);
  a.call = next_call();
  const dim3 grid((unsigned)p.blocks);
  if (f32) hipLaunchKernelGGL((k_verify_largest<float>), grid, threads, 0, stream, a);
  else hipLaunchKernelGGL((k_verify_largest<uint16_t>), grid, threads, 0, stream, a);
  return hipGetLastError() == hipSuccess ? MSQ_OK : MSQ_ERR_HIP;
}
