// Shared pieces of the 8-bit key/value cache kernels (msq_kv.hip: write and
// read back; msq_kv_attn.hip: attention).  Layout and quantiser: msq.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "msq.h"

namespace msq {

constexpr int64_t kMostThreads = 0xFFFFFFFF;  // of one launch

// Cache and sequences as the kernels take them.
struct KvCacheView {
  uint8_t *kc, *vc;
  float *ks, *vs;
  int nblocks, H, shift;  // block_tokens = 1 << shift
};

struct KvSeqsView {
  const int32_t* table;
  const int32_t* offset;  // null: per_seq rows each
  int batch, width, total, max_count, per_seq;
};

// First row and row count of sequence b, kept inside 0 .. total whatever
// offset holds.
__device__ inline void kv_rows(const KvSeqsView& s, int b, int& row0, int& count) {
  if (!s.offset) {
    row0 = b * s.per_seq;
    count = s.per_seq;
    return;
  }
  const int lo = min(max(s.offset[b], 0), s.total);
  const int hi = min(max(s.offset[b + 1], lo), s.total);
  row0 = lo;
  count = min(hi - lo, s.max_count);
}

// Physical block of table entry e of sequence b; -1 if absent.
__device__ inline int kv_block(const KvCacheView& c, const KvSeqsView& s, int b, int64_t e) {
  if (e < 0 || e >= s.width) return -1;
  const int id = s.table[(int64_t)b * s.width + e];
  return (unsigned)id < (unsigned)c.nblocks ? id : -1;
}

// Host checks shared by the three entry points; fills the views.
msq_status kv_views(const msq_kv_cache* cache, const msq_kv_seqs* seqs, KvCacheView& c,
                    KvSeqsView& s);
// The pointers of both structs: present and aligned.
msq_status kv_pointers(const msq_kv_cache* cache, const msq_kv_seqs* seqs);


// A number for one call (msq_kv_attn.hip): never 0, and from a start that depends on the
// time, the process and where it was loaded, so that no call finds its number in what a
// workspace held before.
uint64_t next_call();

}  // namespace msq
