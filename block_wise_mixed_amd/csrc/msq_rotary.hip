// Rotary positions (msq_rotary_apply): formulas and roundings in msq.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "msq.h"
#include "msq_kv.h"
#include "msq_rotary.h"

namespace msq {
namespace {

struct RotaryArgs {
  RotaryView r;
  RotaryRowsView v;
  const int32_t* positions;
  int rows, each;       // of the call, of a workgroup
  int heads, parts;     // of a workgroup; workgroups that share its rows
  unsigned begin;
};

extern __shared__ __align__(16) unsigned char smem_turns[];

// A workgroup takes a few rows of some heads, a unit of 16 values a thread: the turns of a row are
// made once in LDS, in fp64, and used for all of its heads.  HBM bound: 28707 rows of 32 bf16
// heads of 128, 470 MB in 77 to 81 us, 5.8 to 6.1 TB/s (a large copy runs at 5.1 to 5.2).  With four
// units a thread, and so fewer, longer workgroups, 162 us; with 64 rows a workgroup 192.  A
// step of 64 rows of 64 fp32 heads 3.5 us.
__global__ __launch_bounds__(256) void k_rotary(RotaryArgs a) {
  const unsigned id = a.begin + blockIdx.x, chunk = id / (unsigned)a.parts, part = id - chunk * a.parts;
  const int row0 = (int)chunk * a.each, rows = min(a.each, a.rows - row0);
  const int h0 = (int)part * a.heads, heads = min(a.heads, a.v.heads - h0);
  rotate_rows(a.v, a.r, row0, rows, h0, heads, reinterpret_cast<float2*>(smem_turns),
              [&](int i) { return a.positions[row0 + i]; });
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

msq_status rotary_view(const msq_rotary* rot, int head_dim, bool none, RotaryView& r) {
  if (!rot) return MSQ_ERR_INVALID_ARG;
  if (rot->dims < (none ? 0 : 16) || rot->dims % 16 || rot->dims > head_dim) return MSQ_ERR_SHAPE;
  if (!std::isfinite(rot->amplitude)) return MSQ_ERR_INVALID_ARG;
  if (rot->dims && (!rot->freq || !aligned_to(rot->freq, 8))) return MSQ_ERR_INVALID_ARG;
  r.freq = rot->freq;
  r.amplitude = rot->amplitude == 0.0 ? 1.0 : rot->amplitude;
  r.half = rot->dims / 2;
  r.interleaved = rot->interleaved != 0;
  return MSQ_OK;
}

msq_status rotary_rows_view(const msq_rotary_rows* x, RotaryRowsView& v) {
  if (!x) return MSQ_ERR_INVALID_ARG;
  if (x->heads < 1 || x->head_dim < 16 || x->head_dim % 16 || x->head_dim > MSQ_ROTARY_MAX_DIM ||
      (int64_t)x->heads * x->head_dim > 0x7FFFFFFF)
    return MSQ_ERR_SHAPE;
  for (const int32_t t : {x->x_dtype, x->out_dtype})
    if (t != MSQ_DTYPE_BF16 && t != MSQ_DTYPE_F32) return MSQ_ERR_INVALID_ARG;
  v.x = x->x;
  v.out = x->out;
  v.xts = x->x_token_stride;
  v.xhs = x->x_head_stride;
  v.ots = x->out_token_stride;
  v.ohs = x->out_head_stride;
  v.heads = x->heads;
  v.units = x->head_dim / 16;
  v.x_f32 = x->x_dtype == MSQ_DTYPE_F32;
  v.out_f32 = x->out_dtype == MSQ_DTYPE_F32;
  return MSQ_OK;
}

msq_status rotary_rows_pointers(const msq_rotary_rows* x) {
  const int64_t in = x->x_dtype == MSQ_DTYPE_F32 ? 4 : 8, out = x->out_dtype == MSQ_DTYPE_F32 ? 4 : 8;
  if (!x->x || !x->out || !aligned_to(x->x, 16) || !aligned_to(x->out, 16) || x->x_token_stride % in ||
      x->x_head_stride % in || x->out_token_stride % out || x->out_head_stride % out)
    return MSQ_ERR_INVALID_ARG;
  return MSQ_OK;
}

}  // namespace msq

using namespace msq;

extern "C" msq_status msq_rotary_apply(const msq_rotary* rot, const msq_rotary_rows* x,
                                       const int32_t* positions, int64_t rows, hipStream_t stream) {
  RotaryArgs a{};
  msq_status st = rotary_rows_view(x, a.v);
  if (st == MSQ_OK) st = rotary_view(rot, x->head_dim, false, a.r);
  if (st != MSQ_OK) return st;
  if (rows < 0 || rows > 0x7FFFFFFF) return MSQ_ERR_SHAPE;
  if (rows == 0) return MSQ_OK;
  st = rotary_rows_pointers(x);
  if (st != MSQ_OK) return st;
  if (!positions || !aligned_to(positions, 4)) return MSQ_ERR_INVALID_ARG;
  a.positions = positions;
  a.rows = (int)rows;
  const RotaryShare share = rotary_share(a.v, 256, rows);
  a.heads = share.heads;
  a.parts = share.parts;
  a.each = share.rows;
  const int64_t blocks = (rows + a.each - 1) / a.each * a.parts;
  const size_t lds = (size_t)a.each * a.r.half * sizeof(float2);
  const int64_t most = kMostThreads / 256;
  // (workgroup numbers of a launch are added to `begin` in 32 bits)
  if (blocks > 0xFFFFFFFFll) return MSQ_ERR_SHAPE;
  for (int64_t done = 0; done < blocks; done += most) {
    a.begin = (unsigned)done;
    hipLaunchKernelGGL(k_rotary, dim3((unsigned)std::min(blocks - done, most)), dim3(256), lds, stream, a);
    if (hipGetLastError() != hipSuccess) return MSQ_ERR_HIP;
  }
  return MSQ_OK;
}
