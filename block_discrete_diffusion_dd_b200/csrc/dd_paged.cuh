// dd_paged.cuh -- device-side view of a paged batch (dd_paged_batch), shared
// by the cache kernels and the attention over the cache.
//
// Lengths, offsets and page ids live in device memory, where the host cannot
// check them before a launch, so every kernel checks what it uses: a batch
// row with impossible lengths or offsets is taken as empty, a page id outside
// the pool is never followed, and both latch kDevErrBounds in the workspace
// header.  A row that starts before the end of an earlier possible one is
// impossible too, so that a packed row has one owner at most.  Where every
// row's offsets are possible by themselves they are in order, and the owner is
// found by bisection; otherwise the rows are gone through one after the other.
#pragma once

#include "dd_device.cuh"
#include "dd_internal.h"

namespace dd {

struct ChunkRow {
  int q0;   // first row of the packed new-token tensors
  int n;    // new tokens
  int len;  // tokens in the cache, the new ones included
};

// Whether the offsets of row b are possible by themselves, with `most` packed rows.
__device__ __forceinline__ bool offsets_fit(const int32_t* cu, int b, int most) {
  const int q0 = __ldg(cu + b), q1 = __ldg(cu + b + 1);
  return q0 >= 0 && q1 >= q0 && q1 <= most;
}

// Row b, where the possible rows before it end at `end`; an impossible one has
// no tokens and starts (and ends) there.
__device__ __forceinline__ ChunkRow chunk_row(const PagedBatch& p, int b, int end, uint32_t* err) {
  ChunkRow r;
  r.q0 = __ldg(p.cu_new + b);
  const int q1 = __ldg(p.cu_new + b + 1);
  r.len = __ldg(p.kv_len + b);
  if (r.q0 < end || q1 < r.q0 || q1 > p.total_new || q1 - r.q0 > p.max_new || r.len < 0 ||
      (int64_t)r.len > ((int64_t)p.max_pages << p.page_shift)) {
    atomicOr(err, kDevErrBounds);
    return ChunkRow{end, 0, 0};
  }
  r.n = q1 - r.q0;
  return r;
}

// The batch row that owns packed row t, offsets in order: the last b with
// cu[b] <= t (rows of no tokens are passed over), or -1 when t lies at or past
// cu[batch].  (Offsets that are not: some b with cu[b] <= t < cu[b + 1], or -1.)
__device__ __forceinline__ int owner_row(const int32_t* cu, int batch, int t) {
  if (t >= __ldg(cu + batch) || t < __ldg(cu)) return -1;
  int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The pool row of position `pos` of batch row b for kv head 0, in units of
// one head's token: the row of head h is h << page_shift further on.  -1
// (and the error latched) for a page id outside the pool.
__device__ __forceinline__ int64_t pool_row(const PagedBatch& p, int b, int pos, uint32_t* err) {
  const int page = __ldg(p.page_table + (int64_t)b * p.max_pages + (pos >> p.page_shift));
  if ((uint32_t)page >= (uint32_t)p.num_pages) {
    atomicOr(err, kDevErrBounds);
    return -1;
  }
  return (((int64_t)page * p.heads_kv) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((127 + e) << 23); }

// Four E4M3 bytes (lowest first) as two fp16 pairs; exact, NaN stays NaN.
__device__ __forceinline__ uint2 e4m3x4_to_f16(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace dd
