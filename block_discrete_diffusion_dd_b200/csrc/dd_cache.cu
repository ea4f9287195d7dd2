// dd_cache.cu -- the paged K/V cache: writing the K and V of new tokens into
// it (dd_cache_append) and laying it out as the packed prefix that the canvas
// attention takes (dd_cache_read).
//
// Layout: K and V [num_pages, heads_kv, page_size, D], so that one head's
// share of a page is contiguous (page_size * D elements: what a head's
// attention fetches as one box).  An E4M3 cache has one scale byte per
// (token, head) in [num_pages, heads_kv, page_size]: byte s stands for
// 2^(s - 127).
//
// Quantisation of the D values x of one (token, head): with a the largest
// finite |x|, e is the least integer with a <= 448 2^e (448: the largest
// finite E4M3 value), kept within [-120, 120], and 0 when a = 0; the codes
// are E4M3(x 2^-e), rounded to nearest even among those whose product with
// 2^e is a finite bf16 number.  A power of two costs an E4M3
// code no precision (its significand is 4 bits at any scale) and makes the
// product code * 2^e exact in bf16 (exponents down to 2^-129 are bf16
// subnormals, still exact), so reading back adds no rounding of its own, and
// a scale per token means that a later token never changes an earlier one.
// bf16's own exponent and mantissa bits give e without any floating-point
// rounding.  E4M3 has no infinities: non-finite values are stored as NaN.
//
// Both are copies, bound by memory: a group of D / 8 lanes moves one (token,
// head) row of K or V, 16 bytes of bf16 per lane.
#include "dd_paged.cuh"

namespace dd {
namespace {

constexpr int kThreads = 256;

// Largest finite |x| of the 8 bf16 values in v, as bf16 bits.
__device__ __forceinline__ uint32_t amax_bits(uint4 v) {
  uint32_t m = 0;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    if (lo < 0x7f80u) m = max(m, lo);
    if (hi < 0x7f80u) m = max(m, hi);
  }
  return m;
}

// Scale byte (e + 127) for a largest magnitude given as bf16 bits: a =
// (1 + M/128) 2^(E-127) <= 1.75 2^(8+e), i.e. e = E - 135, one more when
// M > 96.
__device__ __forceinline__ uint32_t scale_byte(uint32_t a) {
  if (a == 0) return 127u;
  const int s = (int)(a >> 7) - 8 + ((a & 127u) > 96u ? 1 : 0);
  return (uint32_t)max(s, 7);
}

// Four values as codes; `top` bounds their magnitudes (448, but 240 at the
// largest exponent, 120, where the next code, 256, times 2^120 is no longer
// a finite bf16 number).
__device__ __forceinline__ uint32_t quant4(uint32_t a, uint32_t b, float inv, float top) {
  float x[4] = {bf16lo(a) * inv, bf16hi(a) * inv, bf16lo(b) * inv, bf16hi(b) * inv};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    // (the comparison is false for non-finite inputs only)
    x[i] = fabsf(x[i]) <= 448.f ? fminf(fmaxf(x[i], -top), top) : NAN;
  return pack_e4m3x4(make_float2(x[0], x[1]), make_float2(x[2], x[3]));
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kThreads)
    cache_append_kernel(const PagedBatch p, const uint16_t* __restrict__ k_new,
                        const uint16_t* __restrict__ v_new, int64_t k_stride, int64_t v_stride,
                        void* k_pool, void* v_pool, uint8_t* k_scale, uint8_t* v_scale,
                        uint32_t* err) {
  constexpr int kLanes = D / 8;
  pdl_wait();
  pdl_trigger();
  const int unit = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int l = threadIdx.x % kLanes;
  const int t = unit / (2 * p.heads_kv), hv = unit % (2 * p.heads_kv);
  const int h = hv >> 1;
  int64_t row = -1;
  if (t < p.total_new) {
    const int b = owner_row(p.cu_new, p.batch, t);
    if (b >= 0) {
      const ChunkRow c = chunk_row(p, b, err);
      const int pos = c.len - c.n + (t - c.q0);
      // (a row taken as empty has no position for its tokens)
      if (t - c.q0 < c.n && pos >= 0) row = pool_row(p, b, pos, err);
    }
  }
  const bool ok = row >= 0;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (ok) {
    const uint16_t* src = (hv & 1) ? v_new + t * v_stride : k_new + t * k_stride;
    v = *reinterpret_cast<const uint4*>(src + h * D + l * 8);
    row += (int64_t)h << p.page_shift;
  }
  if constexpr (!kF8) {
    if (ok) reinterpret_cast<uint4*>((hv & 1) ? v_pool : k_pool)[row * kLanes + l] = v;
  } else {
    uint32_t a = amax_bits(v);
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1)
      a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
    const uint32_t s = scale_byte(a);
    const float inv = pow2f(127 - (int)s), top = s == 247u ? 240.f : 448.f;
    if (ok) {
      uint2 c;
      c.x = quant4(v.x, v.y, inv, top);
      c.y = quant4(v.z, v.w, inv, top);
      reinterpret_cast<uint2*>((hv & 1) ? v_pool : k_pool)[row * kLanes + l] = c;
      if (l == 0) ((hv & 1) ? v_scale : k_scale)[row] = (uint8_t)s;
    }
  }
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kThreads)
    cache_read_kernel(const PagedBatch p, const void* k_pool, const void* v_pool,
                      const uint8_t* __restrict__ k_scale, const uint8_t* __restrict__ v_scale,
                      uint4* __restrict__ k_out, uint4* __restrict__ v_out, uint32_t* err) {
  constexpr int kLanes = D / 8;
  pdl_wait();
  pdl_trigger();
  const int unit = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int l = threadIdx.x % kLanes;
  const int t = unit / (2 * p.heads_kv), hv = unit % (2 * p.heads_kv);
  const int h = hv >> 1;
  if (t >= p.total_new) return;
  const int b = owner_row(p.cu_new, p.batch, t);
  if (b < 0) return;
  const int pos = t - __ldg(p.cu_new + b);
  if (pos >= (p.max_pages << p.page_shift)) {
    atomicOr(err, kDevErrBounds);
    return;
  }
  int64_t row = pool_row(p, b, pos, err);
  if (row < 0) return;
  row += (int64_t)h << p.page_shift;
  uint4 o;
  if constexpr (!kF8) {
    o = reinterpret_cast<const uint4*>((hv & 1) ? v_pool : k_pool)[row * kLanes + l];
  } else {
    const uint2 c = reinterpret_cast<const uint2*>((hv & 1) ? v_pool : k_pool)[row * kLanes + l];
    const float f = pow2f((int)((hv & 1) ? v_scale : k_scale)[row] - 127);
    const float2 x0 = e4m3x2_to_float2(c.x), x1 = e4m3x2_to_float2(c.x >> 16);
    const float2 x2 = e4m3x2_to_float2(c.y), x3 = e4m3x2_to_float2(c.y >> 16);
    o = make_uint4(pack_bf16x2(x0.x * f, x0.y * f), pack_bf16x2(x1.x * f, x1.y * f),
                   pack_bf16x2(x2.x * f, x2.y * f), pack_bf16x2(x3.x * f, x3.y * f));
  }
  ((hv & 1) ? v_out : k_out)[((int64_t)t * p.heads_kv + h) * kLanes + l] = o;
}

template <int D, bool kF8>
cudaError_t append_t(const CacheAppendArgs& a, cudaStream_t stream) {
  const int64_t units = (int64_t)a.p.total_new * 2 * a.p.heads_kv;
  const int per = kThreads / (D / 8);
  cudaError_t e = launch_pdl(cache_append_kernel<D, kF8>, dim3((unsigned)((units + per - 1) / per)),
                             dim3(kThreads), 0, stream, a.p,
                             static_cast<const uint16_t*>(a.k_new),
                             static_cast<const uint16_t*>(a.v_new), a.k_stride, a.v_stride,
                             a.pool.k, a.pool.v, a.pool.k_scale, a.pool.v_scale, a.err);
  note_launch();
  return e;
}

template <int D, bool kF8>
cudaError_t read_t(const CacheReadArgs& a, cudaStream_t stream) {
  const int64_t units = (int64_t)a.p.total_new * 2 * a.p.heads_kv;
  const int per = kThreads / (D / 8);
  cudaError_t e = launch_pdl(cache_read_kernel<D, kF8>, dim3((unsigned)((units + per - 1) / per)),
                             dim3(kThreads), 0, stream, a.p, (const void*)a.pool.k,
                             (const void*)a.pool.v, (const uint8_t*)a.pool.k_scale,
                             (const uint8_t*)a.pool.v_scale, static_cast<uint4*>(a.k_out),
                             static_cast<uint4*>(a.v_out), a.err);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendArgs& a, cudaStream_t stream) {
  if (a.p.head_dim == 64)
    return a.pool.e4m3 ? append_t<64, true>(a, stream) : append_t<64, false>(a, stream);
  return a.pool.e4m3 ? append_t<128, true>(a, stream) : append_t<128, false>(a, stream);
}

cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t stream) {
  if (a.p.head_dim == 64)
    return a.pool.e4m3 ? read_t<64, true>(a, stream) : read_t<64, false>(a, stream);
  return a.pool.e4m3 ? read_t<128, true>(a, stream) : read_t<128, false>(a, stream);
}

}  // namespace dd
