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
// Both are copies, bound by memory.  A unit is the row of one (token, K or V,
// head); D / 8 lanes move it, 16 bytes of bf16 each.  A CTA takes N units per
// lane group, all of their loads in flight at once, and looks its few tokens'
// places up once, in shared memory; appending, the loads do not wait for that.
// Measured, 8 kv heads of 128 (replayed from a graph): an E4M3 append of 76,588
// tokens 103 us, 4.6 TB/s, with instructions issued in 73% of the cycles
// (largest magnitude, scale and codes of every row), a bf16 one 97 us, the rate
// of a copy; 81,986 tokens of a bf16 cache read in 104 us, the rate of a copy,
// of an E4M3 cache in 94 (5.4 TB/s); 4,096 tokens of an E4M3 cache in 5.9 us; one
// token of 32 sequences appended in 2.5 us.
#include <climits>

#include "dd_paged.cuh"

namespace dd {
namespace {

constexpr int kThreads = 256;
// CTAs of the append per SM (64 registers with and without it; an E4M3 append of
// prompts takes 106 us with it and 109.6 without)
constexpr int kBlocks = 4;

// Largest |x| of the 8 bf16 values in v, as bf16 bits (which order like the
// magnitudes they stand for; 0x7f80 and above are infinities and NaN).
__device__ __forceinline__ uint32_t amax_bits(uint4 v) {
  const uint32_t k = 0x7fff7fffu;
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
  return max(m & 0xffffu, m >> 16);
}
// The same of the finite ones.
__device__ __forceinline__ uint32_t amax_finite_bits(uint4 v) {
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
// The largest of the values that the kLanes lanes of a row hold.
template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t a) {
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
  return a;
}

// Scale byte (e + 127) for a largest magnitude given as bf16 bits: a =
// (1 + M/128) 2^(E-127) <= 1.75 2^(8+e), i.e. e = E - 135, one more when
// M > 96.
__device__ __forceinline__ uint32_t scale_byte(uint32_t a) {
  if (a == 0) return 127u;
  const int s = (int)(a >> 7) - 8 + ((a & 127u) > 96u ? 1 : 0);
  return (uint32_t)max(s, 7);
}

// Four values as codes.
__device__ __forceinline__ uint32_t quant4(uint32_t a, uint32_t b, float inv) {
  const float2 f = make_float2(inv, inv);
  return pack_e4m3x4(__fmul2_rn(make_float2(bf16lo(a), bf16hi(a)), f),
                     __fmul2_rn(make_float2(bf16lo(b), bf16hi(b)), f));
}
// Four values of a row with non-finite ones (NaN) or of the largest exponent,
// where codes are bounded by 240: the next, 256, times 2^120 is no longer a
// finite bf16 number.
__device__ __forceinline__ uint32_t quant4_rare(uint32_t a, uint32_t b, float inv, float top) {
  float x[4] = {bf16lo(a) * inv, bf16hi(a) * inv, bf16lo(b) * inv, bf16hi(b) * inv};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    // (the comparison is false for non-finite inputs only)
    x[i] = fabsf(x[i]) <= 448.f ? fminf(fmaxf(x[i], -top), top) : NAN;
  return pack_e4m3x4(make_float2(x[0], x[1]), make_float2(x[2], x[3]));
}

// Where the units of a CTA start, and how a unit falls into (token, K or V,
// head): units of a token are the heads of K, then the heads of V.
template <int D, int N>
struct Units {
  static constexpr int kLanes = D / 8;
  static constexpr int kGroups = kThreads / kLanes;  // units in one pass
  static constexpr int kPer = kGroups * N;           // units of a CTA
  static constexpr int kTokens = kPer / 2 + 1;       // the most tokens they touch
};

// From a unit to the one `units` further on, without a division each.
struct Step {
  int dt, dh, per;
  __device__ __forceinline__ Step(int units, int per) : dt(units / per), dh(units % per), per(per) {}
  __device__ __forceinline__ void operator()(int t, int h, int& t2, int& h2) const {
    const bool over = h + dh >= per;
    t2 = t + dt + (over ? 1 : 0);
    h2 = h + dh - (over ? per : 0);
  }
};

// Pool rows (head 0) of the CTA's tokens, -1 for those without a place: row(b,
// end) is sequence b where the possible ones before it end at `end`, of(t, b, c)
// the place of its packed row t, and `most` the packed rows there may be.
// Returns whether the offsets are in order, which other warps find beside the
// search that trusts they are; if not, place_in_turn finds the places.  (The
// first CTA checks rows without tokens of this call too.  The loops over all
// offsets stay rolled: unrolled, they cost the append a CTA per SM.)
template <typename R, typename F>
__device__ __forceinline__ bool place_tokens(int64_t* rows, int first, int count,
                                             const PagedBatch& p, int most, R&& row, F&& of) {
  bool order = true;
#pragma unroll 1
  for (int b = (int)((threadIdx.x + kThreads - 32) % kThreads); b < p.batch; b += kThreads) {
    order = offsets_fit(p.cu_new, b, most) && order;
    if (blockIdx.x == 0) row(b, 0);
  }
  for (int k = threadIdx.x; k < count; k += kThreads) {
    const int t = first + k;
    const int b = t < p.total_new ? owner_row(p.cu_new, p.batch, t) : -1;
    rows[k] = -1;
    if (b < 0) continue;
    const ChunkRow c = row(b, 0);
    if (t >= c.q0 && t - c.q0 < c.n) rows[k] = of(t, b, c);
  }
  return __syncthreads_and(order);
}
template <typename R, typename F>
__device__ __forceinline__ void place_in_turn(int64_t* rows, int first, int count,
                                              const PagedBatch& p, R&& row, F&& of) {
  for (int k = threadIdx.x; k < count; k += kThreads) {
    const int t = first + k;
    rows[k] = -1;
    ChunkRow c{0, 0, 0};
#pragma unroll 1
    for (int b = 0; b < p.batch && t < p.total_new; ++b) {
      c = row(b, c.q0 + c.n);
      if (t >= c.q0 && t - c.q0 < c.n) rows[k] = of(t, b, c);
    }
  }
  __syncthreads();
}

// The place of packed row t of sequence b.
__device__ __forceinline__ int64_t append_row(const PagedBatch& p, int t, int b, const ChunkRow& c,
                                              uint32_t* err) {
  const int pos = c.len - c.n + (t - c.q0);
  return pos >= 0 ? pool_row(p, b, pos, err) : -1;
}

struct Append {
  const uint16_t *k_new, *v_new;
  int64_t k_stride, v_stride;
  void *k_pool, *v_pool;
  uint8_t *k_scale, *v_scale;
  uint32_t* err;
};

// This lane's 16 bytes of the unit (token, hv), and their way into the pool,
// where the token's head 0 has the row `row` (ok: it has one).  The lanes of a
// warp call the second together.
template <int D>
__device__ __forceinline__ uint4 load_unit(const Append& a, int heads, int tok, int hv, int l) {
  const uint16_t* src = hv < heads ? a.k_new + tok * a.k_stride + hv * D
                                   : a.v_new + tok * a.v_stride + (hv - heads) * D;
  return __ldg(reinterpret_cast<const uint4*>(src) + l);
}
template <int D, bool kF8>
__device__ __forceinline__ void store_unit(const PagedBatch& p, const Append& a, int64_t row,
                                           bool ok, int hv, int l, uint4 v) {
  constexpr int kLanes = D / 8;
  const int H = p.heads_kv;
  const bool is_v = hv >= H;
  row += (int64_t)(is_v ? hv - H : hv) << p.page_shift;
  if constexpr (!kF8) {
    if (ok) reinterpret_cast<uint4*>(is_v ? a.v_pool : a.k_pool)[row * kLanes + l] = v;
  } else {
    uint32_t s = scale_byte(row_max<kLanes>(amax_bits(v)));
    uint2 c;
    // one comparison covers non-finite values and the largest exponent
    if (!__any_sync(0xffffffffu, s >= 247u)) {
      const float inv = pow2f(127 - (int)s);
      c.x = quant4(v.x, v.y, inv);
      c.y = quant4(v.z, v.w, inv);
    } else {
      s = scale_byte(row_max<kLanes>(amax_finite_bits(v)));
      const float inv = pow2f(127 - (int)s), top = s == 247u ? 240.f : 448.f;
      c.x = quant4_rare(v.x, v.y, inv, top);
      c.y = quant4_rare(v.z, v.w, inv, top);
    }
    if (ok) {
      reinterpret_cast<uint2*>(is_v ? a.v_pool : a.k_pool)[row * kLanes + l] = c;
      if (l == 0) (is_v ? a.v_scale : a.k_scale)[row] = (uint8_t)s;
    }
  }
}

// A CTA's units where the offsets are not in order.
template <int D, bool kF8, int N>
__device__ __noinline__ void append_in_turn(const PagedBatch& p, const Append& a, int64_t* rows) {
  using U = Units<D, N>;
  const int H = p.heads_kv, l = threadIdx.x % U::kLanes;
  const int first = blockIdx.x * U::kPer / (2 * H);
  place_in_turn(
      rows, first, min(U::kTokens, (U::kPer - 1) / (2 * H) + 2), p,
      [&](int b, int end) { return chunk_row(p, b, end, a.err); },
      [&](int t, int b, const ChunkRow& c) { return append_row(p, t, b, c, a.err); });
  for (int i = 0; i < N; ++i) {
    const int u = blockIdx.x * U::kPer + threadIdx.x / U::kLanes + i * U::kGroups;
    const int tok = u / (2 * H), hv = u - tok * 2 * H;
    const bool in = tok < p.total_new;
    const uint4 v = in ? load_unit<D>(a, H, tok, hv, l) : make_uint4(0u, 0u, 0u, 0u);
    const int64_t row = in ? rows[tok - first] : -1;
    store_unit<D, kF8>(p, a, row, row >= 0, hv, l, v);
  }
}

template <int D, bool kF8, int N>
__global__ void __launch_bounds__(kThreads, kBlocks)
    cache_append_kernel(const __grid_constant__ PagedBatch p, const __grid_constant__ Append a) {
  using U = Units<D, N>;
  __shared__ int64_t rows[U::kTokens];
  pdl_wait();
  pdl_trigger();
  const int H = p.heads_kv, l = threadIdx.x % U::kLanes;
  const int u0 = blockIdx.x * U::kPer + threadIdx.x / U::kLanes;
  const int first = blockIdx.x * U::kPer / (2 * H);
  const Step step(U::kGroups, 2 * H);
  uint4 v[N];
  int tok[N], hv[N];
  tok[0] = u0 / (2 * H);
  hv[0] = u0 - tok[0] * 2 * H;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i > 0) step(tok[i - 1], hv[i - 1], tok[i], hv[i]);
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tok[i] < p.total_new) v[i] = load_unit<D>(a, H, tok[i], hv[i], l);
  }
  const bool order = place_tokens(
      rows, first, min(U::kTokens, (U::kPer - 1) / (2 * H) + 2), p, p.total_new,
      [&](int b, int end) { return chunk_row(p, b, end, a.err); },
      [&](int t, int b, const ChunkRow& c) { return append_row(p, t, b, c, a.err); });
  if (!order) return append_in_turn<D, kF8, N>(p, a, rows);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = rows[min(tok[i] - first, U::kTokens - 1)];
    store_unit<D, kF8>(p, a, row, row >= 0 && tok[i] < p.total_new, hv[i], l, v[i]);
  }
}

template <int D, bool kF8, int N>
__global__ void __launch_bounds__(kThreads)
    cache_read_kernel(const PagedBatch p, const void* k_pool, const void* v_pool,
                      const uint8_t* __restrict__ k_scale, const uint8_t* __restrict__ v_scale,
                      uint4* __restrict__ k_out, uint4* __restrict__ v_out, uint32_t* err) {
  using U = Units<D, N>;
  __shared__ int64_t rows[U::kTokens];
  pdl_wait();
  pdl_trigger();
  const int H = p.heads_kv, l = threadIdx.x % U::kLanes;
  const int u0 = blockIdx.x * U::kPer + threadIdx.x / U::kLanes;
  const int first = blockIdx.x * U::kPer / (2 * H);
  // (a sequence may go on behind the rows that are asked for)
  const int count = min(U::kTokens, (U::kPer - 1) / (2 * H) + 2);
  auto row = [&](int b, int end) {
    const int q0 = __ldg(p.cu_new + b), q1 = __ldg(p.cu_new + b + 1);
    if (q0 >= end && q1 >= q0) return ChunkRow{q0, q1 - q0, q1 - q0};
    atomicOr(err, kDevErrBounds);
    return ChunkRow{end, 0, 0};
  };
  auto place = [&](int t, int b, const ChunkRow& c) {
    const int pos = t - c.q0;
    if (pos < (p.max_pages << p.page_shift)) return pool_row(p, b, pos, err);
    atomicOr(err, kDevErrBounds);
    return (int64_t)-1;
  };
  if (!place_tokens(rows, first, count, p, INT_MAX, row, place))
    place_in_turn(rows, first, count, p, row, place);
  uint4 v[N];
  uint32_t sc[N];
  int64_t out[N];  // output row, -1: none; complemented for V
  bool ok[N];
  const Step step(U::kGroups, 2 * H);
  int tok = u0 / (2 * H), hv = u0 - tok * 2 * H;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i > 0) step(tok, hv, tok, hv);
    const bool is_v = hv >= H;
    const int h = is_v ? hv - H : hv;
    int64_t row = rows[min(tok - first, U::kTokens - 1)];
    ok[i] = row >= 0 && tok < p.total_new;
    row += (int64_t)h << p.page_shift;
    out[i] = (int64_t)tok * H + h;
    if (is_v) out[i] = ~out[i];
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    sc[i] = 127;
    if (ok[i]) {
      const void* pool = is_v ? v_pool : k_pool;
      if constexpr (kF8) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(pool) + row * U::kLanes + l);
        v[i].x = c.x;
        v[i].y = c.y;
        sc[i] = __ldg((is_v ? v_scale : k_scale) + row);
      } else {
        v[i] = __ldg(reinterpret_cast<const uint4*>(pool) + row * U::kLanes + l);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (kF8) {
      const float f = pow2f((int)sc[i] - 127);
      const float2 ff = make_float2(f, f);
      const uint2 a = e4m3x4_to_f16(v[i].x), b = e4m3x4_to_f16(v[i].y);
      auto pair = [&](uint32_t h) {
        const float2 x = __fmul2_rn(f16x2_to_float2(h), ff);
        return pack_bf16x2(x.x, x.y);
      };
      v[i] = make_uint4(pair(a.x), pair(a.y), pair(b.x), pair(b.y));
    }
    const bool is_v = out[i] < 0;
    if (ok[i]) __stcs((is_v ? v_out : k_out) + (is_v ? ~out[i] : out[i]) * U::kLanes + l, v[i]);
  }
}

// Units per lane group: as many as keep every SM busy.
constexpr int kMany = 8;
template <int D>
bool many_units(int64_t units) {
  return units >= (int64_t)Units<D, kMany>::kPer * 2 * 148;
}

template <int D, bool kF8, int N>
cudaError_t append_t(const CacheAppendArgs& a, int64_t units, cudaStream_t stream) {
  using U = Units<D, N>;
  cudaError_t e = launch_pdl(
      cache_append_kernel<D, kF8, N>, dim3((unsigned)((units + U::kPer - 1) / U::kPer)),
      dim3(kThreads), 0, stream, a.p,
      Append{static_cast<const uint16_t*>(a.k_new), static_cast<const uint16_t*>(a.v_new),
             a.k_stride, a.v_stride, a.pool.k, a.pool.v, a.pool.k_scale, a.pool.v_scale, a.err});
  note_launch();
  return e;
}

template <int D, bool kF8, int N>
cudaError_t read_t(const CacheReadArgs& a, int64_t units, cudaStream_t stream) {
  using U = Units<D, N>;
  cudaError_t e = launch_pdl(
      cache_read_kernel<D, kF8, N>, dim3((unsigned)((units + U::kPer - 1) / U::kPer)),
      dim3(kThreads), 0, stream, a.p, (const void*)a.pool.k, (const void*)a.pool.v,
      (const uint8_t*)a.pool.k_scale, (const uint8_t*)a.pool.v_scale,
      static_cast<uint4*>(a.k_out), static_cast<uint4*>(a.v_out), a.err);
  note_launch();
  return e;
}

template <int D, bool kF8>
cudaError_t append_n(const CacheAppendArgs& a, cudaStream_t stream) {
  const int64_t units = (int64_t)a.p.total_new * 2 * a.p.heads_kv;
  return many_units<D>(units) ? append_t<D, kF8, kMany>(a, units, stream)
                              : append_t<D, kF8, 1>(a, units, stream);
}
template <int D, bool kF8>
cudaError_t read_n(const CacheReadArgs& a, cudaStream_t stream) {
  const int64_t units = (int64_t)a.p.total_new * 2 * a.p.heads_kv;
  return many_units<D>(units) ? read_t<D, kF8, kMany>(a, units, stream)
                              : read_t<D, kF8, 1>(a, units, stream);
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendArgs& a, cudaStream_t stream) {
  if (a.p.head_dim == 64)
    return a.pool.e4m3 ? append_n<64, true>(a, stream) : append_n<64, false>(a, stream);
  return a.pool.e4m3 ? append_n<128, true>(a, stream) : append_n<128, false>(a, stream);
}

cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t stream) {
  if (a.p.head_dim == 64)
    return a.pool.e4m3 ? read_n<64, true>(a, stream) : read_n<64, false>(a, stream);
  return a.pool.e4m3 ? read_n<128, true>(a, stream) : read_n<128, false>(a, stream);
}

}  // namespace dd
