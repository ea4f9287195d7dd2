// dd_paged_few.cu -- attention over a paged cache for few query rows: one
// token per sequence, or a few (dd_paged_attn with at most kFewRows packed
// rows per sequence and kv head).
//
// What bounds it is the cache: every key and value is read once and serves
// only a handful of rows, so the products are a small part of the time and
// what counts is bytes in flight (about 45 KB per SM cover the latency at the
// full rate).  A 128-row tensor-core tile would leave one warp with all the
// softmax; here each warp works on its own 16 keys at a time with warp-level
// matrix instructions (m16n8k16, keys as the 16 rows, query rows as the 8
// columns) and its own running softmax, with no barrier in the loop, and the
// warps' results are merged at the end of an item.
//
// No operand passes through shared memory: the order in which the head
// dimension is summed, and the order of output columns, are free, so each lane
// loads 16 consecutive bytes of a row of K or V and uses them as the fragment
// of permuted columns:
//   S^T = K Q^T   lane (g, c) = (lane / 4, lane % 4) holds, of keys g and
//                 g + 8, the 16 bytes at 64 j + 16 c for each 64-byte block j;
//                 Q is loaded in the same order;
//   O^T += V^T W  lane (g, c) holds, of keys 2c, 2c+1, 2c+8, 2c+9, the D / 8
//                 columns from g D / 8 on; byte permutes pair two keys of one
//                 column, the columns 2t and 2t + 1 of the lane being rows g
//                 and g + 8 of the t-th product;
//   W             the softmax weights come out of the first product by key
//                 and enter the second by query row: one 8x8 transpose each.
//
// E4M3 cache: a code is exact in fp16, and the products run on the codes
// themselves, in fp16.  The key's scale 2^ek multiplies its scores.  The
// value's scale 2^ev enters the exponent: with x the log2-domain score, the
// weights are w = 2^(x + ev - n) in O = sum w code, with n a reference that
// follows the maximum of x + ev over the keys whose V is not zero (a row of
// zeros has the scale 2^0, often far above its neighbours', and adds nothing).
// n lies 6 below the maximum when it moves and moves when a weight would pass
// 2^15, so that a weight keeps fp16's 11 bits down to 2^-20 of the largest; what
// a smaller one loses, 2^-25 of its codes at most, is under 2^-30 of what the
// largest adds (as the cache is written, a row's largest code is above 224).
// The softmax's sum is that of 2^(x - m), m the running maximum of x, with
// exponentials of its own: x and x + ev can lie 240 octaves apart, more than
// fp32 holds beside a sum.  The bf16 query is scaled by a power of two per
// row that puts its largest magnitude in [2^14, 2^15); only what lies 2^28
// below it loses bits.
//
// Measured (D = 128, one token per sequence, group of two; replayed from a
// graph): 64 sequences of up to 16,384 tokens, bf16 317 us (6.6 TB/s, the rate of
// a copy), E4M3 194 us (5.5 TB/s; 204 to 208 with other inputs each time;
// expanding the codes and the softmax take the issue slots 43% of the time); one
// sequence of 65,536, bf16 52 us (5.2 TB/s: about 8 us of it are start, merge and
// end).  Two short sequences at D = 64 take 7.1 us, all of it latency: the
// launch, the lengths, the key tiles one after the other.
#include "dd_paged_attn.cuh"

namespace dd {
namespace paged {
namespace {

constexpr int kFixed = 2;  // an item's overhead in key tiles
constexpr int kMinShare = 4;
constexpr float kLazy = 8.0f;
// E4M3 cache: log2 of a weight at the maximum when its reference moves, and of
// the largest that a weight may get
constexpr float kWeight = 6.0f, kMostWeight = 15.0f;

// Warps per CTA and CTAs per SM by what a lane has to keep: 16 keys of data
// (32 registers for 8-bit, 64 for bf16, at D = 128), the output (D / 4 per 8
// query rows) and the query.
template <int D, bool kF8, int NT>
struct Few {
  static constexpr bool kSmall = kF8 ? NT == 1 : NT == 1 && D == 64;
  static constexpr int kWarps = kSmall ? 8 : NT == 1 ? 10 : 8;
  static constexpr int kBlocks = kSmall ? kFewBlocks : 1;
  static constexpr int kRows = 8 * NT;
  // key tiles of an item that a CTA takes whole where there are CTAs enough:
  // two sequences of up to 700 tokens (D = 64) 7.1 us against 8.4 shared out; 16
  // of 512 at D = 128 9.3 against 14.0, of 1,024 13.5 against 18.9 (E4M3: 512
  // 11.3 against 12.7, 768 14.0 against 14.6, but 1,024 16.6 against 15.5)
  static constexpr int kMostWhole = kF8 ? 6 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kLd = D + 4;  // floats per row of the merge area
  static constexpr int kSmem = kWarps * kRows * (kLd + (kF8 ? 3 : 2)) * 4;
};

__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

// C (16 x 8, fp32) += A (16 x 16) B (16 x 8).
template <bool kF16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit elements.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, bool kF8, int NT>
__global__ void __launch_bounds__(Few<D, kF8, NT>::kThreads, Few<D, kF8, NT>::kBlocks)
    paged_few_kernel(const Params p, const uint8_t* __restrict__ k_pool,
                     const uint8_t* __restrict__ v_pool) {
  using F = Few<D, kF8, NT>;
  constexpr int kRow = kF8 ? D : 2 * D;   // bytes of a token's row
  constexpr int kJ = kRow / 64;           // 64-byte blocks of it
  constexpr int kKS = kF8 ? 4 : 2;        // products per block
  constexpr int kMT = D / 16;             // products per 16 keys of V
  constexpr int kVB = kRow / 8;           // bytes of a V row per lane
  extern __shared__ float area[];         // merge area: O, then m and l, and n (8-bit cache)
  __shared__ Share share;
  __shared__ int64_t warp_sums[F::kWarps];
  float* area_m = area + F::kWarps * F::kRows * F::kLd;
  float* area_l = area_m + F::kWarps * F::kRows;
  float* area_n = area_l + F::kWarps * F::kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_trigger();
  find_share<F::kRows, kFixed, kMinShare, F::kMostWhole, F::kThreads>(p, &share, warp_sums);
  auto walk = start_walk<F::kRows, kFixed>(p, share);
  const int shift = p.b.page_shift, in_page = (1 << shift) - 1;
  Seg sg{};
  while (walk.next(p, sg)) {
    const int rows = sg.r.n * p.G;
    const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
    // ---- the query rows nt 8 + g as fragments, and what rows 2c, 2c + 1 need
    uint32_t qf[NT][kJ * kKS * 2];
    float scale[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      const int tok = div_G(p, r);
      const __nv_bfloat16* src = p.q + (int64_t)(sg.r.q0 + min(tok, max(sg.r.n - 1, 0))) * p.q_stride +
                                 (int64_t)(sg.g * p.G + r - tok * p.G) * D;
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        // 16 (8-bit cache) or 8 (bf16 cache) consecutive elements
        constexpr int kE = kF8 ? 2 : 1;
#pragma unroll
        for (int h = 0; h < kE; ++h) {
          const uint4 v = r < rows ? ld16(src + j * (kF8 ? 64 : 32) + c * (kF8 ? 16 : 8) + h * 8)
                                   : make_uint4(0u, 0u, 0u, 0u);
          uint32_t* f = &qf[nt][(j * kE + h) * 4];
          f[0] = v.x;
          f[1] = v.y;
          f[2] = v.z;
          f[3] = v.w;
        }
      }
      float mul = p.scale_log2;
      if constexpr (kF8) {
#pragma unroll
        for (int i = 0; i < kJ * kKS * 2; ++i)
          mx = fmaxf(mx, fmaxf(fabsf(bf16lo(qf[nt][i])), fabsf(bf16hi(qf[nt][i]))));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = row_exponent(mx);
        const float inv = pow2f(-e);
#pragma unroll
        for (int i = 0; i < kJ * kKS * 2; ++i)
          qf[nt][i] = pack_f16x2(bf16lo(qf[nt][i]) * inv, bf16hi(qf[nt][i]) * inv);
        mul *= pow2f(e);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        scale[nt][u] = __shfl_sync(0xffffffffu, mul, (2 * c + u) * 4);
        const int row = nt * 8 + 2 * c + u;
        lim[nt][u] = row >= rows ? 0 : p.causal ? sg.r.len - sg.r.n + div_G(p, row) + 1 : sg.r.len;
      }
    }
    // ---- the keys of this warp: chunks of 16, every kWarps-th of the segment
    float o[NT][kMT][4];
    float m[NT][2], l[NT][2], n[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = n[nt][0] = n[nt][1] = -1e30f;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int t = 0; t < kMT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][t][e] = 0.f;
    }
    const int32_t* table = p.b.page_table + (int64_t)sg.b * p.b.max_pages;
    const int first = sg.t0 * (BN / 16) + warp;
    const int last = min(sg.t1 * (BN / 16), cdiv(sg.r.len, 16));  // chunks end
    // The 8 keys from position 16 i + 8 h on share a page: where they start in
    // the pools, in bytes, and the last of them that exists.  Behind the
    // sequence's end its last key stands in, whose weight is then 0: loads
    // need no condition, and what lies past the end is not read.
    struct Place {
      int64_t at;
      int most;
    };
    const int end8 = (sg.r.len - 1) & ~7;
    auto page_of = [&](int i, int h) { return __ldg(table + (min(i * 16 + h * 8, end8) >> shift)); };
    auto place_of = [&](int i, int h, int page) {
      const int pos = min(i * 16 + h * 8, end8);
      if ((uint32_t)page >= (uint32_t)p.b.num_pages) {
        atomicOr(p.err, kDevErrBounds);
        page = 0;
      }
      const int64_t row = (((int64_t)page * p.b.heads_kv + sg.g) << shift) + (pos & in_page);
      return Place{row, min(7, sg.r.len - 1 - pos)};
    };
    uint4 kd[2][kJ];               // keys g, g + 8
    uint4 vd[4][(kVB + 15) / 16];  // keys 2c, 2c + 1, 2c + 8, 2c + 9
    uint32_t ks[2], vs[2];         // scale bytes of keys g, g + 8
    auto load_k = [&](const Place (&pl)[2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = pl[h].at + min(g, pl[h].most);
        const uint8_t* src = k_pool + row * kRow + c * 16;
#pragma unroll
        for (int j = 0; j < kJ; ++j) kd[h][j] = ld16(src + j * 64);
        if constexpr (kF8) {
          ks[h] = __ldg(p.k_scale + row);
          vs[h] = __ldg(p.v_scale + row);
        }
      }
    };
    auto load_v = [&](const Place (&pl)[2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* src = v_pool + pl[h].at * kRow + g * kVB;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* at = src + min(2 * c + u, pl[h].most) * kRow;
          if constexpr (kVB >= 16) {
#pragma unroll
            for (int e = 0; e < kVB / 16; ++e) vd[2 * h + u][e] = ld16(at + e * 16);
          } else {
            const uint2 x = ld8(at);
            vd[2 * h + u][0] = make_uint4(x.x, x.y, 0u, 0u);
          }
        }
      }
    };
    // page ids are asked for two chunks ahead, keys and values one
    Place place[2];
    int page[2] = {0, 0};
    if (first < last) {
#pragma unroll
      for (int h = 0; h < 2; ++h) place[h] = place_of(first, h, page_of(first, h));
      load_k(place);
      load_v(place);
#pragma unroll
      for (int h = 0; h < 2; ++h) page[h] = page_of(first + F::kWarps, h);
    }
    for (int i = first; i < last; i += F::kWarps) {
      const bool more = i + F::kWarps < last;
      if (more) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          place[h] = place_of(i + F::kWarps, h, page[h]);
          page[h] = page_of(i + 2 * F::kWarps, h);
        }
      }
      // ---- S^T: keys g, g + 8 by query rows 2c, 2c + 1
      float s[NT][4] = {};
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const uint32_t a[4] = {kd[0][j].x, kd[0][j].y, kd[0][j].z, kd[0][j].w};
        const uint32_t b[4] = {kd[1][j].x, kd[1][j].y, kd[1][j].z, kd[1][j].w};
#pragma unroll
        for (int x = 0; x < kKS; ++x) {
          uint32_t a0, a1, a2, a3;
          if constexpr (kF8) {
            const uint2 h0 = e4m3x4_to_f16(a[x]), h1 = e4m3x4_to_f16(b[x]);
            a0 = h0.x;
            a2 = h0.y;
            a1 = h1.x;
            a3 = h1.y;
          } else {
            a0 = a[2 * x];
            a2 = a[2 * x + 1];
            a1 = b[2 * x];
            a3 = b[2 * x + 1];
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t* f = &qf[nt][(j * kKS + x) * 2];
            mma<kF8>(s[nt], a0, a1, a2, a3, f[0], f[1]);
          }
        }
      }
      // 2^ek and ev of keys g, g + 8
      float fk[2], ev[2];
      if constexpr (kF8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          fk[h] = __uint_as_float(ks[h] << 23);
          ev[h] = __uint_as_float(0x4b000000u + vs[h]) - (8388608.f + 127.f);  // 2^23 + byte
        }
      }
      if (more) load_k(place);  // in flight over the rest of this chunk
      // ---- softmax
      uint32_t wf[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e >> 1, u = e & 1;
          const float x = s[nt][e] * (kF8 ? fk[h] * scale[nt][u] : scale[nt][u]);
          s[nt][e] = i * 16 + h * 8 + g < lim[nt][u] ? x : -INFINITY;
          grow |= s[nt][e] > m[nt][u] + kLazy;
          if constexpr (kF8) grow |= s[nt][e] + ev[h] > n[nt][u] + kMostWeight;
        }
      }
      // the references move only when a score passes one by a margin
      if (__any_sync(0xffffffffu, grow)) {
        if constexpr (kF8) {  // keys whose V is zero: weight 0
          uint32_t some = 0;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4& q = vd[u][0];
            if ((q.x | q.y | q.z | q.w) & 0x7f7f7f7fu) some |= 1u << (2 * c + (u & 1) + 4 * (u & 2));
          }
          some = __reduce_or_sync(0xffffffffu, some);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (!(some >> (g + 8 * h) & 1u)) ev[h] = -INFINITY;
        }
        // to the keys' maximum, less `low`; returns the factor
        auto move = [&](float& ref, float a, float b, float low) {
          a = fmaxf(a, b);
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 8));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
          a = fmaxf(ref, a - low);
          const float f = ex2_approx(ref - a);
          ref = a;
          return f;
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float al = move(m[nt][u], s[nt][u], s[nt][2 + u], 0.f);
            l[nt][u] *= al;
            if constexpr (kF8)
              al = move(n[nt][u], s[nt][u] + ev[0], s[nt][2 + u] + ev[1], kWeight);
#pragma unroll
            for (int t = 0; t < kMT; ++t) {
              o[nt][t][u] *= al;
              o[nt][t][2 + u] *= al;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = ex2_approx(s[nt][e] - m[nt][e & 1]);
          l[nt][e & 1] += w[e];
          if constexpr (kF8) w[e] = ex2_approx(s[nt][e] + (ev[e >> 1] - n[nt][e & 1]));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wf[nt][h] = transpose8(kF8 ? pack_f16x2(w[2 * h], w[2 * h + 1])
                                     : pack_bf16x2(w[2 * h], w[2 * h + 1]));
      }
      // ---- O^T
      auto word = [&](int u, int i) {  // 32-bit word i of key u's columns
        const uint4& q = vd[u][i >> 2];
        return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
      };
      if constexpr (kF8) {
#pragma unroll
        for (int t = 0; t < kMT; t += 2) {  // four columns: codes of two keys paired, then expanded
          uint32_t w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) w[u] = word(u, t >> 1);
          const uint2 a = e4m3x4_to_f16(__byte_perm(w[0], w[1], 0x5140));
          const uint2 b = e4m3x4_to_f16(__byte_perm(w[2], w[3], 0x5140));
          const uint2 c2 = e4m3x4_to_f16(__byte_perm(w[0], w[1], 0x7362));
          const uint2 d = e4m3x4_to_f16(__byte_perm(w[2], w[3], 0x7362));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma<kF8>(o[nt][t], a.x, a.y, b.x, b.y, wf[nt][0], wf[nt][1]);
            mma<kF8>(o[nt][t + 1], c2.x, c2.y, d.x, d.y, wf[nt][0], wf[nt][1]);
          }
        }
      } else {
#pragma unroll
        for (int t = 0; t < kMT; ++t) {
          uint32_t w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) w[u] = word(u, t);
          const uint32_t a0 = __byte_perm(w[0], w[1], 0x5410), a1 = __byte_perm(w[0], w[1], 0x7632);
          const uint32_t a2 = __byte_perm(w[2], w[3], 0x5410), a3 = __byte_perm(w[2], w[3], 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma<kF8>(o[nt][t], a0, a1, a2, a3, wf[nt][0], wf[nt][1]);
        }
      }
      if (more) load_v(place);
    }
    // ---- this warp's rows into the merge area
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float v = l[nt][u];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        const int r = warp * F::kRows + nt * 8 + 2 * c + u;
        if (g == 0) {
          area_m[r] = m[nt][u];
          area_l[r] = v;
          if constexpr (kF8) area_n[r] = n[nt][u];
        }
#pragma unroll
        for (int t = 0; t < kMT; ++t)
          *reinterpret_cast<float2*>(area + r * F::kLd + g * (D / 8) + 2 * t) =
              make_float2(o[nt][t][u], o[nt][t][2 + u]);
      }
    __syncthreads();
    // ---- one warp per query row, D / 32 columns per lane
    constexpr int kC = D / 32;
    for (int r = warp; r < min(rows, F::kRows); r += F::kWarps) {
      float top = -1e30f, ntop = -1e30f;
#pragma unroll
      for (int w = 0; w < F::kWarps; ++w) {
        top = fmaxf(top, area_m[w * F::kRows + r]);
        if constexpr (kF8) ntop = fmaxf(ntop, area_n[w * F::kRows + r]);
      }
      float sum = 0.f, acc[kC] = {};
#pragma unroll
      for (int w = 0; w < F::kWarps; ++w) {
        float f = ex2_approx(area_m[w * F::kRows + r] - top);
        sum = fmaf(f, area_l[w * F::kRows + r], sum);
        if constexpr (kF8) f = ex2_approx(area_n[w * F::kRows + r] - ntop);
        const float* src = area + (w * F::kRows + r) * F::kLd + lane * kC;
#pragma unroll
        for (int e = 0; e < kC; ++e) acc[e] = fmaf(f, src[e], acc[e]);
      }
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const float lse = sum > 0.f ? top + __log2f(sum) : -INFINITY;
#pragma unroll
      for (int e = 0; e < kC; ++e) acc[e] *= inv;
      if constexpr (kF8) {  // O is in units of 2^(n - m), which may lie near either end of fp32
        const float half = ex2_approx(0.5f * (ntop - top));
#pragma unroll
        for (int e = 0; e < kC; ++e) acc[e] = acc[e] * half * half;
      }
      if (whole) {
        const int tok = div_G(p, r);
        const int64_t at = (int64_t)(sg.r.q0 + tok) * p.Hq + sg.g * p.G + r - tok * p.G;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * D) + lane * (kC / 2);
#pragma unroll
        for (int e = 0; e < kC / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e], acc[2 * e + 1]);
        if (p.lse && lane == 0) p.lse[at] = lse * 0.6931471805599453f;
      } else {
        float mxa = 0.f;
#pragma unroll
        for (int e = 0; e < kC; ++e) mxa = fmaxf(mxa, fabsf(acc[e]));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) mxa = fmaxf(mxa, __shfl_xor_sync(0xffffffffu, mxa, s));
        const int e2 = row_exponent(mxa);
        const float f = pow2f(-e2);
        const int64_t slot = (2 * (int64_t)blockIdx.x + (sg.t0 > 0 ? 0 : 1)) * p.slot_rows + r;
        uint32_t* dst = p.part_o + slot * (D / 2) + lane * (kC / 2);
#pragma unroll
        for (int e = 0; e < kC / 2; ++e) dst[e] = pack_f16x2(acc[2 * e] * f, acc[2 * e + 1] * f);
        if (lane == 0) p.part_lse[slot] = make_float2(lse, pow2f(e2));
      }
    }
    __syncthreads();
  }
  finish_items<D, F::kRows, kFixed, F::kThreads>(p, share, sg);
}

template <int D, bool kF8, int NT>
cudaError_t launch_t(const Params& p, const PagedPool& pool, int sms, cudaStream_t stream) {
  using F = Few<D, kF8, NT>;
  cudaError_t e = allow_smem<paged_few_kernel<D, kF8, NT>>(F::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_few_kernel<D, kF8, NT>, dim3(F::kBlocks * sms),
                             dim3(F::kThreads), F::kSmem, stream, p,
                             static_cast<const uint8_t*>(pool.k),
                             static_cast<const uint8_t*>(pool.v));
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_few(const Params& p, const PagedPool& pool, int rows, int sms,
                       cudaStream_t stream) {
  const bool two = rows > 8;
  if (p.b.head_dim == 64) {
    if (pool.e4m3)
      return two ? launch_t<64, true, 2>(p, pool, sms, stream) : launch_t<64, true, 1>(p, pool, sms, stream);
    return two ? launch_t<64, false, 2>(p, pool, sms, stream) : launch_t<64, false, 1>(p, pool, sms, stream);
  }
  if (pool.e4m3)
    return two ? launch_t<128, true, 2>(p, pool, sms, stream) : launch_t<128, true, 1>(p, pool, sms, stream);
  return two ? launch_t<128, false, 2>(p, pool, sms, stream) : launch_t<128, false, 1>(p, pool, sms, stream);
}

}  // namespace paged
}  // namespace dd
