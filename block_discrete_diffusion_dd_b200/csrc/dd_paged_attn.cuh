// dd_paged_attn.cuh -- what the kernels of the attention over a paged cache
// share: their parameters, the cut of the work into one share per CTA, and
// the form in which partial results are handed to the merge.
//
// An item is (sequence b, kv head g, group of kRows packed query rows) with
// the 128-key tiles that its last row sees.  Lengths are known on the device
// only and differ widely, so the items are laid end to end, each with kFixed
// units of overhead in front of its tiles, and cut into equal shares, one per
// CTA: every CTA finds its own share from the lengths (a block-wide prefix
// sum) and walks it.  One wave and no host plan, whatever the lengths are.
// (Few rows, short sequences and CTAs enough: an item each.)
// An item that spans CTAs leaves one partial per CTA; at most two of a CTA's
// items are partial, its first (slot 0) and its last (slot 1).  Partials are
// merged in CTA order, whoever does it: with many rows per item a second
// kernel, with few the CTA that delivers an item's last partial.
#pragma once

#include "dd_paged.cuh"

namespace dd {
namespace paged {

constexpr int BN = 128;  // keys per tile

template <int v>
struct Int {
  static constexpr int value = v;
};

struct Params {
  PagedBatch b;
  const uint8_t *k_scale, *v_scale;
  const __nv_bfloat16* q;
  int64_t q_stride;
  int Hq, G, causal;
  uint32_t inv_G;     // ceil(2^32 / G)
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  struct Split* split;  // [CTAs]: the item that starts there and ends elsewhere (merge kernel)
  uint32_t* arrived;    // [CTAs]: partials of that item (few rows); zero between calls
  int slot_rows;      // rows kept per slot
  uint32_t* part_o;   // [2 CTAs][slot_rows][D / 2]: O / l as fp16 pairs times 2^-e_row
  float2* part_lse;   // [2 CTAs][slot_rows]: log2-domain LSE, 2^e_row
  uint32_t* err;
  uint64_t wait_ns;
  int stall;
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// x / G for 0 <= x < 2^31: the product with the rounded-up reciprocal is at
// most one too large.
__device__ __forceinline__ int div_G(const Params& p, int x) {
  if (p.G == 1) return x;
  const int q = (int)__umulhi((uint32_t)x, p.inv_G);
  return q * p.G > x ? q - 1 : q;
}
__device__ __forceinline__ uint64_t div64(uint64_t a, uint32_t b) {
  return (a >> 32) == 0 ? (uint32_t)a / b : a / b;
}

__device__ __forceinline__ int row_exponent(float m) {
  if (!(m > 0.f) || !(m <= 3.4e38f)) return 0;
  return min(113, max(-126, ilogbf(m) - 14));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Query-tile groups of a sequence, and the key tiles of group tp.
template <int kRows>
__device__ __forceinline__ int tile_groups(const ChunkRow& r, int G) {
  return cdiv(r.n * G, kRows);
}
template <int kRows>
__device__ __forceinline__ int key_tiles(const Params& p, const ChunkRow& r, int tp) {
  const int last = div_G(p, min((tp + 1) * kRows, r.n * p.G) - 1);  // last token of the group
  const int seen = p.causal ? r.len - r.n + last + 1 : r.len;
  return cdiv(max(seen, 0), BN);
}

// One CTA's part of an item.
struct Seg {
  int b, g, tp;
  ChunkRow r;
  int t0, t1, nt;  // key tiles [t0, t1) of nt
  int64_t begin;   // the item's first unit
};

// Walks a CTA's share [pos, end) of the items laid end to end.
template <int kRows, int kFixed>
struct Walk {
  int64_t pos, end;
  int b, g, tp, x;  // the item, and the place in it
  ChunkRow r;       // of sequence b
  int groups;

  __device__ __forceinline__ void load(const Params& p) {
    r = chunk_row(p.b, b, r.q0 + r.n, p.err);
    groups = tile_groups<kRows>(r, p.G);
  }
  __device__ __forceinline__ bool next(const Params& p, Seg& s) {
    while (pos < end) {
      while (groups == 0) {  // a sequence without new tokens
        ++b;
        load(p);
      }
      const int nt = key_tiles<kRows>(p, r, tp);
      const int w = nt + kFixed;
      const int x1 = (int)min((int64_t)w, x + (end - pos));
      const int t0 = max(0, x - kFixed), t1 = max(0, x1 - kFixed);
      const bool some = t1 > t0 || (nt == 0 && x == 0);
      if (some) {
        s.b = b;
        s.g = g;
        s.tp = tp;
        s.r = r;
        s.nt = nt;
        s.t0 = t0;
        s.t1 = t1;
        s.begin = pos - x;
      }
      pos += x1 - x;
      x = x1;
      if (x == w) {
        x = 0;
        if (++tp == groups) {
          tp = 0;
          if (++g == p.b.heads_kv) {
            g = 0;
            ++b;
            if (pos < end) load(p);
          }
        }
      }
      if (some) return true;
    }
    return false;
  }
};

// One partial item: its partials are slot 1 of CTA `first` and slot 0 of the
// CTAs first + 1 .. last.
struct Split {
  int b, g, tp, first, last;
  ChunkRow r;
};

// The share of this CTA, [pos, end) of `total` units, and where it starts:
// place x of item (b, g, tp).
struct Share {
  int64_t pos, end, total;
  int ctas, b, g, tp, x;
  int64_t quota;  // units of a CTA: quota + 1 for the first `extra` CTAs, quota for the others
  int extra;
  ChunkRow r;     // of sequence b
  Split split[2]; // items to merge (b < 0: none)
};

__device__ __forceinline__ int64_t share_begin(const Share& s, int c) {
  return s.quota * c + min(c, s.extra);
}
// The CTA whose share holds unit u.
__device__ __forceinline__ int owner(const Share& s, int64_t u) {
  const int64_t big = (s.quota + 1) * s.extra;
  return u < big ? (int)div64(u, (uint32_t)(s.quota + 1))
                 : s.extra + (int)div64(u - big, (uint32_t)s.quota);
}

template <int kRows, int kFixed>
__device__ __forceinline__ int64_t row_weight(const Params& p, const ChunkRow& r) {
  const int groups = tile_groups<kRows>(r, p.G);
  int64_t w = 0;
  for (int tp = 0; tp < groups; ++tp) w += key_tiles<kRows>(p, r, tp) + kFixed;
  return w;
}

// kMin: the least share of a CTA.  kMost > 0 (few rows: one group per sequence
// and head): where there are no more items than CTAs and none has more than
// kMost key tiles, CTA c takes item c whole, so that nothing is searched for
// and nothing has to be merged.
template <int kRows, int kFixed, int kMin, int kMost, int kT>
__device__ void find_share(const Params& p, Share* sh, int64_t* warp_sums) {
  constexpr int kW = kT / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool narrow = p.b.batch <= 32;  // one warp's work
  if (!narrow || warp == 0) {
  // every row's offsets are possible by themselves (a round of rows that is the
  // only one finds that out as it is weighed)
  bool order = true;
  if (p.b.batch > kT) {
    for (int b = threadIdx.x; b < p.b.batch; b += kT)
      order = offsets_fit(p.b.cu_new, b, p.b.total_new) && order;
    order = __syncthreads_and(order);
  }
  bool many = false;  // an item of more than kMost tiles (one barrier serves this too)
  int item = 0;       // units of an item of this thread's sequence
  // exclusive prefix of v over the block; *all gets the block's sum
  auto scan = [&](int64_t v, int64_t* all) {
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (narrow) {
      many = __any_sync(0xffffffffu, many);
      *all = __shfl_sync(0xffffffffu, inc, 31);
      return inc - v;
    }
    if (lane == 31) warp_sums[warp] = inc;
    if constexpr (kMost > 0) many = __syncthreads_or(many);
    else __syncthreads();
    int64_t before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const int64_t x = warp_sums[i];
      if (i < warp) before += x;
      sum += x;
    }
    *all = sum;
    return before + inc - v;
  };
  int64_t total = 0, w = 0, at = 0, all = 0;
  ChunkRow r{0, 0, 0};
  auto weigh = [&](int b0) {
    const int b = b0 + threadIdx.x;
    w = 0;
    if (b < p.b.batch) r = chunk_row(p.b, b, 0, p.err);
    if (p.b.batch <= kT) {
      const bool fits = b >= p.b.batch || offsets_fit(p.b.cu_new, b, p.b.total_new);
      order = narrow ? __all_sync(0xffffffffu, fits) : __syncthreads_and(fits);
    }
    if (b < p.b.batch) {
      if (!order) {
        r = ChunkRow{0, 0, 0};
#pragma unroll 1
        for (int a = 0; a <= b; ++a) r = chunk_row(p.b, a, r.q0 + r.n, p.err);
      }
      w = row_weight<kRows, kFixed>(p, r);
      many = w > kMost + kFixed;
      item = (int)w;
      w *= p.b.heads_kv;
    }
    at = scan(w, &all);
  };
  for (int b0 = 0; b0 < p.b.batch; b0 += kT) {
    if (b0 > 0) __syncthreads();  // warp_sums is read
    weigh(b0);
    total += all;
  }
  // the sequence whose item this CTA takes whole, or -1
  const int whole = kMost > 0 && !many && p.b.batch <= kT &&
                            (int64_t)p.b.batch * p.b.heads_kv <= gridDim.x
                        ? (int)blockIdx.x / p.b.heads_kv
                        : -1;
  const int ctas = whole >= 0 ? 0 : (int)min((int64_t)gridDim.x, (total + kMin - 1) / kMin);
  Share s{};
  if (ctas > 0) {
    s.quota = (int64_t)div64(total, (uint32_t)ctas);
    s.extra = (int)(total - s.quota * ctas);
    if ((int)blockIdx.x < ctas) {
      s.pos = share_begin(s, blockIdx.x);
      s.end = share_begin(s, blockIdx.x + 1);
    }
  }
  s.total = total;
  s.ctas = ctas;
  if (kMost > 0 && whole >= 0 && whole < p.b.batch) {
    if ((int)threadIdx.x == whole) {
      s.end = item;
      s.b = whole;
      s.g = (int)blockIdx.x - whole * p.b.heads_kv;
      s.r = r;
      *sh = s;
    }
    s.end = 0;
  } else if (threadIdx.x == 0 && s.end == s.pos) {
    *sh = s;
  }
  if (s.end > s.pos) {
    int64_t base = 0;
    for (int b0 = 0; b0 < p.b.batch; b0 += kT) {
      if (p.b.batch > kT) {  // (a single round keeps its weights)
        __syncthreads();
        weigh(b0);
      }
      if (s.pos >= base + at && s.pos < base + at + w) {
        uint64_t off = (uint64_t)(s.pos - base - at);
        const uint64_t head = div64((uint64_t)w, (uint32_t)p.b.heads_kv);
        s.b = b0 + threadIdx.x;
        s.g = (int)((off >> 32) == 0 && (head >> 32) == 0 ? (uint32_t)off / (uint32_t)head
                                                          : off / head);
        off -= head * s.g;
        while (true) {
          const int wi = key_tiles<kRows>(p, r, s.tp) + kFixed;
          if ((int64_t)off < wi) break;
          off -= wi;
          ++s.tp;
        }
        s.x = (int)off;
        s.r = r;
        *sh = s;
      }
      base += all;
    }
  }
  }
  __syncthreads();
}

// A walk over the share.
template <int kRows, int kFixed>
__device__ __forceinline__ Walk<kRows, kFixed> start_walk(const Params& p, const Share& share) {
  Walk<kRows, kFixed> w;
  w.pos = share.pos;
  w.end = share.end;
  w.b = share.b;
  w.g = share.g;
  w.tp = share.tp;
  w.x = share.x;
  w.r = share.r;
  w.groups = tile_groups<kRows>(share.r, p.G);
  return w;
}

// Merges rows [begin, end) of a partial item: lse = log2 sum 2^lse_s, O =
// sum_s 2^(lse_s - lse) 2^e_s O_s.  A warp takes every kWarps-th row: lane s
// holds the weight of split s, lane l the columns (D / 32) l ..; sixteen split
// rows are requested before the first is needed (of one query row, or of two
// where there are up to eight splits), since the latency of the requests is
// what a merge spends its time on.
template <int D, int kRows, int kWarps>
__device__ void merge_rows(const Params& p, const Split& s, int begin, int end, int warp) {
  constexpr int kC = D / 64;  // fp16 pairs per lane
  const int lane = threadIdx.x & 31;
  const int row0 = s.tp * kRows, rows = min(min(s.r.n * p.G - row0, end), p.slot_rows);
  const int ns = s.last - s.first + 1;
  auto at = [&](int k, int row) {  // the row of split k
    return (int64_t)(k == 0 ? 2 * s.first + 1 : 2 * (s.first + k)) * p.slot_rows + row;
  };
  auto fetch = [&](int k, int row, uint32_t (&x)[kC]) {
    const uint32_t* src = p.part_o + at(k, row) * (D / 2) + lane * kC;
    if constexpr (kC == 2) {
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(src));
      x[0] = v.x;
      x[1] = v.y;
    } else {
      x[0] = __ldcg(src);
    }
  };
  auto add = [&](float w, const uint32_t (&x)[kC], float (&acc)[2 * kC]) {
#pragma unroll
    for (int e = 0; e < kC; ++e) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&x[e]));
      acc[2 * e] = fmaf(w, v.x, acc[2 * e]);
      acc[2 * e + 1] = fmaf(w, v.y, acc[2 * e + 1]);
    }
  };
  auto store = [&](int row, float ref, float wsum, const float (&acc)[2 * kC]) {
    const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
    const int pr = row0 + row, tok = div_G(p, pr);
    const int64_t orow = (int64_t)(s.r.q0 + tok) * p.Hq + s.g * p.G + pr - tok * p.G;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D) + lane * kC;
#pragma unroll
    for (int e = 0; e < kC; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (p.lse && lane == 0)
      p.lse[orow] = wsum > 0.f ? (ref + __log2f(wsum)) * 0.6931471805599453f : -INFINITY;
  };
  // kI query rows of up to kK splits at once
  auto batch = [&](auto ki, auto kk) {
    constexpr int kI = decltype(ki)::value, kK = decltype(kk)::value;
    for (int r0 = begin + warp; r0 < rows; r0 += kI * kWarps) {
      float2 ls[kI];
      uint32_t x[kI][kK][kC];
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        const int row = r0 + i * kWarps;
        ls[i] = row < rows && lane < ns ? __ldcg(&p.part_lse[at(lane, row)])
                                        : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int k = 0; k < kK; ++k) {
#pragma unroll
          for (int e = 0; e < kC; ++e) x[i][k][e] = 0;
          if (row < rows && k < ns) fetch(k, row, x[i][k]);
        }
      }
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        const int row = r0 + i * kWarps;
        if (row >= rows) break;
        float mx = ls[i].x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float ref = fmaxf(mx, -1e30f);
        const float w = exp2f(ls[i].x - ref), wo = w * ls[i].y;
        float wsum = w, acc[2 * kC] = {};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
#pragma unroll
        for (int k = 0; k < kK; ++k) add(__shfl_sync(0xffffffffu, wo, k), x[i][k], acc);
        store(row, ref, wsum, acc);
      }
    }
  };
  if (ns <= 8) return batch(Int<2>{}, Int<8>{});
  if (ns <= 16) return batch(Int<1>{}, Int<16>{});
  for (int row = begin + warp; row < rows; row += kWarps) {
    float mx = -INFINITY;
    for (int k = lane; k < ns; k += 32) mx = fmaxf(mx, __ldcg(&p.part_lse[at(k, row)]).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float ref = fmaxf(mx, -1e30f);
    float wsum = 0.f, acc[2 * kC] = {};
    for (int k0 = 0; k0 < ns; k0 += 32) {
      const int k = k0 + lane;
      const float2 ls = k < ns ? __ldcg(&p.part_lse[at(k, row)]) : make_float2(-INFINITY, 0.f);
      const float w = exp2f(ls.x - ref), wo = w * ls.y;
      wsum += w;
      const int n = min(32, ns - k0);
      for (int j0 = 0; j0 < n; j0 += 8) {
        uint32_t x[8][kC];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
#pragma unroll
          for (int e = 0; e < kC; ++e) x[u][e] = 0;
          if (j0 + u < n) fetch(k0 + j0 + u, row, x[u]);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) add(__shfl_sync(0xffffffffu, wo, j0 + u), x[u], acc);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
    store(row, ref, wsum, acc);
  }
}

// The item that the last segment `e` of a share starts and does not finish,
// for the merge kernel (one thread, also where the share is empty).
template <int kFixed>
__device__ __forceinline__ void write_split(const Params& p, const Share& share, const Seg& e) {
  Split s{-1, 0, 0, 0, 0, {0, 0, 0}};
  if (share.pos < share.end && e.t0 == 0 && e.t1 > 0 && e.t1 < e.nt)
    s = Split{e.b, e.g, e.tp, (int)blockIdx.x, owner(share, e.begin + kFixed + e.nt - 1), e.r};
  p.split[blockIdx.x] = s;
}

// The end of a CTA of the kernel for few rows, whose last segment is `e`: its
// partials are counted on the CTAs where their items start, and the items
// that are complete now are merged.  Every thread calls it, after its last
// write of a partial.
template <int D, int kRows, int kFixed, int kT>
__device__ __forceinline__ void finish_items(const Params& p, Share& share, const Seg& e) {
  __syncthreads();
  if (share.pos == share.end) return;
  if (share.x <= kFixed && !(e.t0 == 0 && e.t1 > 0 && e.t1 < e.nt)) return;  // whole items only
  if (threadIdx.x == 0) {
    __threadfence();
    // the item the share starts in, with tiles before it and some in it; and
    // the last one, with its first tile and not its last
    const int nt = key_tiles<kRows>(p, share.r, share.tp);
    const bool first = share.x > kFixed && share.x < nt + kFixed;
    const bool last = e.t0 == 0 && e.t1 > 0 && e.t1 < e.nt;
    Split s[2];
    if (first) {
      const int64_t begin = share.pos - share.x + kFixed;
      s[0] = Split{share.b, share.g, share.tp, owner(share, begin), owner(share, begin + nt - 1),
                   share.r};
    }
    if (last)
      s[1] = Split{e.b, e.g, e.tp, (int)blockIdx.x, owner(share, e.begin + kFixed + e.nt - 1), e.r};
    const uint32_t n0 = first ? atomicAdd(&p.arrived[s[0].first], 1u) : 0;
    const uint32_t n1 = last ? atomicAdd(&p.arrived[blockIdx.x], 1u) : 0;
    if (!first || n0 != (uint32_t)(s[0].last - s[0].first)) s[0].b = -1;
    else p.arrived[s[0].first] = 0;  // for the next call
    if (!last || n1 != (uint32_t)(s[1].last - s[1].first)) s[1].b = -1;
    else p.arrived[blockIdx.x] = 0;
    share.split[0] = s[0];
    share.split[1] = s[1];
    __threadfence();
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < 2; ++i)
    if (share.split[i].b >= 0)
      merge_rows<D, kRows, kT / 32>(p, share.split[i], 0, kRows, threadIdx.x >> 5);
}

// Query rows per sequence and kv head up to which the kernel for few rows is
// taken, and its launch (dd_paged_few.cu; up to kFewBlocks CTAs per SM).
constexpr int kFewRows = 16;
constexpr int kFewBlocks = 2;
cudaError_t launch_few(const Params& p, const PagedPool& pool, int rows, int sms,
                       cudaStream_t stream);

}  // namespace paged
}  // namespace dd
