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
// An item that spans CTAs leaves one partial per CTA; at most two of a CTA's
// items are partial, its first and its last.
#pragma once

#include "dd_paged.cuh"

namespace dd {
namespace paged {

constexpr int BN = 128;  // keys per tile

// A partial item that starts in CTA c and ends in CTA `last`: its partials
// are slot 1 of CTA c and slot 0 of CTAs c + 1 .. last.
struct Split {
  int b, g, tp, last;  // b < 0: none starts here
};

struct Params {
  PagedBatch b;
  const uint8_t *k_scale, *v_scale;
  const __nv_bfloat16* q;
  int64_t q_stride;
  int Hq, G, causal, max_ctas;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  Split* split;       // [max_ctas]
  int slot_rows;      // rows kept per slot
  uint32_t* part_o;   // [2 max_ctas][slot_rows][D / 2]: O / l as fp16 pairs times 2^-e_row
  float2* part_lse;   // [2 max_ctas][slot_rows]: log2-domain LSE, 2^e_row
  uint32_t* err;
  uint64_t wait_ns;
  int stall;
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

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
__device__ __forceinline__ int key_tiles(const ChunkRow& r, int G, int causal, int tp) {
  const int last = (min((tp + 1) * kRows, r.n * G) - 1) / G;  // last token of the group
  const int seen = causal ? r.len - r.n + last + 1 : r.len;
  return cdiv(max(seen, 0), BN);
}

// One CTA's part of an item.
struct Seg {
  int b, g, tp;
  ChunkRow r;
  int t0, t1, nt;  // key tiles [t0, t1) of nt
};

// Walks a CTA's share [pos, end) of the items laid end to end.
template <int kRows, int kFixed>
struct Walk {
  int64_t pos, end;
  int b, g, tp, x;  // the item, and the place in it
  ChunkRow r;
  int groups;

  __device__ __forceinline__ void load(const Params& p) {
    r = chunk_row(p.b, b, p.err);
    groups = tile_groups<kRows>(r, p.G);
  }
  __device__ __forceinline__ bool next(const Params& p, Seg& s) {
    while (pos < end) {
      while (groups == 0) {  // a sequence without new tokens
        ++b;
        load(p);
      }
      const int nt = key_tiles<kRows>(r, p.G, p.causal, tp);
      const int w = nt + kFixed;
      const int x1 = (int)min((int64_t)w, x + (end - pos));
      s.b = b;
      s.g = g;
      s.tp = tp;
      s.r = r;
      s.nt = nt;
      s.t0 = max(0, x - kFixed);
      s.t1 = max(0, x1 - kFixed);
      const bool some = s.t1 > s.t0 || (nt == 0 && x == 0);
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

// The share of this CTA: a block-wide prefix sum over the sequences.
struct Share {
  int64_t pos, end, total;
  int ctas, b, g, tp, x;
};

template <int kRows, int kFixed>
__device__ int64_t seq_weight(const Params& p, int b) {
  const ChunkRow r = chunk_row(p.b, b, p.err);
  const int groups = tile_groups<kRows>(r, p.G);
  int64_t w = 0;
  for (int tp = 0; tp < groups; ++tp) w += key_tiles<kRows>(r, p.G, p.causal, tp) + kFixed;
  return w * p.b.heads_kv;
}

template <int kRows, int kFixed, int kT>
__device__ void find_share(const Params& p, Share* sh, int64_t* warp_sums) {
  constexpr int kW = kT / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // exclusive prefix of v over the block; *all gets the block's sum
  auto scan = [&](int64_t v, int64_t* all) {
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int64_t before = 0, sum = 0;
    for (int i = 0; i < kW; ++i) {
      if (i < warp) before += warp_sums[i];
      sum += warp_sums[i];
    }
    __syncthreads();
    *all = sum;
    return before + inc - v;
  };
  int64_t total = 0, w = 0, at = 0, all;
  for (int b0 = 0; b0 < p.b.batch; b0 += kT) {
    const int b = b0 + threadIdx.x;
    w = b < p.b.batch ? seq_weight<kRows, kFixed>(p, b) : 0;
    at = scan(w, &all);
    total += all;
  }
  // no CTA takes less than one item's overhead and as many tiles again
  const int64_t most = (total + 2 * kFixed - 1) / (2 * kFixed);
  const int ctas = (int)min((int64_t)gridDim.x, most);
  const int64_t pos = ctas > 0 && blockIdx.x < ctas ? blockIdx.x * total / ctas : 0;
  const int64_t end = ctas > 0 && blockIdx.x < ctas ? (blockIdx.x + 1) * total / ctas : 0;
  if (threadIdx.x == 0) {
    sh->total = total;
    sh->ctas = ctas;
    sh->pos = pos;
    sh->end = end;
  }
  if (end > pos) {
    int64_t base = 0;
    for (int b0 = 0; b0 < p.b.batch; b0 += kT) {
      const int b = b0 + threadIdx.x;
      if (p.b.batch > kT) {  // (a single round keeps its w and prefix)
        w = b < p.b.batch ? seq_weight<kRows, kFixed>(p, b) : 0;
        at = scan(w, &all);
      }
      if (pos >= base + at && pos < base + at + w) {
        int64_t off = pos - base - at;
        const ChunkRow r = chunk_row(p.b, b, p.err);
        const int64_t head = w / p.b.heads_kv;
        sh->b = b;
        sh->g = (int)(off / head);
        off %= head;
        int tp = 0;
        while (true) {
          const int wi = key_tiles<kRows>(r, p.G, p.causal, tp) + kFixed;
          if (off < wi) break;
          off -= wi;
          ++tp;
        }
        sh->tp = tp;
        sh->x = (int)off;
      }
      base += all;
    }
  }
  __syncthreads();
}

// What the merge needs to know about the item that starts in this CTA's share
// and ends in a later one (one thread).
template <int kRows, int kFixed>
__device__ void write_split(const Params& p, const Share& share) {
  Split s{-1, 0, 0, 0};
  Walk<kRows, kFixed> w;
  w.pos = share.pos;
  w.end = share.end;
  if (w.pos < w.end) {
    w.b = share.b;
    w.g = share.g;
    w.tp = share.tp;
    w.x = share.x;
    w.load(p);
    Seg e;
    while (w.next(p, e))
      if (e.t0 == 0 && e.t1 < e.nt && e.t1 > 0) {
        // its last unit, and the CTA whose share holds it
        const int64_t last = share.end + (e.nt - e.t1) - 1;
        int c = (int)(last * share.ctas / share.total);
        while ((c + 1) * share.total / share.ctas <= last) ++c;
        while (c * share.total / share.ctas > last) --c;
        s = Split{e.b, e.g, e.tp, c};
      }
  }
  p.split[blockIdx.x] = s;
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
  if (w.pos < w.end) w.load(p);
  return w;
}

// Query rows per sequence and kv head up to which the kernel for few rows is
// taken, and its launch (dd_paged_few.cu), which sets p.max_ctas to its 1 or 2
// CTAs per SM.
constexpr int kFewRows = 16;
cudaError_t launch_few(Params& p, const PagedPool& pool, int rows, int sms,
                       cudaStream_t stream);

}  // namespace paged
}  // namespace dd
