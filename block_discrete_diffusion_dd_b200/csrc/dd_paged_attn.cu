// dd_paged_attn.cu -- attention of new tokens over a paged cache
// (dd_paged_attn) on the 5th-generation tensor cores: tcgen05.mma with its
// accumulators in tensor memory, pages gathered by TMA.
//
// Definition: new token i of a sequence with n new tokens and `len` tokens in
// the cache sees the keys j < len - n + i + 1 (causal) or j < len,
//   O = sum_j softmax_j(scale <q, k_j>) v_j,
// zeros (log-sum-exp -inf) where it sees none.  The G = Hq / Hkv query heads
// of a kv head are packed with the new tokens into rows r = i G + h, so that
// one K/V tile serves them all, whatever G is.
//
// Work.  An item is (sequence b, kv head g, kQT query tiles of 128 rows),
// with the 128-key tiles its last row sees.  Lengths are known on the device
// only and differ widely, so the items' tiles are laid end to end, each item
// with kFixed units of overhead in front, and cut into equal shares, one per
// CTA: every CTA finds its own share from the lengths (a block-wide prefix
// sum) and walks it.  One wave, no host plan, and the same code serves one
// token over 65,536 keys and a long chunk.  An item that spans CTAs leaves a
// partial result per CTA (at most two of a CTA's items are partial: its first
// and its last), which a second kernel merges in CTA order.
//
// Inside a CTA:
//   warps 0 .. 8 kQT - 1  softmax.  Each owns 16 query rows through the
//            16-lane tcgen05.ld shape (four threads per row, two shuffles per
//            row reduction), loads them into the Q tile, runs the online
//            softmax in fp32 (base 2; O is rescaled only when the running
//            maximum grows past a margin of 2^8) and writes P back as bf16
//            where S was, for the P.V product.  Warps without valid rows only
//            keep the barriers' count.
//   TMA warp one lane per 8-key group looks the page up; a page's share of the
//            tile is one box of the tensor map.
//   MMA warp issues every MMA from one elected lane, so that the tensor core
//            works ahead of the softmax.  One query tile: two S buffers, used
//            in turn, S(j+2) behind PV(j).  Two query tiles with P in columns
//            of its own (kSep): S_0 and S_1 of a key tile as soon as the
//            softmax has loaded what lay in the buffer, PV_q(j) when its P is
//            written.  Two query tiles with P where S was: PV_0(j) S_0(j+1)
//            PV_1(j) S_1(j+1).
//   convert  (E4M3 cache) expands the 8-bit tiles to bf16 operands: code times
//            2^e, exact in bf16, so that the products see exactly what the
//            cache stands for.  The scale bytes follow the page by cp.async.
// The tensor core runs one thread's MMAs in issue order.  Where P takes S's
// place with two query tiles, S_q(j) complete therefore means PV_q(j-1)
// complete, and O may be rescaled; elsewhere a rescale waits for PV(j-1) on a
// barrier of the P.V products.  A wait tells a phase from its neighbours only
// by parity, so that when it starts, the product before the awaited one on the
// same barrier has to be known complete, and the one behind it not to be
// possible.  The latter needs P of this warp.  The former holds with a barrier
// per query tile where S(j) complete means PV(j-1) complete, or where every
// tile waits for the P.V product before it (kSep); one query tile, where S(j)
// complete means PV(j-2) complete, takes two barriers in turn.
//
// What bounds it (D = 128, 148 CTAs): with 256 query rows the softmax, whose 16
// warps take about 1.4 us per key tile (loads and maximum 0.3, row reductions
// 0.3, exponentials 0.7, stores 0.1) and wait 0.3 us for the tensor core,
// against 1.0 us of tensor-core work: two chunks of 2,048 tokens over 8,192
// take 232 us, or 257 once the power limit holds the clock down (the products
// alone: 135), the tensor pipe being active half of the time.  With an E4M3
// cache the conversion: 1.0 us for K and 0.9 us for V of a tile (blocks of 256
// tokens of eight sequences with up to 16,384 each: 136 us, from bf16 117; the
// two chunks 275, or 290).  (The registers are spent too: with two query tiles
// 96 a thread, or 80, and the kernels spill up to 40 bytes.)  A short past is
// bounded by the chain of single steps: the share's search 2.3 us, the Q tile
// 2.4, the first product 0.8, the epilogue 2.6, and the second kernel 5 to 8
// (one block of 256 over 4,096: 28.3 us).
//
// What the cache holds past a sequence's length may be anything, NaN
// included: masked scores are replaced before they are used, and V rows past
// the length are set to zero in shared memory, since 0 * NaN is NaN.
//
// Every mbarrier wait is bounded in time; on expiry the CTA latches an error,
// drains its copies and MMAs and frees its tensor memory.
#include <algorithm>
#include <type_traits>

#include "dd_paged_attn.cuh"

namespace dd {
namespace {

using namespace paged;

constexpr int BM = 128;  // query rows per tile
constexpr uint32_t kAtom = 128 * 128;  // 128 rows of one 128-byte swizzle atom (64 bf16)
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.0f;          // log2 units
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr int kMaxStages = 6, kMaxRaw = 8;

struct Barriers {
  uint64_t q_full[2];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t mma_final;
  uint64_t never;  // completed by nothing: the target of the test stall
  uint32_t tmem_base;
  int abort;
};

template <int D, bool kF8, int kQT>
struct Lay {
  static constexpr uint32_t kTile = BM * D * 2;  // a bf16 operand tile
  static constexpr uint32_t kRaw = BN * D;       // an E4M3 tile
  // 8-bit caches: with two query tiles one expanded K tile suffices (the next
  // one is expanded while the softmax works), which leaves room for three 8-bit
  // tiles in flight
  static constexpr int kStagesK = D == 64 ? 4 : kF8 ? 3 - kQT : 4 - kQT;
  static constexpr int kStagesV = D == 64 ? 4 : 2;
  static constexpr int kRawStages = !kF8 ? 0 : D == 64 ? 4 : 3;
  static constexpr int kSoftWarps = 8 * kQT;
  static constexpr int kConvWarps = kF8 ? 6 : 0;
  static constexpr int kWarpTMA = kSoftWarps, kWarpMMA = kSoftWarps + 1;
  static constexpr int kThreads = (kSoftWarps + 2 + kConvWarps) * 32;
  static constexpr uint32_t kOffK = kQT * kTile;
  static constexpr uint32_t kOffV = kOffK + kStagesK * kTile;
  static constexpr uint32_t kOffRaw = kOffV + kStagesV * kTile;
  static constexpr uint32_t kOffScale = kOffRaw + kRawStages * kRaw;
  static constexpr uint32_t kOffBar = kOffScale + kRawStages * BN;
  static constexpr uint32_t kSmem = kOffBar + sizeof(Barriers) + 1024;
  // Tensor memory: S buffers, then (two query tiles) P, then O.  With two query
  // tiles P has columns of its own, so that a score buffer is free again as
  // soon as the softmax has loaded it; at D = 128 that leaves one for both.
  // (With an 8-bit cache the softmax loads its scores twice, and holds a single
  // buffer too long: ragged blocks of 8 took 176 us against 137.)
  static constexpr bool kSep = kQT == 2 && (!kF8 || D == 64);
  static constexpr int kSBufs = kSep && D == 128 ? 1 : 2;
  static constexpr uint32_t kTmemP = kSBufs * BN;
  static constexpr uint32_t kTmemO = kTmemP + (kSep ? kQT * BN / 2 : 0);
  static_assert(kTmemO + kQT * D <= kTmemCols, "tensor memory");
  // an item's overhead (its Q tile, first product and epilogue) in key tiles
  static constexpr int kFixed = kQT == 1 ? 2 : 3;
  static constexpr int kMinShare = kFixed;
  static_assert(kStagesK <= kMaxStages && kStagesV <= kMaxStages && kRawStages <= kMaxRaw,
                "barrier arrays");
  static_assert(kSmem + 3 * 1024 <= 227 * 1024, "shared memory budget, static part included");
};

__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t off) {
  return base + (uint64_t)(off >> 4);
}

// S = Q K^T: K-major operands, 16 elements (32 bytes) per MMA through the
// 128-byte swizzle atoms.
template <int D>
__device__ __forceinline__ void issue_s(uint32_t dS, uint64_t aq, uint64_t bk) {
  constexpr uint32_t id = idesc_bf16_f32(BM, BN, 0, 0);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk >> 2) * kAtom + (kk & 3) * 32;
    tc_mma_ss(dS, desc_at(aq, off), desc_at(bk, off), id, kk > 0);
  }
}
// O (+)= P V: P from tensor memory, two keys per column; V MN-major.
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t dO, uint32_t aP, uint64_t bv, bool acc) {
  constexpr uint32_t id = idesc_bf16_f32(BM, D, 0, 1);
#pragma unroll
  for (int kk = 0; kk < BN / 16; ++kk)
    tc_mma_ts(dO, aP + (uint32_t)(kk * 8), desc_at(bv, kk * 16 * 128), id,
              (acc || kk > 0) ? 1u : 0u);
}

// 16 E4M3 codes (16 bytes) times f as bf16.
__device__ __forceinline__ void expand16(uint4 c, float f, uint4& lo, uint4& hi) {
  const float2 ff = make_float2(f, f);
  auto four = [&](uint32_t w, uint32_t& a, uint32_t& b) {
    const uint2 h = e4m3x4_to_f16(w);
    const float2 x = __fmul2_rn(f16x2_to_float2(h.x), ff), y = __fmul2_rn(f16x2_to_float2(h.y), ff);
    a = pack_bf16x2(x.x, x.y);
    b = pack_bf16x2(y.x, y.y);
  };
  four(c.x, lo.x, lo.y);
  four(c.y, lo.z, lo.w);
  four(c.z, hi.x, hi.y);
  four(c.w, hi.z, hi.w);
}

template <int D, bool kF8, int kQT>
__global__ void __launch_bounds__(Lay<D, kF8, kQT>::kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const Params p) {
  using L = Lay<D, kF8, kQT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Share share;
  __shared__ int64_t warp_sums[L::kThreads / 32];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Barriers* bars = reinterpret_cast<Barriers*>(smem + L::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStagesK; ++i) {
      mbar_init(&bars->k_full[i], kF8 ? L::kConvWarps : 1);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < L::kStagesV; ++i) {
      mbar_init(&bars->v_full[i], kF8 ? L::kConvWarps : 1);
      mbar_init(&bars->v_empty[i], 1);
    }
    for (int i = 0; i < L::kRawStages; ++i) {
      mbar_init(&bars->raw_full[i], 1 + BN / 8);  // the pages, and each lane's scale bytes
      mbar_init(&bars->raw_empty[i], L::kConvWarps);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&bars->q_full[q], 8);
      mbar_init(&bars->s_full[q], 1);
      mbar_init(&bars->s_free[q], 8);
      mbar_init(&bars->p_full[q], 8);
      mbar_init(&bars->pv_done[q], 1);
    }
    mbar_init(&bars->mma_final, 1);
    mbar_init(&bars->never, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == L::kWarpMMA) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  find_share<kQT * BM, L::kFixed, L::kMinShare, 0, L::kThreads>(p, &share, warp_sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // Each warp walks the share by itself; the walk's state lies in shared memory,
  // since the softmax has no registers to spare for it.
  __shared__ Walk<kQT * BM, L::kFixed> walks[L::kThreads / 32];
  __shared__ Seg segs[L::kThreads / 32];
  const bool work = share.pos < share.end;
  const Seg& sg = segs[warp];
  if (lane == 0) {
    walks[warp] = start_walk<kQT * BM, L::kFixed>(p, share);
    segs[warp] = Seg{};
  }
  auto next = [&]() {
    bool got = false;
    __syncwarp();
    if (lane == 0) got = walks[warp].next(p, segs[warp]);
    __syncwarp();
    return __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
  };

  if (warp < L::kSoftWarps) {
    // ------------------------------------------------------------ softmax
    const int q = warp >> 3, wl = warp & 3, hv = (warp >> 2) & 1;
    const int t4 = lane & 3;
    const int rbase = wl * 32 + hv * 16;
    const int rA = rbase + (lane >> 2), rB = rA + 8;  // query rows in tile q
    const uint32_t lane_base = (uint32_t)rbase << 16;
    const uint32_t tO = tmem + lane_base + L::kTmemO + (uint32_t)(q * D);
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    constexpr int kChunks = D / 8;  // 16-byte pieces of a row
    uint8_t* tileQ = smem + q * L::kTile;
    int cnt = 0;  // tiles of this query tile
    bool ok = true;
    auto quad_max = [](float v) {
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
      return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
    };
    auto quad_sum = [](float v) {
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      return v + __shfl_xor_sync(0xffffffffu, v, 2);
    };
    // P.V product t of this query tile is complete
    auto wait_pv = [&](int t) {
      const int bar = kQT == 1 ? t & 1 : q, phase = kQT == 1 ? t >> 1 : t;
      const bool done = __all_sync(
          0xffffffffu, mbar_wait_bounded(&bars->pv_done[bar], phase & 1, abort_flag, p.wait_ns));
      tc_fence_after();
      return done;
    };
    while (ok && next()) {
      const int row0 = (sg.tp * kQT + q) * BM;         // packed row of the tile's row 0
      const int rows = sg.r.n * p.G - row0;            // valid rows of this tile
      if (rows <= 0) continue;
      const bool active = rbase < rows;
      const int first_head = sg.g * p.G;
      // global row (token, head) of the tile's row r, in elements of q / out
      auto token = [&](int r, int& head) {
        const int pr = row0 + r, i = div_G(p, pr);
        head = first_head + pr - i * p.G;
        return sg.r.q0 + i;
      };
      if (sg.nt == 0) {  // nothing to see: zeros
        for (int r = rbase + lane / kChunks; r < rbase + 16; r += 32 / kChunks)
          if (r < rows) {
            int h;
            const int64_t at = (int64_t)token(r, h) * p.Hq + h;
            reinterpret_cast<uint4*>(p.out + at * D)[lane % kChunks] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse && lane % kChunks == 0) p.lse[at] = -INFINITY;
          }
        continue;
      }
      if (active) {  // this warp's 16 rows of Q, into the K-major swizzled tile
        uint4 v[16 * kChunks / 32];
#pragma unroll
        for (int i = 0; i < 16 * kChunks / 32; ++i) {
          const int r = rbase + i * (32 / kChunks) + lane / kChunks;
          v[i] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows) {
            int h;
            const int64_t t = token(r, h);
            v[i] = __ldg(reinterpret_cast<const uint4*>(p.q + t * p.q_stride + (int64_t)h * D) +
                         lane % kChunks);
          }
        }
#pragma unroll
        for (int i = 0; i < 16 * kChunks / 32; ++i) {
          const int r = rbase + i * (32 / kChunks) + lane / kChunks, c = lane % kChunks;
          *reinterpret_cast<uint4*>(tileQ + (c >> 3) * kAtom + r * 128 +
                                    (((c & 7) ^ (r & 7)) << 4)) = v[i];
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->q_full[q]);
      // keys seen by rows A and B, and the fewest of the warp's rows
      auto limit = [&](int r) {
        if (r >= rows) return 0;
        const int i = div_G(p, row0 + r);
        return p.causal ? sg.r.len - sg.r.n + i + 1 : sg.r.len;
      };
      const int limA = limit(rA), limB = limit(rB), lim0 = limit(rbase);
      const int full_to = rbase + 16 <= rows ? lim0 : 0;
      float mrefA = -1e30f, mrefB = -1e30f, lA = 0.f, lB = 0.f;
      const int n = sg.t1 - sg.t0;
      for (int j = 0; j < n; ++j, ++cnt) {
        const int buf = kQT == 1 ? cnt & 1 : q;
        const uint32_t par = (kQT == 1 ? cnt >> 1 : cnt) & 1;
        const uint32_t tS = tmem + lane_base + (uint32_t)((L::kSBufs == 1 ? 0 : buf) * BN);
        const uint32_t tP = L::kSep ? tmem + lane_base + L::kTmemP + (uint32_t)(q * (BN / 2)) : tS;
        // wait outcomes are made warp-uniform: tcgen05.ld/st are .sync.aligned
        if (!__all_sync(0xffffffffu,
                        mbar_wait_bounded(&bars->s_full[buf], par, abort_flag, p.wait_ns))) {
          ok = false;
          break;
        }
        if (active) {
          tc_fence_after();
          const int k0 = (sg.t0 + j) * BN;
          // The scores in kH parts of 128 / kH columns: with an 8-bit cache and
          // two query tiles 24 warps leave 80 registers each, and the upper
          // half is loaded twice, first for the maximum, then for P, whose
          // columns by then only overlie scores that are used up.
          constexpr int kH = kF8 && kQT == 2 ? 2 : 1, kI = 16 / kH;
          uint32_t sv[4 * kI];
          auto load = [&](int h) {
            if constexpr (kH == 1) tmem_ld16x256b_x16(tS, sv);
            else tmem_ld16x256b_x8(tS + (uint32_t)(h * 64), sv);
            if (k0 + BN > full_to) {
              const int vA = limA - k0 - h * 64, vB = limB - k0 - h * 64;
#pragma unroll
              for (int i = 0; i < kI; ++i) {
                const int c = 8 * i + 2 * t4;
                if (c >= vA) sv[4 * i] = __float_as_uint(-INFINITY);
                if (c + 1 >= vA) sv[4 * i + 1] = __float_as_uint(-INFINITY);
                if (c >= vB) sv[4 * i + 2] = __float_as_uint(-INFINITY);
                if (c + 1 >= vB) sv[4 * i + 3] = __float_as_uint(-INFINITY);
              }
            }
          };
          auto free_s = [&]() {  // the score buffer may be written again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->s_free[q]);
          };
          float ma = -INFINITY, mb = -INFINITY;
#pragma unroll
          for (int h = kH - 1; h >= 0; --h) {
            load(h);
            if (L::kSep && kH == 1) free_s();
#pragma unroll
            for (int i = 0; i < kI; ++i) {
              ma = fmaxf(ma, fmaxf(__uint_as_float(sv[4 * i]), __uint_as_float(sv[4 * i + 1])));
              mb = fmaxf(mb, fmaxf(__uint_as_float(sv[4 * i + 2]), __uint_as_float(sv[4 * i + 3])));
            }
          }
          const float xa = quad_max(ma) * p.scale_log2, xb = quad_max(mb) * p.scale_log2;
          if (j == 0) {
            // the reference is the row's maximum (a row that sees none of
            // this tile keeps a finite one: its exponentials are 0)
            mrefA = fmaxf(mrefA, xa);
            mrefB = fmaxf(mrefB, xb);
          } else if (__any_sync(0xffffffffu, xa > mrefA + kLazy || xb > mrefB + kLazy)) {
            // rescale (rare, a warp-uniform decision); the last P.V product
            // has to be complete (where P lies in the place of S, and there
            // are two query tiles, it is: S came behind it)
            if ((kQT == 1 || L::kSep) && !wait_pv(cnt - 1)) {
              ok = false;
              break;
            }
            const float na = fmaxf(mrefA, xa), nb = fmaxf(mrefB, xb);
            const float alA = ex2_approx(mrefA - na), alB = ex2_approx(mrefB - nb);
            lA *= alA;
            lB *= alB;
#pragma unroll 1
            for (int c16 = 0; c16 < D / 16; ++c16) {
              uint32_t o[8];
              tmem_ld16x256b_x2(tO + (uint32_t)(c16 * 16), o);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                o[e] = __float_as_uint(__uint_as_float(o[e]) * ((e & 2) ? alB : alA));
              tmem_st16x256b_x2(tO + (uint32_t)(c16 * 16), o);
            }
            mrefA = na;
            mrefB = nb;
          }
          // P has columns of its own: the last P.V product has to have read them
          if (L::kSep && cnt > 0 && !wait_pv(cnt - 1)) {
            ok = false;
            break;
          }
          const float2 na = make_float2(-mrefA, -mrefA), nb = make_float2(-mrefB, -mrefB);
          float2 sa = make_float2(0.f, 0.f), sb = make_float2(0.f, 0.f);
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            if (h > 0) {
              load(h);
              if (L::kSep) free_s();
            }
            uint32_t w[2 * kI];  // 16x128b: w[2i] row A, w[2i + 1] row B, column 4 i + t % 4
#pragma unroll
            for (int i = 0; i < kI; ++i) {
              const float2 da = __ffma2_rn(
                  make_float2(__uint_as_float(sv[4 * i]), __uint_as_float(sv[4 * i + 1])), sl2, na);
              const float2 db = __ffma2_rn(
                  make_float2(__uint_as_float(sv[4 * i + 2]), __uint_as_float(sv[4 * i + 3])), sl2,
                  nb);
              const float2 pa = make_float2(ex2_approx(da.x), ex2_approx(da.y));
              const float2 pb = make_float2(ex2_approx(db.x), ex2_approx(db.y));
              sa = __fadd2_rn(sa, pa);
              sb = __fadd2_rn(sb, pb);
              w[2 * i] = pack_bf16x2(pa.x, pa.y);
              w[2 * i + 1] = pack_bf16x2(pb.x, pb.y);
            }
            if constexpr (kH == 1) tmem_st16x128b_x16(tP, w);
            else tmem_st16x128b_x8(tP + (uint32_t)(h * 32), w);
          }
          lA += sa.x + sa.y;
          lB += sb.x + sb.y;
          tmem_wait_st();
          tc_fence_before();
        } else if (L::kSep) {
          // (an arrival must not run ahead of the other warps' previous one)
          if (lane == 0) mbar_arrive(&bars->s_free[q]);
          if (cnt > 0 && !wait_pv(cnt - 1)) {
            ok = false;
            break;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[buf]);
      }
      if (!ok) break;
      // epilogue: O / l and the log-sum-exp
      if (!wait_pv(cnt - 1)) {
        ok = false;
        break;
      }
      if (!active) continue;
      tc_fence_after();
      const float lrowA = quad_sum(lA), lrowB = quad_sum(lB);
      const float invA = lrowA > 0.f ? 1.f / lrowA : 0.f, invB = lrowB > 0.f ? 1.f / lrowB : 0.f;
      const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (sg.t0 > 0 ? 0 : 1);
      float sA = invA, sB = invB;
      int eA = 0, eB = 0;
      if (!whole) {
        // fp16 pairs, each row scaled by a power of two that puts its largest
        // magnitude in [2^14, 2^15): 11 significant bits against the row's
        // maximum in half the bytes of fp32
        float mA = 0.f, mB = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint32_t o[32];
          tmem_ld16x256b_x8(tO + (uint32_t)(h * 64), o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            mA = fmaxf(mA, fmaxf(fabsf(__uint_as_float(o[4 * i])), fabsf(__uint_as_float(o[4 * i + 1]))));
            mB = fmaxf(mB, fmaxf(fabsf(__uint_as_float(o[4 * i + 2])),
                                 fabsf(__uint_as_float(o[4 * i + 3]))));
          }
        }
        eA = row_exponent(quad_max(mA) * invA);
        eB = row_exponent(quad_max(mB) * invB);
        sA = invA * pow2f(-eA);
        sB = invB * pow2f(-eB);
      }
      // staged in this warp's own rows of the Q tile (whose products are
      // complete), in the Q tile's swizzled layout: a store hits 32 banks
      auto piece = [&](int r, int c) {
        return tileQ + (c >> 3) * kAtom + r * 128 + (((c & 7) ^ (r & 7)) << 4);
      };
      auto put = [&](int r, int i, float x, float y, float s) {
        reinterpret_cast<uint32_t*>(piece(r, i))[t4] =
            whole ? pack_bf16x2(x * s, y * s) : pack_f16x2(x * s, y * s);
      };
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t o[32];
        tmem_ld16x256b_x8(tO + (uint32_t)(h * 64), o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          put(rA, h * 8 + i, __uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), sA);
          put(rB, h * 8 + i, __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]), sB);
        }
      }
      if (t4 == 0) {
        const float lseA = lrowA > 0.f ? mrefA + __log2f(lrowA) : -INFINITY;
        const float lseB = lrowB > 0.f ? mrefB + __log2f(lrowB) : -INFINITY;
        auto put_lse = [&](int r, float l, int e) {
          if (r >= rows) return;
          if (whole) {
            int h;
            const int64_t t = token(r, h);
            if (p.lse) p.lse[t * p.Hq + h] = l * 0.6931471805599453f;
          } else {
            p.part_lse[slot * p.slot_rows + q * BM + r] = make_float2(l, pow2f(e));
          }
        };
        put_lse(rA, lseA, eA);
        put_lse(rB, lseB, eB);
      }
      __syncwarp();
      for (int r = rbase + lane / kChunks; r < rbase + 16; r += 32 / kChunks) {
        if (r >= rows) break;
        const int c = lane % kChunks;
        const uint4 v = *reinterpret_cast<const uint4*>(piece(r, c));
        if (whole) {
          int h;
          const int64_t t = token(r, h);
          reinterpret_cast<uint4*>(p.out + (t * p.Hq + h) * D)[c] = v;
        } else {
          reinterpret_cast<uint4*>(p.part_o + (slot * p.slot_rows + q * BM + r) * (D / 2))[c] = v;
        }
      }
      __syncwarp();
    }
  } else {
    if (warp == L::kWarpTMA) {
      // ------------------------------------------------------------ TMA
      // Lane l < 16 looks up the page of the tile's 8-key group l, and issues
      // the copy where that group starts a page (or the tile).
      int tile = 0;  // tiles issued
      const int ps = 1 << p.b.page_shift, per = min(ps, BN);
      if (lane == 0 && work) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
      }
      bool ok = true;
      while (ok && next()) {
        const int32_t* table = p.b.page_table + (int64_t)sg.b * p.b.max_pages;
        auto look = [&](int t) {
          const int pos = t * BN + lane * 8;
          return lane < BN / 8 && t < sg.t1 && pos < sg.r.len
                     ? __ldg(table + (pos >> p.b.page_shift)) : -1;
        };
        int page = look(sg.t0);
        for (int t = sg.t0; t < sg.t1 && ok; ++t, ++tile) {
          const int after = look(t + 1);
          const int pos = t * BN + lane * 8;
          const bool live = lane < BN / 8 && pos < sg.r.len;
          int at = page;
          if (live && (uint32_t)page >= (uint32_t)p.b.num_pages) {
            atomicOr(p.err, kDevErrBounds);
            at = p.b.num_pages;  // outside the tensor map: read as zero
          }
          const bool lead = live && (lane * 8) % per == 0;
          const uint32_t bytes =
              (uint32_t)__popc(__ballot_sync(0xffffffffu, lead)) * per * D * (kF8 ? 1 : 2);
          const int c1 = pos & (ps - 1) & ~(per - 1), c2 = at * p.b.heads_kv + sg.g;
          for (int v = 0; v < 2 && ok; ++v) {
            const CUtensorMap* map = v ? &tmV : &tmK;
            uint64_t *full, *empty;
            uint8_t* dst;
            int round;
            if constexpr (kF8) {
              const int n = 2 * tile + v, st = n % L::kRawStages;
              round = n / L::kRawStages;
              full = &bars->raw_full[st];
              empty = &bars->raw_empty[st];
              dst = smem + L::kOffRaw + st * L::kRaw;
            } else {
              const int stages = v ? L::kStagesV : L::kStagesK, st = tile % stages;
              round = tile / stages;
              full = v ? &bars->v_full[st] : &bars->k_full[st];
              empty = v ? &bars->v_empty[st] : &bars->k_empty[st];
              dst = smem + (v ? L::kOffV : L::kOffK) + st * L::kTile;
            }
            if (round > 0)
              ok = __all_sync(0xffffffffu,
                              mbar_wait_bounded(empty, (round - 1) & 1, abort_flag, p.wait_ns));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(full, bytes);
            __syncwarp();
            if constexpr (kF8) {
              if (lead) tma_load_3d(dst + lane * 8 * D, map, full, 0, c1, c2);
              if (lane < BN / 8) {
                if (live && at == page) {
                  const int64_t row = ((int64_t)c2 << p.b.page_shift) + (pos & (ps - 1));
                  uint8_t* sc = smem + L::kOffScale + ((2 * tile + v) % L::kRawStages) * BN;
                  cp_async8(sc + lane * 8, (v ? p.v_scale : p.k_scale) + row);
                }
                cp_async_arrive(full);
              }
            } else if (lead) {
#pragma unroll
              for (int a = 0; a < D / 64; ++a)
                tma_load_3d(dst + a * kAtom + lane * 8 * 128, map, full, a * 64, c1, c2);
            }
            __syncwarp();
          }
          page = after;
        }
      }
      if (lane == 0) write_split<L::kFixed>(p, share, sg);
      // copies still in flight must land before the CTA exits (all have, unless
      // the CTA gave up: then the last tiles' barriers are waited for, those of
      // copies that were not issued any more running out)
      if (*abort_flag) {
        for (int n = max(0, tile - kMaxStages); n <= tile; ++n)
          for (int v = 0; v < 2; ++v) {
            const int i = 2 * n + v;
            uint64_t* full = kF8 ? &bars->raw_full[i % max(1, L::kRawStages)]
                             : v ? &bars->v_full[n % L::kStagesV] : &bars->k_full[n % L::kStagesK];
            const int round = kF8 ? i / max(1, L::kRawStages) : n / (v ? L::kStagesV : L::kStagesK);
            mbar_wait_bounded(full, round & 1, nullptr, kDrainNs / 64);
          }
      }
      __syncwarp();
    } else if (warp == L::kWarpMMA) {
      // ------------------------------------------------------------ MMA
      const bool leader = elect_one_sync();
      const uint64_t dQ = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dK = smem_desc_sw128(smem_u32(smem + L::kOffK), 16, 1024);
      const uint64_t dV = smem_desc_sw128(smem_u32(smem + L::kOffV), kAtom, 1024);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool r = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, p.wait_ns));
        tc_fence_after();
        return r;
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) tc_commit(bar);
        __syncwarp();
      };
      int kt = 0, vt = 0;            // K and V tiles consumed
      int cnt[2] = {0, 0};           // tiles of the query tiles (kQT = 1: of the S buffers)
      int segs[2] = {0, 0};          // segments per query tile
      int sbuf = 0, pbuf = 0;        // kQT = 1: the next S / P buffer
      bool ok = true, first = true;
      auto wait_k = [&](int t) { return wait(&bars->k_full[t % L::kStagesK], (t / L::kStagesK) & 1); };
      auto s_product = [&](int q, int buf, int t, uint64_t* full) {
        if (leader) {
          issue_s<D>(tmem + buf * BN, desc_at(dQ, q * L::kTile),
                     desc_at(dK, t % L::kStagesK * L::kTile));
          tc_commit(full);
        }
        __syncwarp();
      };
      while (ok && next()) {
        const int n = sg.t1 - sg.t0;
        if (n == 0) continue;
        const int rows = sg.r.n * p.G - sg.tp * kQT * BM;
        const int nq = kQT == 1 ? 1 : min(kQT, cdiv(rows, BM));
        for (int q = 0; q < nq && ok; ++q) ok = wait(&bars->q_full[q], segs[q]++ & 1);
        // S of the segment's tile j for query tile q.  A shared S buffer is
        // waited for until the other query tile has loaded it, an own one
        // until this one has (one query tile: P has taken its place, and the
        // P.V product issued before has read it).
        auto s_of = [&](int q, int j) {
          const int t = kt + j;
          if (q == 0 && !wait_k(t)) return false;
          if constexpr (kQT == 1) {
            s_product(0, sbuf, t, &bars->s_full[sbuf]);
            sbuf ^= 1;
          } else {
            constexpr bool kOne = L::kSBufs == 1;
            if (L::kSep) {
              // tile j of q = 0 comes after tile j - 1 of q = 1, tile j of
              // q = 1 after tile j of q = 0
              const int o = kOne && nq == 2 ? 1 - q : q;
              const int past = kOne && nq == 2 && q == 1 ? j : j - 1;
              if (past >= 0 && !wait(&bars->s_free[o], (cnt[o] + past) & 1)) return false;
            }
            s_product(q, kOne ? 0 : q, t, &bars->s_full[q]);
          }
          if (q == nq - 1) commit(&bars->k_empty[t % L::kStagesK]);
          return true;
        };
        ok = ok && s_of(0, 0);
        if (kQT == 1) ok = ok && (n == 1 || s_of(0, 1));
        else ok = ok && (nq == 1 || s_of(1, 0));
        if (ok && first && p.stall) ok = wait(&bars->never, 0);
        first = false;
        for (int j = 0; j < n && ok; ++j) {
          // separate P: the next S of a query tile goes ahead of its P.V
          if (L::kSep && j + 1 < n && !(ok = s_of(0, j + 1))) break;
          const int vst = vt % L::kStagesV;
          if (!(ok = wait(&bars->v_full[vst], (vt / L::kStagesV) & 1))) break;
          if constexpr (!kF8) {
            // V rows past the sequence's length: zero, whatever the page holds
            const int valid = sg.r.len - (sg.t0 + j) * BN;
            if (valid < BN) {
              uint8_t* v = smem + L::kOffV + vst * L::kTile;
              for (int i = lane; i < (BN - valid) * 8; i += 32)
#pragma unroll
                for (int a = 0; a < D / 64; ++a)
                  *reinterpret_cast<uint4*>(v + a * kAtom + valid * 128 + i * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          const uint64_t bv = desc_at(dV, vst * L::kTile);
          for (int q = 0; q < nq && ok; ++q) {
            if (L::kSep && q == 1 && j + 1 < n && !(ok = s_of(1, j + 1))) break;
            const int buf = kQT == 1 ? pbuf : q;
            const uint32_t par = kQT == 1 ? cnt[buf]++ : cnt[q] + j;
            if (!(ok = wait(&bars->p_full[buf], par & 1))) break;
            const uint32_t aP = L::kSep ? L::kTmemP + q * (BN / 2) : buf * BN;
            if (leader) issue_pv<D>(tmem + L::kTmemO + q * D, tmem + aP, bv, j > 0);
            __syncwarp();
            commit(&bars->pv_done[buf]);  // (one query tile: two in turn, as P's buffers)
            // P in the place of S: the next S has to come behind its P.V
            if (!L::kSep && kQT == 2 && j + 1 < n) ok = s_of(q, j + 1);
          }
          if (!ok) break;
          pbuf ^= 1;
          commit(&bars->v_empty[vst]);
          ++vt;
          if (kQT == 1 && j + 2 < n) ok = s_of(0, j + 2);
        }
        if (!ok) break;
        kt += n;
        if (kQT == 2)
          for (int q = 0; q < nq; ++q) cnt[q] += n;
      }
      // every MMA issued above has completed before TMEM is released
      commit(&bars->mma_final);
      mbar_wait_bounded(&bars->mma_final, 0, nullptr, kDrainNs);
      __syncwarp();
    } else if constexpr (kF8) {
      // ------------------------------------------------------------ convert
      // A group of 8 lanes takes two rows, four 16-byte pieces of each; the
      // rows are paired (r, r ^ 5) at D = 128 and (r, r + 1) at D = 64 so that
      // both the reads of the 8-bit tile and the writes of the bf16 tile, each
      // swizzled by its row, touch every bank once.
      const int cw = warp - L::kWarpMMA - 1;
      const int oct = lane >> 3, sel = (lane >> 2) & 1, kk = lane & 3;
      const int sub = D == 128 ? (sel ? oct ^ 5 : oct) : 2 * oct + sel;  // row in its group of 8
      int tile = 0;
      bool ok = true;
      while (ok && next()) {
        for (int t = sg.t0; t < sg.t1 && ok; ++t, ++tile) {
          const int valid = sg.r.len - t * BN;
          for (int v = 0; v < 2; ++v) {
            const int stages = v ? L::kStagesV : L::kStagesK;
            const int n = 2 * tile + v, rs = n % L::kRawStages, st = tile % stages;
            uint64_t* empty = v ? &bars->v_empty[st] : &bars->k_empty[st];
            uint64_t* full = v ? &bars->v_full[st] : &bars->k_full[st];
            ok = mbar_wait_bounded(&bars->raw_full[rs], (n / L::kRawStages) & 1, abort_flag,
                                   p.wait_ns);
            if (ok && tile >= stages)
              ok = mbar_wait_bounded(empty, (tile / stages - 1) & 1, abort_flag, p.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint8_t* raw = smem + L::kOffRaw + rs * L::kRaw;
            const uint8_t* sc = smem + L::kOffScale + rs * BN;
            uint8_t* dst = smem + (v ? L::kOffV : L::kOffK) + st * L::kTile;
#pragma unroll 2
            for (int grp = cw; grp < BN / 8; grp += L::kConvWarps) {
              const int r = grp * 8 + sub;
              const float f = pow2f((int)sc[r] - 127);
#pragma unroll
              for (int half = 0; half < D / 64; ++half) {
                const int c = kk + 4 * half;
                const uint8_t* src = D == 128 ? raw + r * 128 + ((c ^ sub) << 4) : raw + r * 64 + (c << 4);
                uint4 lo, hi;
                expand16(*reinterpret_cast<const uint4*>(src), f, lo, hi);
                if (r >= valid) lo = hi = make_uint4(0u, 0u, 0u, 0u);
                uint8_t* d = dst + half * kAtom + r * 128;
                *reinterpret_cast<uint4*>(d + (((2 * kk) ^ sub) << 4)) = lo;
                *reinterpret_cast<uint4*>(d + (((2 * kk + 1) ^ sub) << 4)) = hi;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bars->raw_empty[rs]);
              mbar_arrive(full);
            }
          }
        }
      }
    }
  }

  if (*abort_flag && threadIdx.x == 0) atomicOr(p.err, kDevErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == L::kWarpMMA) tmem_dealloc(tmem, kTmemCols);
}

// Block (c, part): kMergeRows rows of the item that starts in CTA c and ends
// in another.
constexpr int kMergeWarps = 8, kMergeRows = 16;

template <int D, int kRows>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(const Params p) {
  pdl_wait();
  pdl_trigger();
  const int parts = cdiv(p.slot_rows, kMergeRows);
  const int c = blockIdx.x / parts, begin = blockIdx.x % parts * kMergeRows;
  const Split s = p.split[c];
  if (s.b >= 0)
    merge_rows<D, kRows, kMergeWarps>(p, s, begin, begin + kMergeRows, threadIdx.x >> 5);
}

// ----------------------------------------------------------------- host
// The pool as [pages * heads, page_size, D]: a box is one head's share of a
// page, or 128 rows of it, 64 bf16 columns (one swizzle atom) or a whole
// E4M3 row wide.  E4M3 tiles of 128-byte rows are swizzled as well, for the
// conversion's reads.
bool encode_pages(CUtensorMap* m, const void* base, const PagedBatch& p, bool f8) {
  const int64_t es = f8 ? 1 : 2, ps = (int64_t)1 << p.page_shift;
  const int64_t dims[3] = {p.head_dim, ps, (int64_t)p.num_pages * p.heads_kv};
  const int64_t strides[2] = {p.head_dim * es, ps * p.head_dim * es};
  const int box[3] = {f8 ? p.head_dim : 64, (int)std::min<int64_t>(ps, BN), 1};
  return encode_3d(m, base, f8, dims, strides, box, !f8 || p.head_dim == 128);
}

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = 148;
  }
  return n;
}

// Query rows that one sequence can have at most; more than one tile of them
// takes the two-tile kernel (each key tile then serves 256 rows).
int64_t max_rows(const PagedAttnArgs& a) {
  return (int64_t)std::min(a.p.max_new, a.p.total_new) * (a.heads_q / a.p.heads_kv);
}

template <int D, bool kF8, int kQT>
cudaError_t launch_t(const CUtensorMap& mk, const CUtensorMap& mv, const Params& p, int sms,
                     cudaStream_t stream) {
  using L = Lay<D, kF8, kQT>;
  cudaError_t e = allow_smem<paged_attn_kernel<D, kF8, kQT>>((int)L::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_attn_kernel<D, kF8, kQT>, dim3(sms), dim3(L::kThreads), L::kSmem,
                             stream, mk, mv, p);
  note_launch();
  return e;
}

template <int D, int kRows>
cudaError_t launch_merge(const Params& p, int sms, cudaStream_t stream) {
  const int parts = (p.slot_rows + kMergeRows - 1) / kMergeRows;
  cudaError_t e = launch_pdl(paged_merge_kernel<D, kRows>, dim3(sms * parts),
                             dim3(kMergeWarps * 32), 0, stream, p);
  note_launch();
  return e;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

size_t paged_attn_scratch_bytes(const PagedAttnArgs& a) {
  const size_t ctas = kFewBlocks * num_sms();
  const size_t rows = (size_t)std::min<int64_t>(max_rows(a), 2 * BM);
  return align256(ctas * sizeof(Split)) + align256(2 * ctas * rows * sizeof(float2)) +
         2 * ctas * rows * a.p.head_dim * 2;
}

// Up to kFewRows query rows per sequence and kv head, the kernel for few rows
// (dd_paged_few.cu).  Measured against the tensor-core kernel, D = 128, groups
// of two, 64 sequences of up to 16,384 tokens: E4M3, one token each 194 us
// against 423, eight tokens (16 rows) 325 against 426; bf16 317 against 397 and
// 346 against 414.  One sequence of 65,536: bf16 52 against 58 us (16 rows: 56
// against 62), E4M3 37 against 67 (58 against 70).
// Above that and up to one tile of rows the tensor-core kernel with one query
// tile: eight sequences, 32 and 128 rows, bf16 48 and 51 us against 52 and 55
// with the other, E4M3 55 and 60 against 60 and 67.  More rows: two query
// tiles, so that a key tile is fetched (and expanded) once for 256 rows.
// (The host knows the bound max_new, not the lengths: in a batch of single tokens
// and one chunk, or under a loose bound, the single tokens take the kernel of the
// longest.  63 of them beside a chunk of 2,048 tokens: E4M3 630 us, bf16 503, of
// which the single tokens alone, with their own bound, would be 180 and 296.)
cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  const bool f8 = a.pool.e4m3;
  const int D = a.p.head_dim;
  const int64_t rows = max_rows(a);  // (none: the lengths are checked all the same)
  const int sms = num_sms();
  Params p{};
  p.b = a.p;
  p.k_scale = a.pool.k_scale;
  p.v_scale = a.pool.v_scale;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.Hq = a.heads_q;
  p.G = a.heads_q / a.p.heads_kv;
  p.causal = a.causal ? 1 : 0;
  p.inv_G = (uint32_t)((0x100000000ull + p.G - 1) / p.G);  // (unused where G = 1)
  p.arrived = a.arrived;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.slot_rows = (int)std::min<int64_t>(rows, 2 * BM);
  uint8_t* s = static_cast<uint8_t*>(a.scratch);
  p.split = reinterpret_cast<Split*>(s);
  s += align256((size_t)kFewBlocks * sms * sizeof(Split));
  p.part_lse = reinterpret_cast<float2*>(s);
  s += align256((size_t)2 * kFewBlocks * sms * p.slot_rows * sizeof(float2));
  p.part_o = reinterpret_cast<uint32_t*>(s);
  p.err = a.err;
  p.wait_ns = pipeline_wait_ns();
  p.stall = pipeline_test_stall() ? 1 : 0;
  if (rows <= kFewRows) return launch_few(p, a.pool, (int)rows, sms, stream);
  CUtensorMap mk, mv;
  if (!encode_pages(&mk, a.pool.k, a.p, f8) || !encode_pages(&mv, a.pool.v, a.p, f8))
    return cudaErrorInvalidValue;
  const bool two = rows > BM;
  auto go = [&](auto d, auto e4m3) {
    constexpr int kD = decltype(d)::value;
    constexpr bool k8 = decltype(e4m3)::value;
    const cudaError_t e = two ? launch_t<kD, k8, 2>(mk, mv, p, sms, stream)
                              : launch_t<kD, k8, 1>(mk, mv, p, sms, stream);
    if (e != cudaSuccess) return e;
    return two ? launch_merge<kD, 2 * BM>(p, sms, stream) : launch_merge<kD, BM>(p, sms, stream);
  };
  using std::integral_constant;
  using D64 = integral_constant<int, 64>;
  using D128 = integral_constant<int, 128>;
  if (D == 64) return f8 ? go(D64{}, std::true_type{}) : go(D64{}, std::false_type{});
  return f8 ? go(D128{}, std::true_type{}) : go(D128{}, std::false_type{});
}

}  // namespace dd
