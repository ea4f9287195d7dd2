// dd_verify.cu -- verification of drafted tokens against the target's
// probabilities (dd_verify_draft).
//
// Sequence b drafted tokens x_0 .. x_{k-1}, x_i with probability `conf_i`
// from q_i = softmax(draft_i / tau_d); the target gives p_i = softmax(
// target_i / tau), i = 0 .. k.  x_i is accepted while u_i conf_i < p_i(x_i),
// for given uniform numbers u in [0, 1); with n the accepted ones, the next
// token is drawn from the weights w = max(p_n - q_n, 0) (n < k) or w = p_k
// (n = k) by inverting their running sum at u_s: the least v whose running
// sum exceeds u_s W.  Accepted tokens and the next one are then distributed
// as the target's own samples.
//
// Three kernels:
//   scan    one read of all the target's rows: per chunk of 1,024 16-byte
//           blocks a reference r and the sum of 2^(x c - r), c = log2(e) / tau,
//           in fp32.  Bound by memory, with the exponentials close behind (one
//           per entry: 23 us of MUFU time against 30 us of HBM time for 390
//           bf16 rows of 262,144).  The chunk that finishes a row merges its
//           chunks, forms p(x_i) and tests it.  A test within kNear of equality
//           is left open.  kNear covers what p(x_i) may be off by: c is within
//           2^-24 of itself, which moves log2 p(x_i) by 2^-24 |log2 p(x_i) + H|,
//           H the row's entropy in bits, hence p by 1.2e-5 at 2^-298, the least
//           that u_i conf_i (fp32 factors) can be; a lane adds up to 128 terms
//           (7.6e-6), its warp and the row's chunks 14 more (0.8e-6); a sum is
//           scaled up to eight times (2.4e-6); exponents are rounded by 2^-24 of
//           themselves, twice (5e-6 where they count: H <= 30, a reference up to
//           32 above the maximum), exponentials by 2^-22, three times (0.7e-6).
//           In all 3e-5.
//   norm    finds the first refusal, repeating open tests with 64-bit sums over
//           their rows, so that the decision is the one exact arithmetic takes;
//           then, for the one row the next token is drawn at, the 64-bit sums of
//           the target's and the draft's exponentials per chunk of
//           logits.  The running sum has a border per vocabulary entry (up
//           to 262,144 of them), and a relative error of e in the weights
//           moves each border by about e: with fp32 sums one draw in ten to
//           a hundred would land on another token, with 64 bits none does.
//   pick    the weights' sums per chunk; the last chunk to finish finds the
//           chunk that holds u_s W and walks it.
// The last two are latency: each thread asks for all it needs at once, and a
// phase is one or two barriers.  Sums are taken in a fixed order, so a call's
// result does not depend on scheduling.
//
// Measured, bf16, 262,144 entries: eight sequences with 358 drafted tokens 65.5
// us (fp32 89), of which the scan 40 (4.8 TB/s; instructions issued in 59% of
// the cycles) and norm and pick 25; one sequence with eight drafted tokens 18.5
// us (fp32 20.3), nearly all of it the chain of the three kernels.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "dd_paged.cuh"

namespace dd {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 4;               // 16-byte blocks of a thread of the scan
constexpr int kScanBlocks = 5;           // CTAs of the scan per SM (48 registers)
// entries of a thread of norm and pick (kPer): 8, or 4 where that makes few
// chunks (launch_verify_t)
constexpr int kFew = 4, kMany = 8;
constexpr double kNear = 4e-5;
// Scaled logits up to which a row's fp32 reference is good enough: a step of
// 2^28 is 32, which fp32 exponentials have room for.  Rows beyond it (a mask of
// the type's lowest value that leaves nothing, say) are summed in 64 bits, by a
// warp each.
constexpr float kWide = 268435456.f;

// What `norm` hands on about sequence b's draw.
struct Draw {
  int t_row;   // target row
  int d_row;   // draft row, or -1: draw from the target's own distribution
  int out;     // index of the next token in `tokens`, or -1: no draw
  int arrived; // chunks of `pick` done
};
struct Part {  // one chunk of one row, exponentials relative to its maximum
  double s;
  float m;
  int pad;
};

struct VerifyParams {
  const void *target, *draft;
  int batch, total, vocab;
  int64_t target_stride, draft_stride;
  double c, cd;       // log2(e) / tau
  const int32_t* draft_tokens;
  const float* draft_conf;
  const int32_t* cu;
  const float *u_accept, *u_sample;
  int32_t *accepted, *tokens;
  float* target_prob;
  float2* scan;       // [total + batch][segments]: reference, sum
  uint32_t* arrived;  // [kPagedCounters]: chunks done of the rows = i mod their number
  float* ref;         // [total + batch]: the rows' references
  int* owner;         // [total + batch]: the sequence a row is of (if any is)
  uint8_t* state;     // [total]: 0 accepted, 1 refused, 2 near
  Draw* draw;         // [batch]
  Part* part;         // [batch][2][pick chunks]
  double* weight;     // [batch][pick chunks]
  uint32_t* err;
};

template <typename T>
__device__ __forceinline__ float logit(const T* p, int64_t i) {
  if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)__ldg(p + i) << 16);
  else return __uint_as_float(__ldg(p + i));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Block-wide maxima of two values, or sums of two, in every thread (the sums
// in a fixed order).  `sm` is not reused before the next barrier.
struct Pair {
  double x, y;
};
__device__ __forceinline__ float2 block_max2(float x, float y, float2* sm) {
  x = warp_max(x);
  y = warp_max(y);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = make_float2(x, y);
  __syncthreads();
  float2 r = sm[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) r = make_float2(fmaxf(r.x, sm[i].x), fmaxf(r.y, sm[i].y));
  return r;
}
__device__ __forceinline__ Pair block_sum2(double x, double y, Pair* sm) {
  x = warp_sum(x);
  y = warp_sum(y);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = Pair{x, y};
  __syncthreads();
  Pair r{0, 0};
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    r.x += sm[i].x;
    r.y += sm[i].y;
  }
  return r;
}

// A maximum that exponents may be taken against: rows (chunks) of -inf only
// get a finite one, against which every term is 0.
__device__ __forceinline__ float safe_max(float m) { return fmaxf(m, -FLT_MAX); }

// Entries of a 16-byte block as floats.
template <typename T>
__device__ __forceinline__ void unpack(uint4 v, float (&x)[16 / sizeof(T)]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}

// The largest entry of some blocks: packed comparisons for bf16.
template <typename T>
__device__ __forceinline__ float blocks_max(const uint4 (&v)[kBlocks]) {
  if constexpr (sizeof(T) == 2) {
    auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    __nv_bfloat162 m = h(v[0].x);
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
      m = __hmax2(m, __hmax2(__hmax2(h(v[i].x), h(v[i].y)), __hmax2(h(v[i].z), h(v[i].w))));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
      m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y))),
                fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w)));
    return m;
  }
}

// p of the entry x1 of one row in 64 bits throughout (one warp; not inlined, so
// that the scan stays at 48 registers: at 62 a call takes 1.5 to 2.5 us more).
template <typename T>
__device__ __noinline__ double wide_prob(const T* x, int vocab, double c, float x1) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int v = lane; v < vocab; v += 32) m = fmaxf(m, logit(x, v));
  m = safe_max(warp_max(m));
  double s = 0;
  for (int v = lane; v < vocab; v += 32) s += exp2(((double)logit(x, v) - (double)m) * c);
  s = warp_sum(s);
  return s > 0 ? exp2(((double)x1 - (double)m) * c) / s : 0;
}

// A row is read in aligned 16-byte blocks, whatever its start; entries of the
// first and the last block that are not the row's count as -inf.  A CTA takes
// `per` chunks of kThreads * kBlocks blocks of one row, the next one's blocks
// in flight while the exponentials of one are summed.
template <typename T>
__global__ void __launch_bounds__(kThreads, kScanBlocks)
    verify_scan_kernel(const VerifyParams p, int segs, int per) {
  constexpr int kE = 16 / sizeof(T);
  __shared__ float2 sm[kThreads / 32];
  __shared__ int last;
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x / segs, seg = blockIdx.x % segs;
  const T* x = static_cast<const T*>(p.target) + row * p.target_stride;
  const int skew = (int)(reinterpret_cast<uintptr_t>(x) & 15u) / (int)sizeof(T);
  const uint4* base = reinterpret_cast<const uint4*>(x - skew);
  const int blocks = (p.vocab + skew + kE - 1) / kE;
  const bool whole = (p.vocab + skew) % kE == 0;  // the last block is all the row's
  const int chunk0 = seg * per;
  // whether the offsets are in order: asked before the logits are and needed
  // after them, or (large batches) asked by the rows' last CTAs alone
  const bool large = p.batch > kThreads;
  bool order = large || (int)threadIdx.x >= p.batch || offsets_fit(p.cu, threadIdx.x, p.total);
  auto load = [&](int ch, uint4 (&v)[kBlocks]) {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int b = (ch * kBlocks + i) * kThreads + threadIdx.x;
      constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
      v[i] = make_uint4(kNone, kNone, kNone, kNone);
      if ((b > 0 || skew == 0) && (b < blocks - 1 || (b == blocks - 1 && whole))) {
        v[i] = __ldcs(base + b);
      } else if (b < blocks) {  // an end of the row: entry by entry
        uint32_t w[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const int at = b * kE + e - skew;
          if (at < 0 || at >= p.vocab) continue;
          if constexpr (sizeof(T) == 2) {
            const uint32_t bits = __ldg(x + at);
            w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | (bits << 16) : (w[e / 2] & 0xffff0000u) | bits;
          } else {
            w[e] = __ldg(x + at);
          }
        }
        v[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  // each warp has a reference of its own, which follows its maximum; rounded
  // up, so that no exponent is above 0: where logits are large (a warp of
  // masked entries, -1e10 say) half a step of their product with c is hundreds
  const float c = (float)p.c;
  const float2 c2 = make_float2(c, c);
  float ref = safe_max(safe_max(-INFINITY) * c);
  float2 s2 = make_float2(0.f, 0.f);
  uint4 next[kBlocks];
  load(chunk0, next);
  for (int ch = 0; ch < per && (chunk0 + ch) * kThreads * kBlocks < blocks; ++ch) {
    uint4 v[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) v[i] = next[i];
    if (ch + 1 < per) load(chunk0 + ch + 1, next);
    const float top = fmaxf(ref, __fmul_ru(warp_max(blocks_max<T>(v)), c));
    const float f = ex2_approx(ref - top);
    s2 = __fmul2_rn(s2, make_float2(f, f));
    ref = top;
    const float2 r2 = make_float2(-ref, -ref);
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      float e[kE];
      unpack<T>(v[i], e);
#pragma unroll
      for (int k = 0; k < kE; k += 2) {
        const float2 d = __ffma2_rn(make_float2(e[k], e[k + 1]), c2, r2);
        s2 = __fadd2_rn(s2, make_float2(ex2_approx(d.x), ex2_approx(d.y)));
      }
    }
  }
  const float s = warp_sum(s2.x + s2.y);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = make_float2(ref, s);
  __syncthreads();
  const int cls = row % (int)kPagedCounters, rows = p.total + p.batch;
  if (threadIdx.x == 0) {
    float top = sm[0].x, sum = 0.f;
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) top = fmaxf(top, sm[i].x);
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) sum = fmaf(sm[i].y, exp2f(sm[i].x - top), sum);
    p.scan[(int64_t)row * segs + seg] = make_float2(top, sum);
    // rows that share a counter are finished together (there are
    // kPagedCounters of them, so mostly that is one row)
    __threadfence();
    const uint32_t all = (uint32_t)(((rows - 1 - cls) / (int)kPagedCounters + 1) * segs);
    last = atomicAdd(&p.arrived[cls], 1u) == all - 1;
    if (last) p.arrived[cls] = 0;  // for the next call
    __threadfence();
  }
  order = __syncthreads_and(order);
  if (!last) return;
  if (large) {
#pragma unroll 1
    for (int b = threadIdx.x; b < p.batch; b += kThreads)
      order = offsets_fit(p.cu, b, p.total) && order;
    order = __syncthreads_and(order);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = cls + warp * (int)kPagedCounters; r < rows; r += kThreads / 32 * (int)kPagedCounters) {
    // the sequence whose rows cu[b] + b .. cu[b + 1] + b hold r: by bisection,
    // or in turn, of the rows of `cu` that stand, where they are not in order
    int lo = order ? 0 : -1, hi = order ? p.batch : 0;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) + mid <= r) lo = mid;
      else hi = mid;
    }
#pragma unroll 1
    for (int a = 0, end = 0; !order && a < p.batch; ++a) {
      if (!offsets_fit(p.cu, a, p.total) || __ldg(p.cu + a) < end) continue;
      end = __ldg(p.cu + a + 1);
      if (__ldg(p.cu + a) + a <= r) lo = a;
    }
    const int q0 = lo < 0 ? 0 : __ldg(p.cu + lo), q1 = lo < 0 ? 0 : __ldg(p.cu + lo + 1), t = r - lo;
    const bool drafted = q0 >= 0 && q1 <= p.total && t >= q0 && t < q1;
    int tok = -1;
    double bar = 0;
    if (drafted) {
      tok = __ldg(p.draft_tokens + t);
      bar = (double)__ldg(p.u_accept + t) * (double)__ldg(p.draft_conf + t);
    }
    const bool in = (uint32_t)tok < (uint32_t)p.vocab;
    const float x1 = in ? logit(static_cast<const T*>(p.target) + r * p.target_stride, tok) : 0.f;
    const float2* sc = p.scan + (int64_t)r * segs;
    const float2 mine = lane < segs ? __ldcg(sc + lane) : make_float2(-INFINITY, 0.f);
    float top = mine.x;
    for (int k = lane + 32; k < segs; k += 32) top = fmaxf(top, __ldcg(sc + k).x);
    top = warp_max(top);
    double sum = (double)mine.y * exp2f(mine.x - top);
    for (int k = lane + 32; k < segs; k += 32) {
      const float2 v = __ldcg(sc + k);
      sum += (double)v.y * exp2f(v.x - top);
    }
    sum = warp_sum(sum);
    const bool wide = !(fabsf(top) < kWide);
    double pr = 0;
    if (wide && drafted && in)
      pr = wide_prob(static_cast<const T*>(p.target) + r * p.target_stride, p.vocab, p.c, x1);
    if (lane == 0) {
      p.ref[r] = top;
      p.owner[r] = lo;
      if (drafted) {
        if (!in) atomicOr(p.err, kDevErrBounds);
        if (!wide && in && sum > 0) pr = exp2((double)x1 * (double)c - (double)top) / sum;
        p.target_prob[t] = (float)pr;
        p.state[t] = pr == 0 ? 1 : !wide && fabs(bar - pr) <= kNear * pr ? 2 : bar < pr ? 0 : 1;
      }
    }
  }
}

// p(x) of one row with 64-bit sums relative to 2^ref (the whole CTA; the
// near-tie path).
template <typename T>
__device__ double exact_prob(const T* x, int vocab, double c, double ref, int tok, double* smd) {
  double s = 0;
  for (int v = threadIdx.x; v < vocab; v += kThreads) s += exp2((double)logit(x, v) * c - ref);
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) smd[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0;
  for (int i = 0; i < kThreads / 32; ++i) s += smd[i];
  __syncthreads();
  return exp2((double)logit(x, tok) * c - ref) / s;
}

// The draw of sequence b: its first refusal, by every CTA of `norm` alike; the
// first of them (`mine`) also writes the outputs that follow from it.
template <typename T>
__device__ Draw find_draw(const VerifyParams& p, int b, bool mine) {
  __shared__ double smd[kThreads / 32];
  __shared__ int first;
  Draw dr{0, -1, -1, 0};
  const int q0 = __ldg(p.cu + b), q1 = __ldg(p.cu + b + 1);
  // possible by itself, and the scan gave it its target rows
  if (q0 < 0 || q1 < q0 || q1 > p.total || p.owner[q0 + b] != b) {
    if (mine && threadIdx.x == 0) {
      atomicOr(p.err, kDevErrBounds);
      p.accepted[b] = 0;
      p.draw[b] = dr;
    }
    return dr;
  }
  const int k = q1 - q0;
  int n = 0;
  while (true) {
    if (threadIdx.x == 0) first = k;
    __syncthreads();
    for (int i = n + threadIdx.x; i < k; i += kThreads)
      if (p.state[q0 + i] != 0) {
        atomicMin(&first, i);
        break;
      }
    __syncthreads();
    n = first;
    if (n == k || p.state[q0 + n] == 1) break;
    const int row = q0 + b + n;
    const double pr = exact_prob(static_cast<const T*>(p.target) + row * p.target_stride, p.vocab,
                                 p.c, (double)p.ref[row], p.draft_tokens[q0 + n], smd);
    if (!((double)p.u_accept[q0 + n] * (double)p.draft_conf[q0 + n] < pr)) break;
    ++n;
  }
  dr.t_row = q0 + b + n;
  dr.d_row = n < k ? q0 + n : -1;
  dr.out = q0 + b + n;
  if (mine) {
    for (int i = threadIdx.x; i <= k; i += kThreads)
      if (i != n) p.tokens[q0 + b + i] = i < n ? p.draft_tokens[q0 + i] : -1;
    if (threadIdx.x == 0) {
      p.accepted[b] = n;
      p.draw[b] = dr;
    }
  }
  return dr;
}

// This thread's kPer consecutive entries of a chunk: one or two wide loads
// where the row is aligned, entry by entry where not.
template <typename T, int kPer>
__device__ __forceinline__ void load_entries(const T* x, int v0, int vocab, float (&e)[kPer]) {
  constexpr int kE = 16 / sizeof(T);
  if ((reinterpret_cast<uintptr_t>(x) & 15u) == 0 && v0 + kPer <= vocab) {
    if constexpr (kPer < kE) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(x + v0));
      e[0] = bf16lo(v.x);
      e[1] = bf16hi(v.x);
      e[2] = bf16lo(v.y);
      e[3] = bf16hi(v.y);
    } else {
#pragma unroll
      for (int i = 0; i < kPer / kE; ++i) {
        float f[kE];
        unpack<T>(__ldg(reinterpret_cast<const uint4*>(x + v0) + i), f);
#pragma unroll
        for (int k = 0; k < kE; ++k) e[i * kE + k] = f[k];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = v0 + i < vocab ? logit(x, v0 + i) : -INFINITY;
  }
}

// What the target's row and the draft's (if any) hold at the draw of b.
template <typename T, int kPer>
__device__ __forceinline__ void load_rows(const VerifyParams& p, const Draw& dr, int ch,
                                          float (&xt)[kPer], float (&xd)[kPer]) {
  const int v0 = (ch * kThreads + threadIdx.x) * kPer;
  load_entries<T, kPer>(static_cast<const T*>(p.target) + dr.t_row * p.target_stride, v0, p.vocab, xt);
  if (dr.d_row >= 0)
    load_entries<T, kPer>(static_cast<const T*>(p.draft) + dr.d_row * p.draft_stride, v0, p.vocab, xd);
  else
#pragma unroll
    for (int i = 0; i < kPer; ++i) xd[i] = -INFINITY;
}

template <typename T, int kPer>
__global__ void __launch_bounds__(kThreads) verify_norm_kernel(const VerifyParams p, int chunks) {
  __shared__ float2 smf[kThreads / 32];
  __shared__ Pair smd[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / chunks, ch = blockIdx.x % chunks;
  const Draw dr = find_draw<T>(p, b, ch == 0);
  if (dr.out < 0) return;
  float xt[kPer], xd[kPer];
  load_rows<T, kPer>(p, dr, ch, xt, xd);
  float mt = xt[0], md = xd[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) {
    mt = fmaxf(mt, xt[i]);
    md = fmaxf(md, xd[i]);
  }
  float2 m = block_max2(mt, md, smf);
  m = make_float2(safe_max(m.x), safe_max(m.y));
  double st = 0, sd = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) st += exp2(((double)xt[i] - (double)m.x) * p.c);
  if (dr.d_row >= 0)
#pragma unroll
    for (int i = 0; i < kPer; ++i) sd += exp2(((double)xd[i] - (double)m.y) * p.cd);
  const Pair s = block_sum2(st, sd, smd);
  if (threadIdx.x == 0) {
    Part* part = p.part + (int64_t)b * 2 * chunks + ch;
    part[0] = Part{s.x, m.x, 0};
    part[chunks] = Part{s.y, m.y, 0};
  }
}

template <typename T, int kPer>
__global__ void __launch_bounds__(kThreads) verify_pick_kernel(const VerifyParams p, int chunks) {
  __shared__ float2 smf[kThreads / 32];
  __shared__ Pair smd[3][kThreads / 32];
  __shared__ int s_last, s_chunk, s_tok;
  __shared__ double s_bar;
  constexpr int kWarps = kThreads / 32;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / chunks, ch = blockIdx.x % chunks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Draw dr = p.draw[b];
  if (dr.out < 0) return;
  const bool drafted = dr.d_row >= 0;
  float xt[kPer], xd[kPer];
  load_rows<T, kPer>(p, dr, ch, xt, xd);
  // both rows' maxima and sums from the chunks'
  const Part* part = p.part + (int64_t)b * 2 * chunks;
  const Part none{0, -INFINITY, 0};
  const Part pt = (int)threadIdx.x < chunks ? part[threadIdx.x] : none;
  const Part pd = (int)threadIdx.x < chunks ? part[chunks + threadIdx.x] : none;
  float mt = pt.m, md = pd.m;
  for (int i = threadIdx.x + kThreads; i < chunks; i += kThreads) {
    mt = fmaxf(mt, part[i].m);
    md = fmaxf(md, part[chunks + i].m);
  }
  const float2 m = block_max2(mt, md, smf);
  double st = pt.s * exp2(((double)pt.m - (double)m.x) * p.c);
  double sd = pd.s * exp2(((double)pd.m - (double)m.y) * p.cd);
  for (int i = threadIdx.x + kThreads; i < chunks; i += kThreads) {
    st += part[i].s * exp2(((double)part[i].m - (double)m.x) * p.c);
    sd += part[chunks + i].s * exp2(((double)part[chunks + i].m - (double)m.y) * p.cd);
  }
  const Pair z = block_sum2(st, sd, smd[0]);
  const double it = z.x > 0 ? 1.0 / z.x : 0.0, id = z.y > 0 ? 1.0 / z.y : 0.0;
  // this thread's weights in a chunk whose logits are loaded (-inf: 0), and
  // their sum; consecutive entries per thread, so that thread order is
  // vocabulary order
  auto weigh = [&](bool rest, double (&w)[kPer]) {
    double s = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      w[e] = exp2(((double)xt[e] - (double)m.x) * p.c) * it;
      if (rest) w[e] = fmax(w[e] - exp2(((double)xd[e] - (double)m.y) * p.cd) * id, 0.0);
      s += w[e];
    }
    return s;
  };
  double w[kPer];
  const double ws = block_sum2(weigh(drafted, w), 0, smd[1]).x;
  double* weights = p.weight + (int64_t)b * chunks;
  if (threadIdx.x == 0) {
    weights[ch] = ws;
    __threadfence();
    s_last = atomicAdd(&p.draw[b].arrived, 1) == chunks - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  // every chunk's sum is there: this CTA finds the chunk, then the entry.
  // A scan of per-thread sums of `n` consecutive values: exclusive prefix.
  auto prefix = [&](double mine, Pair* sm, double& total) {
    double inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    __syncthreads();
    if (lane == 31) sm[warp].x = inc;
    if (threadIdx.x == 0) {
      s_chunk = -1;
      s_tok = p.vocab;
    }
    __syncthreads();
    double before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += sm[i].x;
      total += sm[i].x;
    }
    return before + inc - mine;
  };
  const int each = (chunks + kThreads - 1) / kThreads;  // chunks of a thread
  bool rest = drafted;
  double total = 0, at = 0;
  auto chunk_weight = [&](int i) {
    return rest || !drafted ? __ldcg(weights + i)
                            : part[i].s * exp2(((double)part[i].m - (double)m.x) * p.c) * it;
  };
  while (true) {
    double mine = 0;
    for (int i = threadIdx.x * each; i < min(chunks, (int)(threadIdx.x + 1) * each); ++i)
      mine += chunk_weight(i);
    at = prefix(mine, smd[2], total);
    if (total > 0 || !rest) break;
    rest = false;  // no residual mass: the target itself
  }
  const double bar = (double)p.u_sample[b] * total;
  // the first chunk that passes the bar; none does (rounding): the last with
  // mass.  Its thread keeps the weight before it.
  int pass = -1, mass = -1;
  double before_pass = 0, before_mass = 0;
  for (int i = threadIdx.x * each; i < min(chunks, (int)(threadIdx.x + 1) * each); ++i) {
    const double wi = chunk_weight(i);
    if (wi > 0) {
      mass = i;
      before_mass = at;
      if (pass < 0 && at + wi > bar) {
        pass = i;
        before_pass = at;
      }
    }
    at += wi;
  }
  // (one candidate per warp: thread order is vocabulary order)
  auto offer = [&](int lowest, int highest) {
    const uint32_t lo = __ballot_sync(0xffffffffu, lowest >= 0);
    const uint32_t hi = __ballot_sync(0xffffffffu, highest >= 0);
    if (lo && lane == __ffs(lo) - 1) atomicMin(&s_tok, lowest);
    if (hi && lane == 31 - __clz(hi)) atomicMax(&s_chunk, highest);
  };
  offer(pass, mass);
  __syncthreads();
  const int c = s_tok < p.vocab ? s_tok : s_chunk;
  if (c < 0) {  // no mass at all: every logit of the target's row is -inf
    if (threadIdx.x == 0) p.tokens[dr.out] = -1;
    return;
  }
  if (c == pass) s_bar = bar - before_pass;
  else if (c == mass && s_tok == p.vocab) s_bar = bar - before_mass;
  load_rows<T, kPer>(p, dr, c, xt, xd);
  double sum;
  at = prefix(weigh(rest, w), smd[2], sum);  // (its barriers publish s_bar)
  int found = -1, last = -1;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    at += w[e];
    if (w[e] > 0) {
      last = (c * kThreads + threadIdx.x) * kPer + e;
      if (found < 0 && at > s_bar) found = last;
    }
  }
  offer(found, last);
  __syncthreads();
  // (rounding may leave the bar at the chunk's end: its last entry with mass)
  if (threadIdx.x == 0) p.tokens[dr.out] = s_tok < p.vocab ? s_tok : s_chunk;
}

size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }
// (one entry short of a block more than the row has, for any alignment)
template <typename T>
int scan_chunks(int vocab) {
  constexpr int kE = 16 / sizeof(T), kChunk = kThreads * kBlocks * kE;
  return (int)(((int64_t)vocab + kE - 1 + kChunk - 1) / kChunk);
}
int pick_chunks(int vocab, int per) { return (vocab + kThreads * per - 1) / (kThreads * per); }

template <typename T>
cudaError_t launch_verify_t(const VerifyParams& p, cudaStream_t stream) {
  // several chunks per CTA once there are many more than the SMs hold (up to
  // eight CTAs each), so that what a CTA does besides reading is done less often
  const int sc = scan_chunks<T>(p.vocab), rows = p.total + p.batch;
  const int per = (int)std::min<int64_t>(8, std::max<int64_t>(1, (int64_t)rows * sc / (148 * 16)));
  const int segs = (sc + per - 1) / per;
  cudaError_t e = launch_pdl(verify_scan_kernel<T>, dim3(rows * segs), dim3(kThreads), 0, stream, p,
                             segs, per);
  note_launch();
  if (e != cudaSuccess) return e;
  auto draw = [&](auto per_thread) {
    constexpr int kPer = decltype(per_thread)::value;
    const int pc = pick_chunks(p.vocab, kPer);
    cudaError_t e = launch_pdl(verify_norm_kernel<T, kPer>, dim3(p.batch * pc), dim3(kThreads), 0,
                               stream, p, pc);
    note_launch();
    if (e != cudaSuccess) return e;
    e = launch_pdl(verify_pick_kernel<T, kPer>, dim3(p.batch * pc), dim3(kThreads), 0, stream, p,
                   pc);
    note_launch();
    return e;
  };
  // Few chunks (one per SM at most) are waited for, each thread's entries one
  // after the other: with half as many bf16 entries per thread one sequence of
  // 262,144 takes 18.5 us (20.1), of 32,000 16.3 (19.1).  Many chunks cost by
  // their number: eight sequences take 65.5 us with 8 entries, 68.8 with 4 (and
  // one of fp32 rows, whose 8 are two loads, 20.3 and 20.9).
  if constexpr (sizeof(T) == 2)
    if ((int64_t)p.batch * pick_chunks(p.vocab, kMany) <= 148)
      return draw(std::integral_constant<int, kFew>{});
  return draw(std::integral_constant<int, kMany>{});
}

}  // namespace

size_t verify_scratch_bytes(int batch, int total, int vocab) {
  const size_t sc = scan_chunks<uint32_t>(vocab), pc = pick_chunks(vocab, kFew);  // the more of them
  return align16((size_t)(total + batch) * sc * sizeof(float2)) +
         2 * align16((size_t)(total + batch) * sizeof(float)) + align16((size_t)total) +
         align16((size_t)batch * sizeof(Draw)) + (size_t)batch * 2 * pc * sizeof(Part) +
         (size_t)batch * pc * sizeof(double);
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
  VerifyParams p{};
  p.target = a.target;
  p.draft = a.draft;
  p.batch = a.batch;
  p.total = a.total;
  p.vocab = a.vocab;
  p.target_stride = a.target_stride;
  p.draft_stride = a.draft_stride;
  p.c = 1.4426950408889634074 / a.tau;
  p.cd = 1.4426950408889634074 / a.draft_tau;
  p.draft_tokens = a.draft_tokens;
  p.draft_conf = a.draft_conf;
  p.cu = a.cu_draft;
  p.u_accept = a.u_accept;
  p.u_sample = a.u_sample;
  p.accepted = a.accepted;
  p.tokens = a.tokens;
  p.target_prob = a.target_prob;
  p.err = a.err;
  p.arrived = a.arrived;
  const size_t sc = scan_chunks<uint32_t>(a.vocab), pc = pick_chunks(a.vocab, kFew);
  uint8_t* s = static_cast<uint8_t*>(a.scratch);
  p.scan = reinterpret_cast<float2*>(s);
  s += align16((size_t)(a.total + a.batch) * sc * sizeof(float2));
  p.ref = reinterpret_cast<float*>(s);
  s += align16((size_t)(a.total + a.batch) * sizeof(float));
  p.owner = reinterpret_cast<int*>(s);
  s += align16((size_t)(a.total + a.batch) * sizeof(int));
  p.state = s;
  s += align16((size_t)a.total);
  p.draw = reinterpret_cast<Draw*>(s);
  s += align16((size_t)a.batch * sizeof(Draw));
  p.part = reinterpret_cast<Part*>(s);
  s += (size_t)a.batch * 2 * pc * sizeof(Part);
  p.weight = reinterpret_cast<double*>(s);
  return a.bf16 ? launch_verify_t<uint16_t>(p, stream) : launch_verify_t<uint32_t>(p, stream);
}

}  // namespace dd
