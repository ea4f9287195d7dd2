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
// Four kernels:
//   scan    one read of all the target's rows: per chunk of kScan logits the
//           maximum and the sum of 2^((x - max) c), c = log2(e) / tau, in
//           fp32 (c as two floats, so that the long argument of a small term
//           does not lose what its many peers add up to).  Bound by memory.
//   decide  one CTA per sequence merges the chunks of its rows, forms p(x_i)
//           in 64 bits and takes the first refusal.  A test within kNear of
//           equality is repeated with a 64-bit sum over the row, so that the
//           decision is the one exact arithmetic takes.
//   norm    for the one row the next token is drawn at: the 64-bit sums of
//           the target's and the draft's exponentials per chunk of kPick
//           logits.  The running sum has a border per vocabulary entry (up
//           to 262,144 of them), and a relative error of e in the weights
//           moves each border by about e: with fp32 sums one draw in ten to
//           a hundred would land on another token, with 64 bits none does.
//   pick    the weights' sums per chunk; the last chunk to finish finds the
//           chunk that holds u_s W and walks it.
// Sums are taken in a fixed order, so a call's result does not depend on
// scheduling.
#include "dd_paged.cuh"

namespace dd {
namespace {

constexpr int kScan = 8192;  // logits per scan chunk
constexpr int kPick = 2048;  // logits per norm / pick chunk
constexpr int kThreads = 256;
constexpr double kNear = 1e-5;

// What `decide` hands on about sequence b's draw.
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
  float2* scan;       // [total + batch][scan chunks]: maximum, sum
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
// Block-wide sum / maximum in every thread (a fixed order; 2 barriers).
template <typename F>
__device__ F block_sum(F v, F* sm) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  F r = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) r += sm[i];
  __syncthreads();
  return r;
}
__device__ float block_max(float v, float* sm) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = sm[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) r = fmaxf(r, sm[i]);
  __syncthreads();
  return r;
}

// A maximum that exponents may be taken against: rows (chunks) of -inf only
// get a finite one, against which every term is 0.
__device__ __forceinline__ float safe_max(float m) { return fmaxf(m, -3.0e38f); }

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_scan_kernel(const VerifyParams p, int chunks) {
  __shared__ float smf[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x / chunks, ch = blockIdx.x % chunks;
  const T* x = static_cast<const T*>(p.target) + row * p.target_stride;
  const int v0 = ch * kScan, v1 = min(p.vocab, v0 + kScan);
  float m = -INFINITY;
  for (int v = v0 + threadIdx.x; v < v1; v += kThreads) m = fmaxf(m, logit(x, v));
  m = block_max(m, smf);
  const float mr = safe_max(m), c = (float)p.c, c_lo = (float)(p.c - (double)c);
  float s = 0.f;
  for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
    const float d = logit(x, v) - mr;
    s += ex2_approx(fmaf(d, c, d * c_lo));
  }
  s = block_sum(s, smf);
  if (threadIdx.x == 0) p.scan[(int64_t)row * chunks + ch] = make_float2(m, s);
}

// p(x) of one row with 64-bit sums (the whole CTA; the near-tie path).
template <typename T>
__device__ double exact_prob(const T* x, int vocab, double c, float m, int tok, double* smd) {
  double s = 0;
  for (int v = threadIdx.x; v < vocab; v += kThreads)
    s += exp2(((double)logit(x, v) - (double)m) * c);
  s = block_sum(s, smd);
  return exp2(((double)logit(x, tok) - (double)m) * c) / s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    verify_decide_kernel(const VerifyParams p, int chunks) {
  __shared__ double smd[kThreads / 32];
  __shared__ int first;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q0 = p.cu[b], q1 = p.cu[b + 1];
  Draw dr{0, -1, -1, 0};
  if (q0 < 0 || q1 < q0 || q1 > p.total) {
    if (threadIdx.x == 0) {
      atomicOr(p.err, kDevErrBounds);
      p.accepted[b] = 0;
      p.draw[b] = dr;
    }
    return;
  }
  const int k = q1 - q0;
  auto row_of = [&](int i) {
    return static_cast<const T*>(p.target) + (int64_t)(q0 + b + i) * p.target_stride;
  };
  auto row_max = [&](int i) {  // the row's maximum, in every lane
    const float2* sc = p.scan + (int64_t)(q0 + b + i) * chunks;
    float m = -INFINITY;
    for (int c = lane; c < chunks; c += 32) m = fmaxf(m, sc[c].x);
    return safe_max(warp_max(m));
  };
  for (int i = warp; i < k; i += kThreads / 32) {
    const float2* sc = p.scan + (int64_t)(q0 + b + i) * chunks;
    const float m = row_max(i);
    double s = 0;
    for (int c = lane; c < chunks; c += 32)
      s += (double)sc[c].y * exp2(((double)safe_max(sc[c].x) - (double)m) * p.c);
    s = warp_sum(s);
    if (lane == 0) {
      const int tok = p.draft_tokens[q0 + i];
      double pr = 0;
      uint8_t st = 1;
      if ((uint32_t)tok >= (uint32_t)p.vocab) {
        atomicOr(p.err, kDevErrBounds);
      } else {
        if (s > 0) pr = exp2(((double)logit(row_of(i), tok) - (double)m) * p.c) / s;
        const double bar = (double)p.u_accept[q0 + i] * (double)p.draft_conf[q0 + i];
        st = fabs(bar - pr) <= kNear * pr ? 2 : bar < pr ? 0 : 1;
        if (pr == 0) st = 1;
      }
      p.target_prob[q0 + i] = (float)pr;
      p.state[q0 + i] = st;
    }
  }
  __syncthreads();
  int n = 0;
  while (true) {  // the first row that is not accepted; near ones are decided in 64 bits
    if (threadIdx.x == 0) first = k;
    __syncthreads();
    for (int i = n + threadIdx.x; i < k; i += kThreads)
      if (p.state[q0 + i] != 0) {
        atomicMin(&first, i);
        break;
      }
    __syncthreads();
    n = first;
    __syncthreads();
    if (n == k || p.state[q0 + n] == 1) break;
    const float m = row_max(n);
    const double pr = exact_prob(row_of(n), p.vocab, p.c, m, p.draft_tokens[q0 + n], smd);
    if (!((double)p.u_accept[q0 + n] * (double)p.draft_conf[q0 + n] < pr)) break;
    ++n;
  }
  for (int i = threadIdx.x; i <= k; i += kThreads)
    if (i != n) p.tokens[q0 + b + i] = i < n ? p.draft_tokens[q0 + i] : -1;
  if (threadIdx.x == 0) {
    p.accepted[b] = n;
    dr.t_row = q0 + b + n;
    dr.d_row = n < k ? q0 + n : -1;
    dr.out = q0 + b + n;
    p.draw[b] = dr;
  }
}

// Maximum and 64-bit sum of one chunk of a row (the whole CTA).
template <typename T>
__device__ Part chunk_part(const T* x, int v0, int v1, double c, float* smf, double* smd) {
  float m = -INFINITY;
  for (int v = v0 + threadIdx.x; v < v1; v += kThreads) m = fmaxf(m, logit(x, v));
  Part r;
  r.m = safe_max(block_max(m, smf));
  double s = 0;
  for (int v = v0 + threadIdx.x; v < v1; v += kThreads)
    s += exp2(((double)logit(x, v) - (double)r.m) * c);
  r.s = block_sum(s, smd);
  r.pad = 0;
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_norm_kernel(const VerifyParams p, int chunks) {
  __shared__ float smf[kThreads / 32];
  __shared__ double smd[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / chunks, ch = blockIdx.x % chunks;
  const Draw dr = p.draw[b];
  if (dr.out < 0) return;
  const int v0 = ch * kPick, v1 = min(p.vocab, v0 + kPick);
  Part* part = p.part + (int64_t)b * 2 * chunks + ch;
  const Part a = chunk_part(static_cast<const T*>(p.target) + dr.t_row * p.target_stride, v0, v1,
                            p.c, smf, smd);
  if (threadIdx.x == 0) part[0] = a;
  if (dr.d_row >= 0) {
    const Part d = chunk_part(static_cast<const T*>(p.draft) + dr.d_row * p.draft_stride, v0, v1,
                              p.cd, smf, smd);
    if (threadIdx.x == 0) part[chunks] = d;
  }
}

// Maximum and sum of a whole row from its chunks (the whole CTA).
__device__ Part row_part(const Part* part, int chunks, double c, float* smf, double* smd) {
  float m = -INFINITY;
  for (int i = threadIdx.x; i < chunks; i += kThreads) m = fmaxf(m, part[i].m);
  Part r;
  r.m = safe_max(block_max(m, smf));
  double s = 0;
  for (int i = threadIdx.x; i < chunks; i += kThreads)
    s += part[i].s * exp2(((double)part[i].m - (double)r.m) * c);
  r.s = block_sum(s, smd);
  r.pad = 0;
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_pick_kernel(const VerifyParams p, int chunks) {
  __shared__ float smf[kThreads / 32];
  __shared__ double smd[kThreads / 32];
  __shared__ int s_last, s_chunk, s_tok, s_any;
  __shared__ double s_before;
  constexpr int kPer = kPick / kThreads;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / chunks, ch = blockIdx.x % chunks;
  const Draw dr = p.draw[b];
  if (dr.out < 0) return;
  const Part* part = p.part + (int64_t)b * 2 * chunks;
  const T* xt = static_cast<const T*>(p.target) + dr.t_row * p.target_stride;
  const T* xd = static_cast<const T*>(p.draft) + max(dr.d_row, 0) * p.draft_stride;
  const Part zt = row_part(part, chunks, p.c, smf, smd);
  Part zd{};
  if (dr.d_row >= 0) zd = row_part(part + chunks, chunks, p.cd, smf, smd);
  const double it = zt.s > 0 ? 1.0 / zt.s : 0.0, id = zd.s > 0 ? 1.0 / zd.s : 0.0;
  // weight of entry v; `rest`: the residual rather than the target itself
  auto weight = [&](int v, bool rest) {
    double w = exp2(((double)logit(xt, v) - (double)zt.m) * p.c) * it;
    if (rest) w = fmax(w - exp2(((double)logit(xd, v) - (double)zd.m) * p.cd) * id, 0.0);
    return w;
  };
  // consecutive entries per thread, so that a walk in thread order is one
  // in vocabulary order
  auto thread_sum = [&](int c, bool rest, double (&w)[kPer]) {
    double s = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int v = c * kPick + threadIdx.x * kPer + e;
      w[e] = v < p.vocab ? weight(v, rest) : 0.0;
      s += w[e];
    }
    return s;
  };
  double w[kPer];
  bool rest = dr.d_row >= 0;
  const double ws = block_sum(thread_sum(ch, rest, w), smd);
  double* weights = p.weight + (int64_t)b * chunks;
  if (threadIdx.x == 0) {
    weights[ch] = ws;
    __threadfence();
    s_last = atomicAdd(&p.draw[b].arrived, 1) == chunks - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // every chunk's sum is there: find the chunk, then the entry
  if (threadIdx.x == 0) {
    double total = 0;
    for (int i = 0; i < chunks; ++i) total += __ldcg(weights + i);
    if (!(total > 0) && rest) {  // no residual mass: the target itself
      rest = false;
      total = 0;
      for (int i = 0; i < chunks; ++i) {
        weights[i] = part[i].s * exp2(((double)part[i].m - (double)zt.m) * p.c) * it;
        total += weights[i];
      }
    }
    const double bar = (double)p.u_sample[b] * total;
    int pick = -1;
    double run = 0, before = 0;
    for (int i = 0; i < chunks; ++i) {
      const double wi = __ldcg(weights + i);
      if (wi > 0) {  // the last chunk with mass, unless an earlier one passes the bar
        pick = i;
        before = run;
      }
      run += wi;
      if (run > bar) break;
    }
    s_chunk = pick;
    s_before = bar - before;
    s_any = rest ? 1 : 0;
    s_tok = p.vocab;
  }
  __syncthreads();
  const int c = s_chunk;
  if (c < 0) {  // no mass at all: every logit of the target's row is -inf
    if (threadIdx.x == 0) p.tokens[dr.out] = -1;
    return;
  }
  double run = thread_sum(c, s_any != 0, w);
  // exclusive prefix over the threads, in a fixed order
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double inc = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) smd[warp] = inc;
  __syncthreads();
  double at = inc - run;
  for (int i = 0; i < warp; ++i) at += smd[i];
  int last = -1;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int v = c * kPick + threadIdx.x * kPer + e;
    at += w[e];
    if (w[e] > 0) {
      last = v;
      if (at > s_before) {
        atomicMin(&s_tok, v);
        break;
      }
    }
  }
  __syncthreads();
  const int tok = s_tok;
  __syncthreads();
  if (tok < p.vocab) {
    if (threadIdx.x == 0) p.tokens[dr.out] = tok;
    return;
  }
  // rounding left the bar at the chunk's end: its last entry with mass
  if (threadIdx.x == 0) s_chunk = -1;
  __syncthreads();
  if (last >= 0) atomicMax(&s_chunk, last);
  __syncthreads();
  if (threadIdx.x == 0) p.tokens[dr.out] = s_chunk;
}

size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }
int scan_chunks(int vocab) { return (vocab + kScan - 1) / kScan; }
int pick_chunks(int vocab) { return (vocab + kPick - 1) / kPick; }

template <typename T>
cudaError_t launch_verify_t(const VerifyParams& p, cudaStream_t stream) {
  const int sc = scan_chunks(p.vocab), pc = pick_chunks(p.vocab);
  cudaError_t e = launch_pdl(verify_scan_kernel<T>, dim3((p.total + p.batch) * sc), dim3(kThreads),
                             0, stream, p, sc);
  note_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(verify_decide_kernel<T>, dim3(p.batch), dim3(kThreads), 0, stream, p, sc);
  note_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(verify_norm_kernel<T>, dim3(p.batch * pc), dim3(kThreads), 0, stream, p, pc);
  note_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(verify_pick_kernel<T>, dim3(p.batch * pc), dim3(kThreads), 0, stream, p, pc);
  note_launch();
  return e;
}

}  // namespace

size_t verify_scratch_bytes(int batch, int total, int vocab) {
  const size_t sc = scan_chunks(vocab), pc = pick_chunks(vocab);
  return align16((size_t)(total + batch) * sc * sizeof(float2)) + align16((size_t)total) +
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
  const size_t sc = scan_chunks(a.vocab), pc = pick_chunks(a.vocab);
  uint8_t* s = static_cast<uint8_t*>(a.scratch);
  p.scan = reinterpret_cast<float2*>(s);
  s += align16((size_t)(a.total + a.batch) * sc * sizeof(float2));
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
