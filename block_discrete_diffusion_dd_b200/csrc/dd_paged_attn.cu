// dd_paged_attn.cu -- attention of a chunk of new tokens over a paged cache
// (dd_paged_attn): new token i of a sequence with n new tokens and `len`
// tokens in the cache sees the keys j < len - n + i + 1 (causal) or j < len,
//   O = sum_j softmax_j(scale <q, k_j>) v_j,
// zeros (log-sum-exp -inf) where it sees none.
//
// One warp per (token, query head): lane j scores key j of a block of 32,
// the warp runs an online softmax in base 2, and each lane accumulates D/32
// output columns.
#include "dd_paged.cuh"

namespace dd {
namespace {

constexpr int kWarps = 4;

template <int D, bool kF8>
__global__ void __launch_bounds__(kWarps * 32)
    paged_attn_kernel(const PagedBatch p, const PagedPool pool, int Hq,
                      const __nv_bfloat16* __restrict__ q, int64_t q_stride, float scale2,
                      int causal, __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                      uint32_t* err) {
  constexpr int DPL = D / 32;
  __shared__ float sQ[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
  const int t = (int)(unit / Hq), h = (int)(unit % Hq);
  if (t >= p.total_new) return;
  const int b = owner_row(p.cu_new, p.batch, t);
  if (b < 0) return;
  const ChunkRow c = chunk_row(p, b, err);
  if (t - c.q0 >= c.n) return;
  const int seen = causal ? c.len - c.n + (t - c.q0) + 1 : c.len;
  const int64_t head = (int64_t)(h / (Hq / p.heads_kv)) << p.page_shift;
  for (int d = lane; d < D; d += 32) sQ[warp][d] = (float)q[t * q_stride + h * D + d];
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[DPL] = {};
  for (int j0 = 0; j0 < seen; j0 += 32) {
    const int j = j0 + lane;
    int64_t row = -1;
    float s = -INFINITY, fv = 1.f;
    if (j < seen) {
      row = pool_row(p, b, j, err);
      if (row >= 0) {
        row += head;
        float x = 0.f;
        if constexpr (kF8) {
          const uint8_t* kr = static_cast<const uint8_t*>(pool.k) + row * D;
          for (int d = 0; d < D; d += 2) {
            const float2 kd = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(kr + d));
            x = fmaf(sQ[warp][d], kd.x, fmaf(sQ[warp][d + 1], kd.y, x));
          }
          x *= pow2f((int)pool.k_scale[row] - 127);
          fv = pow2f((int)pool.v_scale[row] - 127);
        } else {
          const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(pool.k) + row * D;
          for (int d = 0; d < D; ++d) x = fmaf(sQ[warp][d], (float)kr[d], x);
        }
        s = x * scale2;
      }
    }
    float mx = s;
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = ex2_approx(m - ref), pr = ex2_approx(s - ref);
    float ps = pr;
    for (int off = 16; off > 0; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
    l = l * alpha + ps;
    m = mn;
    for (int k = 0; k < DPL; ++k) o[k] *= alpha;
    for (int jj = 0; jj < 32; ++jj) {
      const float w = __shfl_sync(0xffffffffu, pr * fv, jj);
      const int64_t r = __shfl_sync(0xffffffffu, row, jj);
      if (r < 0) continue;
      for (int k = 0; k < DPL; ++k) {
        const int64_t at = r * D + lane + 32 * k;
        float x;
        if constexpr (kF8)
          x = e4m3x2_to_float2(static_cast<const uint8_t*>(pool.v)[at]).x;
        else
          x = (float)static_cast<const __nv_bfloat16*>(pool.v)[at];
        o[k] = fmaf(w, x, o[k]);
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t at = (int64_t)t * Hq + h;
  for (int k = 0; k < DPL; ++k) out[at * D + lane + 32 * k] = (__nv_bfloat16)(o[k] * inv);
  if (lse && lane == 0)
    lse[at] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int D, bool kF8>
cudaError_t launch_t(const PagedAttnArgs& a, cudaStream_t stream) {
  const int64_t units = (int64_t)a.p.total_new * a.heads_q;
  paged_attn_kernel<D, kF8><<<(unsigned)((units + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(
      a.p, a.pool, a.heads_q, static_cast<const __nv_bfloat16*>(a.q), a.q_stride,
      a.scale * 1.4426950408889634f, a.causal ? 1 : 0, static_cast<__nv_bfloat16*>(a.out), a.lse,
      a.err);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

size_t paged_attn_scratch_bytes(const PagedAttnArgs&) { return 0; }

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  if (a.p.head_dim == 64)
    return a.pool.e4m3 ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
  return a.pool.e4m3 ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
}

}  // namespace dd
