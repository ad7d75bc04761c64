// pnb_pkv_attn.cu - attention over the paged KV cache, one warp per (token, query head) row.
#include <cuda_bf16.h>
#include <math.h>

#include "pnb_pkv.cuh"

namespace pnb {
namespace {

constexpr int kWarps = 8;

template <int HD, typename TQ, typename TO>
__global__ void __launch_bounds__(kWarps * 32) k_pkv_attn(const PkvAttnArgs a) {
  constexpr int N = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  pdl_wait();
  const int tok = (int)(row / a.n_head), h = (int)(row % a.n_head);
  if (tok >= a.seqs.n_tok) return;
  const int b = pkv_seq_of(a.seqs, tok);
  if (b < 0) return;
  int t0, n;
  pkv_tokens(a.seqs, b, t0, n);
  if (tok < t0 || tok - t0 >= n) {   // `start` decreases
    set_error(a.err, kErrRange);
    return;
  }
  const int last = pkv_len(a.seqs, a.pool.page_log2, b, a.err) - n + (tok - t0);
  const int lo = a.window > 0 ? max(0, last - a.window + 1) : 0;
  const int g = h / (a.n_head / a.pool.n_kv);
  const int32_t *pages = a.seqs.pages + (int64_t)b * a.seqs.max_page;
  float q[N], o[N] = {};
  load_vals<TQ, N>(static_cast<const TQ *>(a.q.p) + tok * a.q.token + h * a.q.head + lane * N, q);
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] *= a.qscale;
  float m = -INFINITY, sum = 0.f;
  for (int j = lo; j <= last; ++j) {
    const __nv_bfloat16 *k = pkv_row<HD>(a.pool, pages, j, 0, g);
    if (!k) {
      if (lane == 0) set_error(a.err, kErrRange);
      continue;
    }
    float x[N], s = 0.f;
    load_vals<__nv_bfloat16, N>(k + lane * N, x);
#pragma unroll
    for (int i = 0; i < N; ++i) s += q[i] * x[i];
    s = warp_sum(s);
    const float mn = fmaxf(m, s), c = exp2f(m - mn), p = exp2f(s - mn);
    load_vals<__nv_bfloat16, N>(k + ((int64_t)a.pool.n_kv << a.pool.page_log2) * HD + lane * N, x);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * c + p * x[i];
    sum = sum * c + p;
    m = mn;
  }
  TO *out = static_cast<TO *>(a.out.p) + tok * a.out.token + h * a.out.head + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) Elem<TO>::store(out, i, last < lo ? 0.f : o[i] / sum);
}

template <int HD>
cudaError_t launch_attn(const PkvAttnArgs &a, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)a.seqs.n_tok * a.n_head + kWarps - 1) / kWarps)), block(kWarps * 32);
  typedef __nv_bfloat16 H;
  if (a.q.dtype == PNB_F32)
    return a.out.dtype == PNB_F32 ? launch_pdl(k_pkv_attn<HD, float, float>, grid, block, 0, 1, st, a)
                                  : launch_pdl(k_pkv_attn<HD, float, H>, grid, block, 0, 1, st, a);
  return a.out.dtype == PNB_F32 ? launch_pdl(k_pkv_attn<HD, H, float>, grid, block, 0, 1, st, a)
                                : launch_pdl(k_pkv_attn<HD, H, H>, grid, block, 0, 1, st, a);
}

}  // namespace

cudaError_t launch_pkv_attn(int hd, const PkvAttnArgs &a, cudaStream_t st) {
  return hd == 128 ? launch_attn<128>(a, st) : launch_attn<64>(a, st);
}

}  // namespace pnb
