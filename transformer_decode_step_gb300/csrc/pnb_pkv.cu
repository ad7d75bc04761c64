// pnb_pkv.cu - append of the paged KV cache: rotation of queries and keys and
// the store of keys and values into pages.
//
// Token t at position p turns pair i of a row by the angle p theta^(-2i/hd):
// (x, y) -> (x cos - y sin, x sin + y cos).  The frequency is held in turns as a
// 64-bit fraction, so that position times frequency, cut off at whole turns by
// the multiplication itself, is the exact turn; its rounding to fp32 is off by
// at most 2^-24 of the turn, whatever the position.  Bound by bytes: each row is
// read and written once.
//
// An 8k MHA prompt (32 heads, head_dim 128, bf16, 403 MB) takes 68.5 us, 5.9 TB/s (88 % of a
// plain copy), its warps waiting for loads; 64 single tokens 11 us with the host's part, 7
// without: lengths, starts and page ids, then rows, in turn.
#include <cuda_bf16.h>

#include "pnb_pkv.cuh"

namespace pnb {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxPairs = 64;
// Loads on their way come from many warps rather than from many rows per lane: an 8k MHA
// prompt (half-split, bf16) with 1, 2, 3 rows per lane takes 68, 73, 96 us, and with 2, 4, 5, 6
// CTAs per SM 92, 68, 78, 108 (the registers of the last do not hold the rows).
constexpr int kCtasPerSm = 4;

// A lane's part of a row: E elements (8 l ..), or, half-split, E / 2 of each half, as 16-byte
// loads where the type allows: 8 elements, and 16 of bf16 half-split rows.
template <bool NEOX, typename T>
constexpr int kElems = NEOX && sizeof(T) == 2 ? 16 : 8;

template <int HD, bool NEOX, typename T>
__device__ __forceinline__ void load_part(const T *p, int l, float (&f)[kElems<NEOX, T>]) {
  constexpr int E = kElems<NEOX, T>, V = sizeof(T) == 2 ? 8 : 4;   // elements of a 16-byte load
#pragma unroll
  for (int i = 0; i < E; i += V) {
    const T *from = !NEOX ? p + E * l + i : i < E / 2 ? p + E / 2 * l + i : p + HD / 2 + E / 2 * l + i - E / 2;
    load_vals<T, V>(from, reinterpret_cast<float(&)[V]>(f[i]));
  }
}

// the same part of a row of type T, computed as E elements
template <int HD, bool NEOX, int E, typename T>
__device__ __forceinline__ void store_part(T *p, int l, const float (&f)[E]) {
  constexpr int V = sizeof(T) == 4 ? 4 : NEOX && E == 8 ? 4 : 8;
#pragma unroll
  for (int i = 0; i < E; i += V) {
    T *to = !NEOX ? p + E * l + i : i < E / 2 ? p + E / 2 * l + i : p + HD / 2 + E / 2 * l + i - E / 2;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4 *>(to) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    else if constexpr (V == 4)
      *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16(f[i], f[i + 1]), pack_bf16(f[i + 2], f[i + 3]));
    else
      *reinterpret_cast<uint4 *>(to) = make_uint4(pack_bf16(f[i], f[i + 1]), pack_bf16(f[i + 2], f[i + 3]),
                                                  pack_bf16(f[i + 4], f[i + 5]), pack_bf16(f[i + 6], f[i + 7]));
  }
}

// a.wpt warps (1, 2, 4 or 8) take a token: they compute its cosines and sines once, in
// shared memory, while its first rows load
template <int HD, bool NEOX, typename T, typename TQ>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) k_pkv_append(const PkvAppendArgs a) {
  constexpr int E = kElems<NEOX, T>, LPR = HD / E, RPW = 32 / LPR;   // lanes per row, rows per warp
  constexpr int U = E == 16 ? 1 : sizeof(T) == 2 ? 4 : 2;                // rows on their way per lane
  __shared__ float2 turns[kWarps][kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tok = blockIdx.x * (kWarps / a.wpt) + warp / a.wpt, rank = warp % a.wpt;
  pdl_wait();
  // the lane's pairs turn by positions that are there, or by the token's entry
  constexpr int PAIRS = HD / 2 / 32;   // per lane, at one warp per token
  int pos[PAIRS] = {};
  if (a.pos && a.freq && tok < a.seqs.n_tok)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      const int i = (rank + j * a.wpt) * 32 + lane;
      if (i < HD / 2) pos[j] = a.pos[(int64_t)((i >= a.sec0) + (i >= a.sec1)) * a.seqs.n_tok + tok];
    }
  int b, t0, n, len = 0;
  if (tok >= a.seqs.n_tok) {
    b = -1;
  } else if (a.seqs.start && a.seqs.n_seq <= 32) {
    // all sequences' starts and lengths in one trip to memory, a lane each
    const int at = min(lane, a.seqs.n_seq - 1);
    const int from = a.seqs.start[at], to = a.seqs.start[at + 1], held = a.seqs.len[at];
    b = __popc(__ballot_sync(0xffffffffu, lane < a.seqs.n_seq && to <= tok));
    const int src = min(b, a.seqs.n_seq - 1);
    t0 = min(max(__shfl_sync(0xffffffffu, from, src), 0), a.seqs.n_tok);
    n = max(min(__shfl_sync(0xffffffffu, to, src), a.seqs.n_tok) - t0, 0);
    len = __shfl_sync(0xffffffffu, held, src);
    if (b >= a.seqs.n_seq) b = -1;
  } else {
    b = pkv_seq_of(a.seqs, tok);
    if (b >= 0) {
      pkv_tokens(a.seqs, b, t0, n);
      len = a.seqs.len[b];
    }
  }
  // (tokens before the first sequence are no one's, as are any that a `start` that decreases leaves out)
  const bool live = b >= 0 && tok >= t0 && tok - t0 < n;
  if (blockIdx.x == 0 && a.seqs.start &&
      pkv_bad_starts(a.seqs.start, a.seqs.n_seq, -1, -1, a.seqs.n_tok, threadIdx.x, kWarps * 32))
    set_error(a.err, kErrRange);
  const int64_t e64 = live ? (int64_t)len - n + (tok - t0) : 0;   // the token's entry
  const int e = (int)e64;

  const bool held = live && e64 >= 0 && e64 < (int64_t)a.seqs.max_page << a.pool.page_log2;
  // the entry's K row of KV head 0
  __nv_bfloat16 *const page =
      held ? pkv_row<HD>(a.pool, a.seqs.pages + (int64_t)b * a.seqs.max_page, e, 0, 0) : nullptr;

  const int l = lane % LPR, sub = lane / LPR;
  const int nq = a.q.p ? a.n_head : 0, nkv = a.pool.n_kv, rows = nq + 2 * nkv, step = a.wpt * RPW;
  const T *q = static_cast<const T *>(a.q.p) + tok * a.q.token;
  const T *k = static_cast<const T *>(a.k.p) + tok * a.k.token;
  const T *v = static_cast<const T *>(a.v.p) + tok * a.v.token;
  float x[U][E];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * step;
      if (r >= rows) break;
      const T *p = r < nq ? q + r * a.q.head : r < nq + nkv ? k + (r - nq) * a.k.head : v + (r - nq - nkv) * a.v.head;
      load_part<HD, NEOX, T>(p, l, x[u]);
    }
  };
  int r0 = rank * RPW + sub;
  if (live) load(r0);

  float2 *mine = turns[warp / a.wpt * a.wpt];
  if (live && a.freq) {
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      const int i = (rank + j * a.wpt) * 32 + lane;
      if (i >= HD / 2) break;
      const int p = a.pos ? pos[j] : e;
      const long long turn = (long long)((unsigned long long)(long long)p * a.freq[i]);
      float sn, cs;
      sincospif(__ll2float_rn(turn) * 0x1p-63f, &sn, &cs);
      mine[i] = make_float2(cs, sn);
    }
  }
  if (a.wpt > 1) __syncthreads();
  else __syncwarp();
  if (!live) return;

  if (!page && lane == 0 && rank == 0) set_error(a.err, held ? kErrRange : kErrFull);
  const int64_t head_step = (int64_t)HD << a.pool.page_log2;
  float2 cs[E / 2];
#pragma unroll
  for (int j = 0; j < E / 2; ++j) cs[j] = a.freq ? mine[E / 2 * l + j] : make_float2(1.f, 0.f);
  TQ *q_out = static_cast<TQ *>(a.q_out.p) + tok * a.q_out.token;
  while (r0 < rows) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * step;
      if (r >= rows) break;
      if (r < nq + nkv && a.freq) {
        float(&f)[E] = x[u];
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          float &y = f[NEOX ? j : 2 * j], &z = f[NEOX ? E / 2 + j : 2 * j + 1];
          const float y0 = y, z0 = z;
          y = y0 * cs[j].x - z0 * cs[j].y;
          z = y0 * cs[j].y + z0 * cs[j].x;
        }
      }
      if (r < nq) store_part<HD, NEOX, E, TQ>(q_out + r * a.q_out.head, l, x[u]);
      else if (page) store_part<HD, NEOX, E, __nv_bfloat16>(page + (r - nq) * head_step, l, x[u]);   // V lies n_kv heads behind K
    }
    r0 += step * U;
    if (r0 < rows) load(r0);
  }
}

template <int HD, bool NEOX>
cudaError_t launch_append(const PkvAppendArgs &a, int grid, cudaStream_t st) {
  const bool in32 = a.k.dtype == PNB_F32, out32 = a.q.p ? a.q_out.dtype == PNB_F32 : in32;
  typedef __nv_bfloat16 H;
  if (in32)
    return out32 ? launch_pdl(k_pkv_append<HD, NEOX, float, float>, dim3(grid), dim3(kWarps * 32), 0, 1, st, a)
                 : launch_pdl(k_pkv_append<HD, NEOX, float, H>, dim3(grid), dim3(kWarps * 32), 0, 1, st, a);
  return out32 ? launch_pdl(k_pkv_append<HD, NEOX, H, float>, dim3(grid), dim3(kWarps * 32), 0, 1, st, a)
               : launch_pdl(k_pkv_append<HD, NEOX, H, H>, dim3(grid), dim3(kWarps * 32), 0, 1, st, a);
}

}  // namespace

cudaError_t launch_pkv_append(int hd, bool neox, const PkvAppendArgs &args, cudaStream_t st) {
  PkvAppendArgs a = args;
  // few tokens: a token's rows go to several warps, so that they load at once
  a.wpt = 8;
  while (a.wpt > 1 && (int64_t)a.seqs.n_tok * a.wpt > (int64_t)a.sms * 32) a.wpt /= 2;
  const int per = kWarps / a.wpt, grid = (a.seqs.n_tok + per - 1) / per;
  if (hd == 128) return neox ? launch_append<128, true>(a, grid, st) : launch_append<128, false>(a, grid, st);
  return neox ? launch_append<64, true>(a, grid, st) : launch_append<64, false>(a, grid, st);
}

}  // namespace pnb
