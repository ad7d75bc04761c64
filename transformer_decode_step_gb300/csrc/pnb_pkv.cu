// pnb_pkv.cu - append of the paged KV cache: rotation of queries and keys and
// the store of keys and values into pages.
//
// Token t at position p turns pair i of a row by the angle p theta^(-2i/hd):
// (x, y) -> (x cos - y sin, x sin + y cos).  The frequency is held in turns as a
// 64-bit fraction, so that position times frequency, cut off at whole turns by
// the multiplication itself, is the exact turn; its rounding to fp32 is off by
// at most 2^-24 of the turn, whatever the position.  Bound by bytes: each row is
// read and written once.
#include <cuda_bf16.h>

#include "pnb_pkv.cuh"

namespace pnb {
namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;      // rows on their way per lane group

// 8 elements of a row: 8 l .. 8 l + 7, or, half-split, 4 l .. 4 l + 3 of each half
template <int HD, bool NEOX, typename T>
__device__ __forceinline__ void load8(const T *p, int l, float (&f)[8]) {
  if constexpr (NEOX) {
    load_vals<T, 4>(p + 4 * l, reinterpret_cast<float(&)[4]>(f[0]));
    load_vals<T, 4>(p + HD / 2 + 4 * l, reinterpret_cast<float(&)[4]>(f[4]));
  } else if constexpr (sizeof(T) == 2) {
    load_vals<T, 8>(p + 8 * l, f);
  } else {
    load_vals<T, 4>(p + 8 * l, reinterpret_cast<float(&)[4]>(f[0]));
    load_vals<T, 4>(p + 8 * l + 4, reinterpret_cast<float(&)[4]>(f[4]));
  }
}

template <int HD, bool NEOX, typename T>
__device__ __forceinline__ void store8(T *p, int l, const float (&f)[8]) {
  T *a = NEOX ? p + 4 * l : p + 8 * l, *b = NEOX ? p + HD / 2 + 4 * l : p + 8 * l + 4;
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4 *>(a) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(b) = make_float4(f[4], f[5], f[6], f[7]);
  } else if constexpr (NEOX) {
    *reinterpret_cast<uint2 *>(a) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
    *reinterpret_cast<uint2 *>(b) = make_uint2(pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  } else {
    *reinterpret_cast<uint4 *>(a) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
}

template <int HD, bool NEOX, typename T, typename TQ>
__global__ void __launch_bounds__(kWarps * 32) k_pkv_append(const PkvAppendArgs a) {
  constexpr int LPR = HD / 8, RPW = 32 / LPR;   // lanes per row, rows per warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tok = blockIdx.x * (kWarps / a.wpt) + warp / a.wpt;
  pdl_wait();
  if (tok >= a.seqs.n_tok) return;
  const int b = pkv_seq_of(a.seqs, tok);
  if (b < 0) return;
  int t0, n;
  pkv_tokens(a.seqs, b, t0, n);
  if (tok < t0 || tok - t0 >= n) {   // `start` decreases
    set_error(a.err, kErrRange);
    return;
  }
  const int64_t e64 = (int64_t)a.seqs.len[b] - n + (tok - t0);   // the token's entry
  const int e = (int)e64;
  const int l = lane % LPR, sub = lane / LPR, rank = warp % a.wpt;

  float cs[4], sn[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = 4 * l + j;
    cs[j] = 1.f;
    sn[j] = 0.f;
    if (a.freq) {
      const int axis = (i >= a.sec0) + (i >= a.sec1);
      const int p = a.pos ? a.pos[(int64_t)axis * a.seqs.n_tok + tok] : e;
      const long long turn = (long long)((unsigned long long)(long long)p * a.freq[i]);
      sincospif(__ll2float_rn(turn) * 0x1p-63f, &sn[j], &cs[j]);
    }
  }

  __nv_bfloat16 *page = nullptr;   // the entry's K row of KV head 0
  if (e64 < 0 || e64 >= (int64_t)a.seqs.max_page << a.pool.page_log2) {
    if (lane == 0 && rank == 0) set_error(a.err, kErrFull);
  } else {
    page = pkv_row<HD>(a.pool, a.seqs.pages + (int64_t)b * a.seqs.max_page, e, 0, 0);
    if (!page && lane == 0 && rank == 0) set_error(a.err, kErrRange);
  }
  const int64_t head_step = (int64_t)HD << a.pool.page_log2;

  const int nq = a.q.p ? a.n_head : 0, nkv = a.pool.n_kv, rows = nq + 2 * nkv;
  const T *q = static_cast<const T *>(a.q.p) + tok * a.q.token;
  const T *k = static_cast<const T *>(a.k.p) + tok * a.k.token;
  const T *v = static_cast<const T *>(a.v.p) + tok * a.v.token;
  TQ *q_out = static_cast<TQ *>(a.q_out.p) + tok * a.q_out.token;
  const int step = a.wpt * RPW;
  for (int r0 = rank * RPW + sub; r0 < rows; r0 += step * kUnroll) {
    float x[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * step;
      if (r >= rows) break;
      const T *p = r < nq ? q + r * a.q.head : r < nq + nkv ? k + (r - nq) * a.k.head : v + (r - nq - nkv) * a.v.head;
      load8<HD, NEOX>(p, l, x[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * step;
      if (r >= rows) break;
      if (r < nq + nkv && a.freq) {
        float(&f)[8] = x[u];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float &y = f[NEOX ? j : 2 * j], &z = f[NEOX ? 4 + j : 2 * j + 1];
          const float y0 = y, z0 = z;
          y = y0 * cs[j] - z0 * sn[j];
          z = y0 * sn[j] + z0 * cs[j];
        }
      }
      if (r < nq) store8<HD, NEOX>(q_out + r * a.q_out.head, l, x[u]);
      else if (page) store8<HD, NEOX>(page + (r - nq) * head_step, l, x[u]);   // V lies n_kv heads behind K
    }
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
