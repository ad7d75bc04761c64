// pnb_pkv.cuh - the paged KV cache: layout, kernel arguments and launchers.
//
// A layer of the pool is [n_page][2 (K, V)][n_kv][page][head_dim] bf16: the
// entries of one page, K or V and KV head are a contiguous run of rows, so that
// a tiled bulk copy brings them as they lie.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pnb.h"
#include "pnb_device.cuh"
#include "pnb_rows.cuh"

namespace pnb {

constexpr int kPkvMaxSeq = 1024;
constexpr int kPkvMaxGroup = 64;       // query heads per KV head

// one layer of a pool
struct PkvPool {
  __nv_bfloat16 *base;
  int32_t n_page, page_log2, n_kv;
};

// the sequences of a call
struct PkvSeqs {
  const int32_t *start, *len, *pages;   // start NULL: `each` tokens per sequence
  int32_t n_seq, max_page, n_tok, each;
};

struct PkvAppendArgs {
  PkvPool pool;
  PkvSeqs seqs;
  DevRows k, v, q, q_out;               // q.p NULL: no queries
  int32_t n_head;
  const int32_t *pos;                   // [1 or 3][n_tok] or NULL
  int32_t sec0, sec1;                   // pairs before the second and the third axis (one axis: head_dim / 2)
  const unsigned long long *freq;       // [head_dim / 2] turns per position in units of 2^-64, NULL: no rotation
  int32_t *err;
  int32_t wpt;                          // warps per token (set by the launcher)
  int32_t sms;
};

struct PkvAttnArgs {
  PkvPool pool;
  PkvSeqs seqs;
  DevRows q, out;
  int32_t n_head, window;
  float qscale;                         // log2(e) / sqrt(head_dim)
  int32_t *err;
};

cudaError_t launch_pkv_append(int hd, bool neox, const PkvAppendArgs &a, cudaStream_t st);
cudaError_t launch_pkv_attn(int hd, const PkvAttnArgs &a, cudaStream_t st);

// Tokens of sequence b: the first one and their number, kept inside the packed
// rows whatever `start` holds.
__device__ __forceinline__ void pkv_tokens(const PkvSeqs &s, int b, int &t0, int &n) {
  if (s.start) {
    t0 = min(max(s.start[b], 0), s.n_tok);
    n = max(min(s.start[b + 1], s.n_tok) - t0, 0);
  } else {
    t0 = b * s.each;
    n = s.each;
  }
}

// entries of sequence b, no more than its page table names
__device__ __forceinline__ int pkv_len(const PkvSeqs &s, int page_log2, int b, int32_t *err) {
  const int n = s.len[b], most = (int)min((int64_t)s.max_page << page_log2, (int64_t)0x7fffffff);
  if (n < 0 || n > most) set_error(err, kErrRange);
  return min(max(n, 0), most);
}

// The sequence of a packed token (the calling warp; every lane answers), -1
// behind the last one.  Two rounds of 32 loads for up to 1024 sequences.
__device__ __forceinline__ int pkv_seq_of(const PkvSeqs &s, int tok) {
  if (!s.start) return tok / s.each;
  const int lane = threadIdx.x & 31;
  // sequences whose end is not behind the token
  const int step = (s.n_seq + 31) / 32;
  const int e = min((lane + 1) * step, s.n_seq);
  const int blk = __popc(__ballot_sync(0xffffffffu, s.start[e] <= tok));
  if (blk == 32) return -1;
  if (step == 1) return blk < s.n_seq ? blk : -1;
  const int b0 = blk * step;
  const int f = min(b0 + lane + 1, s.n_seq);
  const int b = b0 + __popc(__ballot_sync(0xffffffffu, lane < step && b0 + lane < s.n_seq && s.start[f] <= tok));
  return b < s.n_seq ? b : -1;
}

// row `e` of the page that holds an entry, K (0) or V (1); NULL when the table
// names no page of the pool
template <int HD>
__device__ __forceinline__ __nv_bfloat16 *pkv_row(const PkvPool &p, const int32_t *pages, int e, int kv, int head) {
  const int id = pages[e >> p.page_log2];
  if (id < 0 || id >= p.n_page) return nullptr;
  const int64_t row = (((int64_t)id * 2 + kv) * p.n_kv + head) << p.page_log2;
  return p.base + (row + (e & ((1 << p.page_log2) - 1))) * HD;
}

}  // namespace pnb
