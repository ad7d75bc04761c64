// pnb_pkv.cuh - the paged KV cache: layout, kernel arguments and launchers.
//
// A layer of the pool is [n_page][2 (K, V)][n_kv][page][head_dim] bf16: the
// entries of one page, K or V and KV head are a contiguous run of rows, so that
// a tiled bulk copy brings them as they lie.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "pnb.h"
#include "pnb_device.cuh"
#include "pnb_rows.cuh"

namespace pnb {

constexpr int kPkvMaxSeq = 1024;
constexpr int kPkvMaxGroup = 64;       // query heads per KV head
constexpr int kPkvMaxCtas = 512;       // most CTAs of an attention kernel

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

// Rows (token, query head of a KV head's group) that share their K and V are
// attended together: the tokens of one sequence, or, over a shared prefix, those
// of all the sequences of a group.  A block is up to kPkvBlockRows such rows, an
// item a block with its tiles of kPkvTile entries; the flat list of all items'
// tiles (and a few units more per item, for its queries and its end) is cut into
// equal runs, one per CTA.  What a run holds of an item that others share goes to
// the run's partial sums, which a second kernel adds up in the list's order.
constexpr int kPkvBoxLog2 = 6;          // rows of a TMA box: a page's, at most 64
// what a kernel attends to: everything, the groups' prefixes, or what lies behind them;
// the rows of the last two are unfinished, and a kernel behind both adds them up
enum { kPkvAll = 0, kPkvPrefix = 1, kPkvOwn = 2 };
constexpr int kPkvTile = 128;          // of the prompts' kernel
constexpr int kPkvChunk = 64;          // of the steps' kernel
constexpr int kPkvBlockRows = 256;     // at most; see pkv_block_rows
// rows of a block of the prompts' kernel
__host__ __device__ constexpr int pkv_block_rows(int hd, bool split) { return split && hd == 128 ? 128 : 256; }

// what a CTA left of an item that others share
struct PkvPart {
  int32_t flags;      // 1: holds something, 2: the item ends here
  int32_t b, j, h;    // sequence (or group), block, KV head
};

// the whole pages that a group shares, as far as every query of the group sees
// them, and its sequences' shortest and longest length
struct PkvGroup {
  int32_t prefix, len_min, len_max, pad;
};

struct PkvAttnArgs {
  PkvPool pool;
  PkvSeqs seqs;
  DevRows q, out;
  int32_t n_head, window;
  float qscale;                         // log2(e) / sqrt(head_dim)
  int32_t *err;
  int32_t pass;                         // kPkvAll, kPkvPrefix, kPkvOwn
  // groups of sequences with a common prefix
  const int32_t *group_start, *prefix;
  int32_t n_group;
  PkvGroup *groups;                     // [n_group] workspace
  // unfinished rows, sums and (reference, their weights' sum): of whole items, of the prefix's
  // and of the own pass [n_tok][n_head][head_dim], [..][2], and of what items share, per CTA
  float *row_o[2], *row_ml[2];
  float *part_o, *part_ml;              // [2 grid][kPkvBlockRows][head_dim], [..][2]
  PkvPart *part;                        // [2 grid]
  int32_t grid;
  int32_t block_rows;
  int32_t heads_inner;                  // the list's order (set by the launchers)
  // what an item costs beside its tiles, in tiles, and a tile's time on an SM; the same of the
  // pass beside this one, and its tiles' entries (set by the launchers)
  int32_t item_units, unit_ns, other_item_units, other_ns, other_tile;
};

cudaError_t prepare_pkv_rows(int hd);
cudaError_t prepare_pkv_step(int hd);
cudaError_t launch_pkv_append(int hd, bool neox, const PkvAppendArgs &a, cudaStream_t st);
cudaError_t launch_pkv_rows(int hd, const CUtensorMap &map, const PkvAttnArgs &a, cudaStream_t st);
cudaError_t launch_pkv_step(int hd, const CUtensorMap &map, const PkvAttnArgs &a, cudaStream_t st);
// adds up the parts that the CTAs left, up to `rows` rows per item, and with a.pass not kPkvAll
// the parts of both passes and then the passes
cudaError_t launch_pkv_join(int hd, const PkvAttnArgs &a, int rows, cudaStream_t st);
// a tile's time, and what an item costs beside its tiles
void pkv_rows_cost(int hd, bool split, int *unit_ns, int *item_units);
void pkv_step_cost(int hd, int *unit_ns, int *item_units);
inline bool pkv_split(const PkvAttnArgs &a) { return a.q.dtype == PNB_F32 || a.out.dtype == PNB_F32; }

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

// Whether the calling threads (thread i of n) find starts that are out of range or decrease,
// from `first` (-1: from anywhere) to `last` (-1: to anywhere) in 0 .. most.
__device__ __forceinline__ bool pkv_bad_starts(const int32_t *start, int count, int first, int last, int most, int i, int n) {
  bool bad = false;
  for (; i <= count; i += n) {
    const int at = start[i], before = i ? start[i - 1] : 0;
    bad |= at < before || at > most || (i == 0 && first >= 0 && at != first) || (i == count && last >= 0 && at != last);
  }
  return bad;
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

// the group of sequence s, -1 when none holds it (group starts that decrease or
// do not reach it)
__device__ __forceinline__ int pkv_group_of(const int32_t *start, int n_group, int s) {
  int lo = 0, hi = n_group;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (start[m] <= s) lo = m;
    else hi = m;
  }
  return start[lo] <= s && s < start[lo + 1] ? lo : -1;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// 2^x by the hardware's approximation (2 ulp; subnormal results are 0)
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// N consecutive outputs o * f
template <int N>
__device__ __forceinline__ void pkv_store(const DevRows &out, int64_t at, const float *o, float f) {
  if (out.dtype == PNB_F32) {
    float *p = static_cast<float *>(out.p) + at;
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4 *>(p + i) = make_float4(o[i] * f, o[i + 1] * f, o[i + 2] * f, o[i + 3] * f);
    } else {
      *reinterpret_cast<float2 *>(p) = make_float2(o[0] * f, o[1] * f);
    }
  } else {
    __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(out.p) + at;
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 8)
        *reinterpret_cast<uint4 *>(p + i) =
            make_uint4(pack_bf16(o[i] * f, o[i + 1] * f), pack_bf16(o[i + 2] * f, o[i + 3] * f),
                       pack_bf16(o[i + 4] * f, o[i + 5] * f), pack_bf16(o[i + 6] * f, o[i + 7] * f));
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) *reinterpret_cast<uint32_t *>(p + i) = pack_bf16(o[i] * f, o[i + 1] * f);
    }
  }
}

// Sums of R rows over entries [from, to) of each, by the calling warp, without matrix
// instructions: lanes take an entry each for the scores and HD / 32 elements each (l * HD / 32 ..)
// for the outputs.  A page that the table does not name counts as zeros, and what a row
// does not see is no part of its sums, whatever it holds.  *work changes every 32 entries.
template <int HD, int R>
__device__ __forceinline__ void pkv_attend_rows(const PkvPool &pool, const int32_t *pages, int h, const DevRows &q,
                                             const int64_t (&q_at)[R], float scale, const int (&from)[R],
                                             const int (&to)[R], float (&o)[R][HD / 32], float (&m)[R], float (&sum)[R],
                                             uint32_t *work) {
  constexpr int N = HD / 32;
  const int lane = threadIdx.x & 31;
  int begin = INT_MAX, end = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (from[r] < to[r]) {
      begin = min(begin, from[r]);
      end = max(end, to[r]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) o[r][i] = 0.f;
    m[r] = -INFINITY;
    sum[r] = 0.f;
  }
  for (int e0 = begin; e0 < end; e0 += 32) {
    const int e = e0 + lane;
    const __nv_bfloat16 *k = e < end ? pkv_row<HD>(pool, pages, e, 0, h) : nullptr;
    float s[R] = {};
    if (k) {
#pragma unroll 4
      for (int i = 0; i < HD; i += 4) {
        float y[4];
        load_vals<__nv_bfloat16, 4>(k + i, y);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float x[4];
          if (q.dtype == PNB_F32) load_vals<float, 4>(static_cast<const float *>(q.p) + q_at[r] + i, x);
          else load_vals<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16 *>(q.p) + q_at[r] + i, x);
#pragma unroll
          for (int c = 0; c < 4; ++c) s[r] = fmaf(x[c], y[c], s[r]);
        }
      }
    }
    float p[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float x = e >= from[r] && e < to[r] ? s[r] * scale : -INFINITY;
      const float top = fmaxf(m[r], warp_max(x)), ref = top == -INFINITY ? 0.f : top, f = exp2f(m[r] - ref);
      p[r] = exp2f(x - ref);
      sum[r] = sum[r] * f + warp_sum(p[r]);
#pragma unroll
      for (int i = 0; i < N; ++i) o[r][i] *= f;
      m[r] = top;
    }
    const long long v = (long long)(uintptr_t)(k ? k + ((int64_t)pool.n_kv << pool.page_log2) * HD : nullptr);
#pragma unroll 4
    for (int j = 0; j < 32; ++j) {
      const long long at = __shfl_sync(0xffffffffu, v, j);
      float y[N] = {};
      if (at) load_vals<__nv_bfloat16, N>(reinterpret_cast<const __nv_bfloat16 *>((uintptr_t)at) + lane * N, y);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = __shfl_sync(0xffffffffu, p[r], j);
        const bool sees = e0 + j >= from[r] && e0 + j < to[r];
#pragma unroll
        for (int i = 0; i < N; ++i) o[r][i] = sees ? fmaf(f, y[i], o[r][i]) : o[r][i];
      }
    }
    if (lane == 0) atomicAdd(work, 1u);
  }
}

// the same for one row, by a call
template <int HD>
__device__ __noinline__ void pkv_attend_row(const PkvPool &pool, const int32_t *pages, int h, const DevRows &q,
                                            int64_t q_at, float scale, int from, int to, float (&o)[HD / 32], float &m,
                                            float &sum, uint32_t *work) {
  const int64_t at[1] = {q_at};
  const int f[1] = {from}, t[1] = {to};
  float ms[1], sums[1];
  pkv_attend_rows<HD, 1>(pool, pages, h, q, at, scale, f, t, reinterpret_cast<float(&)[1][HD / 32]>(o), ms, sums, work);
  m = ms[0];
  sum = sums[0];
}

// what brings sums with references m and m2 to a common one
__device__ __forceinline__ void pkv_join_factors(float m, float m2, float &f, float &f2) {
  const float top = fmaxf(m, m2);
  f = m == -INFINITY ? 0.f : exp2f(m - top);
  f2 = m2 == -INFINITY ? 0.f : exp2f(m2 - top);
}

}  // namespace pnb
