// pnb_pkv_sched.cuh - the list of work of the paged cache's attention kernels: blocks of
// rows, their tiles of entries, and each CTA's run through them.
#pragma once

#include "pnb_pkv.cuh"

namespace pnb {

constexpr int kPkvMinRun = 4;      // units that a CTA starts for
struct PkvItem {
  int b, j, h;              // sequence or group, block, KV head
  int tok0, ntok;           // its tokens
  int base;                 // first token's last entry (prompts)
  int hi, lo;               // entries [lo, hi): those that some row sees
  int hi_min, lo_max;       // entries [lo_max, hi_min): those that every row sees
  int len;                  // the sequence's entries (the prefix's)
  int floor;                // entries below are the prefix's, another pass's
  int t0, nt;               // tiles of the whole item
  int ta, tb;               // this CTA's tiles
  bool ends;                // the item's end is this CTA's
};

// tokens of a sequence, or of a group's sequences in the prefix's pass
__device__ __forceinline__ void pkv_members(const PkvAttnArgs &a, int b, int &t0, int &n) {
  if (a.pass == kPkvPrefix) {
    const int gs = min(max(a.group_start[b], 0), a.seqs.n_seq), ge = min(max(a.group_start[b + 1], gs), a.seqs.n_seq);
    t0 = gs * a.seqs.each;
    n = (ge - gs) * a.seqs.each;
  } else {
    pkv_tokens(a.seqs, b, t0, n);
  }
}

// the j-th block of a sequence or group; false behind the last one
template <int TILE>
__device__ __forceinline__ bool pkv_block(const PkvAttnArgs &a, int TB, int b, int j, PkvItem &it) {
  int t0, n;
  pkv_members(a, b, t0, n);
  if (j * TB >= n) return false;
  it.b = b;
  it.j = j;
  it.tok0 = t0 + j * TB;
  it.ntok = min(TB, n - j * TB);
  const int W = a.window;
  it.floor = 0;
  if (a.pass == kPkvPrefix) {
    const PkvGroup g = a.groups[b];
    it.base = 0;
    it.len = INT_MAX;   // (a shared prefix is whole pages, all of them entries)
    it.hi = it.hi_min = g.prefix;
    it.lo = W > 0 ? min(max(0, g.len_min - a.seqs.each - W + 1), g.prefix) : 0;
    it.lo_max = W > 0 ? max(0, g.len_max - W) : 0;
  } else {
    it.len = pkv_len(a.seqs, a.pool.page_log2, b, a.err);
    it.base = it.len - n + j * TB;
    it.hi = max(0, it.base + it.ntok);
    it.hi_min = it.base + 1;
    it.lo = W > 0 ? max(0, it.base - W + 1) : 0;
    it.lo_max = W > 0 ? max(0, it.base + it.ntok - W) : 0;
    if (a.pass == kPkvOwn) {
      const int g = pkv_group_of(a.group_start, a.n_group, b);
      const int p = g < 0 ? 0 : a.groups[g].prefix;
      it.lo = min(max(it.lo, p), it.hi);
      it.lo_max = max(it.lo_max, p);
      it.floor = p;
    }
  }
  it.t0 = it.lo / TILE;
  it.nt = max(1, (it.hi + TILE - 1) / TILE - it.t0);
  return true;
}

// a CTA's way through its run of units
struct PkvWalk {
  int h, b, j, x;       // next item, units of it that lie before the run
  int64_t left;         // units
  int n_b;              // sequences or groups

  template <int TILE>
  __device__ __forceinline__ bool next(const PkvAttnArgs &a, int TB, PkvItem &it) {
    while (left > 0 && h < a.pool.n_kv) {
      if (!pkv_block<TILE>(a, TB, b, j, it)) {
        j = 0;
        if (++b == n_b) {
          b = 0;
          ++h;
        }
        continue;
      }
      const int units = it.nt + a.item_units;
      const int end = (int)min((int64_t)units, x + left);
      it.h = h;
      it.ta = max(0, x - a.item_units);
      it.tb = max(0, end - a.item_units);
      it.ends = end == units;
      left -= end - x;
      x = end;
      if (it.ends) {
        ++j;
        x = 0;
      }
      if (it.tb > it.ta) return true;
    }
    return false;
  }
};

// The shared prefix of every group as all of its queries see it.  Every CTA writes
// the same numbers, so each finds its own.
template <int THREADS>
__device__ __forceinline__ void pkv_find_groups(const PkvAttnArgs &a, int *scratch) {
  int *gmin = scratch, *gmax = scratch + a.n_group;
  for (int g = threadIdx.x; g < a.n_group; g += THREADS) {
    gmin[g] = INT_MAX;
    gmax[g] = 0;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < a.seqs.n_seq; s += THREADS) {
    const int g = pkv_group_of(a.group_start, a.n_group, s);
    if (g < 0) {
      set_error(a.err, kErrRange);
      continue;
    }
    const int n = pkv_len(a.seqs, a.pool.page_log2, s, a.err);
    atomicMin(&gmin[g], n);
    atomicMax(&gmax[g], n);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < a.n_group; g += THREADS) {
    const int p = min(max(a.prefix[g], 0), max(0, gmin[g] - a.seqs.each));
    a.groups[g] = PkvGroup{p >> a.pool.page_log2 << a.pool.page_log2, gmin[g], gmax[g], 0};
  }
  __syncthreads();
}

// Where this CTA's run starts.  The blocks of one KV head are counted and their
// units added up by all threads; heads follow one another in the list.
template <int TILE, int THREADS>
__device__ __forceinline__ void pkv_find_run(const PkvAttnArgs &a, int TB, int *scratch, PkvWalk *out) {
  const int n_b = a.pass == kPkvPrefix ? a.n_group : a.seqs.n_seq, tid = threadIdx.x, lane = tid & 31;
  int *first = scratch;                                             // [n_b + 1] blocks before a sequence
  long long *sums = reinterpret_cast<long long *>(scratch + 1026);   // [THREADS + 1]
  for (int b = tid; b < n_b; b += THREADS) {
    int t0, n;
    pkv_members(a, b, t0, n);
    first[b + 1] = (n + TB - 1) / TB;
  }
  if (tid == 0) first[0] = 0;
  __syncthreads();
  if (tid < 32) {
    int base = 0;
    for (int b0 = 1; b0 <= n_b; b0 += 32) {
      int v = b0 + lane <= n_b ? first[b0 + lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (b0 + lane <= n_b) first[b0 + lane] = base + v;
      base += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  const int blocks = first[n_b];
  const int i0 = (int)((int64_t)blocks * tid / THREADS), i1 = (int)((int64_t)blocks * (tid + 1) / THREADS);
  // the sequence of block i0: the last one that starts at or before it
  int b0 = 0;
  if (i0 < i1) {
    int lo = 0, hi = n_b;   // first[lo] <= i0 < first[hi]
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (first[m] <= i0) lo = m;
      else hi = m;
    }
    b0 = lo;
  }
  auto walk = [&](auto &&f) {
    int b = b0, j = i0 - first[b0];
    for (int i = i0; i < i1; ++i) {
      PkvItem it;
      while (!pkv_block<TILE>(a, TB, b, j, it)) {
        ++b;
        j = 0;
      }
      if (!f(b, j, it.nt + a.item_units)) return;
      ++j;
    }
  };
  long long mine = 0;
  walk([&](int, int, int u) {
    mine += u;
    return true;
  });
  sums[tid + 1] = mine;
  if (tid == 0) sums[0] = 0;
  __syncthreads();
  if (tid < 32) {
    long long base = 0;
    for (int k0 = 1; k0 <= THREADS; k0 += 32) {
      long long v = sums[k0 + lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      sums[k0 + lane] = base + v;
      base += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  const long long per_head = sums[THREADS], total = per_head * a.pool.n_kv;
  // as many CTAs as get a run of a few units each
  const long long ctas = max(1ll, min((long long)gridDim.x, total / kPkvMinRun));
  const long long c = min((long long)blockIdx.x, ctas), u0 = total * c / ctas, u1 = total * min(c + 1, ctas) / ctas;
  if (u1 <= u0) {
    if (tid == 0) *out = PkvWalk{0, 0, 0, 0, 0, n_b};
  } else {
    const int h = (int)(u0 / per_head);
    const long long in_head = u0 - h * per_head;
    if (in_head >= sums[tid] && in_head < sums[tid + 1]) {
      long long at = sums[tid];
      walk([&](int b, int j, int u) {
        if (in_head >= at + u) {
          at += u;
          return true;
        }
        *out = PkvWalk{h, b, j, (int)(in_head - at), u1 - u0, n_b};
        return false;
      });
    }
  }
  __syncthreads();
}

}  // namespace pnb
