// pnb_pkv_sched.cuh - the list of work of the paged cache's attention kernels: blocks of
// rows, their tiles of entries, and each CTA's run through them.
//
// Over a shared prefix two lists are worked through at once, the groups' prefixes and what
// the sequences have of their own: each gets CTAs by its share of the work, and the two
// kernels run side by side on their SMs (one bound by products, one by bytes).
//
// The list holds the sequences (or groups) and their blocks in order, once per KV head: the
// heads innermost for prompts, so that the CTAs that read the same entries for different
// blocks read them at about the same time (512 tokens on a 60k context, whose K and V do
// not fit in L2: 413 -> 369 us), and outermost otherwise, so that a run holds items of
// different lengths and what the units get wrong evens out (64 slots of 1 to 1024 entries:
// 47 -> 40 us).  A block's units are its tiles and what its start and end cost;
// a sequence's units have a closed form, so that a CTA finds its run with one load per
// sequence, a prefix sum over the sequences, and a search within one of them.
#pragma once

#include "pnb_pkv.cuh"

namespace pnb {

constexpr int kPkvMinRun = 4;      // units that a CTA starts for

// a sequence, or in the prefix's pass a group
struct PkvSeq {
  int t0, n;                // its tokens
  int len;                  // its entries (the prefix's whole pages)
  int floor;                // entries below are the prefix's, another pass's
  int lo, lo_max;           // prefix: entries that some row, and that every row sees, start here
};

struct PkvItem {
  int b, j, h;              // sequence or group, block, KV head
  int tok0, ntok;           // its tokens
  int base;                 // first token's last entry (not the prefix's pass)
  int hi, lo;               // entries [lo, hi): those that some row sees
  int hi_min, lo_max;       // entries [lo_max, hi_min): those that every row sees
  int len, floor;           // of its sequence
  int t0, nt;               // tiles of the whole item
  int ta, tb;               // this CTA's tiles
  bool ends;                // the item's end is this CTA's
};

__device__ __forceinline__ PkvSeq pkv_seq(const PkvAttnArgs &a, int pass, int b) {
  PkvSeq s{};
  const int W = a.window;
  if (pass == kPkvPrefix) {
    const int gs = min(max(a.group_start[b], 0), a.seqs.n_seq), ge = min(max(a.group_start[b + 1], gs), a.seqs.n_seq);
    s.t0 = gs * a.seqs.each;
    s.n = (ge - gs) * a.seqs.each;
    const PkvGroup g = a.groups[b];
    s.len = g.prefix;
    s.lo = W > 0 ? min(max(0, g.len_min - a.seqs.each - W + 1), g.prefix) : 0;
    s.lo_max = W > 0 ? max(0, g.len_max - W) : 0;
  } else {
    pkv_tokens(a.seqs, b, s.t0, s.n);
    s.len = pkv_len(a.seqs, a.pool.page_log2, b, a.err);
    if (pass == kPkvOwn) {
      const int g = pkv_group_of(a.group_start, a.n_group, b);
      s.floor = g < 0 ? 0 : min(a.groups[g].prefix, max(s.len - s.n, 0));
    }
  }
  return s;
}

// a sequence's j-th block (j * TB < n)
template <int TILE>
__device__ __forceinline__ void pkv_block(const PkvAttnArgs &a, int pass, const PkvSeq &s, int TB, int b, int j,
                                          PkvItem &it) {
  const int W = a.window;
  it.b = b;
  it.j = j;
  it.tok0 = s.t0 + j * TB;
  it.ntok = min(TB, s.n - j * TB);
  it.len = s.len;
  it.floor = s.floor;
  if (pass == kPkvPrefix) {
    it.base = 0;
    it.hi = it.hi_min = s.len;
    it.lo = s.lo;
    it.lo_max = s.lo_max;
  } else {
    it.base = s.len - s.n + j * TB;
    it.hi = max(0, it.base + it.ntok);
    it.hi_min = it.base + 1;
    // (before entry 0 a window starts at no entry either: what may be far below 0 is left out)
    it.lo = max(s.floor, W > 0 ? max(it.base, 0) - W + 1 : 0);
    it.lo_max = max(s.floor, W > 0 ? max(it.base + it.ntok, 0) - W : 0);
  }
  it.t0 = it.lo / TILE;
  it.nt = max(1, (it.hi + TILE - 1) / TILE - it.t0);
}

// sum of floor((a i + b) / m) for i = 0 .. n - 1 (the steps of Euclid's algorithm on a and
// m); a n + b below 2^32 once a and b are below m
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  unsigned long long sum = 0;
  while (n > 0) {
    if (a >= m) {
      sum += (unsigned long long)n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += (unsigned long long)n * (b / m);
      b %= m;
    }
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return (long long)sum;
}

__device__ __forceinline__ int pkv_blocks(const PkvSeq &s, int TB) { return (s.n + TB - 1) / TB; }

// units of a sequence's first J blocks, per KV head; `each` of them for an item's start and end
template <int TILE>
__device__ __forceinline__ long long pkv_units(const PkvAttnArgs &a, int pass, int each, const PkvSeq &s, int TB, int J) {
  if (J <= 0) return 0;
  PkvItem it;
  if (pass == kPkvPrefix) {
    pkv_block<TILE>(a, pass, s, TB, 0, 0, it);
    return (long long)J * (it.nt + each);
  }
  // the last block may have fewer tokens
  long long sum = 0;
  int K = J;
  if (J == pkv_blocks(s, TB)) {
    pkv_block<TILE>(a, pass, s, TB, 0, J - 1, it);
    sum = it.nt;
    --K;
  }
  if (K > 0) {
    const int base = s.len - s.n;
    // blocks z .. K - 1 end behind entry base + (j + 1) TB; those before see nothing: a tile each
    const int z = base < 0 ? min(K, -base / TB) : 0;
    sum += z;
    if (K > z) sum += floor_sum(K - z, TILE, TB, base + (z + 1) * TB + TILE - 1);
    // first entries: the floor, and from block y on the window's
    int y = K;
    if (a.window > 0) {
      const int64_t d = (int64_t)s.floor + a.window - 1 - base;   // base + j TB - window + 1 > floor
      y = d < 0 ? z : (int)min((int64_t)K, max((int64_t)z, d / TB + 1));
    }
    sum -= (long long)(y - z) * (s.floor / TILE);
    if (K > y) sum -= floor_sum(K - y, TILE, TB, base + y * TB - a.window + 1);
  }
  return sum + (long long)J * each;
}

// a CTA's way through its run of units
struct PkvWalk {
  int b, j, h, x;       // next item, units of it that lie before the run
  int n_b;              // sequences or groups
  int64_t left;         // units
  PkvSeq seq;           // sequence b

  template <int TILE>
  __device__ __forceinline__ bool next(const PkvAttnArgs &a, int TB, PkvItem &it) {
    while (left > 0) {
      if (a.heads_inner && h == a.pool.n_kv) {
        h = 0;
        ++j;
      }
      while (j * TB >= seq.n) {
        j = 0;
        if (++b == n_b) {
          b = 0;
          if (a.heads_inner || ++h == a.pool.n_kv) return false;
        }
        seq = pkv_seq(a, a.pass, b);
      }
      pkv_block<TILE>(a, a.pass, seq, TB, b, j, it);
      const int units = it.nt + a.item_units;
      const int end = (int)min((int64_t)units, x + left);
      it.h = h;
      it.ta = max(0, x - a.item_units);
      it.tb = max(0, end - a.item_units);
      it.ends = end == units;
      left -= end - x;
      x = end;
      if (it.ends) {
        x = 0;
        if (a.heads_inner) ++h;
        else ++j;
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
    const int n = pkv_len(a.seqs, a.pool.page_log2, s, a.err);
    const int g = pkv_group_of(a.group_start, a.n_group, s);
    if (g < 0) {
      set_error(a.err, kErrRange);
      continue;
    }
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

// Inclusive prefix sum over the CTA's threads; `all` gets their sum.  scratch: 32 numbers.
template <int THREADS>
__device__ __forceinline__ long long pkv_scan(long long v, long long *scratch, long long &all) {
  constexpr int WARPS = THREADS / 32;
  static_assert(WARPS <= 32, "warps");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  long long w = lane < WARPS ? scratch[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  return v + (warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
}

// The work of the pass that runs beside this one, in nanoseconds of an SM.
template <int THREADS>
__device__ __forceinline__ long long pkv_other_work(const PkvAttnArgs &a, long long *scratch) {
  const int pass = a.pass == kPkvPrefix ? kPkvOwn : kPkvPrefix, n = pass == kPkvPrefix ? a.n_group : a.seqs.n_seq;
  long long mine = 0, all;
  for (int b = threadIdx.x; b < n; b += THREADS) {
    const PkvSeq s = pkv_seq(a, pass, b);
    const int TB = a.other_tile == kPkvTile ? a.block_rows / (a.n_head / a.pool.n_kv) : a.seqs.each;
    mine += a.other_tile == kPkvTile ? pkv_units<kPkvTile>(a, pass, a.other_item_units, s, TB, pkv_blocks(s, TB))
                                     : pkv_units<kPkvChunk>(a, pass, a.other_item_units, s, TB, pkv_blocks(s, TB));
  }
  pkv_scan<THREADS>(mine, scratch, all);
  return all * a.other_ns;
}

// Where this CTA's run starts (every warp answers for itself).  scratch: 64 numbers.
template <int TILE, int THREADS>
__device__ __forceinline__ PkvWalk pkv_find_run(const PkvAttnArgs &a, int TB, long long *scratch) {
  constexpr int PASSES = (kPkvMaxSeq + THREADS - 1) / THREADS;
  const int n_b = a.pass == kPkvPrefix ? a.n_group : a.seqs.n_seq, tid = threadIdx.x, lane = tid & 31;
  long long before[PASSES], units[PASSES], total = 0;
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    before[k] = units[k] = 0;
    if (k * THREADS >= n_b) continue;   // (the same for all threads)
    const int b = k * THREADS + tid;
    if (b < n_b) {
      const PkvSeq s = pkv_seq(a, a.pass, b);
      units[k] = pkv_units<TILE>(a, a.pass, a.item_units, s, TB, pkv_blocks(s, TB));
    }
    long long all;
    before[k] = total + pkv_scan<THREADS>(units[k], scratch, all) - units[k];
    total += all;
  }
  // as many CTAs as get a run of a few units each, and this pass's share of them
  const int n_kv = a.pool.n_kv;
  const long long list = total * n_kv;
  long long ctas = gridDim.x;
  if (a.pass != kPkvAll) {
    const long long here = total * a.unit_ns, there = pkv_other_work<THREADS>(a, scratch);
    // (the prefix's pass rounds down and the other one up)
    const long long prefix = a.pass == kPkvPrefix ? here : there;
    ctas = max(1ll, min(ctas - 1, ctas * prefix / max(here + there, 1ll)));
    if (a.pass == kPkvOwn) ctas = gridDim.x - ctas;
  }
  ctas = max(1ll, min(ctas, list / kPkvMinRun));
  const long long c = min((long long)blockIdx.x, ctas), u0 = list * c / ctas, u1 = list * min(c + 1, ctas) / ctas;
  PkvWalk r{};
  r.n_b = n_b;
  if (u1 <= u0) return r;
  // in units of one KV head: which sequence, which block
  if (!a.heads_inner) r.h = (int)(u0 / total);
  const long long at = a.heads_inner ? u0 / n_kv : u0 - r.h * total;
#pragma unroll
  for (int k = 0; k < PASSES; ++k)
    if (at >= before[k] && at < before[k] + units[k]) {
      scratch[40] = k * THREADS + tid;
      scratch[41] = before[k];
    }
  __syncthreads();
  r.b = (int)scratch[40];
  r.seq = pkv_seq(a, a.pass, r.b);
  const long long in_seq = at - scratch[41];
  // the last block j with units(j) <= in_seq: 32 candidates at a time
  int lo = 0, hi = pkv_blocks(r.seq, TB);
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, j = lo + lane * step;
    const bool in = j < hi && pkv_units<TILE>(a, a.pass, a.item_units, r.seq, TB, j) <= in_seq;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, in));
    lo += k * step;
    hi = min(hi, lo + step);
  }
  r.j = lo;
  const long long block = pkv_units<TILE>(a, a.pass, a.item_units, r.seq, TB, lo);
  if (a.heads_inner) {
    PkvItem it;
    pkv_block<TILE>(a, a.pass, r.seq, TB, r.b, lo, it);
    const long long rest = u0 - (scratch[41] + block) * n_kv;   // of the block, over its heads
    r.h = (int)(rest / (it.nt + a.item_units));
    r.x = (int)(rest % (it.nt + a.item_units));
  } else {
    r.x = (int)(in_seq - block);
  }
  r.left = u1 - u0;
  return r;
}

}  // namespace pnb
