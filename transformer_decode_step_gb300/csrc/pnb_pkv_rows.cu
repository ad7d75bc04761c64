// pnb_pkv_rows.cu - attention over the paged KV cache on tcgen05 tensor cores, for
// blocks of up to 256 rows (token, query head) that share a KV head's entries:
// prompts, prompt chunks, and the shared prefix of a group of sequences.
//
// Row i attends to entries [lo_i, hi_i).  With x_ij = q_i.k_j log2(e) / sqrt(hd) and a
// reference r_i, p_ij = 2^(x_ij - r_i), l_i = sum_j p_ij, o_i = sum_j p_ij v_j / l_i.
// r_i only moves when a tile's largest score passes it by 2^8, so that sums and
// outputs are rarely rescaled; p stays below 2^8 and sums are held in fp32.
//
// One CTA per SM works through a run of (block, 128-entry tile) units:
//   warps 0-3, 4-7  softmax of the block's rows 0-127 and 128-255, one row per thread:
//                   S from tensor memory, masks, reference, p as bf16 back over S;
//   warp 8          K and V tiles by tiled TMA loads of a page's rows each, into a ring;
//   warp 9          S = Q K^T (both operands in shared memory) and O += P V (P in tensor
//                   memory), the two halves in turn, so that one half's softmax runs
//                   beside the other's products;
//   warps 10, 11    V rows that no row of the block sees become zero (0 x NaN is NaN), and
//                   tiles that some rows see only in part are searched for NaN and
//                   infinities: a block that has one is done again row by row.
// Tensor memory (512 columns): S of both halves (128 each), O of both halves.
//
// fp32 on either side (SPLIT): Q and P enter as two bf16 numbers, high and low part, in
// twice the products.
#include <cuda_bf16.h>
#include <math.h>

#include "pnb_pkv.cuh"
#include "pnb_tc.cuh"

namespace pnb {
namespace {

extern __shared__ __align__(1024) uint8_t r_smem[];

constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;
constexpr int kBadSlots = 8;       // items that the V search may be ahead of the softmax, and more
constexpr float kTau = 8.f;
// the V search waits for a tile that may be a whole item away
constexpr unsigned long long kItemLimitNs = 10000000000ull;
// registers per thread: 384 x 168 at launch = 256 x 216 + 128 x 72
constexpr int kRegsSoft = 216, kRegsRest = 72;

template <int HD, bool SPLIT>
struct RL {
  static constexpr int NB = HD / 64;                        // 64-column boxes of a row
  static constexpr int BOX = kPkvTile * 128;                // bytes of a 128-row box
  static constexpr int UNIT = NB * BOX;                     // a K or V tile
  static constexpr int QHALF = UNIT * (SPLIT ? 2 : 1);      // Q of 128 rows (high, then low parts)
  static constexpr int NU = (229376 - 2 * QHALF) / UNIT;    // ring units
  static constexpr int SMEM = 1024 + 2 * QHALF + NU * UNIT + 1024;
};

struct RItem {
  int b, j, h;              // sequence or group, block, KV head
  int tok0, ntok;           // its tokens
  int base;                 // first token's last entry (prompts)
  int hi, lo;               // entries [lo, hi): those that some row sees
  int hi_min, lo_max;       // entries [lo_max, hi_min): those that every row sees
  int t0, nt;               // tiles of the whole item
  int ta, tb;               // this CTA's tiles
  bool ends;                // the item's end is this CTA's
};

// the j-th block of a sequence or group; false behind the last one
__device__ __forceinline__ bool block_of(const PkvAttnArgs &a, int TB, int b, int j, RItem &it) {
  int t0, n;
  if (a.groups) {
    const int gs = min(max(a.group_start[b], 0), a.seqs.n_seq), ge = min(max(a.group_start[b + 1], gs), a.seqs.n_seq);
    t0 = gs * a.seqs.each;
    n = (ge - gs) * a.seqs.each;
  } else {
    pkv_tokens(a.seqs, b, t0, n);
  }
  if (j * TB >= n) return false;
  it.b = b;
  it.j = j;
  it.tok0 = t0 + j * TB;
  it.ntok = min(TB, n - j * TB);
  const int W = a.window;
  if (a.groups) {
    const PkvGroup g = a.groups[b];
    it.base = 0;
    it.hi = it.hi_min = g.prefix;
    it.lo = W > 0 ? min(max(0, g.len_min - a.seqs.each - W + 1), g.prefix) : 0;
    it.lo_max = W > 0 ? max(0, g.len_max - W) : 0;
  } else {
    it.base = pkv_len(a.seqs, a.pool.page_log2, b, a.err) - n + j * TB;
    it.hi = max(0, it.base + it.ntok);
    it.hi_min = it.base + 1;
    it.lo = W > 0 ? max(0, it.base - W + 1) : 0;
    it.lo_max = W > 0 ? max(0, it.base + it.ntok - W) : 0;
  }
  it.t0 = it.lo / kPkvTile;
  it.nt = max(1, (it.hi + kPkvTile - 1) / kPkvTile - it.t0);
  return true;
}

// a CTA's way through its run of units
struct RWalk {
  int h, b, j, x;       // next item, units of it that lie before the run
  int64_t left;         // units
  int n_b;              // sequences or groups

  __device__ __forceinline__ bool next(const PkvAttnArgs &a, int TB, RItem &it) {
    while (left > 0 && h < a.pool.n_kv) {
      if (!block_of(a, TB, b, j, it)) {
        j = 0;
        if (++b == n_b) {
          b = 0;
          ++h;
        }
        continue;
      }
      const int units = it.nt + kPkvItemUnits;
      const int end = (int)min((int64_t)units, x + left);
      it.h = h;
      it.ta = max(0, x - kPkvItemUnits);
      it.tb = max(0, end - kPkvItemUnits);
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
__device__ void find_groups(const PkvAttnArgs &a, int *scratch) {
  int *gmin = scratch, *gmax = scratch + a.n_group;
  for (int g = threadIdx.x; g < a.n_group; g += kThreads) {
    gmin[g] = INT_MAX;
    gmax[g] = 0;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < a.seqs.n_seq; s += kThreads) {
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
  for (int g = threadIdx.x; g < a.n_group; g += kThreads) {
    const int p = min(max(a.prefix[g], 0), max(0, gmin[g] - a.seqs.each));
    a.groups[g] = PkvGroup{p >> a.pool.page_log2 << a.pool.page_log2, gmin[g], gmax[g], 0};
  }
  __syncthreads();
}

// Where this CTA's run starts.  The blocks of one KV head are counted and their
// units added up by all threads; heads follow one another in the list.
__device__ void find_run(const PkvAttnArgs &a, int TB, int *scratch, RWalk *out) {
  const int n_b = a.groups ? a.n_group : a.seqs.n_seq, tid = threadIdx.x, lane = tid & 31;
  int *first = scratch;                                             // [n_b + 1] blocks before a sequence
  long long *sums = reinterpret_cast<long long *>(scratch + 1026);   // [kThreads + 1]
  for (int b = tid; b < n_b; b += kThreads) {
    int t0, n;
    if (a.groups) {
      const int gs = min(max(a.group_start[b], 0), a.seqs.n_seq);
      n = (min(max(a.group_start[b + 1], gs), a.seqs.n_seq) - gs) * a.seqs.each;
    } else {
      pkv_tokens(a.seqs, b, t0, n);
    }
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
  const int i0 = (int)((int64_t)blocks * tid / kThreads), i1 = (int)((int64_t)blocks * (tid + 1) / kThreads);
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
      RItem it;
      while (!block_of(a, TB, b, j, it)) {
        ++b;
        j = 0;
      }
      if (!f(b, j, it.nt + kPkvItemUnits)) return;
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
    for (int k0 = 1; k0 <= kThreads; k0 += 32) {
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
  const long long per_head = sums[kThreads], total = per_head * a.pool.n_kv;
  const int ctas = gridDim.x;
  const long long u0 = total * blockIdx.x / ctas, u1 = total * (blockIdx.x + 1) / ctas;
  if (u1 <= u0) {
    if (tid == 0) *out = RWalk{0, 0, 0, 0, 0, n_b};
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
        *out = RWalk{h, b, j, (int)(in_head - at), u1 - u0, n_b};
        return false;
      });
    }
  }
  __syncthreads();
}

struct RBars {
  uint64_t full[16], empty[16], q_ready[2], s_full[2], p_ready[2], o_full[2], v_go, v_ok, drain;
  uint32_t tmem, pad;
  int bad[kBadSlots];
  RWalk walk;
};
static_assert(sizeof(RBars) <= 1024, "barriers");

// 8 elements of a query row as bf16, and with SPLIT what the rounding left
template <bool SPLIT>
__device__ __forceinline__ void load_q8(const DevRows &q, int64_t at, uint4 &hi, uint4 &lo) {
  if (q.dtype == PNB_BF16) {
    hi = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(q.p) + at);
    lo = make_uint4(0, 0, 0, 0);
    return;
  }
  float f[8];
  const float *p = static_cast<const float *>(q.p) + at;
  load_vals<float, 4>(p, reinterpret_cast<float(&)[4]>(f[0]));
  load_vals<float, 4>(p + 4, reinterpret_cast<float(&)[4]>(f[4]));
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    l[i] = pack_bf16(f[2 * i] - bf16lo(h[i]), f[2 * i + 1] - bf16hi(h[i]));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

template <int HD, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_pkv_rows(const __grid_constant__ CUtensorMap kvmap, const PkvAttnArgs a) {
  typedef RL<HD, SPLIT> L;
  constexpr int NU = L::NU;
  static_assert(NU <= 16 && NU >= 2, "ring");
  uint8_t *sm = r_smem + ((1024u - (smem_addr(r_smem) & 1023u)) & 1023u);
  uint8_t *Q = sm, *ring = sm + 2 * L::QHALF;
  RBars &bar = *reinterpret_cast<RBars *>(ring + NU * L::UNIT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.n_head / a.pool.n_kv, TB = kPkvBlockRows / G;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NU; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_ready[i], 4);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_ready[i], 4);
      mbar_init(&bar.o_full[i], 1);
    }
    mbar_init(&bar.v_go, 1);
    mbar_init(&bar.v_ok, 64);
    mbar_init(&bar.drain, 1);
    for (int i = 0; i < kBadSlots; ++i) bar.bad[i] = 0;
    fence_barrier_init();
    bar.walk = RWalk{0, 0, 0, 0, 0, 1};
  }
  if (warp == 9) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 2) a.part[2 * blockIdx.x + threadIdx.x].flags = 0;
  if (a.groups) find_groups(a, reinterpret_cast<int *>(ring));
  find_run(a, TB, reinterpret_cast<int *>(ring), &bar.walk);
  RWalk walk = bar.walk;
  RItem it;
  const uint32_t tmem = bar.tmem;
  const uint32_t t_s[2] = {tmem, tmem + 128}, t_o[2] = {tmem + 256, tmem + 384};
  // the ring held the schedule's sums: order them before the tiles that TMA writes
  fence_async_smem();
  __syncthreads();

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == 8) {
      // ------------------------------------------------------ K and V tiles
      bool ok = true;
      uint32_t u = 0;   // units issued
      const int log2p = a.pool.page_log2, per_tile = kPkvTile >> log2p, page = 1 << log2p;
      const int rows_total = a.pool.n_page * 2 * a.pool.n_kv << log2p;
      while (ok && walk.next(a, TB, it)) {
        // page ids are the first sequence's of a group
        const int seq = a.groups ? min(max(a.group_start[it.b], 0), a.seqs.n_seq - 1) : it.b;
        const int32_t *pages = a.seqs.pages + (int64_t)seq * a.seqs.max_page;
        auto page_id = [&](int t) {
          const int e = (it.t0 + t) * kPkvTile + (lane << log2p);
          return lane < per_tile && e < it.hi && e + page > it.lo ? pages[e >> log2p] : -1;
        };
        int id = page_id(it.ta);
        for (int t = it.ta; t < it.tb && ok; ++t) {
          const int e = (it.t0 + t) * kPkvTile + (lane << log2p);
          const bool needed = lane < per_tile && e < it.hi && e + page > it.lo;
          const bool good = id >= 0 && id < a.pool.n_page;
          if (needed && !good) set_error(a.err, kErrRange);
          const int now = id;
          if (t + 1 < it.tb) id = page_id(t + 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++u) {
            const int s = u % NU;
            if (u >= NU && !mbar_wait(&bar.empty[s], (u / NU - 1) & 1)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&bar.full[s], L::UNIT);
            __syncwarp();
            if (lane < per_tile) {
              // rows behind the pool's end read as zero
              const int y = needed && good ? ((now * 2 + kv) * a.pool.n_kv + it.h) << log2p : rows_total;
              uint8_t *dst = ring + s * L::UNIT + (lane << log2p) * 128;
#pragma unroll
              for (int c = 0; c < L::NB; ++c) tma_load_2d(dst + c * L::BOX, &kvmap, c * 64, y, &bar.full[s]);
            }
          }
        }
      }
      if (!ok) {
        if (lane == 0) set_error(a.err, kErrTimeout);
        // what is still on its way lands before the CTA ends
        for (uint32_t i = u > NU ? u - NU : 0; i < u; ++i) mbar_wait(&bar.full[i % NU], (i / NU) & 1);
      }
    } else if (warp == 9) {
      // ----------------------------------------------------------- products
      if (lane == 0) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, kPkvTile);
        constexpr uint32_t idesc_o = idesc_bf16_f32(128, HD) | (1u << 16);   // V: N contiguous
        bool ok = true;
        uint32_t u = 0, nq[2] = {0, 0}, np[2] = {0, 0}, nv = 0;
        auto issue_s = [&](int w, int s) {
          const uint8_t *k = ring + s * L::UNIT, *q = Q + w * L::QHALF;
#pragma unroll
          for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
            for (int c = 0; c < L::NB; ++c)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                mma_bf16(t_s[w], desc_k_sw128(q + part * L::UNIT + c * L::BOX, x * 32),
                         desc_k_sw128(k + c * L::BOX, x * 32), idesc_s, part > 0 || c > 0 || x > 0);
          mma_commit(&bar.s_full[w]);
        };
        auto issue_o = [&](int w, int s, bool first) {
          const uint8_t *v = ring + s * L::UNIT;
#pragma unroll
          for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
            for (int x = 0; x < kPkvTile / 16; ++x)
              mma_bf16_ts(t_o[w], t_s[w] + part * 64 + x * 8, desc_mn_sw128(v + x * 2048, L::BOX), idesc_o,
                          !first || part > 0 || x > 0);
        };
        while (ok && walk.next(a, TB, it)) {
          const int halves = it.ntok * G > 128 ? 2 : 1;
          for (int w = 0; w < halves && ok; ++w) {
            ok = mbar_wait(&bar.q_ready[w], nq[w]++ & 1) && (w || mbar_wait(&bar.full[u % NU], (u / NU) & 1));
            if (!ok) break;
            tc_fence_after();
            issue_s(w, u % NU);
          }
          if (ok) mma_commit(&bar.empty[u % NU]);
          ++u;
          for (int t = it.ta; t < it.tb && ok; ++t) {
            // u: this tile's V; u + 1: the next one's K
            const int sv = u % NU, sk = (u + 1) % NU;
            const bool more = t + 1 < it.tb;
            const int e = (it.t0 + t) * kPkvTile;
            ok = mbar_wait(&bar.full[sv], (u / NU) & 1);
            if (ok && (e < it.lo_max || e + kPkvTile > it.hi_min)) {
              mbar_arrive(&bar.v_go);
              ok = mbar_wait(&bar.v_ok, nv++ & 1);
            }
            for (int w = 0; w < halves && ok; ++w) {
              ok = mbar_wait(&bar.p_ready[w], np[w]++ & 1);
              if (!ok) break;
              tc_fence_after();
              issue_o(w, sv, t == it.ta);
              if (!more) mma_commit(&bar.o_full[w]);
              if (w == halves - 1) mma_commit(&bar.empty[sv]);
              if (more) {
                if (w == 0) ok = mbar_wait(&bar.full[sk], ((u + 1) / NU) & 1);
                if (!ok) break;
                issue_s(w, sk);
                if (w == halves - 1) mma_commit(&bar.empty[sk]);
              }
            }
            u += more ? 2 : 1;
          }
        }
        if (!ok) {
          set_error(a.err, kErrTimeout);
          mma_commit(&bar.drain);   // the products in flight end before tensor memory is given back
          mbar_wait(&bar.drain, 0);
        }
      }
      __syncwarp();
    } else {
      // --------------------------------------------- V rows that are not seen
      const int tid = threadIdx.x - 320;
      bool ok = true;
      uint32_t u = 0, item = 0, nv = 0;
      while (ok && walk.next(a, TB, it)) {
        for (int t = it.ta; t < it.tb && ok; ++t, u += 2) {
          const int e0 = (it.t0 + t) * kPkvTile;
          if (e0 >= it.lo_max && e0 + kPkvTile <= it.hi_min) continue;
          const int s = (u + 1) % NU;
          // (the ring's own barriers would not do: this warp skips tiles, and the ring
          // may be a whole turn ahead or behind)
          ok = mbar_wait_for(&bar.v_go, nv++ & 1, kItemLimitNs);
          if (!ok) break;
          uint8_t *v = ring + s * L::UNIT;
          bool bad = false;
          for (int i = tid; i < L::UNIT / 16; i += 64) {
            const int e = e0 + ((i >> 3) & (kPkvTile - 1));
            uint4 *p = reinterpret_cast<uint4 *>(v) + i;
            if (e >= it.hi || e < it.lo) {
              *p = make_uint4(0, 0, 0, 0);
            } else {
              const uint4 x = *p;
              // an exponent of ones in either half of a word
              auto odd = [](uint32_t w) {
                return (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u;
              };
              bad |= odd(x.x) || odd(x.y) || odd(x.z) || odd(x.w);
            }
          }
          if (bad) *reinterpret_cast<volatile int *>(&bar.bad[item % kBadSlots]) = (int)item + 1;
          fence_async_smem();
          mbar_arrive(&bar.v_ok);
        }
        ++item;
      }
      if (!ok && lane == 0) set_error(a.err, kErrTimeout);
    }
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int w = warp >> 2, quad = warp & 3, r = (warp << 5) + lane;   // r: row of the block
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t ts = t_s[w] + lanes, to = t_o[w] + lanes;
    const float c = a.qscale;
    uint32_t ns = 0, no = 0, item = 0;
    bool ok = true;

    // the warp's 32 query rows of an item into shared memory
    auto load_q = [&](const RItem &x) {
      constexpr int LPR = HD / 8, RPW = 32 / LPR;   // lanes per row, rows at a time
      const int l = lane % LPR, sub = lane / LPR;
      uint8_t *q = Q + w * L::QHALF;
#pragma unroll 4
      for (int k = 0; k < 32; k += RPW) {
        const int row = (warp << 5) + k + sub;
        uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
        if (row < x.ntok * G) {
          const int tok = x.tok0 + row / G, head = x.h * G + row % G;
          load_q8<SPLIT>(a.q, tok * a.q.token + head * a.q.head + 8 * l, hi, lo);
        }
        uint8_t *p = q + (l >> 3) * L::BOX + sw128(row & 127, (l & 7) * 16);
        *reinterpret_cast<uint4 *>(p) = hi;
        if (SPLIT) *reinterpret_cast<uint4 *>(p + L::UNIT) = lo;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_ready[w]);
    };
    // the next item with rows for this half
    auto next = [&](RItem &x) {
      while (walk.next(a, TB, x)) {
        ++item;
        if (x.ntok * G > 128 * w) return true;
      }
      return false;
    };

    bool have = next(it);
    if (have) load_q(it);
    while (have && ok) {
      const bool live = r < it.ntok * G;
      const int tok = it.tok0 + (live ? r / G : 0), head = it.h * G + (live ? r % G : 0);
      int lo = it.lo, hi = it.hi;
      if (a.groups) {
        if (a.window > 0) {
          const int seq = tok / a.seqs.each;
          const int last = pkv_len(a.seqs, a.pool.page_log2, seq, a.err) - a.seqs.each + tok % a.seqs.each;
          lo = max(0, last - a.window + 1);
        }
      } else {
        const int last = it.base + (tok - it.tok0);
        hi = last + 1;
        if (a.window > 0) lo = max(0, last - a.window + 1);
      }
      float m = -INFINITY, sum = 0.f;
      for (int t = it.ta; t < it.tb; ++t) {
        if (!mbar_wait(&bar.s_full[w], ns++ & 1)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32_async(ts + 32 * i, s + 32 * i);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_landed(s + 32 * i);
        const int e = (it.t0 + t) * kPkvTile;
        if (e < it.lo_max || e + kPkvTile > it.hi_min) {
          // columns [from, from + n) of the tile are this row's
          const int from = max(lo - e, 0), n = max(min(hi - e, kPkvTile) - from, 0);
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if ((unsigned)(i - from) >= (unsigned)n) s[i] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 124; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], s[i + k]), s[i + k + 4]);
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[124 + k]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        const bool move = top > m + kTau;
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? (m == -INFINITY ? 0.f : exp2_approx(m - top)) : 1.f;
          if (move) m = top;
          sum *= f;
          if (t > it.ta) {
            // the products of the tile before are done: S of this one came behind them
#pragma unroll 1
            for (int i = 0; i < HD; i += 32) {
              float o[32];
              tmem_ld32_async(to + i, o);
              tmem_wait_ld();
              tmem_landed(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= f;
              tmem_st32_async(to + i, reinterpret_cast<const uint32_t *>(o));
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;   // nothing seen yet: every p is 2^-inf
        const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
        float2 acc[4] = {};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float2 x = make_float2(s[64 * half + 2 * i], s[64 * half + 2 * i + 1]);
            x = ffma2(x, c2, r2);
            x.x = exp2_approx(x.x);
            x.y = exp2_approx(x.y);
            acc[i & 3] = fadd2(acc[i & 3], x);
            p[i] = pack_bf16(x.x, x.y);
            if (SPLIT) {
              s[64 * half + 2 * i] = x.x - bf16lo(p[i]);
              s[64 * half + 2 * i + 1] = x.y - bf16hi(p[i]);
            }
          }
          tmem_st32_async(ts + 32 * half, p);
          if (SPLIT) {
#pragma unroll
            for (int i = 0; i < 32; ++i) p[i] = pack_bf16(s[64 * half + 2 * i], s[64 * half + 2 * i + 1]);
            tmem_st32_async(ts + 64 + 32 * half, p);
          }
        }
        acc[0] = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
        sum += acc[0].x + acc[0].y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_ready[w]);
      }
      if (!ok) break;
      // the next item's queries go where this one's lay: its last S is done
      const uint32_t id = item;
      RItem nx;
      have = next(nx);
      if (have) load_q(nx);

      if (!mbar_wait(&bar.o_full[w], no++ & 1)) {
        ok = false;
        break;
      }
      __syncwarp();
      tc_fence_after();
      const bool redo = *reinterpret_cast<volatile int *>(&bar.bad[(id - 1) % kBadSlots]) == (int)id;
      const bool whole = it.ta == 0 && it.ends;
      const int side = it.ta > 0 ? 0 : 1;   // of the run's two partial sums
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      float *po = nullptr, *pml = nullptr;
      if (!whole) {
        const int64_t at = (int64_t)(2 * blockIdx.x + side) * kPkvBlockRows + r;
        po = a.part_o + at * HD;
        pml = a.part_ml + at * 2;
        if (r == 0) a.part[2 * blockIdx.x + side] = PkvPart{it.ends ? 3 : 1, it.b, it.j, it.h};
      } else if (a.groups) {
        const int64_t at = (int64_t)tok * a.n_head + head;
        po = a.row_o + at * HD;
        pml = a.row_ml + at * 2;
      }
      if (!redo) {
#pragma unroll 1
        for (int i = 0; i < HD; i += 32) {
          float o[32];
          tmem_ld32_async(to + i, o);
          tmem_wait_ld();
          tmem_landed(o);
          if (live && po) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4 *>(po + i + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          } else if (live) {
            // a row that saw nothing has only zeros summed up
            pkv_store<32>(a.out, tok * a.out.token + head * a.out.head + i, o, inv);
          }
          __syncwarp();
        }
        if (live && po) *reinterpret_cast<float2 *>(pml) = make_float2(m, sum);
      } else {
        // a NaN or an infinity among values that only some rows see: each row by itself
        const int seq = a.groups ? min(max(a.group_start[it.b], 0), a.seqs.n_seq - 1) : it.b;
        for (int k = 0; k < 32; ++k) {
          const int from = max(__shfl_sync(0xffffffffu, lo, k), (it.t0 + it.ta) * kPkvTile);
          const int to_e = min(__shfl_sync(0xffffffffu, hi, k), (it.t0 + it.tb) * kPkvTile);
          const int tk = __shfl_sync(0xffffffffu, tok, k), hd_k = __shfl_sync(0xffffffffu, head, k);
          const long long po_k = __shfl_sync(0xffffffffu, (long long)(uintptr_t)po, k);
          const long long pml_k = __shfl_sync(0xffffffffu, (long long)(uintptr_t)pml, k);
          if (!__shfl_sync(0xffffffffu, (int)live, k)) continue;
          float o[HD / 32], mk, lk;
          pkv_attend_row<HD>(a.pool, a.seqs.pages + (int64_t)seq * a.seqs.max_page, it.h, a.q,
                             tk * a.q.token + hd_k * a.q.head, c, from, to_e, o, mk, lk);
          if (po_k) {
            float *dst = reinterpret_cast<float *>((uintptr_t)po_k);
#pragma unroll
            for (int i = 0; i < HD / 32; ++i) dst[lane * (HD / 32) + i] = o[i];
            if (lane == 0) *reinterpret_cast<float2 *>((uintptr_t)pml_k) = make_float2(mk, lk);
          } else {
            const float d = to_e > from ? 1.f / lk : 0.f;
            pkv_store<HD / 32>(a.out, tk * a.out.token + hd_k * a.out.head + lane * (HD / 32), o, d);
          }
        }
      }
      tc_fence_before();
      it = nx;
    }
    if (!ok && lane == 0) set_error(a.err, kErrTimeout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Adds up the parts of the items that several CTAs shared, in the list's order.  The
// CTA whose run holds an item's first tiles has it in its second partial sum; the
// runs behind it hold the rest in their first ones.  A warp per row.
template <int HD>
__global__ void __launch_bounds__(256) k_pkv_join(const PkvAttnArgs a) {
  constexpr int N = HD / 32;
  const int lane = threadIdx.x & 31, c0 = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const PkvPart p = a.part[2 * c0 + 1];
  if (!(p.flags & 1)) return;
  const int G = a.n_head / a.pool.n_kv, TB = kPkvBlockRows / G;
  RItem it;
  if (!block_of(a, TB, p.b, p.j, it)) return;
  int last = c0;   // the run that ends the item
  if (!(p.flags & 2))
    for (last = c0 + 1; last < a.grid - 1 && !(a.part[2 * last].flags & 2);) ++last;
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < it.ntok * G; r += 8 * gridDim.y) {
    float m = -INFINITY;
    for (int k = c0; k <= last; ++k) {
      const int slot = k == c0 ? 2 * k + 1 : 2 * k;
      if (!(a.part[slot].flags & 1)) continue;   // (a run without units)
      m = fmaxf(m, a.part_ml[((int64_t)slot * kPkvBlockRows + r) * 2]);
    }
    const float ref = m == -INFINITY ? 0.f : m;
    float o[N] = {}, sum = 0.f;
    for (int k = c0; k <= last; ++k) {
      const int slot = k == c0 ? 2 * k + 1 : 2 * k;
      if (!(a.part[slot].flags & 1)) continue;
      const int64_t at = (int64_t)slot * kPkvBlockRows + r;
      const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + at * 2);
      const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - ref);
      float x[N];
      load_vals<float, N>(a.part_o + at * HD + lane * N, x);
      if (ml.x == -INFINITY && ml.y == 0.f) continue;   // a part without entries of this row
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] += f * x[i];
      sum += f * ml.y;
    }
    const int tok = it.tok0 + r / G, head = p.h * G + r % G;
    if (a.groups) {
      const int64_t at = (int64_t)tok * a.n_head + head;
#pragma unroll
      for (int i = 0; i < N; ++i) a.row_o[at * HD + lane * N + i] = o[i];
      if (lane == 0) *reinterpret_cast<float2 *>(a.row_ml + at * 2) = make_float2(m, sum);
    } else {
      pkv_store<N>(a.out, tok * a.out.token + head * a.out.head + lane * N, o, sum == 0.f ? 0.f : 1.f / sum);
    }
  }
}

template <int HD, bool SPLIT>
cudaError_t launch_rows(const CUtensorMap &map, const PkvAttnArgs &a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(a.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = RL<HD, SPLIT>::SMEM;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_pkv_rows<HD, SPLIT>, map, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_pkv_join<HD>, dim3(a.grid, 8), dim3(256), 0, 1, st, a);
}

template <int HD>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(k_pkv_rows<HD, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       RL<HD, false>::SMEM);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(k_pkv_rows<HD, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, RL<HD, true>::SMEM);
}

}  // namespace

cudaError_t prepare_pkv_kernels(int hd) { return hd == 128 ? prepare<128>() : prepare<64>(); }

cudaError_t launch_pkv_rows(int hd, const CUtensorMap &map, const PkvAttnArgs &a, cudaStream_t st) {
  const bool split = a.q.dtype == PNB_F32 || a.out.dtype == PNB_F32;
  if (hd == 128) return split ? launch_rows<128, true>(map, a, st) : launch_rows<128, false>(map, a, st);
  return split ? launch_rows<64, true>(map, a, st) : launch_rows<64, false>(map, a, st);
}

}  // namespace pnb
