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

#include "pnb_pkv_sched.cuh"
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

struct RBars {
  uint64_t full[16], empty[16], q_ready[2], s_full[2], p_ready[2], o_full[2], v_go, v_ok, drain;
  uint32_t tmem, pad;
  int bad[kBadSlots];
  PkvWalk walk;
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
    bar.walk = PkvWalk{0, 0, 0, 0, 0, 1};
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
  if (a.pass == kPkvPrefix) pkv_find_groups<kThreads>(a, reinterpret_cast<int *>(ring));
  pkv_find_run<kPkvTile, kThreads>(a, TB, reinterpret_cast<int *>(ring), &bar.walk);
  PkvWalk walk = bar.walk;
  PkvItem it;
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
      // a lane per copied box: a page's rows, at most 64 of them
      const int log2p = a.pool.page_log2, log2b = min(log2p, kPkvBoxLog2), per_tile = kPkvTile >> log2b, box = 1 << log2b;
      const int rows_total = a.pool.n_page * 2 * a.pool.n_kv << log2p;
      while (ok && walk.next<kPkvTile>(a, TB, it)) {
        // page ids are the first sequence's of a group
        const int seq = a.pass == kPkvPrefix ? min(max(a.group_start[it.b], 0), a.seqs.n_seq - 1) : it.b;
        const int32_t *pages = a.seqs.pages + (int64_t)seq * a.seqs.max_page;
        auto page_id = [&](int t) {
          const int e = (it.t0 + t) * kPkvTile + (lane << log2b);
          return lane < per_tile && e < it.hi && e + box > it.lo ? pages[e >> log2p] : -1;
        };
        int id = page_id(it.ta);
        for (int t = it.ta; t < it.tb && ok; ++t) {
          const int e = (it.t0 + t) * kPkvTile + (lane << log2b);
          const bool needed = lane < per_tile && e < it.hi && e + box > it.lo;
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
              const int y = needed && good
                                ? (((now * 2 + kv) * a.pool.n_kv + it.h) << log2p) + (e & ((1 << log2p) - 1))
                                : rows_total;
              uint8_t *dst = ring + s * L::UNIT + (lane << log2b) * 128;
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
        while (ok && walk.next<kPkvTile>(a, TB, it)) {
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
      while (ok && walk.next<kPkvTile>(a, TB, it)) {
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
    auto load_q = [&](const PkvItem &x) {
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
    auto next = [&](PkvItem &x) {
      while (walk.next<kPkvTile>(a, TB, x)) {
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
      if (a.pass == kPkvPrefix) {
        if (a.window > 0) {
          const int seq = tok / a.seqs.each;
          const int last = pkv_len(a.seqs, a.pool.page_log2, seq, a.err) - a.seqs.each + tok % a.seqs.each;
          lo = max(0, last - a.window + 1);
        }
      } else {
        const int last = it.base + (tok - it.tok0);
        hi = last + 1;
        lo = max(it.floor, a.window > 0 ? last - a.window + 1 : 0);
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
      PkvItem nx;
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
      // the prefix's part of the row
      float f_own = 1.f, f_pre = 0.f, all = sum;
      const float *bo = nullptr;
      if (whole && it.floor > 0) {
        const int64_t at = (int64_t)tok * a.n_head + head;
        const float2 ml = *reinterpret_cast<const float2 *>(a.row_ml + at * 2);
        bo = a.row_o + at * HD;
        pkv_join_factors(m, ml.x, f_own, f_pre);
        all = sum * f_own + ml.y * f_pre;
      }
      const float inv = all == 0.f ? 0.f : 1.f / all;
      float *po = nullptr, *pml = nullptr;
      if (!whole) {
        const int64_t at = (int64_t)(2 * blockIdx.x + side) * kPkvBlockRows + r;
        po = a.part_o + at * HD;
        pml = a.part_ml + at * 2;
        if (r == 0) a.part[2 * blockIdx.x + side] = PkvPart{it.ends ? 3 : 1, it.b, it.j, it.h};
      } else if (a.pass == kPkvPrefix) {
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
            if (it.floor > 0) {
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(bo + i + k);
                o[k] = o[k] * f_own + x.x * f_pre;
                o[k + 1] = o[k + 1] * f_own + x.y * f_pre;
                o[k + 2] = o[k + 2] * f_own + x.z * f_pre;
                o[k + 3] = o[k + 3] * f_own + x.w * f_pre;
              }
            }
            pkv_store<32>(a.out, tok * a.out.token + head * a.out.head + i, o, inv);
          }
          __syncwarp();
        }
        if (live && po) *reinterpret_cast<float2 *>(pml) = make_float2(m, sum);
      } else {
        // a NaN or an infinity among values that only some rows see: each row by itself
        const int seq = a.pass == kPkvPrefix ? min(max(a.group_start[it.b], 0), a.seqs.n_seq - 1) : it.b;
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
            if (it.floor > 0) pkv_add_prefix<HD / 32>(a, tk, hd_k, o, mk, lk);
            const float d = lk == 0.f ? 0.f : 1.f / lk;
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
  PkvItem it;
  if (!pkv_block<kPkvTile>(a, TB, p.b, p.j, it)) return;
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
    if (it.floor > 0) pkv_add_prefix<N>(a, tok, head, o, m, sum);
    if (a.pass == kPkvPrefix) {
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
  return cudaLaunchKernelEx(&cfg, k_pkv_rows<HD, SPLIT>, map, a);
}

template <int HD>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(k_pkv_rows<HD, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       RL<HD, false>::SMEM);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(k_pkv_rows<HD, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, RL<HD, true>::SMEM);
}

}  // namespace

cudaError_t launch_pkv_join(int hd, const PkvAttnArgs &a, int rows, cudaStream_t st) {
  const dim3 grid(a.grid, (rows + 31) / 32), block(256);
  return hd == 128 ? launch_pdl(k_pkv_join<128>, grid, block, 0, 1, st, a)
                   : launch_pdl(k_pkv_join<64>, grid, block, 0, 1, st, a);
}

cudaError_t prepare_pkv_rows(int hd) { return hd == 128 ? prepare<128>() : prepare<64>(); }

cudaError_t launch_pkv_rows(int hd, const CUtensorMap &map, const PkvAttnArgs &a, cudaStream_t st) {
  const bool split = a.q.dtype == PNB_F32 || a.out.dtype == PNB_F32;
  cudaError_t e;
  if (hd == 128) e = split ? launch_rows<128, true>(map, a, st) : launch_rows<128, false>(map, a, st);
  else e = split ? launch_rows<64, true>(map, a, st) : launch_rows<64, false>(map, a, st);
  return e == cudaSuccess ? launch_pkv_join(hd, a, kPkvBlockRows, st) : e;
}

}  // namespace pnb
