// pnb_pkv_rows.cu - attention over the paged KV cache on tcgen05 tensor cores, for
// blocks of up to 256 rows (token, query head) that share a KV head's entries:
// prompts, prompt chunks, and the shared prefix of a group of sequences.
//
// Row i attends to entries [lo_i, hi_i).  With x_ij = q_i.k_j log2(e) / sqrt(hd) and a
// reference r_i, p_ij = 2^(x_ij - r_i), l_i = sum_j p_ij, o_i = sum_j p_ij v_j / l_i.
// r_i is the largest of the first scores seen, and moves when the sum of 64 p passes
// 2^16, so that no maximum is taken and nothing is rescaled in most tiles; sums are held
// in fp32.
//
// One CTA per SM works through a run of (block, 128-entry tile) units:
//   warps 0-3, 4-7  softmax of the block's rows 0-127 and 128-255, one row per thread:
//                   S from tensor memory, masks, reference, p as bf16 back over S;
//   warp 8          K and V tiles by tiled TMA loads of a page's rows each, into a ring;
//   warp 9          S = Q K^T (both operands in shared memory) and O += P V (P in tensor
//                   memory), the two halves in turn, so that one half's softmax runs
//                   beside the other's products (issued by a thread each, the halves ran
//                   in step, softmax beside softmax: a third slower);
//   warps 10, 11    V rows behind a sequence's last entry become zero (0 x NaN is NaN).
// A NaN or an infinity among a sequence's own values reaches, through tiles that a block's
// rows see only in part, rows that do not attend to it: a row whose output is not finite
// is done again by itself where such a value lies, and so is one of scores above 2^26.
// Tensor memory (512 columns): S of both halves (128 each), O of both halves, with SPLIT
// beside each half's O the sum over the tiles before.
//
// fp32 on either side (SPLIT): Q enters as three bf16 numbers (24 bits: a score's error is its
// weight's relative one), P as two (16 bits: 2^-17 of a weight at most), in 5/2
// times the products.  At head_dim 128 that leaves room for the queries of 128 rows: warps 4-7
// idle, S of two tiles takes both halves' columns, and the products of S run ahead of the softmax
// (two prompts up to 8191 under a window of 4096: 1468 us one tile at a time, 1149 so).  With ONE
// the same is done for calls whose blocks all have at most 128 rows.
//
// Bound by the hand-over between softmax and products: a tile's S and O take 2048 cycles for the two
// halves at head_dim 128, the exponentials, conversions and sums of 64 scores 367 cycles of a
// scheduler, 654 with both halves' warps on it, so that 128 scores of one half (1308) outlast the
// other's products (1024).  A 16k prompt (32 / 8 heads, head_dim 128, bf16) takes 1565 us, 1.41 PFLOP/s
// or 72 % of cuBLAS's bf16 rate on the same part; 512 tokens behind 60k entries 372 us, 70 %; DRAM is
// idle (2 to 12 %), K and V come from L2.
// Not kept: two threads per row (16 softmax warps meet at a barrier per tile: 2078 against 1661),
// an issuing thread per half (2145), a warp that serves whichever half is ready (2077).
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "pnb_pkv_sched.cuh"
#include "pnb_tc.cuh"

namespace pnb {
namespace {

extern __shared__ __align__(1024) uint8_t r_smem[];

constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;
constexpr float kLarge = 65536.f;   // a sum of 64 p that moves the reference
// A reference that is rounded by many powers of two puts p, exact products less the reference,
// out of any range: such rows are done again by themselves.
constexpr float kFar = 67108864.f;
// registers per thread: 384 x 168 at launch = 256 x 208 + 128 x 88
constexpr int kRegsSoft = 208, kRegsRest = 88;

// a place in the ring and the parity of its turn
template <int NU>
struct RingAt {
  int s = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void next() {
    if (++s == NU) {
      s = 0;
      turn ^= 1;
    }
  }
};

// With SPLIT the products' sums start anew every so many tiles, and are added up outside: the
// matrix unit cuts off what it adds, always towards zero, and over 475 tiles outputs came out
// 5e-5 too small.
constexpr int kFold = 4;
// Without SPLIT, where bf16's own roundings are of 2e-3, only every so many tiles (64k entries: 2.6e-4
// at most; without, values of mean 1 came out 4e-3 too small over 1M entries and 7e-2 over 16M).
// The sum over the tiles before then lies in the CTA's partial sums, in global memory: tensor
// memory has no columns left.
constexpr int kFoldLong = 512;

template <int HD, bool SPLIT, bool ONE>
struct RL {
  static constexpr int NB = HD / 64;                        // 64-column boxes of a row
  static constexpr int BOX = kPkvTile * 128;                // bytes of a 128-row box
  static constexpr int UNIT = NB * BOX;                     // a K or V tile
  // fp32 on either side: queries of three bf16 parts, for which one half of rows leaves room at
  // head_dim 128
  // (ONE: no block of the call has more)
  static constexpr int HALVES = ONE ? 1 : pkv_block_rows(HD, SPLIT) / 128;
  static constexpr int PARTS = SPLIT ? 3 : 1;
  static constexpr int QHALF = UNIT * PARTS;                // Q of 128 rows, part by part
  static constexpr int NU = (229376 - HALVES * QHALF) / UNIT;   // ring units
  static constexpr int SMEM = 1024 + HALVES * QHALF + NU * UNIT + 1024;
};

struct RBars {
  uint64_t full[16], empty[16], q_ready[2], s_full[2], p_ready[2][2], pv_half[2], o_full[2], v_go, v_ok, drain;
  uint32_t tmem;
  uint32_t work;   // changes with every tile that is loaded, and with rows done again
  uint32_t stop;   // a warp gave up
};
static_assert(sizeof(RBars) <= 1024, "barriers");

// S = Q K^T of one half and tile: hd / 16 products (three times with SPLIT, the smallest part
// first: a product cuts off what it adds to a large sum, and to a small one next to nothing)
template <int HD, bool SPLIT, int I = 0>
__device__ __forceinline__ void products_s(uint32_t d, uint64_t q, uint64_t k) {
  typedef RL<HD, SPLIT, true> L;   // (the same for both)
  constexpr int KS = HD / 16, part = L::PARTS - 1 - I / KS, c = I % KS / 4, x = I % 4;
  if constexpr (I < L::PARTS * KS) {
    mma_bf16_off<(part * L::UNIT + c * L::BOX + x * 32) / 16, (c * L::BOX + x * 32) / 16>(
        d, q, k, idesc_bf16_f32(128, kPkvTile), I > 0);
    products_s<HD, SPLIT, I + 1>(d, q, k);
  }
}
// O += P V of half a tile: four products of 16 entries (twice with SPLIT), V with N contiguous
template <int HD, bool SPLIT, int HALF, int I = 0>
__device__ __forceinline__ void products_o(uint32_t d, uint32_t p, uint64_t v, bool first) {
  constexpr int part = I / 4, x = I % 4;
  if constexpr (I < (SPLIT ? 8 : 4)) {
    mma_bf16_ts_off<HALF * 64 + part * 32 + x * 8, (HALF * 4 + x) * 2048 / 16>(
        d, p, v, idesc_bf16_f32(128, HD) | (1u << 16), I > 0 || !first);
    products_o<HD, SPLIT, HALF, I + 1>(d, p, v, first);
  }
}

// 8 elements of a query row as three bf16 parts each, what a rounding leaves in the next
__device__ __forceinline__ void split8(const float4 &a, const float4 &b, uint4 (&part)[3]) {
  float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
      f[2 * i] -= bf16lo(w[i]);
      f[2 * i + 1] -= bf16hi(w[i]);
    }
    part[p] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Adds a row's outputs in tensor memory to its sum in global memory (with `first`, sets it).
template <int HD>
__device__ __noinline__ void fold_long(uint32_t to, float *all, bool first) {
#pragma unroll 1
  for (int i = 0; i < HD; i += 32) {
    float o[32];
    tmem_ld32_async(to + i, o);
    tmem_wait_ld();
    tmem_landed(o);
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      float4 *p = reinterpret_cast<float4 *>(all + i + k);
      const float4 x = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *p;
      *p = make_float4(x.x + o[k], x.y + o[k + 1], x.z + o[k + 2], x.w + o[k + 3]);
    }
  }
}
template <int HD>
__device__ __noinline__ void scale_long(float *all, float f) {
#pragma unroll 1
  for (int i = 0; i < HD; i += 4) {
    float4 *p = reinterpret_cast<float4 *>(all + i);
    *p = make_float4(p->x * f, p->y * f, p->z * f, p->w * f);
  }
}

// Whether a value that some row of a block sees and another does not is NaN or infinite
// (the calling warp, a lane per entry; entries of tiles that the block's rows see in part).
template <int HD>
__device__ __noinline__ bool hidden_odd_values(const PkvAttnArgs &a, const PkvItem &it, uint32_t *work) {
  const int lane = threadIdx.x & 31;
  const int seq = a.pass == kPkvPrefix ? min(max(a.group_start[it.b], 0), a.seqs.n_seq - 1) : it.b;
  const int32_t *pages = a.seqs.pages + (int64_t)seq * a.seqs.max_page;
  const int first = it.t0 * kPkvTile, end = (it.t0 + it.nt) * kPkvTile;
  bool bad = false;
  for (int part = 0; part < 2; ++part) {
    const int from = part ? max(it.hi_min, first) : first;
    const int to = min(part ? end : min(it.lo_max, end), it.len);
    for (int e0 = max(from, 0); e0 < to; e0 += 32) {
      const __nv_bfloat16 *v = e0 + lane < to ? pkv_row<HD>(a.pool, pages, e0 + lane, 1, it.h) : nullptr;
#pragma unroll 4
      for (int i = 0; i < HD && v; i += 4) {
        float x[4];
        load_vals<__nv_bfloat16, 4>(v + i, x);
#pragma unroll
        for (int c = 0; c < 4; ++c) bad |= !(x[c] * 0.f == 0.f);
      }
      if (lane == 0) atomicAdd(work, 1u);
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// Does rows of a warp (bits of `rows`, a lane's row each) again by themselves: entries [lo, hi) of
// this CTA's tiles.  Sums go to po and pml, or where these are NULL answers to their place.
// An item's 256 rows over 400k entries (head_dim 64) take 0.8 s, over 2M 4.5 s: bound by latency, for
// a mishap.  The pipeline's waits count this as work.
template <int HD>
__device__ __noinline__ void repair_rows(const PkvAttnArgs &a, const PkvItem &it, uint32_t rows, int lo, int hi, int tok,
                                         int head, float *po, float *pml, uint32_t *work) {
  constexpr int R = 4, N = HD / 32;   // four rows at a time share the loads of K and V
  const int lane = threadIdx.x & 31;
  const int seq = a.pass == kPkvPrefix ? min(max(a.group_start[it.b], 0), a.seqs.n_seq - 1) : it.b;
  const int first = (it.t0 + it.ta) * kPkvTile, end = (it.t0 + it.tb) * kPkvTile;
  while (rows) {
    int64_t q_at[R];
    int from[R], to[R], src[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      src[i] = rows ? __ffs(rows) - 1 : -1;
      rows &= rows - 1;   // (0 stays 0)
      const int k = max(src[i], 0);
      from[i] = max(__shfl_sync(0xffffffffu, lo, k), first);
      to[i] = src[i] < 0 ? 0 : min(__shfl_sync(0xffffffffu, hi, k), end);
      q_at[i] = __shfl_sync(0xffffffffu, tok, k) * a.q.token + __shfl_sync(0xffffffffu, head, k) * a.q.head;
    }
    float o[R][N], m[R], sum[R];
    pkv_attend_rows<HD, R>(a.pool, a.seqs.pages + (int64_t)seq * a.seqs.max_page, it.h, a.q, q_at, a.qscale, from, to, o, m,
                           sum, work);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (src[i] < 0) break;
      float *dst = reinterpret_cast<float *>((uintptr_t)__shfl_sync(0xffffffffu, (long long)(uintptr_t)po, src[i]));
      float *ml = reinterpret_cast<float *>((uintptr_t)__shfl_sync(0xffffffffu, (long long)(uintptr_t)pml, src[i]));
      const int t = __shfl_sync(0xffffffffu, tok, src[i]), hd = __shfl_sync(0xffffffffu, head, src[i]);
      if (dst) {
#pragma unroll
        for (int n = 0; n < N; ++n) dst[lane * N + n] = o[i][n];
        if (lane == 0) *reinterpret_cast<float2 *>(ml) = make_float2(m[i], sum[i]);
      } else {
        pkv_store<N>(a.out, t * a.out.token + hd * a.out.head + lane * N, o[i], sum[i] == 0.f ? 0.f : 1.f / sum[i]);
      }
    }
  }
}

template <int HD, bool SPLIT, bool ONE>
__global__ void __launch_bounds__(kThreads, 1)
    k_pkv_rows(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ PkvAttnArgs a) {
  typedef RL<HD, SPLIT, ONE> L;
  constexpr int NU = L::NU;
  static_assert(NU <= 16 && NU >= 2, "ring");
  uint8_t *sm = r_smem + ((1024u - (smem_addr(r_smem) & 1023u)) & 1023u);
  uint8_t *Q = sm, *ring = sm + L::HALVES * L::QHALF;
  RBars &bar = *reinterpret_cast<RBars *>(ring + NU * L::UNIT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.n_head / a.pool.n_kv, TB = a.block_rows / G;

  // Waits behind other warps' tiles, items and repairs, of any number and length, go by the work that
  // is done meanwhile.  The products' warp, for which the others wait, only looks whether one of them
  // gave up (with the others' wait 16 packed prompts took 311 to 316 us against 305, so 307 to 311).
  auto working = [&](uint64_t *b, uint32_t parity) { return mbar_wait_working(b, parity, &bar.work); };
  auto give_up = [&]() {
    set_error(a.err, kErrTimeout);
    *reinterpret_cast<volatile uint32_t *>(&bar.stop) = 1;
  };

  if (threadIdx.x == 0) {
    bar.work = bar.stop = 0;
    for (int i = 0; i < NU; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_ready[i], 4);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_ready[i][0], 4);
      mbar_init(&bar.p_ready[i][1], 4);
      mbar_init(&bar.pv_half[i], 1);
      mbar_init(&bar.o_full[i], 1);
    }
    mbar_init(&bar.v_go, 1);
    mbar_init(&bar.v_ok, 64);
    mbar_init(&bar.drain, 1);
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The own pass runs beside the prefix's, which let it start behind its own wait: the call's
  // inputs are there, and it waits for the prefix's end only at its own.
  if (a.pass != kPkvOwn) pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 2) a.part[2 * blockIdx.x + threadIdx.x].flags = 0;
  if (a.pass != kPkvAll) pkv_find_groups<kThreads>(a, reinterpret_cast<int *>(ring));
  PkvWalk walk = pkv_find_run<kPkvTile, kThreads>(a, TB, reinterpret_cast<long long *>(ring));
  PkvItem it;
  const uint32_t tmem = bar.tmem;
  // the ring held the schedule's sums: order them before the tiles that TMA writes
  fence_async_smem();
  __syncthreads();

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == 8) {
      // ------------------------------------------------------ K and V tiles
      bool ok = true;
      uint32_t u = 0;   // units issued
      RingAt<NU> at;
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
          for (int kv = 0; kv < 2; ++kv, ++u, at.next()) {
            const int s = at.s;
            if (u >= NU && !working(&bar.empty[s], at.turn ^ 1)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
              *reinterpret_cast<volatile uint32_t *>(&bar.work) = u;
              mbar_arrive_expect_tx(&bar.full[s], L::UNIT);
            }
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
        if (lane == 0) give_up();
        // what is still on its way lands before the CTA ends
        for (uint32_t i = u > NU ? u - NU : 0; i < u; ++i) mbar_wait(&bar.full[i % NU], (i / NU) & 1);
      }
    } else if (warp == 9) {
      // ----------------------------------------------------------- products
      // The whole warp goes through the loops, with numbers that are the same in every lane,
      // and one elected lane issues: descriptors then stay in uniform registers (21 cycles
      // per product; 47 from a thread of its own, which kept the tensor pipe waiting).
      // A descriptor each for Q, K and V at the buffers' start; what a product adds to it
      // is known at compile time.
      const uint64_t q0 = desc_k_sw128(Q, 0), k0 = desc_k_sw128(ring, 0), v0 = desc_mn_sw128(ring, L::BOX);
      bool ok = true;
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0}, nv = 0, n_s = 0;
      RingAt<NU> at;
      auto wait = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_unless(b, parity, &bar.stop)) != 0; };
      while (ok && __all_sync(0xffffffffu, walk.next<kPkvTile>(a, TB, it))) {
        const int halves = __shfl_sync(0xffffffffu, it.ntok * G > 128 ? 2 : 1, 0);
        const int tiles = __shfl_sync(0xffffffffu, it.tb - it.ta, 0);
        // tiles from this one on reach behind the sequence's last entry (a prefix is whole pages, and
        // what lies behind in its last tile reads as zero)
        const int past = __shfl_sync(0xffffffffu, a.pass == kPkvPrefix ? INT_MAX : it.len / kPkvTile - it.t0 - it.ta, 0);
        if constexpr (L::HALVES == 1) {
          // One half: S of the next two tiles lies in tensor memory before a tile's p is there, so
          // that the softmax goes from tile to tile and the products run beside it.
          RingAt<NU> k = at, v = at;   // a tile's K and V lie side by side in the ring
          v.next();
          auto issue_s = [&]() {
            ok = wait(&bar.full[k.s], k.turn);
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) {
              products_s<HD, SPLIT>(tmem + (n_s & 1) * 128, q0, k0 + k.s * (L::UNIT >> 4));
              mma_commit(&bar.s_full[n_s & 1]);
              mma_commit(&bar.empty[k.s]);
            }
            __syncwarp();
            ++n_s;
            k.next();
            k.next();
          };
          ok = wait(&bar.q_ready[0], nq[0]++ & 1);
          if (ok) issue_s();
          if (ok && tiles > 1) issue_s();
          for (int t = 0; t < tiles && ok; ++t) {
            ok = wait(&bar.full[v.s], v.turn);
            if (ok && t >= past) {
              if (elect_one()) mbar_arrive(&bar.v_go);
              ok = wait(&bar.v_ok, nv++ & 1);
            }
            // (a p_ready for each of the two S: a warp may be a tile ahead of the others)
            const uint32_t i = np[0] & 1, turn = np[0]++ >> 1 & 1, p = tmem + i * 128;
            if (ok) ok = wait(&bar.p_ready[i][0], turn);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              products_o<HD, SPLIT, 0>(tmem + 256, p, v0 + v.s * (L::UNIT >> 4), t % (SPLIT ? kFold : kFoldLong) == 0);
              mma_commit(&bar.pv_half[0]);
            }
            __syncwarp();
            ok = wait(&bar.p_ready[i][1], turn);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              products_o<HD, SPLIT, 1>(tmem + 256, p, v0 + v.s * (L::UNIT >> 4), false);
              mma_commit(&bar.pv_half[1]);   // (of the whole tile)
              mma_commit(&bar.empty[v.s]);
              if (t + 1 == tiles) mma_commit(&bar.o_full[0]);
            }
            __syncwarp();
            v.next();
            v.next();
            if (t + 2 < tiles) issue_s();
          }
          at = k;
          continue;
        }
        ok = wait(&bar.full[at.s], at.turn);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (w >= halves || !ok) break;
          ok = wait(&bar.q_ready[w], nq[w]++ & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            products_s<HD, SPLIT>(tmem + w * 128, q0 + w * (L::QHALF >> 4), k0 + at.s * (L::UNIT >> 4));
            mma_commit(&bar.s_full[w]);
            if (w == halves - 1) mma_commit(&bar.empty[at.s]);
          }
          __syncwarp();
        }
        at.next();
        for (int t = 0; t < tiles && ok; ++t) {
          const RingAt<NU> v = at;   // this tile's V, then the next one's K
          at.next();
          const bool more = t + 1 < tiles;
          ok = wait(&bar.full[v.s], v.turn);
          if (ok && t >= past) {
            if (elect_one()) mbar_arrive(&bar.v_go);
            ok = wait(&bar.v_ok, nv++ & 1);
          }
          if (ok && more) ok = wait(&bar.full[at.s], at.turn);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (w >= halves || !ok) break;
            ok = wait(&bar.p_ready[w][0], np[w] & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              products_o<HD, SPLIT, 0>(tmem + 256 + w * 128, tmem + w * 128, v0 + v.s * (L::UNIT >> 4),
                                      t % (SPLIT ? kFold : kFoldLong) == 0);
              mma_commit(&bar.pv_half[w]);
            }
            __syncwarp();
            ok = wait(&bar.p_ready[w][1], np[w]++ & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              products_o<HD, SPLIT, 1>(tmem + 256 + w * 128, tmem + w * 128, v0 + v.s * (L::UNIT >> 4), false);
              if (more) {
                if (w == halves - 1) mma_commit(&bar.empty[v.s]);
                products_s<HD, SPLIT>(tmem + w * 128, q0 + w * (L::QHALF >> 4), k0 + at.s * (L::UNIT >> 4));
                mma_commit(&bar.s_full[w]);
                if (w == halves - 1) mma_commit(&bar.empty[at.s]);
              } else {
                mma_commit(&bar.o_full[w]);
                if (w == halves - 1) mma_commit(&bar.empty[v.s]);
              }
            }
            __syncwarp();
          }
          if (more) at.next();
        }
      }
      if (!ok) {
        if (elect_one()) {
          give_up();
          mma_commit(&bar.drain);   // the products in flight end before tensor memory is given back
        }
        mbar_wait(&bar.drain, 0);
      }
      __syncwarp();
    } else {
      // --------------------------------------------- V rows that are no entries
      bool ok = true;
      const int tid = threadIdx.x - 320;
      uint32_t nv = 0;
      RingAt<NU> at;
      while (ok && walk.next<kPkvTile>(a, TB, it)) {
        for (int t = it.ta; t < it.tb && ok; ++t, at.next()) {
          at.next();   // K, then V
          const int e0 = (it.t0 + t) * kPkvTile;
          if (it.t0 + t < it.len / kPkvTile || a.pass == kPkvPrefix) continue;
          const int s = at.s;
          // (the ring's own barriers would not do: this warp skips tiles, and the ring
          // may be a whole turn ahead or behind)
          ok = working(&bar.v_go, nv++ & 1);
          if (!ok) break;
          uint4 *v = reinterpret_cast<uint4 *>(ring + s * L::UNIT);
          for (int i = tid; i < L::UNIT / 16; i += 64)
            if (e0 + ((i >> 3) & (kPkvTile - 1)) >= it.len) v[i] = make_uint4(0, 0, 0, 0);
          fence_async_smem();
          mbar_arrive(&bar.v_ok);
        }
      }
      if (!ok && lane == 0) give_up();
      // Starts, groups and prefixes that are out of range are reported by a warp of the last CTA that
      // has nothing else to do (in the join kernel or in the schedule this took small calls 0.5 us).
      if (warp == 11 && blockIdx.x == gridDim.x - 1) {
        bool bad = false;
        if (a.seqs.start) bad = pkv_bad_starts(a.seqs.start, a.seqs.n_seq, -1, -1, a.seqs.n_tok, lane, 32);
        if (a.pass == kPkvPrefix) {
          bad |= pkv_bad_starts(a.group_start, a.n_group, 0, a.seqs.n_seq, a.seqs.n_seq, lane, 32);
          for (int g = lane; g < a.n_group; g += 32) bad |= a.prefix[g] < 0;
        }
        if (bad) set_error(a.err, kErrRange);
      }
    }
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int w = warp >> 2, quad = warp & 3, r = (warp << 5) + lane;   // r: row of the block
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    constexpr bool ALONE = L::HALVES == 1;   // S of consecutive tiles in either half's columns
    const uint32_t ts0 = tmem + w * 128 + lanes, to = tmem + 256 + w * 128 + lanes;
    const float c = a.qscale;
    // row / G as the high half of a product: exact for rows below 2^16 and G up to 64
    const uint32_t g_inv = (uint32_t)((0x100000000ull + G - 1) / G);
    auto div_g = [&](int row) { return G == 1 ? row : (int)__umulhi((uint32_t)row, g_inv); };
    uint32_t ns = 0, no = 0;
    bool ok = true;

    // A warp's 32 rows of a half lie in its own part of the Q buffer: queries before an
    // item, outputs on their way to memory behind it.  LPR lanes have 8 elements each.
    constexpr int LPR = HD / 8, RPW = 32 / LPR, QR = 32 / RPW;
    const int ql = lane % LPR, qsub = lane / LPR;
    uint8_t *const qmine = Q + w * L::QHALF + quad * 4096;   // 4 KB of each box
    uint4 qh[SPLIT ? 1 : QR];
    // A lane finds its own row's address; the lanes that move the row get it from there.
    auto of_lane = [&](long long v, int from) { return __shfl_sync(0xffffffffu, v, from); };
    auto put = [&](int k, const uint4 &v, int part) {
      const int row = k * RPW + qsub;
      *reinterpret_cast<uint4 *>(qmine + part * L::UNIT + (ql >> 3) * L::BOX + sw128(row, (ql & 7) * 16)) = v;
    };
    const bool q32 = a.q.dtype == PNB_F32;
    long long q_row = 0;
    // bf16 queries of the next item load while this one's outputs are on their way; rows
    // behind the block's last one repeat it, so that all loads are on their way at once
    auto fetch_q = [&](const PkvItem &x) {
      const int row = min(r, x.ntok * G - 1), q = div_g(row);
      const int64_t at = (x.tok0 + q) * a.q.token + (x.h * G + row - q * G) * a.q.head;
      q_row = (long long)(uintptr_t)a.q.p + at * (q32 ? 4 : 2);
      if constexpr (!SPLIT) {
#pragma unroll
        for (int k = 0; k < QR; ++k)
          qh[k] = reinterpret_cast<const uint4 *>((uintptr_t)of_lane(q_row, k * RPW + qsub))[ql];
      }
    };
    auto put_q = [&]() {
      if constexpr (!SPLIT) {
#pragma unroll
        for (int k = 0; k < QR; ++k) put(k, qh[k], 0);
      } else {
        constexpr int B = QR < 8 ? QR : 8;
#pragma unroll 1
        for (int k = 0; k < QR; k += B) {
          if (q32) {
            float4 f[B][2];
#pragma unroll
            for (int i = 0; i < B; ++i) {
              const float4 *p = reinterpret_cast<const float4 *>((uintptr_t)of_lane(q_row, (k + i) * RPW + qsub)) + 2 * ql;
              f[i][0] = p[0];
              f[i][1] = p[1];
            }
#pragma unroll
            for (int i = 0; i < B; ++i) {
              uint4 part[3];
              split8(f[i][0], f[i][1], part);
#pragma unroll
              for (int p = 0; p < 3; ++p) put(k + i, part[p], p);
            }
          } else {
            uint4 hi[B];
#pragma unroll
            for (int i = 0; i < B; ++i)
              hi[i] = reinterpret_cast<const uint4 *>((uintptr_t)of_lane(q_row, (k + i) * RPW + qsub))[ql];
#pragma unroll
            for (int i = 0; i < B; ++i) {
              put(k + i, hi[i], 0);
              put(k + i, make_uint4(0, 0, 0, 0), 1);
              put(k + i, make_uint4(0, 0, 0, 0), 2);
            }
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_ready[w]);
    };
    // the next item with rows for this half
    auto next = [&](PkvItem &x) {
      while (walk.next<kPkvTile>(a, TB, x))
        if (x.ntok * G > 128 * w) return true;
      return false;
    };

    bool have = next(it);
    if (have) {
      fetch_q(it);
      put_q();
    }
    while (have && ok) {
      const bool live = r < it.ntok * G;
      const int rq = live ? div_g(r) : 0, tok = it.tok0 + rq, head = it.h * G + (live ? r - rq * G : 0);
      int lo = it.lo, hi = it.hi;
      if (a.pass == kPkvPrefix) {
        if (a.window > 0) {
          const int seq = tok / a.seqs.each;
          const int last = pkv_len(a.seqs, a.pool.page_log2, seq, a.err) - a.seqs.each + tok % a.seqs.each;
          lo = max(0, last - a.window + 1);
        }
      } else {
        const int last = max(it.base + (tok - it.tok0), -1);
        hi = last + 1;
        lo = max(it.floor, a.window > 0 ? last - a.window + 1 : 0);
      }
      float m = -INFINITY, sum = 0.f;
      bool far = false;
      for (int t0 = it.ta; t0 < it.tb && ok; t0 += kFoldLong) {
        if (!SPLIT && t0 > it.ta) {
          // The products of the tiles so far go to the sum: with two halves they end before S of the next
          // tile is there, with one they are waited for.
          if (!working(&bar.s_full[ALONE ? ns & 1 : w], (ALONE ? ns >> 1 : ns) & 1)) ok = false;
          if (ALONE && !working(&bar.pv_half[1], (ns - 1) & 1)) ok = false;
          if (!ok) break;
          __syncwarp();
          tc_fence_after();
          fold_long<HD>(to, a.part_o + ((int64_t)(2 * blockIdx.x + (it.ta > 0 ? 0 : 1)) * kPkvBlockRows + r) * HD,
                        t0 - it.ta == kFoldLong);
          tc_fence_before();
        }
        const int t1 = SPLIT ? it.tb : min(it.tb, t0 + kFoldLong);
        for (int t = t0; t < t1; ++t) {
          const uint32_t ts = ts0 + (ALONE ? (ns & 1) * 128 : 0);
          if (!working(&bar.s_full[ALONE ? ns & 1 : w], (ALONE ? ns >> 1 : ns) & 1)) {
            ok = false;
            break;
          }
          ++ns;
          __syncwarp();
          tc_fence_after();
          // The row's 128 scores in two halves: the products of the first begin beside the
          // second one's exponentials.
          const int e = (it.t0 + t) * kPkvTile;
          const bool masked = e < it.lo_max || e + kPkvTile > it.hi_min;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            float x[64];
#pragma unroll
            for (int i = 0; i < 2; ++i) tmem_ld32_async(ts + 64 * h + 32 * i, x + 32 * i);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 2; ++i) tmem_landed(x + 32 * i);
            if (masked) {
              // columns [from, from + n) of the 64 are this row's
              const int e2 = e + 64 * h, from = max(lo - e2, 0), n = max(min(hi - e2, 64) - from, 0);
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if ((unsigned)(i - from) >= (unsigned)n) x[i] = -INFINITY;
            }
            // No maximum is taken while the reference does: p and its sum tell when it does not,
            // and fp32 and bf16 hold a p far above 1 as well as one below.  p goes over S, high
            // parts (and low parts) of 64 entries in 32 columns each.
            auto exponentials = [&]() {
              const float ref = m == -INFINITY ? 0.f : m;   // nothing seen yet: every p is 2^-inf
              const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
              float2 acc[2] = {};
              uint32_t p[32], low[SPLIT ? 32 : 1];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float2 y = ffma2(make_float2(x[2 * i], x[2 * i + 1]), c2, r2);
                y.x = exp2_approx(y.x);
                y.y = exp2_approx(y.y);
                acc[i & 1] = fadd2(acc[i & 1], y);
                p[i] = pack_bf16(y.x, y.y);
                if constexpr (SPLIT) low[i] = pack_bf16(y.x - bf16lo(p[i]), y.y - bf16hi(p[i]));
              }
              tmem_st32_async(ts + 64 * h, p);
              if constexpr (SPLIT) tmem_st32_async(ts + 64 * h + 32, low);
              acc[0] = fadd2(acc[0], acc[1]);
              return acc[0].x + acc[0].y;
            };
            float part = exponentials();
            if (__any_sync(0xffffffffu, m == -INFINITY || !(part < kLarge))) {
              float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
              for (int i = 4; i < 64; i += 4)
#pragma unroll
                for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], x[i + k]);
              const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
              const bool move = top > m && (m == -INFINITY || !(part < kLarge));
              if (__any_sync(0xffffffffu, move)) {
                const float f = move ? (m == -INFINITY ? 0.f : exp2_approx(m - top)) : 1.f;
                if (move) m = top;
                far |= move && fabsf(top) >= kFar;
                sum *= f;
                if (!SPLIT && t - it.ta >= kFoldLong && move)
                  scale_long<HD>(a.part_o + ((int64_t)(2 * blockIdx.x + (it.ta > 0 ? 0 : 1)) * kPkvBlockRows + r) * HD, f);
                if (t > it.ta || h) {
                  // Outputs so far go to the new reference.  The products of the tile before end
                  // first: with two halves S of this tile came behind them; with one it did not, and they
                  // may wait for another warp's p yet.  Those of this tile's first half end next (only
                  // then: a phase further back has the same parity, and would pass for this one).
                  if (ALONE && t > it.ta && !working(&bar.pv_half[1], ns & 1)) ok = false;
                  if (h && !working(&bar.pv_half[w], (ns - 1) & 1)) ok = false;
                  __syncwarp();
                  tc_fence_after();
#pragma unroll 1
                  for (int i = 0; i < (SPLIT && t - it.ta >= kFold ? 2 * HD : HD); i += 32) {
                    float o[32];
                    tmem_wait_st();
                    tmem_ld32_async(to + i, o);
                    tmem_wait_ld();
                    tmem_landed(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] *= f;
                    tmem_st32_async(to + i, reinterpret_cast<const uint32_t *>(o));
                  }
                }
                // p goes over p, and below a sum that starts anew is read back
                tmem_wait_st();
                part = exponentials();
              }
            }
            sum += part;
            if (SPLIT && h == 0 && t > it.ta && (t - it.ta) % kFold == 0) {
              // the products of the tiles so far (done: S of this one came behind them) go to the
              // sum, and this tile's start anew
              if (ALONE && !working(&bar.pv_half[1], ns & 1)) ok = false;
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < HD; i += 32) {
                float o[32], all[32];
                tmem_ld32_async(to + i, o);
                tmem_ld32_async(to + HD + i, all);
                tmem_wait_ld();
                tmem_landed(o);
                tmem_landed(all);
#pragma unroll
                for (int k = 0; k < 32; ++k) all[k] = t - it.ta == kFold ? o[k] : all[k] + o[k];
                tmem_st32_async(to + HD + i, reinterpret_cast<const uint32_t *>(all));
              }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_ready[ALONE ? (ns - 1) & 1 : w][h]);
          }
        }
        if (SPLIT) break;   // (whose sums start anew beside the softmax)
      }
      if (!ok) break;
      PkvItem nx;
      have = next(nx);
      if (have) fetch_q(nx);
      if (!working(&bar.o_full[w], no++ & 1)) {
        ok = false;
        break;
      }
      __syncwarp();
      tc_fence_after();
      const bool whole = it.ta == 0 && it.ends;
      const int side = it.ta > 0 ? 0 : 1;   // of the run's two partial sums
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      // where the row goes: the answer, or, unfinished, its sums
      float *po = nullptr, *pml = nullptr;
      if (!whole) {
        const int64_t at = (int64_t)(2 * blockIdx.x + side) * kPkvBlockRows + r;
        po = a.part_o + at * HD;
        pml = a.part_ml + at * 2;
        if (r == 0) a.part[2 * blockIdx.x + side] = PkvPart{it.ends ? 3 : 1, it.b, it.j, it.h};
      } else if (a.pass != kPkvAll) {
        const int64_t at = (int64_t)tok * a.n_head + head;
        po = a.row_o[a.pass - 1] + at * HD;
        pml = a.row_ml[a.pass - 1] + at * 2;
      }
      const bool out32 = a.out.dtype == PNB_F32;
      const long long to_row = po ? (long long)(uintptr_t)po
                                  : (long long)(uintptr_t)a.out.p +
                                        (tok * a.out.token + head * a.out.head) * (out32 ? 4 : 2);
      bool redo = false, odd = false;
      uint32_t odd_rows = 0;
      // Outputs go through the warp's part of the Q buffer, so that rows leave in whole lines:
      // 16-byte pieces of a row, turned by the row so that lanes meet different banks.
      auto emit = [&](auto wide) {
        constexpr bool F32 = decltype(wide)::value;
        constexpr int PASSES = F32 && !SPLIT ? 2 : 1;   // without SPLIT there is room for 16 bits per element
        constexpr int ROWS = 32 / PASSES, BYTES = F32 ? HD * 4 : HD * 2, PIECES = BYTES / 16, STEP = 32 / PIECES;
        auto piece = [&](int row, int i, int turn) {
          const int at = row * BYTES + ((i ^ (turn & 7)) << 4);
          return reinterpret_cast<uint4 *>(qmine + (at >> 12) * L::BOX + (at & 4095));   // no row crosses 4 KB
        };
        const float f = po ? 1.f : inv;   // a row that saw nothing has only zeros summed up
#pragma unroll 1
        for (int pass = 0; pass < PASSES; ++pass) {
          const bool mine = lane / ROWS == pass;
          float z = 0.f;   // NaN if an output is not finite
#pragma unroll 1
          for (int i = 0; i < HD; i += 32) {
            float o[32];
            tmem_ld32_async(to + i, o);
            tmem_wait_ld();
            tmem_landed(o);
            if (SPLIT && it.tb - it.ta > kFold) {
              float all[32];
              tmem_ld32_async(to + HD + i, all);
              tmem_wait_ld();
              tmem_landed(all);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] += all[k];
            }
            if (!SPLIT && it.tb - it.ta > kFoldLong) {
              const float *all = a.part_o + ((int64_t)(2 * blockIdx.x + side) * kPkvBlockRows + r) * HD + i;
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(all + k);
                o[k] += x.x;
                o[k + 1] += x.y;
                o[k + 2] += x.z;
                o[k + 3] += x.w;
              }
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) z = fmaf(o[k], 0.f, z);
            if (mine) {
              if constexpr (F32) {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                  *piece(lane % ROWS, (i + k) >> 2, lane) =
                      make_uint4(__float_as_uint(o[k] * f), __float_as_uint(o[k + 1] * f),
                                 __float_as_uint(o[k + 2] * f), __float_as_uint(o[k + 3] * f));
              } else {
#pragma unroll
                for (int k = 0; k < 32; k += 8)
                  *piece(lane, (i + k) >> 3, lane) =
                      make_uint4(pack_bf16(o[k] * f, o[k + 1] * f), pack_bf16(o[k + 2] * f, o[k + 3] * f),
                                 pack_bf16(o[k + 4] * f, o[k + 5] * f), pack_bf16(o[k + 6] * f, o[k + 7] * f));
              }
            }
            __syncwarp();
          }
          if (pass == 0) {
            odd = live && (z != 0.f || far);
            odd_rows = __ballot_sync(0xffffffffu, odd);
            if (odd_rows) {
              const PkvItem copy = it;   // (its address is taken)
              redo = __any_sync(0xffffffffu, far) || hidden_odd_values<HD>(a, copy, &bar.work);
            }
          }
          const uint32_t store = __ballot_sync(0xffffffffu, live && !(redo && odd));
#pragma unroll 4
          for (int k = 0; k < ROWS; k += STEP) {
            const int at = k + lane / PIECES, src = pass * ROWS + at;
            const uint4 x = *piece(at, lane % PIECES, src);
            uint4 *dst = reinterpret_cast<uint4 *>((uintptr_t)of_lane(to_row, src)) + lane % PIECES;
            if (store >> src & 1) *dst = x;
          }
          __syncwarp();
        }
      };
      if (po || out32) emit(std::true_type());
      else emit(std::false_type());
      if (live && po && !(redo && odd)) *reinterpret_cast<float2 *>(pml) = make_float2(m, sum);
      if (redo) {
        const PkvItem copy = it;
        repair_rows<HD>(a, copy, odd_rows, lo, hi, tok, head, po, pml, &bar.work);
      }
      if (have) put_q();
      tc_fence_before();
      it = nx;
    }
    if (!ok && lane == 0) give_up();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
  if (a.pass == kPkvOwn) pdl_wait();
}

// rows r0 .. r0 + 3 of the item whose first tiles CTA c0 had
template <int HD>
__device__ __forceinline__ void join_rows(const PkvAttnArgs &a, int pass, int c0, int r0, const uint8_t *first,
                                          const uint8_t *second) {
  constexpr int N = HD / 32, R = 4;
  const int lane = threadIdx.x & 31;
  const PkvPart p = a.part[2 * c0 + 1];
  const int G = a.n_head / a.pool.n_kv, TB = a.block_rows / G, h = p.h;
  const PkvSeq seq = pkv_seq(a, pass, p.b);
  PkvItem it;
  pkv_block<kPkvTile>(a, pass, seq, TB, p.b, p.j, it);
  const int rows = it.ntok * G;
  if (r0 >= rows) return;
  // the run that ends the item
  const int end = (c0 / a.grid + 1) * a.grid;
  int last = end - 1;
  for (int k0 = c0 + 1; k0 < end; k0 += 32) {
    const uint32_t ends = __ballot_sync(0xffffffffu, k0 + lane < end && (first[k0 + lane] & 2));
    if (ends) {
      last = k0 + __ffs(ends) - 1;
      break;
    }
  }
  float m[R], sum[R], o[R][N] = {};
#pragma unroll
  for (int i = 0; i < R; ++i) m[i] = -INFINITY;
  // a lane per part: references first, then factors
  for (int k0 = c0; k0 <= last; k0 += 32) {
    const int k = k0 + lane, slot = k == c0 ? 2 * k + 1 : 2 * k;
    const bool has = k <= last && ((k == c0 ? second[k] : first[k]) & 1);   // (a run may have no units)
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (has && r0 + i < rows) m[i] = fmaxf(m[i], a.part_ml[((int64_t)slot * kPkvBlockRows + r0 + i) * 2]);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = warp_max(m[i]);
    sum[i] = 0.f;
  }
  for (int k0 = c0; k0 <= last; k0 += 32) {
    const int k = k0 + lane, slot = k == c0 ? 2 * k + 1 : 2 * k;
    const bool has = k <= last && ((k == c0 ? second[k] : first[k]) & 1);
    float f[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      f[i] = 0.f;
      if (has && r0 + i < rows) {
        const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + ((int64_t)slot * kPkvBlockRows + r0 + i) * 2);
        // a part without entries of the row counts 0, one with a NaN score as it is
        f[i] = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - m[i]);
        sum[i] += f[i] * ml.y;
      }
    }
    const uint32_t which = __ballot_sync(0xffffffffu, has);
    // four parts' rows on their way together
    for (int j = 0; j <= last - k0 && j < 32; j += 4) {
      float x[4][R][N];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int kk = min(k0 + j + u, last), from = kk == c0 ? 2 * kk + 1 : 2 * kk;
        const float *src = a.part_o + ((int64_t)from * kPkvBlockRows + r0) * HD + lane * N;
#pragma unroll
        for (int i = 0; i < R; ++i) load_vals<float, N>(src + i * HD, x[u][i]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (j + u > 31 || !(which >> (j + u) & 1)) continue;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float fj = __shfl_sync(0xffffffffu, f[i], j + u);
#pragma unroll
          for (int n = 0; n < N; ++n) o[i][n] += fj * x[u][i][n];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + i;
    sum[i] = warp_sum(sum[i]);
    if (r >= rows) break;
    const int tok = it.tok0 + r / G, head = h * G + r % G;
    if (pass != kPkvAll) {
      const int64_t at = (int64_t)tok * a.n_head + head;
#pragma unroll
      for (int n = 0; n < N; ++n) a.row_o[pass - 1][at * HD + lane * N + n] = o[i][n];
      if (lane == 0) *reinterpret_cast<float2 *>(a.row_ml[pass - 1] + at * 2) = make_float2(m[i], sum[i]);
    } else {
      pkv_store<N>(a.out, tok * a.out.token + head * a.out.head + lane * N, o[i], sum[i] == 0.f ? 0.f : 1.f / sum[i]);
    }
  }
}

// Adds up the parts of the items that several CTAs shared, in the list's order.  The
// CTA whose run holds an item's first tiles has it in its second partial sum; the
// runs behind it hold the rest in their first ones.  A warp takes four rows together, so
// that the parts' loads are on their way at once.  Over a shared prefix the parts of both
// passes are there, the own pass's CTAs behind the prefix's.  Blocks share out the items
// that have something to add: chunks of 32 rows, chunks[pass] of them per item.
template <int HD>
__global__ void __launch_bounds__(256)
    k_pkv_join(const __grid_constant__ PkvAttnArgs a, const int chunks0, const int chunks1) {
  constexpr int R = 4, MAX = 2 * kPkvMaxCtas;
  __shared__ uint8_t first[MAX], second[MAX];   // flags of the CTAs' partial sums
  __shared__ uint16_t leaders[MAX];
  __shared__ int n_leaders[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int passes = a.pass == kPkvAll ? 1 : 2, n = passes * a.grid;
  pdl_wait();
  pdl_trigger();
  int any = 0;
  for (int k = threadIdx.x; k < n; k += 256) {
    first[k] = (uint8_t)a.part[2 * k].flags;
    second[k] = (uint8_t)a.part[2 * k + 1].flags;
    any |= second[k] & 1;
  }
  if (!__syncthreads_or(any)) return;
  if (warp == 0) {
    int at = 0;
    for (int k0 = 0; k0 < n; k0 += 32) {
      const int k = k0 + lane;
      const uint32_t is = __ballot_sync(0xffffffffu, k < n && (second[k] & 1));
      if (is >> lane & 1) leaders[at + __popc(is & ((1u << lane) - 1))] = (uint16_t)k;
      const uint32_t early = __ballot_sync(0xffffffffu, k < a.grid);
      if (lane == 0 && k0 < a.grid) n_leaders[0] = at + __popc(is & early);
      at += __popc(is);
    }
    if (lane == 0) n_leaders[1] = at;
  }
  __syncthreads();
  const int items0 = n_leaders[0], work0 = items0 * chunks0, work = work0 + (n_leaders[1] - items0) * chunks1;
  for (int i = blockIdx.x; i < work; i += gridDim.x) {
    const int own = i >= work0, chunks = own ? chunks1 : chunks0, at = own ? i - work0 : i;
    const int c0 = leaders[own * items0 + at / chunks], r0 = ((at % chunks) * 8 + warp) * R;
    const int pass = a.pass == kPkvAll ? kPkvAll : kPkvPrefix + own;
    join_rows<HD>(a, pass, c0, r0, first, second);
  }
}

// Adds the two passes' parts of every row, a warp each.
template <int HD>
__global__ void __launch_bounds__(256) k_pkv_finish(const __grid_constant__ PkvAttnArgs a) {
  constexpr int N = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  if (row >= (int64_t)a.seqs.n_tok * a.n_head) return;
  const int tok = (int)(row / a.n_head), head = (int)(row - (int64_t)tok * a.n_head);
  float2 ml[2];
  float x[2][N];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ml[i] = *reinterpret_cast<const float2 *>(a.row_ml[i] + row * 2);
    load_vals<float, N>(a.row_o[i] + row * HD + lane * N, x[i]);
  }
  // a sequence that no group holds has no prefix
  const int g = pkv_group_of(a.group_start, a.n_group, tok / a.seqs.each);
  if (g < 0 || a.groups[g].prefix == 0) {
    ml[0] = make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) x[0][i] = 0.f;
  }
  float f0, f1, o[N];
  pkv_join_factors(ml[0].x, ml[1].x, f0, f1);
  const float sum = ml[0].y * f0 + ml[1].y * f1;
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = x[0][i] * f0 + x[1][i] * f1;
  pkv_store<N>(a.out, tok * a.out.token + head * a.out.head + lane * N, o, sum == 0.f ? 0.f : 1.f / sum);
}

template <int HD, bool SPLIT, bool ONE>
cudaError_t launch_rows(const CUtensorMap &map, const PkvAttnArgs &a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(a.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = RL<HD, SPLIT, ONE>::SMEM;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_pkv_rows<HD, SPLIT, ONE>, map, a);
}

template <int HD, bool SPLIT>
cudaError_t launch_halves(bool one, const CUtensorMap &map, const PkvAttnArgs &a, cudaStream_t st) {
  if constexpr (pkv_block_rows(HD, SPLIT) > 128)
    if (!one) return launch_rows<HD, SPLIT, false>(map, a, st);
  return launch_rows<HD, SPLIT, true>(map, a, st);
}

template <int HD, bool SPLIT>
cudaError_t prepare() {
  const cudaError_t e = cudaFuncSetAttribute(
      k_pkv_rows<HD, SPLIT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, RL<HD, SPLIT, true>::SMEM);
  if constexpr (pkv_block_rows(HD, SPLIT) > 128)
    if (e == cudaSuccess)
      return cudaFuncSetAttribute(k_pkv_rows<HD, SPLIT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  RL<HD, SPLIT, false>::SMEM);
  return e;
}

}  // namespace

cudaError_t launch_pkv_join(int hd, const PkvAttnArgs &a, int rows, cudaStream_t st) {
  const bool two = a.pass != kPkvAll;
  const dim3 block(256);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(2 * a.grid);
  cfg.blockDim = block;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const int chunks0 = (two ? kPkvBlockRows : rows) / 32, chunks1 = (rows + 31) / 32;
  cudaError_t e = cudaLaunchKernelEx(&cfg, hd == 128 ? k_pkv_join<128> : k_pkv_join<64>, a, two ? chunks0 : chunks1, chunks1);
  if (e != cudaSuccess || !two) return e;
  const dim3 all((unsigned)(((int64_t)a.seqs.n_tok * a.n_head + 7) / 8));
  return hd == 128 ? launch_pdl(k_pkv_finish<128>, all, block, 0, 1, st, a)
                   : launch_pdl(k_pkv_finish<64>, all, block, 0, 1, st, a);
}

// A tile's time, for the shares of a prefix's and the own pass (against pkv_step_cost's), and an item's
// start and end against a tile.  64 slots of up to 1024 entries behind a shared prefix, us at
//   1200, 1500, 1800, 2200, 2600 ns: 8k, head_dim 128: fp32 110, 104, 95, 98, 104; bf16 96, 84, 86, 88, 90;
//                                    16k, head_dim 64: fp32 84, 80, 77, 75, 76; bf16 65, 63, 67, 69, 73.
// 3, 4, 6, 8 units per item: 16k prompt 1677, 1522, 1556, 1560; 16 packed prompts 317, 300, 311, 330, in
// fp32 692, 642, 656, 693, at head_dim 64 227, 224, 234, 247 and in fp32 351, 345, 365, 386; two prompts under a
// window, fp32, 1287, 1139, 1141, 1165.
void pkv_rows_cost(int hd, bool split, int *unit_ns, int *item_units) {
  *unit_ns = hd == 128 ? (split ? 1800 : 1500) : (split ? 2000 : 1500);
  *item_units = 4;
}

cudaError_t prepare_pkv_rows(int hd) {
  const cudaError_t e = hd == 128 ? prepare<128, false>() : prepare<64, false>();
  if (e != cudaSuccess) return e;
  return hd == 128 ? prepare<128, true>() : prepare<64, true>();
}

cudaError_t launch_pkv_rows(int hd, const CUtensorMap &map, const PkvAttnArgs &args, cudaStream_t st) {
  PkvAttnArgs a = args;
  const bool split = pkv_split(a);
  pkv_rows_cost(hd, split, &a.unit_ns, &a.item_units);
  a.heads_inner = a.pass == kPkvAll;
  // No block has more than a half's rows: the kernel of one half, S running ahead.  16 rows over
  // 64 sequences of 4096 (head_dim 128, bf16, cold L2) 227 against 243 us, 80 over 16 of 3000 92 against
  // 100; 32 rows over 64 of 4096 at head_dim 64 in bf16 164 against 182, in fp32 215 against 258.  Beside
  // a prefix's pass it loses (32 slots of 12 rows behind 30000 entries 132 against 114).
  const int64_t tokens = a.seqs.each ? a.seqs.each : a.seqs.n_tok;
  const bool one = a.pass == kPkvAll && tokens * (a.n_head / a.pool.n_kv) <= 128;
  if (hd == 128) return split ? launch_halves<128, true>(one, map, a, st) : launch_halves<128, false>(one, map, a, st);
  return split ? launch_halves<64, true>(one, map, a, st) : launch_halves<64, false>(one, map, a, st);
}

}  // namespace pnb
