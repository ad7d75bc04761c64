// pnb_pkv_step.cu - attention of a few rows per sequence and KV head (single tokens,
// a few drafted ones) over the paged KV cache.  Bound by the bytes of K and V.
//
// A row is one (token, query head); up to 8 RB rows share a KV head's entries (RB 2 at
// head_dim 64 only: at 128 the tcgen05 kernel is faster from 9 rows on).  Warp
// instructions m16n8k16 take rows 0-7 of A as the rows' bf16 high parts and rows 8-15 as
// their low parts, of the queries in S = Q K^T and of the softmax weights in O = P V: the
// 16 rows that the instruction has anyway give 16 bits of both operands, and a lane
// holds a row's high and low sums side by side.  (fp32 queries' third parts take a second
// instruction.)  tcgen05's 128 rows would be empty but
// for these.
//
// One CTA per SM, eight compute warps and one that loads.  The list of all (sequence, KV
// head) items' 64-entry chunks is cut into equal runs, one per CTA; a chunk's K and V come
// by TMA into a ring; four warps take 16 of its entries each, the other four the next
// chunk.  Every warp keeps its own reference, sums and outputs; they meet at an item's
// end in shared memory, and those of items that CTAs share in the join kernel.
//
// Single tokens of 64 sequences of 4096 entries (32 / 8 heads, head_dim 128, 1.07 GB, L2
// cold) take 194 us, 5.5 TB/s; 8 of 32768 188 us, 5.7; one of 32768 53 us, 2.5: bytes, and
// for few of them the start (schedule, lengths, page ids and first chunk in turn) and the join.
#include <cuda_bf16.h>
#include <math.h>

#include "pnb_pkv_sched.cuh"
#include "pnb_tc.cuh"

namespace pnb {
namespace {

extern __shared__ __align__(1024) uint8_t s_smem[];

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32 + 32;
constexpr int kChunk = kPkvChunk;
constexpr float kTau = 8.f;
// The matrix instructions cut off what they add, always towards zero: without new starts values of mean 1
// came out 1.4e-5 too small over 64k entries and 8e-3 over 16M.  With LONG, in items of more chunks
// than this, outputs go to fp32 sums in shared memory every so many chunks, half of them a warp's
// (1.4e-6 at any length).  It is there for page tables with room for so many entries of a sequence, from
// where on the cut is above 4e-6 (bf16: 5e-5): 8 of 32768 take 173 us with it and 172 without, but 64
// slots behind a shared 8k prefix 105 against 98, for registers.
constexpr int kFoldChunks = 128;
constexpr int64_t kLongF32 = 16384, kLongBf16 = 262144;

template <int HD, int RB>
struct SL {
  static constexpr int NB = HD / 64;
  static constexpr int BOX = kChunk * 128;
  static constexpr int UNIT = NB * BOX;                    // K or V of a chunk
  static constexpr int STAGE = 2 * UNIT;
  static constexpr int LD = HD + 4;                        // a warp's row in the merge buffer, floats
  static constexpr int MERGE = kWarps * RB * 8 * LD * 4;
  static constexpr int FIT = (232448 - 1024 - 2048 - MERGE) / STAGE / 2 * 2;
  static constexpr int NS = FIT < 8 ? FIT : 8;             // even: a stage belongs to one half of the warps
  static constexpr int SMEM = 1024 + NS * STAGE + MERGE + 2048;
};

struct SBars {
  uint64_t full[8], empty[8];
  float2 ml[kWarps][16];
  int bad;
  uint32_t work;   // changes with rows done again
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// two neighbouring elements of a query row: high parts, low parts and the rest
__device__ __forceinline__ void load_q2(const DevRows &q, int64_t at, uint32_t &hi, uint32_t &lo, uint32_t &rest) {
  if (q.dtype == PNB_BF16) {
    hi = *reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(q.p) + at);
    lo = rest = 0;
  } else {
    const float2 f = *reinterpret_cast<const float2 *>(static_cast<const float *>(q.p) + at);
    hi = pack_bf16(f.x, f.y);
    const float x = f.x - bf16lo(hi), y = f.y - bf16hi(hi);
    lo = pack_bf16(x, y);
    rest = pack_bf16(x - bf16lo(lo), y - bf16hi(lo));
  }
}

template <int HD, int RB, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
    k_pkv_step(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ PkvAttnArgs a) {
  typedef SL<HD, RB> L;
  constexpr int NS = L::NS, KS = HD / 16, NT = HD / 8;
  static_assert(NS >= 2 && L::SMEM <= 232448, "ring");
  uint8_t *sm = s_smem + ((1024u - (smem_addr(s_smem) & 1023u)) & 1023u);
  uint8_t *ring = sm;
  float *merge = reinterpret_cast<float *>(sm + NS * L::STAGE);
  SBars &bar = *reinterpret_cast<SBars *>(sm + NS * L::STAGE + L::MERGE);
  static_assert(sizeof(SBars) <= 2048, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.n_head / a.pool.n_kv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], kWarps / 2);
    }
    fence_barrier_init();
    bar.bad = 0;
    bar.work = 0;
  }
  __syncthreads();
  // The own pass runs beside the prefix's, which let it start behind its own wait: the call's
  // inputs are there, and it waits for the prefix's end only at its own.
  if (a.pass != kPkvOwn) pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 2) a.part[2 * blockIdx.x + threadIdx.x].flags = 0;
  if (a.pass == kPkvOwn) pkv_find_groups<kThreads>(a, reinterpret_cast<int *>(ring));
  PkvWalk walk = pkv_find_run<kChunk, kThreads>(a, a.seqs.each, reinterpret_cast<long long *>(ring));
  PkvItem it;
  fence_async_smem();   // the ring held the schedule's sums
  __syncthreads();

  if (warp == kWarps) {
    // -------------------------------------------------------- K and V chunks
    bool ok = true;
    uint32_t u = 0;   // chunks issued
    const int log2p = a.pool.page_log2, log2b = min(log2p, kPkvBoxLog2), per = kChunk >> log2b, box = 1 << log2b;
    const int rows_total = a.pool.n_page * 2 * a.pool.n_kv << log2p;
    while (ok && walk.next<kChunk>(a, a.seqs.each, it)) {
      const int32_t *pages = a.seqs.pages + (int64_t)it.b * a.seqs.max_page;
      auto page_id = [&](int t) {
        const int e = (it.t0 + t) * kChunk + (lane << log2b);
        return lane < per && e < it.hi && e + box > it.lo ? pages[e >> log2p] : -1;
      };
      int id = page_id(it.ta);
      for (int t = it.ta; t < it.tb; ++t, ++u) {
        const int e = (it.t0 + t) * kChunk + (lane << log2b);
        const bool needed = lane < per && e < it.hi && e + box > it.lo;
        const bool good = id >= 0 && id < a.pool.n_page;
        if (needed && !good) set_error(a.err, kErrRange);
        const int now = id;
        if (t + 1 < it.tb) id = page_id(t + 1);
        const int s = u % NS;
        if (u >= NS && !mbar_wait_working(&bar.empty[s], (u / NS - 1) & 1, &bar.work)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar.full[s], L::STAGE);
        __syncwarp();
        if (lane < per) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            // rows behind the pool's end read as zero
            const int y = needed && good ? (((now * 2 + kv) * a.pool.n_kv + it.h) << log2p) + (e & ((1 << log2p) - 1))
                                         : rows_total;
            uint8_t *dst = ring + s * L::STAGE + kv * L::UNIT + (lane << log2b) * 128;
#pragma unroll
            for (int c = 0; c < L::NB; ++c) tma_load_2d(dst + c * L::BOX, &kvmap, c * 64, y, &bar.full[s]);
          }
        }
      }
    }
    if (!ok) {
      if (lane == 0) set_error(a.err, kErrTimeout);
      for (uint32_t i = u > NS ? u - NS : 0; i < u; ++i) mbar_wait(&bar.full[i % NS], (i / NS) & 1);
    }
    return;
  }

  const int half = warp >> 2, p0 = (warp & 3) * 16;   // this warp's entries of a chunk
  const int g = lane >> 2, c = lane & 3;
  const bool q32 = a.q.dtype == PNB_F32;
  uint32_t u = 0, item = 0;
  bool ok = true;
  while (walk.next<kChunk>(a, a.seqs.each, it)) {
    ++item;
    const int rows = it.ntok * G;
    // queries as A operands, and the entries that each row sees
    uint32_t aq[RB][KS][4], ar[RB][KS][2];
    int lo[RB], hi[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r = b * 8 + g, rr = min(r, rows - 1);
      const int tok = it.tok0 + rr / G, head = it.h * G + rr % G;
      const int64_t at = tok * a.q.token + head * a.q.head + 2 * c;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        load_q2(a.q, at + 16 * k, aq[b][k][0], aq[b][k][1], ar[b][k][0]);
        load_q2(a.q, at + 16 * k + 8, aq[b][k][2], aq[b][k][3], ar[b][k][1]);
      }
      const int last = it.base + rr / G;
      hi[b] = last + 1;
      lo[b] = max(it.floor, a.window > 0 ? last - a.window + 1 : 0);
    }
    float o[RB][NT][4] = {}, m[RB], sum[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      m[b] = -INFINITY;
      sum[b] = 0.f;
    }

    // this lane's places of the warp's sums, where they meet at the end
    auto place = [&](int b, int n) {
      return reinterpret_cast<float2 *>(merge + ((warp * RB + b) * 8 + g) * L::LD + 2 * c + n * 8);
    };
    const bool folds = LONG && it.tb - it.ta > kFoldChunks;
    if (folds) {
#pragma unroll 1
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int b = 0; b < RB; ++b) *place(b, n) = make_float2(0.f, 0.f);
    }

    for (int t = it.ta; t < it.tb; ++t, ++u) {
      if ((u & 1) != half) continue;
      const int s = u % NS;
      if (ok && !mbar_wait(&bar.full[s], (u / NS) & 1)) {
        ok = false;
        set_error(a.err, kErrTimeout);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;
      const int e0 = (it.t0 + t) * kChunk + p0;
      const uint32_t ks = smem_addr(ring + s * L::STAGE), vs = ks + L::UNIT;
      const bool masked = e0 < it.lo_max || e0 + 16 > it.hi_min;
      if (masked && (e0 >= it.hi || e0 + 16 <= it.lo)) {   // no row sees any of the 16
        if (lane == 0) mbar_arrive(&bar.empty[s]);
        continue;
      }
      // S = Q K^T of two blocks of eight entries
      float sc[RB][2][4] = {};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int pos = p0 + (lane & 7) + (lane >> 4) * 8, col = (k & 3) * 2 + ((lane >> 3) & 1);
        uint32_t kb[4];
        ldmatrix4(ks + (k >> 2) * L::BOX + pos * 128 + ((col ^ (pos & 7)) << 4), kb);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          mma16816(sc[b][0], aq[b][k], kb[0], kb[1]);
          mma16816(sc[b][1], aq[b][k], kb[2], kb[3]);
          if (q32) {
            const uint32_t rest[4] = {ar[b][k][0], 0, ar[b][k][1], 0};
            mma16816(sc[b][0], rest, kb[0], kb[1]);
            mma16816(sc[b][1], rest, kb[2], kb[3]);
          }
        }
      }
      if (masked) {
        // V rows that no row sees become zero (0 x NaN is NaN), the others are searched
        // for NaN and infinities (a single token's rows all see the same)
        bool bad = false;
        for (int i = lane; i < 16 * HD / 8; i += 32) {
          const int pos = (i >> 3) & 15;
          uint4 *p = reinterpret_cast<uint4 *>(ring + s * L::STAGE + L::UNIT + (i >> 7) * L::BOX + (p0 + pos) * 128) + (i & 7);
          if (e0 + pos >= it.hi || e0 + pos < it.lo) {
            *p = make_uint4(0, 0, 0, 0);
          } else {
            const uint4 x = *p;
            auto odd = [](uint32_t w) { return (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u; };
            bad |= odd(x.x) || odd(x.y) || odd(x.z) || odd(x.w);
          }
        }
        if (bad && it.ntok > 1) *reinterpret_cast<volatile int *>(&bar.bad) = (int)item;
        fence_async_smem();
        __syncwarp();
      }
      // this lane's scores of row g: entries 2c, 2c + 1, 8 + 2c, 9 + 2c
      uint32_t ap[RB][4];
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        float x[4] = {sc[b][0][0] + sc[b][0][2], sc[b][0][1] + sc[b][0][3], sc[b][1][0] + sc[b][1][2],
                      sc[b][1][1] + sc[b][1][3]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] *= a.qscale;
          const int e = e0 + (i >> 1) * 8 + 2 * c + (i & 1);
          if (masked && (e < lo[b] || e >= hi[b])) x[i] = -INFINITY;
        }
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        if (__any_sync(0xffffffffu, top > m[b] + kTau)) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          if (top > m[b]) {
            const float f = m[b] == -INFINITY ? 0.f : exp2_approx(m[b] - top);
            m[b] = top;
            sum[b] *= f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[b][n][i] *= f;
            if (folds) {
#pragma unroll 1
              for (int n = 0; n < NT; ++n) *place(b, n) = make_float2(place(b, n)->x * f, place(b, n)->y * f);
            }
          }
        }
        const float ref = m[b] == -INFINITY ? 0.f : m[b];
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = exp2_approx(x[i] - ref);
        sum[b] += (p[0] + p[1]) + (p[2] + p[3]);
        ap[b][0] = pack_bf16(p[0], p[1]);
        ap[b][2] = pack_bf16(p[2], p[3]);
        ap[b][1] = pack_bf16(p[0] - bf16lo(ap[b][0]), p[1] - bf16hi(ap[b][0]));
        ap[b][3] = pack_bf16(p[2] - bf16lo(ap[b][2]), p[3] - bf16hi(ap[b][2]));
      }
      // O += P V
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        const int pos = p0 + (lane & 15), col = (n & 7) + (lane >> 4);
        uint32_t vb[4];
        ldmatrix4_trans(vs + (n >> 3) * L::BOX + pos * 128 + ((col ^ (pos & 7)) << 4), vb);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          mma16816(o[b][n], ap[b], vb[0], vb[1]);
          mma16816(o[b][n + 1], ap[b], vb[2], vb[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.empty[s]);
      if (folds && ((t - it.ta) | 1) % kFoldChunks == kFoldChunks - 1) {   // (one of two chunks is the warp's)
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float2 all = *place(b, n);
            *place(b, n) = make_float2(all.x + (o[b][n][0] + o[b][n][2]), all.y + (o[b][n][1] + o[b][n][3]));
#pragma unroll
            for (int i = 0; i < 4; ++i) o[b][n][i] = 0.f;
          }
      }
    }

    // the warps' parts of the item meet
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      sum[b] += __shfl_xor_sync(0xffffffffu, sum[b], 1);
      sum[b] += __shfl_xor_sync(0xffffffffu, sum[b], 2);
      if (c == 0) bar.ml[warp][b * 8 + g] = make_float2(m[b], sum[b]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 all = folds ? *place(b, n) : make_float2(0.f, 0.f);
        *place(b, n) = make_float2(all.x + (o[b][n][0] + o[b][n][2]), all.y + (o[b][n][1] + o[b][n][3]));
      }
    }
    consumer_sync<kWarps * 32>();
    const bool redo = *reinterpret_cast<volatile int *>(&bar.bad) == (int)item;
    const bool whole = it.ta == 0 && it.ends;
    const int side = it.ta > 0 ? 0 : 1;
    if (!whole && threadIdx.x == 0) a.part[2 * blockIdx.x + side] = PkvPart{it.ends ? 3 : 1, it.b, it.j, it.h};
    constexpr int N = HD / 32;
    for (int r = warp; r < rows; r += kWarps) {
      const int tok = it.tok0 + r / G, head = it.h * G + r % G;
      float x[N] = {}, mr = -INFINITY, sr = 0.f;
      if (!redo) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mr = fmaxf(mr, bar.ml[w][r].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 ml = bar.ml[w][r];
          const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - mr);
          const float *p = merge + ((w * RB + (r >> 3)) * 8 + (r & 7)) * L::LD + lane * N;
          float y[N];
          load_vals<float, N>(p, y);
#pragma unroll
          for (int i = 0; i < N; ++i) x[i] += f * y[i];
          sr += f * ml.y;
        }
      } else {
        // a NaN or an infinity among values that only some rows see: the row by itself
        const int last = it.base + r / G;
        const int from = max(max(it.floor, a.window > 0 ? last - a.window + 1 : 0), (it.t0 + it.ta) * kChunk);
        pkv_attend_row<HD>(a.pool, a.seqs.pages + (int64_t)it.b * a.seqs.max_page, it.h, a.q,
                           tok * a.q.token + head * a.q.head, a.qscale, from, min(last + 1, (it.t0 + it.tb) * kChunk), x,
                           mr, sr, &bar.work);
      }
      if (whole && a.pass == kPkvAll) {
        pkv_store<N>(a.out, tok * a.out.token + head * a.out.head + lane * N, x, sr == 0.f ? 0.f : 1.f / sr);
      } else {
        const int64_t at =
            whole ? (int64_t)tok * a.n_head + head : (int64_t)(2 * blockIdx.x + side) * kPkvBlockRows + r;
        float *po = whole ? a.row_o[1] : a.part_o, *pml = whole ? a.row_ml[1] : a.part_ml;
#pragma unroll
        for (int i = 0; i < N; ++i) po[at * HD + lane * N + i] = x[i];
        if (lane == 0) *reinterpret_cast<float2 *>(pml + at * 2) = make_float2(mr, sr);
      }
    }
    consumer_sync<kWarps * 32>();
  }
  if (a.pass == kPkvOwn) pdl_wait();
}

template <int HD, int RB, bool LONG>
cudaError_t launch_step(const CUtensorMap &map, const PkvAttnArgs &a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(a.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = SL<HD, RB>::SMEM;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_pkv_step<HD, RB, LONG>, map, a);
}

template <int HD, int RB>
cudaError_t launch_step(const CUtensorMap &map, const PkvAttnArgs &a, cudaStream_t st) {
  const int64_t room = (int64_t)a.seqs.max_page << a.pool.page_log2;
  return room > (a.out.dtype == PNB_F32 ? kLongF32 : kLongBf16) ? launch_step<HD, RB, true>(map, a, st)
                                                                 : launch_step<HD, RB, false>(map, a, st);
}

template <int HD, int RB>
cudaError_t prepare() {
  const cudaError_t e =
      cudaFuncSetAttribute(k_pkv_step<HD, RB, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SL<HD, RB>::SMEM);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(k_pkv_step<HD, RB, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SL<HD, RB>::SMEM);
}

}  // namespace

cudaError_t prepare_pkv_step(int hd) {
  cudaError_t e = hd == 128 ? prepare<128, 1>() : prepare<64, 1>();
  if (e != cudaSuccess || hd == 128) return e;
  return prepare<64, 2>();
}

// A chunk at the GPU's copy rate, shared out over its SMs.  64 slots behind a shared prefix (as at
// pkv_rows_cost) at 350, 500, 700, 1000 ns: head_dim 128 fp32 115, 104, 95, 108, bf16 94, 86, 84, 102; head_dim 64
// fp32 75, 86, 90, 100, bf16 63, 71, 74, 86.
void pkv_step_cost(int hd, int *unit_ns, int *item_units) {
  *unit_ns = hd == 128 ? 700 : 350;
  *item_units = 4;
}

cudaError_t launch_pkv_step(int hd, const CUtensorMap &map, const PkvAttnArgs &args, cudaStream_t st) {
  PkvAttnArgs a = args;
  pkv_step_cost(hd, &a.unit_ns, &a.item_units);
  const int rows = a.seqs.each * (a.n_head / a.pool.n_kv);
  if (hd == 128) return launch_step<128, 1>(map, a, st);
  return rows <= 8 ? launch_step<64, 1>(map, a, st) : launch_step<64, 2>(map, a, st);
}

}  // namespace pnb
