// pnb_kv4_attn.cu - decode attention over the 4-bit KV cache, and the
// accumulation of each cached position's attention weight.
//
// For the rows q_i of one KV head (the query heads of its group times the
// call's tokens), with keys k_j = d_jg (u_j - 8) per 32-dim block g:
//   x_ij = log2(e) / sqrt(hd) sum_g d_jg sum_{n in g} q_in (u_jn - 8)
//   o_i  = sum_j p_ij v_j / l_i,  p_ij = 2^(x_ij - ref_i),  l_i = sum_j p_ij
// and the same for the values: sum_j (p_ij d_jg) (u_jn - 8).
// Codes never become scaled numbers: the matrix instructions multiply the
// integers u - 8 (exact in fp16), so the only roundings are those of the fp32
// operand's split into two fp16 (22 bits) and of the fp32 sums.
//
// Both products take the codes as the A operand (m16n8k16: 16 positions of K by
// 16 dims, 16 dims of V by 16 positions) and the few rows as B's 8 columns:
//  - PAIR (up to four rows): columns 2 q and 2 q + 1 are the high and low fp16
//    parts of row q;
//  - otherwise a row per column, and a second product with the low parts onto the
//    same sums, SPLIT for the queries too: bf16 ones are exact in one fp16.
// Softmax weights are in two parts whatever the outputs' type, so that a bf16
// output is the rounding of what an fp32 one would be.
// Scores come out with a position per lane group r = lane / 4 and rows by c =
// lane % 4; a transposition of 8 x 8 fp16 turns them into B operands of the
// second product.
// (With the rows as A's 16 rows, high parts over low parts, both products took
// twice the matrix instructions and the outputs twice the registers.)
#include <cfloat>

#include "pnb_kv4.cuh"

namespace pnb {

namespace {

// Work units: an item (slot, KV head, block of 8 query rows) takes one per
// chunk of 32 positions and kItemUnits more for its queries and its end (21 slots x
// 4 heads x 3 blocks of rows, lengths up to 200, 10.9 us with one, 10.8 with two,
// 13.3 with three; 64 x 8 heads at 1200 27.6, 26.6, 27.3).
constexpr int kItemUnits = 2;
// While no item has more units than this, none is split over CTAs (head_dim 128,
// us, whole against split: 8 KV heads of one sequence 6 units 6.3, 9.2; 18 units
// 8.7, 9.4; 26 units 9.4, 9.5; 34 units 10.6, 9.6.  21 slots x 4 heads x 3 blocks
// of rows, lengths up to 200 10.8, 13.6; all 800 18.4, 18.9.  64 x 8 heads, all
// 100 11.2, 12.6; all 600 19.6, 18.5; all 1200 27.6, 26.5)
constexpr int kWholeUnits = 28;

template <int NG, bool PAIR, bool SPLIT>
struct AttnSmem {
  static constexpr int kHd = 32 * NG;
  static constexpr int kPitch = kHd + 8;      // floats between partial rows: lanes (r, c) write row c, dims 8 i + r
  static constexpr int kStages = NG == 4 ? 2 : 4;
  static constexpr int kChunk = kv4_chunk_bytes(NG);
  static constexpr int kRing = kKv4Warps * kStages * kChunk;
  static constexpr int kQSets = SPLIT && !PAIR ? 2 : 1;             // high and low parts apart
  static constexpr int kQ = kRing;                                  // uint2 [warps][sets][2 NG][32]
  static constexpr int kBars = kQ + kKv4Warps * kQSets * 2 * NG * 32 * 8;
  static constexpr int kPart = kBars + kKv4Warps * kStages * 8;     // int4 [2 warps]: item of each partial
  static constexpr int kMl = kPart + kKv4Warps * 2 * 16;            // float2 [2 warps][8]: reference, sum
  static constexpr int kFlag = kMl + kKv4Warps * 2 * kKv4Rows * 8;
  static constexpr int kSpan = kFlag + 16;                          // the CTA's units, the number of CTAs
  static constexpr int kPre = kSpan + 16;                           // int [n_slot + 1]
  static int bytes(int n_slot) { return kPre + (2 * n_slot + 3) * 4; }   // and the lengths, their count and largest
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same with a zero accumulator
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }
__device__ __forceinline__ uint32_t as_word(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ float2 half2_pair(uint32_t w) { return __half22float2(as_half2(w)); }

__device__ __forceinline__ uint32_t pack_half2(float2 v) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// the 8 x 8 matrix of fp16 whose row r lane (r, c) holds columns 2 c, 2 c + 1 of, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(w));
  return d;
}

template <int NG>
__device__ __forceinline__ void lds_words(const uint8_t *p, uint32_t (&w)[NG]) {
  if constexpr (NG == 4) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (NG == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

// what V scales below 2^ev are multiplied with, as a power of two
__device__ __forceinline__ int up_of(int ev) { return ev < -3 || ev > 0 ? -ev : 0; }

// the halves of a word that are finite, as a mask (scales have no sign)
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
  return ((w & 0xffffu) < 0x7c00u ? 0xffffu : 0u) | ((w >> 16) < 0x7c00u ? 0xffff0000u : 0u);
}

// The part of a warp's units [x, x1) that lies in one item: chunks [c0, c1) of
// the item's nch (none when only its extra units do), `units` units.
// first is the unit of the item's chunk 0: it identifies the item.
struct Segment {
  int b, h, rb, c0, c1, nch, units, first;
};

__device__ __forceinline__ Segment segment_at(const int *pre, const int *lens, const Kv4AttnArgs &a, int x, int x1) {
  Segment s;
  s.b = kv4_find(pre, a.n_slot, x);
  const int rel = x - pre[s.b];
  s.nch = (lens[s.b] + kKv4Chunk - 1) / kKv4Chunk;
  const int per = s.nch + kItemUnits;
  const int it = (int)((unsigned)rel / (unsigned)per), off = rel - it * per;
  s.h = it;
  s.rb = 0;
  if (a.nrb > 1) {
    s.h = (int)((unsigned)it / (unsigned)a.nrb);
    s.rb = it - s.h * a.nrb;
  }
  s.units = min(x1 - x, per - off);
  s.c0 = max(0, off - kItemUnits);
  s.c1 = max(0, off + s.units - kItemUnits);
  s.first = x - off + kItemUnits;
  return s;
}

// The first unit of the item that unit x belongs to.  Out of line: inlined, its
// code on the way of all calls cost 0.1 to 0.3 us each.
__device__ __noinline__ int item_start(const int *pre, const int *lens, int n_slot, int x) {
  const int b = kv4_find(pre, n_slot, x), per = (lens[b] + kKv4Chunk - 1) / kKv4Chunk + kItemUnits;
  return x - (int)((unsigned)(x - pre[b]) % (unsigned)per);
}

// The equal split of `total` units: part i of n takes [start(i), start(i + 1)),
// start(i) = floor(i total / n), in 32 bits (n < 2^13).
struct Split {
  int n, base, rem;
  __device__ __forceinline__ Split(int total, int parts) : n(parts) {
    base = (int)((unsigned)total / (unsigned)parts);
    rem = total - base * parts;
  }
  __device__ __forceinline__ int start(int i) const { return i * base + (int)((unsigned)(i * rem) / (unsigned)n); }
  // the part that holds unit u
  __device__ __forceinline__ int part_of(int u) const {
    int i = (int)((float)u * ((float)n / ((float)base * (float)n + (float)rem)));
    i = min(max(i, 0), n - 1);
    while (i > 0 && start(i) > u) --i;
    while (i + 1 < n && start(i + 1) <= u) ++i;
    return i;
  }
};

template <int N>
__device__ __forceinline__ void store_row(const DevRows &o, int64_t at, const float (&v)[N]) {
  if (o.dtype == PNB_F32) {
    float *p = static_cast<float *>(o.p) + at;
    if constexpr (N == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else if constexpr (N == 2) *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    else *p = v[0];
  } else {
    __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(o.p) + at;
    if constexpr (N == 1) {
      *p = __float2bfloat16_rn(v[0]);
    } else {
      __nv_bfloat162 h[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      if constexpr (N == 4) *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(h);
      else *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<uint32_t *>(h);
    }
  }
}

// N consecutive fp16 as fp32
template <int N>
__device__ __forceinline__ void lds_halves(const uint8_t *p, float (&v)[N]) {
  if constexpr (N == 4) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    const float2 x = half2_pair(w.x), y = half2_pair(w.y);
    v[0] = x.x; v[1] = x.y; v[2] = y.x; v[3] = y.y;
  } else if constexpr (N == 2) {
    const float2 x = half2_pair(*reinterpret_cast<const uint32_t *>(p));
    v[0] = x.x; v[1] = x.y;
  } else {
    v[0] = __half2float(*reinterpret_cast<const __half *>(p));
  }
}

template <int N>
__device__ __forceinline__ void ldcg_row(const float *p, float (&v)[N]) {
  if constexpr (N == 4) {
    const float4 u = __ldcg(reinterpret_cast<const float4 *>(p));
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  } else if constexpr (N == 2) {
    const float2 u = __ldcg(reinterpret_cast<const float2 *>(p));
    v[0] = u.x; v[1] = u.y;
  } else {
    v[0] = __ldcg(p);
  }
}

// What turns a row's scores into weights: 2^(x - ref) times the sum's reciprocal
// (as one number, ref + log2(sum) would round, most where scores are large).  A
// row with nothing to attend to gets weights of 0.
__device__ __forceinline__ float2 weight_scale(float ref, float sum) {
  return sum != 0.f ? make_float2(ref, 1.f / sum) : make_float2(INFINITY, 0.f);
}

// a row's output from its sums (lane: dims NG lane ..), and what its weights are scaled with
template <int NG, bool TRACK>
__device__ __forceinline__ void finish_row(const Kv4AttnArgs &a, int b, int h, int row, int lane, float mref,
                                           float lsum, float (&os)[NG]) {
  const int t = row / a.G, hq = h * a.G + (row - t * a.G);
  const float f = lsum != 0.f ? 1.f / lsum : 0.f;
#pragma unroll
  for (int i = 0; i < NG; ++i) os[i] = lsum != 0.f ? os[i] * f : 0.f;
  store_row<NG>(a.out, b * a.out.slot + t * a.out.token + hq * a.out.head + lane * NG, os);
  if (TRACK && lane == 0) a.wscale[((int64_t)b * a.n_kv + h) * a.rows + row] = weight_scale(mref, lsum);
}

// Every warp takes an equal, contiguous run of the units and works alone: its
// own ring of bulk copies (one chunk of K and V each, running on across
// items), its own queries and softmax state.  Items that lie in one warp are
// finished by it; the others leave partial rows, which the CTA adds up at its
// end, and for items shared by CTAs the last CTA to arrive does, all in the
// order of the units, so that results do not depend on the run.  (The CTA's
// warps on one item at a time pay two barriers and the queries' load for each.)
// The registers (128) leave 16 warps on an SM.  As one CTA of 16 they share fewer
// items between CTAs than as two of 8, whose barriers and merges are cheaper:
// 128k positions 58.0 us against 60.3, 64 ragged slots 41.5 against 42.7, 16 rows
// of 32 heads at 6007 28.9 against 31.0, 8 KV heads at 32768 15.7 against 16.8;
// but 32 MHA heads at 2048 10.0 against 9.3, 64 x 8 heads at 100 11.2 against 9.5.
// 64 slots at 512..4096 positions (8 x 4 heads, head_dim 128, fp32) take 41.3 us
// (3.8 TB/s), two contexts of 100k and 128k (bf16) 57.8 us (4.6 TB/s).  The bytes
// alone are 23 and 39 of that; the rest is launch, start (lengths, queries and
// first chunk in turn) and merges, which is all that short caches have, and the
// latency of a chunk's chain from codes to sums, at four warps per scheduler
// (issue slots 58 and 64 % busy over the launch, the integer pipe, which
// unpacks 8 codes in 9 instructions, 45 and 50 %).
template <int NG, bool PAIR, bool SPLIT, bool TRACK>
__global__ void __launch_bounds__(kKv4Threads, kKv4CtasPerSm)
    k_kv4_attn(const __grid_constant__ Kv4AttnArgs a) {
  static_assert(SPLIT || !PAIR, "pairs are split");
  using L = AttnSmem<NG, PAIR, SPLIT>;
  constexpr int HD = L::kHd, ST = L::kStages, PITCH = L::kPitch;
  constexpr int RPI = PAIR ? 4 : 8;           // rows per item
  constexpr int RL = PAIR ? 1 : 2;            // rows whose scores and outputs a lane holds
  static_assert(RPI <= kKv4Rows && 2 * RPI * PITCH * 4 <= ST * L::kChunk, "partial rows, in a warp's ring");
  extern __shared__ __align__(128) uint8_t smem[];
  int4 *spart = reinterpret_cast<int4 *>(smem + L::kPart);
  float2 *sml = reinterpret_cast<float2 *>(smem + L::kMl);
  int *sflag = reinterpret_cast<int *>(smem + L::kFlag);
  int4 *sspan = reinterpret_cast<int4 *>(smem + L::kSpan);
  int *pre = reinterpret_cast<int *>(smem + L::kPre), *lens = pre + a.n_slot + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  uint2 *qs = reinterpret_cast<uint2 *>(smem + L::kQ) + warp * L::kQSets * 2 * NG * 32 + lane;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars) + warp * ST;
  uint8_t *ring = smem + warp * ST * L::kChunk;

  pdl_wait();
  if (warp == 0) {
    kv4_prefix(a.l, a.n_slot, kKv4Chunk, kItemUnits, a.n_kv * a.nrb, pre, lens);
  } else {                                    // meanwhile
    if (warp == 1 && lane == 0) {
      for (int s = 0; s < kKv4Warps * ST; ++s) mbar_init(reinterpret_cast<uint64_t *>(smem + L::kBars) + s, 1);
      fence_barrier_init();
    }
    if (warp == 2 && lane < 2 * kKv4Warps) spart[lane].x = -1;
  }
  __syncthreads();
  const int total = pre[a.n_slot], cta = blockIdx.x;
  // One unit per warp at least, except that short items stay in one CTA: rows
  // shared by CTAs cost about 3 us more.
  const int items = lens[a.n_slot] * a.n_kv * a.nrb;
  const int longest = (lens[a.n_slot + 1] + kKv4Chunk - 1) / kKv4Chunk + kItemUnits;
  const bool whole = longest <= kWholeUnits;
  const bool each = whole && total == items * longest && items <= (int)gridDim.x;   // a CTA each
  const int ctas = max(1, min((int)gridDim.x, !whole ? total / kKv4Warps : each ? items : total));
  int x0, x1;
  {
    const Split by_cta(total, ctas);   // and each CTA's part is split over its warps the same way
    int u0 = by_cta.start(cta), u1 = by_cta.start(cta + 1);
    if (whole && !each) {              // the items that begin in it
      if (u0 < total) u0 = item_start(pre, lens, a.n_slot, u0);
      if (u1 < total) u1 = item_start(pre, lens, a.n_slot, u1);
    }
    x0 = u0 + (u1 - u0) * warp / kKv4Warps;
    x1 = u0 + (u1 - u0) * (warp + 1) / kKv4Warps;
    if (tid == 0) *sspan = make_int4(u0, u1, ctas, 0);   // for the end: the loop needs the registers
  }

  // slots with nothing to attend to answer zero
  for (int b = cta; b < a.n_slot; b += gridDim.x) {
    if (pre[b + 1] != pre[b]) continue;
    const float z[NG] = {};
    for (int i = tid; i < a.T * a.n_kv * a.G * 32; i += kKv4Threads) {
      const int row = i >> 5, t = row / (a.n_kv * a.G), hq = row - t * (a.n_kv * a.G);
      store_row<NG>(a.out, b * a.out.slot + t * a.out.token + hq * a.out.head + (i & 31) * NG, z);
    }
  }
  if (cta >= ctas || total == 0) return;

  // producer: next segment's first unit, next chunk, segment's end
  int px = x0, pc = 0, pc1 = 0;
  const uint8_t *pbase = nullptr;
  auto enter = [&](const Segment &ps) {
    px += ps.units;
    pc = ps.c0;
    pc1 = ps.c1;
    pbase = a.l.codes + ((int64_t)ps.b * a.n_kv + ps.h) * (a.l.cap / kKv4Chunk) * L::kChunk;
  };
  int pstage = 0;
  bool dead = false;
  auto produce = [&]() {           // copy the warp's next chunk, if any, into stage pstage
    while (pc >= pc1) {
      if (px >= x1) return;
      enter(segment_at(pre, lens, a, px, x1));
    }
    if (lane == 0 && !dead) {
      mbar_arrive_expect_tx(bars + pstage, L::kChunk);
      bulk_g2s(ring + pstage * L::kChunk, pbase + (int64_t)pc * L::kChunk, L::kChunk, bars + pstage);
    }
    ++pc;
    pstage = pstage + 1 == ST ? 0 : pstage + 1;
  };

  int stage = 0;
  uint32_t phase = 0;
  bool primed = false, early = false;
  auto early_part = [&]() { return a.warp_part + ((int64_t)blockIdx.x * kKv4Warps + warp) * kKv4Rows * HD + lane; };
  const int vunit_off = kv4_vunit(0, r, c);
  uint32_t magic = 0x64006400u;
  asm volatile("" : "+r"(magic));
#pragma unroll 1
  for (int x = x0; x < x1;) {
    const Segment sg = segment_at(pre, lens, a, x, x1);
    if (x == x0) enter(sg);
    x += sg.units;
    if (sg.c0 >= sg.c1) continue;
    const int len = lens[sg.b];
    const int row0 = sg.rb * RPI;
    // the lane's score rows are row0 + lane_row(k), k < RL; its column's row
    // (queries, weights) is row_col
    auto lane_row = [&](int k) { return PAIR ? c : 2 * c + k; };
    const int row_col = row0 + (PAIR ? r >> 1 : r);

    // Queries: lane (r, c) holds dims 32 g + 8 c .. + 7 of its column, which are
    // its own entries of the B operand.  Scaled to a largest magnitude of 2^10 by
    // a power of two that the scores undo; PAIR: high part in even columns.
    float rs[RL];
    {
      float v[NG][8];
      if (row_col < a.rows) {
        const int t = row_col / a.G, hq = sg.h * a.G + (row_col - t * a.G);
        const int64_t at = sg.b * a.q.slot + t * a.q.token + hq * a.q.head + 8 * c;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (SPLIT && a.q.dtype == PNB_F32) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q.p) + at + 32 * g);
            const float4 u = p[0], w = p[1];
            v[g][0] = u.x; v[g][1] = u.y; v[g][2] = u.z; v[g][3] = u.w;
            v[g][4] = w.x; v[g][5] = w.y; v[g][6] = w.z; v[g][7] = w.w;
          } else {
            load_vals<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16 *>(a.q.p) + at + 32 * g, v[g]);
          }
        }
      } else {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[g][i] = 0.f;
      }
      // the first copies go out behind the first queries' loads, which would
      // otherwise wait in their queue
      if (!primed) {
        primed = true;
#pragma unroll 1
        for (int s = 0; s < ST; ++s) produce();
      }
      float mx = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[g][i]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      int e = (int)(__float_as_uint(mx) >> 23) - 127;
      e = min(max(e, -100), 127);
      const float up = __uint_as_float((uint32_t)(10 - e + 127) << 23);
      const float scale = __uint_as_float((uint32_t)(e - 10 + 127) << 23) * a.qscale;
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // dims n, n + 4 with n = 2 h (b0) and 2 h + 1 (b1)
          uint32_t hi[2], lo[2] = {};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 y = make_float2(v[g][2 * h + k] * up, v[g][2 * h + k + 4] * up);
            hi[k] = pack_half2(y);
            if (SPLIT) {
              const float2 z = half2_pair(hi[k]);
              lo[k] = pack_half2(make_float2(y.x - z.x, y.y - z.y));
            }
          }
          const bool low = PAIR && (r & 1);
          qs[(g * 2 + h) * 32] = make_uint2(low ? lo[0] : hi[0], low ? lo[1] : hi[1]);
          if (SPLIT && !PAIR) qs[(2 * NG + g * 2 + h) * 32] = make_uint2(lo[0], lo[1]);
        }
      // the score rows' factors from the lanes of their columns
#pragma unroll
      for (int k = 0; k < RL; ++k) rs[k] = __shfl_sync(0xffffffffu, scale, PAIR ? 8 * c : 4 * (2 * c + k));
    }
    const int limit_all = len - a.T + 1;                       // every row sees positions below it
    int limit[RL];
    float *score[RL];
#pragma unroll
    for (int k = 0; k < RL; ++k) {
      const int row = row0 + lane_row(k);
      limit[k] = row < a.rows ? limit_all + row / a.G : 0;
      if (TRACK)
        score[k] = row < a.rows
                       ? a.scores + (((int64_t)sg.b * a.n_kv + sg.h) * a.rows + row) * a.l.cap + r
                       : nullptr;
    }

    float2 o[NG * 2][2];                                       // the products' accumulators, in 2^(ref - up_of(ev))
#pragma unroll
    for (int i = 0; i < NG * 2; ++i) o[i][0] = o[i][1] = make_float2(0.f, 0.f);
    float l[RL], ref[RL];                                      // sum (in 2^ref), reference
#pragma unroll
    for (int k = 0; k < RL; ++k) {
      l[k] = 0.f;
      ref[k] = -FLT_MAX;
    }
    int ev = 0;
#pragma unroll 1
    for (int ch = sg.c0; ch < sg.c1; ++ch) {
      if (!dead && !mbar_wait(bars + stage, phase)) {
        // a wait that gave up: no more copies; those in flight get another
        // bounded chance to land before the shared memory goes away
        dead = true;
        if (lane == 0) set_error(a.err, kErrTimeout);
        for (int s = 0; s < ST; ++s)
          mbar_wait(bars + (stage + s) % ST, stage + s < ST ? phase : phase ^ 1u);
      }
      const uint8_t *st = ring + stage * L::kChunk;
      const int p0 = ch * kKv4Chunk;
      const bool tail = p0 + kKv4Chunk > limit_all;

      // scores of position p0 + 8 t + r, row lane_row(k)
      float s[4][RL];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t kw[2][NG];
        float kd[2][NG];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = 8 * (2 * mt + h) + r;
          lds_words<NG>(st + kv4_kword(NG, p, c, 0), kw[h]);
          lds_halves<NG>(st + kv4_kscale_off(NG) + kv4_kscale(NG, p, 0), kd[h]);
#pragma unroll
          for (int k = 0; k < RL; ++k) s[2 * mt + h][k] = 0.f;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint32_t u0[4], u1[4];
          code_pairs(kw[0][g], magic, u0);
          code_pairs(kw[1][g], magic, u1);
          float d[4];
          {
            const uint2 qa = qs[(g * 2) * 32], qb = qs[(g * 2 + 1) * 32];
            mma_f16_new(d, u0[0], u1[0], u0[1], u1[1], qa.x, qa.y);
            mma_f16(d, u0[2], u1[2], u0[3], u1[3], qb.x, qb.y);
          }
          if (SPLIT && !PAIR) {
            const uint2 qa = qs[(2 * NG + g * 2) * 32], qb = qs[(2 * NG + g * 2 + 1) * 32];
            mma_f16(d, u0[0], u1[0], u0[1], u1[1], qa.x, qa.y);
            mma_f16(d, u0[2], u1[2], u0[3], u1[3], qb.x, qb.y);
          }
          if (PAIR) {
            s[2 * mt][0] = fmaf(d[0] + d[1], kd[0][g], s[2 * mt][0]);
            s[2 * mt + 1][0] = fmaf(d[2] + d[3], kd[1][g], s[2 * mt + 1][0]);
          } else {
#pragma unroll
            for (int k = 0; k < RL; ++k) {
              s[2 * mt][k] = fmaf(d[k], kd[0][g], s[2 * mt][k]);
              s[2 * mt + 1][k] = fmaf(d[2 + k], kd[1][g], s[2 * mt + 1][k]);
            }
          }
        }
      }
      // The scores, rounded once: the maximum, the weights and what is stored come
      // from the same numbers, so that at any size none lies above the maximum.
#pragma unroll
      for (int k = 0; k < RL; ++k)
#pragma unroll
        for (int t = 0; t < 4; ++t) s[t][k] = __fmul_rn(s[t][k], rs[k]);
      if (tail) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int k = 0; k < RL; ++k)
            if (p0 + 8 * t + r >= limit[k]) s[t][k] = -INFINITY;
      }
      if (TRACK) {
#pragma unroll
        for (int k = 0; k < RL; ++k)
          if (score[k]) {
#pragma unroll
            for (int t = 0; t < 4; ++t) score[k][p0 + 8 * t] = s[t][k];
          }
      }
      // The chunk's V scales lie below 2^evc (the finite ones, inside the sequence).
      // ev follows within a factor of 2^3; scales above 1, or all below 2^-3, are
      // brought to just below 1, in the chunk itself.
      constexpr int kWords = 16 * NG, kPer = (kWords + 31) / 32;
      uint32_t vw[kPer], both;          // the lane's words of V scales, and its two positions' largest
      bool uneven;                      // one of them has far smaller values than another position
      uint8_t *vscales = ring + stage * L::kChunk + kv4_vscale_off(NG) + (lane * kPer % kWords) * 4;
      auto scale_words = [&](uint32_t by) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          reinterpret_cast<uint32_t *>(vscales)[i] = as_word(__hmul2_rn(as_half2(vw[i]), as_half2(by)));
        // ahead of the copy that fills the stage again
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      };
      {
        lds_words<kPer>(vscales, vw);
        uint32_t outside = 0;           // the halves behind the sequence
        const int p = p0 + 2 * (lane * kPer % kWords / NG);
        if (tail) {
          outside = p >= len ? 0xffffffffu : (p + 1 >= len ? 0xffff0000u : 0u);
#pragma unroll
          for (int i = 0; i < kPer; ++i) vw[i] &= ~outside;
        }
        auto largest = [&](const uint32_t (&w)[kPer]) {
          const __half2 m = kPer == 2 ? __hmax2_nan(as_half2(w[0]), as_half2(w[kPer - 1])) : as_half2(w[0]);
          return NG == 1 ? as_word(m) : as_word(__hmax2_nan(m, as_half2(__shfl_xor_sync(0xffffffffu, as_word(m), 1))));
        };
        auto over_warp = [](uint32_t w) { return __reduce_max_sync(0xffffffffu, max(w & 0xffffu, w >> 16)); };
        both = largest(vw);
        uint32_t hmax = over_warp(both);
        if (hmax >= 0x7c00u) {          // a block of NaN: only the finite scales count
          uint32_t finite[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) finite[i] = vw[i] & finite_halves(vw[i]);
          both = largest(finite);
          hmax = over_warp(both);
          if (tail && a.T > 1) {
            // A weight of 0 times NaN is NaN: entries that not all rows see lose
            // their NaN here, and the rows that see them have it from now on.
            for (int q = max(limit_all, p0); q < min(len, p0 + kKv4Chunk); ++q) {
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                const uint32_t d = *reinterpret_cast<const uint16_t *>(st + kv4_vscale_off(NG) + kv4_vscale(NG, q - p0, g));
                if (d < 0x7c00u) continue;
#pragma unroll
                for (int i = 2 * g; i < 2 * g + 2; ++i)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    if (q < limit[0]) o[i][h].x = NAN;
                    if (q < limit[RL - 1]) o[i][h].y = NAN;
                  }
              }
            }
            __syncwarp();
            const uint32_t some = (p >= limit_all ? 0xffffu : 0u) | (p + 1 >= limit_all ? 0xffff0000u : 0u);
#pragma unroll
            for (int i = 0; i < kPer; ++i) vw[i] = (vw[i] & ~some) | (finite[i] & some);
          }
        }
        const uint32_t in = both | outside;
        const __half least = __ushort_as_half((unsigned short)min(in & 0xffffu, in >> 16));
        uneven = __hlt(__hmul(least, __ushort_as_half(0x5400)), __ushort_as_half((unsigned short)hmax));   // 64 times
        const int evc = (int)(hmax >> 10) - 14;
        if ((unsigned)(ev - evc) > 3u && hmax != 0) {
          const float more = __uint_as_float((uint32_t)(127 + up_of(evc) - up_of(ev)) << 23);
          ev = evc;
#pragma unroll
          for (int i = 0; i < NG * 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) o[i][h] = make_float2(o[i][h].x * more, o[i][h].y * more);
        }
        if (up_of(ev) != 0 || tail) {   // and what lies behind the sequence becomes 0
          const float f = __uint_as_float((uint32_t)(127 + up_of(ev)) << 23);
          scale_words(pack_half2(make_float2(f, f)));
        }
      }
      // p = 2^(x - ref) and p d in fp16: the reference follows the chunks' largest
      // scores in whole powers of two, with some play, so that a chunk's largest p lies
      // in 2^2 .. 2^15 whatever the chunks before it held (a first entry that takes
      // nearly all the weight, say).  Products keep 22 bits down to 2^-3 and lose one
      // per power of two from there.  (One reference for all chunks, that of the
      // largest score, left up to 4 % of error beside such an entry.  New references by
      // every chunk's own largest scores, with the sums' factors: 64 slots 47.5 us.)
      bool off = uneven;                // some row's reference does not fit
      float xmax[RL], lmul = 1.f;
#pragma unroll
      for (int k = 0; k < RL; ++k) {
        xmax[k] = fmaxf(fmaxf(s[0][k], s[1][k]), fmaxf(s[2][k], s[3][k]));
        const float d = xmax[k] - ref[k];
        const uint32_t near = __ballot_sync(0xffffffffu, !(d < 2.f));
        off |= d > 15.f;
        off |= (near & (0x11111111u << c)) == 0;
      }
      if (__any_sync(0xffffffffu, off)) {
        // Where positions' values are uneven (next to a first entry with a value of
        // zero), each position's V scales are brought to just below 1/2 and its
        // weight takes the power of two: the reference then goes by what the
        // positions add to the outputs.  The sum takes the weights as they are.
        const bool spread = __any_sync(0xffffffffu, uneven);
        float adj[4];
        if (spread) {
          auto field = [](uint32_t h) { return min(max(28 - (int)(h >> 10), 1), 28); };   // of 2^(field - 15)
          scale_words((uint32_t)field(both & 0xffffu) << 10 | (uint32_t)field(both >> 16) << 26);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t w = __shfl_sync(0xffffffffu, both, (4 * t + (r >> 1)) * (NG > 1 ? 2 : 1));
            const uint32_t h = (r & 1) ? w >> 16 : w & 0xffffu;
            adj[t] = h == 0 ? -INFINITY : (float)(up_of(ev) + 15 - field(h));
          }
        }
        const float room = spread ? 13.f : 15.f;
        float al[RL];
#pragma unroll
        for (int k = 0; k < RL; ++k) {
          auto over_rows = [](float x) {
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          };
          float xm = over_rows(xmax[k]), to = ref[k];
          // the sums stay below 2^80 or so, which bounds how far a reference falls
          const float lm = over_rows(l[k]);
          const float least = fmaxf(ceilf(__fadd_ru(xm, -60.f)), ref[k] + (float)((int)(__float_as_uint(lm) >> 23) - 187));
          if (spread)
            xm = over_rows(fmaxf(fmaxf(s[0][k] + adj[0], s[1][k] + adj[1]), fmaxf(s[2][k] + adj[2], s[3][k] + adj[3])));
          // (where scores are so large that the reference rounds, it rounds up)
          if (xm - to > room || (xm - to < room - 13.f && xm > -INFINITY)) to = ceilf(__fadd_ru(xm, 6.f - room));
          to = fmaxf(to, least);
          al[k] = ex2(ref[k] - to);
          ref[k] = to;
          l[k] *= al[k];
        }
#pragma unroll
        for (int i = 0; i < NG * 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) o[i][h] = make_float2(o[i][h].x * al[0], o[i][h].y * al[RL - 1]);
        if (spread) {
          lmul = 0.f;
#pragma unroll
          for (int k = 0; k < RL; ++k)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              l[k] += ex2(__fadd_rn(s[t][k], -ref[k]));
              s[t][k] += adj[t];
            }
        }
      }
      // softmax weights as columns: xh[t] holds the high parts of positions 8 t + 2 c,
      // + 1 of the lane's column's row, xl[t] the low parts (PAIR: 0 in even columns)
      uint32_t xh[4], xl[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float p[RL];
#pragma unroll
        for (int k = 0; k < RL; ++k) {
          p[k] = ex2(__fadd_rn(s[t][k], -ref[k]));
          l[k] = fmaf(p[k], lmul, l[k]);
        }
        if (PAIR) {
          const uint32_t h = pack_half2(make_float2(p[0], p[0]));
          xh[t] = transpose8(h);
          xl[t] = transpose8(pack_half2(make_float2(0.f, p[0] - __low2float(as_half2(h)))));
        } else {
          const uint32_t h = pack_half2(make_float2(p[0], p[RL - 1]));
          xh[t] = transpose8(h);
          const float2 z = half2_pair(h);
          xl[t] = transpose8(pack_half2(make_float2(p[0] - z.x, p[RL - 1] - z.y)));
        }
      }
      const uint32_t odd = (r & 1) ? 0xffffffffu : 0u;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint4 vw = *reinterpret_cast<const uint4 *>(st + kv4_v_off(NG) + g * 512 + vunit_off);
        uint32_t u[4][4];
        code_pairs(vw.x, magic, u[0]);
        code_pairs(vw.y, magic, u[1]);
        code_pairs(vw.z, magic, u[2]);
        code_pairs(vw.w, magic, u[3]);
        // p d in fp16: its rounding, and the rest of the exact product, the
        // rounding's residual (one fma) + p_lo d.  PAIR: the one in even columns,
        // the other in odd ones.
        uint32_t w[4], wl[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t dw = *reinterpret_cast<const uint32_t *>(st + kv4_vscale_off(NG) + (t * 4 + c) * 4 * NG + 4 * g);
          const __half2 d = as_half2(dw), h = as_half2(xh[t]);
          const uint32_t first = as_word(__hmul2_rn(h, d));
          w[t] = first;
          const uint32_t taken = PAIR ? first & odd : first;
          wl[t] = as_word(__hfma2(as_half2(xl[t]), d, __hfma2(h, d, __hneg2(as_half2(taken)))));
          if (PAIR) w[t] = wl[t];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float d[4];
          mma_f16_new(d, u[2 * j][0], u[2 * j + 1][0], u[2 * j][1], u[2 * j + 1][1], w[0], w[1]);
          mma_f16(d, u[2 * j][2], u[2 * j + 1][2], u[2 * j][3], u[2 * j + 1][3], w[2], w[3]);
          if (!PAIR) {
            mma_f16(d, u[2 * j][0], u[2 * j + 1][0], u[2 * j][1], u[2 * j + 1][1], wl[0], wl[1]);
            mma_f16(d, u[2 * j][2], u[2 * j + 1][2], u[2 * j][3], u[2 * j + 1][3], wl[2], wl[3]);
          }
          // fp32 sums by rounding additions (the matrix instruction cuts off: thousands
          // of entries with a common mean were 2e-6 too small)
          o[2 * g + j][0] = fadd2(o[2 * g + j][0], make_float2(d[0], d[1]));
          o[2 * g + j][1] = fadd2(o[2 * g + j][1], make_float2(d[2], d[3]));
        }
      }
      __syncwarp();
      produce();
      stage = stage + 1 == ST ? 0 : stage + 1;
      phase ^= stage == 0;
    }

    // the lane's outputs: row lane_row(k), dim 8 i + r
    const float vs = __uint_as_float((uint32_t)(127 - up_of(ev)) << 23);
    auto out_of = [&](int k, int i) {
      const float2 v = o[i >> 1][i & 1];
      return (PAIR ? v.x + v.y : k ? v.y : v.x) * vs;
    };
#pragma unroll
    for (int k = 0; k < RL; ++k) {
      l[k] += __shfl_xor_sync(0xffffffffu, l[k], 4);
      l[k] += __shfl_xor_sync(0xffffffffu, l[k], 8);
      l[k] += __shfl_xor_sync(0xffffffffu, l[k], 16);
    }
    if (sg.c0 == 0 && sg.c1 == sg.nch) {
#pragma unroll
      for (int k = 0; k < RL; ++k) {
        const int row = row0 + lane_row(k);
        if (row >= a.rows) continue;
        const int t = row / a.G, hq = sg.h * a.G + (row - t * a.G);
        const int64_t at = sg.b * a.out.slot + t * a.out.token + hq * a.out.head + r;
        const float f = l[k] != 0.f ? 1.f / l[k] : 0.f;
#pragma unroll
        for (int i = 0; i < NG * 4; ++i) {
          const float v[1] = {l[k] != 0.f ? out_of(k, i) * f : 0.f};
          store_row<1>(a.out, at + 8 * i, v);
        }
        if (TRACK && r == 0) a.wscale[((int64_t)sg.b * a.n_kv + sg.h) * a.rows + row] = weight_scale(ref[k], l[k]);
      }
    } else {
      const int which = sg.c0 == 0 ? 1 : 0;    // 1: the item starts here and goes on behind
      if (lane == 0) spart[2 * warp + which] = make_int4(sg.first, sg.nch, sg.b, sg.h * a.nrb + sg.rb);
      // the rows into the warp's ring once its last chunk is used; before that to
      // global memory
      float *pd = x >= x1 ? reinterpret_cast<float *>(ring) + which * RPI * PITCH : nullptr;
      early |= x < x1;
#pragma unroll
      for (int k = 0; k < RL; ++k) {
        const int i0 = lane_row(k);
        if (r == 0) sml[(2 * warp + which) * kKv4Rows + i0] = make_float2(ref[k], l[k]);
#pragma unroll
        for (int i = 0; i < NG * 4; ++i) {
          if (pd) pd[i0 * PITCH + r + 8 * i] = out_of(k, i);
          else early_part()[(k * NG * 4 + i) * 32] = out_of(k, i);
        }
      }
    }
  }
  if (early) {
#pragma unroll
    for (int k = 0; k < RL; ++k) {
      const int i0 = PAIR ? c : 2 * c + k;
#pragma unroll
      for (int i = 0; i < NG * 4; ++i)
        reinterpret_cast<float *>(ring)[i0 * PITCH + r + 8 * i] = early_part()[(k * NG * 4 + i) * 32];
    }
  }
  __syncthreads();

  const int4 span = *sspan;
  const int u0 = span.x, u1 = span.y;
  // The CTA's partial rows, in the units' order: entry 2 w is warp w's item
  // from before, 2 w + 1 the one that it starts.  Consecutive entries of one
  // item form a group; the warps share out the groups' rows.
  const int mine = lane < 2 * kKv4Warps ? spart[lane].x : -1;
  const uint32_t valid = __ballot_sync(0xffffffffu, mine >= 0), below = valid & ((1u << lane) - 1u);
  const int before = __shfl_sync(0xffffffffu, mine, below ? 31 - __clz(below) : 0);
  const uint32_t starts = __ballot_sync(0xffffffffu, mine >= 0 && (!below || before != mine));
  const int groups = __popc(starts), rows = min(RPI, a.rows);
  struct Item {
    int first, nch, b, h, rb;
  };
  auto item_of = [&](int4 e) {
    Item it = {e.x, e.y, e.z, e.w, 0};
    if (a.nrb > 1) {
      it.h = e.w / a.nrb;
      it.rb = e.w - it.h * a.nrb;
    }
    return it;
  };
#pragma unroll 1
  for (int task = warp; task < groups * rows; task += kKv4Warps) {
    const int gi = task / rows, i = task - gi * rows;
    uint32_t m = starts;
    for (int k = 0; k < gi; ++k) m &= m - 1u;
    const uint32_t rest = m & (m - 1u), begin = m & -m;          // begin: the group's first bit
    const uint32_t members = valid & ((rest & -rest) - begin);   // up to the next group's
    const Item it = item_of(spart[__ffs(begin) - 1]);
    const int my_row = it.rb * RPI + i;
    if (my_row >= a.rows) continue;
    // lane e holds entry e's factor
    const float2 ml = (members >> lane) & 1u ? sml[lane * kKv4Rows + i] : make_float2(0.f, 0.f);
    const float mref = warp_max(ml.y != 0.f ? ml.x : -INFINITY);
    float fac = ml.y != 0.f ? ex2(ml.x - mref) : 0.f;
    const float lsum = warp_sum(ml.y * fac);
    // 0 stands for no entry; an entry's factor of 0 is -0, which hands on a NaN
    if (fac == 0.f && ((members >> lane) & 1u)) fac = -0.f;
    float os[NG] = {};
#pragma unroll
    for (int e = 0; e < 2 * kKv4Warps; ++e) {
      const float f = __shfl_sync(0xffffffffu, fac, e);
      if (__float_as_uint(f) == 0u) continue;
      float v[NG];
      load_vals<float, NG>(reinterpret_cast<const float *>(smem + (e >> 1) * ST * L::kChunk) +
                               ((e & 1) * RPI + i) * PITCH + lane * NG, v);
#pragma unroll
      for (int j = 0; j < NG; ++j) os[j] = fmaf(v[j], f, os[j]);
    }
    if (it.first >= u0 && it.first + it.nch <= u1) {
      finish_row<NG, TRACK>(a, it.b, it.h, my_row, lane, mref, lsum, os);
    } else {
      const int64_t at = (int64_t)(2 * cta + (it.first >= u0 ? 1 : 0)) * kKv4Rows + i;
#pragma unroll
      for (int j = 0; j < NG; ++j) a.part[at * HD + lane * NG + j] = os[j];
      if (lane == 0) reinterpret_cast<float2 *>(a.part_ml)[at] = make_float2(mref, lsum);
    }
  }

  // items shared with other CTAs (the CTA's first and last at most): the last
  // CTA to arrive adds them up
  Item front = {}, back = {};
  bool at_front = false, at_back = false;
  if (groups > 0) {
    front = item_of(spart[__ffs(starts) - 1]);
    back = item_of(spart[31 - __clz(starts)]);
    at_front = front.first < u0;
    at_back = back.first + back.nch > u1 && !(at_front && back.first == front.first);
  }
  if (!at_front && !at_back) return;
  const int slot = tid - (kKv4Threads - 32);   // lanes 0 and 1 of the last warp: front and back
  int n = 0, c0 = 0;
  if (slot == 0 || slot == 1) {
    const Split by_cta(pre[a.n_slot], span.z);
    const Item it = slot ? back : front;
    if (slot ? at_back : at_front) {
      c0 = by_cta.part_of(it.first);
      n = by_cta.part_of(it.first + it.nch - 1) - c0 + 1;
    }
  }
  __syncthreads();
  if (slot == 0 || slot == 1) {
    if (n > 0) {
      // releases the CTA's partial rows (ordered by the barrier before), acquires the others'
      unsigned seen;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(seen) : "l"(a.counter + c0) : "memory");
      if (seen == (unsigned)(n - 1)) a.counter[c0] = 0;
      else n = 0;
    }
    sflag[2 * slot] = n;
    sflag[2 * slot + 1] = c0;
  }
  __syncthreads();
  // front and back at once where the warps suffice
  constexpr bool BOTH = 2 * RPI <= kKv4Warps;
#pragma unroll 1
  for (int i = BOTH ? warp / RPI : 0; i < 2; i += BOTH ? 2 : 1) {
    n = sflag[2 * i];
    c0 = sflag[2 * i + 1];
    const Item it = i ? back : front;
    const int w = BOTH ? warp % RPI : warp, my_row = it.rb * RPI + w;
    if (n == 0 || w >= RPI || my_row >= a.rows) continue;
    // the first CTA's partial is its second one, all others' their first
    auto at = [&](int k) { return (int64_t)(2 * (c0 + k) + (k == 0 ? 1 : 0)) * kKv4Rows + w; };
    auto ml_of = [&](int k) {
      return k < n ? __ldcg(reinterpret_cast<const float2 *>(a.part_ml) + at(k)) : make_float2(0.f, 0.f);
    };
    constexpr int AHEAD = 16;                // rows' loads in flight
    float v[AHEAD][NG];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int q = 0; q < AHEAD; ++q)
        if (k0 + q < n) ldcg_row<NG>(a.part + at(k0 + q) * HD + lane * NG, v[q]);
    };
    float2 ml = ml_of(lane);                 // lane k: partial k
    fetch(0);
    float mref = ml.y != 0.f ? ml.x : -INFINITY, lsum = 0.f, fac = 0.f, os[NG] = {};
    for (int k = lane + 32; k < n; k += 32) {
      const float2 x = ml_of(k);
      if (x.y != 0.f) mref = fmaxf(mref, x.x);
    }
    mref = warp_max(mref);
    for (int k0 = 0; k0 < n; k0 += AHEAD) {
      if (k0 > 0) fetch(k0);
      if (k0 % 32 == 0) {                    // the factors of the next 32
        if (k0 > 0) ml = ml_of(k0 + lane);
        fac = ml.y != 0.f ? ex2(ml.x - mref) : 0.f;
        lsum += warp_sum(ml.y != 0.f ? ml.y * fac : 0.f);
      }
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        const float f = __shfl_sync(0xffffffffu, fac, (k0 + q) & 31);
        if (k0 + q < n) {
#pragma unroll
          for (int j = 0; j < NG; ++j) os[j] = fmaf(v[q][j], f, os[j]);
        }
      }
    }
    finish_row<NG, TRACK>(a, it.b, it.h, my_row, lane, mref, lsum, os);
  }
}

// weights[j] = decay * weights[j] + sum over the rows of 2^(x_ij - ref_i) / l_i: each
// position has one owner that adds its rows in order.  Bound by latency (8 slots
// at 512..4096, 8 x 4 heads: 4 us behind the attention's 13) and, with many rows,
// by the scores' bytes (16 rows of 32 heads at 6007 positions, 12 MB: 6 us).
// Each thread has four positions; PARTS groups of threads share out the rows of
// the same positions, and the first adds up the groups' sums in order.
constexpr int kWeightThreads = 128, kWeightCtasPerSm = 8;

template <int PARTS>
__global__ void __launch_bounds__(kWeightThreads) k_kv4_weights(const __grid_constant__ Kv4WeightArgs a) {
  constexpr int GROUP = kWeightThreads / PARTS, UNIT = 4 * GROUP;
  extern __shared__ __align__(16) uint8_t wsmem[];
  float4 *sums = reinterpret_cast<float4 *>(wsmem);       // [PARTS - 1][GROUP]
  int *wpre = reinterpret_cast<int *>(sums + (PARTS - 1) * GROUP);
  const int part = PARTS == 1 ? 0 : threadIdx.x / GROUP, at = threadIdx.x % GROUP;
  pdl_wait();
  if (threadIdx.x < 32) kv4_prefix(a.l, a.n_slot, UNIT, 0, a.n_kv, wpre, nullptr);
  __syncthreads();
  const int total = wpre[a.n_slot], per_part = (a.rows + PARTS - 1) / PARTS;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const int b = kv4_find(wpre, a.n_slot, u), rel = u - wpre[b];
    const int per = (wpre[b + 1] - wpre[b]) / a.n_kv, h = rel / per;
    const int len = kv4_len(a.l, b);
    const int p = (rel - h * per) * UNIT + 4 * at;
    if (PARTS == 1 && p >= len) continue;
    const int64_t bh = (int64_t)b * a.n_kv + h;
    const float *x = a.scores + bh * a.rows * a.l.cap + p;
    const float2 *scale = a.wscale + bh * a.rows;
    float w[4] = {};
    float *dst = a.l.weights + bh * a.l.cap + p;
    float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool live = PARTS == 1 || p < len;
    if (live && part == 0 && a.decay > 0.f) old = *reinterpret_cast<const float4 *>(dst);
    const int end = PARTS == 1 ? a.rows : live ? min((part + 1) * per_part, a.rows) : 0;
    for (int i0 = PARTS == 1 ? 0 : part * per_part; i0 < end; i0 += 8) {     // eight rows' loads in flight
      float4 v[8];
      float2 z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = min(i0 + i, end - 1);
        v[i] = *reinterpret_cast<const float4 *>(x + (int64_t)row * a.l.cap);
        z[i] = i0 + i < end ? scale[row] : make_float2(INFINITY, 0.f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[0] = fmaf(ex2(v[i].x - z[i].x), z[i].y, w[0]); w[1] = fmaf(ex2(v[i].y - z[i].x), z[i].y, w[1]);
        w[2] = fmaf(ex2(v[i].z - z[i].x), z[i].y, w[2]); w[3] = fmaf(ex2(v[i].w - z[i].x), z[i].y, w[3]);
      }
    }
    if constexpr (PARTS > 1) {
      if (part > 0) sums[(part - 1) * GROUP + at] = make_float4(w[0], w[1], w[2], w[3]);
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int k = 0; k < PARTS - 1; ++k) {
          const float4 s = sums[k * GROUP + at];
          w[0] += s.x; w[1] += s.y; w[2] += s.z; w[3] += s.w;
        }
      }
      __syncthreads();
    }
    if (part > 0) continue;
    const float held[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p + i < len) dst[i] = a.decay > 0.f ? fmaf(a.decay, held[i], w[i]) : w[i];
  }
}

template <int NG>
cudaError_t prepare(int *sms) {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto k, int smem) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  auto set_both = [&](auto plain, auto track, int smem) {
    set(plain, smem);
    set(track, smem);
  };
  set_both(k_kv4_attn<NG, false, false, false>, k_kv4_attn<NG, false, false, true>,
           AttnSmem<NG, false, false>::bytes(kKv4MaxSlots));
  set_both(k_kv4_attn<NG, false, true, false>, k_kv4_attn<NG, false, true, true>,
           AttnSmem<NG, false, true>::bytes(kKv4MaxSlots));
  set_both(k_kv4_attn<NG, true, true, false>, k_kv4_attn<NG, true, true, true>,
           AttnSmem<NG, true, true>::bytes(kKv4MaxSlots));
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e;
}

template <int NG, bool PAIR, bool SPLIT>
cudaError_t run_attn(Kv4AttnArgs a, int grid, cudaStream_t st) {
  constexpr int rows = PAIR ? 4 : 8;
  a.nrb = (a.rows + rows - 1) / rows;
  const int smem = AttnSmem<NG, PAIR, SPLIT>::bytes(a.n_slot);
  auto kern = a.scores ? k_kv4_attn<NG, PAIR, SPLIT, true> : k_kv4_attn<NG, PAIR, SPLIT, false>;
  return launch_pdl(kern, dim3(grid), dim3(kKv4Threads), smem, 1, st, a);
}

template <int NG>
cudaError_t run_attn(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  if (a.rows <= 4) return run_attn<NG, true, true>(a, grid, st);
  return a.q.dtype == PNB_BF16 ? run_attn<NG, false, false>(a, grid, st) : run_attn<NG, false, true>(a, grid, st);
}

}  // namespace

cudaError_t prepare_kv4_kernels(int ng, int *sms) {
  return ng == 4 ? prepare<4>(sms) : ng == 2 ? prepare<2>(sms) : prepare<1>(sms);
}

cudaError_t launch_kv4_attn(int ng, const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  return ng == 4 ? run_attn<4>(a, grid, st) : ng == 2 ? run_attn<2>(a, grid, st) : run_attn<1>(a, grid, st);
}

template <int PARTS>
cudaError_t run_weights(const Kv4WeightArgs &a, cudaStream_t st) {
  constexpr int unit = 4 * kWeightThreads / PARTS;
  const int64_t units = (int64_t)a.n_slot * a.n_kv * ((a.l.cap + unit - 1) / unit);
  const int64_t most = (int64_t)kWeightCtasPerSm * a.sms;
  const int grid = (int)(units < most ? units : most);
  const int smem = (PARTS - 1) * (kWeightThreads / PARTS) * 16 + (a.n_slot + 1) * 4;
  return launch_pdl(k_kv4_weights<PARTS>, dim3(grid), dim3(kWeightThreads), smem, 1, st, a);
}

cudaError_t launch_kv4_weights(const Kv4WeightArgs &a, cudaStream_t st) {
  // rows in one or four parts, tracked attention at head_dim 64, us: 64 rows, 2
  // slots at 367 14.7, 12.3; 56 rows, 14 at 958 22.5, 18.6; 64 rows, 8 x 32768 69.3,
  // 69.0; 24 rows, 15 x 20000 35.1, 37.0; 16 rows, 64 x 8 at 1000 43.2, 47.9
  return a.rows < 32 ? run_weights<1>(a, st) : run_weights<4>(a, st);
}

}  // namespace pnb
