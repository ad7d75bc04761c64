// pnb_kv4.cu - the 4-bit KV cache's append (quantisation), read-back and
// eviction kernels.  Layout: pnb_kv4.cuh.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "pnb_kv4.cuh"

namespace cg = cooperative_groups;

namespace pnb {

namespace {

// ------------------------------------------------------------------ append
// One Q4_0 block is held by 4 neighbouring lanes, 8 dims each:
//   d = fp16(max|x| / 7), u = clamp(rint(x / d), -8, 7) + 8
// with correctly rounded quotients.  rint(x / d) is taken as rint(x * (1 / d)),
// which can be off by one next to a border, and put right from the residual
// x - k d (one fma, exact there: x lies within a factor of two of k d, or k is
// 0): a residual beyond d / 2, or of exactly d / 2 with k odd (ties go to the
// even integer), moves k by one.
// NaN and infinities make the block's scale NaN; a scale past fp16's range
// saturates.
__device__ __forceinline__ uint32_t q4_word(const float (&x)[8], __half *scale) {
  uint32_t top = 0;   // as integers, magnitudes order like floats, NaN on top
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (top >= 0x7f800000u) {
    *scale = __ushort_as_half((unsigned short)0x7fffu);
    return 0x88888888u;
  }
  const __half d = __float2half_rn(fminf(__fdiv_rn(__uint_as_float(top), 7.f), 65504.f));
  *scale = d;
  const float df = __half2float(d);
  if (df == 0.f) return 0x88888888u;
  const float inv = __frcp_rn(df), half_d = 0.5f * df;
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float big = 12582912.f;                 // 1.5 * 2^23: adding it rounds to an integer
    float k = __fadd_rn(__fmaf_rn(x[i], inv, big), -big);
    const float e = __fmaf_rn(-k, df, x[i]);
    if (fabsf(e) >= half_d && (fabsf(e) > half_d || (__float_as_uint(k + big) & 1u))) k += copysignf(1.f, e);
    k = fminf(fmaxf(k, -8.f), 7.f);
    w = (w << 4) | (__float_as_uint(k + (big + 8.f)) & 15u);
  }
  return w;
}

template <typename T>
__device__ __forceinline__ void load8(const void *p, int64_t at, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    load_vals<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16 *>(p) + at, x);
  } else {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
    const float4 u = q[0], v = q[1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
  }
}

constexpr int kAppendThreads = 256;

// One CTA per (chunk, KV head, slot): 128 threads quantise the chunk's new K
// rows, 128 its new V rows (16 bytes or 32 of a row per thread).  K words go
// straight to their place; V words hold 8 positions of one dim, so the codes
// cross shared memory, and a chunk that already holds entries keeps their
// nibbles.  Bound by the rows' bytes; a single token by its dependent loads.
template <int NG, typename T>
__global__ void __launch_bounds__(kAppendThreads) k_kv4_append(const __grid_constant__ Kv4AppendArgs a) {
  constexpr int TPR = 4 * NG;                     // threads (words) per row
  constexpr int RPP = 128 / TPR;                  // rows per pass: 8, 16, 32
  constexpr int PASSES = kKv4Chunk / RPP;
  __shared__ __align__(16) uint32_t vcode[kKv4Chunk][TPR];
  const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y;
  pdl_wait();
  const int len = kv4_len(a.l, b), seen = a.l.seen[b];
  int start = a.start ? a.start[b] : len;
  int n = a.n_new ? a.n_new[b] : a.T;
  int bad = 0;
  if (start < 0 || start > len || n < 0 || n > a.T) {
    bad = kErrRange;                              // the slot stays as it was
    start = len;
    n = 0;
  }
  if (n > a.l.cap - start) {
    bad = kErrFull;                               // rows past the capacity are not stored
    n = a.l.cap - start;
  }
  const int end = start + n;
  const int seen0 = seen - (len - start);         // id of the first new entry
  const int ch = start / kKv4Chunk + (int)blockIdx.x, p0 = ch * kKv4Chunk;
  const int lo = max(start, p0), hi = min(end, p0 + kKv4Chunk);
  if (lo < hi) {
    const int64_t bh = (int64_t)b * a.n_kv + h;
    uint8_t *chunk = a.l.codes + (bh * (a.l.cap / kKv4Chunk) + ch) * kv4_chunk_bytes(NG);
    const bool is_v = tid >= 128;
    const int th = tid & 127, sub = th % TPR, j = sub >> 2, cc = sub & 3, r0 = th / TPR;
    const Kv4Rows &rows = is_v ? a.v : a.k;
    uint8_t *scales = chunk + (is_v ? kv4_vscale_off(NG) : kv4_kscale_off(NG));
    const int64_t base = b * rows.slot + h * rows.head + sub * 8 + (int64_t)(p0 - start) * rows.token;
    float x[PASSES][8];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int p = r0 + i * RPP;
      if (p0 + p >= lo && p0 + p < hi) {
        load8<T>(rows.p, base + p * rows.token, x[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int p = r0 + i * RPP;
      const bool live = p0 + p >= lo && p0 + p < hi;
      __half d;
      const uint32_t w = q4_word(x[i], &d);
      if (is_v) vcode[p][sub] = w;
      else if (live) *reinterpret_cast<uint32_t *>(chunk + kv4_kword(NG, p, cc, j)) = w;
      if (live && cc == 0)
        *reinterpret_cast<__half *>(scales + (is_v ? kv4_vscale(NG, p, j) : kv4_kscale(NG, p, j))) = d;
    }
    if (tid < kKv4Chunk && p0 + tid >= lo && p0 + tid < hi) {
      a.l.ids[bh * a.l.cap + p0 + tid] = seen0 + (p0 + tid - start);
      a.l.weights[bh * a.l.cap + p0 + tid] = 0.f;
    }
    __syncthreads();
    if (tid < 32 * NG) {                          // unit (J, r, c): 4 dims of 8 positions
      const int J = tid >> 5, r = (tid >> 2) & 7, c = tid & 3;
      uint32_t w[4] = {}, fresh = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int p = 8 * (k >> 1) + 2 * c + (k & 1), sh = 4 * ((k >> 1) + 4 * (k & 1));
        const uint4 q = *reinterpret_cast<const uint4 *>(&vcode[p][J * 4]);
        if (p0 + p >= lo && p0 + p < hi) fresh |= 15u << sh;
        w[0] |= ((q.x >> (4 * r)) & 15u) << sh;
        w[1] |= ((q.y >> (4 * r)) & 15u) << sh;
        w[2] |= ((q.z >> (4 * r)) & 15u) << sh;
        w[3] |= ((q.w >> (4 * r)) & 15u) << sh;
      }
      uint4 *dst = reinterpret_cast<uint4 *>(chunk + kv4_v_off(NG) + kv4_vunit(J, r, c));
      if (fresh == 0xffffffffu) {
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (fresh) {
        const uint4 old = *dst;
        *dst = make_uint4((old.x & ~fresh) | (w[0] & fresh), (old.y & ~fresh) | (w[1] & fresh),
                          (old.z & ~fresh) | (w[2] & fresh), (old.w & ~fresh) | (w[3] & fresh));
      }
    }
  }
  // the slot's last CTA moves its length: all have read the old one
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    const unsigned ctas = gridDim.x * gridDim.y;
    if (atomicInc(a.arrive + b, ctas - 1) == ctas - 1) {
      if (bad) set_error(a.err, bad);
      if (bad != kErrRange) {
        a.l.len[b] = end;
        a.l.seen[b] = seen0 + n;
      }
    }
  }
}

// -------------------------------------------------------------------- read
template <typename T>
__device__ __forceinline__ void store8(void *p, int64_t at, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + at) = *reinterpret_cast<uint4 *>(v);
  } else {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
    q[0] = make_float4(x[0], x[1], x[2], x[3]);
    q[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

constexpr int kReadThreads = 256;

// One CTA per (chunk, KV head, slot): the chunk through shared memory, then 8
// dims of one position per thread and store (one word of K codes; one nibble
// of each of 8 V words).  Bound by the values' bytes.
template <int NG, typename T>
__global__ void __launch_bounds__(kReadThreads) k_kv4_read(const __grid_constant__ Kv4ReadArgs a) {
  constexpr int CH = kv4_chunk_bytes(NG);
  __shared__ __align__(16) uint8_t sm[CH];
  const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y;
  pdl_wait();
  const int len = kv4_len(a.l, b);
  int first = a.first ? a.first[b] : 0;
  first = first < 0 || first > a.l.cap ? a.l.cap : first;   // outside the cache: nothing but zeros
  const int ch = first / kKv4Chunk + (int)blockIdx.x, p0 = ch * kKv4Chunk;
  const int64_t last = (int64_t)first + a.T;
  const int lo = max(first, p0), hi = (int)min(last, (int64_t)p0 + kKv4Chunk);
  if (lo >= hi) return;
  if (p0 < len) {
    const uint4 *src = reinterpret_cast<const uint4 *>(
        a.l.codes + (((int64_t)b * a.n_kv + h) * (a.l.cap / kKv4Chunk) + ch) * CH);
    for (int i = tid; i < CH / 16; i += kReadThreads) reinterpret_cast<uint4 *>(sm)[i] = src[i];
  }
  __syncthreads();
  for (int i = tid; i < 2 * kKv4Chunk * 4 * NG; i += kReadThreads) {
    const bool is_v = i >= kKv4Chunk * 4 * NG;
    const int k = is_v ? i - kKv4Chunk * 4 * NG : i;
    const int p = k / (4 * NG), w8 = k % (4 * NG), j = w8 >> 2, sub = w8 & 3, pos = p0 + p;
    if (pos < lo || pos >= hi) continue;
    float x[8] = {};
    if (pos < len) {
      if (!is_v) {
        const float d = __half2float(*reinterpret_cast<const __half *>(sm + kv4_kscale_off(NG) + kv4_kscale(NG, p, j)));
        const uint32_t w = *reinterpret_cast<const uint32_t *>(sm + kv4_kword(NG, p, sub, j));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = d * (float)((int)((w >> (4 * e)) & 15u) - 8);
      } else {
        const float d = __half2float(*reinterpret_cast<const __half *>(sm + kv4_vscale_off(NG) + kv4_vscale(NG, p, j)));
        const int c = (p >> 1) & 3, sh = kv4_vshift(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w = *reinterpret_cast<const uint32_t *>(sm + kv4_v_off(NG) + kv4_vunit(j, e, c) + 4 * sub);
          x[e] = d * (float)((int)((w >> sh) & 15u) - 8);
        }
      }
    }
    const Kv4Rows &o = is_v ? a.v : a.k;
    store8<T>(o.p, b * o.slot + (int64_t)(pos - first) * o.token + h * o.head + w8 * 8, x);
  }
}

// ---------------------------------------------------------------- eviction
// Selection, one thread-block cluster per (slot, KV head), the entries' keys
// in registers: entries that must stay have the largest key, the others an
// order-preserving image of their weight.  A radix descent (four 8-bit levels)
// finds the key of rank `budget`; of the entries with exactly that key the
// first ones stay.  Then the kept entries behind the budget ("movers") fill
// the dropped ones' places below it ("holes"), both in index order:
// src_of[hole r] = mover r.
template <int THREADS, int K>
__global__ void __launch_bounds__(THREADS) k_kv4_select(const __grid_constant__ Kv4EvictArgs a) {
  constexpr int WARPS = THREADS / 32, COPIES = 8;
  __shared__ uint32_t hist[COPIES][256];
  __shared__ uint32_t merged[2][256];
  __shared__ uint32_t warp_sum[WARPS], totals[4];
  __shared__ uint32_t s_bin, s_need;
  cg::cluster_group cluster = cg::this_cluster();
  const int CL = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  const int n = kv4_len(a.src, b), seen = a.src.seen[b], m = a.budget;
  const int64_t bh = (int64_t)b * a.n_kv + h;
  const int32_t *ids = a.src.ids + bh * a.src.cap;
  const float *wt = a.src.weights + bh * a.src.cap;
  int32_t *src_of = a.src_of + bh * a.src.cap, *movers = a.movers + bh * a.src.cap;
  // (uniform over the cluster)
  if (n > m) {
    const int base = rank * THREADS * K + warp * 32 * K + lane;   // this lane's entries: base + 32 k
    uint32_t key[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = base + 32 * k;
      key[k] = 0;
      if (i < n) {
        const int id = ids[i];
        const uint32_t u = __float_as_uint(wt[i]);
        const bool stays = id < a.n_sink || (int64_t)id >= (int64_t)seen - a.n_recent;
        key[k] = stays ? 0xffffffffu : ((u & 0x80000000u) ? ~u : (u | 0x80000000u));
      }
    }
    uint32_t prefix = 0, need = (uint32_t)m;   // the need-th largest among keys with this prefix
    uint32_t equal = 0;
#pragma unroll 1
    for (int level = 0; level < 4; ++level) {
      const int sh = 24 - 8 * level;
      for (int i = tid; i < COPIES * 256; i += THREADS) (&hist[0][0])[i] = 0;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const bool in = base + 32 * k < n && (level == 0 || (key[k] >> (sh + 8)) == prefix);
        if (in) atomicAdd(&hist[warp % COPIES][(key[k] >> sh) & 255u], 1u);
      }
      __syncthreads();
      uint32_t *mine = merged[level & 1];
      for (int i = tid; i < 256; i += THREADS) {
        uint32_t s = 0;
#pragma unroll
        for (int q = 0; q < COPIES; ++q) s += hist[q][i];
        mine[i] = s;
      }
      if (CL > 1) cluster.sync();
      else __syncthreads();
      // warp 0: totals over the cluster, then the bin in which the running
      // count from the top reaches `need` (lane l holds bins 255 - 8 l - 7 ..)
      if (warp == 0) {
        uint32_t v[8], sum = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] = 0;
          for (int c = 0; c < CL; ++c)
            v[q] += CL > 1 ? *cluster.map_shared_rank(mine + 255 - 8 * lane - q, c) : mine[255 - 8 * lane - q];
          sum += v[q];
        }
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += u;
        }
        uint32_t above = inc - sum;
        if (above < need && need <= inc) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            if (above < need && need <= above + v[q]) {
              s_bin = 255 - 8 * lane - q;
              s_need = need - above;
              totals[0] = v[q];
            }
            above += v[q];
          }
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | s_bin;
      need = s_need;
      equal = totals[0];
      __syncthreads();
    }
    // the first `need` of the `equal` entries with key == prefix stay
    auto ranks = [&](uint32_t mine, int slot) -> uint32_t {
      // exclusive base of this warp's count over the cluster, in index order
      if (lane == 0) warp_sum[warp] = mine;
      __syncthreads();
      uint32_t before = 0, all = 0;
      for (int w = 0; w < WARPS; ++w) {
        const uint32_t s = warp_sum[w];
        before += w < warp ? s : 0;
        all += s;
      }
      if (CL > 1) {
        if (tid == 0) totals[slot] = all;
        cluster.sync();
        for (int c = 0; c < rank; ++c) before += *cluster.map_shared_rank(&totals[slot], c);
      }
      __syncthreads();
      return before;
    };
    uint32_t kept = 0;                             // bit k: entry base + 32 k stays
    if (need == equal) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (base + 32 * k < n && key[k] >= prefix) kept |= 1u << k;
    } else {
      uint32_t mine = 0;
#pragma unroll
      for (int k = 0; k < K; ++k)
        mine += __popc(__ballot_sync(0xffffffffu, base + 32 * k < n && key[k] == prefix));
      uint32_t at = ranks(mine, 1);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const bool eq = base + 32 * k < n && key[k] == prefix;
        const uint32_t vote = __ballot_sync(0xffffffffu, eq);
        const bool first = eq && at + __popc(vote & ((1u << lane) - 1u)) < need;
        at += __popc(vote);
        if (base + 32 * k < n && (key[k] > prefix || first)) kept |= 1u << k;
      }
    }
    uint32_t holes = 0, moves = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = base + 32 * k;
      const bool s = (kept >> k) & 1u;
      holes += __popc(__ballot_sync(0xffffffffu, i < m && !s));
      moves += __popc(__ballot_sync(0xffffffffu, i >= m && s));
    }
    uint32_t hole_at = ranks(holes, 2), move_at = ranks(moves, 3);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = base + 32 * k;
      const bool go = i >= m && ((kept >> k) & 1u);
      const uint32_t vote = __ballot_sync(0xffffffffu, go);
      if (go) movers[move_at + __popc(vote & ((1u << lane) - 1u))] = i;
      move_at += __popc(vote);
    }
    __threadfence();
    if (CL > 1) cluster.sync();
    else __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = base + 32 * k;
      const bool hole = i < m && !((kept >> k) & 1u);
      const uint32_t vote = __ballot_sync(0xffffffffu, hole);
      if (i < m) src_of[i] = hole ? __ldcg(movers + hole_at + __popc(vote & ((1u << lane) - 1u))) : i;
      hole_at += __popc(vote);
    }
    if (CL > 1) cluster.sync();   // no CTA leaves while a peer may read its shared memory
  }
  __syncthreads();                // every thread has read the old length
  if (tid == 0) {
    if (h == 0 && rank == 0) a.n_old[b] = n;
    __threadfence();
    const unsigned ctas = gridDim.x * gridDim.y;
    if (atomicInc(a.arrive + b, ctas - 1) == ctas - 1) {
      a.dst.len[b] = min(n, m);
      a.dst.seen[b] = seen;
    }
  }
}

constexpr int kMoveThreads = 128;

// The moves, one CTA per (destination chunk, KV head, slot).  Sources of moves
// lie at or behind the budget and destinations below it, so the CTAs do not
// depend on one another; in the chunk that holds the budget's border a V word
// may be read by others while its owner replaces it, with the nibbles that they
// read unchanged (32-bit accesses).
template <int NG>
__global__ void __launch_bounds__(kMoveThreads) k_kv4_move(const __grid_constant__ Kv4EvictArgs a) {
  constexpr int CH = kv4_chunk_bytes(NG);
  __shared__ int src[kKv4Chunk];
  const int tid = threadIdx.x, h = blockIdx.y, b = blockIdx.z, p0 = blockIdx.x * kKv4Chunk;
  pdl_wait();
  const int n = a.n_old[b], out = min(n, a.budget);
  if (p0 >= out || (a.in_place && n <= a.budget)) return;
  const int64_t bh = (int64_t)b * a.n_kv + h;
  const uint8_t *from = a.src.codes + bh * (a.src.cap / kKv4Chunk) * CH;
  uint8_t *to = a.dst.codes + (bh * (a.dst.cap / kKv4Chunk) + blockIdx.x) * CH;
  int moved = 0;
  if (tid < kKv4Chunk) {
    const int p = p0 + tid;
    int s = -1;
    if (p < out) {
      s = n > a.budget ? a.src_of[bh * a.src.cap + p] : p;
      moved = s != p;
      if (!a.in_place || moved) {
        a.dst.ids[bh * a.dst.cap + p] = a.src.ids[bh * a.src.cap + s];
        a.dst.weights[bh * a.dst.cap + p] = a.src.weights[bh * a.src.cap + s];
      }
    }
    src[tid] = s;
  }
  if (!__syncthreads_or(moved) && a.in_place) return;
  // K codes and both kinds of scales, row by row
  for (int i = tid; i < kKv4Chunk * 4 * NG; i += kMoveThreads) {
    const int p = i / (4 * NG), w = i % (4 * NG), s = src[p];
    if (s < 0 || (a.in_place && s == p0 + p)) continue;
    const uint8_t *chunk = from + (int64_t)(s / kKv4Chunk) * CH;
    const int q = s % kKv4Chunk;
    *reinterpret_cast<uint32_t *>(to + p * 16 * NG + w * 4) =
        *reinterpret_cast<const uint32_t *>(chunk + q * 16 * NG + w * 4);
    if (w < 2 * NG) {
      const int j = w % NG;
      const int into = w < NG ? kv4_kscale_off(NG) + kv4_kscale(NG, p, j) : kv4_vscale_off(NG) + kv4_vscale(NG, p, j);
      const int out_of = w < NG ? kv4_kscale_off(NG) + kv4_kscale(NG, q, j) : kv4_vscale_off(NG) + kv4_vscale(NG, q, j);
      *reinterpret_cast<uint16_t *>(to + into) = *reinterpret_cast<const uint16_t *>(chunk + out_of);
    }
  }
  // V codes: unit (J, r, c) holds 4 dims of 8 positions
  for (int u = tid; u < 32 * NG; u += kMoveThreads) {
    const int J = u >> 5, r = (u >> 2) & 7, c = u & 3;
    const uint4 old = *reinterpret_cast<const uint4 *>(from + (int64_t)blockIdx.x * CH + kv4_v_off(NG) +
                                                       kv4_vunit(J, r, c));
    uint32_t w[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int p = 8 * (k >> 1) + 2 * c + (k & 1), s = src[p];
      if (s < 0 || s == p0 + p) continue;
      const int q = s % kKv4Chunk, from_sh = kv4_vshift(q), sh = kv4_vshift(p);
      const uint4 v = *reinterpret_cast<const uint4 *>(from + (int64_t)(s / kKv4Chunk) * CH + kv4_v_off(NG) +
                                                       kv4_vunit(J, r, (q >> 1) & 3));
      w[0] = (w[0] & ~(15u << sh)) | (((v.x >> from_sh) & 15u) << sh);
      w[1] = (w[1] & ~(15u << sh)) | (((v.y >> from_sh) & 15u) << sh);
      w[2] = (w[2] & ~(15u << sh)) | (((v.z >> from_sh) & 15u) << sh);
      w[3] = (w[3] & ~(15u << sh)) | (((v.w >> from_sh) & 15u) << sh);
    }
    *reinterpret_cast<uint4 *>(to + kv4_v_off(NG) + kv4_vunit(J, r, c)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__global__ void k_kv4_reset(int32_t *len, int32_t *seen, int64_t stride, int n_layer, int n_slot, int slot) {
  pdl_wait();
  const int n = n_layer * n_slot;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
    const int l = i / n_slot, b = i - l * n_slot;
    if (slot >= 0 && b != slot) continue;
    len[l * stride + b] = 0;
    seen[l * stride + b] = 0;
  }
}

template <int NG>
cudaError_t run_append(const Kv4AppendArgs &a, cudaStream_t st) {
  // T rows from any position touch at most this many chunks
  const dim3 grid((a.T + kKv4Chunk - 2) / kKv4Chunk + 1, a.n_kv, a.n_slot);
  return a.k.dtype == PNB_F32 ? kv4_launch(k_kv4_append<NG, float>, grid, dim3(kAppendThreads), 0, 1, st, a)
                              : kv4_launch(k_kv4_append<NG, __nv_bfloat16>, grid, dim3(kAppendThreads), 0, 1, st, a);
}

template <int NG>
cudaError_t run_read(const Kv4ReadArgs &a, cudaStream_t st) {
  const dim3 grid((a.T + kKv4Chunk - 2) / kKv4Chunk + 1, a.n_kv, a.n_slot);
  return a.k.dtype == PNB_F32 ? kv4_launch(k_kv4_read<NG, float>, grid, dim3(kReadThreads), 0, 1, st, a)
                              : kv4_launch(k_kv4_read<NG, __nv_bfloat16>, grid, dim3(kReadThreads), 0, 1, st, a);
}

template <int NG>
cudaError_t run_move(const Kv4EvictArgs &a, cudaStream_t st) {
  const int most = a.budget < a.src.cap ? a.budget : a.src.cap;
  const dim3 grid((most + kKv4Chunk - 1) / kKv4Chunk, a.n_kv, a.n_slot);
  return kv4_launch(k_kv4_move<NG>, grid, dim3(kMoveThreads), 0, 1, st, a);
}

}  // namespace

cudaError_t launch_kv4_append(int ng, const Kv4AppendArgs &a, cudaStream_t st) {
  return ng == 4 ? run_append<4>(a, st) : ng == 2 ? run_append<2>(a, st) : run_append<1>(a, st);
}

cudaError_t launch_kv4_read(int ng, const Kv4ReadArgs &a, cudaStream_t st) {
  return ng == 4 ? run_read<4>(a, st) : ng == 2 ? run_read<2>(a, st) : run_read<1>(a, st);
}

cudaError_t launch_kv4_evict(int ng, const Kv4EvictArgs &a, cudaStream_t st) {
  // entries per CTA and CTAs per cluster that hold the whole capacity in registers
  const int per = a.src.cap <= 8 * 256 * 16 ? 256 * 16 : a.src.cap <= 8 * 1024 * 16 ? 1024 * 16 : 1024 * 32;
  int cl = 1;
  while (cl * per < a.src.cap) cl *= 2;
  const dim3 grid(cl, a.n_kv, a.n_slot);
  cudaError_t e;
  if (per == 256 * 16) e = kv4_launch(k_kv4_select<256, 16>, grid, dim3(256), 0, cl, st, a);
  else if (per == 1024 * 16) e = kv4_launch(k_kv4_select<1024, 16>, grid, dim3(1024), 0, cl, st, a);
  else e = kv4_launch(k_kv4_select<1024, 32>, grid, dim3(1024), 0, cl, st, a);
  if (e != cudaSuccess) return e;
  return ng == 4 ? run_move<4>(a, st) : ng == 2 ? run_move<2>(a, st) : run_move<1>(a, st);
}

cudaError_t launch_kv4_reset(int32_t *len, int32_t *seen, int64_t layer_stride, int n_layer, int n_slot,
                             int slot, cudaStream_t st) {
  k_kv4_reset<<<1, 256, 0, st>>>(len, seen, layer_stride, n_layer, n_slot, slot);
  return cudaGetLastError();
}

}  // namespace pnb
