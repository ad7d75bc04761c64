// pnb_kv4.cu - the 4-bit KV cache's append (quantisation), read-back and
// eviction kernels.  Layout: pnb_kv4.cuh.
#include <cooperative_groups.h>

#include "pnb_kv4.cuh"

namespace cg = cooperative_groups;

namespace pnb {

namespace {

// 8 x 8 nibbles transposed: nibble j of word i becomes nibble i of word j.
__device__ __forceinline__ void transpose_nibbles(uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {          // halves of rows i and i + 4
    const uint32_t a = w[i], b = w[i + 4];
    w[i] = __byte_perm(a, b, 0x5410);
    w[i + 4] = __byte_perm(a, b, 0x7632);
  }
#pragma unroll
  for (int g = 0; g < 8; g += 4)
#pragma unroll
    for (int i = g; i < g + 2; ++i) {    // bytes of rows i and i + 2
      const uint32_t a = w[i], b = w[i + 2];
      w[i] = __byte_perm(a, b, 0x6240);
      w[i + 2] = __byte_perm(a, b, 0x7351);
    }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {       // nibbles of rows i and i + 1
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
    w[i + 1] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
  }
}

// position (0..31 in a chunk) of nibble n of a V word of class c
__device__ __forceinline__ int vpos(int c, int n) { return 8 * (n & 3) + 2 * c + (n >> 2); }

// ------------------------------------------------------------------ append
// 8 consecutive elements, as loaded
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const void *p, int64_t at) {
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + at);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = q[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    if constexpr (sizeof(T) == 2) {
      load_vals<__nv_bfloat16, 8>(reinterpret_cast<const __nv_bfloat16 *>(v), x);
    } else {
      x[0] = __uint_as_float(v[0].x); x[1] = __uint_as_float(v[0].y);
      x[2] = __uint_as_float(v[0].z); x[3] = __uint_as_float(v[0].w);
      x[4] = __uint_as_float(v[1].x); x[5] = __uint_as_float(v[1].y);
      x[6] = __uint_as_float(v[1].z); x[7] = __uint_as_float(v[1].w);
    }
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }

// largest magnitude of the 8, NaN when one is
__device__ __forceinline__ float top8(const Raw8<float> &r) {
  float x[8], top = 0.f;
  r.floats(x);
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(x[i]));
  return top;
}
__device__ __forceinline__ float top8(const Raw8<__nv_bfloat16> &r) {
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(r.v);
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
  return max_nan(__low2float(m), __high2float(m));
}

// The codes, where they are hard to round: from the residual x - k d (one fma,
// exact near a border: x lies within a factor of two of k d, or k is 0), one
// beyond d / 2, or of exactly d / 2 with k odd (ties go to the even integer),
// moves k by one; and quotients outside [-8, 7] (a subnormal scale is coarse).
__device__ __noinline__ uint32_t q4_word_checked(float4 a, float4 b, float df, float inv) {
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, big = 12582912.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    float k = __fadd_rn(__fmaf_rn(x[i], inv, big), -big);
    const float e = __fmaf_rn(-k, df, x[i]), half_d = 0.5f * df;
    if (fabsf(e) > half_d || (fabsf(e) == half_d && (__float_as_uint(k + big) & 1u))) k += copysignf(1.f, e);
    k = fminf(fmaxf(k, -8.f), 7.f);
    w = (w << 4) | (__float_as_uint(k + big) & 15u);
  }
  return w ^ 0x88888888u;                // + 8 modulo 16
}

// A block's scale from its largest magnitude: d = fp16(max|x| / 7), the quotient
// correctly rounded by one residual step (Markstein's correction).  NaN and infinities make it NaN; a
// scale past fp16's range saturates.
struct Q4Scale {
  __half d;
  float df;      // d, or 0 where all codes are 8
  bool hard;     // some quotients round outside [-8, 7] (7.5 itself to the even 8)
  __device__ __forceinline__ explicit Q4Scale(float top) {
    const float seventh = 1.f / 7.f, q0 = __fmul_rn(top, seventh);
    const float quot = __fmaf_rn(__fmaf_rn(-q0, 7.f, top), seventh, q0);
    const bool finite = top < INFINITY;  // false for NaN too
    d = __float2half_rn(fminf(quot, 65504.f));
    df = finite ? __half2float(d) : 0.f;
    hard = df != 0.f && top >= 7.5f * df;
    if (!finite) d = __ushort_as_half((unsigned short)0x7fffu);
  }
};

// u = clamp(rint(x / d), -8, 7) + 8 of 8 elements, from x * (1 / d), whose error
// of a few units matters next to a border only:
//  - bf16: x has 8 bits and d 11, so x / d is exactly half an integer or at
//    least 2^-12 away from one; rounded to a multiple of 2^-13 first, the
//    approximate quotient then rounds as the exact one does, ties included.
//  - fp32: blocks with a residual of d / 2 or more are done again, checked.
// Adding 1.5 * 2^23 rounds to an integer and leaves it in the sum's low bits;
// the codes are added up from those modulo 2^32.
template <typename T>
__device__ __forceinline__ uint32_t q4_codes(const Raw8<T> &raw, float df, bool hard) {
  float x[8];
  raw.floats(x);
  const float big = 12582912.f;          // 1.5 * 2^23
  constexpr uint32_t kBits = 0x4b400000u, kBias = 0x88888888u - kBits * 0x11111111u;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(df));
  float off = 0.f;
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = make_float2(x[2 * i], x[2 * i + 1]);
    float2 k;
    if (sizeof(T) == 2) {
      k = fadd2(ffma2(v, dup(inv), dup(1536.f)), dup(big - 1536.f));
    } else {
      k = ffma2(v, dup(inv), dup(big));
      const float2 e = ffma2(fadd2(k, dup(-big)), dup(-df), v);
      off = fmaxf(off, fmaxf(fabsf(e.x), fabsf(e.y)));
    }
    b[2 * i] = __float_as_uint(k.x);
    b[2 * i + 1] = __float_as_uint(k.y);
  }
  if (df == 0.f) return 0x88888888u;
  if ((sizeof(T) == 4 && off >= 0.5f * df) || hard)
    return q4_word_checked(make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7]), df, inv);
#pragma unroll
  for (int o = 1; o < 8; o *= 2)
#pragma unroll
    for (int i = 0; i < 8; i += 2 * o) b[i] += b[i + o] << (4 * o);
  return b[0] + kBias;
}

// One Q4_0 block is held by 4 neighbouring lanes, 8 dims each.
template <typename T>
__device__ __forceinline__ uint32_t q4_word(const Raw8<T> &raw, __half *scale) {
  float top = top8(raw);
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const Q4Scale q(top);
  *scale = q.d;
  return q4_codes(raw, q.df, q.hard);
}

// N blocks at once: the four lanes share out the blocks' scales; lane cc < N
// answers that of block cc.
template <int N, typename T>
__device__ __forceinline__ __half q4_words(const Raw8<T> (&raw)[N], uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "blocks per four lanes");
  const int lane = threadIdx.x & 31;
  float t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = top8(raw[i]);
  if constexpr (N == 4) {
    const bool up = lane & 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float theirs = __shfl_xor_sync(0xffffffffu, up ? t[i] : t[i + 2], 2);
      t[i] = max_nan(up ? t[i + 2] : t[i], theirs);
    }
  }
  if constexpr (N >= 2) {
    const float theirs = __shfl_xor_sync(0xffffffffu, (lane & 1) ? t[0] : t[1], 1);
    t[0] = max_nan((lane & 1) ? t[1] : t[0], theirs);
  } else {
    t[0] = max_nan(t[0], __shfl_xor_sync(0xffffffffu, t[0], 1));
  }
  if constexpr (N < 4) t[0] = max_nan(t[0], __shfl_xor_sync(0xffffffffu, t[0], 2));
  const Q4Scale q(t[0]);
  const bool hard = __any_sync(0xffffffffu, q.hard);
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = q4_codes(raw[i], __shfl_sync(0xffffffffu, q.df, (lane & ~3) | i), hard);
  return q.d;
}

// What a slot's append does, from the device's counts.
struct AppendRange {
  int start, end, seen0, bad;   // entries [start, end), id of the first
  __device__ __forceinline__ AppendRange(const Kv4AppendArgs &a, int b) {
    const int len = kv4_len(a.l, b), seen = a.l.seen[b];
    int n = a.n_new ? a.n_new[b] : a.T;
    start = a.start ? a.start[b] : len;
    bad = 0;
    if (start < 0 || start > len || n < 0 || n > a.T) {
      bad = kErrRange;          // the slot stays as it was
      start = len;
      n = 0;
    }
    if (n > a.l.cap - start) {
      bad = kErrFull;           // rows past the capacity are not stored
      n = a.l.cap - start;
    }
    end = start + n;
    seen0 = seen - (len - start);
  }
  __device__ __forceinline__ void commit(const Kv4AppendArgs &a, int b) const {
    if (bad) set_error(a.err, bad);
    if (bad != kErrRange) {
      a.l.len[b] = end;
      a.l.seen[b] = seen0 + (end - start);
    }
  }
};

// Few tokens: one CTA per slot, so that it alone reads and moves the length.
// First every (token, head, K or V) row is quantised, TPR threads each; then
// each 16-byte unit of V words (8 positions of 4 dims) that holds a new
// position is read, completed and written by one thread.  Bound by its four
// dependent trips to memory (one token of 64 slots x 8 heads, bf16: 2.6 us).
constexpr int kStepThreads = 512;

template <int NG, typename T>
__global__ void __launch_bounds__(kStepThreads) k_kv4_append_step(const __grid_constant__ Kv4AppendArgs a) {
  constexpr int TPR = 4 * NG, CH = kv4_chunk_bytes(NG);
  extern __shared__ __align__(16) uint32_t vrow[];       // [T][n_kv][TPR] V codes
  const int tid = threadIdx.x, b = blockIdx.x;
  pdl_wait();
  const AppendRange r(a, b);
  const int n = r.end - r.start, rows = n * a.n_kv;
  uint8_t *slot = a.l.codes + (int64_t)b * a.n_kv * (a.l.cap / kKv4Chunk) * CH;
  auto chunk_of = [&](int h, int pos) { return slot + ((int64_t)h * (a.l.cap / kKv4Chunk) + pos / kKv4Chunk) * CH; };
  // whole warps run the block maximum's shuffles: 2 rows TPR is a multiple of 32 only by padding
  const int work = (2 * rows * TPR + 31) / 32 * 32;
  for (int i = tid; i < work; i += kStepThreads) {
    const int row = i / TPR, sub = i % TPR, rr = row >> 1, h = rr % a.n_kv, t = rr / a.n_kv;
    const bool live = rr < rows, is_v = row & 1;
    const Kv4Rows &src = is_v ? a.v : a.k;
    Raw8<T> raw;
    if (live) raw.load(src.p, b * src.slot + t * src.token + h * src.head + sub * 8);
    else raw.clear();
    __half d;
    const uint32_t w = q4_word(raw, &d);
    if (!live) continue;
    const int pos = r.start + t, p = pos % kKv4Chunk, j = sub >> 2, cc = sub & 3;
    uint8_t *chunk = chunk_of(h, pos);
    if (is_v) vrow[(t * a.n_kv + h) * TPR + sub] = w;
    else *reinterpret_cast<uint32_t *>(chunk + kv4_kword(NG, p, cc, j)) = w;
    if (cc == 0)
      *reinterpret_cast<__half *>(chunk + (is_v ? kv4_vscale_off(NG) + kv4_vscale(NG, p, j)
                                                : kv4_kscale_off(NG) + kv4_kscale(NG, p, j))) = d;
    if (sub == 0 && !is_v) {
      const int64_t at = ((int64_t)b * a.n_kv + h) * a.l.cap + pos;
      a.l.ids[at] = r.seen0 + t;
      a.l.weights[at] = 0.f;
    }
  }
  __syncthreads();
  // units (h, J, rr, token): the first token of its chunk and class does the unit's work
  for (int i = tid; i < rows * 8 * NG; i += kStepThreads) {
    const int rr = i % 8, J = (i / 8) % NG, h = (i / (8 * NG)) % a.n_kv, t0 = i / (8 * NG * a.n_kv);
    const int pos = r.start + t0, c = (pos >> 1) & 3;
    bool first = true;
    for (int t = 0; t < t0; ++t) {
      const int q = r.start + t;
      first &= q / kKv4Chunk != pos / kKv4Chunk || ((q >> 1) & 3) != c;
    }
    if (!first) continue;
    uint4 *unit = reinterpret_cast<uint4 *>(chunk_of(h, pos) + kv4_v_off(NG) + kv4_vunit(J, rr, c));
    uint4 u = *unit;
    for (int t = t0; t < n; ++t) {
      const int q = r.start + t;
      if (q / kKv4Chunk != pos / kKv4Chunk || ((q >> 1) & 3) != c) continue;
      const int sh = kv4_vshift(q % kKv4Chunk);
      const uint4 w = *reinterpret_cast<const uint4 *>(vrow + (t * a.n_kv + h) * TPR + 4 * J);
      const uint32_t keep = ~(15u << sh);
      u.x = (u.x & keep) | (((w.x >> (4 * rr)) & 15u) << sh);
      u.y = (u.y & keep) | (((w.y >> (4 * rr)) & 15u) << sh);
      u.z = (u.z & keep) | (((w.z >> (4 * rr)) & 15u) << sh);
      u.w = (u.w & keep) | (((w.w >> (4 * rr)) & 15u) << sh);
    }
    *unit = u;
  }
  if (tid == 0) r.commit(a, b);
}

// Many tokens: CTAs of up to kAppendChunks chunks of one (slot, KV head).  128
// threads quantise a chunk's new K rows, 128 its V rows, 16 bytes of a row (32
// for fp32) per thread and pass, the next chunk's rows on their way meanwhile.
// K words go straight to their place; V words hold 8 positions of one dim, so
// 8 x 8 nibbles are transposed by one thread each through shared memory, and a
// chunk that already holds entries keeps their nibbles.  The last of the slot's
// CTAs to have read the length moves it.  Bound by the rows' bytes in fp32
// (8191 tokens of 32 heads at head_dim 128 in 48.9 us, 6.3 TB/s) and by the
// quantiser's instructions in bf16 (32.8 us, 5.2 TB/s; at head_dim 64 4.2 TB/s).
// Four CTAs per SM: fp32 would take 71 registers and 52.3 us instead of 50.4.
constexpr int kAppendThreads = 256, kAppendChunks = 8;

template <int NG, typename T>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 4 ? 4 : 0) k_kv4_append(const __grid_constant__ Kv4AppendArgs a) {
  constexpr int TPR = 4 * NG;                     // threads (words) per row
  constexpr int RPP = 128 / TPR;                  // rows per pass: 8, 16, 32
  constexpr int PASSES = kKv4Chunk / RPP;
  constexpr int VP = TPR + 4;                     // V row pitch in words, against bank conflicts
  __shared__ __align__(16) uint32_t vcode[2][kKv4Chunk * VP];
  const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y;
  pdl_wait();
  const AppendRange rg(a, b);
  __syncthreads();
  if (tid == 0) {                                 // all the CTA's threads have read the old length
    __threadfence();
    const unsigned ctas = gridDim.x * gridDim.y;
    if (atomicInc(a.arrive + b, ctas - 1) == ctas - 1) rg.commit(a, b);
  }
  const int64_t bh = (int64_t)b * a.n_kv + h;
  const bool is_v = tid >= 128;
  const int th = tid & 127, sub = th % TPR, j = sub >> 2, cc = sub & 3, r0 = th / TPR;
  const Kv4Rows &rows = is_v ? a.v : a.k;
  const int ch0 = rg.start / kKv4Chunk + (int)blockIdx.x * a.group;
  const int ch1 = min(ch0 + a.group, (rg.end + kKv4Chunk - 1) / kKv4Chunk);
  const T *src = static_cast<const T *>(rows.p) + b * rows.slot + h * rows.head + sub * 8;
  Raw8<T> raw[PASSES];
  auto fetch = [&](int ch) {
    const int first = ch * kKv4Chunk + r0 - rg.start, count = rg.end - rg.start;
    const T *at = src + first * rows.token;
    if (ch * kKv4Chunk >= rg.start && (ch + 1) * kKv4Chunk <= rg.end) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) raw[i].load(at + i * (RPP * rows.token), 0);
    } else {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int t = first + i * RPP;
        if (t >= 0 && t < count) raw[i].load(at + i * (RPP * rows.token), 0);
        else raw[i].clear();
      }
    }
  };
  if (ch0 < ch1) fetch(ch0);
  for (int ch = ch0; ch < ch1; ++ch) {
    const int p0 = ch * kKv4Chunk, lo = max(rg.start, p0) - p0, hi = min(rg.end - p0, kKv4Chunk);
    uint8_t *chunk = a.l.codes + (bh * (a.l.cap / kKv4Chunk) + ch) * kv4_chunk_bytes(NG);
    uint8_t *scales = chunk + (is_v ? kv4_vscale_off(NG) : kv4_kscale_off(NG));
    uint32_t *vc = vcode[ch & 1];
    uint32_t w[PASSES];
    const __half d = q4_words(raw, w);            // the scale of row r0 + cc RPP
    if (ch + 1 < ch1) fetch(ch + 1);
    if (is_v) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) vc[(r0 + i * RPP) * VP + sub] = w[i];
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int p = r0 + i * RPP;
      if (!is_v && p >= lo && p < hi) *reinterpret_cast<uint32_t *>(chunk + kv4_kword(NG, p, cc, j)) = w[i];
    }
    if (const int p = r0 + cc * RPP; cc < PASSES && p >= lo && p < hi)
      *reinterpret_cast<__half *>(scales + (is_v ? kv4_vscale(NG, p, j) : kv4_kscale(NG, p, j))) = d;
    if (tid >= lo && tid < hi) {
      a.l.ids[bh * a.l.cap + p0 + tid] = rg.seen0 + (p0 + tid - rg.start);
      a.l.weights[bh * a.l.cap + p0 + tid] = 0.f;
    }
    __syncthreads();
    // (J, c, i): 8 dims 32 J + 8 i .. of 8 positions; another pair of warps for each chunk
    const int u = tid - 64 * (ch & 3);
    if (u >= 0 && u < 16 * NG) {
      const int i = u & 3, c = (u >> 2) & 3, J = u >> 4;
      uint32_t n[8], fresh = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int p = vpos(c, k);
        n[k] = vc[p * VP + J * 4 + i];
        if (p >= lo && p < hi) fresh |= 15u << (4 * k);
      }
      transpose_nibbles(n);
      uint8_t *unit = chunk + kv4_v_off(NG) + 4 * i;
      auto to = [&](int r) { return reinterpret_cast<uint32_t *>(unit + kv4_vunit(J, r, c)); };   // dim r of the eight
      if (fresh != 0xffffffffu && fresh != 0) {   // all loads first
        uint32_t old[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) old[r] = *to(r);
#pragma unroll
        for (int r = 0; r < 8; ++r) n[r] = (old[r] & ~fresh) | (n[r] & fresh);
      }
      if (fresh != 0) {
#pragma unroll
        for (int r = 0; r < 8; ++r) *to(r) = n[r];
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

// 16 bytes of the 8: all of them as bf16, or four (part 0 or 1) as fp32
template <typename T>
__device__ __forceinline__ void store16(void *p, int64_t at, int part, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2)
    store8<T>(p, at, x);
  else
    *reinterpret_cast<float4 *>(static_cast<float *>(p) + at + 4 * part) =
        part ? make_float4(x[4], x[5], x[6], x[7]) : make_float4(x[0], x[1], x[2], x[3]);
}

// d (u - 8) of a word's 8 codes
__device__ __forceinline__ void q4_values(uint32_t w, float d, float (&x)[8]) {
  uint32_t b[4];
  code_pairs(w, 0x64006400u, b);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&b[n]));
    x[n] = d * v.x;
    x[n + 4] = d * v.y;
  }
}

__device__ __forceinline__ float half_at(const uint8_t *p) {
  return __half2float(*reinterpret_cast<const __half *>(p));
}

// Few tokens: a thread per 8 dims of a row, straight from the cache.  Bound by
// latency (one token of 64 slots x 8 heads 2.3 us).
template <int NG, typename T>
__global__ void __launch_bounds__(256) k_kv4_read_step(const __grid_constant__ Kv4ReadArgs a) {
  constexpr int TPR = 4 * NG, CH = kv4_chunk_bytes(NG);
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.n_slot * a.T * a.n_kv * 2 * TPR) return;
  const int sub = (int)(i % TPR), j = sub >> 2, cc = sub & 3;
  const bool is_v = (i / TPR) & 1;
  int64_t k = i / (2 * TPR);
  const int h = (int)(k % a.n_kv);
  k /= a.n_kv;
  const int t = (int)(k % a.T), b = (int)(k / a.T);
  const int first = a.first ? a.first[b] : 0;
  const int64_t pos = first < 0 ? -1 : (int64_t)first + t;
  float x[8] = {};
  if (pos >= 0 && pos < kv4_len(a.l, b)) {
    const int p = (int)(pos % kKv4Chunk);
    const uint8_t *chunk = a.l.codes + (((int64_t)b * a.n_kv + h) * (a.l.cap / kKv4Chunk) + pos / kKv4Chunk) * CH;
    if (!is_v) {
      q4_values(*reinterpret_cast<const uint32_t *>(chunk + kv4_kword(NG, p, cc, j)),
                half_at(chunk + kv4_kscale_off(NG) + kv4_kscale(NG, p, j)), x);
    } else {
      const float d = half_at(chunk + kv4_vscale_off(NG) + kv4_vscale(NG, p, j));
      const int sh = kv4_vshift(p);
      uint32_t w = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        w |= ((*reinterpret_cast<const uint32_t *>(chunk + kv4_v_off(NG) + kv4_vunit(j, r, (p >> 1) & 3) + 4 * cc) >>
               sh) & 15u) << (4 * r);
      q4_values(w, d, x);
    }
  }
  const Kv4Rows &o = is_v ? a.v : a.k;
  store8<T>(o.p, b * o.slot + t * o.token + h * o.head + sub * 8, x);
}

// Many tokens: CTAs of up to kReadChunks chunks of one (slot, KV head), which one
// bulk copy brings into shared memory; then 8 dims of a K position per thread,
// and 8 x 8 nibbles of V (8 positions, 8 dims) per thread.  Bound by the
// values' bytes (8191 tokens of 32 heads at head_dim 128: bf16 28.0 us, fp32 49.3
// us, 6.2 TB/s).
constexpr int kReadThreads = 256, kReadChunks = 4, kReadStepTokens = 16;

template <int NG, typename T>
__global__ void __launch_bounds__(kReadThreads) k_kv4_read(const __grid_constant__ Kv4ReadArgs a) {
  constexpr int CH = kv4_chunk_bytes(NG), TPR = 4 * NG;
  __shared__ __align__(128) uint8_t sm[kReadChunks * CH];
  __shared__ __align__(8) uint64_t bar;
  const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y;
  if (tid == 0) {
    mbar_init(&bar, 1);
    fence_barrier_init();
  }
  pdl_wait();
  const int len = kv4_len(a.l, b);
  int first = a.first ? a.first[b] : 0;
  first = first < 0 || first > a.l.cap ? a.l.cap : first;   // outside the cache: nothing but zeros
  const int ch0 = first / kKv4Chunk + (int)blockIdx.x * a.group;
  const int64_t p0 = (int64_t)ch0 * kKv4Chunk, lo = max((int64_t)first, p0);
  const int64_t hi = min((int64_t)first + a.T, p0 + a.group * kKv4Chunk);
  if (lo >= hi) return;
  // chunks that hold entries to be read
  const int held = (int)max((int64_t)0, (min(hi, (int64_t)len) - p0 + kKv4Chunk - 1) / kKv4Chunk);
  __syncthreads();
  bool ok = true;
  if (held > 0) {
    if (tid == 0) {
      mbar_arrive_expect_tx(&bar, held * CH);
      bulk_g2s(sm, a.l.codes + (((int64_t)b * a.n_kv + h) * (a.l.cap / kKv4Chunk) + ch0) * CH, held * CH, &bar);
    }
    ok = mbar_wait(&bar, 0);
    if (!ok && tid == 0) {
      set_error(a.err, kErrTimeout);
      mbar_wait(&bar, 0);          // another bounded chance to land before the shared memory goes away
    }
  }
  // a row's threads: one per 16 bytes, 8 dims of bf16 or 4 of fp32, so that
  // every store of a warp is contiguous
  constexpr int HALF = sizeof(T) == 4 ? 2 : 1, LPR = TPR * HALF;
  const int64_t slot_k = b * a.k.slot + h * a.k.head, slot_v = b * a.v.slot + h * a.v.head;
  for (int i = tid; i < a.group * kKv4Chunk * LPR; i += kReadThreads) {
    const int q = i / LPR, sub = (i % LPR) / HALF, part = i % HALF, j = sub >> 2, cc = sub & 3, p = q % kKv4Chunk;
    const int64_t pos = p0 + q;
    if (pos < lo || pos >= hi) continue;
    const uint8_t *chunk = sm + (q / kKv4Chunk) * CH;
    float x[8] = {};
    if (pos < len)
      q4_values(*reinterpret_cast<const uint32_t *>(chunk + kv4_kword(NG, p, cc, j)),
                half_at(chunk + kv4_kscale_off(NG) + kv4_kscale(NG, p, j)), x);
    store16<T>(a.k.p, slot_k + (pos - first) * a.k.token + sub * 8, part, x);
  }
  for (int i = tid; i < a.group * 4 * LPR; i += kReadThreads) {
    const int sub = (i % LPR) / HALF, part = i % HALF, j = sub >> 2, cc = sub & 3, c = (i / LPR) & 3, q = i / (4 * LPR);
    const uint8_t *chunk = sm + q * CH;
    uint32_t w[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      w[r] = *reinterpret_cast<const uint32_t *>(chunk + kv4_v_off(NG) + kv4_vunit(j, r, c) + 4 * cc);
    transpose_nibbles(w);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int p = vpos(c, n);
      const int64_t pos = p0 + q * kKv4Chunk + p;
      if (pos < lo || pos >= hi) continue;
      float x[8] = {};
      if (pos < len) q4_values(w[n], half_at(chunk + kv4_vscale_off(NG) + kv4_vscale(NG, p, j)), x);
      store16<T>(a.v.p, slot_v + (pos - first) * a.v.token + sub * 8, part, x);
    }
  }
}

// ---------------------------------------------------------------- eviction
// Selection, one thread-block cluster per (slot, KV head), the entries' keys
// (order-preserving images of their weights) in registers.  Entries that must
// stay are set apart; a radix descent over the others' distances from their
// smallest key, ten bits at a time, finds the key of the rank that is left, and
// ends as soon as a bin is kept whole (mostly after two levels); of the entries with exactly that key the
// first ones stay.  Then the kept entries behind the budget ("movers") fill the
// dropped ones' places below it ("holes"), both in index order: src_of[p] is p
// or, for hole r, -1 - r, and movers[r] what goes there.  Bound by the latency
// of its barriers (8 heads each: 64 slots at 1000 entries 8 us, four at 32k in
// clusters of eight CTAs 17 us, of 1024 threads each 25 us).
template <int THREADS, int K>
__global__ void __launch_bounds__(THREADS, THREADS >= 1024 ? 1 : 3) k_kv4_select(const __grid_constant__ Kv4EvictArgs a) {
  constexpr int WARPS = THREADS / 32, COPIES = 4, BITS = 10, BINS = 1 << BITS;
  static_assert(THREADS >= BINS / 4, "four bins per thread");
  __shared__ __align__(16) uint32_t hist[COPIES][BINS];
  __shared__ __align__(16) uint32_t merged[2][BINS];
  __shared__ uint32_t warp_sum[WARPS], warp_min[WARPS], warp_max_[WARPS];
  __shared__ uint2 warp_pair[WARPS], totals[2];
  __shared__ uint32_t range[3];                    // the CTA's smallest and largest loose key, entries that stay
  __shared__ uint32_t s_bin, s_need, s_equal;
  cg::cluster_group cluster = cg::this_cluster();
  const int CL = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y, b = blockIdx.z;
  auto sync_all = [&]() {
    if (CL > 1) cluster.sync();
    else __syncthreads();
  };
  pdl_trigger();                  // the moves' CTAs may settle beside these, and wait
  pdl_wait();
  const int n = kv4_len(a.src, b), seen = a.src.seen[b], m = a.budget;
  const int64_t bh = (int64_t)b * a.n_kv + h;
  const int32_t *ids = a.src.ids + bh * a.src.cap;
  const float *wt = a.src.weights + bh * a.src.cap;
  int32_t *src_of = a.src_of + bh * a.src.cap, *movers = a.movers + bh * a.src.cap;
  auto arrive = [&]() {           // the last of the slot's CTAs to have read the length moves it
    __syncthreads();
    if (tid != 0) return;
    if (h == 0 && rank == 0) a.n_old[b] = n;
    __threadfence();
    const unsigned ctas = gridDim.x * gridDim.y;
    if (atomicInc(a.arrive + b, ctas - 1) == ctas - 1) {
      a.dst.len[b] = min(n, m);
      a.dst.seen[b] = seen;
    }
  };
  // (uniform over the cluster)
  if (n > m) {
    // The chunk that holds the budget's border gives entries and takes some, in
    // one V word even: in place, its V codes are read from a copy.
    if (a.in_place && rank == 0 && tid < 32 * a.ng) {
      const uint8_t *from = a.src.codes + (bh * (a.src.cap / kKv4Chunk) + m / kKv4Chunk) * kv4_chunk_bytes(a.ng) + kv4_v_off(a.ng);
      reinterpret_cast<uint4 *>(a.border + bh * (512 * a.ng))[tid] = reinterpret_cast<const uint4 *>(from)[tid];
    }
    const int base = rank * THREADS * K + warp * 32 * K + lane;   // this lane's entries: base + 32 k
    uint32_t key[K], loose = 0, lo = 0xffffffffu, hi = 0, stay = 0;
    constexpr int LOADS = K < 16 ? K : 16;        // in flight at once
#pragma unroll
    for (int k0 = 0; k0 < K; k0 += LOADS) {
      int id[LOADS];
      float w[LOADS];
#pragma unroll
      for (int k = 0; k < LOADS; ++k) {
        const int i = min(base + 32 * (k0 + k), n - 1);
        id[k] = ids[i];
        w[k] = wt[i];
      }
      if (k0 == 0) arrive();
#pragma unroll
      for (int k = 0; k < LOADS; ++k) {
        const uint32_t u = w[k] == 0.f ? 0u : __float_as_uint(w[k]);   // -0 and 0 are equal
        key[k0 + k] = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
        if (base + 32 * (k0 + k) >= n) continue;
        if (id[k] < a.n_sink || (int64_t)id[k] >= (int64_t)seen - a.n_recent) {
          ++stay;
        } else {
          loose |= 1u << (k0 + k);
          lo = min(lo, key[k0 + k]);
          hi = max(hi, key[k0 + k]);
        }
      }
    }
    for (int i = tid; i < COPIES * BINS; i += THREADS) (&hist[0][0])[i] = 0;
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    stay = __reduce_add_sync(0xffffffffu, stay);
    if (lane == 0) {
      warp_min[warp] = lo;
      warp_max_[warp] = hi;
      warp_sum[warp] = stay;
    }
    __syncthreads();
    if (warp == 0) {
      lo = __reduce_min_sync(0xffffffffu, lane < WARPS ? warp_min[lane] : 0xffffffffu);
      hi = __reduce_max_sync(0xffffffffu, lane < WARPS ? warp_max_[lane] : 0u);
      stay = __reduce_add_sync(0xffffffffu, lane < WARPS ? warp_sum[lane] : 0u);
      if (lane == 0) {
        range[0] = lo;
        range[1] = hi;
        range[2] = stay;
      }
    }
    sync_all();
    {   // over the cluster: a CTA per lane
      const uint32_t *r = CL > 1 ? cluster.map_shared_rank(range, min(lane, CL - 1)) : range;
      lo = __reduce_min_sync(0xffffffffu, r[0]);
      hi = __reduce_max_sync(0xffffffffu, r[1]);
      stay = __reduce_add_sync(0xffffffffu, lane < CL ? r[2] : 0u);
    }
    // distances from the smallest loose key; the need-th largest is sought.
    // prefix: its bits from `shift` up
#pragma unroll
    for (int k = 0; k < K; ++k) key[k] -= lo;
    int shift = hi > lo ? 32 - __clz(hi - lo) : 1;
    uint32_t prefix = 0, equal = 0xffffffffu;
    uint32_t need = (uint32_t)m > stay ? (uint32_t)m - stay : 0u;
#pragma unroll 1
    for (int level = 0; need > 0 && shift > 0 && need != equal; ++level) {
      const int width = min(BITS, shift);
      shift -= width;
      const uint32_t digit = (1u << width) - 1u;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint32_t d = key[k] >> shift;
        if (((loose >> k) & 1u) && (level == 0 || (d >> width) == prefix)) atomicAdd(&hist[warp % COPIES][d & digit], 1u);
      }
      __syncthreads();
      // thread t: the four bins 1023 - 4 t - 3 .. 1023 - 4 t, over the copies and the cluster
      const int first = BINS - 4 - 4 * tid;
      uint4 v = make_uint4(0, 0, 0, 0);
      auto add = [&](uint4 x) { v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w; };
      uint32_t *mine = merged[level & 1];
      if (tid < BINS / 4) {
#pragma unroll
        for (int q = 0; q < COPIES; ++q) {
          uint4 *h4 = reinterpret_cast<uint4 *>(&hist[q][first]);
          add(*h4);
          *h4 = make_uint4(0, 0, 0, 0);
        }
        if (CL > 1) *reinterpret_cast<uint4 *>(mine + first) = v;
      }
      if (CL > 1) {
        cluster.sync();
        if (tid < BINS / 4) {
          uint4 x[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            x[c] = c < CL ? *reinterpret_cast<const uint4 *>(cluster.map_shared_rank(mine + first, c)) : make_uint4(0, 0, 0, 0);
          v = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < 8; ++c) add(x[c]);
        }
      }
      // the bin in which the running count from the top reaches `need`
      const uint32_t sum = v.x + v.y + v.z + v.w;
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      if (lane == 31) warp_sum[warp] = inc;
      __syncthreads();
      const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u);
      uint32_t above = before + inc - sum;
      if (above < need && need <= above + sum) {
        const uint32_t four[4] = {v.w, v.z, v.y, v.x};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (above < need && need <= above + four[q]) {
            s_bin = first + 3 - q;
            s_need = need - above;
            s_equal = four[q];
          }
          above += four[q];
        }
      }
      __syncthreads();
      prefix = (prefix << width) | s_bin;
      need = s_need;
      equal = s_equal;
    }
    // the first `need` of the `equal` entries with key == prefix stay (shift is 0 unless all do)
    // exclusive bases of this warp's two counts over the cluster, in index order
    auto ranks = [&](uint32_t first, uint32_t second, int slot) -> uint2 {
      if (lane == 0) warp_pair[warp] = make_uint2(first, second);
      __syncthreads();
      const uint2 w = lane < WARPS ? warp_pair[lane] : make_uint2(0, 0);
      uint2 before = make_uint2(__reduce_add_sync(0xffffffffu, lane < warp ? w.x : 0u),
                                __reduce_add_sync(0xffffffffu, lane < warp ? w.y : 0u));
      if (CL > 1) {
        const uint2 all = make_uint2(__reduce_add_sync(0xffffffffu, w.x), __reduce_add_sync(0xffffffffu, w.y));
        if (tid == 0) totals[slot] = all;
        cluster.sync();
        const uint2 t = lane < rank ? *cluster.map_shared_rank(&totals[slot], lane) : make_uint2(0, 0);
        before.x += __reduce_add_sync(0xffffffffu, t.x);
        before.y += __reduce_add_sync(0xffffffffu, t.y);
      }
      __syncthreads();
      return before;
    };
    uint32_t kept = 0;                             // bit k: entry base + 32 k stays
    if (need == 0 || need == equal) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (base + 32 * k < n && (!((loose >> k) & 1u) || (need > 0 && (key[k] >> shift) >= prefix))) kept |= 1u << k;
    } else {
      uint32_t mine = 0;
#pragma unroll
      for (int k = 0; k < K; ++k)
        mine += __popc(__ballot_sync(0xffffffffu, ((loose >> k) & 1u) && key[k] == prefix));
      uint32_t at = ranks(mine, 0, 0).x;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const bool is_loose = (loose >> k) & 1u, eq = is_loose && key[k] == prefix;
        const uint32_t vote = __ballot_sync(0xffffffffu, eq);
        const bool first = eq && at + __popc(vote & ((1u << lane) - 1u)) < need;
        at += __popc(vote);
        if (base + 32 * k < n && (!is_loose || key[k] > prefix || first)) kept |= 1u << k;
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
    const uint2 at = ranks(holes, moves, 1);
    uint32_t hole_at = at.x, move_at = at.y;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = base + 32 * k;
      const bool go = i >= m && ((kept >> k) & 1u);
      const uint32_t vote = __ballot_sync(0xffffffffu, go);
      if (go) movers[move_at + __popc(vote & ((1u << lane) - 1u))] = i;
      move_at += __popc(vote);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = base + 32 * k;
      const bool hole = i < m && !((kept >> k) & 1u);
      const uint32_t vote = __ballot_sync(0xffffffffu, hole);
      if (i < m) src_of[i] = hole ? -1 - (int)(hole_at + __popc(vote & ((1u << lane) - 1u))) : i;
      hole_at += __popc(vote);
    }
    if (CL > 1) cluster.sync();   // no CTA leaves while a peer may read its shared memory
  } else {
    arrive();
  }
}

constexpr int kMoveThreads = 128, kMoveChunks = 2;

// The moves, one CTA per (kMoveChunks destination chunks, KV head, slot).
// Sources of moves lie at or behind the budget and destinations below it, so
// the CTAs do not depend on one another; V words of the chunk that holds both
// are read from the selection's copy.  Bound by the gathered V
// words, which hold 8 positions each (8 heads, head_dim 128: four slots of 32k to
// 8192 29 us, 130 MB; copies of 64 slots at 1000 entries 25.5 us, 157 MB, 6.2 TB/s).
template <int NG>
__global__ void __launch_bounds__(kMoveThreads, 8) k_kv4_move(const __grid_constant__ Kv4EvictArgs a) {
  constexpr int CH = kv4_chunk_bytes(NG), POS = kMoveChunks * kKv4Chunk;
  static_assert(POS <= kMoveThreads, "a position per thread");
  __shared__ int src[POS];
  __shared__ const uint8_t *vfrom[POS];     // the V codes of a source's chunk
  __shared__ int moved_chunk[kMoveChunks];
  const int tid = threadIdx.x, h = blockIdx.y, b = blockIdx.z, p0 = blockIdx.x * POS;
  pdl_wait();
  const int n = a.n_old[b], out = min(n, a.budget);
  if (p0 >= out || (a.in_place && n <= a.budget)) return;
  const int64_t bh = (int64_t)b * a.n_kv + h;
  const uint8_t *from = a.src.codes + bh * (a.src.cap / kKv4Chunk) * CH;
  uint8_t *to = a.dst.codes + (bh * (a.dst.cap / kKv4Chunk) + blockIdx.x * kMoveChunks) * CH;
  // V units (J, r, c), 4 dims of 8 positions: those of the same place,
  // at once unless most chunks will not be touched
  constexpr int UNITS = 32 * NG, PER = (kMoveChunks * UNITS + kMoveThreads - 1) / kMoveThreads;
  constexpr int VECS = (POS * NG + kMoveThreads - 1) / kMoveThreads;
  uint4 w[PER];
  auto same_place = [&](int k, int u) {   // unit u in their order in memory
    return *reinterpret_cast<const uint4 *>(from + (int64_t)(p0 / kKv4Chunk + k) * CH + kv4_v_off(NG) + u * 16);
  };
  if (!a.in_place) {
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const int i = x * kMoveThreads + tid, k = i / UNITS;
      if (k < kMoveChunks && p0 + k * kKv4Chunk < out) w[x] = same_place(k, i % UNITS);
    }
  }
  int my_src = -1;
  if (tid < POS) {
    const int p = p0 + tid;
    int s = -1;
    if (p < out) {
      s = n > a.budget ? a.src_of[bh * a.src.cap + p] : p;
      if (s < 0) s = a.movers[bh * a.src.cap - 1 - s];
    }
    my_src = s;
    src[tid] = s;
    vfrom[tid] = a.in_place && s >= a.budget && s / kKv4Chunk == a.budget / kKv4Chunk
                     ? a.border + bh * (512 * NG)
                     : from + (int64_t)(s / kKv4Chunk) * CH + kv4_v_off(NG);
    const bool any = __any_sync(0xffffffffu, s >= 0 && s != p);
    if ((tid & 31) == 0) moved_chunk[tid >> 5] = any;
  }
  __syncthreads();
  // K rows, NG 16-byte vectors each, and a position per thread its scales, id and
  // weight; all loads before the stores
  {
    const bool mine = my_src >= 0 && !(a.in_place && my_src == p0 + tid);
    int32_t id = 0;
    float weight = 0.f;
    uint16_t ks[NG] = {}, vs[NG] = {};
    if (mine) {
      id = a.src.ids[bh * a.src.cap + my_src];
      weight = a.src.weights[bh * a.src.cap + my_src];
      const uint8_t *f = from + (int64_t)(my_src / kKv4Chunk) * CH;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        ks[j] = *reinterpret_cast<const uint16_t *>(f + kv4_kscale_off(NG) + kv4_kscale(NG, my_src % kKv4Chunk, j));
        vs[j] = *reinterpret_cast<const uint16_t *>(f + kv4_vscale_off(NG) + kv4_vscale(NG, my_src % kKv4Chunk, j));
      }
    }
    uint4 v[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int p = (i * kMoveThreads + tid) / NG, s = p < POS ? src[p] : -1;
      if (s >= 0 && !(a.in_place && s == p0 + p))
        v[i] = reinterpret_cast<const uint4 *>(from + (int64_t)(s / kKv4Chunk) * CH + (s % kKv4Chunk) * 16 * NG)[tid % NG];
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int p = (i * kMoveThreads + tid) / NG, s = p < POS ? src[p] : -1;
      if (s >= 0 && !(a.in_place && s == p0 + p))
        reinterpret_cast<uint4 *>(to + (p / kKv4Chunk) * CH + (p % kKv4Chunk) * 16 * NG)[tid % NG] = v[i];
    }
    if (mine) {
      a.dst.ids[bh * a.dst.cap + p0 + tid] = id;
      a.dst.weights[bh * a.dst.cap + p0 + tid] = weight;
      uint8_t *t = to + (tid / kKv4Chunk) * CH;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        *reinterpret_cast<uint16_t *>(t + kv4_kscale_off(NG) + kv4_kscale(NG, tid % kKv4Chunk, j)) = ks[j];
        *reinterpret_cast<uint16_t *>(t + kv4_vscale_off(NG) + kv4_vscale(NG, tid % kKv4Chunk, j)) = vs[j];
      }
    }
  }
  auto live = [&](int k) { return k < kMoveChunks && p0 + k * kKv4Chunk < out && (!a.in_place || moved_chunk[k]); };
  if (a.in_place) {
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const int i = x * kMoveThreads + tid, k = i / UNITS;
      if (live(k)) w[x] = same_place(k, i % UNITS);
    }
  }
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    const int i = x * kMoveThreads + tid, k = i / UNITS, u = i % UNITS, J = u >> 5, c = (u >> 3) & 3, r = (u - 2 * c) & 7;
    if (!live(k)) continue;
    if (moved_chunk[k]) {
      uint4 v[8];
      int s[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int p = vpos(c, e);
        s[e] = src[k * kKv4Chunk + p];
        if (s[e] == p0 + k * kKv4Chunk + p) s[e] = -1;
        if (s[e] >= 0)
          v[e] = *reinterpret_cast<const uint4 *>(vfrom[k * kKv4Chunk + p] + kv4_vunit(J, r, (s[e] >> 1) & 3));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (s[e] < 0) continue;
        const int from_sh = kv4_vshift(s[e] % kKv4Chunk), sh = 4 * e;
        w[x].x = (w[x].x & ~(15u << sh)) | (((v[e].x >> from_sh) & 15u) << sh);
        w[x].y = (w[x].y & ~(15u << sh)) | (((v[e].y >> from_sh) & 15u) << sh);
        w[x].z = (w[x].z & ~(15u << sh)) | (((v[e].z >> from_sh) & 15u) << sh);
        w[x].w = (w[x].w & ~(15u << sh)) | (((v[e].w >> from_sh) & 15u) << sh);
      }
    }
    *reinterpret_cast<uint4 *>(to + k * CH + kv4_v_off(NG) + u * 16) = w[x];
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

// chunks that T rows from any position touch at most, in groups
int chunk_groups(int T, int group) { return ((T + kKv4Chunk - 2) / kKv4Chunk + group) / group; }

// Chunks per CTA: up to `most` (append 8: one prompt of 8191 in fp32 48.9 us against
// 50.4 with four and 57.0 with two; 8 x 4096 at head_dim 32 in fp32 15.0, 16.9,
// 20.5), fewer while all CTAs fit the GPU at once (four on each SM).  bf16 append /
// fp32 read, us, always four chunks against this rule and against always one: 1 sequence x 8 heads x 256 tokens 6.1 / 5.9,
// 3.1 / 3.0, 3.0 / 3.1; 4 x 8 x 1031 7.8 / 8.4, 6.6 / 8.1, 7.2 / 8.4; 1 x 32 x
// 8191 35.4 / 49.5, 35.3 / 49.6, 43.6 / 53.8.
constexpr int kChunkCtasPerSm = 4;

int chunk_group(int T, int n_kv, int n_slot, int sms, int most) {
  const int64_t chunks = (int64_t)chunk_groups(T, 1) * n_kv * n_slot, at_once = (int64_t)kChunkCtasPerSm * sms;
  const int64_t per = (chunks + at_once - 1) / at_once;
  return (int)(per < 1 ? 1 : per > most ? most : per);
}

template <int NG, typename T>
cudaError_t run_append(Kv4AppendArgs a, cudaStream_t st) {
  // One CTA per slot against one per chunk and head, us, step form first, at
  // head_dim 128 bf16, then 64 fp32, then 32 fp32 (the types differ by less than
  // a tenth):
  //   64 slots x 8 heads, 1 token    2.6, 3.8    2.6, 3.6    2.5, 3.6
  //   64 x 8, 8 tokens               7.3, 4.0    4.8, 3.4    3.3, 3.8
  //   1 x 32, 1 token                3.9, 2.8    2.9, 2.9    2.6, 2.9
  //   256 x 8, 4 tokens              5.8, 11.8   3.9, 9.9    3.2, 10.1
  //   1024 x 1, 8 tokens             7.9, 6.6    7.4, 5.7    7.9, 5.9
  // (the last, many tokens of few heads, is where the rule picks the slower form)
  const int64_t values = (int64_t)a.T * a.n_kv * 32 * NG;
  if (values <= 2048 || (values <= 8192 && (int64_t)a.n_slot * a.n_kv > 1024))
    return kv4_launch(k_kv4_append_step<NG, T>, dim3(a.n_slot), dim3(kStepThreads), (size_t)values / 2, 1, st, a);
  a.group = chunk_group(a.T, a.n_kv, a.n_slot, a.sms, kAppendChunks);
  const dim3 grid(chunk_groups(a.T, a.group), a.n_kv, a.n_slot);
  return kv4_launch(k_kv4_append<NG, T>, grid, dim3(kAppendThreads), 0, 1, st, a);
}

template <int NG, typename T>
cudaError_t run_read(Kv4ReadArgs a, cudaStream_t st) {
  // few rows per chunk: straight from the cache, or through whole chunks (64
  // slots x 8 heads at head_dim 128, fp32, us: 1 token 2.3, 4.8; 16 tokens 4.6, 6.0;
  // 32 tokens 7.0 both)
  if (a.T <= kReadStepTokens) {
    const int64_t threads = (int64_t)a.n_slot * a.T * a.n_kv * 8 * NG;
    return kv4_launch(k_kv4_read_step<NG, T>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, 1, st, a);
  }
  a.group = chunk_group(a.T, a.n_kv, a.n_slot, a.sms, kReadChunks);
  const dim3 grid(chunk_groups(a.T, a.group), a.n_kv, a.n_slot);
  return kv4_launch(k_kv4_read<NG, T>, grid, dim3(kReadThreads), 0, 1, st, a);
}

template <int NG>
cudaError_t run_append(const Kv4AppendArgs &a, cudaStream_t st) {
  return a.k.dtype == PNB_F32 ? run_append<NG, float>(a, st) : run_append<NG, __nv_bfloat16>(a, st);
}

template <int NG>
cudaError_t run_read(const Kv4ReadArgs &a, cudaStream_t st) {
  return a.k.dtype == PNB_F32 ? run_read<NG, float>(a, st) : run_read<NG, __nv_bfloat16>(a, st);
}

template <int NG>
cudaError_t run_move(const Kv4EvictArgs &a, cudaStream_t st) {
  const int most = a.budget < a.src.cap ? a.budget : a.src.cap, pos = kMoveChunks * kKv4Chunk;
  const dim3 grid((most + pos - 1) / pos, a.n_kv, a.n_slot);
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
  // entries per CTA and CTAs per cluster that hold the whole capacity in
  // registers; up to 4096 entries in one CTA, then in growing clusters of such
  // CTAs (which keep many SMs busy when there are few rows), then larger CTAs
  const int cap = a.src.cap;
  const int per = cap <= 1024 ? 1024 : cap <= 2048 ? 2048 : cap <= 8 * 4096 ? 4096 : cap <= 8 * 16384 ? 16384 : 32768;
  int cl = 1;
  while (cl * per < cap) cl *= 2;
  const dim3 grid(cl, a.n_kv, a.n_slot);
  cudaError_t e;
  if (per == 1024) e = kv4_launch(k_kv4_select<256, 4>, grid, dim3(256), 0, cl, st, a);
  else if (per == 2048) e = kv4_launch(k_kv4_select<256, 8>, grid, dim3(256), 0, cl, st, a);
  else if (per == 4096) e = kv4_launch(k_kv4_select<256, 16>, grid, dim3(256), 0, cl, st, a);
  else if (per == 16384) e = kv4_launch(k_kv4_select<1024, 16>, grid, dim3(1024), 0, cl, st, a);
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
