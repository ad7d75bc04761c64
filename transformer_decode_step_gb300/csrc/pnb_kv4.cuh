// pnb_kv4.cuh - the 4-bit KV cache: layout, kernel arguments and launchers.
//
// Every K and V row is held in Q4_0 blocks of 32 consecutive head dimensions:
// one fp16 scale d and 32 codes u, value = d * (u - 8).  A (layer, slot, KV
// head) is a list of chunks of 32 positions, each one contiguous run of
// 1152 * NG bytes (NG = head_dim / 32; 4608 at head_dim 128), so that a single
// bulk copy brings the K and V of 32 positions into shared memory:
//
//   [K codes 512 NG][K scales 64 NG][V codes 512 NG][V scales 64 NG]
//
// The codes lie as the attention kernel's matrix instructions (m16n8k16, fp16)
// want their A operand, so that one 32-bit word of 8 codes becomes four
// registers of two fp16 each with four masks, one shift and four packed fp16
// operations:
//   - a word's nibbles n and n + 4 are a pair, in the two halves of the word;
//   - K: a lane (r = lane / 4, c = lane % 4) holds position 8 t + r and, per
//     32-dim block j, the word of dims 32 j + 8 c + n;
//   - V: the lane holds dim 32 J + 8 i + r and the word whose nibble t + 4 e
//     is position 8 t + 2 c + e.
// A position's K scales are its blocks' fp16 in a row: what a lane multiplies
// its position's partial scores with.  The V scales of positions 8 t + 2 c and
// 8 t + 2 c + 1 are a half2 per block, next to one another over the blocks: what
// a lane (r, c) multiplies its softmax weights of that position pair with.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pnb.h"
#include "pnb_device.cuh"

namespace pnb {

constexpr int kKv4Chunk = 32;              // positions per chunk
constexpr int kKv4Rows = 8;                // most query rows (tokens x heads of a group) per work item
constexpr int kKv4Warps = 16;              // warps per attention CTA
constexpr int kKv4Threads = kKv4Warps * 32;
constexpr int kKv4CtasPerSm = 1;
constexpr int kKv4MaxRows = 64;            // tokens x heads of a group in one call
constexpr int kKv4MaxSlots = 1024;
constexpr int kKv4MaxCap = 1 << 20;        // positions per slot
constexpr int kKv4MaxEvictCap = 1 << 18;   // largest cache the eviction selects from
constexpr int kErrFull = 4;                // mirror of PNB_DEV_ERR_FULL
constexpr int kErrRange = 8;               // mirror of PNB_DEV_ERR_RANGE

__host__ __device__ constexpr int kv4_chunk_bytes(int ng) { return 1152 * ng; }
__host__ __device__ constexpr int kv4_kscale_off(int ng) { return 512 * ng; }
__host__ __device__ constexpr int kv4_v_off(int ng) { return 576 * ng; }
__host__ __device__ constexpr int kv4_vscale_off(int ng) { return 1088 * ng; }
// K word of position p (0..31 in the chunk), block j, dims 8 c .. 8 c + 7 of it
__host__ __device__ constexpr int kv4_kword(int ng, int p, int c, int j) {
  return p * 16 * ng + c * 4 * ng + j * 4;
}
// scale of position p, block j, relative to the K and to the V scale area
__host__ __device__ constexpr int kv4_kscale(int ng, int p, int j) { return p * 2 * ng + j * 2; }
__host__ __device__ constexpr int kv4_vscale(int ng, int p, int j) {
  return (p >> 1) * 4 * ng + j * 4 + (p & 1) * 2;
}
// V words of dims 32 J + 8 i + r (i = 0..3, 16 bytes) for position class c: a
// position's 32 dims lie in 128 contiguous bytes, the units rotated so that the
// attention's lanes (r, c) read them without bank conflicts
__host__ __device__ constexpr int kv4_vunit(int J, int r, int c) {
  return J * 512 + c * 128 + ((r + 2 * c) & 7) * 16;
}
// bit position of position p's nibble in its V word; its class is (p / 2) % 4
__host__ __device__ constexpr int kv4_vshift(int p) { return 4 * ((p >> 3) + 4 * (p & 1)); }

// rows of a caller's tensor [slot][token][head][head_dim], strides in elements
struct Kv4Rows {
  void *p;
  int64_t slot, token, head;
  int32_t dtype;
};

// one layer of a cache
struct Kv4Layer {
  uint8_t *codes;       // [n_slot][n_kv][cap / 32] chunks
  int32_t *ids;         // [n_slot][n_kv][cap] original position of each entry
  float *weights;       // [n_slot][n_kv][cap] accumulated attention weights
  int32_t *len, *seen;  // [n_slot] entries held, tokens ever appended
  int32_t cap;
};

struct Kv4AppendArgs {
  Kv4Layer l;
  Kv4Rows k, v;
  const int32_t *n_new, *start;   // [n_slot] or NULL
  int32_t n_slot, n_kv, T, sms;   // (sms: the device's SM count)
  int32_t group;                  // chunks per CTA (set by the launcher)
  uint32_t *arrive;               // [n_slot]
  int32_t *err;
};

struct Kv4ReadArgs {
  Kv4Layer l;
  Kv4Rows k, v;
  const int32_t *first;           // [n_slot] or NULL
  int32_t n_slot, n_kv, T, sms;   // (sms: the device's SM count)
  int32_t group;                  // chunks per CTA (set by the launcher)
  int32_t *err;
};

struct Kv4AttnArgs {
  Kv4Layer l;
  Kv4Rows q, out;
  int32_t n_slot, n_kv, G, T, rows;  // rows = T * G
  int32_t nrb;                    // items per KV head (set by the launcher)
  float qscale;                   // log2(e) / sqrt(head_dim)
  float *warp_part;               // [grid][kKv4Warps][kKv4Rows][head_dim]: rows a warp puts aside
  float *part;                    // [2 grid][kKv4Rows][head_dim]: a CTA's partial rows
  float *part_ml;                 // [2 grid][kKv4Rows][2]: their reference and sum
  unsigned *counter;              // [grid]
  int32_t *err;
  float *scores;                  // [n_slot][n_kv][rows][cap], log2 units (NULL: not tracked)
  float2 *wscale;                 // [n_slot][n_kv][rows] reference, reciprocal of the sum
};

struct Kv4WeightArgs {
  Kv4Layer l;
  const float *scores;
  const float2 *wscale;
  int32_t n_slot, n_kv, rows, sms;
  float decay;
};

struct Kv4EvictArgs {
  Kv4Layer src, dst;
  int32_t n_slot, n_kv, budget, n_sink, n_recent;
  int32_t in_place, ng;
  int32_t *src_of, *movers;       // [n_slot][n_kv][src.cap]
  int32_t *n_old;                 // [n_slot]
  uint8_t *border;                // [n_slot][n_kv][512 ng] V codes of the chunk that holds the budget's border
  uint32_t *arrive;               // [n_slot]
};

cudaError_t prepare_kv4_kernels(int ng, int *sms);
cudaError_t launch_kv4_append(int ng, const Kv4AppendArgs &a, cudaStream_t st);
cudaError_t launch_kv4_read(int ng, const Kv4ReadArgs &a, cudaStream_t st);
cudaError_t launch_kv4_attn(int ng, const Kv4AttnArgs &a, int grid, cudaStream_t st);
cudaError_t launch_kv4_weights(const Kv4WeightArgs &a, cudaStream_t st);
cudaError_t launch_kv4_evict(int ng, const Kv4EvictArgs &a, cudaStream_t st);
cudaError_t launch_kv4_reset(int32_t *len, int32_t *seen, int64_t layer_stride, int n_layer, int n_slot,
                             int slot, cudaStream_t st);

// launch with programmatic dependent launch: every kernel of the cache waits
// (griddepcontrol.wait) before its first access to global memory
template <typename K, typename A>
inline cudaError_t kv4_launch(K kern, dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st,
                              const A &a) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int na = 0;
  attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[na].val.programmaticStreamSerializationAllowed = 1;
  ++na;
  if (cluster > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = cluster;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// The code pairs of a word as fp16 pairs u - 8, exactly: nibbles 0 and 4
// (b[0]), 1 and 5 (b[1]), 2 and 6 (b[2]), 3 and 7 (b[3]).  As published for 4-bit
// weights: a masked nibble under the exponent of 1024 is the number 1024 + u (or
// 1024 + 16 u), and one packed operation takes the rest away.  (Left as subnormals u * 2^-24, which
// saves that operation, the codes lose up to 10 bits in the matrix
// instruction's alignment: outputs were 8e-5 off instead of 1e-6.)  `magic` is
// 0x64006400 in a register: as a second immediate it would cost a second
// logic instruction per mask.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(magic));
  return d;
}

__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t magic, uint32_t (&b)[4]) {
  const __half2 off = __half2half2(__ushort_as_half(0x6408)), sixteenth = __half2half2(__ushort_as_half(0x2c00)),
                m72 = __half2half2(__ushort_as_half(0xd480));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = and_or(w, 0x000f000fu, magic), hi = and_or(w, 0x00f000f0u, magic);
    const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&lo), off);
    const __half2 h = __hfma2(*reinterpret_cast<const __half2 *>(&hi), sixteenth, m72);
    b[2 * i] = *reinterpret_cast<const uint32_t *>(&l);
    b[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&h);
    w >>= 8;
  }
}

// a + b on packed pairs of fp32
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
  return *reinterpret_cast<float2 *>(&d);
}

// Entries of slot b as the kernels use them: a length outside [0, cap] (the
// buffer is the caller's) never leads an access out of the cache.
__device__ __forceinline__ int kv4_len(const Kv4Layer &l, int b) {
  const int n = l.len[b];
  return n < 0 ? 0 : (n > l.cap ? l.cap : n);
}

// Prefix sums over the slots of mult * (ceil(len / unit) + extra), 0 for an
// empty slot, into pre[0 .. n_slot] (shared memory), and when lens is given the
// lengths and, behind them, the number of slots that are not empty and the
// largest length, by the calling warp; the caller synchronises.
__device__ __forceinline__ void kv4_prefix(const Kv4Layer &l, int n_slot, int unit, int extra, int mult, int *pre,
                                           int *lens) {
  const int lane = threadIdx.x & 31;
  int base = 0, live = 0, most = 0;
  for (int b0 = 0; b0 < n_slot; b0 += 32) {
    const int b = b0 + lane;
    const int n = b < n_slot ? kv4_len(l, b) : 0;
    if (lens && b < n_slot) lens[b] = n;
    live += __popc(__ballot_sync(0xffffffffu, n > 0));
    most = max(most, n);
    int v = n > 0 ? mult * ((n + unit - 1) / unit + extra) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (b < n_slot) pre[b + 1] = base + v;
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) pre[0] = 0;
  if (lens) {
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      lens[n_slot] = live;
      lens[n_slot + 1] = most;
    }
  }
}

// The slot whose range of the prefix sums holds x (0 <= x < pre[n_slot]; the same
// x in all lanes): the number of ranges that end at or before it.  (A binary
// search, six dependent loads for 64 slots, adds 1 us to attention over them.)
__device__ __forceinline__ int kv4_find(const int *pre, int n_slot, int x) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 2
  for (int b0 = 1; b0 < n_slot; b0 += 32)
    n += __popc(__ballot_sync(0xffffffffu, pre[min(b0 + lane, n_slot)] <= x));
  return n;
}

}  // namespace pnb
