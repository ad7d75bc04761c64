// pnb_rows.cuh - what the KV-cache entry points share: rows of a caller's tensor
// and their checks, the clearing of a workspace, launches.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "pnb.h"

namespace pnb {

// rows of a caller's tensor [slot][token][head][head_dim], strides in elements
struct DevRows {
  void *p;
  int64_t slot, token, head;
  int32_t dtype;
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Zeroes device memory before it returns: the first call that reads it may be on
// any stream, and a non-blocking one does not wait for a clear on the default
// stream (which may itself be behind other work there).
inline cudaError_t clear_now(void *p, size_t n) {
  cudaStream_t st;
  cudaError_t e = cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(p, 0, n, st);
  const cudaError_t done = cudaStreamSynchronize(st);
  cudaStreamDestroy(st);
  return e != cudaSuccess ? e : done;
}

// a caller's rows: type, 16-byte alignment of every row, no negative strides;
// rows that are written must not lie over one another
inline int check_rows(const pnb_rows *r, int T, int n_slot, int heads, int head_dim, bool written, DevRows *out) {
  if (!r->dev) return PNB_E_NULL;
  if (r->dtype != PNB_F32 && r->dtype != PNB_BF16) return PNB_E_INVAL;
  if (r->slot < 0 || r->token < 0 || r->head < 0) return PNB_E_INVAL;
  const int64_t per = r->dtype == PNB_F32 ? 4 : 8;   // elements in 16 bytes
  if (!aligned16(r->dev) || r->slot % per || r->token % per || r->head % per) return PNB_E_ALIGN;
  if (written) {
    // sorted by stride, each dimension must step past the extent of the ones
    // below it
    int64_t s[3] = {r->head, r->token, r->slot}, n[3] = {heads, T, n_slot};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (s[j] > s[j + 1]) {
          const int64_t a = s[j], b = n[j];
          s[j] = s[j + 1]; n[j] = n[j + 1];
          s[j + 1] = a; n[j + 1] = b;
        }
    int64_t extent = head_dim;
    for (int i = 0; i < 3; ++i) {
      if (n[i] <= 1) continue;
      if (s[i] < extent) return PNB_E_INVAL;
      extent += s[i] * (n[i] - 1);
    }
  }
  out->p = const_cast<void *>(r->dev);
  out->slot = r->slot;
  out->token = r->token;
  out->head = r->head;
  out->dtype = r->dtype;
  return PNB_OK;
}

// Whether rows x, already checked as written rows, and rows y are apart in
// memory: far from one another, or with the same type and strides (K and V side
// by side in one tensor).  `same` answers for x and y being the same rows.
inline bool apart(const DevRows &x, const DevRows &y, int T, int n_slot, int heads, int head_dim, bool same) {
  int64_t s[3] = {x.slot, x.token, x.head}, n[3] = {n_slot, T, heads};
  const int64_t sy[3] = {y.slot, y.token, y.head};
  const int64_t ex = x.dtype == PNB_F32 ? 4 : 2, ey = y.dtype == PNB_F32 ? 4 : 2;
  int64_t bx = head_dim, by = head_dim;
  bool alike = x.dtype == y.dtype;
  for (int i = 0; i < 3; ++i) {
    bx += s[i] * (n[i] - 1);
    by += sy[i] * (n[i] - 1);
    alike &= n[i] == 1 || s[i] == sy[i];
  }
  const int64_t diff = static_cast<uint8_t *>(y.p) - static_cast<uint8_t *>(x.p);
  if (diff >= bx * ex || -diff >= by * ey) return true;
  if (!alike) return false;
  if (diff == 0) return same;
  for (int i = 0; i < 2; ++i)          // strides in descending order
    for (int j = 0; j < 2 - i; ++j)
      if (s[j] < s[j + 1]) {
        std::swap(s[j], s[j + 1]);
        std::swap(n[j], n[j + 1]);
      }
  // Do steps i_d, |i_d| < n_d, lead from a row of x to within a row of one of y?
  // A stride is no shorter than what lies below it, so that only the two steps
  // about the distance can.
  for (int c = 0; c < 8; ++c) {
    int64_t left = diff / ex;
    for (int d = 0; d < 3; ++d) {
      if (n[d] <= 1) continue;
      int64_t i = left / s[d] - (left % s[d] < 0) + (c >> d & 1);
      i = std::min(std::max(i, 1 - n[d]), n[d] - 1);
      left -= i * s[d];
    }
    if (left < head_dim && left > -head_dim) return false;
  }
  return true;
}

// launch with programmatic dependent launch: every kernel of the caches waits
// (griddepcontrol.wait) before its first access to global memory
template <typename K, typename A>
inline cudaError_t launch_pdl(K kern, dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st,
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

}  // namespace pnb
