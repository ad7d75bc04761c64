// pnb_kv4_api.cu - the C ABI of the 4-bit KV cache: checks, the layout of the
// caller's buffer, the library's workspace.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <utility>

#include "pnb.h"
#include "pnb_kv4.cuh"

using namespace pnb;

struct pnb_kvq {
  pnb_kvq_config cfg;
  int device = 0, ng = 0, sms = 0, grid = 0;   // grid: the attention's CTAs
  uint8_t *buf = nullptr;
  // byte offsets within a layer, and a layer's bytes
  size_t o_ids = 0, o_weights = 0, o_len = 0, o_seen = 0, layer_bytes = 0;
  uint8_t *ws = nullptr;
  float *part = nullptr, *part_ml = nullptr, *warp_part = nullptr, *scores = nullptr;
  float2 *wscale = nullptr;
  unsigned *counter = nullptr;
  uint32_t *arrive = nullptr;
  int32_t *err = nullptr, *n_old = nullptr, *src_of = nullptr, *movers = nullptr;
  uint8_t *border = nullptr;
};

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }

int check_config(const pnb_kvq_config &c) {
  if (c.n_layer <= 0 || c.n_slot <= 0 || c.n_head <= 0 || c.n_kv_head <= 0 || c.cap <= 0 || c.track < 0)
    return PNB_E_INVAL;
  if (c.n_head % c.n_kv_head || c.cap % kKv4Chunk) return PNB_E_INVAL;
  const int G = c.n_head / c.n_kv_head;
  if (c.head_dim != 32 && c.head_dim != 64 && c.head_dim != 128) return PNB_E_UNSUPPORTED;
  if (G > kKv4MaxRows || (int64_t)c.track * G > kKv4MaxRows || c.n_slot > kKv4MaxSlots ||
      c.n_kv_head > 1024 || c.n_layer > 4096 || c.cap > kKv4MaxCap)
    return PNB_E_UNSUPPORTED;
  // the flat list of work chunks is indexed with 32 bits
  const int64_t chunks = (int64_t)c.n_slot * c.n_kv_head * (c.cap / kKv4Chunk + 2);
  if (chunks * (kKv4MaxRows / 4) >= (int64_t)1 << 31) return PNB_E_UNSUPPORTED;
  return PNB_OK;
}

void lay_out(pnb_kvq *k) {
  const pnb_kvq_config &c = k->cfg;
  k->ng = c.head_dim / 32;
  const size_t entries = (size_t)c.n_slot * c.n_kv_head * c.cap;
  k->o_ids = align256(entries / kKv4Chunk * kv4_chunk_bytes(k->ng));
  k->o_weights = k->o_ids + align256(entries * 4);
  k->o_len = k->o_weights + align256(entries * 4);
  k->o_seen = k->o_len + align256((size_t)c.n_slot * 4);
  k->layer_bytes = k->o_seen + align256((size_t)c.n_slot * 4);
}

Kv4Layer layer_of(const pnb_kvq *k, int layer) {
  uint8_t *base = k->buf + (size_t)layer * k->layer_bytes;
  Kv4Layer l;
  l.codes = base;
  l.ids = reinterpret_cast<int32_t *>(base + k->o_ids);
  l.weights = reinterpret_cast<float *>(base + k->o_weights);
  l.len = reinterpret_cast<int32_t *>(base + k->o_len);
  l.seen = reinterpret_cast<int32_t *>(base + k->o_seen);
  l.cap = k->cfg.cap;
  return l;
}

// Zeroes device memory before it returns: the first call that reads it may be on
// any stream, and a non-blocking one does not wait for a clear on the default
// stream (which may itself be behind other work there).
cudaError_t clear_now(void *p, size_t n) {
  cudaStream_t st;
  cudaError_t e = cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(p, 0, n, st);
  const cudaError_t done = cudaStreamSynchronize(st);
  cudaStreamDestroy(st);
  return e != cudaSuccess ? e : done;
}

int check_call(const pnb_kvq *k, int layer) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return PNB_E_CUDA;
  if (dev != k->device) return PNB_E_WRONG_DEVICE;
  return layer >= 0 && layer < k->cfg.n_layer ? PNB_OK : PNB_E_INVAL;
}

// a caller's rows: type, 16-byte alignment of every row, no negative strides;
// rows that are written must not lie over one another
int check_rows(const pnb_rows *r, int T, int n_slot, int heads, int head_dim, bool written, Kv4Rows *out) {
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
bool apart(const Kv4Rows &x, const Kv4Rows &y, int T, int n_slot, int heads, int head_dim, bool same) {
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

}  // namespace

extern "C" {

size_t pnb_kvq_bytes(const pnb_kvq_config *cfg) {
  if (!cfg || check_config(*cfg) != PNB_OK) return 0;
  pnb_kvq k;
  k.cfg = *cfg;
  lay_out(&k);
  return k.layer_bytes * cfg->n_layer;
}

int pnb_kvq_new(const pnb_kvq_config *cfg, void *buf_dev, size_t bytes, pnb_kvq **out) {
  if (!cfg || !buf_dev || !out) return PNB_E_NULL;
  *out = nullptr;
  const int rc = check_config(*cfg);
  if (rc != PNB_OK) return rc;
  if (reinterpret_cast<uintptr_t>(buf_dev) & 127u) return PNB_E_ALIGN;
  if (bytes < pnb_kvq_bytes(cfg)) return PNB_E_INVAL;
  pnb_kvq *k = new (std::nothrow) pnb_kvq();
  if (!k) return PNB_E_NOMEM;
  k->cfg = *cfg;
  lay_out(k);
  k->buf = static_cast<uint8_t *>(buf_dev);
  if (cudaGetDevice(&k->device) != cudaSuccess || prepare_kv4_kernels(k->ng, &k->sms) != cudaSuccess) {
    cudaGetLastError();
    delete k;
    return PNB_E_CUDA;
  }
  k->grid = k->sms * kKv4CtasPerSm;
  const pnb_kvq_config &c = *cfg;
  const size_t entries = (size_t)c.n_slot * c.n_kv_head * c.cap;
  const size_t part_rows = (size_t)2 * k->grid * kKv4Rows;
  const size_t rows = (size_t)c.n_slot * c.n_head * c.track;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  const size_t o_err = take(4), o_counter = take(4 * (size_t)k->grid), o_arrive = take(4 * (size_t)c.n_slot);
  const size_t zeroed = at;
  const size_t o_nold = take(4 * (size_t)c.n_slot), o_ml = take(part_rows * 8);
  const size_t o_part = take(part_rows * c.head_dim * 4);
  const size_t o_wpart = take(part_rows / 2 * kKv4Warps * c.head_dim * 4);
  const size_t o_src = take(entries * 4), o_mov = take(entries * 4);
  const size_t o_border = take((size_t)c.n_slot * c.n_kv_head * 512 * k->ng);
  const size_t o_wscale = take(rows * 8), o_scores = take(rows * c.cap * 4);
  cudaError_t e = cudaMalloc(&k->ws, at);
  if (e == cudaSuccess) e = clear_now(k->ws, zeroed);
  if (e != cudaSuccess) {
    cudaGetLastError();
    if (k->ws) cudaFree(k->ws);
    delete k;
    return e == cudaErrorMemoryAllocation ? PNB_E_NOMEM : PNB_E_CUDA;
  }
  k->err = reinterpret_cast<int32_t *>(k->ws + o_err);
  k->counter = reinterpret_cast<unsigned *>(k->ws + o_counter);
  k->arrive = reinterpret_cast<uint32_t *>(k->ws + o_arrive);
  k->n_old = reinterpret_cast<int32_t *>(k->ws + o_nold);
  k->part_ml = reinterpret_cast<float *>(k->ws + o_ml);
  k->part = reinterpret_cast<float *>(k->ws + o_part);
  k->warp_part = reinterpret_cast<float *>(k->ws + o_wpart);
  k->src_of = reinterpret_cast<int32_t *>(k->ws + o_src);
  k->movers = reinterpret_cast<int32_t *>(k->ws + o_mov);
  k->border = k->ws + o_border;
  k->wscale = reinterpret_cast<float2 *>(k->ws + o_wscale);
  k->scores = reinterpret_cast<float *>(k->ws + o_scores);
  *out = k;
  return PNB_OK;
}

void pnb_kvq_free(pnb_kvq *k) {
  if (!k) return;
  cudaFree(k->ws);
  delete k;
}

int pnb_kvq_reset(pnb_kvq *k, int32_t slot, pnb_stream stream) {
  if (!k) return PNB_E_NULL;
  if (slot < -1 || slot >= k->cfg.n_slot) return PNB_E_INVAL;
  const int rc = check_call(k, 0);
  if (rc != PNB_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Kv4Layer l = layer_of(k, 0);
  if (launch_kv4_reset(l.len, l.seen, (int64_t)(k->layer_bytes / 4), k->cfg.n_layer, k->cfg.n_slot, slot, st) !=
      cudaSuccess)
    return PNB_E_CUDA;
  if (slot < 0 && cudaMemsetAsync(k->err, 0, 4, st) != cudaSuccess) return PNB_E_CUDA;
  return PNB_OK;
}

int pnb_kvq_append(pnb_kvq *c, int32_t layer, const pnb_rows *k, const pnb_rows *v, int32_t T,
                   const int32_t *n_new_dev, const int32_t *start_dev, pnb_stream stream) {
  if (!c || !k || !v) return PNB_E_NULL;
  if (T < 1 || T > c->cfg.cap) return PNB_E_INVAL;
  if (!aligned4(n_new_dev) || !aligned4(start_dev)) return PNB_E_ALIGN;
  const pnb_kvq_config &g = c->cfg;
  Kv4AppendArgs a{};
  int rc = check_rows(k, T, g.n_slot, g.n_kv_head, g.head_dim, false, &a.k);
  if (rc == PNB_OK) rc = check_rows(v, T, g.n_slot, g.n_kv_head, g.head_dim, false, &a.v);
  if (rc != PNB_OK) return rc;
  if (k->dtype != v->dtype) return PNB_E_INVAL;
  rc = check_call(c, layer);
  if (rc != PNB_OK) return rc;
  a.l = layer_of(c, layer);
  a.n_new = n_new_dev;
  a.start = start_dev;
  a.n_slot = g.n_slot;
  a.n_kv = g.n_kv_head;
  a.T = T;
  a.sms = c->sms;
  a.arrive = c->arrive;
  a.err = c->err;
  return launch_kv4_append(c->ng, a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PNB_OK : PNB_E_CUDA;
}

int pnb_kvq_read(pnb_kvq *c, int32_t layer, const int32_t *first_dev, int32_t T, const pnb_rows *k,
                 const pnb_rows *v, pnb_stream stream) {
  if (!c || !k || !v) return PNB_E_NULL;
  if (T < 1 || T > c->cfg.cap) return PNB_E_INVAL;
  if (!aligned4(first_dev)) return PNB_E_ALIGN;
  const pnb_kvq_config &g = c->cfg;
  Kv4ReadArgs a{};
  int rc = check_rows(k, T, g.n_slot, g.n_kv_head, g.head_dim, true, &a.k);
  if (rc == PNB_OK) rc = check_rows(v, T, g.n_slot, g.n_kv_head, g.head_dim, true, &a.v);
  if (rc != PNB_OK) return rc;
  if (k->dtype != v->dtype || !apart(a.k, a.v, T, g.n_slot, g.n_kv_head, g.head_dim, false)) return PNB_E_INVAL;
  rc = check_call(c, layer);
  if (rc != PNB_OK) return rc;
  a.l = layer_of(c, layer);
  a.first = first_dev;
  a.err = c->err;
  a.n_slot = g.n_slot;
  a.n_kv = g.n_kv_head;
  a.T = T;
  a.sms = c->sms;
  return launch_kv4_read(c->ng, a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PNB_OK : PNB_E_CUDA;
}

int pnb_kvq_attention(pnb_kvq *c, int32_t layer, const pnb_rows *q, int32_t T, const pnb_rows *out,
                      float decay, pnb_stream stream) {
  if (!c || !q || !out) return PNB_E_NULL;
  const pnb_kvq_config &g = c->cfg;
  const int G = g.n_head / g.n_kv_head;
  const bool track = decay >= 0.f;
  if (T < 1 || std::isnan(decay) || std::isinf(decay)) return PNB_E_INVAL;
  if ((int64_t)T * G > kKv4MaxRows) return PNB_E_UNSUPPORTED;
  if (track && T > g.track) return PNB_E_INVAL;
  Kv4AttnArgs a{};
  int rc = check_rows(q, T, g.n_slot, g.n_head, g.head_dim, false, &a.q);
  if (rc == PNB_OK) rc = check_rows(out, T, g.n_slot, g.n_head, g.head_dim, true, &a.out);
  if (rc != PNB_OK) return rc;
  if (!apart(a.out, a.q, T, g.n_slot, g.n_head, g.head_dim, true)) return PNB_E_INVAL;
  rc = check_call(c, layer);
  if (rc != PNB_OK) return rc;
  a.l = layer_of(c, layer);
  a.n_slot = g.n_slot;
  a.n_kv = g.n_kv_head;
  a.G = G;
  a.T = T;
  a.rows = T * G;
  a.qscale = (float)(1.4426950408889634 / std::sqrt((double)g.head_dim));
  a.part = c->part;
  a.part_ml = c->part_ml;
  a.warp_part = c->warp_part;
  a.counter = c->counter;
  a.err = c->err;
  a.scores = track ? c->scores : nullptr;
  a.wscale = track ? c->wscale : nullptr;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (launch_kv4_attn(c->ng, a, c->grid, st) != cudaSuccess) return PNB_E_CUDA;
  if (track) {
    Kv4WeightArgs w{};
    w.l = a.l;
    w.scores = a.scores;
    w.wscale = a.wscale;
    w.n_slot = a.n_slot;
    w.n_kv = a.n_kv;
    w.rows = a.rows;
    w.sms = c->sms;
    w.decay = decay;
    if (launch_kv4_weights(w, st) != cudaSuccess) return PNB_E_CUDA;
  }
  return PNB_OK;
}

int pnb_kvq_evict(pnb_kvq *src, int32_t src_layer, pnb_kvq *dst, int32_t dst_layer, int32_t budget,
                  int32_t n_sink, int32_t n_recent, pnb_stream stream) {
  if (!src || !dst) return PNB_E_NULL;
  const pnb_kvq_config &s = src->cfg, &d = dst->cfg;
  if (budget < 1 || n_sink < 0 || n_recent < 0 || (int64_t)n_sink + n_recent > budget) return PNB_E_INVAL;
  if (s.n_slot != d.n_slot || s.n_kv_head != d.n_kv_head || s.head_dim != d.head_dim) return PNB_E_INVAL;
  if (budget > d.cap) return PNB_E_INVAL;
  // one buffer, or two that are apart
  if (src->buf == dst->buf ? s.cap != d.cap
                           : src->buf < dst->buf + dst->layer_bytes * d.n_layer &&
                                 dst->buf < src->buf + src->layer_bytes * s.n_layer)
    return PNB_E_INVAL;
  if (s.cap > kKv4MaxEvictCap) return PNB_E_UNSUPPORTED;
  int rc = check_call(src, src_layer);
  if (rc == PNB_OK) rc = check_call(dst, dst_layer);
  if (rc != PNB_OK) return rc;
  Kv4EvictArgs a{};
  a.src = layer_of(src, src_layer);
  a.dst = layer_of(dst, dst_layer);
  a.n_slot = s.n_slot;
  a.n_kv = s.n_kv_head;
  a.budget = budget;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.in_place = a.src.codes == a.dst.codes;
  a.src_of = src->src_of;
  a.movers = src->movers;
  a.border = src->border;
  a.ng = src->ng;
  a.n_old = src->n_old;
  a.arrive = src->arrive;
  return launch_kv4_evict(src->ng, a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PNB_OK : PNB_E_CUDA;
}

int pnb_kvq_layer_views(const pnb_kvq *k, int32_t layer, pnb_kvq_views *out) {
  if (!k || !out) return PNB_E_NULL;
  if (layer < 0 || layer >= k->cfg.n_layer) return PNB_E_INVAL;
  const Kv4Layer l = layer_of(k, layer);
  out->len = l.len;
  out->seen = l.seen;
  out->ids = l.ids;
  out->weights = l.weights;
  return PNB_OK;
}

int pnb_kvq_check(pnb_kvq *k, int32_t *device_error) {
  if (!k) return PNB_E_NULL;
  const int rc = check_call(k, 0);
  if (rc != PNB_OK) return rc;
  int32_t e = 0;
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(&e, k->err, sizeof(e), cudaMemcpyDeviceToHost) != cudaSuccess)
    return PNB_E_CUDA;
  if (device_error) *device_error = e;
  return e ? PNB_E_DEVICE : PNB_OK;
}

}  // extern "C"
