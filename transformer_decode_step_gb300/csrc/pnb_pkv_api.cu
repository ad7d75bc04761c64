// pnb_pkv_api.cu - the C ABI of the paged KV cache: checks, the library's workspace.
#include <cuda_runtime.h>

#include <cmath>
#include <new>
#include <vector>

#include "pnb.h"
#include "pnb_pkv.cuh"
#include "pnb_tmap.cuh"

using namespace pnb;

struct pnb_pkv {
  pnb_pkv_config cfg;
  int device = 0, sms = 0, page_log2 = 0;
  uint8_t *pool = nullptr;
  size_t layer_bytes = 0;
  uint8_t *ws = nullptr;
  unsigned long long *freq = nullptr;
  int32_t *err = nullptr;
  PkvGroup *groups = nullptr;
  PkvPart *part = nullptr;
  float *part_o = nullptr, *part_ml = nullptr, *row_o[2] = {}, *row_ml[2] = {};
  std::vector<CUtensorMap> maps;   // one per layer
};

namespace {

int check_config(const pnb_pkv_config &c) {
  if (c.n_layer <= 0 || c.n_page <= 0 || c.n_head <= 0 || c.n_kv_head <= 0 || c.shared_tok < 0) return PNB_E_INVAL;
  if (c.n_head % c.n_kv_head || (c.rope_neox != 0 && c.rope_neox != 1)) return PNB_E_INVAL;
  if (c.head_dim != 64 && c.head_dim != 128) return PNB_E_UNSUPPORTED;
  const int32_t *s = c.rope_section;
  if (s[0] < 0 || s[1] < 0 || s[2] < 0) return PNB_E_INVAL;
  if ((s[0] || s[1] || s[2]) && (int64_t)s[0] + s[1] + s[2] != c.head_dim / 2) return PNB_E_INVAL;
  if (!(c.rope_theta >= 0.0) || std::isinf(c.rope_theta)) return PNB_E_INVAL;
  if (c.page != 16 && c.page != 32 && c.page != 64 && c.page != 128) return PNB_E_UNSUPPORTED;
  if (c.n_head / c.n_kv_head > kPkvMaxGroup || c.n_head > 4096 || c.n_layer > 4096) return PNB_E_UNSUPPORTED;
  // a layer's rows are indexed with 32 bits, and so are the rows of a shared call
  if ((int64_t)c.n_page * 2 * c.n_kv_head >= (((int64_t)1 << 31) - 4096) / c.page) return PNB_E_UNSUPPORTED;
  if ((int64_t)c.shared_tok * c.n_head >= (int64_t)1 << 24) return PNB_E_UNSUPPORTED;
  return PNB_OK;
}

size_t layer_bytes_of(const pnb_pkv_config &c) {
  return (size_t)c.n_page * 2 * c.n_kv_head * c.page * c.head_dim * 2;
}

int check_call(const pnb_pkv *k, int layer) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return PNB_E_CUDA;
  if (dev != k->device) return PNB_E_WRONG_DEVICE;
  return layer >= 0 && layer < k->cfg.n_layer ? PNB_OK : PNB_E_INVAL;
}

int check_batch(const pnb_pkv *c, const pnb_pkv_batch *b, int32_t n_tok, PkvSeqs *out) {
  if (!b->len_dev || !b->pages_dev) return PNB_E_NULL;
  if (!aligned4(b->len_dev) || !aligned4(b->pages_dev) || !aligned4(b->start_dev)) return PNB_E_ALIGN;
  if (b->n_seq < 1 || b->max_page < 1 || n_tok < 1) return PNB_E_INVAL;
  if (!b->start_dev && n_tok % b->n_seq) return PNB_E_INVAL;
  if (b->n_seq > kPkvMaxSeq || (int64_t)n_tok * c->cfg.n_head >= (int64_t)1 << 31) return PNB_E_UNSUPPORTED;
  // a sequence's entries and row numbers are indexed with 32 bits
  if ((int64_t)b->max_page * c->cfg.page > (int64_t)1 << 30) return PNB_E_UNSUPPORTED;
  *out = PkvSeqs{b->start_dev, b->len_dev, b->pages_dev, b->n_seq, b->max_page, n_tok,
                 b->start_dev ? 0 : n_tok / b->n_seq};
  return PNB_OK;
}

PkvPool pool_of(const pnb_pkv *c, int layer) {
  return PkvPool{reinterpret_cast<__nv_bfloat16 *>(c->pool + (size_t)layer * c->layer_bytes), c->cfg.n_page,
                 c->page_log2, c->cfg.n_kv_head};
}

// whether a tensor's rows lie apart from the pool
bool off_pool(const pnb_pkv *c, const DevRows &r, int n_tok, int heads) {
  const int64_t es = r.dtype == PNB_F32 ? 4 : 2;
  const int64_t bytes = (r.token * (n_tok - 1) + r.head * (heads - 1) + c->cfg.head_dim) * es;
  const uint8_t *p = static_cast<const uint8_t *>(r.p);
  return p + bytes <= c->pool || p >= c->pool + c->layer_bytes * c->cfg.n_layer;
}

// Whether rows x and rows y (tokens by heads) are apart in memory: one behind the
// other, or side by side in the tokens of one tensor (a fused projection's).
bool rows_apart(const DevRows &x, int x_heads, const DevRows &y, int y_heads, int n_tok, int hd) {
  const int64_t ex = x.dtype == PNB_F32 ? 4 : 2, ey = y.dtype == PNB_F32 ? 4 : 2;
  const int64_t bx = (x.head * (x_heads - 1) + hd) * ex, by = (y.head * (y_heads - 1) + hd) * ey;   // a token's bytes
  const int64_t sx = x.token * ex, sy = y.token * ey;
  const int64_t diff = static_cast<uint8_t *>(y.p) - static_cast<uint8_t *>(x.p);
  if (diff >= bx + sx * (n_tok - 1) || -diff >= by + sy * (n_tok - 1)) return true;
  if (sx != sy || sx < bx || sx < by) return false;
  const int64_t at = ((diff % sx) + sx) % sx;   // y's token behind x's, within one stride
  return at >= bx && at + by <= sx;
}

int check_tokens(const pnb_pkv *c, const pnb_rows *r, int n_tok, int heads, bool written, DevRows *out) {
  pnb_rows one = *r;
  one.slot = 0;
  const int rc = check_rows(&one, n_tok, 1, heads, c->cfg.head_dim, written, out);
  if (rc != PNB_OK) return rc;
  return off_pool(c, *out, n_tok, heads) ? PNB_OK : PNB_E_INVAL;
}

// Up to this many rows (tokens x query heads of a KV head) of every sequence go
// through the kernel for steps (its registers hold 16).  At head_dim 128 a second block of 8
// rows costs it more than the tcgen05 kernel's empty rows do: 16 rows over 64 sequences of 4096,
// 64 of 300, 8 of 1000, 1 of 32768, 1 of 200, in bf16, cold L2: 421, 88, 49, 86, 29 us against 227, 72,
// 43, 61, 33; in fp32 430, 92, 49, 88, 33 against 291, 90, 53, 74, 37; at head_dim 64 in bf16
// 166, 47, 31, 41, 21 against 162, 57, 39, 49, 29, in fp32 178, 53, 35, 45, 23 against 215, 74, 47, 57, 35.
constexpr int kStepRows = 16, kStepRows128 = 8;
// A batch whose page tables have room for no more than this goes sequence by sequence, shared
// prefix or not: the pages that sequences share come from L2, at some 11 TB/s, and one kernel
// and its join take less than two passes.  Single tokens of 32 / 8 heads, head_dim 128, bf16, cold L2,
// tables of 10, 75, 151, 285, 302, 2416 MB: 25, 37, 46, 59, 68, 285 us against 44, 50, 52, 52, 67, 99.
// The host knows the tables' room, not the lengths: a batch of few entries in wide tables takes the second.
constexpr int64_t kDirectBytes = (int64_t)256 << 20;

int attend(pnb_pkv *c, int32_t layer, const pnb_pkv_batch *b, int32_t n_group, const int32_t *group_start,
           const int32_t *prefix, int32_t n_tok, const pnb_rows *q, const pnb_rows *out, int32_t window,
           pnb_stream stream) {
  const pnb_pkv_config &g = c->cfg;
  if (window < 0) return PNB_E_INVAL;
  PkvAttnArgs a{};
  int rc = check_batch(c, b, n_tok, &a.seqs);
  if (rc == PNB_OK) rc = check_tokens(c, q, n_tok, g.n_head, false, &a.q);
  if (rc == PNB_OK) rc = check_tokens(c, out, n_tok, g.n_head, true, &a.out);
  if (rc != PNB_OK) return rc;
  if (!apart(a.out, a.q, n_tok, 1, g.n_head, g.head_dim, true)) return PNB_E_INVAL;
  rc = check_call(c, layer);
  if (rc != PNB_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  a.pool = pool_of(c, layer);
  a.n_head = g.n_head;
  // a window that reaches past the page tables is none
  a.window = window < (int64_t)b->max_page * g.page ? window : 0;
  a.qscale = (float)(1.4426950408889634 / std::sqrt((double)g.head_dim));
  a.err = c->err;
  a.part = c->part;
  a.part_o = c->part_o;
  a.part_ml = c->part_ml;
  a.grid = c->sms;
  a.block_rows = pkv_block_rows(g.head_dim, pkv_split(a));
  a.pass = kPkvAll;
  const CUtensorMap &map = c->maps[layer];
  const int group = g.n_head / g.n_kv_head;
  const bool step = a.seqs.each > 0 && (int64_t)a.seqs.each * group <= (g.head_dim == 128 ? kStepRows128 : kStepRows);
  const int64_t held = (int64_t)b->n_seq * b->max_page * g.page * g.n_kv_head * g.head_dim * 4;
  cudaError_t e = cudaSuccess;
  if (group_start && held > kDirectBytes) {
    a.group_start = group_start;
    a.prefix = prefix;
    a.n_group = n_group;
    a.groups = c->groups;
    for (int i = 0; i < 2; ++i) {
      a.row_o[i] = c->row_o[i];
      a.row_ml[i] = c->row_ml[i];
    }
    // the prefix's pass, and beside it, with partial sums of its own, the other
    PkvAttnArgs p = a, o = a;
    p.pass = kPkvPrefix;
    o.pass = kPkvOwn;
    if (step) pkv_step_cost(g.head_dim, &p.other_ns, &p.other_item_units);
    else pkv_rows_cost(g.head_dim, pkv_split(a), &p.other_ns, &p.other_item_units);
    p.other_tile = step ? kPkvChunk : kPkvTile;
    pkv_rows_cost(g.head_dim, pkv_split(a), &o.other_ns, &o.other_item_units);
    o.other_tile = kPkvTile;
    o.part += 2 * c->sms;
    o.part_o += (size_t)2 * c->sms * kPkvBlockRows * g.head_dim;
    o.part_ml += (size_t)2 * c->sms * kPkvBlockRows * 2;
    e = launch_pkv_rows(g.head_dim, map, p, st);
    if (e == cudaSuccess)
      e = step ? launch_pkv_step(g.head_dim, map, o, st) : launch_pkv_rows(g.head_dim, map, o, st);
    a.pass = kPkvPrefix;
  } else {
    e = step ? launch_pkv_step(g.head_dim, map, a, st) : launch_pkv_rows(g.head_dim, map, a, st);
  }
  if (e == cudaSuccess)
    e = launch_pkv_join(g.head_dim, a, step ? a.seqs.each * group : kPkvBlockRows, st);
  return e == cudaSuccess ? PNB_OK : PNB_E_CUDA;
}

}  // namespace

extern "C" {

size_t pnb_pkv_bytes(const pnb_pkv_config *cfg) {
  if (!cfg || check_config(*cfg) != PNB_OK) return 0;
  return layer_bytes_of(*cfg) * cfg->n_layer;
}

int pnb_pkv_new(const pnb_pkv_config *cfg, void *pool_dev, size_t bytes, pnb_pkv **out) {
  if (!cfg || !pool_dev || !out) return PNB_E_NULL;
  *out = nullptr;
  const int rc = check_config(*cfg);
  if (rc != PNB_OK) return rc;
  if (reinterpret_cast<uintptr_t>(pool_dev) & 127u) return PNB_E_ALIGN;
  if (bytes < pnb_pkv_bytes(cfg)) return PNB_E_INVAL;
  pnb_pkv *k = new (std::nothrow) pnb_pkv();
  if (!k) return PNB_E_NOMEM;
  const pnb_pkv_config &c = *cfg;
  k->cfg = c;
  k->pool = static_cast<uint8_t *>(pool_dev);
  k->layer_bytes = layer_bytes_of(c);
  while (1 << k->page_log2 < c.page) ++k->page_log2;
  // turns per position, theta^(-2i/hd) / (2 pi), as fractions of 2^64
  unsigned long long freq[64] = {};
  for (int i = 0; i < c.head_dim / 2 && c.rope_theta > 0.0; ++i) {
    const double turns = std::pow(c.rope_theta, -2.0 * i / c.head_dim) * 0.15915494309189533577;
    freq[i] = (unsigned long long)std::ldexp(turns - std::floor(turns), 64);
  }
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  cudaError_t e = cudaGetDevice(&k->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&k->sms, cudaDevAttrMultiProcessorCount, k->device);
  if (e == cudaSuccess) e = prepare_pkv_rows(c.head_dim);
  if (e == cudaSuccess) e = prepare_pkv_step(c.head_dim);
  k->sms = k->sms < kPkvMaxCtas ? k->sms : kPkvMaxCtas;
  bool maps = e == cudaSuccess;
  try {
    if (maps) k->maps.resize(c.n_layer);
  } catch (...) {
    delete k;
    return PNB_E_NOMEM;
  }
  for (int l = 0; l < c.n_layer && maps; ++l)
    maps = encode_map(&k->maps[l], k->pool + (size_t)l * k->layer_bytes, (int64_t)c.n_page * 2 * c.n_kv_head * c.page,
                      c.head_dim, c.page < 1 << kPkvBoxLog2 ? c.page : 1 << kPkvBoxLog2);
  if (e == cudaSuccess && !maps) e = cudaErrorUnknown;
  // two partial sums per CTA, for either of the passes over a shared prefix
  const size_t parts = (size_t)2 * k->sms * (c.shared_tok ? 2 : 1), part_rows = parts * kPkvBlockRows;
  const size_t rows = (size_t)c.shared_tok * c.n_head;
  const size_t o_err = take(4), o_freq = take(sizeof(freq)), o_part = take(parts * sizeof(PkvPart));
  const size_t zeroed = at;
  const size_t o_groups = take(kPkvMaxSeq * sizeof(PkvGroup));
  const size_t o_pml = take(part_rows * 8), o_po = take(part_rows * c.head_dim * 4);
  const size_t o_rml = take(rows * 8), o_ro = take(rows * c.head_dim * 4);
  const size_t o_rml2 = take(rows * 8), o_ro2 = take(rows * c.head_dim * 4);
  if (e == cudaSuccess) e = cudaMalloc(&k->ws, at);
  if (e == cudaSuccess) e = clear_now(k->ws, zeroed);
  if (e == cudaSuccess) e = cudaMemcpy(k->ws + o_freq, freq, sizeof(freq), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) {
    cudaGetLastError();
    if (k->ws) cudaFree(k->ws);
    delete k;
    return e == cudaErrorMemoryAllocation ? PNB_E_NOMEM : PNB_E_CUDA;
  }
  k->err = reinterpret_cast<int32_t *>(k->ws + o_err);
  k->freq = reinterpret_cast<unsigned long long *>(k->ws + o_freq);
  k->groups = reinterpret_cast<PkvGroup *>(k->ws + o_groups);
  k->part = reinterpret_cast<PkvPart *>(k->ws + o_part);
  k->part_ml = reinterpret_cast<float *>(k->ws + o_pml);
  k->part_o = reinterpret_cast<float *>(k->ws + o_po);
  k->row_ml[0] = reinterpret_cast<float *>(k->ws + o_rml);
  k->row_o[0] = reinterpret_cast<float *>(k->ws + o_ro);
  k->row_ml[1] = reinterpret_cast<float *>(k->ws + o_rml2);
  k->row_o[1] = reinterpret_cast<float *>(k->ws + o_ro2);
  *out = k;
  return PNB_OK;
}

void pnb_pkv_free(pnb_pkv *c) {
  if (!c) return;
  cudaFree(c->ws);
  delete c;
}

int pnb_pkv_append(pnb_pkv *c, int32_t layer, const pnb_pkv_batch *b, int32_t n_tok, const pnb_rows *k,
                   const pnb_rows *v, const pnb_rows *q, const pnb_rows *q_out, const int32_t *pos_dev,
                   pnb_stream stream) {
  if (!c || !b || !k || !v || !q != !q_out) return PNB_E_NULL;
  const pnb_pkv_config &g = c->cfg;
  PkvAppendArgs a{};
  int rc = check_batch(c, b, n_tok, &a.seqs);
  if (rc == PNB_OK) rc = check_tokens(c, k, n_tok, g.n_kv_head, false, &a.k);
  if (rc == PNB_OK) rc = check_tokens(c, v, n_tok, g.n_kv_head, false, &a.v);
  if (rc == PNB_OK && q) rc = check_tokens(c, q, n_tok, g.n_head, false, &a.q);
  if (rc == PNB_OK && q) rc = check_tokens(c, q_out, n_tok, g.n_head, true, &a.q_out);
  if (rc != PNB_OK) return rc;
  if (!aligned4(pos_dev)) return PNB_E_ALIGN;
  if (k->dtype != v->dtype || (q && q->dtype != k->dtype)) return PNB_E_INVAL;
  if (q) {
    // the rotated queries lie over no other rows of the call but q's own
    if (!apart(a.q_out, a.q, n_tok, 1, g.n_head, g.head_dim, true)) return PNB_E_INVAL;
    // (k and v of as many heads may also lie between q's heads)
    auto clear = [&](const DevRows &r) {
      return rows_apart(a.q_out, g.n_head, r, g.n_kv_head, n_tok, g.head_dim) ||
             (g.n_head == g.n_kv_head && apart(a.q_out, r, n_tok, 1, g.n_head, g.head_dim, false));
    };
    if (!clear(a.k) || !clear(a.v)) return PNB_E_INVAL;
  }
  rc = check_call(c, layer);
  if (rc != PNB_OK) return rc;
  a.pool = pool_of(c, layer);
  a.n_head = g.n_head;
  a.pos = pos_dev;
  const bool axes = g.rope_section[0] || g.rope_section[1] || g.rope_section[2];
  a.sec0 = axes ? g.rope_section[0] : g.head_dim / 2;
  a.sec1 = axes ? g.rope_section[0] + g.rope_section[1] : g.head_dim / 2;
  a.freq = g.rope_theta > 0.0 ? c->freq : nullptr;
  a.err = c->err;
  a.sms = c->sms;
  return launch_pkv_append(g.head_dim, g.rope_neox != 0, a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PNB_OK
             : PNB_E_CUDA;
}

int pnb_pkv_attention(pnb_pkv *c, int32_t layer, const pnb_pkv_batch *b, int32_t n_tok, const pnb_rows *q,
                      const pnb_rows *out, int32_t window, pnb_stream stream) {
  if (!c || !b || !q || !out) return PNB_E_NULL;
  return attend(c, layer, b, 0, nullptr, nullptr, n_tok, q, out, window, stream);
}

int pnb_pkv_attention_shared(pnb_pkv *c, int32_t layer, const pnb_pkv_batch *b, int32_t n_group,
                             const int32_t *group_start_dev, const int32_t *prefix_dev, int32_t n_tok,
                             const pnb_rows *q, const pnb_rows *out, int32_t window, pnb_stream stream) {
  if (!c || !b || !group_start_dev || !prefix_dev || !q || !out) return PNB_E_NULL;
  if (!aligned4(group_start_dev) || !aligned4(prefix_dev)) return PNB_E_ALIGN;
  if (n_group < 1 || n_group > b->n_seq || b->start_dev || n_tok > c->cfg.shared_tok) return PNB_E_INVAL;
  return attend(c, layer, b, n_group, group_start_dev, prefix_dev, n_tok, q, out, window, stream);
}

int pnb_pkv_check(pnb_pkv *c, int32_t *device_error) {
  if (!c) return PNB_E_NULL;
  const int rc = check_call(c, 0);
  if (rc != PNB_OK) return rc;
  int32_t e = 0;
  const int32_t zero = 0;
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(&e, c->err, sizeof(e), cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemcpy(c->err, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
    return PNB_E_CUDA;
  if (device_error) *device_error = e;
  return e ? PNB_E_DEVICE : PNB_OK;
}

}  // extern "C"
