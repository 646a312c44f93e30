// The C ABI of the 4-bit KV cache (include/gdn.h): argument checks, then one
// launcher per call.
#include <cmath>

#include "kv4.cuh"

using namespace gdn;

namespace {

constexpr int kMaxSms = 160;  // what the workspaces are sized for, so that their size needs no device

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_E_CUDA; }

// SMs of the current device (0: the query failed).
int num_sms() {
  static int known[64] = {};
  int dev = -1, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < 64 && known[dev]) return known[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev] = n;
  return n;
}

// The cache and the batch; rows = T * heads of the largest tensor.
gdn_status check(const kv4_cache *c, const kv4_batch *b, Kv4Args &a, int32_t *status) {
  if (!c || !b) return GDN_E_NULL;
  if (b->B < 0 || b->T < 0 || b->max_pages < 0) return GDN_E_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return GDN_E_SHAPE;
  const int p = c->page_tokens;
  if (p != 16 && p != 32 && p != 64 && p != 128 && p != 256) return GDN_E_SHAPE;
  if (c->num_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024) return GDN_E_SHAPE;
  if (b->B == 0 && b->T != 0) return GDN_E_SHAPE;
  if (!std::isfinite(c->k_scale) || !std::isfinite(c->v_scale)) return GDN_E_NONFINITE;
  if (!(c->k_scale > 0.0f) || !(c->v_scale > 0.0f)) return GDN_E_BAD_SCALE;
  if (b->T > 0) {
    if (!c->pages || !b->kv_len || !b->block_table) return GDN_E_NULL;
    if (b->max_pages < 1 || (!b->q_start && b->T % b->B)) return GDN_E_SHAPE;
    if (!aligned16(c->pages)) return GDN_E_ALIGN;
    if ((reinterpret_cast<uintptr_t>(b->kv_len) | reinterpret_cast<uintptr_t>(b->block_table) |
         reinterpret_cast<uintptr_t>(b->q_start)) & 3u)
      return GDN_E_ALIGN;
    if ((long long)b->max_pages * p > 0x7fffffffLL) return GDN_E_OVERFLOW;
  }
  a = Kv4Args{c->pages, c->num_pages, p, c->n_kv_heads, c->head_dim, c->k_scale, c->v_scale, b->kv_len,
              b->block_table, b->q_start, b->B, b->max_pages, b->T, status, wait_budget(),
              b->q_start ? b->zero_padding & 3 : 0};
  return GDN_OK;
}

bool heads_fit(const kv4_cache *c, int Hq) { return Hq > 0 && Hq % c->n_kv_heads == 0 && Hq / c->n_kv_heads <= 64; }

gdn_status check_attn(const kv4_cache *c, const kv4_batch *b, const uint16_t *q, int64_t q_stride, int Hq, float sm,
                      uint16_t *out, float *lse, int32_t *status, Kv4AttnArgs &a) {
  gdn_status st = check(c, b, a.c, status);
  if (st != GDN_OK) return st;
  if (!heads_fit(c, Hq)) return GDN_E_SHAPE;
  if (!std::isfinite(sm)) return GDN_E_NONFINITE;
  if (!(sm > 0.0f)) return GDN_E_BAD_SCALE;
  if (b->T > 0) {
    if (!q || !out) return GDN_E_NULL;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u)) return GDN_E_ALIGN;
    if (q_stride % 8 || q_stride < (int64_t)Hq * c->head_dim) return GDN_E_SHAPE;
    if ((long long)b->T * Hq > 0x7fffffffLL) return GDN_E_OVERFLOW;
  }
  a.q = q;
  a.q_stride = q_stride;
  a.Hq = Hq;
  a.sm_scale = sm;
  a.out = out;
  a.lse = lse;
  return GDN_OK;
}

gdn_status check_pages(const Kv4PageArgs &a) {
  if (a.layers < 1 || a.num_pages < 1 || a.page_bytes < 16 || a.page_bytes % 16 || a.n < 0) return GDN_E_SHAPE;
  if (a.page_bytes > (1LL << 40) / a.num_pages) return GDN_E_OVERFLOW;
  if (a.layers > 1 && (a.layer_stride % 16 || a.layer_stride < a.num_pages * a.page_bytes)) return GDN_E_SHAPE;
  if (!a.pages) return GDN_E_NULL;
  if (!aligned16(a.pages)) return GDN_E_ALIGN;
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status kv4_append(const kv4_cache *c, const kv4_batch *b, const uint16_t *k, int64_t k_stride, const uint16_t *v,
                      int64_t v_stride, int32_t *dev_status, void *stream) {
  Kv4Args a{};
  gdn_status st = check(c, b, a, dev_status);
  if (st != GDN_OK || b->T == 0) return st;
  if (!k || !v) return GDN_E_NULL;
  if (!aligned16(k) || !aligned16(v)) return GDN_E_ALIGN;
  const int64_t row = (int64_t)c->n_kv_heads * c->head_dim;
  if (k_stride % 8 || v_stride % 8 || k_stride < row || v_stride < row) return GDN_E_SHAPE;
  return cuda_status(launch_kv4_append(a, k, k_stride, v, v_stride, static_cast<cudaStream_t>(stream)));
}

gdn_status kv4_read(const kv4_cache *c, const kv4_batch *b, uint16_t *k, uint16_t *v, int32_t *dev_status,
                    void *stream) {
  Kv4Args a{};
  gdn_status st = check(c, b, a, dev_status);
  if (st != GDN_OK || b->T == 0) return st;
  if (!k || !v) return GDN_E_NULL;
  if (!aligned16(k) || !aligned16(v)) return GDN_E_ALIGN;
  return cuda_status(launch_kv4_read(a, k, v, static_cast<cudaStream_t>(stream)));
}

// 0 for arguments that kv4_decode refuses.
size_t kv4_decode_workspace(const kv4_cache *c, const kv4_batch *b, int n_q_heads) {
  Kv4AttnArgs a{};
  if (check(c, b, a.c, nullptr) != GDN_OK || b->T == 0 || b->q_start || !heads_fit(c, n_q_heads)) return 0;
  a.Hq = n_q_heads;
  return kv4_decode_bytes(a, kMaxSms);
}

gdn_status kv4_decode(const kv4_cache *c, const kv4_batch *b, const uint16_t *q, int64_t q_stride, int n_q_heads,
                      float sm_scale, uint16_t *out, float *lse, void *workspace, size_t workspace_bytes,
                      int32_t *dev_status, void *stream) {
  Kv4AttnArgs a{};
  gdn_status st = check_attn(c, b, q, q_stride, n_q_heads, sm_scale, out, lse, dev_status, a);
  if (st != GDN_OK) return st;
  if (b->q_start) return GDN_E_SHAPE;
  if (b->T == 0) return GDN_OK;
  const size_t need = kv4_decode_bytes(a, kMaxSms);
  if (need && !workspace) return GDN_E_NULL;
  if (workspace_bytes < need) return GDN_E_SHAPE;
  if (!aligned16(workspace)) return GDN_E_ALIGN;
  const int sms = num_sms();
  if (sms < 1) return GDN_E_CUDA;
  return cuda_status(launch_kv4_decode(a, workspace, sms < kMaxSms ? sms : kMaxSms, static_cast<cudaStream_t>(stream)));
}

// 0 for arguments that kv4_prefill refuses.
size_t kv4_prefill_workspace(const kv4_cache *c, const kv4_batch *b, int64_t total_kv, int n_q_heads) {
  Kv4AttnArgs a{};
  if (check(c, b, a.c, nullptr) != GDN_OK || b->T == 0 || !heads_fit(c, n_q_heads)) return 0;
  if (total_kv < 0 || total_kv > 0x7fffffffLL) return 0;
  return kv4_prefill_bytes(a, total_kv);
}

gdn_status kv4_prefill(const kv4_cache *c, const kv4_batch *b, int64_t total_kv, const uint16_t *q, int64_t q_stride,
                       int n_q_heads, float sm_scale, uint16_t *out, float *lse, void *workspace,
                       size_t workspace_bytes, int32_t *dev_status, void *stream) {
  Kv4AttnArgs a{};
  gdn_status st = check_attn(c, b, q, q_stride, n_q_heads, sm_scale, out, lse, dev_status, a);
  if (st != GDN_OK) return st;
  if (total_kv < 0) return GDN_E_SHAPE;
  if (b->T == 0) return GDN_OK;
  const size_t need = total_kv > 0x7fffffffLL ? 0 : kv4_prefill_bytes(a, total_kv);
  if (need == 0) return GDN_E_OVERFLOW;
  if (!workspace) return GDN_E_NULL;
  if (workspace_bytes < need) return GDN_E_SHAPE;
  if (!aligned16(workspace)) return GDN_E_ALIGN;
  const int sms = num_sms();
  if (sms < 1) return GDN_E_CUDA;
  return cuda_status(launch_kv4_prefill(a, total_kv, workspace, sms, static_cast<cudaStream_t>(stream)));
}

gdn_status kv4_copy_pages(uint8_t *pages, int n_layers, int64_t layer_stride, int num_pages, int64_t page_bytes,
                          const int32_t *src, const int32_t *dst, int n, int32_t *dev_status, void *stream) {
  Kv4PageArgs a{};
  a.pages = pages;
  a.layers = n_layers;
  a.num_pages = num_pages;
  a.layer_stride = layer_stride;
  a.page_bytes = page_bytes;
  a.src = src;
  a.dst = dst;
  a.n = n;
  a.status = dev_status;
  gdn_status st = check_pages(a);
  if (st != GDN_OK || n == 0) return st;
  if (!src || !dst) return GDN_E_NULL;
  if ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 3u) return GDN_E_ALIGN;
  return cuda_status(launch_kv4_copy_pages(a, static_cast<cudaStream_t>(stream)));
}

size_t kv4_compact_workspace(int num_pages) { return num_pages > 0 ? kv4_compact_bytes(num_pages) : 0; }

gdn_status kv4_compact(uint8_t *pages, int n_layers, int64_t layer_stride, int num_pages, int64_t page_bytes,
                       const int32_t *block_table, int rows, int cols, int32_t *tables_out, int32_t *page_map,
                       int32_t *n_live, void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
  Kv4PageArgs a{};
  a.pages = pages;
  a.layers = n_layers;
  a.num_pages = num_pages;
  a.layer_stride = layer_stride;
  a.page_bytes = page_bytes;
  a.table = block_table;
  a.rows = rows;
  a.cols = cols;
  a.tables_out = tables_out;
  a.page_map = page_map;
  a.n_live = n_live;
  a.workspace = workspace;
  a.status = dev_status;
  gdn_status st = check_pages(a);
  if (st != GDN_OK) return st;
  if (num_pages > (1 << 20) || rows < 0 || cols < 0) return GDN_E_SHAPE;
  if ((long long)rows * cols > 0x7fffffffLL) return GDN_E_OVERFLOW;
  if (!page_map || !n_live || !workspace || ((long long)rows * cols > 0 && (!block_table || !tables_out)))
    return GDN_E_NULL;
  if (workspace_bytes < kv4_compact_bytes(num_pages)) return GDN_E_SHAPE;
  const uintptr_t words = reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(tables_out) |
                          reinterpret_cast<uintptr_t>(page_map) | reinterpret_cast<uintptr_t>(n_live);
  if ((words & 3u) || !aligned16(workspace))
    return GDN_E_ALIGN;
  return cuda_status(launch_kv4_compact(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
