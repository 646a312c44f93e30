// The C ABI of the 4-bit KV cache (include/gdn.h): argument checks, then one
// launcher per call.
#include <cmath>
#include <initializer_list>

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

bool words(std::initializer_list<const void *> ps) {
  uintptr_t all = 0;
  for (const void *p : ps) all |= reinterpret_cast<uintptr_t>(p);
  return (all & 3u) == 0;
}

// The sequences of a batch whose rows do not matter (or may be none).
gdn_status check_seqs(const kv4_cache *c, const kv4_batch *b, Kv4Args &a, int32_t *status) {
  if (!b) return GDN_E_NULL;
  kv4_batch one = *b;
  one.T = b->B > 0 ? b->B : 0;
  one.q_start = nullptr;
  return check(c, &one, a, status);
}

// Shared decode, scores and eviction step past a sequence's last token, or a row's last kept place, by a block's
// stride at most before they stop: what is longer than this their 31-bit places cannot count.
constexpr long long kMostTokens = 0x7fffffffLL - (1 << 15);
long long table_tokens(const Kv4Args &a) { return (long long)a.cols * a.page_tokens; }

// The score rows of n_layers layers, `stride` floats apart.
gdn_status check_scores(const kv4_cache *c, const kv4_scores *s, int n_layers, int64_t stride, Kv4ScoreRows &r) {
  if (!s) return GDN_E_NULL;
  if (s->n_slots < 0 || s->tokens < 0) return GDN_E_SHAPE;
  const long long row = (long long)c->n_kv_heads * s->tokens;  // below 2^42
  if (s->n_slots > 0 && row > (1LL << 44) / s->n_slots) return GDN_E_OVERFLOW;
  const long long layer = row * s->n_slots;
  if (n_layers > 1 && stride < layer) return GDN_E_SHAPE;
  if (layer > 0) {
    if (!s->in || !s->out) return GDN_E_NULL;
    if (!words({s->in, s->out, s->slots})) return GDN_E_ALIGN;
    if (n_layers > 1 && stride > (1LL << 58) / n_layers) return GDN_E_OVERFLOW;
    const uintptr_t x = reinterpret_cast<uintptr_t>(s->in), y = reinterpret_cast<uintptr_t>(s->out);
    const uintptr_t size = 4 * (uintptr_t)((n_layers - 1) * stride + layer);
    if (x != y && (x < y ? y - x : x - y) < size) return GDN_E_SHAPE;
  }
  r = Kv4ScoreRows{s->in, s->out, s->slots, s->n_slots, s->tokens};
  return GDN_OK;
}

gdn_status check_shared(const kv4_shared *s, int Hq, Kv4SharedArgs &a) {
  if (!s) return GDN_E_NULL;
  if (s->groups < 0 || s->max_shared < 0) return GDN_E_SHAPE;
  if (s->groups > 0 && (!s->group_start || !s->shared_len)) return GDN_E_NULL;
  if (s->groups > 0 && !words({s->group_start, s->shared_len})) return GDN_E_ALIGN;
  if (table_tokens(a.a.c) > kMostTokens) return GDN_E_OVERFLOW;
  if ((long long)a.a.c.T * Hq + s->groups > 0x7ffffff0LL) return GDN_E_OVERFLOW;  // T is B or more
  a.group_start = s->group_start;
  a.shared_len = s->shared_len;
  a.groups = s->groups;
  a.max_shared = s->max_shared;
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

// 0 for arguments that kv4_decode_shared refuses.
size_t kv4_decode_shared_workspace(const kv4_cache *c, const kv4_batch *b, const kv4_shared *s, int n_q_heads) {
  Kv4SharedArgs a{};
  if (check(c, b, a.a.c, nullptr) != GDN_OK || b->T == 0 || b->q_start || !heads_fit(c, n_q_heads)) return 0;
  if (check_shared(s, n_q_heads, a) != GDN_OK) return 0;
  a.a.Hq = n_q_heads;
  return kv4_decode_shared_bytes(a, kMaxSms);
}

gdn_status kv4_decode_shared(const kv4_cache *c, const kv4_batch *b, const kv4_shared *s, const uint16_t *q,
                             int64_t q_stride, int n_q_heads, float sm_scale, uint16_t *out, float *lse,
                             void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
  Kv4SharedArgs a{};
  gdn_status st = check_attn(c, b, q, q_stride, n_q_heads, sm_scale, out, lse, dev_status, a.a);
  if (st != GDN_OK) return st;
  if (b->q_start) return GDN_E_SHAPE;
  st = check_shared(s, n_q_heads, a);
  if (st != GDN_OK || b->T == 0) return st;
  const size_t need = kv4_decode_shared_bytes(a, kMaxSms);
  if (!workspace) return GDN_E_NULL;
  if (workspace_bytes < need) return GDN_E_SHAPE;
  if (!aligned16(workspace)) return GDN_E_ALIGN;
  const int sms = num_sms();
  if (sms < 1) return GDN_E_CUDA;
  return cuda_status(
      launch_kv4_decode_shared(a, workspace, sms < kMaxSms ? sms : kMaxSms, static_cast<cudaStream_t>(stream)));
}

// 0 where none is needed, and for arguments that kv4_score refuses.
size_t kv4_score_workspace(const kv4_cache *c, const kv4_batch *b, int n_q_heads) {
  Kv4ScoreArgs a{};
  if (check(c, b, a.c, nullptr) != GDN_OK || b->T == 0 || !heads_fit(c, n_q_heads)) return 0;
  a.Hq = n_q_heads;
  return kv4_score_bytes(a, kMaxSms);
}

gdn_status kv4_score(const kv4_cache *c, const kv4_batch *b, const uint16_t *q, int64_t q_stride, int n_q_heads,
                     float sm_scale, const float *lse, const kv4_scores *s, const int32_t *scored, void *workspace,
                     size_t workspace_bytes, int32_t *dev_status, void *stream) {
  Kv4ScoreArgs a{};
  gdn_status st = check_seqs(c, b, a.c, dev_status);
  if (st == GDN_OK) st = check(c, b, a.c, dev_status);
  if (st != GDN_OK) return st;
  if (!heads_fit(c, n_q_heads)) return GDN_E_SHAPE;
  if (!std::isfinite(sm_scale)) return GDN_E_NONFINITE;
  if (!(sm_scale > 0.0f)) return GDN_E_BAD_SCALE;
  st = check_scores(c, s, 1, 0, a.s);
  if (st != GDN_OK) return st;
  if (b->T > 0) {
    if (!q || !lse) return GDN_E_NULL;
    if (!aligned16(q) || !words({lse})) return GDN_E_ALIGN;
    if (q_stride % 8 || q_stride < (int64_t)n_q_heads * c->head_dim) return GDN_E_SHAPE;
    if ((long long)b->T * n_q_heads > 0x7fffffffLL) return GDN_E_OVERFLOW;
  }
  if (!words({scored})) return GDN_E_ALIGN;
  if (b->B == 0 || b->max_pages == 0 || s->n_slots == 0) return GDN_OK;
  if (table_tokens(a.c) > kMostTokens) return GDN_E_OVERFLOW;
  // a CTA per so many tokens of a sequence and head
  if (((long long)b->max_pages * c->page_tokens / 128 + 1) * b->B > 0x7fffffffLL / c->n_kv_heads) return GDN_E_OVERFLOW;
  a.q = q;
  a.q_stride = q_stride;
  a.Hq = n_q_heads;
  a.sm_scale = sm_scale;
  a.lse = lse;
  a.scored = scored;
  const size_t need = b->T > 0 ? kv4_score_bytes(a, kMaxSms) : 0;
  if (need && !workspace) return GDN_E_NULL;
  if (workspace_bytes < need) return GDN_E_SHAPE;
  if (!aligned16(workspace)) return GDN_E_ALIGN;
  const int sms = num_sms();
  if (sms < 1) return GDN_E_CUDA;
  return cuda_status(launch_kv4_score(a, workspace, sms < kMaxSms ? sms : kMaxSms, static_cast<cudaStream_t>(stream)));
}

gdn_status kv4_evict(const kv4_cache *c, int n_layers, int64_t layer_stride, const kv4_batch *b, const int32_t *keep,
                     int recent, const kv4_scores *s, int64_t score_stride, const int32_t *new_table, int new_pages,
                     int32_t *kept, int max_keep, int32_t *new_len, int32_t *dev_status, void *stream) {
  Kv4EvictArgs a{};
  gdn_status st = check_seqs(c, b, a.c, dev_status);
  if (st != GDN_OK) return st;
  if (n_layers < 1 || recent < 0 || new_pages < 0 || max_keep < 0) return GDN_E_SHAPE;
  const int64_t page_bytes = (int64_t)c->n_kv_heads * (c->page_tokens / 16) * 18 * c->head_dim;
  if (page_bytes > (1LL << 40) / c->num_pages) return GDN_E_OVERFLOW;
  if (n_layers > 1 && (layer_stride % 16 || layer_stride < c->num_pages * page_bytes)) return GDN_E_SHAPE;
  st = check_scores(c, s, n_layers, score_stride, a.s);
  if (st != GDN_OK || b->B == 0) return st;
  if (!keep || !new_len || (max_keep > 0 && !kept) || (new_pages > 0 && !new_table)) return GDN_E_NULL;
  if (!words({keep, new_len, kept, new_table})) return GDN_E_ALIGN;
  if (max_keep > kMostTokens || (table_tokens(a.c) > kMostTokens && s->tokens > kMostTokens)) return GDN_E_OVERFLOW;
  const long long rows = (long long)b->B * c->n_kv_heads;
  // up to 16 CTAs choose for a row, one moves 128 of its tokens
  if (rows > 0x7fffffffLL / 16 / n_layers || rows * n_layers > 0x7fffffffLL / (max_keep / 128 + 1)) return GDN_E_OVERFLOW;
  a.layers = n_layers;
  a.layer_stride = layer_stride;
  a.score_layer = score_stride;
  a.keep = keep;
  a.recent = recent;
  a.new_table = new_table;
  a.new_cols = new_pages;
  a.kept = kept;
  a.new_len = new_len;
  a.max_keep = max_keep;
  return cuda_status(launch_kv4_evict(a, static_cast<cudaStream_t>(stream)));
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
