// Eviction by accumulated attention weight (include/gdn.h): of each KV head's n
// tokens the newest r stay, and of the others the k - r of the highest scores;
// they move to new pages in order, and their scores with them.
//
// What bounds it: the bytes. The scores are read once and written once, and a
// kept token-head's 9/8 d bytes are read and written.
#include "kv4.cuh"

namespace gdn {

namespace {

constexpr int kSelThreads = 1024;

// A score's place in the order, as an unsigned integer: NaN below everything,
// the two zeros equal.
GDN_DEV uint32_t order_of(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.0f);  // -0 + 0 = +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A sequence of the batch, checked.
struct Evictee {
  int n, k, slot;  // tokens, tokens to keep; slot < 0: left out
};
GDN_DEV Evictee evictee(const Kv4EvictArgs &p, int b) {
  const Kv4Args &c = p.c;
  Evictee e{c.kv_len[b], p.keep[b], p.s.slots ? p.s.slots[b] : b};
  const bool bad = e.n < 0 || e.n > (long long)c.cols * c.page_tokens || e.n > p.s.tokens || e.k < 0 ||
                   (min(e.k, e.n) > p.max_keep) || min(e.k, e.n) > (long long)p.new_cols * c.page_tokens ||
                   e.slot < -1 || e.slot >= p.s.n_slots;
  if (bad) {
    flag_status(c.status, GDN_E_RANGE);
    e.slot = -1;
  }
  e.k = min(e.k, e.n);
  return e;
}

// The sum of v over the block's threads before this one; total: of all of them.
// sums: 33 words of shared memory. All threads.
GDN_DEV unsigned block_before(unsigned v, unsigned *sums, unsigned &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    unsigned x = lane < (int)blockDim.x / 32 ? sums[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    sums[lane] = x;
  }
  __syncthreads();
  const unsigned before = incl - v + (warp ? sums[warp - 1] : 0u);
  total = sums[31];
  __syncthreads();
  return before;
}

// One CTA per (layer, sequence, KV head): the places of the kept tokens, in order,
// and their scores.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(Kv4EvictArgs p) {
  __shared__ unsigned hist[256], sums[33];
  __shared__ unsigned found[2];
  kv4_begin();
  const Kv4Args &c = p.c;
  const int tid = threadIdx.x;
  const int h = blockIdx.x % c.Hkv, b = blockIdx.x / c.Hkv % c.B, l = blockIdx.x / c.Hkv / c.B;
  Evictee e = evictee(p, b);
  if (p.s.slots && e.slot >= 0) {  // a slot that another sequence has too: both are left out
    int twice = 0;
    for (int i = tid; i < c.B; i += kSelThreads) twice |= i != b && p.s.slots[i] == e.slot;
    if (__syncthreads_or(twice)) {
      flag_status(c.status, GDN_E_RANGE);
      e.slot = -1;
    }
  }
  int32_t *kept = p.kept + (((size_t)l * c.B + b) * c.Hkv + h) * p.max_keep;
  if (h == 0 && l == 0 && tid == 0) p.new_len[b] = e.slot < 0 ? -1 : e.k;
  if (e.slot < 0) {
    for (int i = tid; i < p.max_keep; i += kSelThreads) kept[i] = -1;
    return;
  }
  const size_t row = (size_t)l * p.score_layer + ((size_t)e.slot * c.Hkv + h) * p.s.tokens;
  const float *in = p.s.in + row;
  float *out = p.s.out + row;
  const int n = e.n, k = e.k, r = min(p.recent, k), m = n - r;  // m tokens compete for k - r places
  // ---- the lowest order that is kept, 8 bits at a time
  uint32_t low = 0;
  unsigned need = k - r;  // places left for tokens whose higher bits are low's
  for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < m; i += kSelThreads) {
      const uint32_t o = order_of(in[i]);
      if (shift == 24 || (o >> (shift + 8)) == (low >> (shift + 8))) atomicAdd(&hist[o >> shift & 255], 1u);
    }
    __syncthreads();
    // bin x holds the place `need` when the bins above it hold fewer than `need` and with it at least as many
    unsigned total, v = tid < 256 ? hist[255 - tid] : 0u;
    const unsigned before = block_before(v, sums, total);
    if (tid < 256 && before < need && before + v >= need) {
      found[0] = 255 - tid;
      found[1] = before;
    }
    __syncthreads();
    low |= found[0] << shift;
    need -= found[1];
    __syncthreads();
  }
  // ---- in order: the tokens above low, the first `need` of those at it, the newest
  // (only tokens of a chunk that has been read are overwritten: a token moves to a place not past its own)
  const bool some = k - r > 0;
  unsigned above = 0, at = 0;  // of the chunks before
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const float f = i < n ? in[i] : 0.0f;
    const uint32_t o = order_of(f);
    const bool over = some && i < m && o > low, same = some && i < m && o == low;
    unsigned total;
    const unsigned before = block_before((unsigned)over | (unsigned)same << 16, sums, total);
    const unsigned a = above + (before & 0xffffu), t = at + (before >> 16);
    int to = -1;
    if (over || (same && t < need)) to = (int)(a + min(t, need));
    else if (i >= m && i < n) to = k - r + (i - m);
    if (to >= 0) {
      kept[to] = i;
      out[to] = f;
    }
    above += total & 0xffffu;
    at += total >> 16;
  }
  __syncthreads();
  for (int i = k + tid; i < n; i += kSelThreads) out[i] = 0.0f;
  for (int i = k + tid; i < p.max_keep; i += kSelThreads) kept[i] = -1;
}

// One warp per group of 16 kept tokens of a (layer, sequence, KV head): from where
// they lie into the new pages, with zeros where the last group has no token.
template <int D>
__global__ void __launch_bounds__(256) kv4_move_kernel(Kv4EvictArgs p) {
  kv4_begin();
  const Kv4Args &c = p.c;
  const int lane = threadIdx.x & 31;
  const int chunks = (p.max_keep + 127) / 128, row = blockIdx.x / chunks;
  const int h = row % c.Hkv, b = row / c.Hkv % c.B, l = row / c.Hkv / c.B;
  const int k = p.new_len[b];
  const int group = blockIdx.x % chunks * 8 + (threadIdx.x >> 5);
  if (group * 16 >= k) return;  // (k < 0: left out)
  const int32_t *kept = p.kept + (((size_t)l * c.B + b) * c.Hkv + h) * p.max_keep;
  const long long layer = l * p.layer_stride;
  // lane t < 16 (and t + 16): where token t lies
  const int place = group * 16 + (lane & 15);
  const uint8_t *src = nullptr;
  int st = 0;
  if (place < k) {
    const int pos = kept[place];
    const uint8_t *g = kv4_group<D>(c, b, pos);
    if (g) src = g + layer + h * kv4_head_bytes<D>(c);
    st = pos & 15;
  }
  const int page = p.new_table[(size_t)b * p.new_cols + group * 16 / c.page_tokens];
  if (page < 0 || page >= c.num_pages) {
    flag_status(c.status, GDN_E_RANGE);
    return;
  }
  uint8_t *dst = c.pages + layer + ((size_t)page * c.Hkv * (c.page_tokens / 16) + group * 16 % c.page_tokens / 16) * (18 * D) +
                 h * kv4_head_bytes<D>(c);
  auto from = [&](int t, int &s) {
    s = __shfl_sync(0xffffffffu, st, t);
    return reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), t));
  };
  constexpr int P = D / 32;  // 16-byte pieces of a token's codes
  uint4 x[2][16 * P / 32];
#pragma unroll
  for (int q = 0; q < 16 * P / 32; ++q) {
    const int t = (q * 32 + lane) / P, i = lane % P * 16;
    int s;
    const uint8_t *g = from(t, s);
    x[0][q] = g ? *reinterpret_cast<const uint4 *>(g + kv4_k_code<D>(s, i)) : make_uint4(0, 0, 0, 0);
    x[1][q] = g ? *reinterpret_cast<const uint4 *>(g + kv4_v_code<D>(s, i)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int q = 0; q < 16 * P / 32; ++q) {
    const int t = (q * 32 + lane) / P, i = lane % P * 16;
    *reinterpret_cast<uint4 *>(dst + kv4_k_code<D>(t, i)) = x[0][q];
    *reinterpret_cast<uint4 *>(dst + kv4_v_code<D>(t, i)) = x[1][q];
  }
  // scales: lane w writes word w of each (D = 64: lanes 0 .. 15)
  uint32_t ks = 0, vs = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = (lane * 4 + j) % D;  // d = 64: the upper lanes repeat the lower ones
    {  // K: token at / (D / 16), block at % (D / 16)
      const int t = at / (D / 16);
      int s;
      const uint8_t *g = from(t, s);
      if (g) ks |= (uint32_t)g[kv4_k_scale<D>(s, at % (D / 16))] << (8 * j);
    }
    {  // V: block at / 16, tokens 2 q, 2 q + 1, 2 q + 8, 2 q + 9 of word q
      const int t = 2 * (lane & 3) + (j & 1) + 8 * (j >> 1);
      int s;
      const uint8_t *g = from(t, s);
      if (g) vs |= (uint32_t)g[kv4_v_scale<D>(s, at / 16)] << (8 * j);
    }
  }
  if (lane * 4 >= D) return;
  reinterpret_cast<uint32_t *>(dst + 16 * D)[lane] = ks;
  reinterpret_cast<uint32_t *>(dst + 17 * D)[lane] = vs;
}

}  // namespace

cudaError_t launch_kv4_evict(const Kv4EvictArgs &p, cudaStream_t stream) {
  const Kv4Args &c = p.c;
  cudaError_t e = kv4_launch(kv4_select_kernel, (unsigned)(p.layers * c.B * c.Hkv), kSelThreads, 0, stream, p);
  if (e != cudaSuccess || p.max_keep == 0) return e;
  const unsigned grid = (unsigned)((p.max_keep + 127) / 128) * c.B * c.Hkv * p.layers;
  return kv4_launch(c.D == 128 ? kv4_move_kernel<128> : kv4_move_kernel<64>, grid, 256, 0, stream, p);
}

}  // namespace gdn
