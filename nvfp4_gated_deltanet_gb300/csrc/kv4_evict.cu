// Eviction by accumulated attention weight (include/gdn.h): of each KV head's n
// tokens the newest r stay, and of the others the k - r of the highest scores;
// they move to new pages in order, and their scores with them.
//
// What bounds it: the bytes. The scores are read once and written once, and a
// kept token-head's 9/8 d bytes are read and written.
#include <algorithm>

#include "kv4.cuh"

namespace gdn {

namespace {

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
template <int THREADS>
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
  unsigned x = lane < THREADS / 32 ? sums[lane] : 0u;  // every warp for itself: no second barrier
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  total = __shfl_sync(0xffffffffu, x, 31);
  const unsigned before = __shfl_sync(0xffffffffu, x, max(warp - 1, 0));
  __syncthreads();
  return incl - v + (warp ? before : 0u);
}

// ---------------------------------------------------------------- the choice
// A CTA, or a cluster of them, per (layer, sequence, KV head); a CTA holds its
// slice of the row in shared memory and the tokens' orders in registers, so that
// the row is read once (and may be overwritten once all have read). The lowest
// order that is kept is found in passes that split its range into bins, first from
// the least order to the greatest. (Bins of the leading bits put the scores' few
// exponents into few bins, whose counters the lanes of a warp then wait for.) A
// cluster adds its CTAs' counts up a share of the bins each: remote loads take a
// warp about 34 cycles each, and every CTA reading all counts took 35000 cycles a
// pass. Then the kept tokens' places follow from prefix counts, in order: a warp
// has neighbouring tokens, counts them, and after one barrier writes them.
// Bound by instructions and by the passes' barriers (512 rows of up to
// 8190: 23.0 us, issue 67% busy; 4 rows of 200001, sixteen CTAs each: 26.3).
constexpr int kMaxHeld = 48 * 1024;   // tokens that shared memory holds beside the counts
constexpr int kSplit = 4096;          // where SMs are idle, a CTA's slice is halved down to this

GDN_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
GDN_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// The word at `p` of this CTA's shared memory, in CTA `rank` of the cluster
GDN_DEV unsigned cluster_load(const unsigned *p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// E: a thread's tokens, whose orders are in registers; 0: any number, worked out
// in each pass. HELD: the slice is in shared memory; without, it is read again
// each time (one CTA, which overwrites only what it has read).
template <int THREADS, int CS, int E, bool HELD>
__global__ void __launch_bounds__(THREADS) kv4_select_kernel(Kv4EvictArgs p) {
  static_assert(HELD || (CS == 1 && E == 0), "a CTA overwrites only what it has read");
  // (one CTA, 11 bits for all: 1152 rows of up to 1501 46.5 us for choice and move instead of 45.7, 512 of up to 8190
  // 74.5 instead of 73.2, 1296 of 27 15.2 instead of 12.8)
  constexpr int BITS = CS > 1 ? 8 : E == 0 ? 11 : E == 16 ? 9 : 8, BINS = 1 << BITS;
  constexpr int PER = BINS > THREADS ? BINS / THREADS : 1, WARPS = THREADS / 32;
  static_assert(CS == 1 || PER == 1);
  constexpr int SHARE = CS > 1 ? BINS / CS : 1;  // bins whose counts a CTA of the cluster adds up
  extern __shared__ __align__(16) float held[];  // the slice's scores
  __shared__ __align__(16) unsigned hist[2][BINS];
  __shared__ unsigned gathered[2][SHARE], sums[33], range[2][32], ext[2], mine[2], found[3];
  kv4_begin();
  const Kv4Args &c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CS > 1 ? (int)cluster_rank() : 0, row_id = blockIdx.x / CS;
  const int h = row_id % c.Hkv, b = row_id / c.Hkv % c.B, l = row_id / c.Hkv / c.B;
  Evictee e = evictee(p, b);
  const size_t row = (size_t)l * p.score_layer + ((size_t)max(e.slot, 0) * c.Hkv + h) * p.s.tokens;
  const float *in = p.s.in + row;
  float *out = p.s.out + row;
  if (e.slot < 0) e.n = e.k = 0;
  const int n = e.n, k = e.k, r = min(p.recent, k), m = n - r;  // m tokens compete for k - r places
  const int slice = (n + CS - 1) / CS, i0 = min(n, rank * slice), len = min(n - i0, slice);  // this CTA's tokens
  const int rivals = max(0, min(len, m - i0));                                               // of them, those that compete
  // a warp has `part` neighbours, of which this lane takes every 32nd
  const int part = (len + THREADS - 1) / THREADS * 32, w0 = min(len, warp * part), w1 = min(len, w0 + part);
  float f[E > 0 ? E : 1];
  if constexpr (E > 0) {
#pragma unroll
    for (int x = 0; x < E; ++x) f[x] = w0 + x * 32 + lane < w1 ? in[i0 + w0 + x * 32 + lane] : 0.0f;
  }
  if (p.s.slots && e.slot >= 0) {  // a slot that another sequence has too: both are left out
    int twice = 0;
    for (int i = tid; i < c.B; i += THREADS) twice |= i != b && p.s.slots[i] == e.slot;
    if (__syncthreads_or(twice)) {
      flag_status(c.status, GDN_E_RANGE);
      e.slot = -1;
    }
  }
  int32_t *kept = p.kept + (size_t)row_id * p.max_keep;
  if (h == 0 && l == 0 && tid == 0 && rank == 0) p.new_len[b] = e.slot < 0 ? -1 : k;
  if (e.slot < 0) {  // all CTAs of the cluster alike
    for (int i = rank * THREADS + tid; i < p.max_keep; i += CS * THREADS) kept[i] = -1;
    return;
  }
  for (int x = tid; x < BINS; x += THREADS) hist[0][x] = 0;
  auto score = [&](int i) { return HELD ? held[i] : in[i0 + i]; };
  // ---- read: the least and the greatest order of the tokens that compete
  uint32_t lo = ~0u, hi = 0u, o[E > 0 ? E : 1];
  if constexpr (E > 0) {
#pragma unroll
    for (int x = 0; x < E; ++x) {
      const int i = w0 + x * 32 + lane;
      if (i < w1) held[i] = f[x];
      const bool rival = i < min(w1, rivals);
      o[x] = rival ? order_of(f[x]) : 0u;  // 0 is never above what is kept
      lo = min(lo, rival ? o[x] : ~0u);
      hi = max(hi, o[x]);
    }
  } else {
    for (int i = tid; i < len; i += THREADS) {
      const float f = in[i0 + i];
      if (HELD) held[i] = f;
      if (i < rivals) {
        lo = min(lo, order_of(f));
        hi = max(hi, order_of(f));
      }
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    range[0][warp] = lo;
    range[1][warp] = hi;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < WARPS ? range[0][lane] : ~0u);
  hi = __reduce_max_sync(0xffffffffu, lane < WARPS ? range[1][lane] : 0u);
  if (CS > 1) {
    if (tid == 0) {
      ext[0] = lo;
      ext[1] = hi;
    }
    cluster_sync();  // (also: everybody has read the row)
    lo = __reduce_min_sync(0xffffffffu, cluster_load(&ext[0], lane % CS));
    hi = __reduce_max_sync(0xffffffffu, cluster_load(&ext[1], lane % CS));
  }
  // ---- the lowest order that is kept: of the tokens in [low, low + 2^width) the need-th from the top
  uint32_t low = lo;
  unsigned need = k - r;
  const bool some = need > 0;
  int width = 32, shift = hi > lo ? max(0, 32 - __clz(hi - lo) - BITS) : 0;
  for (int pass = 0; some; ++pass) {
    unsigned *cnt = hist[pass & 1];
    unsigned first = 0;  // tokens in the lowest bin: many scores are equal where attention never looked
    const uint32_t last = width >= 32 ? ~0u : (1u << width) - 1u;
    auto count = [&](uint32_t x) {
      const uint32_t t = x - low;
      if (x >= low && t <= last) {
        if ((t >> shift) == 0) ++first;
        else atomicAdd(&cnt[t >> shift], 1u);
      }
    };
    if constexpr (E > 0) {
      // (one that does not compete is an order of 0: where that is in a bin at all it is the lowest one, whose count
      // then is too large for an early end, and for nothing else)
#pragma unroll
      for (int x = 0; x < E; ++x) count(o[x]);
    } else {
      for (int i = tid; i < rivals; i += THREADS) count(order_of(score(i)));
    }
    first = __reduce_add_sync(0xffffffffu, first);
    if (lane == 0 && first) atomicAdd(&cnt[0], first);
    // the other counts are cleared for the next pass (everybody has read them: the last pass's barriers)
    for (int x = tid; x < BINS; x += THREADS) hist[(pass & 1) ^ 1][x] = 0;
    unsigned v[PER], sum = 0, total;
    if constexpr (CS > 1) {
      cluster_sync();
      if (tid < BINS) {  // thread: bin rank SHARE + tid / CS of CTA tid % CS
        unsigned x = cluster_load(&cnt[rank * SHARE + tid / CS], tid % CS);
#pragma unroll
        for (int d = 1; d < CS; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (tid % CS == 0) gathered[pass & 1][tid / CS] = x;
      }
      cluster_sync();
      const int bin = BINS - 1 - tid;  // from the top
      v[0] = tid < BINS ? cluster_load(&gathered[pass & 1][bin % SHARE], bin / SHARE) : 0u;
      sum = v[0];
    } else {
      __syncthreads();
      constexpr int W = PER % 4 == 0 ? 4 : PER;  // words of a load
#pragma unroll
      for (int x = 0; x < PER; x += W) {
        const unsigned *at = cnt + max(BINS - (tid * PER + x) - W, 0);
        if constexpr (W == 4) {
          const uint4 y = *reinterpret_cast<const uint4 *>(at);
          v[x] = y.w, v[x + 1] = y.z, v[x + 2] = y.y, v[x + 3] = y.x;
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) v[x + e] = at[W - 1 - e];
        }
#pragma unroll
        for (int e = 0; e < W; ++e) sum += v[x + e] = PER * tid < BINS ? v[x + e] : 0u;  // (more threads than bins)
      }
    }
    // bin x holds the place `need` when the bins above it hold fewer than `need` and with it at least as many
    unsigned before = block_before<THREADS>(sum, sums, total);
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      if (before < need && before + v[x] >= need) {
        found[0] = BINS - 1 - (tid * PER + x);
        found[1] = before;
        found[2] = v[x];
      }
      before += v[x];
    }
    __syncthreads();
    low += found[0] << shift;
    need -= found[1];
    if (shift == 0) break;
    if (found[2] == need && low > 0) {  // the whole bin is kept
      --low;
      need = 0;
      break;
    }
    width = shift;
    shift = max(0, shift - BITS);
    __syncthreads();  // everybody has read `found`, and (one CTA) the counts
  }
  // ---- in order: the tokens above low, the first `need` of those at it, the newest
  auto kinds = [&](int j, uint32_t x, unsigned &over, unsigned &same) {  // of the 32 tokens from j, this lane's order being x
    const bool in_m = some && j + lane < min(w1, rivals);
    over = __ballot_sync(0xffffffffu, in_m && x > low);
    same = __ballot_sync(0xffffffffu, in_m && x == low);
  };
  unsigned above = 0, at = 0;
  if constexpr (E > 0) {
#pragma unroll
    for (int x = 0; x < E; ++x) above += some && o[x] > low;
    above = __reduce_add_sync(0xffffffffu, above);
    if (need > 0) {
#pragma unroll
      for (int x = 0; x < E; ++x) at += o[x] == low && w0 + x * 32 + lane < min(w1, rivals);
      at = __reduce_add_sync(0xffffffffu, at);
    }
  } else if (HELD) {
    for (int j = w0; j < w1; j += 32) {
      unsigned over, same;
      kinds(j, j + lane < w1 ? order_of(held[j + lane]) : 0u, over, same);
      above += __popc(over);
      at += __popc(same);
    }
  }
  unsigned a_all, t_all;
  if constexpr (E > 0) {  // a slice has fewer than 2^16 tokens
    static_assert(THREADS * E < 65536);
    const unsigned both = __shfl_sync(0xffffffffu, block_before<THREADS>(lane == 0 ? above | at << 16 : 0u, sums, a_all), 0);
    above = both & 0xffffu;
    at = both >> 16;
    t_all = a_all >> 16;
    a_all &= 0xffffu;
  } else {
    const unsigned a0 = block_before<THREADS>(lane == 0 ? above : 0u, sums, a_all);
    const unsigned t0 = block_before<THREADS>(lane == 0 ? at : 0u, sums, t_all);
    above = __shfl_sync(0xffffffffu, a0, 0);
    at = __shfl_sync(0xffffffffu, t0, 0);
  }
  if (CS > 1) {
    if (tid == 0) {
      mine[0] = a_all;
      mine[1] = t_all;
    }
    cluster_sync();
    above += __reduce_add_sync(0xffffffffu, lane < rank ? cluster_load(&mine[0], lane) : 0u);
    at += __reduce_add_sync(0xffffffffu, lane < rank ? cluster_load(&mine[1], lane) : 0u);
  }
  auto write = [&](int j, uint32_t x) {
    unsigned over, same;
    kinds(j, x, over, same);
    const unsigned before = (1u << lane) - 1u, a = above + __popc(over & before), t = at + __popc(same & before);
    if ((over >> lane & 1) || ((same >> lane & 1) && t < need)) {
      const unsigned to = a + min(t, need);
      kept[to] = i0 + j + lane;
      out[to] = held[j + lane];
    }
    above += __popc(over);
    at += __popc(same);
  };
  if constexpr (E > 0) {
    if (!some) {
    } else if (need > 0) {
#pragma unroll
      for (int x = 0; x < E; ++x)
        if (w0 + x * 32 < w1) write(w0 + x * 32, o[x]);
    } else {  // none of those at low
#pragma unroll
      for (int x = 0; x < E; ++x) {
        const unsigned over = __ballot_sync(0xffffffffu, o[x] > low);
        if (o[x] > low) {
          const unsigned to = above + __popc(over & ((1u << lane) - 1u));
          kept[to] = i0 + w0 + x * 32 + lane;
          out[to] = held[w0 + x * 32 + lane];
        }
        above += __popc(over);
      }
    }
  } else if (HELD) {
    for (int j = w0; j < w1; j += 32) write(j, j + lane < w1 ? order_of(held[j + lane]) : 0u);
  } else {  // in steps of the block, each read by all before any of it is written
    above = at = 0;
    for (int j0 = 0; j0 < len; j0 += THREADS) {
      const int j = j0 + warp * 32;
      const float f = j + lane < len ? in[j + lane] : 0.0f;
      const uint32_t x = order_of(f);
      const bool in_m = some && j + lane < rivals;
      const unsigned over = __ballot_sync(0xffffffffu, in_m && x > low), same = __ballot_sync(0xffffffffu, in_m && x == low);
      unsigned all;
      const unsigned b4 = block_before<THREADS>(lane == 0 ? (unsigned)__popc(over) | (unsigned)__popc(same) << 16 : 0u, sums, all);
      const unsigned first = __shfl_sync(0xffffffffu, b4, 0), keep_a = above, keep_t = at;
      above += first & 0xffffu;
      at += first >> 16;
      const int i = j + lane;
      const unsigned before = (1u << lane) - 1u, a = above + __popc(over & before), t = at + __popc(same & before);
      int to = -1;
      if ((over >> lane & 1) || ((same >> lane & 1) && t < need)) to = (int)(a + min(t, need));
      else if (i < len && i >= m) to = k - r + (i - m);
      if (to >= 0) {
        kept[to] = i;
        out[to] = f;
      }
      above = keep_a + (all & 0xffffu);
      at = keep_t + (all >> 16);
    }
    __syncthreads();
  }
  if (HELD)  // the newest
    for (int i = rivals + tid; i < len; i += THREADS) {
      kept[k - r + (i0 + i - m)] = i0 + i;
      out[k - r + (i0 + i - m)] = held[i];
    }
  for (int i = k + rank * THREADS + tid; i < n; i += CS * THREADS) out[i] = 0.0f;
  for (int i = k + rank * THREADS + tid; i < p.max_keep; i += CS * THREADS) kept[i] = -1;
  if (CS > 1) cluster_sync();  // nobody leaves while its counts are read
}

// ---------------------------------------------------------------- the move
// A warp per group of 16 kept tokens of a (layer, sequence, KV head): from where
// they lie into the new pages, with zeros where the last group has no token.
// Bound by the bytes, and by a chain of three loads before them (the kept places,
// the page table, the bytes) that many warps hide.
template <int D>
__global__ void __launch_bounds__(256) kv4_move_kernel(Kv4EvictArgs p) {
  kv4_begin();
  const Kv4Args &c = p.c;
  const int lane = threadIdx.x & 31;
  const int chunks = (p.max_keep + 127) / 128, row = blockIdx.x / chunks;
  const int h = row % c.Hkv, b = row / c.Hkv % c.B, l = row / c.Hkv / c.B;
  const int group = blockIdx.x % chunks * 8 + (threadIdx.x >> 5);
  // lane t < 16 (and t + 16): token t
  const int place = group * 16 + (lane & 15), col = group * 16 / c.page_tokens;
  const int k = p.new_len[b];
  const int pos = place < p.max_keep ? p.kept[(size_t)row * p.max_keep + place] : -1;
  const int page = col < p.new_cols ? p.new_table[(size_t)b * p.new_cols + col] : -1;
  if (group * 16 >= k) return;  // (k < 0: left out)
  if (page < 0 || page >= c.num_pages) {
    flag_status(c.status, GDN_E_RANGE);
    return;
  }
  const long long layer = l * p.layer_stride;
  const uint8_t *src = nullptr;
  const int st = pos & 15;
  if (place < k) {
    const uint8_t *g = kv4_group<D>(c, b, pos);
    if (g) src = g + layer + h * kv4_head_bytes<D>(c);
  }
  uint8_t *dst = c.pages + layer + ((size_t)page * c.Hkv * (c.page_tokens / 16) + group * 16 % c.page_tokens / 16) * (18 * D) +
                 h * kv4_head_bytes<D>(c);
  constexpr int P = D / 32, Q = P / 2;  // 16-byte pieces of a token's codes; of those that a lane moves
  uint4 x[2][Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int t = (q * 32 + lane) / P, i = lane % P * 16;
    const int s = __shfl_sync(0xffffffffu, st, t);
    const uint8_t *g = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), t));
    x[0][q] = g ? *reinterpret_cast<const uint4 *>(g + kv4_k_code<D>(s, i)) : make_uint4(0, 0, 0, 0);
    x[1][q] = g ? *reinterpret_cast<const uint4 *>(g + kv4_v_code<D>(s, i)) : make_uint4(0, 0, 0, 0);
  }
  // scales: lanes t and t + 16 take half of token t's blocks each
  constexpr int H = D / 32;
  const int t = lane & 15, b0 = (lane >> 4) * H;
  uint8_t ks[H], vs[H];
#pragma unroll
  for (int i = 0; i < H; ++i) {
    ks[i] = src ? src[kv4_k_scale<D>(st, b0 + i)] : (uint8_t)0;
    vs[i] = src ? src[kv4_v_scale<D>(st, b0 + i)] : (uint8_t)0;
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int t2 = (q * 32 + lane) / P, i = lane % P * 16;
    *reinterpret_cast<uint4 *>(dst + kv4_k_code<D>(t2, i)) = x[0][q];
    *reinterpret_cast<uint4 *>(dst + kv4_v_code<D>(t2, i)) = x[1][q];
  }
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < H; ++i) {
    word |= (uint32_t)ks[i] << (8 * i);
    dst[kv4_v_scale<D>(t, b0 + i)] = vs[i];
  }
  if (D == 128) *reinterpret_cast<uint32_t *>(dst + kv4_k_scale<D>(t, b0)) = word;
  else *reinterpret_cast<uint16_t *>(dst + kv4_k_scale<D>(t, b0)) = (uint16_t)word;
}

template <int THREADS, int CS, int E, bool HELD = true>
cudaError_t launch_select(const Kv4EvictArgs &p, int slice, cudaStream_t stream) {
  static bool allowed[64];
  const auto kernel = kv4_select_kernel<THREADS, CS, E, HELD>;
  cudaError_t e = kv4_allow_smem(kernel, HELD ? 4 * (E ? THREADS * E : kMaxHeld) : 0, allowed, CS > 8);
  if (e != cudaSuccess) return e;
  return kv4_launch_cluster(kernel, (unsigned)(p.layers * p.c.B * p.c.Hkv) * CS, CS, THREADS, HELD ? 4 * (size_t)slice : 0,
                            stream, p);
}

}  // namespace

cudaError_t launch_kv4_evict(const Kv4EvictArgs &p, cudaStream_t stream) {
  const Kv4Args &c = p.c;
  const long long rows = (long long)p.layers * c.B * c.Hkv;
  const int most = (int)std::min((long long)p.s.tokens, (long long)c.cols * c.page_tokens);  // tokens of a row
  // CTAs of a row: as many as registers need, and while SMs are idle and the slices long
  int cs = 1;
  while (cs < 16 && ((most + cs - 1) / cs > 16384 || (most / cs > kSplit && rows * cs < 152))) cs *= 2;
  const int slice = (most + cs - 1) / cs;
  cudaError_t e;
  if (slice > kMaxHeld) e = launch_select<1024, 1, 0, false>(p, 0, stream);
  else if (slice > 16384) e = launch_select<1024, 16, 0>(p, slice, stream);
  else if (cs == 16) e = launch_select<1024, 16, 16>(p, slice, stream);
  else if (cs == 8) e = launch_select<1024, 8, 16>(p, slice, stream);
  else if (cs == 4) e = launch_select<1024, 4, 16>(p, slice, stream);
  else if (cs == 2) e = launch_select<1024, 2, 16>(p, slice, stream);
  else if (slice > 8192) e = launch_select<1024, 1, 16>(p, slice, stream);
  else if (slice > 4096) e = launch_select<512, 1, 16>(p, slice, stream);
  else if (slice > 2048) e = launch_select<256, 1, 16>(p, slice, stream);
  else if (slice > 1024) e = launch_select<256, 1, 8>(p, slice, stream);
  else e = launch_select<256, 1, 4>(p, slice, stream);
  if (e != cudaSuccess || p.max_keep == 0) return e;
  const unsigned grid = (unsigned)((p.max_keep + 127) / 128) * c.B * c.Hkv * p.layers;
  return kv4_launch(c.D == 128 ? kv4_move_kernel<128> : kv4_move_kernel<64>, grid, 256, 0, stream, p);
}

}  // namespace gdn
