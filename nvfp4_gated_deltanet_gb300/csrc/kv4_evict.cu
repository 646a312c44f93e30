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
// A cluster of CTAs per (layer, sequence, KV head); a CTA holds the scores of its
// slice of the row in shared memory, so that the row is read once (and may be
// overwritten once all have read). The lowest order that is kept is found 11 bits
// at a time: each CTA counts its own, all read all counts. Then the kept tokens'
// places follow from prefix counts, in order.
// Bound by latency: three counting passes, a barrier of the cluster in each, and
// the row's one read.
constexpr int kBins = 2048;
constexpr int kMaxSlice = 48 * 1024;  // tokens whose scores fit beside the counts
constexpr int kSplit = 8192;          // where SMs are idle, a CTA's slice is halved down to this
constexpr int kShort = 4096;          // rows up to this take CTAs of 256 threads

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

// HELD: the row is in shared memory; without, it is read again in each pass (one CTA, any length).
template <int THREADS, int CS, bool HELD>
__global__ void __launch_bounds__(THREADS) kv4_select_kernel(Kv4EvictArgs p) {
  static_assert(HELD || CS == 1, "a CTA overwrites only what it has read");
  constexpr int PER = kBins / THREADS;
  extern __shared__ __align__(16) float held[];  // the slice's scores
  __shared__ unsigned hist[2][kBins], sums[33], mine[2];
  __shared__ unsigned found[2];
  kv4_begin();
  const Kv4Args &c = p.c;
  const int tid = threadIdx.x, rank = CS > 1 ? (int)cluster_rank() : 0, row_id = blockIdx.x / CS;
  const int h = row_id % c.Hkv, b = row_id / c.Hkv % c.B, l = row_id / c.Hkv / c.B;
  Evictee e = evictee(p, b);
  if (p.s.slots && e.slot >= 0) {  // a slot that another sequence has too: both are left out
    int twice = 0;
    for (int i = tid; i < c.B; i += THREADS) twice |= i != b && p.s.slots[i] == e.slot;
    if (__syncthreads_or(twice)) {
      flag_status(c.status, GDN_E_RANGE);
      e.slot = -1;
    }
  }
  int32_t *kept = p.kept + (size_t)row_id * p.max_keep;
  if (h == 0 && l == 0 && tid == 0 && rank == 0) p.new_len[b] = e.slot < 0 ? -1 : e.k;
  if (e.slot < 0) {  // all CTAs of the cluster alike
    for (int i = rank * THREADS + tid; i < p.max_keep; i += CS * THREADS) kept[i] = -1;
    return;
  }
  const size_t row = (size_t)l * p.score_layer + ((size_t)e.slot * c.Hkv + h) * p.s.tokens;
  const float *in = p.s.in + row;
  float *out = p.s.out + row;
  const int n = e.n, k = e.k, r = min(p.recent, k), m = n - r;  // m tokens compete for k - r places
  const int slice = (n + CS - 1) / CS, i0 = min(n, rank * slice), len = min(n - i0, slice);  // this CTA's tokens
  auto score = [&](int i) { return HELD ? held[i] : in[i]; };
  for (int x = tid; x < kBins; x += THREADS) hist[0][x] = 0;
  __syncthreads();
  // ---- read: orders kept, the first count beside it (tokens that compete: i0 + i < m)
#pragma unroll 4
  for (int i = tid; i < len; i += THREADS) {
    const float f = in[i0 + i];
    if (HELD) held[i] = f;
    if (i0 + i < m) atomicAdd(&hist[0][order_of(f) >> 21], 1u);
  }
  // ---- the lowest order that is kept
  uint32_t low = 0;
  unsigned need = k - r;  // places left for tokens whose higher bits are low's
  const bool some = need > 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    unsigned *cnt = hist[pass & 1];
    if (pass > 0) {
      if (some)
#pragma unroll 4
        for (int i = tid; i < len; i += THREADS) {
          const uint32_t o = order_of(score(i));
          if (i0 + i < m && (o >> (shift + bits)) == (low >> (shift + bits)))
            atomicAdd(&cnt[o >> shift & ((1 << bits) - 1)], 1u);
        }
    }
    // the other counts are cleared for the next pass (everybody has read them: a barrier of the last pass)
    if (pass < 2)
      for (int x = tid; x < kBins; x += THREADS) hist[(pass & 1) ^ 1][x] = 0;
    if (CS > 1) cluster_sync();
    else __syncthreads();
    // bins from the top: this thread's PER of them, summed over the cluster
    unsigned v[PER], sum = 0, total;
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const int bin = kBins - 1 - (tid * PER + x);
      v[x] = 0;
      if (CS > 1) {
#pragma unroll
        for (int y = 0; y < CS; ++y) v[x] += cluster_load(&cnt[bin], y);
      } else {
        v[x] = cnt[bin];
      }
      sum += v[x];
    }
    // bin x holds the place `need` when the bins above it hold fewer than `need` and with it at least as many
    unsigned before = block_before<THREADS>(sum, sums, total);
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      if (before < need && before + v[x] >= need) {
        found[0] = kBins - 1 - (tid * PER + x);
        found[1] = before;
      }
      before += v[x];
    }
    __syncthreads();
    if (some) {
      low |= found[0] << shift;
      need -= found[1];
    }
    if (CS > 1) cluster_sync();  // everybody has read these counts
    else __syncthreads();
  }
  // ---- this slice's tokens above low and at it, and those of the slices before
  unsigned above = 0, at = 0;
  if (CS > 1) {
    unsigned a = 0, s = 0;
    for (int i = tid; i < len; i += THREADS) {
      const uint32_t o = order_of(score(i));
      a += i0 + i < m && o > low;
      s += i0 + i < m && o == low;
    }
    unsigned ta, ts;
    block_before<THREADS>(a, sums, ta);
    block_before<THREADS>(s, sums, ts);
    if (tid == 0) {
      mine[0] = ta;
      mine[1] = ts;
    }
    cluster_sync();
    for (int y = 0; y < rank; ++y) {
      above += cluster_load(&mine[0], y);
      at += cluster_load(&mine[1], y);
    }
  }
  // ---- in order: the tokens above low, the first `need` of those at it, the newest
  for (int j0 = 0; j0 < len; j0 += 4 * THREADS) {
    const int j = j0 + 4 * tid;
    float f[4];
    unsigned over = 0, same = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      f[x] = j + x < len ? score(j + x) : 0.0f;
      const uint32_t o = order_of(f[x]);
      const bool in_m = some && j + x < len && i0 + j + x < m;
      over |= (unsigned)(in_m && o > low) << x;
      same |= (unsigned)(in_m && o == low) << x;
    }
    unsigned total;
    const unsigned before = block_before<THREADS>((unsigned)__popc(over) | (unsigned)__popc(same) << 16, sums, total);
    unsigned a = above + (before & 0xffffu), t = at + (before >> 16);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = i0 + j + x;
      const bool is_over = over >> x & 1, is_same = same >> x & 1;
      int to = -1;
      if (is_over || (is_same && t < need)) to = (int)(a + min(t, need));
      else if (j + x < len && i >= m) to = k - r + (i - m);
      a += is_over;
      t += is_same;
      if (to >= 0) {
        kept[to] = i;
        out[to] = f[x];
      }
    }
    above += total & 0xffffu;
    at += total >> 16;
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

template <int THREADS, int CS, bool HELD>
cudaError_t launch_select(const Kv4EvictArgs &p, int slice, cudaStream_t stream) {
  const size_t smem = HELD ? 4 * (size_t)slice : 0;
  static bool allowed[64];
  cudaError_t e = kv4_allow_smem(kv4_select_kernel<THREADS, CS, HELD>, HELD ? 4 * kMaxSlice : 0, allowed);
  if (e != cudaSuccess) return e;
  return kv4_launch_cluster(kv4_select_kernel<THREADS, CS, HELD>, (unsigned)(p.layers * p.c.B * p.c.Hkv) * CS, CS, THREADS,
                            smem, stream, p);
}

}  // namespace

cudaError_t launch_kv4_evict(const Kv4EvictArgs &p, cudaStream_t stream) {
  const Kv4Args &c = p.c;
  const long long rows = (long long)p.layers * c.B * c.Hkv;
  const int most = (int)std::min((long long)p.s.tokens, (long long)c.cols * c.page_tokens);  // tokens of a row
  int cs = 1;
  while (cs < 8 && ((most + cs - 1) / cs > kMaxSlice || (most / cs > kSplit && rows * cs < 152))) cs *= 2;
  const int slice = (most + cs - 1) / cs;
  cudaError_t e;
  if (slice > kMaxSlice) e = launch_select<1024, 1, false>(p, 0, stream);
  else if (cs == 8) e = launch_select<1024, 8, true>(p, slice, stream);
  else if (cs == 4) e = launch_select<1024, 4, true>(p, slice, stream);
  else if (cs == 2) e = launch_select<1024, 2, true>(p, slice, stream);
  else if (most > kShort) e = launch_select<1024, 1, true>(p, slice, stream);
  else e = launch_select<256, 1, true>(p, slice, stream);
  if (e != cudaSuccess || p.max_keep == 0) return e;
  const unsigned grid = (unsigned)((p.max_keep + 127) / 128) * c.B * c.Hkv * p.layers;
  return kv4_launch(c.D == 128 ? kv4_move_kernel<128> : kv4_move_kernel<64>, grid, 256, 0, stream, p);
}

}  // namespace gdn
