// The 4-bit KV cache's data movement: new tokens into pages, tokens read back,
// pages copied and compacted.
#include "kv4.cuh"

namespace gdn {

namespace {

// New rows into their pages, or back: one CTA per 16-token group that the new
// rows touch and up to four heads (fewer where that leaves SMs idle). Bound by
// the bytes: per token, head and K or V, 2 d in BF16 and 9/16 d in 4 bits.
constexpr int kHeads = 4;

struct RowsArgs {
  Kv4Args a;
  uint16_t *k, *v;
  long long k_stride, v_stride;
  int heads;  // of a CTA
  int items;  // append: (group, chunk of heads) pairs at most
};
// A group's new tokens [t0, t1) of sequence b (-1: none); token t is row n0 + t.
// pos0 < 0: no tokens, rows of a batch that counts more new rows than the sequence has tokens.
struct Group {
  int b, pos0, t0, t1;
  long long n0;
};
// The x-th group that new rows touch, with ALL those before a sequence's start too. One warp.
template <bool ALL>
GDN_DEV Group find_group(const Kv4Args &a, int x, int lane) {
  Group r{-1, 0, 0, 0, 0};
  int base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    Kv4Seq s{0, 0, 0};
    int n = 0, lo = 0;
    if (b0 + lane < a.B) {
      s = kv4_seq(a, b0 + lane);
      lo = s.len - (s.q1 - s.q0);  // the first new token
      if (!ALL) lo = max(0, lo);
      n = s.q1 > s.q0 && s.len > lo ? ((s.len - 1) >> 4) - (lo >> 4) + 1 : 0;
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, base + incl > x);
    if (past) {
      const int l = __ffs(past) - 1;
      const int pos0 = ((lo >> 4) + x - (base + incl - n)) * 16;
      r.b = b0 + l;
      r.pos0 = __shfl_sync(0xffffffffu, pos0, l);
      r.t0 = __shfl_sync(0xffffffffu, max(0, lo - pos0), l);
      r.t1 = __shfl_sync(0xffffffffu, min(16, s.len - pos0), l);
      r.n0 = __shfl_sync(0xffffffffu, s.q1 - s.len + pos0, l);
      return r;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

GDN_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four pairs of floats -> eight E2M1 codes, the first in the lowest nibble
GDN_DEV uint32_t e2m1x8_from_f32(const float2 (&v)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return r;
}
GDN_DEV float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long *>(&r))
      : "l"(*reinterpret_cast<unsigned long long *>(&x)), "l"(*reinterpret_cast<unsigned long long *>(&y)));
  return r;
}
// quant_block16 of 16 BF16 values, the same steps two at a time (264 instructions a
// block with it): the largest magnitude as an integer maximum of the bits, NaN and
// infinity above all others.
GDN_DEV bool quant_bf16x16(const uint4 (&x)[2], float ts, float inv6ts, uint32_t (&codes)[2], uint32_t &scale) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_u16x2(m, w[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  codes[0] = codes[1] = scale = 0u;
  if (m >= 0x7F80u) return false;
  scale = e4m3_from_f32(__fmul_rn(__uint_as_float(m << 16), inv6ts));
  const float sv = e4m3_to_f32(scale);
  if (sv == 0.0f) return true;
  const float r = __frcp_rn(__fmul_rn(sv, ts));
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = mul2(make_float2(__uint_as_float(w[4 * k + i] << 16), __uint_as_float(w[4 * k + i] & 0xFFFF0000u)), make_float2(r, r));
    codes[k] = e2m1x8_from_f32(v);
  }
  return true;
}

// Append. A CTA goes through its groups with two buffers: while it quantises one
// group, a thread per 16-element block, the next one's rows come to shared memory
// (a token's heads lie together: one bulk copy per token, 32 KB a buffer, three
// CTAs an SM). Its warps find eight groups at once, one each: finding them one by
// one, a chain of three loads, took longer than the group itself. The scales are
// gathered in shared memory and leave as 16-byte words where all of the group's
// tokens are new: a V scale is a byte 16 bytes from its token's next one, and
// single bytes cost more memory transactions than all the codes.
// Bound by neither the bytes nor the issue slots (a block's 16 values: a maximum, a
// division, 16 products, 8 conversions; 51% of them used) but by the two barriers of
// a group, the largest stall: 22638 rows of 8 heads, d = 128, 93 MB read and 26
// written: 22.9 us in a graph, where the bytes take 17.5.
template <int D>
struct AppendSmem {
  uint16_t rows[2][2][16][kHeads * D];  // [buffer][K, V][token]
  uint8_t scales[kHeads * 2 * D];
  Group found[8];
  uint8_t *place[8];
  uint64_t landed[2];
  int gave_up;
};
template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(RowsArgs p) {
  constexpr int NB = D / 16, ITEMS = 2 * 16 * NB;  // of a head: K and V blocks of 16 tokens
  extern __shared__ __align__(128) unsigned char raw[];
  AppendSmem<D> &sm = *reinterpret_cast<AppendSmem<D> *>(raw);
  const Kv4Args &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int chunks = (a.Hkv + p.heads - 1) / p.heads;  // an item: a group, and a chunk of its heads
  if (tid == 0) {
    mbar_init(&sm.landed[0], 1);
    mbar_init(&sm.landed[1], 1);
    sm.gave_up = 0;
    fence_barrier_init();
  }
  kv4_begin();
  uint32_t armed = 0, turns = 0;  // bit `buf`: parity of the buffer's next fetch (thread 0), of its next wait
  auto fetch = [&](int item, int k, int buf) {  // warp 0: the rows of found[k]
    const Group r = sm.found[k];
    if (r.b < 0) return;
    const int h0 = item % chunks * p.heads, hn = min(p.heads, a.Hkv - h0);
    if (lane == 0) mbar_arrive_expect_tx(&sm.landed[buf], 2 * (r.t1 - r.t0) * hn * D * 2);
    armed ^= 1u << buf;
    __syncwarp();
    const int t = lane & 15;
    if (t >= r.t0 && t < r.t1)
      bulk_g2s(sm.rows[buf][lane >> 4][t],
               (lane < 16 ? p.k + (r.n0 + t) * p.k_stride : p.v + (r.n0 + t) * p.v_stride) + h0 * D, hn * D * 2,
               &sm.landed[buf]);
  };
  const size_t head = kv4_head_bytes<D>(a);
  const float invk = inv6ts_of(a.ks), invv = inv6ts_of(a.vs);
  for (int item = blockIdx.x, n = 0;; item += gridDim.x, ++n) {
    const int k = n & 7, buf = n & 1;
    __syncthreads();  // the other buffer, the scales and the last found group have been read
    if (k == 0) {
      const long long mine = item + (long long)(tid >> 5) * gridDim.x;
      const Group r = mine < p.items ? find_group<false>(a, (int)(mine / chunks), lane) : Group{-1, 0, 0, 0, 0};
      if (lane == 0) {
        sm.found[tid >> 5] = r;
        sm.place[tid >> 5] = r.b >= 0 ? kv4_group<D>(a, r.b, r.pos0) : nullptr;
      }
      __syncthreads();
      if (tid < 32) fetch(item, 0, buf);
    }
    const Group r = sm.found[k];
    if (r.b < 0) break;  // items are in order: none follows
    if (tid < 32 && k < 7) fetch(item + gridDim.x, k + 1, buf ^ 1);
    const bool ok = mbar_wait_within(&sm.landed[buf], turns >> buf & 1u, a.wait);
    turns ^= 1u << buf;
    if (!ok) {
      flag_status(a.status, GDN_E_TIMEOUT);
      sm.gave_up = 1;
    }
    const int h0 = item % chunks * p.heads, hn = min(p.heads, a.Hkv - h0);
    uint8_t *g = sm.place[k];  // null: a bad page, flagged
    if (g) g += h0 * head;
    if (g && ok) {
      for (int i = tid; i < hn * ITEMS; i += 256) {
        const int blk = i % NB, t = i / NB % 16, is_v = i / (16 * NB) & 1, h = i / ITEMS;
        if (t < r.t0 || t >= r.t1) continue;
        const uint4 *row = reinterpret_cast<const uint4 *>(&sm.rows[buf][is_v][t][h * D + blk * 16]);
        const uint4 x[2] = {row[0], row[1]};
        uint32_t codes[2], scale;
        if (!quant_bf16x16(x, is_v ? a.vs : a.ks, is_v ? invv : invk, codes, scale)) flag_status(a.status, GDN_E_NONFINITE);
        *reinterpret_cast<uint2 *>(g + h * head + (is_v ? kv4_v_code<D>(t, blk * 8) : kv4_k_code<D>(t, blk * 8))) =
            make_uint2(codes[0], codes[1]);
        sm.scales[h * 2 * D + (is_v ? kv4_v_scale<D>(t, blk) : kv4_k_scale<D>(t, blk)) - 16 * D] = (uint8_t)scale;
      }
    }
    __syncthreads();
    const bool stop = sm.gave_up;  // set between the loop's first barrier and this one only: the same for all
    if (g) {  // (what a group gets whose rows a thread gave up waiting for is unspecified)
      if (r.t0 == 0 && r.t1 == 16) {
        for (int i = tid; i < hn * (2 * D / 16); i += 256) {
          const int h = i / (2 * D / 16), w = i % (2 * D / 16);
          reinterpret_cast<uint4 *>(g + h * head + 16 * D)[w] = reinterpret_cast<const uint4 *>(sm.scales + h * 2 * D)[w];
        }
      } else {  // the other tokens' scales stay
        for (int i = tid; i < hn * ITEMS; i += 256) {
          const int blk = i % NB, t = i / NB % 16, is_v = i / (16 * NB) & 1, h = i / ITEMS;
          if (t < r.t0 || t >= r.t1) continue;
          const int at = is_v ? kv4_v_scale<D>(t, blk) : kv4_k_scale<D>(t, blk);
          (g + h * head)[at] = sm.scales[h * 2 * D + at - 16 * D];
        }
      }
    }
    if (stop) break;
  }
  if (tid == 0 && sm.gave_up) {  // the copies in flight land (or a bounded wait for each ends) before the CTA leaves
    mbar_wait(&sm.landed[0], (armed & 1u) ^ 1u);
    mbar_wait(&sm.landed[1], (armed >> 1 & 1u) ^ 1u);
  }
}

// The zeros of kv4_read: group r's rows where it is `empty` (they hold no token, or
// its page is bad), and the padding rows. Out of line: in line they cost a read of 16 tokens 0.2 us of 2.2.
template <int D>
__device__ __noinline__ void read_zeros(const RowsArgs &p, Group r, bool empty, int padding, int h0, int hn) {
  const int words = hn * (D / 8);  // of 16 bytes
  auto clear = [&](long long row, bool k, bool v) {
    for (int i = threadIdx.x; i < 2 * words; i += 256)
      if (i < words ? k : v)
        reinterpret_cast<uint4 *>((i < words ? p.k + row * p.k_stride : p.v + row * p.v_stride) + h0 * D)[i % words] =
            make_uint4(0, 0, 0, 0);
  };
  for (long long row = (long long)padding + blockIdx.x; row < p.a.T; row += gridDim.x)
    clear(row, p.a.zero_padding & 1, p.a.zero_padding & 2);
  if (empty)
    for (int t = r.t0; t < r.t1; ++t) clear(r.n0 + t, true, true);
}

// Read back: a thread takes half a block (4 code bytes in, 16 bytes out), so that a
// warp's stores are whole lines. 22638 rows of 8 heads, d = 128, 26 MB read and
// 93 written: 21.9 us (a block a thread, whose stores are half lines, took 5 more).
template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ RowsArgs p) {
  constexpr int NH = D / 8, ITEMS = 2 * 16 * NH;  // half blocks of a row; of a head's K and V of 16 tokens
  constexpr int U = 4;                            // loads in flight
  __shared__ Group found;
  __shared__ uint8_t *place;
  __shared__ int padding;
  const Kv4Args &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  kv4_begin();
  if (tid >> 5 == 1) {
    const int first = kv4_padding(a, lane);
    if (lane == 0) padding = first;
  }
  if (tid < 32) {
    const Group r = find_group<true>(a, blockIdx.x, lane);
    if (lane == 0) {
      found = r;
      place = r.b >= 0 && r.pos0 >= 0 ? kv4_group<D>(a, r.b, r.pos0) : nullptr;
    }
  }
  __syncthreads();
  const Group r = found;
  const int h0 = blockIdx.y * p.heads, hn = min(p.heads, a.Hkv - h0);
  if (padding < a.T || !place) {
    read_zeros<D>(p, r, r.b >= 0 && !place, padding, h0, hn);
    if (!place) return;
  }
  const size_t head = kv4_head_bytes<D>(a);
  const uint8_t *g = place + h0 * head;
  for (int i0 = tid; i0 < hn * ITEMS; i0 += 256 * U) {
    uint32_t code[U];
    uint8_t sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 256 * u, e = i % NH, t = i / NH % 16, is_v = i / (16 * NH) & 1, h = i / ITEMS;
      if (i >= hn * ITEMS) continue;
      const uint8_t *q = g + h * head;  // the group's other tokens lie in the page too: they are read and dropped
      code[u] = *reinterpret_cast<const uint32_t *>(q + (is_v ? kv4_v_code<D>(t, e * 4) : kv4_k_code<D>(t, e * 4)));
      sc[u] = q[is_v ? kv4_v_scale<D>(t, e / 2) : kv4_k_scale<D>(t, e / 2)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 256 * u, e = i % NH, t = i / NH % 16, is_v = i / (16 * NH) & 1, h = i / ITEMS;
      if (i >= hn * ITEMS || t < r.t0 || t >= r.t1) continue;
      __half2 v[4];
      e2m1x8_to_h2x4(code[u], v);
      const float f = e4m3_to_f32(sc[u]), ts = is_v ? a.vs : a.ks;
      uint32_t o[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        // e2m1 x e4m3 is exact; one FP32 rounding by ts, one to BF16
        const float2 y = mul2(mul2(__half22float2(v[m]), make_float2(f, f)), make_float2(ts, ts));
        o[m] = bf16x2(y.x, y.y);
      }
      uint16_t *row = is_v ? p.v + (r.n0 + t) * p.v_stride : p.k + (r.n0 + t) * p.k_stride;
      reinterpret_cast<uint4 *>(row + (h0 + h) * D)[e] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// The arguments, and the groups that the new rows touch at most: n rows of a
// sequence touch at most n, and (n + 30) / 16.
RowsArgs rows_args(const Kv4Args &a, uint16_t *k, long long ks, uint16_t *v, long long vs, long long &groups, int &chunks) {
  groups = min((long long)a.T, (long long)a.T / 16 + 2LL * a.B);
  RowsArgs p{a, k, v, ks, vs, min(a.Hkv, kHeads), 0};
  auto parts = [&]() { return (a.Hkv + p.heads - 1) / p.heads; };
  while (p.heads > 1 && groups * parts() < 2 * 152) p.heads = (p.heads + 1) / 2;  // fill the SMs
  chunks = parts();
  return p;
}

template <int D>
cudaError_t launch_append(const RowsArgs &p, cudaStream_t stream) {
  static bool allowed[64];
  cudaError_t e = kv4_allow_smem(kv4_append_kernel<D>, sizeof(AppendSmem<D>), allowed);
  if (e != cudaSuccess) return e;
  return kv4_launch(kv4_append_kernel<D>, min(p.items, 3 * 152), 256, sizeof(AppendSmem<D>), stream, p);
}

// ---------------------------------------------------------------- pages
constexpr int kCopyChunk = 16384;  // bytes of one page and layer that one CTA moves: 4 x 16 bytes a thread

// Bound by the bytes: 700 pages, 413 MB read and written, 62 us cold, 0.98 of the
// copy bandwidth.
// n_dev (compaction): the number of copies comes from the plan, and the tables
// are rewritten by its map beside the copies.
__global__ void __launch_bounds__(256) copy_pages_kernel(Kv4PageArgs a, const int32_t *n_dev) {
  int n = a.n;
  kv4_begin();
  if (n_dev) {
    n = *n_dev;
    const long long entries = (long long)a.rows * a.cols;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < entries; i += gridDim.x * 256LL) {
      const int p = a.table[i];
      a.tables_out[i] = p >= 0 && p < a.num_pages ? a.page_map[p] : -1;
    }
  }
  const int chunks = (int)((a.page_bytes + kCopyChunk - 1) / kCopyChunk);
  const long long total = (long long)n * a.layers * chunks;
  for (long long i = blockIdx.x; i < total; i += gridDim.x) {
    const int c = (int)(i % chunks);
    const long long j = i / chunks;
    const int l = (int)(j % a.layers), m = (int)(j / a.layers);
    const int s = a.src[m], d = a.dst[m];
    if (s < 0 || s >= a.num_pages || d < 0 || d >= a.num_pages) {
      if (threadIdx.x == 0) flag_status(a.status, GDN_E_RANGE);
      continue;
    }
    uint8_t *base = a.pages + l * a.layer_stride;
    const long long at = (long long)c * kCopyChunk;
    const uint4 *from = reinterpret_cast<const uint4 *>(base + s * a.page_bytes + at);
    uint4 *to = reinterpret_cast<uint4 *>(base + d * a.page_bytes + at);
    const int words = (int)(min((long long)kCopyChunk, a.page_bytes - at) / 16);
    uint4 x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int w = threadIdx.x + q * 256;
      if (w < words) x[q] = from[w];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int w = threadIdx.x + q * 256;
      if (w < words) to[w] = x[q];
    }
  }
}

// ---------------------------------------------------------------- compaction
// Workspace: [0] the number of moves, then the moved pages and their places.
struct CompactWs {
  int32_t *n_moves, *src, *dst;
};
CompactWs compact_ws(void *p, int num_pages) {
  int32_t *w = static_cast<int32_t *>(p);
  return {w, w + 4, w + 4 + (num_pages + 3) / 4 * 4};
}

// One CTA: a bitmap of the live pages in shared memory, its prefix counts, and
// from them every page's new id, a thread per page. With before(p) the live pages
// below p: a hole p < L is the (p - before(p))-th, a live p >= L the
// (before(p) - before(L))-th to move. A chain of one CTA's barriers and of the
// tables' loads: 5 to 8 us whatever the size.
__global__ void __launch_bounds__(1024) compact_plan_kernel(Kv4PageArgs a, CompactWs w) {
  extern __shared__ uint32_t bits[];
  __shared__ int sums[32], prefix[1024], live_total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  kv4_begin();
  const int words = (a.num_pages + 31) / 32;
  for (int i = tid; i < words; i += 1024) bits[i] = 0;
  __syncthreads();
  const long long entries = (long long)a.rows * a.cols;
  for (long long i = tid; i < entries; i += 4 * 1024) {
    int p[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) p[u] = i + u * 1024 < entries ? a.table[i + u * 1024] : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (p[u] >= a.num_pages) flag_status(a.status, GDN_E_RANGE);
      else if (p[u] >= 0) atomicOr(&bits[p[u] >> 5], 1u << (p[u] & 31));
    }
  }
  __syncthreads();
  // live pages before each thread's words
  const int per = (words + 1023) / 1024, w0 = min(tid * per, words), w1 = min(w0 + per, words);
  int mine = 0;
  for (int i = w0; i < w1; ++i) mine += __popc(bits[i]);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int x = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    sums[lane] = x;
    if (lane == 31) live_total = x;
  }
  __syncthreads();
  prefix[tid] = incl - mine + (warp ? sums[warp - 1] : 0);
  __syncthreads();
  const int L = live_total;
  auto before = [&](int p) {
    const int word = p >> 5;
    int t = word / per, n = prefix[t];
    for (int i = t * per; i < word; ++i) n += __popc(bits[i]);
    return n + __popc(bits[word] & ((1u << (p & 31)) - 1u));
  };
  const int bl = L < a.num_pages ? before(L) : L;
  for (int p = tid; p < a.num_pages; p += 1024) {
    const bool live = bits[p >> 5] >> (p & 31) & 1u;
    if (!live && p < L) w.dst[p - before(p)] = p;
    if (live && p >= L) w.src[before(p) - bl] = p;
  }
  if (tid == 0) {
    *w.n_moves = L - bl;
    *a.n_live = L;
  }
  __syncthreads();  // the lists are complete, and visible within this CTA
  for (int p = tid; p < a.num_pages; p += 1024) {
    const bool live = bits[p >> 5] >> (p & 31) & 1u;
    a.page_map[p] = !live ? -1 : p < L ? p : w.dst[before(p) - bl];
  }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Args &a, const uint16_t *k, long long k_stride, const uint16_t *v,
                              long long v_stride, cudaStream_t stream) {
  if (a.T == 0 || a.B == 0) return cudaSuccess;
  long long groups;
  int chunks;
  RowsArgs p = rows_args(a, const_cast<uint16_t *>(k), k_stride, const_cast<uint16_t *>(v), v_stride, groups, chunks);
  if (groups * chunks > 0x7fffffffLL - 3 * 152) return cudaErrorInvalidValue;
  p.items = (int)(groups * chunks);
  return a.D == 128 ? launch_append<128>(p, stream) : launch_append<64>(p, stream);
}
cudaError_t launch_kv4_read(const Kv4Args &a, uint16_t *k, uint16_t *v, cudaStream_t stream) {
  if (a.T == 0 || a.B == 0) return cudaSuccess;
  const long long stride = (long long)a.Hkv * a.D;
  long long groups;
  int chunks;
  const RowsArgs p = rows_args(a, k, stride, v, stride, groups, chunks);
  const dim3 grid((unsigned)groups, (unsigned)chunks);
  return kv4_launch(a.D == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>, grid, 256, 0, stream, p);
}

cudaError_t launch_kv4_copy_pages(const Kv4PageArgs &a, cudaStream_t stream) {
  const long long total = (long long)a.n * a.layers * ((a.page_bytes + kCopyChunk - 1) / kCopyChunk);
  if (total == 0) return cudaSuccess;
  return kv4_launch(copy_pages_kernel, (unsigned)min(total, 152LL * 8), 256, 0, stream, a, nullptr);
}

size_t kv4_compact_bytes(int num_pages) { return sizeof(int32_t) * (4 + 2 * (size_t)((num_pages + 3) / 4 * 4)); }

cudaError_t launch_kv4_compact(const Kv4PageArgs &a, cudaStream_t stream) {
  const CompactWs w = compact_ws(a.workspace, a.num_pages);
  const size_t smem = (size_t)(a.num_pages + 31) / 32 * 4;
  static bool allowed[64];
  cudaError_t e = kv4_allow_smem(compact_plan_kernel, 128 * 1024, allowed);
  if (e != cudaSuccess) return e;
  e = kv4_launch(compact_plan_kernel, 1, 1024, smem, stream, a, w);
  if (e != cudaSuccess) return e;
  Kv4PageArgs c = a;
  c.src = w.src;
  c.dst = w.dst;
  return kv4_launch(copy_pages_kernel, 152 * 8, 256, 0, stream, c, w.n_moves);
}

}  // namespace gdn
