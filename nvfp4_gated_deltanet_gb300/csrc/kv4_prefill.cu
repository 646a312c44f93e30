// Prefill attention over the 4-bit paged cache (include/gdn.h): ragged prompt
// chunks, causal, on the fifth-generation tensor cores.
//
// What bounds it: 4 d operations per (query row, key) on the tensor cores,
// and beside them one 2^x per (row, key); the cached bytes matter only for a
// chunk of a few tokens. Two kernels:
//
// kv4_expand_kernel decodes every sequence's cache once into tiles of 128
// tokens, exactly (E2M1 x E4M3 has at most six significant bits, 3 x 15 = 45, and is
// 0 or between 2^-10 and 2688 in magnitude): K in BF16 as the
// B operand of S = Q K^T, whose A operand is q as it came, and V transposed in
// FP16 as the B operand of O += P V, both already in the 128-byte swizzle that
// the MMA reads: each tile is one bulk copy. Decoding inside the attention kernel
// would repeat it for every 256 query rows (at 4096 tokens 64 times per KV head)
// on issue slots that the softmax needs. It is 5 % of the time of two long chunks
// (13 us for 10321 tokens of 8 heads, 12 MB read, 42 written into L2).
//
// kv4_prefill_kernel: an item is 256 query rows of one KV head -- two tiles of
// 128 rows, a row being a (token, query head of the group), so the whole group
// shares the tiles of K and V. While one tile's scores are in its softmax, the
// tensor cores run the other's products. A CTA per SM takes items, the longest
// first, until none is left; the next one's query rows and first products come
// while the last one's results are written:
//   warps 0..3, 4..7  softmax of row tile 0 / 1, one row per thread: S from
//                     tensor memory, weights back into tensor memory as FP16
//                     in the place of S's second half (the A operand of O += P V);
//                     the item's results
//   warp 8            TMEM allocation; one thread issues the MMAs
//   warp 9            one thread streams K and V tiles by bulk copies and an
//                     item's query rows by TMA (a box of tokens x the group's heads)
//   warp 10           finds the next item
//   warp 11           the padding rows, where they are asked for
// The softmax warps take over the others' registers (232 and 40 of 168 each), so
// that a thread holds its row's 128 scores: with 168 they had to be read from
// tensor memory twice, half at a time (284 against 272 us for the chunks below).
// Measured: two chunks of 4096 and 789 tokens, 32 query heads on 8 of d = 128,
// over 8100 and 2221 cached: 268 us in a graph, 1.60 PFLOP/s, 0.84 of a large BF16
// product; call after call 280 us, 1.54.
// What is left: a row tile's chain of softmax (1500 cycles), O += P V and S = Q K^T
// (1024) takes longer than the tensor cores' 2048 for both tiles.
// A row's weights are 2^(z - m + 6) with a maximum m that is only moved (and O
// rescaled in tensor memory) when the row's true maximum passes it by 8: they
// stay below 2^14, and normal FP16 numbers down to 2^-20 of the largest.
// Rounding: q, K and V enter exactly, the weights in FP16, all else is FP32.
// Every wait is bounded; one that gives up sets GDN_E_TIMEOUT and an abort flag
// that ends every role's loop.
#include "kv4.cuh"
#include "tc.cuh"

namespace gdn {

namespace {

constexpr int kKv = 128;          // tokens of a K / V tile
constexpr int kM = 128;           // rows of a query tile
constexpr int kThreads = 384;
constexpr float kShift = 6.0f;    // weights are 2^(z - m + 6)
constexpr float kSlack = 8.0f;    // how far a row's maximum may pass m before m moves
constexpr float kLog2e = 1.4426950408889634f;

struct PrefillKv4 {
  Kv4AttnArgs a;
  int G, tpt;                     // query heads per KV head; tokens of a query tile: 128 / G
  uint32_t inv_g;                 // ceil(2^16 / G): r / G = r inv_g >> 16 for r < 128
  int cap;                        // K / V tiles (of all KV heads) that the workspace holds
  int *next;                      // items handed out beside each CTA's first one; zeroed by the expansion
  uint16_t *tiles;                // [cap][Hkv][K: d / 64 x 128 rows x 64, BF16; V^T: 2 x d rows x 64, FP16], swizzled
};

// The sequence that holds item x when sequence b has count(b) of them, and the
// items before it; -1 past the end. All lanes of a warp.
template <typename F>
GDN_DEV int find_item(int B, int x, int lane, F count, int &before, int &total) {
  int base = 0, b = -1;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int n = b0 + lane < B ? count(b0 + lane) : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, base + incl > x);
    if (b < 0 && past) {
      const int l = __ffs(past) - 1;
      b = b0 + l;
      before = base + __shfl_sync(0xffffffffu, incl - n, l);
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  total = base;
  return b;
}

// One CTA per tile of 128 tokens and KV head. Tokens past the end become 0.
template <int D>
__global__ void __launch_bounds__(256) kv4_expand_kernel(PrefillKv4 p) {
  const Kv4Args &c = p.a.c;
  kv4_begin();
  const int tid = threadIdx.x, lane = tid & 31;
  const int x = blockIdx.x / c.Hkv, h = blockIdx.x % c.Hkv;
  int before = 0, total = 0;
  const int b = find_item(c.B, x, lane, [&](int i) { return (kv4_len(c, i) + kKv - 1) / kKv; }, before, total);
  if (blockIdx.x == 0) {
    if (tid == 0) {
      if (total > p.cap) flag_status(c.status, GDN_E_RANGE);
      *p.next = 0;
    }
    for (int i = tid; i < c.B; i += 256) kv4_seq(c, i);  // flags bad entries
  }
  if (b < 0) return;
  const int pos0 = (x - before) * kKv, len = kv4_len(c, b);
  __shared__ const uint8_t *groups[kKv / 16];
  if (tid < kKv / 16) {
    const uint8_t *g = pos0 + tid * 16 < len ? kv4_group<D>(c, b, pos0 + tid * 16) : nullptr;
    groups[tid] = g ? g + h * kv4_head_bytes<D>(c) : nullptr;
  }
  __syncthreads();
  uint8_t *tile = reinterpret_cast<uint8_t *>(p.tiles) + ((size_t)x * c.Hkv + h) * (4 * kKv * D);
  // K: 16-byte pieces, eight channels of one token
#pragma unroll
  for (int i = tid; i < kKv * (D / 8); i += 256) {
    const int row = i / (D / 8), w = i % (D / 8);
    const uint8_t *g = groups[row / 16];
    uint32_t o[4] = {0, 0, 0, 0};
    if (g && pos0 + row < len) {
      // an FP16 code moved down 3 bits is the BF16 value 2^-112 times as large; the scale (at most 448) makes that good
      const float s = e4m3_to_f32(g[kv4_k_scale<D>(row & 15, w / 2)]) * 5.192296858534828e33f;  // 2^112
      const __nv_bfloat162 s2 = __float2bfloat162_rn(s);
      __half2 e[4];
      e2m1x8_to_h2x4(*reinterpret_cast<const uint32_t *>(g + kv4_k_code<D>(row & 15, w * 4)), e);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t x = h2u(e[q]);
        uint32_t y = ((x >> 3) & 0x0FFF0FFFu) | (x & 0x80008000u);
        const __nv_bfloat162 z = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&y), s2);
        o[q] = *reinterpret_cast<const uint32_t *>(&z);
      }
    }
    *reinterpret_cast<uint4 *>(tile + (w / 8) * (kKv * 128) + sw_off16(row, (w & 7) * 8)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  // V^T: eight tokens of eight channels; neighbouring lanes take neighbouring
  // tokens, so that eight of them write whole 128-byte rows
  uint8_t *vt = tile + 2 * kKv * D;
#pragma unroll
  for (int i = tid; i < (kKv / 8) * (D / 8); i += 256) {
    const int oct = (i & 7) + 8 * (i / (8 * (D / 8))), w = (i / 8) % (D / 8);  // tokens 8 oct .., channels 8 w ..
    const uint8_t *g = groups[oct / 2];
    uint32_t code[8], o[4][2][4];  // o[pair of tokens][even / odd channels][channel pair]
    uint8_t sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = (oct & 1) * 8 + j;
      const bool in = g && pos0 + oct * 8 + j < len;
      code[j] = in ? *reinterpret_cast<const uint32_t *>(g + kv4_v_code<D>(t, w * 4)) : 0u;
      sc[j] = in ? g[kv4_v_scale<D>(t, w / 2)] : (uint8_t)0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 s = __floats2half2_rn(e4m3_to_f32(sc[2 * j]), e4m3_to_f32(sc[2 * j + 1]));
      decode8((code[2 * j] & 0x0F0F0F0Fu) | ((code[2 * j + 1] << 4) & 0xF0F0F0F0u), s, o[j][0]);
      decode8(((code[2 * j] >> 4) & 0x0F0F0F0Fu) | (code[2 * j + 1] & 0xF0F0F0F0u), s, o[j][1]);
    }
#pragma unroll
    for (int ch = 0; ch < 8; ++ch)
      *reinterpret_cast<uint4 *>(vt + (oct / 8) * (D * 128) + sw_off16(w * 8 + ch, (oct & 7) * 8)) =
          make_uint4(o[0][ch & 1][ch >> 1], o[1][ch & 1][ch >> 1], o[2][ch & 1][ch >> 1], o[3][ch & 1][ch >> 1]);
  }
}

template <int D>
struct PrefillShape {
  static constexpr int kStages = D == 128 ? 2 : 4;   // of K and of V each
  static constexpr int kTileBytes = kKv * D * 2;     // a K tile, a V tile, and 128 query rows
  static constexpr int kOut = 8 * 4096;              // per softmax warp: 32 rows x 128 bytes of results on their way
  static constexpr int kBars = 512;
  static constexpr int kBytes = (2 + 2 * kStages) * kTileBytes + kOut + kBars;
  static constexpr int kO = 2 * kKv;                 // TMEM columns: S0, S1, then O0, O1
  static_assert(kO + 2 * D <= 512, "tensor memory");
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};

// 256 query rows of one KV head: sequence rows q0 + t0 .., and the K / V tiles
// that each row tile sees.
struct Item {
  int h, q0, n, t0, len, nkv[2], tile0;  // h < 0: no more items
};

// The x-th item by falling cost (K / V tiles) of all sequences, without its
// head; false past the end. All lanes of a warp. items: of all sequences, for a
// head.
GDN_DEV bool find_work(const PrefillKv4 &p, int x, int lane, Item &w, int &items) {
  const Kv4Args &c = p.a.c;
  const int step = 2 * p.tpt;
  auto own_of = [&](const Kv4Seq &s) { return (int)((unsigned)(s.q1 - s.q0 + step - 1) / (unsigned)step); };
  Kv4Seq s0 = {0, 0, 0};  // of sequence `lane`
  if (lane < c.B) s0 = kv4_seq(c, lane);
  const int own0 = own_of(s0);
  auto seq_of = [&](int b) { return b < 32 ? s0 : kv4_seq(c, b); };  // b % 32 == lane
  auto count = [&](const Kv4Seq &s, int own, int cost) {  // the sequence's items of at least this cost
    const int n = s.q1 - s.q0;
    if (cost == 0) return own;
    const long long at = (long long)(cost - 1) * kKv - (s.len - n);  // an item's last token, at least
    return at <= 0 ? own : at >= n ? 0 : own - (int)((unsigned)at / (unsigned)step);
  };
  auto sum = [&](int v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  auto all = [&](int cost) {
    int v = lane < c.B ? count(s0, own0, cost) : 0;
    for (int b = lane + 32; b < c.B; b += 32) {
      const Kv4Seq s = kv4_seq(c, b);
      v += count(s, own_of(s), cost);
    }
    return sum(v);
  };
  items = all(0);
  if (x >= items) return false;
  // Where every item has a CTA of its own the order does not matter: then, and
  // for one sequence, whose costs rise from item to item, no search (it takes 2 us
  // of one warp, before the first product).
  const bool any_order = c.B == 1 || (long long)items * c.Hkv <= gridDim.x;
  int lo = 0;
  if (!any_order) {
    int hi = 0;
    for (int b = lane; b < c.B; b += 32) hi = max(hi, (seq_of(b).len + kKv - 1) / kKv);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    ++hi;  // all(lo) > x >= all(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (all(mid) > x) lo = mid; else hi = mid;
    }
  }
  int r = any_order ? x : x - all(lo + 1);  // among the items of cost lo (or all), by sequence
  int tiles = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const Kv4Seq s = b0 + lane < c.B ? seq_of(b0 + lane) : Kv4Seq{0, 0, 0};
    const int own = b0 ? own_of(s) : own0;
    const int above = any_order ? 0 : count(s, own, lo + 1), e = count(s, own, lo) - above, kt = (s.len + kKv - 1) / kKv;
    int incl = e, kincl = kt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o), z = __shfl_up_sync(0xffffffffu, kincl, o);
      if (lane >= o) {
        incl += y;
        kincl += z;
      }
    }
    const unsigned past = __ballot_sync(0xffffffffu, incl > r);
    if (past) {
      const int l = __ffs(past) - 1;
      w.q0 = __shfl_sync(0xffffffffu, s.q0, l);
      w.n = __shfl_sync(0xffffffffu, s.q1 - s.q0, l);
      w.len = __shfl_sync(0xffffffffu, s.len, l);
      w.t0 = __shfl_sync(0xffffffffu, own - 1 - above - (r - (incl - e)), l) * step;
      w.tile0 = tiles + __shfl_sync(0xffffffffu, kincl - kt, l);
      break;
    }
    r -= __shfl_sync(0xffffffffu, incl, 31);
    tiles += __shfl_sync(0xffffffffu, kincl, 31);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t1 = min(w.n, w.t0 + (i + 1) * p.tpt) - 1;  // the row tile's last token
    const int last = w.len - w.n + t1;
    w.nkv[i] = t1 >= w.t0 + i * p.tpt && last >= 0 ? last / kKv + 1 : 0;
    if (w.tile0 + w.nkv[i] > p.cap) w.nkv[i] = 0;         // the workspace was too small (flagged by the expansion)
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, PrefillKv4 p) {
  using S = PrefillShape<D>;
  constexpr int NS = S::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];  // the swizzled tiles start on 1024 bytes
  uint8_t *qs = sm, *kbuf = sm + 2 * S::kTileBytes, *vbuf = kbuf + NS * S::kTileBytes, *obuf = vbuf + NS * S::kTileBytes;
  uint64_t *k_full = reinterpret_cast<uint64_t *>(obuf + S::kOut);
  uint64_t *v_full = k_full + NS, *k_free = v_full + NS, *v_free = k_free + NS;
  uint64_t *s_full = v_free + NS, *p_ready = s_full + 2, *o_done = p_ready + 4;
  uint64_t *q_full = o_done + 2, *q_free = q_full + 1;
  uint64_t *item_full = q_free + 1, *item_free = item_full + 2, *fin = item_free + 2;
  Item *items = reinterpret_cast<Item *>(fin + 1);  // [2]
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(items + 2);
  volatile uint32_t *abort_flag = tmem_holder + 1;
  const Kv4Args &c = p.a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(v_full + s, 1);
      mbar_init(k_free + s, 1);
      mbar_init(v_free + s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_ready + 2 * i, 128);
      mbar_init(p_ready + 2 * i + 1, 128);
      mbar_init(o_done + i, 1);
      mbar_init(item_full + i, 1);
      mbar_init(item_free + i, 10);  // every warp but the one that fills it
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(fin, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  auto wait = [&](uint64_t *bar, uint32_t use) { return wait_or_abort(bar, use & 1u, abort_flag, c.status, c.wait); };
  auto warp_wait_all = [&](uint64_t *bar, uint32_t use) { return __all_sync(0xffffffffu, wait(bar, use)) != 0; };
  // Item `it` of this CTA; false when there is none (or a wait gave up). A whole warp.
  auto take = [&](int it, Item &w) {
    if (!warp_wait_all(item_full + (it & 1), it >> 1)) return false;
    w = items[it & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(item_free + (it & 1));
    return w.h >= 0;
  };

  // registers: 384 threads x 168 at launch = 256 x 232 + 128 x 40
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    // ------------------------------------------------ softmax: thread = row r of row tile i
    const int i = warp >> 2, r = tid & 127;
    const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = base + i * kKv, tO = base + S::kO + i * D;
    const float cs = p.a.sm_scale * c.ks * kLog2e;
    uint32_t uses = 0, dones = 0;  // of this row tile's scores, and items that had any
    for (int it = 0; warp_wait_all(item_full + (it & 1), it >> 1); ++it) {
      const Item &w = items[it & 1];  // read where it is needed, and given back at the end: registers are short
      if (w.h < 0) break;
      const int off_t = i * p.tpt + (int)(r * p.inv_g >> 16);                      // the row's token, from the item's first
      const int sure = w.len - w.n + w.t0 + i * p.tpt;            // every row of the tile sees up to here
      const int last = r < p.tpt * p.G && w.t0 + off_t < w.n ? w.len - w.n + w.t0 + off_t : -1;  // the last token this row sees
      const int nkv = w.nkv[i];
      float m = -INFINITY, l = 0.0f;
      bool ok = true;
      for (int j = 0; j < nkv; ++j, ++uses) {
        if (!warp_wait_all(s_full + i, uses)) { ok = false; break; }
        tc_fence_after();
        const bool mask = j * kKv + kKv - 1 > sure;
        // The second half's weights go to the MMAs (columns 96..127) while the first half's, columns 64..95, are made.
        float s[128];
        {
          uint32_t raw[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, raw + 32 * q);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 128; ++q) s[q] = __uint_as_float(raw[q]);
          if (mask) {
#pragma unroll
            for (int q = 0; q < 128; ++q)
              if (j * kKv + q > last) s[q] = -INFINITY;
          }
        }
        float x4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int q = 4; q < 128; q += 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) x4[e] = fmaxf(x4[e], s[q + e]);
        const float top = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * cs;
        const bool up = top > m + kSlack;  // decided row by row: a row's result depends on no other row
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, up)) {
          // S of this tile is complete, so the O += P V issued before it is too
          const float f = up ? ex2(m - top) : 1.0f;
          if (up) m = top;
          l *= f;
#pragma unroll
          for (int q = 0; q < D; q += 32) {
            uint32_t o[32];
            tmem_ld32(tO + q, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(tO + q, o);
          }
        }
        const float off = kShift - (m == -INFINITY ? 0.0f : m);
        const float2 cs2 = make_float2(cs, cs), off2 = make_float2(off, off);
        float2 sum[2] = {make_float2(l, 0.0f), make_float2(0.0f, 0.0f)};
        auto weigh = [&](int half) {
          uint32_t x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float2 z = fma2(make_float2(s[64 * half + 2 * e], s[64 * half + 2 * e + 1]), cs2, off2);
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            sum[e & 1] = add2(sum[e & 1], z);
            x[e] = h2u(__floats2half2_rn(z.x, z.y));
          }
          tmem_st32(tS + 64 + 32 * half, x);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(p_ready + 2 * i + half);
        };
        weigh(1);
        weigh(0);
        sum[0] = add2(sum[0], sum[1]);
        l = sum[0].x + sum[0].y;
      }
      // ---------------------------------------------- the rows' results, 64 channels at a time: each lane's row
      // into the warp's staging rows, from there whole 128-byte lines to memory (16 bytes of 32 rows at a time
      // straight from the lanes took 5000 cycles an item)
      if (!ok || (nkv > 0 && !warp_wait_all(o_done + i, dones++))) break;
      tc_fence_after();
      const float inv = l == 0.0f ? 0.0f : c.vs / l;
      uint8_t *st = obuf + warp * 4096;
#pragma unroll
      for (int q0 = 0; q0 < D; q0 += 64) {
#pragma unroll
        for (int q = 0; q < 64; q += 32) {
          uint32_t o[32];
          if (nkv > 0) {
            tmem_ld32(tO + q0 + q, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          uint32_t x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            x[e] = bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4 *>(st + lane * 128 + (((q / 8 + e) ^ (lane & 7)) << 4)) =
                make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = k * 4 + (lane >> 3), rr = (warp & 3) * 32 + row;
          const int tr = (int)(rr * p.inv_g >> 16), tk = w.t0 + i * p.tpt + tr;
          if (rr < p.tpt * p.G && tk < w.n)
            reinterpret_cast<uint4 *>(p.a.out + ((long long)(w.q0 + tk) * p.a.Hq + w.h * p.G + rr - tr * p.G) * D +
                                      q0)[lane & 7] =
                *reinterpret_cast<const uint4 *>(st + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
        }
        __syncwarp();
      }
      tc_fence_before();  // O has been read: the next item's products follow this row tile's next weights
      const int tok = w.t0 + off_t;
      if (p.a.lse && r < p.tpt * p.G && tok < w.n)
        p.a.lse[(long long)(w.q0 + tok) * p.a.Hq + w.h * p.G + r - (off_t - i * p.tpt) * p.G] = (m + (log2f(l) - kShift)) * 0.6931471805599453f;
      __syncwarp();
      if (lane == 0) mbar_arrive(item_free + (it & 1));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 8) {
      // ------------------------------------------------ MMAs
      constexpr uint32_t idS = idesc_bf16(kKv), idO = idesc_f16(D);
      constexpr uint64_t kStep = S::kTileBytes / 16;  // from one stage or tile to the next, in a descriptor
      const uint64_t qd = desc_sw128(smem_u32(qs)), kd = desc_sw128(smem_u32(kbuf)), vd = desc_sw128(smem_u32(vbuf));
      const bool me = elect_one();
      uint32_t kv = 0, uses[2] = {0, 0};  // K / V tiles taken, and each row tile's
      Item w;
      bool ok = true;
      for (int it = 0; ok && take(it, w); ++it) {
        const int nmax = max(w.nkv[0], w.nkv[1]);
        if (me) {
          auto scores = [&](int i, uint32_t use) {  // S_i = Q_i K^T
            const uint64_t q = qd + i * kStep, kk = kd + (uint64_t)(use % NS) * kStep;
            const uint32_t d = tmem + i * kKv;
            mma_f16_ss_c<false>(d, q, kk, idS);
  #pragma unroll
            for (int k = 1; k < D / 16; ++k)
              mma_f16_ss_c<true>(d, q + (k / 4) * (kM * 128 / 16) + 2 * (k & 3), kk + (k / 4) * (kKv * 128 / 16) + 2 * (k & 3), idS);
            tc_commit(s_full + i);
          };
          auto values = [&](int i, uint32_t use, bool first) {  // O_i += P_i V
            const uint64_t v = vd + (uint64_t)(use % NS) * kStep;
            const uint32_t d = tmem + S::kO + i * D, a = tmem + i * kKv + 64;
            if (!(ok = wait(p_ready + 2 * i + 1, uses[i]))) return;  // tokens 64..127 first
            tc_fence_after();
            if (first) mma_f16_ts_c<false>(d, a + 32, v + D * 128 / 16, idO);
            else mma_f16_ts_c<true>(d, a + 32, v + D * 128 / 16, idO);
  #pragma unroll
            for (int k = 1; k < 4; ++k) mma_f16_ts_c<true>(d, a + 32 + 8 * k, v + D * 128 / 16 + 2 * k, idO);
            if (!(ok = wait(p_ready + 2 * i, uses[i]))) return;
            tc_fence_after();
  #pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ts_c<true>(d, a + 8 * k, v + 2 * k, idO);
            ++uses[i];
          };
          ok = wait(q_full, it);
          if (ok && nmax > 0 && (ok = wait(k_full + kv % NS, kv / NS))) {
            tc_fence_after();
  #pragma unroll
            for (int i = 0; i < 2; ++i)
              if (w.nkv[i] > 0) scores(i, kv);
            tc_commit(k_free + kv % NS);
          }
          if (ok && nmax <= 1) tc_commit(q_free);
          for (int j = 0; j < nmax && ok; ++j) {
            const uint32_t u = kv + j;
            ok = wait(v_full + u % NS, u / NS) && (j + 1 >= nmax || wait(k_full + (u + 1) % NS, (u + 1) / NS));
  #pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || j >= w.nkv[i]) continue;
              values(i, u, j == 0);
              if (!ok) break;
              if (j + 1 < w.nkv[i]) scores(i, u + 1);
              else tc_commit(o_done + i);
            }
            if (!ok) break;
            tc_commit(v_free + u % NS);
            if (j + 1 < nmax) tc_commit(k_free + (u + 1) % NS);
            if (j + 2 == nmax) tc_commit(q_free);  // the item's last scores are issued
          }
        }
        ok = __any_sync(0xffffffffu, me && ok);
        kv += nmax;
      }
      // every MMA issued has completed before the CTA may leave
      if (me) {
        tc_commit(fin);
        mbar_wait(fin, 0u);
      }
    } else if (warp == 9) {
      // ------------------------------------------------ query rows, K and V tiles
      const int q_bytes = p.tpt * p.G * D * 2;  // of a row tile
      uint32_t u = 0, ku = 0, taken = 0;  // V tiles, K tiles and items whose copies were issued
      Item w;
      bool ok = true;
      for (int it = 0; ok && take(it, w); ++it) {
        const int nmax = max(w.nkv[0], w.nkv[1]);
        if (lane == 0 && it > 0) ok = wait(q_free, it - 1);
        if (lane == 0 && ok) {
          mbar_arrive_expect_tx(q_full, 2 * q_bytes);
          ++taken;
  #pragma unroll
          for (int x = 0; x < 2 * (D / 64); ++x)
            tma_load_3d(qs + (x / (D / 64)) * S::kTileBytes + (x % (D / 64)) * (kM * 128), &tmQ, x % (D / 64) * 64, w.h * p.G,
                        w.q0 + w.t0 + x / (D / 64) * p.tpt, q_full);
          if (it == 0) pdl_wait();  // the expansion has finished
          const uint8_t *src = reinterpret_cast<const uint8_t *>(p.tiles) + ((size_t)w.tile0 * c.Hkv + w.h) * (2 * S::kTileBytes);
          const size_t step = (size_t)c.Hkv * 2 * S::kTileBytes;
          for (int j = 0; j < nmax; ++j, ++u) {
            const int s = u % NS;
            if (u >= NS && !(ok = wait(k_free + s, u / NS - 1))) break;
            mbar_arrive_expect_tx(k_full + s, S::kTileBytes);
            bulk_g2s(kbuf + s * S::kTileBytes, src + j * step, S::kTileBytes, k_full + s);
            ku = u + 1;
            if (u >= NS && !(ok = wait(v_free + s, u / NS - 1))) break;
            mbar_arrive_expect_tx(v_full + s, S::kTileBytes);
            bulk_g2s(vbuf + s * S::kTileBytes, src + j * step + S::kTileBytes, S::kTileBytes, v_full + s);
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      }
      if (lane == 0 && u == 0) pdl_wait();
      if (lane == 0) {  // the last copies land (or a bounded wait for each ends) before the CTA leaves, whoever gives up when
        if (taken > 0) mbar_wait(q_full, (taken - 1) & 1u);
        for (uint32_t x = ku < NS ? 0 : ku - NS; x < ku; ++x) mbar_wait(k_full + x % NS, (x / NS) & 1u);
        for (uint32_t x = u < NS ? 0 : u - NS; x < u; ++x) mbar_wait(v_full + x % NS, (x / NS) & 1u);
      }
    } else if (warp == 10) {
      // ------------------------------------------------ the next item
      int all_items = 0;
      for (int it = 0;; ++it) {
        Item w{-1, 0, 0, 0, 0, {0, 0}, 0};
        if (it == 0 || (long long)all_items * c.Hkv > gridDim.x) {  // else every item has its CTA
          if (it == 1) pdl_wait();  // the counter is zeroed by the expansion
          int x = blockIdx.x;
          if (it > 0) {
            if (lane == 0) x = (int)gridDim.x + atomicAdd(p.next, 1);
            x = __shfl_sync(0xffffffffu, x, 0);
          }
          if (find_work(p, x / c.Hkv, lane, w, all_items)) w.h = x % c.Hkv;
        }
        if (it >= 2 && !warp_wait_all(item_free + (it & 1), (it >> 1) - 1)) break;
        if (lane == 0) {
          items[it & 1] = w;
          mbar_arrive(item_full + (it & 1));
        }
        __syncwarp();
        if (w.h < 0) break;
      }
      kv4_begin();  // on every path: this grid must not end before the one it follows
    } else {
      // ------------------------------------------------ padding rows (in the expansion they cost each of its CTAs a load)
      for (long long row = (long long)kv4_padding(c, lane) + blockIdx.x; row < c.T; row += gridDim.x) {
        if (c.zero_padding & 1)
          for (int i = lane; i < p.a.Hq * (D / 8); i += 32)
            reinterpret_cast<uint4 *>(p.a.out + row * p.a.Hq * D)[i] = make_uint4(0, 0, 0, 0);
        if ((c.zero_padding & 2) && p.a.lse)
          for (int i = lane; i < p.a.Hq; i += 32) p.a.lse[row * p.a.Hq + i] = -INFINITY;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_prefill_t(const PrefillKv4 &p, int num_sms, cudaStream_t stream) {
  using S = PrefillShape<D>;
  CUtensorMap tmQ;
  if (!make_heads_map(&tmQ, p.a.q, p.a.c.T, p.a.Hq, D, p.a.q_stride, p.tpt, p.G)) return cudaErrorInvalidValue;
  static bool allowed[64];
  cudaError_t e = kv4_allow_smem(kv4_prefill_kernel<D>, S::kBytes, allowed);
  if (e != cudaSuccess) return e;
  const Kv4Args &c = p.a.c;
  e = kv4_launch(kv4_expand_kernel<D>, (unsigned)p.cap * c.Hkv, 256, 0, stream, p);
  if (e != cudaSuccess) return e;
  const long long items = (long long)(c.T / (2 * p.tpt) + c.B) * c.Hkv;  // at most
  return kv4_launch(kv4_prefill_kernel<D>, (unsigned)(items < num_sms ? items : num_sms), kThreads, S::kBytes, stream, tmQ, p);
}

// K / V tiles: every sequence's last one may be partly filled.
long long tile_cap(const Kv4AttnArgs &a, long long total_kv) { return total_kv / kKv + a.c.B; }

}  // namespace

// 0 where the tiles would pass what a grid can index.
size_t kv4_prefill_bytes(const Kv4AttnArgs &a, long long total_kv) {
  const long long n = tile_cap(a, total_kv) * a.c.Hkv;
  return n > 0x7fffffffLL ? 0 : (size_t)n * 4 * kKv * a.c.D + 16;
}

cudaError_t launch_kv4_prefill(const Kv4AttnArgs &a, long long total_kv, void *workspace, int num_sms, cudaStream_t stream) {
  const int G = a.Hq / a.c.Hkv, cap = (int)tile_cap(a, total_kv);
  const size_t tiles = (size_t)cap * a.c.Hkv * 4 * kKv * a.c.D;
  const PrefillKv4 p{a, G, kM / G, (65536u + G - 1) / G, cap, reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + tiles),
                     static_cast<uint16_t *>(workspace)};
  return a.c.D == 128 ? launch_prefill_t<128>(p, num_sms, stream) : launch_prefill_t<64>(p, num_sms, stream);
}

}  // namespace gdn
