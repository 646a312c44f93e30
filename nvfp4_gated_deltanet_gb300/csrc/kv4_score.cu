// Accumulated attention weights over the 4-bit paged cache (include/gdn.h): what
// the rows of a call gave to each cached token, by the log-sum-exp that the
// attention call returned.
//
//   out_j = (j < scored ? in_j : 0) + sum_i exp(sm q_i . k_j - lse_i),  over the rows i (tokens x
//   the KV head's query heads) that see token j
//
// What bounds it: for a few rows the cached K, d/2 + d/16 bytes per token and KV
// head, read once (V is not), and 8 bytes of scores; for a prompt's rows 2 d
// operations and one 2^x per (row, token).
#include <algorithm>
#include <type_traits>

#include "kv4.cuh"
#include "tc.cuh"

namespace gdn {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// What a row's weights go by: 2^(s c - hi) w, w = 2^-lo near 1 holding what FP32 cannot: the lse in bits is
// hi + lo, and `skew` is by how much c misses the exact factor of a score in bits, relatively, which at the
// scores that matter (near the lse) moves the difference by skew hi.
struct RowWeight {
  float hi, w;
};
GDN_DEV RowWeight row_weight(float lse, float skew) {
  if (lse == -INFINITY) return {0.0f, 0.0f};  // the row saw nothing
  const float hi = lse * kLog2e, lo = fmaf(lse, kLog2e, -hi) + lse * 1.925963e-8f;  // log2 e - kLog2e
  return {hi, ex2(fmaf(skew, hi, -lo))};
}

// A sequence's scores, checked: its row in the slots, or -1 where it is left out.
GDN_DEV int score_slot(const Kv4ScoreArgs &p, int b, int len) {
  const int slot = p.s.slots ? p.s.slots[b] : b;
  if (slot < -1 || slot >= p.s.n_slots || len > p.s.tokens) {
    flag_status(p.c.status, GDN_E_RANGE);
    return -1;
  }
  return slot;
}
// A slot that another sequence of the batch has too (both are left out). A whole warp.
GDN_DEV bool slot_twice(const Kv4ScoreArgs &p, int b, int slot, int lane) {
  bool twice = false;
  if (p.s.slots)
    for (int i = lane; i < p.c.B; i += 32) twice |= i != b && p.s.slots[i] == slot;
  twice = __any_sync(0xffffffffu, twice) != 0;
  if (twice) flag_status(p.c.status, GDN_E_RANGE);
  return twice;
}

// d += A B, m16n8k16, FP16 in, FP32 accumulation
GDN_DEV void mma_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

GDN_DEV __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
// Two E4M3 bytes -> two FP16 (exact)
GDN_DEV uint32_t e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}

// ---------------------------------------------------------------- few rows: a warp per 64 tokens
// All sequences' and KV heads' tokens, 64 at a time (a unit), are cut into runs of
// equal length, one per warp. A warp holds a unit's K bytes in registers: as soon
// as a group of 16 tokens is decoded into MMA operands, the same group of the next
// unit is on its way. No part of a token's sum leaves the warp, nothing is joined.
// Measured: 64 sequences of up to 8190 tokens, 8 KV heads of d = 128, 4 rows each, 162
// MB: 39 us, 4.1 TB/s (0.61 of the copy bandwidth). A unit takes about 700 instructions,
// half of them the decoding; with 16 warps an SM 52% of the issue slots are used, and
// what is left is their latency (per issue 2.1 warps wait for loads, 1.8 for the
// instruction before; 32 tokens a unit and a third more warps: 48 to 56). The tiles
// below would write the decoded K down first.
constexpr int kGroups = 4, kUnit = 16 * kGroups;  // (a lane of four writes a group's sums)
constexpr int kLook = 32 / kGroups;  // units whose groups' places are worked out at once, a group per lane
constexpr int kRowWarps = 8;

struct Unit {
  int b, h, pos, len;  // sequence, KV head, first token; the sequence's tokens
};
GDN_DEV int units_of(int len) { return (len + kUnit - 1) / kUnit; }
GDN_DEV void next_unit(const Kv4Args &c, Unit &k) {
  if ((k.pos += kUnit) < k.len) return;
  k.pos = 0;
  if (++k.h < c.Hkv) return;
  k.h = 0;
  do k.len = kv4_len(c, ++k.b);  // only called while there is another
  while (k.len == 0);
}

template <int D, int NQ>
__global__ void __launch_bounds__(32 * kRowWarps, NQ == 1 ? 2 : 1) kv4_score_rows_kernel(Kv4ScoreArgs p, float c2, float skew) {
  constexpr int KS = D / 16, W = D / 32;
  kv4_begin();
  const Kv4Args &c = p.c;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = p.Hq / c.Hkv;
  // ---- the warp's run
  long long total = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    int n = b0 + lane < c.B ? units_of(kv4_len(c, b0 + lane)) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    total += n;
  }
  total *= c.Hkv;
  const long long warps = (long long)gridDim.x * kRowWarps, me = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const long long u0 = total / warps * me + total % warps * me / warps;
  int left = (int)(total / warps * (me + 1) + total % warps * (me + 1) / warps - u0);
  if (blockIdx.x == 0 && threadIdx.x < 32)
    for (int b = lane; b < c.B; b += 32) kv4_seq(c, b);  // flags bad entries
  if (left == 0) return;
  Unit cur{0, 0, 0, 0};
  {
    long long before = 0;
    for (int b0 = 0;; b0 += 32) {  // (ends: u0 < total)
      const int n = b0 + lane < c.B ? units_of(kv4_len(c, b0 + lane)) : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned past = __ballot_sync(0xffffffffu, (before + incl) * c.Hkv > u0);
      if (past) {
        const int l = __ffs(past) - 1;
        const long long off = u0 - (before + __shfl_sync(0xffffffffu, incl - n, l)) * c.Hkv;
        const int own = __shfl_sync(0xffffffffu, n, l);
        cur.b = b0 + l;
        cur.len = kv4_len(c, cur.b);
        cur.h = (int)(off / own);
        cur.pos = (int)(off - (long long)cur.h * own) * kUnit;
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // ---- loads
  Unit ahead = cur;              // the unit that is loaded next
  int ahead_left = left, ahead_i = kLook;
  const uint8_t *where = c.pages;
  auto look = [&]() {
    if (ahead_i == kLook) {
      ahead_i = 0;
      where = c.pages;  // (past the run's or the sequence's end: read, and not used)
      Unit k = ahead;
      if (lane / kGroups < ahead_left) {
        for (int i = 0; i < lane / kGroups; ++i) next_unit(c, k);
        const int pos = k.pos + lane % kGroups * 16;
        const uint8_t *grp = pos < k.len ? kv4_group<D>(c, k.b, pos) : nullptr;  // a bad page id is flagged
        if (grp) where = grp + k.h * kv4_head_bytes<D>(c);
      }
    }
  };
  // (no loads by the read-only path: pages may have been written by a kernel that had not ended when this one began)
  uint32_t kw[kGroups][2][W];  // [group][token g, g + 8]: 16 (d = 64: 8) code bytes, and their scales
  uint32_t ks[kGroups][2];
  auto load = [&](int q) {
    const uint8_t *src = reinterpret_cast<const uint8_t *>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(where), ahead_i * kGroups + q));
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int tok = g + 8 * x;
      if constexpr (D == 128) {
        const uint4 v = *reinterpret_cast<const uint4 *>(src + kv4_k_code<D>(tok, t * 16));
        kw[q][x][0] = v.x, kw[q][x][1] = v.y, kw[q][x][2 % W] = v.z, kw[q][x][3 % W] = v.w;
        ks[q][x] = *reinterpret_cast<const uint16_t *>(src + kv4_k_scale<D>(tok, 2 * t));
      } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(src + kv4_k_code<D>(tok, t * 8));
        kw[q][x][0] = v.x, kw[q][x][1] = v.y;
        ks[q][x] = src[kv4_k_scale<D>(tok, t)];
      }
    }
  };
  auto loaded = [&]() {
    ++ahead_i;
    if (--ahead_left > 0 && ahead_i == kLook)
      for (int i = 0; i < kLook; ++i) next_unit(c, ahead);
  };
  look();
#pragma unroll
  for (int q = 0; q < kGroups; ++q) load(q);
  loaded();

  uint2 qf[NQ][KS];              // B operand: lane (g, t) = row g of the block, channels t D / 4 ...
  float rc[NQ][2], hi[NQ][2], wt[NQ][2];
  int last[NQ][2];
  int at_b = -1, at_h = -1, slot = -1, scored = 0, rows_b = 0;
  bool some_out = false;         // a row's lse is -infinity: its query may be anything, NaN too
  for (; left > 0; --left) {
    if (cur.b != at_b || cur.h != at_h) {
      // ---- another sequence or head: its rows
      const Kv4Seq s = kv4_seq(c, cur.b);
      const int n = s.q1 - s.q0, R = n * G;
      if (cur.b != at_b) {
        slot = score_slot(p, cur.b, s.len);
        if (slot >= 0 && slot_twice(p, cur.b, slot, lane)) slot = -1;
        scored = p.scored ? p.scored[cur.b] : s.len;
        rows_b = n;
      }
      at_b = cur.b;
      at_h = cur.h;
      some_out = false;
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
        const int row = nq * 8 + g, tok = row / G;
        const bool have = row < R;
        uint4 w[W];
        const uint16_t *src = p.q + (long long)(s.q0 + tok) * p.q_stride + (long long)(cur.h * G + row - tok * G) * D + t * (D / 4);
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = have ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
        const float lse = have ? p.lse[(long long)(s.q0 + tok) * p.Hq + cur.h * G + row - tok * G] : -INFINITY;
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) mx = max(mx, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
        }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = min(140 - (int)(mx >> 7), 60);
        const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          uint32_t y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            y[j] = h2u(__floats2half2_rn(__uint_as_float(x[j] << 16) * sc, __uint_as_float(x[j] & 0xFFFF0000u) * sc));
          qf[nq][2 * i] = make_uint2(y[0], y[1]);
          qf[nq][2 * i + 1] = make_uint2(y[2], y[3]);
        }
        // columns 2t and 2t + 1 are rows 2t and 2t + 1 of this block: held by lanes 4 (2t), 4 (2t + 1)
        const RowWeight rw = row_weight(lse, skew);
        const int sees = lse == -INFINITY ? -1 : s.len - n + tok;
        some_out |= __any_sync(0xffffffffu, have && lse == -INFINITY) != 0;
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          // (a row that is none, or saw nothing: 0 throughout)
          rc[nq][e2] = c2 * __shfl_sync(0xffffffffu, sees < 0 ? 0.0f : __uint_as_float((uint32_t)(127 - e) << 23), (2 * t + e2) * 4);
          hi[nq][e2] = __shfl_sync(0xffffffffu, rw.hi, (2 * t + e2) * 4);
          wt[nq][e2] = __shfl_sync(0xffffffffu, rw.w, (2 * t + e2) * 4);
          last[nq][e2] = __shfl_sync(0xffffffffu, sees, (2 * t + e2) * 4);
        }
      }
    }
    // this lane writes tokens g and g + 8 of group t
    const size_t row = ((size_t)max(slot, 0) * c.Hkv + cur.h) * p.s.tokens;
    float old[2];
    int pos[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      pos[x] = cur.pos + t * 16 + g + 8 * x;
      old[x] = slot >= 0 && pos[x] < min(scored, cur.len) ? p.s.in[row + pos[x]] : 0.0f;
    }
    const bool edge = some_out || cur.pos + kUnit > cur.len - rows_b + 1;
    const bool more = left > 1;
    if (more) look();
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      float d[NQ][4];
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[nq][j] = 0.0f;
      const uint32_t sa = e4m3x2(ks[q][0]), sb = e4m3x2(ks[q][1]);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t xa[4], xb[4];
        decode8(kw[q][0][w], w < 2 ? __low2half2(u2h(sa)) : __high2half2(u2h(sa)), xa);
        decode8(kw[q][1][w], w < 2 ? __low2half2(u2h(sb)) : __high2half2(u2h(sb)), xb);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
            mma_acc(d[nq], xa[2 * i], xb[2 * i], xa[2 * i + 1], xb[2 * i + 1], qf[nq][2 * w + i].x, qf[nq][2 * w + i].y);
      }
      if (more) load(q);
      float v[2] = {0.0f, 0.0f};
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float z = ex2(fmaf(d[nq][2 * x + e2], rc[nq][e2], -hi[nq][e2]));
            if (!edge || cur.pos + q * 16 + g + 8 * x <= last[nq][e2]) v[x] = fmaf(z, wt[nq][e2], v[x]);
          }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        v[x] += __shfl_xor_sync(0xffffffffu, v[x], 1);
        v[x] += __shfl_xor_sync(0xffffffffu, v[x], 2);
        if (t == q) old[x] += v[x];
      }
    }
    if (more) loaded();
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (slot >= 0 && pos[x] < cur.len) p.s.out[row + pos[x]] = old[x];
    if (more) next_unit(c, cur);
  }
}

// ---------------------------------------------------------------- many rows: tiles of 128 tokens by 128 rows
// S^T = K Q^T on tcgen05, a token per lane of tensor memory and a row per column: a
// thread adds its token's weights over the columns, and nothing crosses lanes. An
// item is 128 tokens of a sequence and KV head against the tiles of rows (tokens x
// the KV head's query heads) that see any of them. All items' tiles, in order, are
// cut into runs of equal cost, one per CTA (one per SM); what a run has of an item
// that it does not hold whole goes to the workspace and kv4_score_join_kernel adds
// the pieces in order. Within a CTA:
//   warps 0..11       weights, four warps a tile, a thread per token: three tiles at once
//                     for the exponentials' latency (with two, and K in shared memory, 225 us
//                     instead of 191 for the chunks below)
//   warps 12..15      decode an item's K into the A operand in tensor memory, BF16,
//                     exactly (from shared memory it would take half of its bandwidth)
//   warp 16           TMEM allocation; one thread issues the MMAs
//   warp 17           streams row tiles by TMA, as they came (BF16, the B operand)
//   warps 18, 19      the rows' lse in bits, of every other tile. A row whose lse is -infinity
//                     weighs nothing, its z being -infinity, unless its query is no number or too
//                     large for one: it is overwritten with zeros before the MMAs
// Measured: two chunks of 4096 and 789 tokens, 32 query heads on 8 of d = 128, over
// 8100 and 2221 cached: 168 us, 1.28 PFLOP/s, 0.67 of a large BF16 product; no unit is
// full (exponentials and tensor pipe 57%, issue 62%): a tile's products and weights
// wait for one another, with three of them in flight. Four windows of 64 rows on up to
// 16001 tokens: 38 us, 1.4 us an item of two tiles per CTA, of which each role's own code
// for an item -- a few hundred instructions of one warp per scheduler -- takes most. Every
// wait is bounded; one that gives up sets GDN_E_TIMEOUT and an abort flag that ends every
// role's loop.
constexpr int kTok = 128, kRow = 128;
constexpr int kAccs = 3;          // tiles of sums in tensor memory, 128 columns each: one for each four warps
constexpr int kWeigh = 4 * kAccs; // warps
constexpr int kTileThreads = 32 * (kWeigh + 8);
constexpr int kKCol = kAccs * kRow;  // TMEM column of the two items' K
constexpr int kLses = 8;          // tiles whose rows' lse is in shared memory
constexpr int kTileItem = 8;      // what an item costs beside its tiles, in tiles (some of them are masked): 1, 4, 8 and 12
                                  // gave 196, 169, 167 and 170 us for the chunks above
constexpr int kOpen = 4;          // items whose sums are not all there

struct ScoreInfo {  // of a run: what it leaves to be joined
  int head;         // its first part continues an item: 0 no, 1 and does not end it, 2 and ends it
  int tail;         // its last part begins an item that it does not end
  int b, h, kt;     // that item
};
struct TileKv4 {
  Kv4ScoreArgs a;
  int G, tpt;       // query heads per KV head; tokens of a row tile: 128 / G
  uint32_t inv_g;   // ceil(2^16 / G): x / G = x inv_g >> 16 for x < 128
  float c2, skew;
  float *pieces;    // [runs][head, tail][128]
  ScoreInfo *info;  // [runs]
};

// A sequence's rows and tokens. Its item kt: tokens [128 kt, ...), row tiles [first(kt), tiles).
struct ScoreSeq {
  int q0, n, len, tiles, items, tpt;
  GDN_DEV ScoreSeq(const TileKv4 &p, int b) : tpt(p.tpt) {
    const Kv4Seq s = kv4_seq(p.a.c, b);
    q0 = s.q0;
    n = s.q1 - s.q0;
    len = s.len;
    tiles = (int)((unsigned)(n + tpt - 1) / (unsigned)tpt);
    items = (len + kTok - 1) / kTok;
  }
  GDN_DEV int first(int kt) const {
    const int row = kt * kTok - (len - n);  // the first row (token) that sees any of them
    return row > 0 ? (int)((unsigned)row / (unsigned)tpt) : 0;
  }
  // The cost of items before kt for a KV head, in tiles x tpt, the tiles before the first one taken as a fraction.
  GDN_DEV long long cost(int kt) const {
    const long long o = len - n, k = kt, f = o >= 0 ? o / kTok + 1 : 0;
    return k * (kTileItem + tiles) * tpt - (k > f ? 64 * (k * (k - 1) - f * (f - 1)) - o * (k - f) : 0);
  }
};
struct ScorePlace {
  int b, h, kt, r;  // an item, and a tile of it from its first one
  GDN_DEV bool same_item(const ScorePlace &o) const { return b == o.b && h == o.h && kt == o.kt; }
};
// The place at cost u; b = B past the end. total: all items' cost. A whole warp.
GDN_DEV ScorePlace find_score(const TileKv4 &p, long long u, int lane, long long &total) {
  const Kv4Args &c = p.a.c;
  ScorePlace k{c.B, 0, 0, 0};
  total = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    long long own = 0;
    if (b0 + lane < c.B) {
      const ScoreSeq s(p, b0 + lane);
      own = s.cost(s.items) * c.Hkv;
    }
    long long incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, total + incl > u);
    if (k.b == c.B && past) {
      const int l = __ffs(past) - 1;
      k.b = b0 + l;
      long long off = u - total - __shfl_sync(0xffffffffu, incl - own, l);
      const ScoreSeq s(p, k.b);
      const long long head = s.cost(s.items);
      k.h = (int)(off / head);
      off -= k.h * head;
      int lo = 0, hi = s.items;  // cost(lo) <= off < cost(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.cost(mid) <= off) lo = mid; else hi = mid;
      }
      k.kt = lo;
      k.r = min(s.tiles - s.first(lo), max(0, (int)((off - s.cost(lo)) / p.tpt) - kTileItem));
    }
    total += __shfl_sync(0xffffffffu, incl, 31);
  }
  return k;
}

// Asynchronous copies of B bytes by the thread for itself; the rest of them, from `have` on, becomes zeros.
template <int B>
GDN_DEV void async_copy(void *dst, const void *src, int have) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(B), "r"(have) : "memory");
}
GDN_DEV void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
GDN_DEV void async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D>
struct TileShape {
  static constexpr int kBytesTile = 128 * D * 2;        // 128 rows
  static constexpr int kQs = D == 128 ? 6 : 8;          // row tiles on their way
  static_assert(kKCol + 2 * (D / 2) <= 512, "tensor memory");
  static constexpr int kToken = D / 2 + 16;             // a token's K bytes as they come: an odd number of 16-byte words
  static constexpr int kConst = kLses * kRow * 4;       // -lse in bits of the tiles' rows
  // the barriers, then the tensor memory's address and the abort flag, the run's ends
  static constexpr int kBars = 512, kBarriers = 4 + 2 * kQs + 2 * kAccs + 2 * kLses + 2 * kOpen + 1;
  static_assert(kBarriers * 8 + 8 + 2 * sizeof(ScorePlace) <= kBars, "barriers");
  static constexpr int kBytes = kQs * kBytesTile + kConst + kOpen * kAccs * kTok * 4 + 2 * kTok * kToken + kBars;
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};

template <int D>
__global__ void __launch_bounds__(kTileThreads, 1) kv4_score_tile_kernel(const __grid_constant__ CUtensorMap tmQ, TileKv4 p) {
  using S = TileShape<D>;
  constexpr int NQ = S::kQs;
  extern __shared__ __align__(1024) uint8_t sm[];  // the swizzled tiles start on 1024 bytes
  uint8_t *qbuf = sm;
  float *row_hi = reinterpret_cast<float *>(qbuf + NQ * S::kBytesTile);  // [kLses][128]
  float *parts = row_hi + kLses * kRow;                                  // [kOpen][kAccs][128]: each four warps' sums
  uint8_t *kbytes = reinterpret_cast<uint8_t *>(parts + kOpen * kAccs * kTok);  // [2][128][kToken]
  uint64_t *k_full = reinterpret_cast<uint64_t *>(kbytes + 2 * kTok * S::kToken), *k_free = k_full + 2;
  uint64_t *q_full = k_free + 2, *q_free = q_full + NQ;
  uint64_t *acc_full = q_free + NQ, *acc_free = acc_full + kAccs, *row_full = acc_free + kAccs, *row_free = row_full + kLses,
           *item_full = row_free + kLses, *item_free = item_full + kOpen, *fin = item_free + kOpen;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(fin + 1);
  volatile uint32_t *abort_flag = tmem_holder + 1;
  ScorePlace *ends = reinterpret_cast<ScorePlace *>(tmem_holder + 2);  // [2]
  const Kv4Args &c = p.a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 128);
      mbar_init(k_free + i, 1);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_free + i, 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_free + i, 128);
    }
    for (int i = 0; i < kLses; ++i) {
      mbar_init(row_full + i, 32);
      mbar_init(row_free + i, 128);
    }
    for (int i = 0; i < kOpen; ++i) {
      mbar_init(item_full + i, 32 * kWeigh);
      mbar_init(item_free + i, 128);
    }
    mbar_init(fin, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (p.tpt * p.G < kRow) {  // rows that no copy fills: zeros, so that what comes of them is a number
    for (int i = tid; i < NQ * S::kBytesTile / 16; i += kTileThreads) reinterpret_cast<uint4 *>(qbuf)[i] = make_uint4(0, 0, 0, 0);
    fence_async_shared();
  }
  if (warp == kWeigh + 4) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  kv4_begin();
  if (warp < 2) {  // the run's two ends
    long long total = 0;
    find_score(p, 0x7fffffffffffffffLL, lane, total);
    const long long x = blockIdx.x + warp, n = gridDim.x;
    const ScorePlace k = find_score(p, total / n * x + total % n * x / n, lane, total);
    if (lane == 0) ends[warp] = k;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const ScorePlace from = ends[0], to = ends[1];
  auto wait = [&](uint64_t *bar, uint32_t use) { return wait_or_abort(bar, use & 1u, abort_flag, c.status, c.wait); };
  auto warp_wait_all = [&](uint64_t *bar, uint32_t use) { return __all_sync(0xffffffffu, wait(bar, use)) != 0; };
  // For each item of the run with what the run has of it: f(place, sequence, the first row tile, one past the last,
  // whether that is all), until it returns false.
  auto items = [&](auto f) {
    ScorePlace k = from;
    while (k.b < c.B) {
      const ScoreSeq s(p, k.b);
      for (; k.h < c.Hkv; ++k.h, k.kt = 0)
        for (; k.kt < s.items; ++k.kt) {
          const bool last = k.same_item(to);
          if (last && to.r == 0) return;
          const int t0 = s.first(k.kt), all = s.tiles - t0;
          const int r0 = k.same_item(from) ? from.r : 0, r1 = last ? to.r : all;
          if (r0 == 0 || r0 < r1) {
            if (!f(k, s, t0 + r0, t0 + r1, r0 == 0 && r1 == all)) return;
          }
          if (last) return;
        }
      k.h = 0;
      ++k.b;
    }
  };
  if (tid == 0) {
    ScoreInfo x{0, 0, to.b, to.h, to.kt};
    const bool one = from.same_item(to);
    if (from.b < c.B && from.r > 0) {
      const ScoreSeq s(p, from.b);
      const int all = s.tiles - s.first(from.kt), r1 = one ? to.r : all;
      if (from.r < r1) x.head = r1 == all ? 2 : 1;
    }
    if (to.b < c.B && to.r > 0 && !(one && from.r > 0)) {
      const ScoreSeq s(p, to.b);
      if (to.r < s.tiles - s.first(to.kt)) x.tail = 1;
    }
    p.info[blockIdx.x] = x;
  }

  if (warp < kWeigh) {
    // ------------------------------------------------ weights: thread = token r; tiles u with u % kAccs == i
    const uint32_t i = warp >> 2, r = tid & 127;
    const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t u = 0, it = 0;
    int at_b = -1, slot = -1, scored = 0;
    // The item before the last, where these four warps add its sums up: by then the others' are there.
    struct {
      bool on = false;
      uint32_t it = 0;
      float old = 0.0f, *dst = nullptr;  // null: goes nowhere
    } open;
    auto close = [&]() {
      const uint32_t e = open.it % kOpen;
      if (!warp_wait_all(item_full + e, open.it / kOpen)) return false;
      float v = 0.0f;
#pragma unroll
      for (int x = 0; x < kAccs; ++x) v += parts[(e * kAccs + x) * kTok + r];
      mbar_arrive(item_free + e);
      if (open.dst) *open.dst = open.old + v;
      open.on = false;
      return true;
    };
    items([&](const ScorePlace &w, const ScoreSeq &s, int t0, int t1, bool whole) {
      if (w.b != at_b) {
        at_b = w.b;
        slot = score_slot(p.a, w.b, s.len);
        if (slot >= 0 && slot_twice(p.a, w.b, slot, lane)) slot = -1;
        scored = p.a.scored ? p.a.scored[w.b] : s.len;
      }
      const int pos = w.kt * kTok + r;
      const bool mine = it % kAccs == i;  // these four warps close the item
      float old = 0.0f, *dst = nullptr;
      if (mine) {
        const size_t at = ((size_t)max(slot, 0) * c.Hkv + w.h) * p.a.s.tokens + pos;
        if (!whole) {
          dst = p.pieces + ((size_t)blockIdx.x * 2 + (w.same_item(from) && from.r > 0 ? 0 : 1)) * kTok + r;
        } else if (slot >= 0 && pos < s.len) {
          dst = p.a.s.out + at;
          if (pos < scored) old = p.a.s.in[at];
        }
      }
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      for (int t = t0; t < t1; ++t, ++u) {
        if (u % kAccs != i) continue;
        const uint32_t e8 = u % kLses;
        if (!warp_wait_all(row_full + e8, u / kLses) || !warp_wait_all(acc_full + i, u / kAccs)) return false;
        tc_fence_after();
        // whole tiles: every row sees every token; their rows that are none have hi = -infinity
        const bool mask = (w.kt + 1) * kTok - 1 > s.len - s.n + t * p.tpt || (t + 1) * p.tpt > s.n;
        // the tile's columns that see this token: from its first row that does, and only those that are rows
        const int lo = max(0, pos - (s.len - s.n) - t * p.tpt) * p.G;
        const unsigned width = (unsigned)max(0, (s.n - t * p.tpt) * p.G - lo);
        const float2 c2 = make_float2(p.c2, p.c2);
        const float4 *hi = reinterpret_cast<const float4 *>(row_hi + e8 * kRow);
        const uint32_t acc = base + i * kRow;
        auto weigh = [&](const uint32_t(&y)[16], int q, auto masked) {  // columns 16 q ..
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 h = hi[q * 4 + e];
            float2 z0 = fma2(make_float2(__uint_as_float(y[4 * e]), __uint_as_float(y[4 * e + 1])), c2, make_float2(h.x, h.y));
            float2 z1 = fma2(make_float2(__uint_as_float(y[4 * e + 2]), __uint_as_float(y[4 * e + 3])), c2, make_float2(h.z, h.w));
            z0.x = ex2(z0.x), z0.y = ex2(z0.y), z1.x = ex2(z1.x), z1.y = ex2(z1.y);
            if constexpr (masked()) {
              auto sees = [&](int col) { return (unsigned)(col - lo) < width; };
              z0.x = sees(q * 16 + 4 * e) ? z0.x : 0.0f;
              z0.y = sees(q * 16 + 4 * e + 1) ? z0.y : 0.0f;
              z1.x = sees(q * 16 + 4 * e + 2) ? z1.x : 0.0f;
              z1.y = sees(q * 16 + 4 * e + 3) ? z1.y : 0.0f;
            }
            sum[0] = add2(sum[0], z0);
            sum[1] = add2(sum[1], z1);
          }
        };
        uint32_t x[2][16];
        tmem_ld16(acc, x[0]);
        if (mask) {
#pragma unroll 1
          for (int q = 0; q < 8; q += 2) {
            tmem_ld_wait();
            tmem_ld16(acc + 16 * (q + 1), x[1]);
            weigh(x[0], q, std::true_type{});
            tmem_ld_wait();
            if (q < 6) tmem_ld16(acc + 16 * (q + 2), x[0]);
            weigh(x[1], q + 1, std::true_type{});
          }
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            tmem_ld_wait();
            if (q < 7) tmem_ld16(acc + 16 * (q + 1), x[(q + 1) & 1]);
            weigh(x[q & 1], q, std::false_type{});
          }
        }
        tc_fence_before();
        mbar_arrive(acc_free + i);
        mbar_arrive(row_free + e8);
      }
      const float2 v = add2(sum[0], sum[1]);
      const uint32_t e = it % kOpen;
      if (it >= kOpen && !warp_wait_all(item_free + e, it / kOpen - 1)) return false;
      parts[(e * kAccs + i) * kTok + r] = v.x + v.y;
      mbar_arrive(item_full + e);
      if (open.on && !close()) return false;
      if (mine) {
        open.on = true;
        open.it = it;
        open.old = old;
        open.dst = dst;
      }
      ++it;
      return true;
    });
    if (open.on) close();
  } else if (warp < kWeigh + 4) {
    // ------------------------------------------------ K: a thread per token, 2 BF16 a column
    const int r = tid & 127;
    const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kKCol;
    constexpr int W = D / 8;  // words of eight codes
    // A token's bytes go to shared memory two items ahead, by and for its own thread. (Loops are kept short: the roles'
    // code, all of it in use at once, has to fit the instruction caches.)
    uint8_t *mine = kbytes + r * S::kToken;
    uint32_t it = 0;
    auto convert = [&](uint32_t it) {
      const uint32_t st = it & 1;
      const uint8_t *src = mine + st * (kTok * S::kToken);
      if (it >= 2 && !warp_wait_all(k_free + st, it / 2 - 1)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int y = 0; y < W / 4; ++y) {  // 32 channels, 16 columns
        const uint4 v4 = *reinterpret_cast<const uint4 *>(src + 16 * y);
        const uint32_t code[4] = {v4.x, v4.y, v4.z, v4.w}, sc = *reinterpret_cast<const uint16_t *>(src + D / 2 + 2 * y);
        uint32_t o[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // an FP16 code moved down 3 bits is the BF16 value 2^-112 times as large; the scale (at most 448) makes that good
          const float f = e4m3_to_f32(sc >> (8 * (j / 2))) * 5.192296858534828e33f;  // 2^112
          const __nv_bfloat162 f2 = __float2bfloat162_rn(f);
          __half2 e[4];
          e2m1x8_to_h2x4(code[j], e);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t v = h2u(e[q]);
            uint32_t u = ((v >> 3) & 0x0FFF0FFFu) | (v & 0x80008000u);
            const __nv_bfloat162 z = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&u), f2);
            o[4 * j + q] = *reinterpret_cast<const uint32_t *>(&z);
          }
        }
        tmem_st16(base + st * (D / 2) + 16 * y, o);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(k_full + st);
      return true;
    };
    // where an item's token lies: looked up an item before its bytes are asked for, so that nothing waits for the
    // page id (those windows 39 -> 36 us)
    struct Found {
      int page, within, h;
      bool in;
    } found{};
    auto fetch = [&](uint32_t it) {
      const bool bad = found.page < 0 || found.page >= c.num_pages;
      if (found.in && bad) flag_status(c.status, GDN_E_RANGE);
      const int have = found.in && !bad ? 16 : 0;  // none: zeros
      const uint8_t *g = c.pages;
      if (have) g += ((size_t)found.page * c.Hkv * (c.page_tokens / 16) + found.within / 16) * (18 * D) + found.h * kv4_head_bytes<D>(c);
      uint8_t *dst = mine + (it & 1) * (kTok * S::kToken);
#pragma unroll
      for (int y = 0; y < W / 4; ++y) async_copy<16>(dst + 16 * y, g + kv4_k_code<D>(r & 15, 0) + 16 * y, have);
      async_copy<D / 16>(dst + D / 2, g + kv4_k_scale<D>(r & 15, 0), min(have, D / 16));
      async_commit();
    };
    bool ok = true;
    items([&](const ScorePlace &w, const ScoreSeq &s, int, int, bool) {
      const int pos = w.kt * kTok + r, col = pos / c.page_tokens;
      Found f{0, pos - col * c.page_tokens, w.h, pos < s.len};
      if (f.in) f.page = c.table[(size_t)w.b * c.cols + col];
      if (it > 0) fetch(it - 1);
      if (it > 1) {
        async_wait<1>();
        ok = convert(it - 2);
      }
      found = f;
      ++it;
      return ok;
    });
    if (ok && it > 0) fetch(it - 1);
    if (ok && it > 1) {
      async_wait<1>();
      ok = convert(it - 2);
    }
    async_wait<0>();
    if (ok && it > 0) convert(it - 1);
  } else if (warp == kWeigh + 4) {
    // ------------------------------------------------ MMAs
    constexpr uint32_t id = idesc_bf16(kRow);
    constexpr uint64_t kStep = S::kBytesTile / 16;  // from one stage to the next, in a descriptor
    const uint64_t qd = desc_sw128(smem_u32(qbuf));
    const bool me = elect_one();
    uint32_t u = 0, it = 0;
    items([&](const ScorePlace &, const ScoreSeq &, int t0, int t1, bool) {
      bool ok = true;
      if (me) {
        ok = wait(k_full + (it & 1), it / 2);
        for (int t = t0; t < t1 && ok; ++t) {
          const uint32_t v = u + (t - t0), a = v % kAccs, q = v % NQ;
          ok = wait(q_full + q, v / NQ) && wait(row_full + v % kLses, v / kLses) && (v < kAccs || wait(acc_free + a, v / kAccs - 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t qq = qd + (uint64_t)q * kStep;
          const uint32_t d = tmem + a * kRow, kk = tmem + kKCol + (it & 1) * (D / 2);
          mma_f16_ts_c<false>(d, kk, qq, id);
#pragma unroll
          for (int k = 1; k < D / 16; ++k)
            mma_f16_ts_c<true>(d, kk + 8 * k, qq + (k / 4) * (kRow * 128 / 16) + 2 * (k & 3), id);
          tc_commit(acc_full + a);
          tc_commit(q_free + q);
        }
        if (ok) tc_commit(k_free + (it & 1));
      }
      u += t1 - t0;
      ++it;
      return __any_sync(0xffffffffu, me && ok) != 0;
    });
    // every MMA issued has completed before the CTA may leave
    if (me) {
      tc_commit(fin);
      mbar_wait(fin, 0u);
    }
  } else if (warp == kWeigh + 5) {
    // ------------------------------------------------ row tiles
    uint32_t u = 0;
    items([&](const ScorePlace &w, const ScoreSeq &s, int t0, int t1, bool) {
      bool ok = true;
      for (int t = t0; t < t1; ++t, ++u) {
        const uint32_t q = u % NQ;
        if (u >= NQ && !(ok = warp_wait_all(q_free + q, u / NQ - 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full + q, p.tpt * p.G * D * 2);
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tma_load_3d(qbuf + q * S::kBytesTile + x * (kRow * 128), &tmQ, x * 64, w.h * p.G, s.q0 + t * p.tpt, q_full + q);
        }
        __syncwarp();
      }
      return ok;
    });
    // the last copies land (or a bounded wait for each ends) before the CTA leaves, whoever gives up when
    if (lane == 0)
      for (uint32_t x = u < NQ ? 0 : u - NQ; x < u; ++x) mbar_wait(q_full + x % NQ, (x / NQ) & 1u);
  } else {
    // ------------------------------------------------ what the tiles' rows are weighed by: tiles u with u % 2 == warp % 2
    uint32_t u = 0;
    items([&](const ScorePlace &w, const ScoreSeq &s, int t0, int t1, bool) {
      unsigned out = 0;  // of a lane's four rows of the tile looked up last: those that are left out
      auto lses = [&](int t, float (&hi)[4]) {
        out = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int x = lane + 32 * j, over = (int)(x * p.inv_g >> 16), tok = t * p.tpt + over;
          const bool have = x < p.tpt * p.G && tok < s.n;
          hi[j] = have ? p.a.lse[(long long)(s.q0 + tok) * p.a.Hq + w.h * p.G + x - over * p.G] : -INFINITY;
          out |= (unsigned)(have && hi[j] == -INFINITY) << j;
        }
      };
      float next[4];
      const int mine = t0 + ((u ^ warp) & 1);
      if (mine < t1) lses(mine, next);
      for (int t = mine; t < t1; t += 2) {
        const uint32_t v = u + (t - t0), e8 = v % kLses;
        float hi[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)  // a row that saw nothing, or is none, adds nothing
          hi[j] = next[j] == -INFINITY ? -INFINITY : -fmaf(next[j], kLog2e, next[j] * (1.925963e-8f - p.skew * kLog2e));
        // (A copy of the weighing for such tiles instead: the windows 39.1 us, the chunks 182; one that found NaN in a
        // tile's sum and weighed it again 39.5 and 183; this 38.5 and 178, before such rows were looked at 36.9 and 177.)
        if (__any_sync(0xffffffffu, out != 0)) {
          const uint32_t q = v % NQ;
          if (!warp_wait_all(q_full + q, v / NQ)) return false;
#pragma unroll 1
          for (int j = 0; j < 4; ++j)
            if (out >> j & 1)
              for (int x = 0; x < D / 64 * 8; ++x)  // a row has 128 bytes in each 64 channels' part
                *reinterpret_cast<uint4 *>(qbuf + q * S::kBytesTile + x / 8 * (kRow * 128) + (lane + 32 * j) * 128 + x % 8 * 16) =
                    make_uint4(0, 0, 0, 0);
          fence_async_shared();
        }
        if (t + 2 < t1) lses(t + 2, next);
        if (v >= kLses && !warp_wait_all(row_free + e8, v / kLses - 1)) return false;
#pragma unroll
        for (int j = 0; j < 4; ++j) row_hi[e8 * kRow + lane + 32 * j] = hi[j];
        mbar_arrive(row_full + e8);
      }
      u += t1 - t0;
      return true;
    });
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWeigh + 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A CTA per run: the item that it begins and does not end, its pieces in order.
__global__ void __launch_bounds__(kTok) kv4_score_join_kernel(TileKv4 p, int runs) {
  kv4_begin();
  const Kv4Args &c = p.a.c;
  const ScoreInfo x = p.info[blockIdx.x];
  if (!x.tail) return;
  const int r = threadIdx.x, pos = x.kt * kTok + r, len = kv4_len(c, x.b);
  float v = p.pieces[((size_t)blockIdx.x * 2 + 1) * kTok + r];
  for (int y = blockIdx.x + 1; y < runs; ++y) {
    const int head = p.info[y].head;
    if (head) v += p.pieces[(size_t)y * 2 * kTok + r];
    if (head == 2) break;
  }
  const int slot = score_slot(p.a, x.b, len);
  if (slot < 0 || slot_twice(p.a, x.b, slot, r & 31) || pos >= len) return;
  const int scored = p.a.scored ? p.a.scored[x.b] : len;
  const size_t at = ((size_t)slot * c.Hkv + x.h) * p.a.s.tokens + pos;
  p.a.s.out[at] = v + (pos < scored ? p.a.s.in[at] : 0.0f);
}

// Rows of one sequence and KV head that a call may have, at most.
int most_rows(const Kv4ScoreArgs &p) {
  const Kv4Args &c = p.c;
  return (c.q_start ? c.T : c.T / c.B) * (p.Hq / c.Hkv);
}

template <int D, int NQ>
cudaError_t launch_rows(const Kv4ScoreArgs &p, float c2, float skew, int num_sms, cudaStream_t stream) {
  const Kv4Args &c = p.c;
  const long long units = (long long)c.B * c.Hkv * (((long long)c.cols * c.page_tokens + kUnit - 1) / kUnit);  // at most
  const int most = num_sms * (NQ == 1 ? 2 : 1);
  return kv4_launch(kv4_score_rows_kernel<D, NQ>, (unsigned)std::min((long long)most, (units + kRowWarps - 1) / kRowWarps),
                    32 * kRowWarps, 0, stream, p, c2, skew);
}

// CTAs: no more than there can be tiles.
int tile_runs(const Kv4ScoreArgs &a, int num_sms) {
  const Kv4Args &c = a.c;
  const long long tpt = kRow / (a.Hq / c.Hkv), tiles = (c.q_start ? c.T : c.T / c.B) / tpt + 1;
  const long long items = (long long)c.B * c.Hkv * (((long long)c.cols * c.page_tokens + kTok - 1) / kTok);
  return (int)(items >= num_sms ? num_sms : std::min((long long)num_sms, items * tiles));
}

template <int D>
cudaError_t launch_tile(const TileKv4 &p, int num_sms, cudaStream_t stream) {
  using S = TileShape<D>;
  CUtensorMap tmQ;
  if (!make_heads_map(&tmQ, p.a.q, p.a.c.T, p.a.Hq, D, p.a.q_stride, p.tpt, p.G)) return cudaErrorInvalidValue;
  static bool allowed[64];
  cudaError_t e = kv4_allow_smem(kv4_score_tile_kernel<D>, S::kBytes, allowed);
  if (e != cudaSuccess) return e;
  const int runs = tile_runs(p.a, num_sms);
  e = kv4_launch(kv4_score_tile_kernel<D>, runs, kTileThreads, S::kBytes, stream, tmQ, p);
  if (e != cudaSuccess || runs == 1) return e;
  return kv4_launch(kv4_score_join_kernel, runs - 1, kTok, 0, stream, p, runs);
}

}  // namespace

size_t kv4_score_bytes(const Kv4ScoreArgs &p, int num_sms) {
  return most_rows(p) <= 16 ? 0 : (size_t)tile_runs(p, num_sms) * (2 * kTok * sizeof(float) + sizeof(ScoreInfo));
}

cudaError_t launch_kv4_score(const Kv4ScoreArgs &p, void *workspace, int num_sms, cudaStream_t stream) {
  const Kv4Args &c = p.c;
  const double exact = (double)p.sm_scale * c.ks * 1.4426950408889634074;  // a score in bits
  const float c2 = (float)exact, skew = (float)(exact / c2 - 1.0);
  const int R = most_rows(p), G = p.Hq / c.Hkv;
  // 64 sequences of up to 8190 tokens, 8 KV heads of 128: 4 and 8 rows 38 us, 12 and 16 60, by tiles 176 whatever the rows
  // up to 64; 8 of them, 2 heads of 64: 8 rows 5.4, 16 5.6, by tiles 13.6. (Of ragged rows the host knows the sum only.)
  if (R <= 8) return c.D == 128 ? launch_rows<128, 1>(p, c2, skew, num_sms, stream) : launch_rows<64, 1>(p, c2, skew, num_sms, stream);
  if (R <= 16) return c.D == 128 ? launch_rows<128, 2>(p, c2, skew, num_sms, stream) : launch_rows<64, 2>(p, c2, skew, num_sms, stream);
  float *pieces = static_cast<float *>(workspace);
  const TileKv4 t{p, G, kRow / G, (65536u + G - 1) / G, c2, skew, pieces,
                  reinterpret_cast<ScoreInfo *>(pieces + (size_t)tile_runs(p, num_sms) * 2 * kTok)};
  return c.D == 128 ? launch_tile<128>(t, num_sms, stream) : launch_tile<64>(t, num_sms, stream);
}

}  // namespace gdn
