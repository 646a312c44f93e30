// Decode attention for sequences that share a prefix (include/gdn.h): a group's
// shared tokens are read once for all rows of the group, what follows them by
// kv4_decode's kernels, and the parts joined row by row:
//
//   out = sum_p 2^(m_p - m) O_p / sum_p 2^(m_p - m) l_p,  m = max_p m_p
//
// What bounds it: with the G r rows of many sequences on one cached token the
// prefix is a matrix product, 4 d operations per (row, token) on the tensor cores
// (from about 80 rows per KV head they take longer than the token's bytes), and
// beside them one 2^x per (row, token) and the decoding of the token's 2 d values.
#include <algorithm>
#include <type_traits>

#include "kv4.cuh"
#include "tc.cuh"

namespace gdn {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPlanThreads = 256;

// The workspace. Rows of one KV head are numbered row = (batch row) G + (query head of the group).
struct SharedWs {
  int32_t *own_len;    // [B]: a sequence's tokens behind its shared ones
  int32_t *own_table;  // [B][cols]: their pages
  int2 *seq_item;      // [B]: the first row of its group, and that row's item slot; -1: it shares nothing
  int32_t *len, *lead; // [groups]: shared tokens (0: none), the sequence through whose pages they are read
  float *own, *own_ml;   // [T][Hq][D], [T][Hq][2]: kv4_decode's sums and their (maximum, weight), whole items
  int32_t *ends;         // [Hkv][slots][2]: an item's first piece, or -1: it is whole; the run of its last piece
  float *pre, *pre_ml;   // whole items: [Hkv][D][rows], [Hkv][rows][2]
  float *part, *part_ml; // pieces [2 runs][D][ld], [2 runs][ld][2]
  void *decode;
};

struct SharedKv4 {
  Kv4SharedArgs s;
  SharedWs w;
  int r, G, rows;  // new tokens per sequence, query heads per KV head, T G
  int runs;        // CTAs of the prefix kernel
  int slots, ld;   // items of a KV head, at most; rows of a piece
  Kv4Pieces own;   // of what each sequence has for itself
};

constexpr int kItemRows = 256;  // query rows of an item: two tiles of 128

// Items of all KV heads together have at most this many tiles of 128 tokens.
long long prefix_tiles(const Kv4SharedArgs &s, int slots) {
  return (long long)s.a.c.Hkv * slots * ((std::min((long long)s.max_shared, (long long)s.a.c.cols * s.a.c.page_tokens) + 127) / 128);
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// The sizes of a call, its workspace laid out from `base` (which may be null), and how large that is.
size_t lay_out(const Kv4SharedArgs &s, uint8_t *base, int num_sms, SharedKv4 &p) {
  const Kv4Args &c = s.a.c;
  SharedWs &w = p.w;
  p.s = s;
  p.r = c.T / c.B;
  p.G = s.a.Hq / c.Hkv;
  p.rows = c.T * p.G;
  p.slots = p.rows / kItemRows + s.groups + 1;  // Place::slot
  p.ld = std::min(kItemRows, (p.rows + 31) / 32 * 32);
  p.runs = s.groups ? (int)std::min((long long)num_sms, prefix_tiles(s, p.slots)) : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t *p = base + at;
    at += up16(bytes);
    return p;
  };
  const size_t rows = p.rows, all = (size_t)c.T * s.a.Hq;
  w.own_len = reinterpret_cast<int32_t *>(take(4 * (size_t)c.B));
  w.own_table = reinterpret_cast<int32_t *>(take(4 * (size_t)c.B * c.cols));
  w.seq_item = reinterpret_cast<int2 *>(take(8 * (size_t)c.B));
  w.len = reinterpret_cast<int32_t *>(take(4 * (size_t)s.groups));
  w.lead = reinterpret_cast<int32_t *>(take(4 * (size_t)s.groups));
  w.own = reinterpret_cast<float *>(take(4 * all * c.D));
  w.own_ml = reinterpret_cast<float *>(take(8 * all));
  w.ends = reinterpret_cast<int32_t *>(take(8 * (size_t)c.Hkv * p.slots));
  w.pre = reinterpret_cast<float *>(take(4 * rows * c.Hkv * c.D));
  w.pre_ml = reinterpret_cast<float *>(take(8 * rows * c.Hkv));
  w.part = reinterpret_cast<float *>(take(8 * (size_t)p.runs * p.ld * c.D));
  w.part_ml = reinterpret_cast<float *>(take(16 * (size_t)p.runs * p.ld));
  w.decode = take(kv4_decode_bytes(s.a, num_sms, true));
  p.own = kv4_decode_pieces(s.a, w.decode, num_sms);
  return at;
}

// A CTA per sequence and one per group: what the group shares -- the least of its
// members' bounds, in whole pages -- and where the sequence's own tokens lie.
__global__ void __launch_bounds__(kPlanThreads) kv4_shared_plan_kernel(SharedKv4 p) {
  kv4_begin();
  const Kv4Args &c = p.s.a.c;
  const int32_t *start = p.s.group_start;
  const int tid = threadIdx.x, G = p.s.groups, b = blockIdx.x < c.B ? (int)blockIdx.x : -1;
  // the groups' bounds have to ascend within the batch: else nothing is shared
  int bad = 0, mine = b < 0 ? (int)blockIdx.x - c.B : -1;
  __shared__ int found;
  if (tid == 0) found = mine;
  __syncthreads();
  for (int g = tid; g < G; g += kPlanThreads) {
    const int x = start[g], y = start[g + 1];
    bad |= x < 0 || y < x || y > c.B;
    if (b >= 0 && x <= b && b < y) found = g;  // at most one g where they ascend
  }
  bad = __syncthreads_or(bad);
  if (bad) flag_status(c.status, GDN_E_RANGE);
  const int g = bad ? -1 : found;
  int S = 0, lead = -1;
  if (g >= 0) {
    S = min(p.s.shared_len[g], p.s.max_shared);
    if (S < 0) {
      flag_status(c.status, GDN_E_RANGE);
      S = 0;
    }
    int least = S, first = c.B, live = 0;  // live: members with tokens
    for (int i = start[g] + tid; i < start[g + 1]; i += kPlanThreads) {
      const int n = kv4_len(c, i);
      if (n > 0) {
        least = min(least, max(n - p.r + 1, 0));
        first = min(first, i);
        ++live;
      }
    }
    __shared__ int sl[kPlanThreads / 32], sf[kPlanThreads / 32], sn[kPlanThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
      live += __shfl_xor_sync(0xffffffffu, live, o);
    }
    if ((tid & 31) == 0) {
      sl[tid >> 5] = least;
      sf[tid >> 5] = first;
      sn[tid >> 5] = live;
    }
    __syncthreads();
    live = 0;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
      least = min(least, sl[i]);
      first = min(first, sf[i]);
      live += sn[i];
    }
    lead = first < c.B ? first : -1;
    // a group of one sequence with tokens, of rows that kv4_decode takes together, reads for itself: 5 of 38016 tokens,
    // 8 KV heads of 128, 40 us instead of 99 (2 of 512, 24 rows each, 19.3 instead of 17.6)
    const bool alone = live == 1 && p.own.groups == 1;
    S = lead < 0 || alone ? 0 : least / c.page_tokens * c.page_tokens;
  }
  if (b < 0) {
    if (tid == 0) {
      p.w.len[mine] = bad ? 0 : S;
      p.w.lead[mine] = lead;
    }
    return;
  }
  const int len = kv4_len(c, b), skip = len > 0 ? S : 0;
  if (tid == 0) {
    if (c.kv_len[b] != len) flag_status(c.status, GDN_E_RANGE);
    const int row0 = skip > 0 ? start[g] * p.r * p.G : -1;
    p.w.own_len[b] = len - skip;
    p.w.seq_item[b] = make_int2(row0, skip > 0 ? row0 / kItemRows + g : -1);
  }
  const int from = skip / c.page_tokens, pages = (len - skip + c.page_tokens - 1) / c.page_tokens;
  for (int i = tid; i < pages; i += kPlanThreads)  // (from + pages is at most cols: the length is checked)
    p.w.own_table[(size_t)b * c.cols + i] = c.table[(size_t)b * c.cols + from + i];
}

// ---------------------------------------------------------------- the shared tokens
// kv4_prefix_kernel: an item is 256 query rows of a group and KV head -- two tiles
// of 128, a row being (sequence, token, query head) -- against the group's shared
// tokens. All items' tiles of 128 tokens, in order, are cut into runs of equal
// cost, one per CTA (one per SM); a run's part of an item that it does not hold
// whole goes to the workspace as a piece. Within a CTA:
//   warps 0..3, 4..7  one row per thread: its query in FP16 (scaled by a power of
//                     two) to shared memory, then softmax of row tile 0 / 1, the
//                     weights back into tensor memory; the row's sums
//   warps 8..11       decode a tile's K from its 4-bit bytes into the MMAs' operand
//   warps 12..15      decode its V
//   warp 16           TMEM allocation; one thread issues the MMAs
//   warp 17           streams the cached bytes by bulk copies
// The softmax warps take over registers (160, 56 and 48 of 96 each), enough for half
// of a row's 128 scores at a time, which are read from tensor memory twice (with all
// of them in registers there was room for four decoding warps only, one on each
// scheduler, which then set the pace: 177 us instead of 150 for 1024 rows of each of 4
// KV heads on 65536 tokens, the whole call). K and V are exact in FP16 (six
// significant bits). Measured now, those rows: 103 us in this kernel, 1.33 PFLOP/s
// (0.70 of a large BF16 product); the tensor pipe is busy 62% of the time. Counted for two
// row tiles and 128 tokens, its products take 2048 cycles and shared memory about 2300
// (queries and K of S = Q K^T both come from there, and the decoded tiles go there); the
// rest is a row tile's chain of softmax and products, with two of them in flight.
// The weights are 2^(z - m + 6), with a maximum m that is only moved (and O
// rescaled in tensor memory) when a tile's weights come to 2^14 or more by it.
// Every wait is bounded; one that gives up sets GDN_E_TIMEOUT and an abort flag
// that ends every role's loop.
constexpr int kKv = 128;
constexpr int kPrefixThreads = 640;
constexpr float kShift = 6.0f, kMost = 16384.0f;
// What an item costs beside its tiles, in tiles: its queries, its sums and their joining.
constexpr int kItemCost = 2;
// Few long items are cut into less runs than there are CTAs, sqrt(16 tiles items): joining a piece takes about a
// sixteenth of a tile. One item of 17, 26 or 4 sequences, 274, 301 and 204 tiles: 43.9, 39.6 and 39.8 us by all CTAs,
// now 39.4, 28.4 and 31.9; by sqrt(8 ..) 38.1, 29.0 and 33.2, by sqrt(32 ..) 40.3, 31.3 and 35.1.
constexpr float kFewPieces = 16.0f;

template <int D>
struct PrefixShape {
  static constexpr int kStages = D == 128 ? 2 : 4;      // of K and of V each
  static constexpr int kTileBytes = kKv * D * 2;        // a K tile, a V tile, and 128 query rows
  static constexpr int kRaw = 4 * 18 * D, kRaws = D == 128 ? 3 : 6;  // 64 tokens' bytes as they come
  // the barriers, then the tensor memory's address and the abort flag, the run's first place, its ends
  static constexpr int kBarriers = 4 * kStages + 10 + 2 * kRaws + 1, kBars = 512;
  static_assert(kBarriers * 8 + 8 + 40 + 16 <= kBars, "barriers");
  static constexpr int kBytes = (2 + 2 * kStages) * kTileBytes + kRaws * kRaw + kBars;
  static constexpr int kO = 2 * kKv;                    // TMEM columns: S0, S1, then O0, O1
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};

// A place in the sequence of all tiles: an item, and a tile of it.
struct Place {
  int g, h, pair, tile;
  int nt, S, lead, row0, rows, pairs;  // the group's tiles and tokens, through whom; its first row, rows, items per KV head
  GDN_DEV void group(const SharedKv4 &p, int at) {
    g = at;
    S = p.w.len[g];
    lead = p.w.lead[g];
    nt = (S + kKv - 1) / kKv;
    const int first = p.s.group_start[g];
    row0 = first * p.r * p.G;
    rows = (p.s.group_start[g + 1] - first) * p.r * p.G;
    pairs = (rows + kItemRows - 1) / kItemRows;
  }
  GDN_DEV int item_row0() const { return row0 + pair * kItemRows; }
  GDN_DEV int item_rows() const { return min(kItemRows, rows - pair * kItemRows); }
  // Unique among the items of a KV head: each group takes at most rows / 256 + 1 places
  GDN_DEV int slot() const { return row0 / kItemRows + g + pair; }
  // The next item; only called while there is one.
  GDN_DEV void next(const SharedKv4 &p) {
    tile = 0;
    if (++pair < pairs) return;
    pair = 0;
    if (++h < p.s.a.c.Hkv) return;
    h = 0;
    int at = g + 1;
    while (p.w.len[at] == 0) ++at;
    group(p, at);
  }
};
static_assert(sizeof(Place) == 40, "what the prefix kernel's shared memory has for it");
// a / b, in 32 bits where they fit (64 bits take some 200 instructions)
GDN_DEV long long quot(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}
// Lane's group g0 + lane: its items' cost and tiles.
struct GroupCost {
  long long cost, tiles;
  int nt;
  GDN_DEV GroupCost(const SharedKv4 &p, int g) : cost(0), tiles(0), nt(0) {
    if (g >= p.s.groups) return;
    const int first = p.s.group_start[g], last = p.s.group_start[g + 1], S = p.w.len[g];
    if (S == 0) return;
    nt = (S + kKv - 1) / kKv;
    const long long items = (long long)(((last - first) * p.r * p.G + kItemRows - 1) / kItemRows) * p.s.a.c.Hkv;
    cost = items * (nt + kItemCost);
    tiles = items * nt;
  }
};
GDN_DEV long long warp_lsum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Cut `cut` of the runs' cuts: the tile there, and how many lie before it. No more
// runs than tiles: then the pieces of an item lie in neighbouring ones. A whole warp.
GDN_DEV long long find_cut(const SharedKv4 &p, int cut, int lane, Place &k) {
  const GroupCost mine(p, lane);  // of the first 32 groups
  long long total = warp_lsum(mine.cost), tiles = warp_lsum(mine.tiles);
  for (int g0 = 32; g0 < p.s.groups; g0 += 32) {
    const GroupCost x(p, g0 + lane);
    total += warp_lsum(x.cost);
    tiles += warp_lsum(x.tiles);
  }
  const long long items = (total - tiles) / kItemCost;
  const float fine = sqrtf(kFewPieces * (float)tiles * (float)items);
  const long long n = max(1LL, min(min((long long)gridDim.x, tiles), (long long)fine));
  if (cut >= n || tiles == 0) return tiles;
  const long long q = quot(total, n);
  long long u = q * cut + quot((total - q * n) * cut, n), before = 0;  // the cost at the cut, the tiles of the groups before
  for (int g0 = 0;; g0 += 32) {  // (ends: u < total)
    const GroupCost x = g0 == 0 ? mine : GroupCost(p, g0 + lane);
    long long incl = x.cost, tincl = x.tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o), z = __shfl_up_sync(0xffffffffu, tincl, o);
      if (lane >= o) {
        incl += y;
        tincl += z;
      }
    }
    const unsigned past = __ballot_sync(0xffffffffu, incl > u);
    if (past) {
      const int l = __ffs(past) - 1;
      k.group(p, g0 + l);
      const long long off = u - __shfl_sync(0xffffffffu, incl - x.cost, l), item = quot(off, k.nt + kItemCost);
      k.tile = max((int)(off - item * (k.nt + kItemCost)) - kItemCost, 0);  // an item's own cost comes before its tiles
      k.h = (int)quot(item, k.pairs);
      k.pair = (int)(item - (long long)k.h * k.pairs);
      return before + __shfl_sync(0xffffffffu, tincl - x.tiles, l) + item * k.nt + k.tile;
    }
    u -= __shfl_sync(0xffffffffu, incl, 31);
    before += __shfl_sync(0xffffffffu, tincl, 31);
  }
}

template <int D>
__global__ void __launch_bounds__(kPrefixThreads, 1) kv4_prefix_kernel(SharedKv4 p) {
  using S = PrefixShape<D>;
  constexpr int NS = S::kStages, NR = S::kRaws;
  extern __shared__ __align__(1024) uint8_t sm[];  // the swizzled tiles start on 1024 bytes
  uint8_t *qs = sm, *kbuf = sm + 2 * S::kTileBytes, *vbuf = kbuf + NS * S::kTileBytes, *raw = vbuf + NS * S::kTileBytes;
  uint64_t *k_full = reinterpret_cast<uint64_t *>(raw + NR * S::kRaw);
  uint64_t *v_full = k_full + NS, *k_free = v_full + NS, *v_free = k_free + NS;
  uint64_t *s_full = v_free + NS, *p_ready = s_full + 2, *o_done = p_ready + 4;
  uint64_t *q_full = o_done + 2, *raw_full = q_full + 2, *raw_free = raw_full + NR, *fin = raw_free + NR;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(fin + 1);
  volatile uint32_t *abort_flag = tmem_holder + 1;
  Place *first = reinterpret_cast<Place *>(tmem_holder + 2);
  long long *ends = reinterpret_cast<long long *>(raw + NR * S::kRaw + S::kBars - 16);
  const Kv4Args &c = p.s.a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(k_full + s, 128);
      mbar_init(v_full + s, 128);
      mbar_init(k_free + s, 1);
      mbar_init(v_free + s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_ready + 2 * i, 128);
      mbar_init(p_ready + 2 * i + 1, 128);
      mbar_init(o_done + i, 1);
      mbar_init(q_full + i, 128);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(raw_full + s, 1);
      mbar_init(raw_free + s, 8);
    }
    mbar_init(fin, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 16) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  kv4_begin();
  if (warp < 2) {  // the run's two ends
    Place k{};
    const long long at = find_cut(p, blockIdx.x + warp, lane, k);
    if (lane == 0) {
      if (warp == 0) *first = k;
      ends[warp] = at;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int n_tiles = (int)(ends[1] - ends[0]);
  auto wait = [&](uint64_t *bar, uint32_t use) { return wait_or_abort(bar, use & 1u, abort_flag, c.status, c.wait); };
  auto warp_wait_all = [&](uint64_t *bar, uint32_t use) { return __all_sync(0xffffffffu, wait(bar, use)) != 0; };
  // For each of the run's segments (a part of one item): f(its number, place, tiles), until it returns false.
  auto segments = [&](auto f) {
    if (n_tiles == 0) return;
    Place k = *first;
    for (int at = 0, sg = 0;; ++sg) {
      const int n = min(k.nt - k.tile, n_tiles - at);
      if (!f(sg, k, n)) return;
      at += n;
      if (at == n_tiles) return;
      k.next(p);
    }
  };

  // registers: 640 threads x 96 at launch = 256 x 160 + 256 x 56 + 128 x 48
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    // ------------------------------------------------ softmax: thread = row r of row tile i
    const int i = warp >> 2, r = tid & 127;
    const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = base + i * kKv, tO = base + S::kO + i * D;
    uint32_t uses = 0, dones = 0;  // of this row tile's scores, and items that had any
    segments([&](int sg, const Place &w, int nkv) {
      const int rows = w.item_rows(), row = w.item_row0() + i * 128 + r;  // the row's number among the KV head's
      const bool have = i * 128 + r < rows;
      if (i * 128 >= rows) return true;  // no rows in this tile
      // ---- the row's query: FP16, scaled so that its largest lies in [2^13, 2^14)
      float cs = p.s.a.sm_scale * c.ks * kLog2e;
      {
        const int tok = row / p.G;
        const uint4 *src = reinterpret_cast<const uint4 *>(p.s.a.q + (long long)tok * p.s.a.q_stride +
                                                           (long long)(w.h * p.G + row - tok * p.G) * D);
        uint4 x[D / 8];
        uint32_t mx = 0;
#pragma unroll
        for (int q = 0; q < D / 8; ++q) x[q] = have ? src[q] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < D / 8; ++q) {
          const uint32_t y[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = max(mx, max(y[e] & 0x7FFFu, (y[e] >> 16) & 0x7FFFu));
        }
        const int e = min(140 - (int)(mx >> 7), 60);
        const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
        cs *= __uint_as_float((uint32_t)(127 - e) << 23);
        uint8_t *dst = qs + i * S::kTileBytes;
#pragma unroll
        for (int q = 0; q < D / 8; ++q) {
          const uint32_t y[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = h2u(__floats2half2_rn(__uint_as_float(y[k] << 16) * sc, __uint_as_float(y[k] & 0xFFFF0000u) * sc));
          *reinterpret_cast<uint4 *>(dst + (q / 8) * (128 * 128) + sw_off16(r, (q & 7) * 8)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_async_shared();
        mbar_arrive(q_full + i);
      }
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < nkv; ++j, ++uses) {
        if (!warp_wait_all(s_full + i, uses)) return false;
        tc_fence_after();
        const int valid = w.S - (w.tile + j) * kKv;  // tokens of this tile
        auto half_scores = [&](int half, float (&s)[64]) {
          uint32_t x[64];
#pragma unroll
          for (int q = 0; q < 2; ++q) tmem_ld32(tS + 64 * half + 32 * q, x + 32 * q);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 64; ++q) s[q] = __uint_as_float(x[q]);
          if (valid < kKv) {
#pragma unroll
            for (int q = 0; q < 64; ++q)
              if (64 * half + q >= valid) s[q] = -INFINITY;
          }
        };
        // The weights by the maximum so far, and their sum over the tile: below kMost it shows that no weight passes
        // what FP16 holds, without a look at every score before (the whole call on those 1024 rows of 4 KV heads: 128.5 -> 124.9
        // us). Where it does not, and in an item's first tile, the maximum is found first. Decided by a row's own sum: a
        // row's result depends on no other row.
        float s[64];
        uint32_t weight[2][32];
        float2 sum[2];
        bool up = j == 0;
        for (bool look = j == 0;; look = true) {
          if (look) {
            float x4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              half_scores(half, s);
#pragma unroll
              for (int q = 0; q < 64; q += 4)
#pragma unroll
                for (int e = 0; e < 4; ++e) x4[e] = fmaxf(x4[e], s[q + e]);
            }
            const float top = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * cs;
            if (j > 0) {
              // S of this tile is complete, so the O += P V issued before it is too
              const float f = up && top != m ? ex2(m - top) : 1.0f;
              l *= f;
#pragma unroll 1
              for (int q = 0; q < D; q += 32) {
                uint32_t o[32];
                tmem_ld32(tO + q, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(tO + q, o);
              }
            }
            if (up) m = top;
          }
          const float off = kShift - (m == -INFINITY ? 0.0f : m);
          const float2 cs2 = make_float2(cs, cs), off2 = make_float2(off, off);
          sum[0] = sum[1] = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            half_scores(half, s);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float2 z = fma2(make_float2(s[2 * e], s[2 * e + 1]), cs2, off2);
              z.x = ex2(z.x);
              z.y = ex2(z.y);
              sum[e & 1] = add2(sum[e & 1], z);
              weight[half][e] = h2u(__floats2half2_rn(z.x, z.y));
            }
          }
          sum[0] = add2(sum[0], sum[1]);
          if (look) break;
          up = !(sum[0].x + sum[0].y < kMost && m > -INFINITY);
          if (!__any_sync(0xffffffffu, up)) break;
        }
        l += sum[0].x + sum[0].y;
        // P overlies S's second half; tokens 64 .. go to the products first
#pragma unroll
        for (int half = 1; half >= 0; --half) {
          tmem_st32(tS + 64 + 32 * half, weight[half]);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(p_ready + 2 * i + half);
        }
      }
      // ---- the row's sums, channel by channel: 32 rows are a line
      const bool whole = nkv == w.nt;
      const int piece = 2 * (int)blockIdx.x + (sg == 0 ? 0 : 1);
      {
        if (!warp_wait_all(o_done + i, dones++)) return false;
        tc_fence_after();
        float *dst = whole ? p.w.pre + (size_t)w.h * D * p.rows + row : p.w.part + (size_t)piece * D * p.ld + i * 128 + r;
        const size_t step = whole ? p.rows : p.ld;
#pragma unroll
        for (int q = 0; q < D; q += 32) {
          uint32_t o[32];
          tmem_ld32(tO + q, o);
          tmem_ld_wait();
          if (have) {
#pragma unroll
            for (int e = 0; e < 32; ++e) dst[(q + e) * step] = __uint_as_float(o[e]);
          }
        }
        tc_fence_before();  // O has been read: the next item's products follow this row tile's next weights
        if (have) {
          const float2 ml = make_float2(m - kShift, l);
          if (whole) reinterpret_cast<float2 *>(p.w.pre_ml)[(size_t)w.h * p.rows + row] = ml;
          else reinterpret_cast<float2 *>(p.w.part_ml)[(size_t)piece * p.ld + i * 128 + r] = ml;
        }
      }
      if (tid == 0) {
        int32_t *e = p.w.ends + 2 * ((size_t)w.h * p.slots + w.slot());
        if (w.tile == 0) e[0] = whole ? -1 : piece;
        if (w.tile + nkv == w.nt) e[1] = blockIdx.x;
      }
      return true;
    });
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // ------------------------------------------------ 4-bit bytes into the operands: four warps for K, four for V.
    // Both as they lie, a token's channels in a row: K is the product's B operand with the summed index (channels)
    // along the rows, V with the summed index (tokens) across them.
    // Row r of a group (D = 128: r0 and r0 + 8, D = 64: r0) is K's token r, and V's kv4_v_row's token.
    const int t0 = tid & 127, r0 = t0 / (D / 8), ww = t0 % (D / 8);  // eight channels of rows r0, r0 + 1024 / D, ... of 64
    constexpr int N = D / 16, PER = D == 128 ? 2 : 1;                 // rows of this thread: of 64, of a group
    auto decode = [&](auto values, uint64_t *full, uint64_t *free, uint8_t *tiles) {
      constexpr bool V = values();
      const int t = V ? (r0 & 8) | ((r0 >> 1 & 1) << 2) | ((r0 & 1) << 1) | (r0 >> 2 & 1) : r0;
      const int code_at = V ? kv4_v_code<D>(t, ww * 4) : kv4_k_code<D>(t, ww * 4);
      const int scale_at = V ? kv4_v_scale<D>(t, ww / 2) : kv4_k_scale<D>(t, ww / 2);
      constexpr int scale_step = V ? 2 : 8 * (D / 16);                // from token t's to token t + 8's
      uint8_t *const to = tiles + (ww / 8) * (kKv * 128) + sw_off16(t, (ww & 7) * 8);
      uint32_t u = 0;
      segments([&](int, const Place &w, int n) {
        for (int j = 0; j < n; ++j, ++u) {
          const uint32_t s = u % NS;
          if (u >= NS && !warp_wait_all(free + s, u / NS - 1)) return false;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const uint32_t x = 2 * u + half;
            if (!warp_wait_all(raw_full + x % NR, x / NR)) return false;
            const uint8_t *rb = raw + x % NR * S::kRaw;
            uint8_t *dst = to + s * S::kTileBytes + half * (64 * 128);
            const int valid = w.S - (w.tile + j) * kKv - half * 64;
            uint32_t code[N];
            uint32_t sc[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
              code[i] = *reinterpret_cast<const uint32_t *>(rb + code_at + i / PER * (18 * D) + i % PER * (8 * (D / 2)));
              sc[i] = rb[scale_at + i / PER * (18 * D) + i % PER * scale_step];
            }
            if (V && valid < 64) {  // places that hold no token hold anything, NaN scales too
#pragma unroll
              for (int i = 0; i < N; ++i)
                if (i / PER * 16 + i % PER * 8 + t >= valid) sc[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
              uint32_t h, o[4];
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(sc[i] * 0x0101u)));
              decode8(code[i], *reinterpret_cast<__half2 *>(&h), o);
              *reinterpret_cast<uint4 *>(dst + (i / PER * 16 + i % PER * 8) * 128) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(raw_free + x % NR);
          }
          fence_async_shared();
          mbar_arrive(full + s);
        }
        return true;
      });
    };
    if (warp < 12) decode(std::false_type{}, k_full, k_free, kbuf);
    else decode(std::true_type{}, v_full, v_free, vbuf);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 16) {
      // ------------------------------------------------ MMAs
      constexpr uint32_t idS = idesc_f16(kKv), idO = idesc_f16(D) | (1u << 16);  // V: N runs along the rows
      constexpr uint64_t kStep = S::kTileBytes / 16;  // from one stage or tile to the next, in a descriptor
      const uint64_t qd = desc_sw128(smem_u32(qs)), kd = desc_sw128(smem_u32(kbuf));
      const uint64_t vd = desc_sw128_n(smem_u32(vbuf), kKv * 128);
      const bool me = elect_one();
      uint32_t kv = 0, uses[2] = {0, 0}, items[2] = {0, 0};  // K / V tiles taken, each row tile's, and its items
      segments([&](int, const Place &w, int n) {
        bool ok = true;
        if (me) {
          const int two = w.item_rows() > 128 ? 2 : 1;
          auto scores = [&](int i, uint32_t use) {  // S_i = Q_i K^T
            const uint64_t q = qd + i * kStep, kk = kd + (uint64_t)(use % NS) * kStep;
            const uint32_t d = tmem + i * kKv;
            mma_f16_ss_c<false>(d, q, kk, idS);
#pragma unroll
            for (int k = 1; k < D / 16; ++k)
              mma_f16_ss_c<true>(d, q + (k / 4) * (128 * 128 / 16) + 2 * (k & 3), kk + (k / 4) * (kKv * 128 / 16) + 2 * (k & 3), idS);
            tc_commit(s_full + i);
          };
          auto values = [&](int i, uint32_t use, bool zero) {  // O_i += P_i V
            const uint64_t v = vd + (uint64_t)(use % NS) * kStep;
            const uint32_t d = tmem + S::kO + i * D, a = tmem + i * kKv + 64;
            if (!(ok = wait(p_ready + 2 * i + 1, uses[i]))) return;  // tokens 64..127 first
            tc_fence_after();
            if (zero) mma_f16_ts_c<false>(d, a + 32, v + 4 * (2048 / 16), idO);
            else mma_f16_ts_c<true>(d, a + 32, v + 4 * (2048 / 16), idO);
#pragma unroll
            for (int k = 1; k < 4; ++k) mma_f16_ts_c<true>(d, a + 32 + 8 * k, v + (4 + k) * (2048 / 16), idO);
            if (!(ok = wait(p_ready + 2 * i, uses[i]))) return;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ts_c<true>(d, a + 8 * k, v + k * (2048 / 16), idO);
            ++uses[i];
          };
          ok = wait(q_full, items[0]++) && (two == 1 || wait(q_full + 1, items[1]++)) && wait(k_full + kv % NS, kv / NS);
          if (ok) {
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (i < two) scores(i, kv);
            tc_commit(k_free + kv % NS);
          }
          for (int j = 0; j < n && ok; ++j) {
            const uint32_t u = kv + j;
            ok = wait(v_full + u % NS, u / NS) && (j + 1 >= n || wait(k_full + (u + 1) % NS, (u + 1) / NS));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || i >= two) continue;
              values(i, u, j == 0);
              if (!ok) break;
              if (j + 1 < n) scores(i, u + 1);
              else tc_commit(o_done + i);
            }
            if (!ok) break;
            tc_commit(v_free + u % NS);
            if (j + 1 < n) tc_commit(k_free + (u + 1) % NS);
          }
        }
        kv += n;
        return __any_sync(0xffffffffu, me && ok) != 0;
      });
      // every MMA issued has completed before the CTA may leave
      if (me) {
        tc_commit(fin);
        mbar_wait(fin, 0u);
      }
    } else if (warp == 17) {
      // ------------------------------------------------ the cached bytes, 64 tokens at a time: a copy for the groups of a
      // page, which lie together (a copy's cost is near 100 cycles whatever its size)
      const int per = min(c.page_tokens / 16, 4);  // groups of a copy
      uint32_t x = 0;
      segments([&](int, const Place &w, int n) {
        const uint8_t *src = nullptr;
        for (int j = 0; j < 2 * n; ++j, ++x) {
          const uint32_t s = x % NR;
          // the places of 512 tokens at once, 16 a lane (64 at a time, tiles waited for the page table: the 1024 rows above
          // 124 us instead of 120, six groups of ten rows on up to 38928 tokens 160 instead of 122)
          if (j % 8 == 0) {
            const int pos = (w.tile * 2 + j) * 64 + lane * 16;
            src = nullptr;
            if (lane % per == 0 && pos < w.S && j + lane / 4 < 2 * n) {
              const uint8_t *g = kv4_group<D>(c, w.lead, pos);  // a bad page id (flagged) reads page 0
              src = (g ? g : c.pages) + w.h * kv4_head_bytes<D>(c);
            }
          }
          const bool now = src != nullptr && lane / 4 == j % 8;
          const int copies = __popc(__ballot_sync(0xffffffffu, now));  // (whole pages are shared)
          if (x >= NR && !warp_wait_all(raw_free + s, x / NR - 1)) return false;
          if (lane == 0) mbar_arrive_expect_tx(raw_full + s, copies * per * 18 * D);
          __syncwarp();
          if (now) bulk_g2s(raw + s * S::kRaw + lane % 4 * 18 * D, src, per * 18 * D, raw_full + s);
        }
        return true;
      });
      // the last copies land (or a bounded wait for each ends) before the CTA leaves, whoever gives up when
      if (lane == 0)
        for (uint32_t y = x < NR ? 0 : x - NR; y < x; ++y) mbar_wait(raw_full + y % NR, (y / NR) & 1u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- the parts joined
// A CTA per 32 rows of a KV head and 32 channels. First the prefix's pieces, lane =
// row, U of them in flight; then, four channels a thread, what the sequence has for
// itself. Bound by latency: the row's item, its ends, the pieces.
template <int D>
__global__ void __launch_bounds__(256, 2) kv4_merge_kernel(SharedKv4 p) {
  constexpr int U = 12;
  __shared__ float sums[32][33], pre_m[32], pre_l[32];
  kv4_begin();
  const Kv4Args &c = p.s.a.c;
  const int h = blockIdx.y, ch0 = blockIdx.z * 32;
  const int r = threadIdx.x / 8, ch = ch0 + threadIdx.x % 8 * 4, row = blockIdx.x * 32 + r;
  const bool have = row < p.rows;
  const int tok = have ? row / p.G : 0, b = tok / p.r, q = row - tok * p.G;
  const long long out = (long long)tok * p.s.a.Hq + h * p.G + q;
  // where its own lies: asked for before the prefix's pieces, whose loads take as long again
  const int own_f = row - b * p.r * p.G, own_g = p.own.groups == 1 ? 0 : own_f / p.own.rows;
  const int2 own_e = have ? reinterpret_cast<const int2 *>(p.own.ends)[((size_t)b * c.Hkv + h) * p.own.groups + own_g] : make_int2(0, -1);
  {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x * 32 + lane;
    const int2 item = row < p.rows && p.runs ? p.w.seq_item[row / p.G / p.r] : make_int2(-1, -1);
    const float *src = nullptr;   // the first piece's channel
    const float2 *ml = nullptr;
    int np = 0, second = 0;       // pieces; from the first to the second, in pieces: then one in each run
    size_t ch_step = p.rows;
    if (item.x >= 0) {
      const int pair = (row - item.x) / kItemRows, in = row - item.x - pair * kItemRows;
      const int2 e = reinterpret_cast<const int2 *>(p.w.ends)[(size_t)h * p.slots + item.y + pair];
      if (e.x < 0) {
        np = 1;
        src = p.w.pre + ((size_t)h * D + ch0 + warp * 4) * p.rows + row;
        ml = reinterpret_cast<const float2 *>(p.w.pre_ml) + (size_t)h * p.rows + row;
      } else if (e.x < 2 * p.runs && e.y >= e.x / 2 && e.y < p.runs) {  // (else a wait gave up before they were written)
        np = e.y - e.x / 2 + 1;
        src = p.w.part + ((size_t)e.x * D + ch0 + warp * 4) * p.ld + in;
        ml = reinterpret_cast<const float2 *>(p.w.part_ml) + (size_t)e.x * p.ld + in;
        ch_step = p.ld;
        second = 2 - (e.x & 1);
      }
    }
    float m = -INFINITY, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < np; j += U) {
      float2 x[U];
      float v[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = j + u == 0 ? 0 : second + 2 * (j + u - 1);
        const bool in = j + u < np;
        x[u] = in ? ml[(size_t)at * p.ld] : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[u][k] = in ? src[(size_t)at * D * p.ld + k * ch_step] : 0.0f;
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, x[u].x);
      const float safe = top == -INFINITY ? 0.0f : top, f = ex2(m - safe);
      m = top;
      l *= f;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] *= f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float fu = ex2(x[u].x - safe);
        l = fmaf(x[u].y, fu, l);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = fmaf(v[u][k], fu, acc[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[lane][warp * 4 + k] = acc[k];
    if (warp == 0) {
      pre_m[lane] = m;
      pre_l[lane] = l;
    }
  }
  // ---- the sequence's own: whole, or its pieces
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (have) {
    const int2 e = own_e;
    if (e.x < 0) {
      const float2 x = reinterpret_cast<const float2 *>(p.w.own_ml)[out];
      o = *reinterpret_cast<const float4 *>(p.w.own + out * D + ch);
      m = x.x;
      l = x.y;
    } else if (e.x < 2 * p.own.runs && e.y >= e.x / 2 && e.y < p.own.runs) {
      const int in = own_f - own_g * p.own.rows, np = e.y - e.x / 2 + 1;
      for (int j = 0; j < np; ++j) {
        const size_t at = (size_t)(j == 0 ? e.x : 2 * (e.x / 2 + j)) * p.own.rows + in;
        float2 x = reinterpret_cast<const float2 *>(p.own.ml)[at];
        const float4 v = *reinterpret_cast<const float4 *>(p.own.part + at * D + ch);
        x.x -= kKv4PieceShift;
        const float top = fmaxf(m, x.x), safe = top == -INFINITY ? 0.0f : top, fm = ex2(m - safe), fx = ex2(x.x - safe);
        m = top;
        l = l * fm + x.y * fx;
        o.x = o.x * fm + v.x * fx;
        o.y = o.y * fm + v.y * fx;
        o.z = o.z * fm + v.z * fx;
        o.w = o.w * fm + v.w * fx;
      }
    }
  }
  __syncthreads();
  if (!have) return;
  const float mp = pre_m[r], top = fmaxf(m, mp), safe = top == -INFINITY ? 0.0f : top, fo = ex2(m - safe), fp = ex2(mp - safe);
  l = l * fo + pre_l[r] * fp;
  const float inv = l == 0.0f ? 0.0f : c.vs / l, go = fo * inv, gp = fp * inv;
  const float *s = sums[r] + (ch - ch0);
  *reinterpret_cast<uint2 *>(p.s.a.out + out * D + ch) = make_uint2(bf16x2(o.x * go + s[0] * gp, o.y * go + s[1] * gp),
                                                                    bf16x2(o.z * go + s[2] * gp, o.w * go + s[3] * gp));
  if (p.s.a.lse && ch == 0) p.s.a.lse[out] = (top + log2f(l)) * 0.6931471805599453f;
}

template <int D>
cudaError_t launch_t(const SharedKv4 &p, int num_sms, cudaStream_t stream) {
  using S = PrefixShape<D>;
  const Kv4Args &c = p.s.a.c;
  cudaError_t e = kv4_launch(kv4_shared_plan_kernel, c.B + p.s.groups, kPlanThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  if (p.runs > 0) {
    static bool allowed[64];
    e = kv4_allow_smem(kv4_prefix_kernel<D>, S::kBytes, allowed);
    if (e == cudaSuccess) e = kv4_launch(kv4_prefix_kernel<D>, p.runs, kPrefixThreads, S::kBytes, stream, p);
    if (e != cudaSuccess) return e;
  }
  Kv4AttnArgs own = p.s.a;
  own.c.kv_len = p.w.own_len;
  own.c.table = p.w.own_table;
  e = launch_kv4_decode(own, p.w.decode, num_sms, stream, p.w.own, p.w.own_ml, p.runs > 0);
  if (e != cudaSuccess) return e;
  return kv4_launch(kv4_merge_kernel<D>, dim3((p.rows + 31) / 32, c.Hkv, D / 32), 256, 0, stream, p);
}

}  // namespace

size_t kv4_decode_shared_bytes(const Kv4SharedArgs &s, int num_sms) {
  SharedKv4 p{};
  return s.a.c.T ? lay_out(s, nullptr, num_sms, p) : 0;
}

cudaError_t launch_kv4_decode_shared(const Kv4SharedArgs &s, void *workspace, int num_sms, cudaStream_t stream) {
  SharedKv4 p{};
  lay_out(s, static_cast<uint8_t *>(workspace), num_sms, p);
  return s.a.c.D == 128 ? launch_t<128>(p, num_sms, stream) : launch_t<64>(p, num_sms, stream);
}

}  // namespace gdn
