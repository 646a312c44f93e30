// Decode attention over the 4-bit paged cache (include/gdn.h): r new tokens of
// each of B sequences against everything the sequence has cached.
//
//   z_ij = sm q_i . k_j,  out_i = sum_j 2^(z_ij' - m_i) v_j / sum_j 2^(z_ij' - m_i),  z' = z log2 e
//
// What bounds it: the cached bytes, each read once (2 (d/2 + d/16) per token
// and KV head); at the measured copy bandwidth an SM gets 23 bytes a cycle, so
// a token-head of d = 128 (144 bytes) lasts about 6 cycles, in which its 256
// values are to be decoded and used G r times. So the work is on the warp
// MMAs, transposed: tokens are the rows (m16n8k16, A = 16 tokens of K, or 16
// channels of V), the G r query rows that share a KV head the 8 columns --
// the operand that has to be decoded is decoded straight into A's registers,
// exactly (E2M1 x E4M3 fits FP16), with no pass through shared memory.
//   S^T = K Q^T: lane (g, t) of the warp holds tokens g and g + 8 of a group;
//     the k order is free, so it takes 16 (d = 64: 8) consecutive code bytes.
//   O^T += V^T P^T: lane (g, t) holds channels of block g (d = 64: half a
//     block) of tokens 2t, 2t + 1, 2t + 8, 2t + 9: two tokens' nibbles are
//     joined into one byte, which converts to the FP16 pair that A wants.
//   P^T's registers are S^T's, packed and transposed by movmatrix.
// tcgen05 is no use here: it reads its operands from shared or tensor memory,
// so the decoded cache would have to be written there first (7 times the bytes
// that are loaded), for at most 64 columns.
//
// Rounding: q enters in FP16 scaled by a power of two per row (exact but for
// elements 2^-27 below the row's largest); the weights 2^(z - m + 7) are rounded
// to FP16 (2^-11 relative down to 2^-21 of the largest weight, in steps of 2^-31
// of it below); the scores, the sums and the output are FP32.
//
// Work: a tile is 32 tokens (64 for d = 64) of one item = a (sequence, KV head,
// group of query rows). All items' tiles, in order, are cut into runs of equal
// cost, one per team of warps -- ragged lengths leave no SM idle. The team's
// warps take the run's tiles in turn, each with two slots of its own that it
// refills by bulk copies as soon as it has read them, and its own (m, l, O),
// which meet in shared memory at the end of an item or of the run. An item that
// lies in one run is finished there; the pieces of others go to the workspace
// and kv4_join_kernel adds them in order.
// A team is a whole CTA where there are fewer items than SMs (long contexts:
// few pieces to join), else four warps: the other teams of the CTA work while
// one's parts meet, and fewer warps wait for the slowest.
//
// Measured (32 query heads, d = 128): 64 sequences of up to 8190 tokens, 8 KV
// heads, 291 MB: 56 us, 5.2 TB/s (0.76 of the copy bandwidth); one of 200001, 4 KV
// heads, 115 MB: 28 us. Before the first tile pass 10000 cycles, 5 us (the lengths,
// the run's ends, the page table, the query rows, the first tiles, one after the
// other); the join adds 3. When both took 59 and 29.6, the loads alone took 54 and
// 24, the arithmetic alone 55 and 26. A tile costs about 570 issue slots a warp: 128
// conversions, 96 shifts that bring bytes to them, 128 scale products, 32 MMAs.
#include "kv4.cuh"
#include "tc.cuh"

namespace gdn {

namespace {

// A column's weights are 2^(z - m + 7); m only moves (and O is rescaled) when a
// score passes it by 7, so that a tile whose scores do not costs no exchange
// between lanes and no rescaling. Weights stay below 2^14 in FP16.
constexpr float kShift = 7.0f, kSlack = 7.0f;

// Warps by the registers they need: 128, 168 or 255 each. NQ: 8-row column
// blocks of an item.
// TEAM: warps of a team, 0 for the whole CTA.
template <int D, int NQ, int TEAM>
struct DecodeShape {
  static constexpr int kWarps = D == 128 ? (NQ == 1 ? 16 : NQ == 2 ? 12 : 8) : (NQ <= 2 ? 16 : 12);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTeam = TEAM ? TEAM : kWarps, kTeams = kWarps / kTeam;
  static_assert(kWarps % kTeam == 0, "teams fill the CTA");
  static constexpr int kGroups = D == 64 && NQ <= 2 ? 4 : 2;  // 16-token groups of a tile
  static constexpr int kTile = kGroups * 16;
  static constexpr int kSlot = kGroups * 18 * D;
  static constexpr int kRows = 8 * NQ;
  static constexpr int kLd = D + 4;                           // row of the meeting buffer, floats
  static constexpr bool kQShared = D == 128 && NQ == 4;       // 64 registers of q would not fit beside 128 of O
  static constexpr int kMeet = kWarps * kRows * kLd * 4;
  static constexpr int kStats = 2 * 2 * kWarps * kRows * 4;   // m and l, two segments
  static constexpr int kQRaw = kTeams * kRows * D * 2;        // a segment's query rows
  static constexpr int kQ = kQShared ? (D / 16) * NQ * 32 * 8 : 0;
  static_assert(!kQShared || kTeams == 1, "one converted copy of q");
  static constexpr int kFixed = kMeet + kStats + kQRaw + kQ + 1024;
  static constexpr int kSlots = 2 * kWarps;
  static constexpr int kRing = kSlots * kSlot;
  static constexpr int kBytes = kRing + kFixed;
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};

struct DecodeArgs {
  Kv4AttnArgs a;
  int r, G, RG;      // new tokens per sequence, query heads per KV head, row groups per (sequence, KV head)
  uint32_t inv_g;    // ceil(2^16 / G): x / G = x inv_g >> 16 for x < 128 (G <= 64)
  int extra;         // cost of an item beside its tiles, in tiles; kWhole: runs hold whole items, nothing to join
  int items;         // (sequence, KV head, row group)
  float *part;       // pieces [2 runs][rows][D], their (m, l) [2 runs][rows][2], the items' ends [items][2]
};
// What the plan goes by, all measured on GB300 (d = 128, us):
// An item's query rows, its meeting and its output take a team about as long as
// this many tiles of its run. A whole CTA: 16 / 24 / 32 gave 25.7 / 24.3 / 24.0 at
// 16 sequences of up to 8000 tokens (8 KV heads), 21.4 / 20.8 / 20.3 at 8 of up to
// 30000 (4, d = 64, 16 rows); four warps: 3 / 6 / 10 gave 67.7 / 64.4 / 64.7 at 64
// of up to 8190.
constexpr int kExtraCta = 32, kExtraTeam = 6;
// From as many items as a GB300 has SMs, teams of four warps instead of whole
// CTAs: 59 against 72 with 512 items (64 sequences, above), 26.7 against 29.2 with
// 192 (24 of up to 6000); with 128 items 25.3 against 24.2, with 4 of 200001 tokens
// 56 against 30.
constexpr int kManyItems = 152;
// Items stay whole while a team goes through the longest in this many rounds. Whole
// against cut and joined: 64 items of 1000 tokens (2 rounds of a CTA) 8.8 and 10.7,
// 4 of 3000 (6 rounds) 16.7 and 11.9; 1600 of up to 250 (2 rounds of a team) 21.4
// and 29.4, of up to 400 (4) 27.5 and 29.6, 768 of up to 600 (5) 21.7 and 21.1.
constexpr int kRoundsCta = 3, kRoundsTeam = 4;
constexpr int kWhole = 1 << 20;  // the `extra` of whole items

// a / b, mostly in 32 bits
__device__ __noinline__ long long quot64(long long a, long long b) { return a / b; }
GDN_DEV long long quot(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : quot64(a, b);
}

// A sequence's tiles: an empty one has one tile with no tokens, so that its rows are written.
template <int TILE>
GDN_DEV int tiles_of(int len) { return len > 0 ? (len + TILE - 1) / TILE : 1; }

GDN_DEV int warp_isum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Runs that share `tiles` tiles: each warp gets at least one (`warps` per run).
GDN_DEV int runs(long long tiles, int warps, int most) {
  return tiles < (long long)warps * most ? (int)(((int)tiles + warps - 1) / warps) : most;
}

// A place in the sequence of all tiles: an item and a tile of it.
struct Cursor {
  int b, hr, tile, nt, len;
};
template <int TILE>
GDN_DEV void seek(const Kv4Args &c, Cursor &k, int b) {
  k.b = b;
  k.len = kv4_len(c, b);
  k.nt = tiles_of<TILE>(k.len);
}
template <int TILE>
GDN_DEV void next_item(const Kv4Args &c, Cursor &k, int HR) {
  k.tile = 0;
  if (++k.hr == HR) {
    k.hr = 0;
    seek<TILE>(c, k, k.b + 1);
  }
}
// The tiles of sequences b0 + lane (0 past the end), for one KV head and row group.
template <int TILE>
GDN_DEV int lane_tiles(const Kv4Args &c, int b0, int lane) {
  return b0 + lane < c.B ? tiles_of<TILE>(kv4_len(c, b0 + lane)) : 0;
}
// The tile at cost u (each item costs its tiles and `extra`, which comes
// first), and how many tiles lie before it. All lanes of a warp. n0:
// lane_tiles of the first 32 sequences.
template <int TILE>
GDN_DEV long long find_tile(const Kv4Args &c, long long u, int HR, int extra, int lane, int n0, Cursor &k) {
  long long cost = 0, tiles = 0;  // of the sequences before, per (KV head, row group)
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const int n = b0 ? lane_tiles<TILE>(c, b0, lane) : n0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const int seqs = min(lane + 1, c.B - b0);
    const unsigned past = __ballot_sync(0xffffffffu, b0 + lane < c.B && (cost + incl + (long long)seqs * extra) * HR > u);
    if (past) {
      const int l = __ffs(past) - 1;
      const int before = __shfl_sync(0xffffffffu, incl - n, l);
      seek<TILE>(c, k, b0 + l);
      const long long off = u - (cost + before + (long long)l * extra) * HR;
      k.hr = (int)quot(off, k.nt + extra);
      k.tile = max((int)(off - (long long)k.hr * (k.nt + extra)) - extra, 0);
      return (tiles + before) * HR + (long long)k.hr * k.nt + k.tile;
    }
    const int all = __shfl_sync(0xffffffffu, incl, 31);
    cost += all + (long long)min(32, c.B - b0) * extra;
    tiles += all;
  }
  return tiles * HR;  // past the end
}
// The runs: N of them, cut k at cost floor(units k / N).
struct Cuts {
  int N, rest, n0;
  long long tiles, q;
  GDN_DEV long long at(int k) const { return q * k + rest * k / N; }
};
template <int TILE>
GDN_DEV Cuts find_cuts(const DecodeArgs &p, int warps, int HR, int lane, int most) {
  const Kv4Args &c = p.a.c;
  Cuts k;
  k.n0 = lane_tiles<TILE>(c, 0, lane);
  long long tiles = warp_isum(k.n0);
  for (int b0 = 32; b0 < c.B; b0 += 32) tiles += warp_isum(lane_tiles<TILE>(c, b0, lane));
  const long long units = (tiles + (long long)c.B * p.extra) * HR;
  k.tiles = tiles * HR;
  k.N = runs(k.tiles, warps, most);
  k.q = quot(units, k.N);
  k.rest = (int)(units - k.q * k.N);
  return k;
}
// Cut `cut` of at most `most` runs: the tile there, and how many lie before it.
// With whole items, runs have as many each, and a run's tiles are counted from
// its own beginning: `from` is the run's first cut.
template <int TILE>
GDN_DEV long long find_cut(const DecodeArgs &p, int warps, int HR, int lane, int from, int cut, int most, Cursor &k) {
  const Kv4Args &c = p.a.c;
  k = Cursor{0, 0, 0, 0, 0};
  if (p.extra == kWhole) {
    const int items = c.B * HR;
    const int i0 = (int)quot((long long)items * from, most), i1 = (int)quot((long long)items * cut, most);
    int n = 0;
    for (int i = i0; i < i1; ++i) n += tiles_of<TILE>(kv4_len(c, i / HR));
    if (i1 < items) {
      seek<TILE>(c, k, i1 / HR);
      k.hr = i1 % HR;
    }
    return n;
  }
  const Cuts x = find_cuts<TILE>(p, warps, HR, lane, most);
  return cut >= x.N ? x.tiles : find_tile<TILE>(c, x.at(cut), HR, p.extra, lane, x.n0, k);
}

// A group of an item's query rows, `most` at most: row x is a (token, query head).
struct RowGroup {
  int h, rows;       // the KV head, the rows
  int tok, off, G;   // the first row's token, and its place among that token's heads
  uint32_t inv_g;
  GDN_DEV int over(int x) const { return (int)((uint32_t)(off + x) * inv_g >> 16); }
  GDN_DEV int token(int x) const { return tok + over(x); }
  GDN_DEV int head(int x) const { return off + x - over(x) * G; }
};
GDN_DEV RowGroup row_group(const DecodeArgs &p, int hr, int most) {
  const int h = p.RG == 1 ? hr : hr / p.RG, row0 = (hr - h * p.RG) * most;
  const int tok = row0 ? row0 / p.G : 0;
  return {h, min(most, p.r * p.G - row0), tok, row0 - tok * p.G, p.G, p.inv_g};
}

GDN_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
GDN_DEV uint32_t e4m3x2_to_h2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}

template <int D>
GDN_DEV int32_t *join_ends(const DecodeArgs &p, int runs, int rows) {
  return reinterpret_cast<int32_t *>(p.part + 2 * (size_t)runs * rows * (D + 2));
}

template <int D, int NQ, int TEAM>
__global__ void __launch_bounds__(DecodeShape<D, NQ, TEAM>::kThreads, 1) kv4_decode_kernel(DecodeArgs p) {
  using S = DecodeShape<D, NQ, TEAM>;
  constexpr int TILE = S::kTile, GR = S::kGroups, W = S::kTeam;
  constexpr int KS = D / 16;  // k steps of S, and MMAs of 16 channels of O
  extern __shared__ __align__(128) unsigned char sm[];
  const Kv4Args &c = p.a.c;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int team = threadIdx.x / (32 * W), tid = threadIdx.x - team * (32 * W), warp = tid >> 5;  // within the team
  const int run = blockIdx.x * S::kTeams + team;
  float *meet = reinterpret_cast<float *>(sm + S::kRing) + team * (W * S::kRows * S::kLd);
  float *stats = reinterpret_cast<float *>(sm + S::kRing + S::kMeet) + team * (4 * W * S::kRows);
  unsigned char *qraw = sm + S::kRing + S::kMeet + S::kStats + team * (S::kRows * D * 2);
  unsigned char *tail_sm = sm + S::kRing + S::kMeet + S::kStats + S::kQRaw;
  uint2 *qsm = reinterpret_cast<uint2 *>(tail_sm);
  uint64_t *full = reinterpret_cast<uint64_t *>(tail_sm + S::kQ), *q_full = full + S::kSlots + team;
  volatile uint32_t *abort_flag = reinterpret_cast<uint32_t *>(full + S::kSlots + S::kTeams);
  const int HR = c.Hkv * p.RG;
  auto team_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * W) : "memory"); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kSlots + S::kTeams; ++s) mbar_init(full + s, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  kv4_begin();
  __syncthreads();
  Cursor cur;
  int n_tiles;
  {  // the team's first two warps find its run's ends for all (16 warps at once took 2 us of the issue slots)
    struct Found {
      Cursor k;
      long long at;
    };
    volatile Found *found = reinterpret_cast<volatile Found *>(meet);
    if (warp < 2) {
      const long long n = find_cut<TILE>(p, W, HR, lane, run, run + warp, gridDim.x * S::kTeams, cur);
      if (lane == 0) {
        found[warp].k.b = cur.b;
        found[warp].k.hr = cur.hr;
        found[warp].k.tile = cur.tile;
        found[warp].k.nt = cur.nt;
        found[warp].k.len = cur.len;
        found[warp].at = n;
      }
    }
    team_sync();
    cur.b = found[0].k.b;
    cur.hr = found[0].k.hr;
    cur.tile = found[0].k.tile;
    cur.nt = found[0].k.nt;
    cur.len = found[0].k.len;
    n_tiles = (int)(found[1].at - found[0].at);
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < c.B; b += S::kThreads)
      if (c.kv_len[b] != kv4_len(c, b)) flag_status(c.status, GDN_E_RANGE);

  int at = 0, next = warp;  // the segment's first tile (cur), and this warp's next one, within the run
  // ------------------------------------------------ loads
  // This warp's tiles warp, warp + W, ... go into its two slots in turn. Where
  // the groups of the next TB of them lie is worked out at once, one group per
  // lane (a tile at a time cost 100 instructions a tile, of 820).
  constexpr int TB = 32 / GR;
  uint64_t *my_full = full + 2 * (team * W + warp);
  unsigned char *my_slots = sm + 2 * (team * W + warp) * S::kSlot;
  int ld = warp, ld_i = TB;       // the next tile to load, and its place in the batch
  const uint8_t *ld_src = nullptr;
  auto load = [&](int s) {
    if (ld_i == TB) {
      ld_i = 0;
      ld_src = nullptr;
      const int off = ld + W * (lane / GR);
      if (off < n_tiles) {
        Cursor k = cur;
        for (int step = off - at;;) {
          if (step < k.nt - k.tile) {
            k.tile += step;
            break;
          }
          step -= k.nt - k.tile;
          next_item<TILE>(c, k, HR);
        }
        const int pos = k.tile * TILE + (lane % GR) * 16;
        if (pos < k.len) {
          ld_src = kv4_group<D>(c, k.b, pos);
          if (ld_src) ld_src += (p.RG == 1 ? k.hr : k.hr / p.RG) * kv4_head_bytes<D>(c);
        }
      }
    }
    const uint8_t *src = reinterpret_cast<const uint8_t *>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(ld_src), ld_i * GR + lane % GR));
    const unsigned goods = __ballot_sync(0xffffffffu, lane < GR && src != nullptr);
    if (lane == 0) mbar_arrive_expect_tx(my_full + s, __popc(goods) * 18 * D);
    __syncwarp();
    if (goods >> lane & 1) bulk_g2s(my_slots + s * S::kSlot + lane * 18 * D, src, 18 * D, my_full + s);
    ++ld_i;
    ld += W;
  };
  // The team's warp 0 loads the query rows of a segment, one per lane.
  auto load_q = [&](const Cursor &k) {
    const RowGroup rg = row_group(p, k.hr, S::kRows);
    const int rows = rg.rows;
    if (lane == 0) mbar_arrive_expect_tx(q_full, rows * D * 2);
    __syncwarp();
    if (lane < rows)
      bulk_g2s(qraw + lane * (D * 2),
               p.a.q + ((long long)k.b * p.r + rg.token(lane)) * p.a.q_stride + (long long)(rg.h * p.G + rg.head(lane)) * D,
               D * 2, q_full);
  };
  if (warp == 0 && n_tiles > 0) load_q(cur);
#pragma unroll 1
  for (int i = 0; i < 2; ++i)
    if (ld < n_tiles) load(i);

  int slot = 0, flip = 0;
  uint32_t turn = 0;  // parity of the slots' round
  bool alive = true;
  for (int sg = 0; at < n_tiles; ++sg) {
    const int seg = min(cur.nt - cur.tile, n_tiles - at);
    const bool mine = next < at + seg;
    // ------------------------------------------------ q: B operand, lane (g, t) = row g, channels t D/4 ...
    uint2 qf[S::kQShared ? 1 : NQ][S::kQShared ? 1 : KS];
    float cs[NQ][2];   // sm k_scale log2 e / the row's scale, of columns 2t and 2t + 1
    int last[NQ][2];   // the last token that the row sees
    float O[KS][NQ][4], m[NQ][2], l[NQ][2];
    const RowGroup qg = row_group(p, cur.hr, S::kRows);
    if (alive && !__all_sync(0xffffffffu, wait_or_abort(q_full, (uint32_t)sg & 1u, abort_flag, c.status, c.wait))) {
      alive = false;
      if (warp == 0) mbar_wait(q_full, (uint32_t)sg & 1u);  // its copies: no more follow once it has given up
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int row = n * 8 + g;
      uint4 w[D / 32];
      const uint4 *qp = reinterpret_cast<const uint4 *>(qraw + row * (D * 2) + t * (D / 2));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) w[i] = row < qg.rows ? qp[i] : make_uint4(0, 0, 0, 0);
      uint32_t mx = 0;  // the largest magnitude, as BF16 bits (a NaN counts as the largest: its row is NaN anyway)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = max(mx, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^k that takes the largest to [2^13, 2^14); k <= 60 and the inverse 2^-k are normal
      const int e = (int)(mx >> 7), k = min(140 - e, 60);
      const float sc = __uint_as_float((uint32_t)(k + 127) << 23);
      const float inv = p.a.sm_scale * c.ks * 1.4426950408889634f * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[j] = h2u(__floats2half2_rn(__uint_as_float(x[j] << 16) * sc, __uint_as_float(x[j] & 0xFFFF0000u) * sc));
        if constexpr (!S::kQShared) {
          qf[n][2 * i] = make_uint2(y[0], y[1]);
          qf[n][2 * i + 1] = make_uint2(y[2], y[3]);
        } else {
          if (warp == n) {  // all warps work on this item: warp n puts row block n down for them
            qsm[((2 * i) * NQ + n) * 32 + lane] = make_uint2(y[0], y[1]);
            qsm[((2 * i + 1) * NQ + n) * 32 + lane] = make_uint2(y[2], y[3]);
          }
        }
      }
      // columns 2t and 2t + 1 are rows 2t and 2t + 1 of this block: held by lanes 4 (2t), 4 (2t + 1)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        cs[n][e2] = __shfl_sync(0xffffffffu, inv, (2 * t + e2) * 4);
        const int rr = n * 8 + 2 * t + e2;
        last[n][e2] = rr < qg.rows ? cur.len - p.r + qg.token(rr) : -1;
        m[n][e2] = -INFINITY;
        l[n][e2] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) O[i][n][j] = 0.0f;
    }
    if constexpr (S::kQShared) team_sync();

    // ------------------------------------------------ the warp's tiles of this segment
    for (; next < at + seg; next += W) {
      if (alive && !__all_sync(0xffffffffu, wait_or_abort(my_full + slot, turn, abort_flag, c.status, c.wait))) alive = false;
      if (!alive) continue;
      const unsigned char *buf = my_slots + slot * S::kSlot;
      const int pos0 = (cur.tile + next - at) * TILE;
      float s[GR][NQ][4];
#pragma unroll
      for (int q = 0; q < GR; ++q) {
        const unsigned char *gb = buf + q * 18 * D;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[q][n][j] = 0.0f;
        uint32_t ka[D / 32], kb[D / 32], sa, sb;
        if (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4 *>(gb + g * 64 + t * 16);
          const uint4 y = *reinterpret_cast<const uint4 *>(gb + (g + 8) * 64 + t * 16);
          ka[0] = x.x; ka[1] = x.y; ka[2 % (D / 32)] = x.z; ka[3 % (D / 32)] = x.w;
          kb[0] = y.x; kb[1] = y.y; kb[2 % (D / 32)] = y.z; kb[3 % (D / 32)] = y.w;
          sa = e4m3x2_to_h2(*reinterpret_cast<const uint16_t *>(gb + 16 * D + g * 8 + t * 2));
          sb = e4m3x2_to_h2(*reinterpret_cast<const uint16_t *>(gb + 16 * D + (g + 8) * 8 + t * 2));
        } else {
          const uint2 x = *reinterpret_cast<const uint2 *>(gb + g * 32 + t * 8);
          const uint2 y = *reinterpret_cast<const uint2 *>(gb + (g + 8) * 32 + t * 8);
          ka[0] = x.x; ka[1] = x.y;
          kb[0] = y.x; kb[1] = y.y;
          sa = e4m3x2_to_h2(gb[16 * D + g * 4 + t]);
          sb = e4m3x2_to_h2(gb[16 * D + (g + 8) * 4 + t]);
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const __half2 fa = w < 2 ? __low2half2(u2h(sa)) : __high2half2(u2h(sa));
          const __half2 fb = w < 2 ? __low2half2(u2h(sb)) : __high2half2(u2h(sb));
          uint32_t xa[4], xb[4];
          decode8(ka[w], fa, xa);
          decode8(kb[w], fb, xb);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              uint2 qv;
              if constexpr (S::kQShared) qv = qsm[((2 * w + i) * NQ + n) * 32 + lane];
              else qv = qf[n][2 * w + i];
              mma_acc(s[q][n], xa[2 * i], xb[2 * i], xa[2 * i + 1], xb[2 * i + 1], qv.x, qv.y);
            }
        }
      }
      // ---- mask: only the tiles that reach past the first row's last token (unused columns hold q = 0 and go nowhere)
      if (pos0 + TILE > cur.len - p.r + 1) {
#pragma unroll
        for (int q = 0; q < GR; ++q)
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (pos0 + q * 16 + g + (j >> 1) * 8 > last[n][j & 1]) s[q][n][j] = -INFINITY;
      }
      // ---- the maximum (moved only where a score passes it by kSlack)
      float x[NQ][2];
      bool up = false;
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          x[n][e2] = -INFINITY;
#pragma unroll
          for (int q = 0; q < GR; ++q) x[n][e2] = fmaxf(x[n][e2], fmaxf(s[q][n][e2], s[q][n][2 + e2]));
          x[n][e2] *= cs[n][e2];
          up |= x[n][e2] > m[n][e2] + kSlack;
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float f[2];
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            float top = x[n][e2];
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const bool move = top > m[n][e2] + kSlack;  // decided column by column: no row's result depends on another's
            f[e2] = move ? ex2(m[n][e2] - top) : 1.0f;
            if (move) m[n][e2] = top;
            l[n][e2] *= f[e2];
          }
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) O[i][n][j] *= f[j & 1];
        }
      }
      // ---- weights, and P^T as the B operand
      uint32_t pb[GR][NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float2 c2 = make_float2(cs[n][0], cs[n][1]);
        const float2 o2 = make_float2(kShift - (m[n][0] == -INFINITY ? 0.0f : m[n][0]),
                                      kShift - (m[n][1] == -INFINITY ? 0.0f : m[n][1]));
        float2 sum = make_float2(l[n][0], l[n][1]);
#pragma unroll
        for (int q = 0; q < GR; ++q)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float2 z = fma2(make_float2(s[q][n][2 * j], s[q][n][2 * j + 1]), c2, o2);
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            sum = add2(sum, z);
            pb[q][n][j] = transpose8x8(h2u(__floats2half2_rn(z.x, z.y)));
          }
        l[n][0] = sum.x;
        l[n][1] = sum.y;
      }
      // ---- O^T += V^T P^T
      const bool tail = pos0 + TILE > cur.len;  // places past the end hold anything: their scales count as 0
#pragma unroll
      for (int q = 0; q < GR; ++q) {
        const unsigned char *gb = buf + q * 18 * D;
        uint32_t vs4 = *reinterpret_cast<const uint32_t *>(gb + 17 * D + (D == 128 ? g : g >> 1) * 16 + t * 4);
        if (tail) {
          const int n0 = cur.len - (pos0 + q * 16);  // tokens of this group
          const uint32_t keep = (2 * t < n0 ? 0xFFu : 0u) | (2 * t + 1 < n0 ? 0xFF00u : 0u) |
                                (2 * t + 8 < n0 ? 0xFF0000u : 0u) | (2 * t + 9 < n0 ? 0xFF000000u : 0u);
          vs4 &= keep;
        }
        const __half2 s0 = u2h(e4m3x2_to_h2(vs4 & 0xFFFFu)), s1 = u2h(e4m3x2_to_h2(vs4 >> 16));
        uint32_t v[4][D / 64];  // this lane's four tokens
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = t + 4 * j;
          if (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2 *>(gb + 8 * D + row * 64 + (((g >> 2) ^ (t >> 1)) << 5) + (g & 3) * 8);
            v[j][0] = x.x;
            v[j][1 % (D / 64)] = x.y;
          } else {
            v[j][0] = *reinterpret_cast<const uint32_t *>(gb + 8 * D + row * 32 + g * 4);
          }
        }
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          // byte i of lo: channel 2i of the word (token 2t low, 2t + 1 high); of hi: channel 2i + 1
          uint32_t lo0[4], hi0[4], lo1[4], hi1[4];
          decode8((v[0][w] & 0x0F0F0F0Fu) | ((v[1][w] << 4) & 0xF0F0F0F0u), s0, lo0);
          decode8(((v[0][w] >> 4) & 0x0F0F0F0Fu) | (v[1][w] & 0xF0F0F0F0u), s0, hi0);
          decode8((v[2][w] & 0x0F0F0F0Fu) | ((v[3][w] << 4) & 0xF0F0F0F0u), s1, lo1);
          decode8(((v[2][w] >> 4) & 0x0F0F0F0Fu) | (v[3][w] & 0xF0F0F0F0u), s1, hi1);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NQ; ++n)
              mma_acc(O[w * 4 + i][n], lo0[i], hi0[i], lo1[i], hi1[i], pb[q][n][0], pb[q][n][1]);
        }
      }
      __syncwarp();  // every lane has read the slot
      if (ld < n_tiles) load(slot);
      slot ^= 1;
      turn ^= slot == 0;
    }
    // ------------------------------------------------ the segment's end: the warps' parts meet
    const bool done = seg == cur.nt;  // the item lies in this run
    const size_t piece = 2 * (size_t)run + (sg == 0 ? 0 : 1);
    float *mw = stats + flip * 2 * W * S::kRows, *lw = mw + W * S::kRows;
    flip ^= 1;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        float x = l[n][e2];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) {
          mw[warp * S::kRows + n * 8 + 2 * t + e2] = m[n][e2];
          lw[warp * S::kRows + n * 8 + 2 * t + e2] = mine ? x : -1.0f;  // -1: a warp that had no tile
        }
      }
    team_sync();
    if (warp == 0 && alive && at + seg < n_tiles) {  // every warp has read this segment's query rows: the next one's
      Cursor k = cur;
      next_item<TILE>(c, k, HR);
      load_q(k);
    }
    if (mine) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float fw[2];
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < W; ++w) top = fmaxf(top, mw[w * S::kRows + n * 8 + 2 * t + e2]);
          fw[e2] = ex2(m[n][e2] - (top == -INFINITY ? 0.0f : top));
        }
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          float *dst = meet + (size_t)(warp * S::kRows + n * 8 + 2 * t + e2) * S::kLd + g * (D / 8);
#pragma unroll
          for (int i = 0; i < KS; i += 2)  // MMA i: channels 2i and 2i + 1 of this lane's D / 8
            *reinterpret_cast<float4 *>(dst + 2 * i) =
                make_float4(O[i][n][e2] * fw[e2], O[i][n][2 + e2] * fw[e2], O[i + 1][n][e2] * fw[e2],
                            O[i + 1][n][2 + e2] * fw[e2]);
        }
      }
    }
    team_sync();
    const RowGroup rg = row_group(p, cur.hr, S::kRows);
    for (int i = tid; i < rg.rows * (D / 4); i += 32 * W) {
      const int row = i / (D / 4), d4 = i % (D / 4) * 4;
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, mw[w * S::kRows + row]);
      const float safe = top == -INFINITY ? 0.0f : top;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float lx = lw[w * S::kRows + row];
        if (lx == -1.0f) continue;
        sum += lx * ex2(mw[w * S::kRows + row] - safe);
        const float4 y = *reinterpret_cast<const float4 *>(meet + (size_t)(w * S::kRows + row) * S::kLd + d4);
        o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
      }
      if (done) {
        const long long out = ((long long)cur.b * p.r + rg.token(row)) * p.a.Hq + rg.h * p.G + rg.head(row);
        const float inv = sum == 0.0f ? 0.0f : c.vs / sum;
        *reinterpret_cast<uint2 *>(p.a.out + out * D + d4) =
            make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
        if (p.a.lse && d4 == 0) p.a.lse[out] = (top + (log2f(sum) - kShift)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4 *>(p.part + (piece * S::kRows + row) * D + d4) = o;
        if (d4 == 0)
          *reinterpret_cast<float2 *>(p.part + 2 * (size_t)gridDim.x * S::kTeams * S::kRows * D + (piece * S::kRows + row) * 2) =
              make_float2(top, sum);
      }
    }
    // for the join: an item's first piece (-1: it is done) and the run of its last one
    if (tid == 0 && p.extra != kWhole) {
      int32_t *ends = join_ends<D>(p, gridDim.x * S::kTeams, S::kRows) + 2 * ((long long)cur.b * HR + cur.hr);
      if (cur.tile == 0) ends[0] = done ? -1 : (int)piece;
      if (cur.tile + seg == cur.nt) ends[1] = run;
    }
    at += seg;
    if (at < n_tiles) next_item<TILE>(c, cur, HR);
  }
  // A wait gave up: this warp's copies in flight land (or a bounded wait for each ends) before it leaves. It has
  // loaded (ld - warp) / W tiles and taken slot + 2 turn, modulo 4: two, one or none of them are on their way.
  if (!alive) {
    const int held = ((ld - warp) / W - (slot + 2 * (int)turn)) & 3;
    if (held > 0) mbar_wait(my_full + slot, turn);
    if (held > 1) mbar_wait(my_full + (slot ^ 1), slot == 0 ? turn : turn ^ 1u);
  }
}

// Join R rows, from `row`, of pieces j0, j0 + step, ... < np: U at a time are in flight.
template <int D, int U, int R, typename Piece>
GDN_DEV void join_pieces(const float *part, const float *ml, Piece piece, int row, int rows, int j0, int step, int np,
                         float (&m)[R], float (&l)[R], float (&o)[R][D / 32]) {
  constexpr int E = D / 32;
  struct alignas(4 * E) Lane {
    float v[E];
  };
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[i][e] = 0.0f;
  }
  for (; j0 < np; j0 += U * step) {
    float2 v[U][R];
    float y[U][R][E];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        v[u][i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int e = 0; e < E; ++e) y[u][i][e] = 0.0f;
        if (j0 + u * step < np && row + i < rows) {
          const size_t at = piece(j0 + u * step) + row + i;
          v[u][i] = *reinterpret_cast<const float2 *>(ml + at * 2);
          const Lane x = reinterpret_cast<const Lane *>(part + at * D)[lane];
#pragma unroll
          for (int e = 0; e < E; ++e) y[u][i][e] = x.v[e];
        }
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float mn = fmaxf(m[i], v[u][i].x), safe = mn == -INFINITY ? 0.0f : mn;
        const float f = ex2(m[i] - safe), fx = ex2(v[u][i].x - safe);
        l[i] = l[i] * f + v[u][i].y * fx;
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = o[i][e] * f + y[u][i][e] * fx;
        m[i] = mn;
      }
  }
}

// The items that lie in several runs: their pieces, which the decode kernel wrote
// down, are joined in order. Up to eight pieces: a warp per row. More: a warp for
// every eighth of them -- of one row, with a CTA per row (SPLIT, after whole-CTA
// teams: few items of many pieces; eight rows a CTA took 26 us instead of 22 at 16
// sequences of which one has 131072 tokens), else of four rows at a time.
// Bound by latency: two loads, one after the other, and the launch.
// runs, most: as the decode kernel's runs and rows of an item.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(256, 3) kv4_join_kernel(DecodeArgs p, int runs, int most) {
  constexpr int E = D / 32, R = SPLIT ? 1 : 8, H = SPLIT ? 1 : 4;  // rows of the CTA, and at a time
  struct alignas(4 * E) Lane {
    float v[E];
  };
  __shared__ float sh[8][R][D + 4];
  const Kv4Args &c = p.a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, HR = c.Hkv * p.RG, row0 = blockIdx.y * R;
  const float *ml = p.part + 2 * (size_t)runs * most * D;
  const int2 *ends = reinterpret_cast<const int2 *>(join_ends<D>(p, runs, most));
  int b = blockIdx.x / HR;
  RowGroup rg = row_group(p, blockIdx.x - b * HR, most);
  kv4_begin();  // on every path: this grid must not end before the one it follows
  for (long long item = blockIdx.x;;) {
    const int2 e = ends[item];  // the first piece, or -1; then one in each run up to e.y
    const int first = e.x / 2, np = e.y - first + 1;
    auto piece = [&](int j) { return (size_t)(j > 0 ? 2 * (first + j) : e.x) * most; };
    auto put = [&](int row, int ch, float m, float l, auto &v) {  // channels ch ... of a row
      const long long out = ((long long)b * p.r + rg.token(row)) * p.a.Hq + rg.h * p.G + rg.head(row);
      const float inv = l == 0.0f ? 0.0f : c.vs / l;
#pragma unroll
      for (int x = 0; x < (int)(sizeof(v) / sizeof(float)); x += 2)
        *reinterpret_cast<uint32_t *>(p.a.out + out * D + ch + x) = bf16x2(v[x] * inv, v[x + 1] * inv);
      if (p.a.lse && ch == 0) p.a.lse[out] = (m + (log2f(l) - kShift)) * 0.6931471805599453f;
    };
    if (e.x >= 0 && np <= 8) {
      const int row = row0 + warp;
      if (row0 % 8 == 0 && row < rg.rows) {
        float m[1], l[1], o[1][E];
        join_pieces<D, 8>(p.part, ml, piece, row, rg.rows, 0, 1, np, m, l, o);
        put(row, lane * E, m[0], l[0], o[0]);
      }
    } else if (e.x >= 0 && row0 < rg.rows) {
#pragma unroll 1
      for (int i0 = 0; i0 < R; i0 += H) {
        float m[H], l[H], o[H][E];
        join_pieces<D, 8 / H>(p.part, ml, piece, row0 + i0, rg.rows, warp, 8, np, m, l, o);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          Lane x;
#pragma unroll
          for (int k = 0; k < E; ++k) x.v[k] = o[i][k];
          reinterpret_cast<Lane *>(sh[warp][i0 + i])[lane] = x;
          if (lane == 0) {
            sh[warp][i0 + i][D] = m[i];
            sh[warp][i0 + i][D + 1] = l[i];
          }
        }
      }
      __syncthreads();
      for (int x = threadIdx.x; x < R * (D / 2); x += 256) {
        const int i = x / (D / 2), ch = x % (D / 2) * 2;
        if (row0 + i >= rg.rows) break;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < 8; ++w) top = fmaxf(top, sh[w][i][D]);
        const float safe = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f, v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float f = ex2(sh[w][i][D] - safe);
          sum += sh[w][i][D + 1] * f;
          v[0] += sh[w][i][ch] * f;
          v[1] += sh[w][i][ch + 1] * f;
        }
        put(row0 + i, ch, top, sum, v);
      }
      __syncthreads();
    }
    item += gridDim.x;
    if (item >= p.items) return;
    b = (int)item / HR;
    rg = row_group(p, (int)item - b * HR, most);
  }
}

template <int D, int NQ, int TEAM>
cudaError_t launch_decode_t(const DecodeArgs &p, int ctas, cudaStream_t stream) {
  using S = DecodeShape<D, NQ, TEAM>;
  static bool allowed[64];
  cudaError_t e = kv4_allow_smem(kv4_decode_kernel<D, NQ, TEAM>, S::kBytes, allowed);
  if (e != cudaSuccess) return e;
  e = kv4_launch(kv4_decode_kernel<D, NQ, TEAM>, ctas, S::kThreads, S::kBytes, stream, p);
  const int most = ctas * S::kTeams;  // runs, and cuts but one
  if (e != cudaSuccess || p.extra == kWhole || most < 2) return e;
  const int rows = std::min(int(S::kRows), p.r * p.G);
  const dim3 grid(TEAM ? std::min(p.items, 8 * 152) : p.items, TEAM ? (rows + 7) / 8 : rows);
  return kv4_launch(kv4_join_kernel<D, TEAM == 0>, grid, 256, 0, stream, p, most, int(S::kRows));
}

// Query rows per (sequence, KV head) -> 8-row column blocks of one item.
int blocks_of(int R) { return R <= 8 ? 1 : R <= 16 ? 2 : 4; }

// What a kernel's shape says to the host.
struct ShapeInfo {
  int team, teams, tile;
};
template <int D, int NQ>
ShapeInfo shape_info(bool small) {
  if constexpr (!DecodeShape<D, NQ, 0>::kQShared)
    if (small) return {DecodeShape<D, NQ, 4>::kTeam, DecodeShape<D, NQ, 4>::kTeams, DecodeShape<D, NQ, 4>::kTile};
  return {DecodeShape<D, NQ, 0>::kTeam, DecodeShape<D, NQ, 0>::kTeams, DecodeShape<D, NQ, 0>::kTile};
}

struct DecodePlan {
  int NQ, RG, ctas, extra;
  bool small;    // teams of four warps
  size_t bytes;
};
// Everything the host knows: an upper bound of the lengths. Where it says that an
// item takes a team few rounds of tiles, items stay whole: no piece to join.
DecodePlan decode_plan(const Kv4AttnArgs &a, int num_sms) {
  DecodePlan d{};
  const int R = a.c.T / a.c.B * (a.Hq / a.c.Hkv);
  d.NQ = blocks_of(R);
  d.RG = (R + 8 * d.NQ - 1) / (8 * d.NQ);
  const long long items = (long long)a.c.B * a.c.Hkv * d.RG;
  d.small = items >= kManyItems && !(a.c.D == 128 && d.NQ == 4);
  const ShapeInfo s = a.c.D == 128 ? (d.NQ == 1 ? shape_info<128, 1>(d.small) : d.NQ == 2 ? shape_info<128, 2>(d.small)
                                                                                          : shape_info<128, 4>(d.small))
                                   : (d.NQ == 1 ? shape_info<64, 1>(d.small) : d.NQ == 2 ? shape_info<64, 2>(d.small)
                                                                                         : shape_info<64, 4>(d.small));
  const long long most = ((long long)a.c.cols * a.c.page_tokens + s.tile - 1) / s.tile;  // tiles of an item
  d.extra = most <= (long long)s.team * (d.small ? kRoundsTeam : kRoundsCta) ? kWhole : d.small ? kExtraTeam : kExtraCta;
  const long long n = d.extra == kWhole ? items : (items * most + s.team - 1) / s.team;  // runs that could have work
  d.ctas = (int)(n < (long long)num_sms * s.teams ? (n + s.teams - 1) / s.teams : num_sms);
  d.bytes = d.extra == kWhole ? 0 : 2 * (size_t)d.ctas * s.teams * 8 * d.NQ * (a.c.D + 2) * sizeof(float) + 8 * (size_t)items;
  return d;
}

template <int D, int NQ>
cudaError_t launch_decode(const DecodeArgs &p, const DecodePlan &d, cudaStream_t stream) {
  if constexpr (!DecodeShape<D, NQ, 0>::kQShared)
    if (d.small) return launch_decode_t<D, NQ, 4>(p, d.ctas, stream);
  return launch_decode_t<D, NQ, 0>(p, d.ctas, stream);
}

}  // namespace

size_t kv4_decode_bytes(const Kv4AttnArgs &a, int num_sms) { return a.c.T ? decode_plan(a, num_sms).bytes : 0; }

cudaError_t launch_kv4_decode(const Kv4AttnArgs &a, void *workspace, int num_sms, cudaStream_t stream) {
  const DecodePlan d = decode_plan(a, num_sms);
  const int G = a.Hq / a.c.Hkv;
  const DecodeArgs p{a, a.c.T / a.c.B, G, d.RG, (uint32_t)((65536 + G - 1) / G), d.extra, (int)(a.c.B * a.c.Hkv * d.RG),
                     static_cast<float *>(workspace)};
  if (a.c.D == 128)
    return d.NQ == 1 ? launch_decode<128, 1>(p, d, stream) : d.NQ == 2 ? launch_decode<128, 2>(p, d, stream)
                                                                       : launch_decode<128, 4>(p, d, stream);
  return d.NQ == 1 ? launch_decode<64, 1>(p, d, stream) : d.NQ == 2 ? launch_decode<64, 2>(p, d, stream)
                                                                    : launch_decode<64, 4>(p, d, stream);
}

}  // namespace gdn
