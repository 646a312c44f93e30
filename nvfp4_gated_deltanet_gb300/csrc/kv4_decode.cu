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
// elements 2^-27 below the row's largest); the weights 2^(z - m + 14) are
// rounded to FP16 (2^-11 relative, down to 2^-28 of the largest weight); the
// scores, the sums and the output are FP32.
//
// Work: a tile is 64 tokens (32 with more than 16 query rows) of one item = a
// (sequence, KV head, group of query rows). All items' tiles, in order, are
// cut into equal runs, one per CTA -- ragged lengths cost no idle SM -- and a
// run's tiles go round its 8 warps, each with its own ring of stages that it
// fills by bulk copies. At the end of an item (or run) the warps' (m, l, O)
// meet in shared memory; an item that lies in one run is finished there, the
// pieces of others go to the workspace and kv4_join_kernel adds them in order.
#include "kv4.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 8;
constexpr float kShift = 14.0f;  // weights are 2^(z - m + 14): at most 2^14 in FP16, normal down to 2^-28 of that

template <int D, int NQ>
struct DecodeShape {
  static constexpr int kGroups = NQ == 4 ? 2 : 4;           // 16-token groups of a tile
  static constexpr int kTile = kGroups * 16;
  static constexpr int kStage = kGroups * 18 * D;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kRows = 8 * NQ;
  static constexpr int kLd = D + 4;                         // row of the meeting buffer, floats
  static constexpr bool kQShared = D == 128 && NQ == 4;     // 64 registers of q would not fit beside 128 of O
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMeet = kWarps * kRows * kLd * 4;
  static constexpr int kStats = 2 * 2 * kWarps * kRows * 4;  // m and l, two segments
  static constexpr int kQ = kQShared ? (D / 16) * NQ * 32 * 8 : 0;
  static constexpr int kBytes = kRing + kMeet + kStats + kQ + kWarps * kStages * 8;
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};

struct DecodeArgs {
  Kv4AttnArgs a;
  int r, G, RG;      // new tokens per sequence, query heads per KV head, row groups per (sequence, KV head)
  int whole;         // every item fits one CTA's warps: runs hold whole items, nothing to join
  float *part;       // [2 CTAs][rows][D] and, after them, their (m, l) [2 CTAs][rows][2]
};

// Sequence b's tokens, checked (kv4_seq without rows), and its tiles: an empty
// sequence has one tile with no tokens, so that its rows are written.
GDN_DEV int seq_len(const Kv4Args &c, int b) {
  const int n = c.kv_len[b];
  return n < 0 || n > (long long)c.cols * c.page_tokens ? 0 : n;
}
template <int TILE>
GDN_DEV int tiles_of(int len) { return len > 0 ? (len + TILE - 1) / TILE : 1; }

GDN_DEV int warp_isum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// All sequences' tiles (of one KV head and row group).
template <int TILE>
GDN_DEV long long total_tiles(const Kv4Args &c, int lane) {
  long long n = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) n += warp_isum(b0 + lane < c.B ? tiles_of<TILE>(seq_len(c, b0 + lane)) : 0);
  return n;
}
// The sequence that holds unit u of all units (each sequence has HR times its
// tiles of them), and the units before it.
template <int TILE>
GDN_DEV int find_seq(const Kv4Args &c, long long u, int HR, int lane, long long &before) {
  long long base = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const int n = b0 + lane < c.B ? tiles_of<TILE>(seq_len(c, b0 + lane)) : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, (base + incl) * HR > u);
    if (past) {
      const int l = __ffs(past) - 1;
      before = (base + __shfl_sync(0xffffffffu, incl - n, l)) * HR;
      return b0 + l;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  before = 0;
  return -1;
}
// CTAs that share the tiles: each gets at least one per warp.
GDN_DEV int runs(long long units, int ctas) {
  const long long most = (units + kWarps - 1) / kWarps;
  return (int)(most < ctas ? most : ctas);
}

GDN_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
GDN_DEV uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
GDN_DEV __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
// Two E4M3 bytes -> two FP16 (exact)
GDN_DEV uint32_t e4m3x2_to_h2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}
// Eight E2M1 codes times a pair of scales
GDN_DEV void decode8(uint32_t w, __half2 s, uint32_t (&o)[4]) {
  __half2 h[4];
  e2m1x8_to_h2x4(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = h2u(__hmul2(h[i], s));
}

// Where a warp stands in the run: an item and a tile of it.
struct Cursor {
  int b, hr, tile, nt, len;
};
template <int TILE>
GDN_DEV void seek(const Kv4Args &c, Cursor &k, int b) {
  k.b = b;
  k.len = seq_len(c, b);
  k.nt = tiles_of<TILE>(k.len);
}
template <int TILE>
GDN_DEV void advance(const Kv4Args &c, Cursor &k, int step, int HR) {
  while (step >= k.nt - k.tile) {
    step -= k.nt - k.tile;
    k.tile = 0;
    if (++k.hr == HR) {
      k.hr = 0;
      seek<TILE>(c, k, k.b + 1);
    }
  }
  k.tile += step;
}

// This CTA's run: its first tile and how many tiles it has.
template <int TILE>
GDN_DEV long long find_run(const DecodeArgs &p, int HR, int lane, Cursor &k) {
  const Kv4Args &c = p.a.c;
  k.tile = k.hr = k.b = k.nt = k.len = 0;
  if (p.whole) {
    const long long items = (long long)c.B * HR;
    const long long i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
    long long n = 0;
    for (long long i = i0; i < i1; ++i) n += tiles_of<TILE>(seq_len(c, (int)(i / HR)));
    seek<TILE>(c, k, (int)(i0 / HR));
    k.hr = (int)(i0 % HR);
    return n;
  }
  const long long units = total_tiles<TILE>(c, lane) * HR;
  const int N = runs(units, gridDim.x);
  if ((int)blockIdx.x >= N) return 0;
  const long long u0 = units * blockIdx.x / N, u1 = units * (blockIdx.x + 1) / N;
  long long before;
  const int b = find_seq<TILE>(c, u0, HR, lane, before);
  seek<TILE>(c, k, b);
  k.hr = (int)((u0 - before) / k.nt);
  k.tile = (int)((u0 - before) % k.nt);
  return u1 - u0;
}

template <int D, int NQ>
__global__ void __launch_bounds__(kWarps * 32, 1) kv4_decode_kernel(DecodeArgs p) {
  using S = DecodeShape<D, NQ>;
  constexpr int TILE = S::kTile, GR = S::kGroups, KS = D / 16;  // KS: k steps of S, and MMAs of 16 channels of O
  extern __shared__ __align__(128) unsigned char sm[];
  float *meet = reinterpret_cast<float *>(sm + S::kRing);
  float *stats = reinterpret_cast<float *>(sm + S::kRing + S::kMeet);
  uint2 *qsm = reinterpret_cast<uint2 *>(sm + S::kRing + S::kMeet + S::kStats);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::kRing + S::kMeet + S::kStats + S::kQ);
  const Kv4Args &c = p.a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  unsigned char *ring = sm + warp * S::kStages * S::kStage;
  uint64_t *full = bars + warp * S::kStages;
  const int HR = c.Hkv * p.RG, R = p.r * p.G;
  pdl_launch_dependents();  // kv4_join_kernel finds its places meanwhile
  if (lane == 0) {
    for (int s = 0; s < S::kStages; ++s) mbar_init(full + s, 1);
    fence_barrier_init();
  }
  __syncwarp();
  if (blockIdx.x == 0)
    for (int b = tid; b < c.B; b += kWarps * 32)
      if (c.kv_len[b] != seq_len(c, b)) flag_status(c.status, GDN_E_RANGE);

  Cursor cur;
  const long long n_units = find_run<TILE>(p, HR, lane, cur);

  // ------------------------------------------------ this warp's loads: tiles warp, warp + 8, ... of the run
  Cursor load = cur;
  long long load_at = warp;
  if (load_at < n_units) advance<TILE>(c, load, warp, HR);
  auto issue = [&](int s) {  // the warp's next tile into stage s
    const int pos = load.tile * TILE + lane * 16;
    const uint8_t *src = nullptr;
    if (lane < GR && pos < load.len) {
      const int page = c.table[(size_t)load.b * c.cols + pos / c.page_tokens];
      if (page >= 0 && page < c.num_pages)
        src = c.pages + (((size_t)page * c.Hkv + load.hr / p.RG) * (c.page_tokens / 16) + (pos % c.page_tokens) / 16) * (18 * D);
      else
        flag_status(c.status, GDN_E_RANGE);
    }
    const unsigned good = __ballot_sync(0xffffffffu, src != nullptr);
    if (lane == 0) mbar_arrive_expect_tx(full + s, __popc(good) * 18 * D);
    __syncwarp();
    if (src) bulk_g2s(ring + s * S::kStage + lane * 18 * D, src, 18 * D, full + s);
    load_at += kWarps;
    if (load_at < n_units) advance<TILE>(c, load, kWarps, HR);
  };
  for (int s = 0; s < S::kStages; ++s)
    if (load_at < n_units) issue(s);

  int stage = 0, flip = 0;
  uint32_t parity = 0;
  bool alive = true;
  long long at = 0;  // the segment's first tile within the run
  bool first_segment = true;
  while (at < n_units) {
    const int seg = (int)min((long long)(cur.nt - cur.tile), n_units - at);
    const int h = cur.hr / p.RG, row0 = (cur.hr % p.RG) * S::kRows;
    const int rows = min(S::kRows, R - row0);
    const int first = (int)((warp - at % kWarps + kWarps) % kWarps);  // this warp's first tile of the segment
    // ------------------------------------------------ q: B operand, lane (g, t) = row g, channels t D/4 ...
    uint2 qf[S::kQShared ? 1 : NQ][S::kQShared ? 1 : KS];
    float cs[NQ][2];   // sm k_scale log2 e / the row's scale, of columns 2t and 2t + 1
    int last[NQ][2];   // the last token that the row sees
    float O[KS][NQ][4], m[NQ][2], l[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int row = n * 8 + g;
      uint4 w[D / 32];
      const int ri = row0 + row;
      const bool in = row < rows;
      const uint16_t *qp = p.a.q + ((long long)cur.b * p.r + ri / p.G) * p.a.q_stride +
                           (long long)(h * p.G + ri % p.G) * D + t * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) w[i] = in ? reinterpret_cast<const uint4 *>(qp)[i] : make_uint4(0, 0, 0, 0);
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
        const int rr = row0 + n * 8 + 2 * t + e2;
        last[n][e2] = n * 8 + 2 * t + e2 < rows ? cur.len - p.r + rr / p.G : -1;
        m[n][e2] = -INFINITY;
        l[n][e2] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) O[i][n][j] = 0.0f;
    }
    if constexpr (S::kQShared) __syncthreads();

    // ------------------------------------------------ the warp's tiles of this segment
    for (int ti = first; ti < seg && alive; ti += kWarps) {
      if (!__all_sync(0xffffffffu, mbar_wait(full + stage, parity))) {
        flag_status(c.status, GDN_E_TIMEOUT);
        alive = false;
        break;
      }
      const unsigned char *buf = ring + stage * S::kStage;
      const int pos0 = (cur.tile + ti) * TILE;
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
      // ---- running maximum, weights, and P^T as the B operand
      uint32_t pb[GR][NQ][2];
      bool moved = false;
      float f[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          float x = -INFINITY;
#pragma unroll
          for (int q = 0; q < GR; ++q) x = fmaxf(x, fmaxf(s[q][n][e2], s[q][n][2 + e2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = fmaxf(m[n][e2], x * cs[n][e2]);
          const float safe = mn == -INFINITY ? 0.0f : mn;
          f[n][e2] = ex2(m[n][e2] - safe);
          moved |= mn != m[n][e2];
          m[n][e2] = mn;
          const float off = kShift - safe;
          float sum = 0.0f;
#pragma unroll
          for (int q = 0; q < GR; ++q)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float &v = s[q][n][2 * j + e2];
              v = ex2(fmaf(v, cs[n][e2], off));
              sum += v;
            }
          l[n][e2] = fmaf(l[n][e2], f[n][e2], sum);
        }
#pragma unroll
        for (int q = 0; q < GR; ++q)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            pb[q][n][j] = transpose8x8(h2u(__floats2half2_rn(s[q][n][2 * j], s[q][n][2 * j + 1])));
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) O[i][n][j] *= f[n][j & 1];
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
      __syncwarp();  // every lane has read the stage
      if (load_at < n_units) issue(stage);
      if (++stage == S::kStages) {
        stage = 0;
        parity ^= 1u;
      }
    }
    // ------------------------------------------------ the segment's end: the warps' parts meet
    const bool done = seg == cur.nt;  // the item lies in this run
    const size_t slot = 2 * (size_t)blockIdx.x + (first_segment ? 0 : 1);
    float *mw = stats + flip * 2 * kWarps * S::kRows, *lw = mw + kWarps * S::kRows;
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
          lw[warp * S::kRows + n * 8 + 2 * t + e2] = x;
        }
      }
    __syncthreads();
    const int live = min(seg, kWarps);  // warps that had a tile: (at + i) % 8, i < live
    const bool mine = first < seg;
    if (mine) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float fw[2];
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, mw[w * S::kRows + n * 8 + 2 * t + e2]);
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
    __syncthreads();
    const int w0 = (int)(at % kWarps);
    for (int i = tid; i < S::kRows * (D / 4); i += kWarps * 32) {
      const int row = i / (D / 4), d4 = i % (D / 4) * 4;
      if (row >= rows) break;
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, mw[w * S::kRows + row]);
      const float safe = top == -INFINITY ? 0.0f : top;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int j = 0; j < live; ++j) {
        const int w = (w0 + j) & (kWarps - 1);
        sum += lw[w * S::kRows + row] * ex2(mw[w * S::kRows + row] - safe);
        const float4 x = *reinterpret_cast<const float4 *>(meet + (size_t)(w * S::kRows + row) * S::kLd + d4);
        o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
      }
      if (done) {
        const int ri = row0 + row;
        const long long out = ((long long)cur.b * p.r + ri / p.G) * p.a.Hq + h * p.G + ri % p.G;
        const float inv = sum == 0.0f ? 0.0f : c.vs / sum;
        *reinterpret_cast<uint2 *>(p.a.out + out * D + d4) =
            make_uint2(f32_to_bf16_bits(o.x * inv) | (uint32_t)f32_to_bf16_bits(o.y * inv) << 16,
                       f32_to_bf16_bits(o.z * inv) | (uint32_t)f32_to_bf16_bits(o.w * inv) << 16);
        if (p.a.lse && d4 == 0) p.a.lse[out] = (top + (log2f(sum) - kShift)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4 *>(p.part + (slot * S::kRows + row) * D + d4) = o;
        if (d4 == 0)
          *reinterpret_cast<float2 *>(p.part + 2 * (size_t)gridDim.x * S::kRows * D + (slot * S::kRows + row) * 2) =
              make_float2(top, sum);
      }
    }
    at += seg;
    first_segment = false;
    if (at < n_units) advance<TILE>(c, cur, seg, HR);
  }
  if (!alive)  // a wait ran out: give the copies still in flight one more bounded wait each
    for (int s = 0; s < S::kStages; ++s) mbar_wait(full + s, s >= stage ? parity : parity ^ 1u);
}

// The items that lie in several runs: one CTA per query row, its warps taking
// every fourth piece.
template <int D, int NQ>
__global__ void __launch_bounds__(128) kv4_join_kernel(DecodeArgs p, int ctas) {
  using S = DecodeShape<D, NQ>;
  constexpr int E = D / 32;
  __shared__ float sh[4][D + 2];
  const Kv4Args &c = p.a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int HR = c.Hkv * p.RG, R = p.r * p.G;
  const int row_id = blockIdx.x % R, bh = blockIdx.x / R, b = bh / c.Hkv, h = bh % c.Hkv;
  const int hr = h * p.RG + row_id / S::kRows, row = row_id % S::kRows;
  long long units = 0, before = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const int n = b0 + lane < c.B ? tiles_of<S::kTile>(seq_len(c, b0 + lane)) : 0;
    units += warp_isum(n);
    before += warp_isum(b0 + lane < b ? n : 0);
  }
  units *= HR;
  const int nt = tiles_of<S::kTile>(seq_len(c, b));
  const long long a0 = before * HR + (long long)hr * nt;  // the item's tiles are [a0, a0 + nt)
  const int N = runs(units, ctas);
  const int c0 = (int)(((a0 + 1) * N - 1) / units), c1 = (int)(((a0 + nt) * N - 1) / units);
  pdl_wait();  // on every path: this grid must not end before the one it follows
  if (c0 == c1) return;
  float m = -INFINITY, l = 0.0f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  const float *ml = p.part + 2 * (size_t)ctas * S::kRows * D;
  for (int k = c0 + warp; k <= c1; k += 4) {
    const size_t slot = 2 * (size_t)k + (units * k / N >= a0 ? 0 : 1);  // the run's first segment, or its last
    const float2 x = *reinterpret_cast<const float2 *>(ml + (slot * S::kRows + row) * 2);
    const float *op = p.part + (slot * S::kRows + row) * D + lane * E;
    const float mn = fmaxf(m, x.x), safe = mn == -INFINITY ? 0.0f : mn;
    const float f = ex2(m - safe), fx = ex2(x.x - safe);
    l = l * f + x.y * fx;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + op[e] * fx;
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sh[warp][lane * E + e] = o[e];
  if (lane == 0) {
    sh[warp][D] = m;
    sh[warp][D + 1] = l;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float top = fmaxf(fmaxf(sh[0][D], sh[1][D]), fmaxf(sh[2][D], sh[3][D]));
    const float safe = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, v = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = ex2(sh[w][D] - safe);
      sum += sh[w][D + 1] * f;
      v += sh[w][threadIdx.x] * f;
    }
    const long long out = ((long long)b * p.r + row_id / p.G) * p.a.Hq + h * p.G + row_id % p.G;
    p.a.out[out * D + threadIdx.x] = f32_to_bf16_bits(sum == 0.0f ? 0.0f : v * (c.vs / sum));
    if (p.a.lse && threadIdx.x == 0) p.a.lse[out] = (top + (log2f(sum) - kShift)) * 0.6931471805599453f;
  }
}

template <int D, int NQ>
cudaError_t launch_decode_t(DecodeArgs p, int ctas, int num_sms, cudaStream_t stream) {
  using S = DecodeShape<D, NQ>;
  cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  kv4_decode_kernel<D, NQ><<<ctas, kWarps * 32, S::kBytes, stream>>>(p);
  if (p.whole) return cudaGetLastError();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.a.c.B * p.a.Hq * p.r), 1, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NQ>, p, ctas);
}

// Query rows per (sequence, KV head) -> 8-row column blocks of one item.
int blocks_of(int R) { return R <= 8 ? 1 : R <= 16 ? 2 : 4; }

struct DecodePlan {
  int NQ, RG, ctas, whole;
  size_t bytes;
};
// Everything the host knows: an upper bound of the lengths.
DecodePlan decode_plan(const Kv4AttnArgs &a, int num_sms) {
  DecodePlan d{};
  const int R = a.c.T / a.c.B * (a.Hq / a.c.Hkv);
  d.NQ = blocks_of(R);
  d.RG = (R + 8 * d.NQ - 1) / (8 * d.NQ);
  const int tile = d.NQ == 4 ? 32 : 64;
  const long long items = (long long)a.c.B * a.c.Hkv * d.RG;
  const long long most = ((long long)a.c.cols * a.c.page_tokens + tile - 1) / tile;  // tiles of an item
  d.whole = most <= kWarps;
  const long long units = d.whole ? items : (items * most + kWarps - 1) / kWarps;
  d.ctas = (int)(units < num_sms ? units : num_sms);
  d.bytes = d.whole ? 0 : 2 * (size_t)d.ctas * 8 * d.NQ * (a.c.D + 2) * sizeof(float);
  return d;
}

}  // namespace

size_t kv4_decode_bytes(const Kv4AttnArgs &a, int num_sms) { return a.c.T ? decode_plan(a, num_sms).bytes : 0; }

cudaError_t launch_kv4_decode(const Kv4AttnArgs &a, void *workspace, int num_sms, cudaStream_t stream) {
  const DecodePlan d = decode_plan(a, num_sms);
  DecodeArgs p{a, a.c.T / a.c.B, a.Hq / a.c.Hkv, d.RG, d.whole, static_cast<float *>(workspace)};
  if (a.c.D == 128)
    return d.NQ == 1 ? launch_decode_t<128, 1>(p, d.ctas, num_sms, stream)
         : d.NQ == 2 ? launch_decode_t<128, 2>(p, d.ctas, num_sms, stream)
                     : launch_decode_t<128, 4>(p, d.ctas, num_sms, stream);
  return d.NQ == 1 ? launch_decode_t<64, 1>(p, d.ctas, num_sms, stream)
       : d.NQ == 2 ? launch_decode_t<64, 2>(p, d.ctas, num_sms, stream)
                   : launch_decode_t<64, 4>(p, d.ctas, num_sms, stream);
}

}  // namespace gdn
