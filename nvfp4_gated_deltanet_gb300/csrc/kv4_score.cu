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
constexpr int kUnit = 64;
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
  // ---- loads: where the groups of the next eight units lie is worked out at once, a group per lane
  Unit ahead = cur;              // the unit that is loaded next
  int ahead_left = left, ahead_i = 8;
  const uint8_t *where = nullptr;
  auto look = [&]() {
    if (ahead_i == 8) {
      ahead_i = 0;
      where = nullptr;
      Unit k = ahead;
      if (lane / 4 < ahead_left) {
        for (int i = 0; i < lane / 4; ++i) next_unit(c, k);
        const int pos = k.pos + (lane & 3) * 16;
        if (pos < k.len) {
          where = kv4_group<D>(c, k.b, pos);
          if (where) where += k.h * kv4_head_bytes<D>(c);
        }
      }
    }
  };
  uint32_t kw[4][2][W];  // [group][token g, g + 8]: 16 (d = 64: 8) code bytes, and their scales
  uint32_t ks[4][2];
  auto load = [&](int q) {
    const uint8_t *src = reinterpret_cast<const uint8_t *>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(where), ahead_i * 4 + q));
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int tok = g + 8 * x;
      if constexpr (D == 128) {
        const uint4 v = src ? __ldg(reinterpret_cast<const uint4 *>(src + kv4_k_code<D>(tok, t * 16))) : make_uint4(0, 0, 0, 0);
        kw[q][x][0] = v.x, kw[q][x][1] = v.y, kw[q][x][2 % W] = v.z, kw[q][x][3 % W] = v.w;
        ks[q][x] = src ? __ldg(reinterpret_cast<const uint16_t *>(src + kv4_k_scale<D>(tok, 2 * t))) : 0u;
      } else {
        const uint2 v = src ? __ldg(reinterpret_cast<const uint2 *>(src + kv4_k_code<D>(tok, t * 8))) : make_uint2(0, 0);
        kw[q][x][0] = v.x, kw[q][x][1] = v.y;
        ks[q][x] = src ? __ldg(src + kv4_k_scale<D>(tok, t)) : 0u;
      }
    }
  };
  auto loaded = [&]() {
    ++ahead_i;
    if (--ahead_left > 0 && ahead_i == 8)
      for (int i = 0; i < 8; ++i) next_unit(c, ahead);  // (eight more units were looked up, so eight are behind)
  };
  look();
#pragma unroll
  for (int q = 0; q < 4; ++q) load(q);
  loaded();

  uint2 qf[NQ][KS];              // B operand: lane (g, t) = row g of the block, channels t D / 4 ...
  float rc[NQ][2], hi[NQ][2], wt[NQ][2];
  int last[NQ][2];
  int at_b = -1, at_h = -1, slot = -1, scored = 0, rows_b = 0;
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
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          rc[nq][e2] = c2 * __shfl_sync(0xffffffffu, __uint_as_float((uint32_t)(127 - e) << 23), (2 * t + e2) * 4);
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
    const bool edge = cur.pos + kUnit > cur.len - rows_b + 1;
    const bool more = left > 1;
    if (more) look();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
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
            // a weight of 0 belongs to a row that is none (its z may be anything)
            if (edge ? cur.pos + q * 16 + g + 8 * x <= last[nq][e2] : wt[nq][e2] != 0.0f) v[x] = fmaf(z, wt[nq][e2], v[x]);
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

// 32 tokens of one head as the A operand of S^T = K Q^T, m16n8k16: lane (g, t)
// holds tokens g and g + 8 of two groups, 16 (d = 64: 8) consecutive code bytes of
// each -- the k order is free. Exact in FP16.
template <int D>
struct KeyRows {
  uint32_t a[2][D / 32][2][4];  // [group][word][token g, g + 8][channel pairs]
  GDN_DEV void load(const uint8_t *const (&grp)[2], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int tok = g + 8 * x;
        uint32_t w[D / 32];
        float s[D / 64 + 1];
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          w[i] = grp[q] ? reinterpret_cast<const uint32_t *>(grp[q] + kv4_k_code<D>(tok, 0))[t * (D / 32) + i] : 0u;
#pragma unroll
        for (int i = 0; i < (D == 128 ? 2 : 1); ++i)
          s[i] = grp[q] ? e4m3_to_f32(grp[q][kv4_k_scale<D>(tok, t * (D == 128 ? 2 : 1) + i)]) : 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) decode8(w[i], __float2half2_rn(s[i / 2]), a[q][i][x]);
      }
  }
};

constexpr int kRowChunk = 64;   // query rows in shared memory at once
constexpr int kTokChunk = 256;  // tokens of a CTA

template <int D>
__global__ void __launch_bounds__(256) kv4_score_kernel(Kv4ScoreArgs p, int chunks, float c2, float skew) {
  constexpr int KS = D / 16;
  __shared__ uint2 qsm[kRowChunk / 8][KS][32];
  __shared__ float row_c[kRowChunk], row_hi[kRowChunk], row_w[kRowChunk];
  __shared__ int row_last[kRowChunk];
  kv4_begin();
  const Kv4Args &c = p.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int chunk = blockIdx.x % chunks, h = blockIdx.x / chunks % c.Hkv, b = blockIdx.x / chunks / c.Hkv;
  const Kv4Seq s = kv4_seq(c, b);
  if (chunk * kTokChunk >= s.len) return;
  const int slot = score_slot(p, b, s.len);
  if (slot < 0 || slot_twice(p, b, slot, lane)) return;
  const int G = p.Hq / c.Hkv, n = s.q1 - s.q0, R = n * G;
  const int pos0 = chunk * kTokChunk + warp * 32;
  const uint8_t *grp[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    grp[q] = pos0 + q * 16 < s.len ? kv4_group<D>(c, b, pos0 + q * 16) : nullptr;
    if (grp[q]) grp[q] += h * kv4_head_bytes<D>(c);
  }
  KeyRows<D> k;
  k.load(grp, lane);
  float acc[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // tokens g, g + 8 of both groups, this lane's columns
  for (int row0 = 0; row0 < R; row0 += kRowChunk) {
    __syncthreads();
    {  // q: B operand, lane (g, t) = row g of the warp's eight, channels t D/4 ...; scaled to FP16 by a power of two
      const int row = row0 + warp * 8 + g, tok = row / G;
      uint4 w[D / 32];
      const uint16_t *src = p.q + (long long)(s.q0 + tok) * p.q_stride + (long long)(h * G + row - tok * G) * D + t * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) w[i] = row < R ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = max(mx, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = min(140 - (int)(mx >> 7), 60);
      const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[j] = h2u(__floats2half2_rn(__uint_as_float(x[j] << 16) * sc, __uint_as_float(x[j] & 0xFFFF0000u) * sc));
        qsm[warp][2 * i][lane] = make_uint2(y[0], y[1]);
        qsm[warp][2 * i + 1][lane] = make_uint2(y[2], y[3]);
      }
      if (t == 0) {
        const int x = warp * 8 + g;
        const float lse = row < R ? p.lse[(long long)(s.q0 + tok) * p.Hq + h * G + row - tok * G] : -INFINITY;
        const RowWeight rw = row_weight(lse, skew);
        row_c[x] = c2 * __uint_as_float((uint32_t)(127 - e) << 23);
        row_hi[x] = rw.hi;
        row_w[x] = rw.w;
        row_last[x] = lse == -INFINITY ? -1 : s.len - n + tok;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int nb = 0; nb < kRowChunk / 8 && row0 + nb * 8 < R; ++nb) {
      float d[2][4] = {};
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const uint2 qv = qsm[nb][i][lane];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          mma_acc(d[q], k.a[q][i / 2][0][2 * (i & 1)], k.a[q][i / 2][1][2 * (i & 1)], k.a[q][i / 2][0][2 * (i & 1) + 1],
                  k.a[q][i / 2][1][2 * (i & 1) + 1], qv.x, qv.y);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int x = nb * 8 + 2 * t + e;
        const float rc = row_c[x], hi = row_hi[x], w = row_w[x];
        const int last = row_last[x];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (pos0 + q * 16 + g + 8 * y <= last) acc[q][y] = fmaf(ex2(fmaf(d[q][2 * y + e], rc, -hi)), w, acc[q][y]);
      }
    }
  }
  const int scored = p.scored ? p.scored[b] : s.len;
  const size_t row = ((size_t)slot * c.Hkv + h) * p.s.tokens;
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float v = acc[q][y];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      const int pos = pos0 + q * 16 + g + 8 * y;
      if (t == 0 && pos < s.len) p.s.out[row + pos] = v + (pos < scored ? p.s.in[row + pos] : 0.0f);
    }
}

}  // namespace

size_t kv4_score_bytes(const Kv4ScoreArgs &, int) { return 0; }

template <int D, int NQ>
cudaError_t launch_rows(const Kv4ScoreArgs &p, float c2, float skew, int num_sms, cudaStream_t stream) {
  const Kv4Args &c = p.c;
  const long long units = (long long)c.B * c.Hkv * (((long long)c.cols * c.page_tokens + kUnit - 1) / kUnit);  // at most
  const int most = num_sms * (NQ == 1 ? 2 : 1);
  return kv4_launch(kv4_score_rows_kernel<D, NQ>, (unsigned)std::min((long long)most, (units + kRowWarps - 1) / kRowWarps),
                    32 * kRowWarps, 0, stream, p, c2, skew);
}

cudaError_t launch_kv4_score(const Kv4ScoreArgs &p, void *, int num_sms, cudaStream_t stream) {
  const Kv4Args &c = p.c;
  const double exact = (double)p.sm_scale * c.ks * 1.4426950408889634074;  // a score in bits
  const float c2 = (float)exact, skew = (float)(exact / c2 - 1.0);
  const int R = c.q_start ? 0 : c.T / c.B * (p.Hq / c.Hkv);  // rows per sequence and KV head, where they are known
  if (!c.q_start && R <= 8) return c.D == 128 ? launch_rows<128, 1>(p, c2, skew, num_sms, stream) : launch_rows<64, 1>(p, c2, skew, num_sms, stream);
  if (!c.q_start && R <= 16) return c.D == 128 ? launch_rows<128, 2>(p, c2, skew, num_sms, stream) : launch_rows<64, 2>(p, c2, skew, num_sms, stream);
  const int chunks = (int)(((long long)c.cols * c.page_tokens + kTokChunk - 1) / kTokChunk);
  return kv4_launch(c.D == 128 ? kv4_score_kernel<128> : kv4_score_kernel<64>, (unsigned)(chunks * c.Hkv * c.B), 256, 0,
                    stream, p, chunks, c2, skew);
}

}  // namespace gdn
