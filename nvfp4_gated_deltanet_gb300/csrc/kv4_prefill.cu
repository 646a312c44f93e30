// Prefill attention over the 4-bit paged cache (include/gdn.h): ragged prompt
// chunks, causal, on the fifth-generation tensor cores.
//
// What bounds it: 4 d operations per (query row, key) on the tensor cores,
// and beside them one 2^x per (row, key); the cached bytes matter only for a
// chunk of a few tokens. Two kernels:
//
// kv4_expand_kernel decodes every sequence's cache once into tiles of 128
// tokens in FP16 (exact: E2M1 x E4M3 has five significant bits), K as the
// B operand of S = Q K^T and V transposed as the B operand of O += P V, both
// already in the 128-byte swizzle that the MMA reads: each tile is one bulk
// copy, no tensor map. Decoding inside the attention kernel would repeat it for
// every 256 query rows (at 4096 tokens 64 times per KV head) on issue slots
// that the softmax needs.
//
// kv4_prefill_kernel: one CTA per 256 query rows of one KV head -- two tiles of
// 128 rows, a row being a (token, query head of the group), so the whole group
// shares the tiles of K and V. While one tile's scores are in its softmax, the
// tensor cores run the other's products:
//   warps 0..3, 4..7  softmax of row tile 0 / 1, one row per thread: S from
//                     tensor memory, weights back into tensor memory as FP16
//                     in the place of S's second half (the A operand of O += P V)
//   warp 8            TMEM allocation; one thread issues the MMAs
//   warp 9            one thread streams K and V tiles by bulk copies
// A row's weights are 2^(z - m + 6) with a maximum m that is only moved (and O
// rescaled in tensor memory) when the row's true maximum passes it by 8: they
// stay below 2^14, and normal FP16 numbers down to 2^-20 of the largest.
// Rounding as in decode: q in FP16 by a power of two per row (exact but for
// elements 2^-27 below the row's largest), the weights in FP16, all else FP32.
// Every wait is bounded; one that gives up sets GDN_E_TIMEOUT and an abort flag
// that ends every role's loop.
#include "kv4.cuh"
#include "tc.cuh"

namespace gdn {

namespace {

constexpr int kKv = 128;          // tokens of a K / V tile
constexpr int kM = 128;           // rows of a query tile
constexpr int kThreads = 320;
constexpr float kShift = 6.0f;    // weights are 2^(z - m + 6)
constexpr float kSlack = 8.0f;    // how far a row's maximum may pass m before m moves
constexpr float kLog2e = 1.4426950408889634f;

struct PrefillKv4 {
  Kv4AttnArgs a;
  int G, tpt;                     // query heads per KV head; tokens of a query tile: 128 / G
  int cap;                        // K / V tiles (of all KV heads) that the workspace holds
  uint16_t *tiles;                // [cap][Hkv][K: d / 64 x 128 rows x 64, V^T: 2 x d rows x 64] FP16, swizzled
};

GDN_DEV int seq_len(const Kv4Args &c, int b) {
  const int n = c.kv_len[b];
  return n < 0 || n > (long long)c.cols * c.page_tokens ? 0 : n;
}
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
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int x = blockIdx.x / c.Hkv, h = blockIdx.x % c.Hkv;
  int before = 0, total = 0;
  const int b = find_item(c.B, x, lane, [&](int i) { return (seq_len(c, i) + kKv - 1) / kKv; }, before, total);
  if (blockIdx.x == 0) {
    if (tid == 0 && total > p.cap) flag_status(c.status, GDN_E_RANGE);
    for (int i = tid; i < c.B; i += 256) kv4_seq(c, i);  // flags bad entries
  }
  if (b < 0) return;
  const int pos0 = (x - before) * kKv, len = seq_len(c, b);
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
      const __half2 s = __float2half2_rn(e4m3_to_f32(g[kv4_k_scale<D>(row & 15, w / 2)]));
      decode8(*reinterpret_cast<const uint32_t *>(g + kv4_k_code<D>(row & 15, w * 4)), s, o);
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
  static constexpr int kBars = 256;
  static constexpr int kBytes = 1024 + (2 + 2 * kStages) * kTileBytes + kBars;
  static constexpr int kO = 2 * kKv;                 // TMEM columns: S0, S1, then O0, O1
  static_assert(kO + 2 * D <= 512, "tensor memory");
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(PrefillKv4 p) {
  using S = PrefillShape<D>;
  constexpr int NS = S::kStages;
  extern __shared__ uint8_t smraw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  uint8_t *qs = sm, *kbuf = sm + 2 * S::kTileBytes, *vbuf = kbuf + NS * S::kTileBytes;
  uint64_t *k_full = reinterpret_cast<uint64_t *>(vbuf + NS * S::kTileBytes);
  uint64_t *v_full = k_full + NS, *k_free = v_full + NS, *v_free = k_free + NS;
  uint64_t *q_ready = v_free + NS, *s_full = q_ready + 2, *p_ready = s_full + 2, *o_done = p_ready + 4;
  uint64_t *fin = o_done + 2;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(fin + 1);
  volatile uint32_t *abort_flag = tmem_holder + 1;
  const Kv4Args &c = p.a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ------------------------------------------------ which rows: the last, longest ones first
  const int h = blockIdx.x % c.Hkv, x = blockIdx.x / c.Hkv;
  int before = 0, total = 0, unused = 0;
  auto qtiles = [&](int b) {
    const Kv4Seq s = kv4_seq(c, b);
    return (s.q1 - s.q0 + 2 * p.tpt - 1) / (2 * p.tpt);
  };
  find_item(c.B, 0x7fffffff, lane, qtiles, before, total);
  if (x >= total) {
    pdl_wait();  // on every path: this grid must not end before the one it follows
    return;
  }
  const int item = total - 1 - x;
  const int b = find_item(c.B, item, lane, qtiles, before, unused);
  const Kv4Seq seq = kv4_seq(c, b);
  const int n = seq.q1 - seq.q0, t0 = (item - before) * 2 * p.tpt;  // this CTA's first new token
  int tile0 = 0;  // the sequence's first K / V tile
  for (int b0 = 0; b0 < b; b0 += 32) {
    int v = b0 + lane < b ? (seq_len(c, b0 + lane) + kKv - 1) / kKv : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    tile0 += v;
  }
  // K / V tiles that each row tile sees (none where the workspace was too small: flagged by the expansion)
  int nkv[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t1 = min(n, t0 + (i + 1) * p.tpt) - 1;   // the row tile's last token
    const int last = seq.len - n + t1;
    nkv[i] = t1 >= t0 + i * p.tpt && last >= 0 ? last / kKv + 1 : 0;
    if (tile0 + nkv[i] > p.cap) nkv[i] = 0;
  }
  const int nmax = max(nkv[0], nkv[1]);

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(v_full + s, 1);
      mbar_init(k_free + s, 1);
      mbar_init(v_free + s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_ready + i, 128);
      mbar_init(s_full + i, 1);
      mbar_init(p_ready + 2 * i, 128);
      mbar_init(p_ready + 2 * i + 1, 128);
      mbar_init(o_done + i, 1);
    }
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

  if (warp < 8) {
    // ------------------------------------------------ softmax: thread = row r of row tile i
    const int i = warp >> 2, r = tid & 127;
    const int tok = t0 + i * p.tpt + r / p.G;
    const bool in = r < p.tpt * p.G && tok < n;
    const int hq = h * p.G + r % p.G;
    float cs;
    {
      uint4 w[D / 8];
      const uint16_t *qp = p.a.q + (long long)(seq.q0 + tok) * p.a.q_stride + (long long)hq * D;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) w[j] = in ? reinterpret_cast<const uint4 *>(qp)[j] : make_uint4(0, 0, 0, 0);
      uint32_t mx = 0;  // the largest magnitude, as BF16 bits
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const uint32_t y[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = max(mx, max(y[e] & 0x7FFFu, (y[e] >> 16) & 0x7FFFu));
      }
      const int k = min(140 - (int)(mx >> 7), 60);  // 2^k takes the largest to [2^13, 2^14)
      const float sc = __uint_as_float((uint32_t)(k + 127) << 23);
      cs = p.a.sm_scale * c.ks * kLog2e * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const uint32_t y[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        uint32_t z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          z[e] = h2u(__floats2half2_rn(__uint_as_float(y[e] << 16) * sc, __uint_as_float(y[e] & 0xFFFF0000u) * sc));
        *reinterpret_cast<uint4 *>(qs + i * S::kTileBytes + (j / 8) * (kM * 128) + sw_off16(r, (j & 7) * 8)) =
            make_uint4(z[0], z[1], z[2], z[3]);
      }
      fence_async_shared();
      mbar_arrive(q_ready + i);
    }
    const int last = in ? seq.len - n + tok : -1;               // the last token this row sees
    const int sure = seq.len - n + t0 + i * p.tpt;              // every row of the tile sees up to here
    const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = base + i * kKv, tO = base + S::kO + i * D;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < nkv[i]; ++j) {
      if (!__all_sync(0xffffffffu, wait_or_abort(s_full + i, (uint32_t)(j & 1), abort_flag, c.status))) { ok = false; break; }
      tc_fence_after();
      const bool mask = j * kKv + kKv - 1 > sure;
      // Half of the scores at a time (64 registers): the second half's weights
      // take the place of its own scores, columns 96..127, and go to the MMAs
      // while the first half is read again and its weights, columns 64..95, are made.
      float s[64];
      auto fetch = [&](int half) {
        uint32_t raw[64];
        tmem_ld32(tS + 64 * half, raw);
        tmem_ld32(tS + 64 * half + 32, raw + 32);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 64; ++q) s[q] = __uint_as_float(raw[q]);
        if (mask) {
#pragma unroll
          for (int q = 0; q < 64; ++q)
            if (j * kKv + 64 * half + q > last) s[q] = -INFINITY;
        }
      };
      float x4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto largest = [&]() {
#pragma unroll
        for (int q = 0; q < 64; q += 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) x4[e] = fmaxf(x4[e], s[q + e]);
      };
      fetch(0);
      largest();
      fetch(1);
      largest();
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
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float2 z = fma2(make_float2(s[2 * e], s[2 * e + 1]), cs2, off2);
          z.x = ex2(z.x);
          z.y = ex2(z.y);
          sum[e & 1] = add2(sum[e & 1], z);
          w[e] = h2u(__floats2half2_rn(z.x, z.y));
        }
        tmem_st32(tS + 64 + 32 * half, w);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_ready + 2 * i + half);
      };
      weigh(1);
      fetch(0);
      weigh(0);
      sum[0] = add2(sum[0], sum[1]);
      l = sum[0].x + sum[0].y;
    }
    // ------------------------------------------------ the rows' results
    const bool any = nkv[i] > 0 && ok && warp_wait(o_done + i, 0, abort_flag, c.status);
    tc_fence_after();
    const float inv = l == 0.0f ? 0.0f : c.vs / l;
    uint16_t *op = p.a.out + ((long long)(seq.q0 + tok) * p.a.Hq + hq) * D;
#pragma unroll
    for (int q = 0; q < D; q += 32) {
      uint32_t o[32];
      if (any) {
        tmem_ld32(tO + q, o);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        w[e] = f32_to_bf16_bits(__uint_as_float(o[2 * e]) * inv) | (uint32_t)f32_to_bf16_bits(__uint_as_float(o[2 * e + 1]) * inv) << 16;
      if (in) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          reinterpret_cast<uint4 *>(op + q)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
      }
    }
    if (in && p.a.lse)
      p.a.lse[(long long)(seq.q0 + tok) * p.a.Hq + hq] = (m + (log2f(l) - kShift)) * 0.6931471805599453f;
  } else if (warp == 8) {
    // ------------------------------------------------ MMAs
    if (nmax > 0 && elect_one()) {
      constexpr uint32_t idS = idesc_f16(kKv), idO = idesc_f16(D);
      constexpr uint64_t kStep = S::kTileBytes / 16;  // from one stage or tile to the next, in a descriptor
      const uint64_t qd = desc_sw128(smem_u32(qs)), kd = desc_sw128(smem_u32(kbuf)), vd = desc_sw128(smem_u32(vbuf));
      auto wait = [&](uint64_t *bar, int use) { return wait_or_abort(bar, (uint32_t)(use & 1), abort_flag, c.status); };
      auto scores = [&](int i, int j) {  // S_i = Q_i K_j^T
        const uint64_t q = qd + i * kStep, kk = kd + (uint64_t)(j % NS) * kStep;
        const uint32_t d = tmem + i * kKv;
        mma_f16_ss_c<false>(d, q, kk, idS);
#pragma unroll
        for (int k = 1; k < D / 16; ++k)
          mma_f16_ss_c<true>(d, q + (k / 4) * (kM * 128 / 16) + 2 * (k & 3), kk + (k / 4) * (kKv * 128 / 16) + 2 * (k & 3), idS);
        tc_commit(s_full + i);
      };
      bool ok = wait(q_ready, 0) && wait(q_ready + 1, 0) && wait(k_full, 0);
      auto values = [&](int i, int j) {  // O_i += P_i V_j
        const uint64_t v = vd + (uint64_t)(j % NS) * kStep;
        const uint32_t d = tmem + S::kO + i * D, a = tmem + i * kKv + 64;
        if (!(ok = wait(p_ready + 2 * i + 1, j))) return;  // tokens 64..127 first
        tc_fence_after();
        if (j == 0) mma_f16_ts_c<false>(d, a + 32, v + D * 128 / 16, idO);
        else mma_f16_ts_c<true>(d, a + 32, v + D * 128 / 16, idO);
#pragma unroll
        for (int k = 1; k < 4; ++k) mma_f16_ts_c<true>(d, a + 32 + 8 * k, v + D * 128 / 16 + 2 * k, idO);
        if (!(ok = wait(p_ready + 2 * i, j))) return;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16_ts_c<true>(d, a + 8 * k, v + 2 * k, idO);
      };
      if (ok) {
        tc_fence_after();
        for (int i = 0; i < 2; ++i)
          if (nkv[i] > 0) scores(i, 0);
        tc_commit(k_free);
      }
      for (int j = 0; j < nmax && ok; ++j) {
        ok = wait(v_full + j % NS, j / NS) && (j + 1 >= nmax || wait(k_full + (j + 1) % NS, (j + 1) / NS));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!ok || j >= nkv[i]) continue;
          values(i, j);
          if (!ok) break;
          if (j + 1 < nkv[i]) scores(i, j + 1);
          else tc_commit(o_done + i);
        }
        if (!ok) break;
        tc_commit(v_free + j % NS);
        if (j + 1 < nmax) tc_commit(k_free + (j + 1) % NS);
      }
      // every MMA issued has completed before the CTA may leave
      tc_commit(fin);
      mbar_wait(fin, 0u);
    }
  } else if (lane == 0) {
    // ------------------------------------------------ K and V tiles
    pdl_wait();  // the expansion has finished
    const uint8_t *src = reinterpret_cast<const uint8_t *>(p.tiles) + ((size_t)tile0 * c.Hkv + h) * (2 * S::kTileBytes);
    const size_t step = (size_t)c.Hkv * 2 * S::kTileBytes;
    int j = 0;
    for (; j < nmax; ++j) {
      const int s = j % NS, u = j / NS;
      if (u > 0 && !wait_or_abort(k_free + s, (uint32_t)((u - 1) & 1), abort_flag, c.status)) break;
      mbar_arrive_expect_tx(k_full + s, S::kTileBytes);
      bulk_g2s(kbuf + s * S::kTileBytes, src + j * step, S::kTileBytes, k_full + s);
      if (u > 0 && !wait_or_abort(v_free + s, (uint32_t)((u - 1) & 1), abort_flag, c.status)) break;
      mbar_arrive_expect_tx(v_full + s, S::kTileBytes);
      bulk_g2s(vbuf + s * S::kTileBytes, src + j * step + S::kTileBytes, S::kTileBytes, v_full + s);
    }
    if (*abort_flag)  // the copies in flight land (or a bounded wait for each ends) before the CTA leaves
      for (int s = 0; s < NS; ++s) {
        const int uses = (j + NS - 1 - s) / NS;
        if (uses > 0) {
          mbar_wait(k_full + s, (uint32_t)((uses - 1) & 1));
          mbar_wait(v_full + s, (uint32_t)((uses - 1) & 1));
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
cudaError_t launch_prefill_t(const PrefillKv4 &p, cudaStream_t stream) {
  using S = PrefillShape<D>;
  static bool allowed[64];
  cudaError_t e = kv4_allow_smem(kv4_prefill_kernel<D>, S::kBytes, allowed);
  if (e != cudaSuccess) return e;
  const Kv4Args &c = p.a.c;
  kv4_expand_kernel<D><<<(unsigned)p.cap * c.Hkv, 256, 0, stream>>>(p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(c.T / (2 * p.tpt) + c.B) * c.Hkv, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_prefill_kernel<D>, p);
}

// K / V tiles: every sequence's last one may be partly filled.
long long tile_cap(const Kv4AttnArgs &a, long long total_kv) { return total_kv / kKv + a.c.B; }

}  // namespace

// 0 where the tiles would pass what a grid can index.
size_t kv4_prefill_bytes(const Kv4AttnArgs &a, long long total_kv) {
  const long long n = tile_cap(a, total_kv) * a.c.Hkv;
  return n > 0x7fffffffLL ? 0 : (size_t)n * 4 * kKv * a.c.D;
}

cudaError_t launch_kv4_prefill(const Kv4AttnArgs &a, long long total_kv, void *workspace, cudaStream_t stream) {
  const int G = a.Hq / a.c.Hkv;
  const PrefillKv4 p{a, G, kM / G, (int)tile_cap(a, total_kv), static_cast<uint16_t *>(workspace)};
  return a.c.D == 128 ? launch_prefill_t<128>(p, stream) : launch_prefill_t<64>(p, stream);
}

}  // namespace gdn
