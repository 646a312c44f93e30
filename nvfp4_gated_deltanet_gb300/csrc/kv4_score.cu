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
#include "kv4.cuh"
#include "tc.cuh"

namespace gdn {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

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
__global__ void __launch_bounds__(256) kv4_score_kernel(Kv4ScoreArgs p, int chunks, float c2) {
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
        const bool seen = lse != -INFINITY;  // such a row saw nothing
        const float hi = lse * kLog2e, lo = fmaf(lse, kLog2e, -hi) + lse * 1.925963033500899e-8f;  // log2 e - kLog2e
        row_c[x] = c2 * __uint_as_float((uint32_t)(127 - e) << 23);
        row_hi[x] = seen ? hi : 0.0f;
        row_w[x] = seen ? ex2(-lo) : 0.0f;
        row_last[x] = seen ? s.len - n + tok : -1;
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

cudaError_t launch_kv4_score(const Kv4ScoreArgs &p, void *, int, cudaStream_t stream) {
  const Kv4Args &c = p.c;
  const int chunks = (int)(((long long)c.cols * c.page_tokens + kTokChunk - 1) / kTokChunk);
  const float c2 = (float)((double)p.sm_scale * c.ks * 1.4426950408889634074);
  return kv4_launch(c.D == 128 ? kv4_score_kernel<128> : kv4_score_kernel<64>, (unsigned)(chunks * c.Hkv * c.B), 256, 0,
                    stream, p, chunks, c2);
}

}  // namespace gdn
