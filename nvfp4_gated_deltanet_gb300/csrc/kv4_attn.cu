// Softmax attention over the 4-bit paged cache, plainly: one warp per (row,
// query head), one key at a time, FP32 throughout.
#include "kv4.cuh"

namespace gdn {

namespace {

template <int D>
__global__ void __launch_bounds__(128) kv4_attention_kernel(Kv4AttnArgs a) {
  constexpr int EPL = D / 32;  // elements of a row that a lane holds: 2 or 4
  const int lane = threadIdx.x & 31;
  const long long item = blockIdx.x * 4LL + (threadIdx.x >> 5);
  if (item >= (long long)a.c.T * a.Hq) return;
  const int n = (int)(item / a.Hq), hq = (int)(item % a.Hq), h = hq / (a.Hq / a.c.Hkv);
  const int b = kv4_seq_of(a.c, n);
  if (b < 0) return;
  const Kv4Seq s = kv4_seq(a.c, b);
  if (n < s.q0 || n >= s.q1) return;
  const int last = s.len - (s.q1 - s.q0) + (n - s.q0);  // the last token this row sees
  float q[EPL], o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) {
    q[e] = bf16_bits_to_f32(a.q[n * a.q_stride + (long long)hq * D + lane * EPL + e]);
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const float c = a.sm_scale * a.c.ks;
  for (int pos = 0; pos <= last; ++pos) {
    const uint8_t *g = kv4_group<D>(a.c, b, pos);
    if (!g) continue;
    g += h * kv4_head_bytes<D>(a.c);
    const int t = pos & 15, blk = lane * EPL / 16;
    const float ks = e4m3_to_f32(g[kv4_k_scale<D>(t, blk)]), vs = e4m3_to_f32(g[kv4_v_scale<D>(t, blk)]);
    float z = 0.0f, v[EPL];
#pragma unroll
    for (int e = 0; e < EPL; e += 2) {
      const int i = (lane * EPL + e) / 2;
      const float2 kk = __half22float2(e2m1x2_to_h2(g[kv4_k_code<D>(t, i)]));
      const float2 vv = __half22float2(e2m1x2_to_h2(g[kv4_v_code<D>(t, i)]));
      z = fmaf(q[e], kk.x * ks, fmaf(q[e + 1], kk.y * ks, z));
      v[e] = vv.x * vs;
      v[e + 1] = vv.y * vs;
    }
    z = warp_sum(z) * c;
    const float mn = fmaxf(m, z), f = expf(m - mn), p = expf(z - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] = fmaf(o[e], f, p * v[e]);
    m = mn;
  }
  const float inv = l > 0.0f ? a.c.vs / l : l == 0.0f ? 0.0f : l;  // a NaN sum stays NaN
#pragma unroll
  for (int e = 0; e < EPL; ++e)
    a.out[((long long)n * a.Hq + hq) * D + lane * EPL + e] = f32_to_bf16_bits(o[e] * inv);
  if (a.lse && lane == 0) a.lse[(long long)n * a.Hq + hq] = m + logf(l);
}

}  // namespace

cudaError_t launch_kv4_attention(const Kv4AttnArgs &a, cudaStream_t stream) {
  const long long items = (long long)a.c.T * a.Hq;
  if (items == 0 || a.c.B == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)((items + 3) / 4);
  if (a.c.D == 128)
    kv4_attention_kernel<128><<<blocks, 128, 0, stream>>>(a);
  else
    kv4_attention_kernel<64><<<blocks, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
