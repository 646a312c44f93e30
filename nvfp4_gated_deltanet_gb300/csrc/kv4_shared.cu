// Decode attention for sequences that share a prefix (include/gdn.h): a group's
// shared tokens are read once for all rows of the group, what follows them by
// kv4_decode's kernels, and the two joined row by row:
//
//   out = (2^(m0 - m) O0 + 2^(m1 - m) O1) / (2^(m0 - m) l0 + 2^(m1 - m) l1),  m = max(m0, m1)
#include "kv4.cuh"

namespace gdn {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPlanThreads = 256;

// The workspace. Rows of one KV head are numbered row = (batch row) G + (query head of the group).
struct SharedWs {
  int32_t *own_len;    // [B]: a sequence's tokens behind its shared ones
  int32_t *own_table;  // [B][cols]: their pages
  int32_t *seq_group;  // [B]: its group, -1: none
  int32_t *len, *lead; // [groups]: shared tokens (0: none), the sequence through whose pages they are read
  float *own, *own_ml;   // [T][Hq][D], [T][Hq][2]: kv4_decode's sums and their (maximum, weight)
  float *pre, *pre_ml;   // [Hkv][D][rows], [Hkv][rows][2]: the shared tokens'
  void *decode;
};

struct SharedKv4 {
  Kv4SharedArgs s;
  SharedWs w;
  int r, G, rows;  // new tokens per sequence, query heads per KV head, T G
};

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// Lays the workspace out from `base` (which may be null) and returns its size.
size_t lay_out(const Kv4SharedArgs &s, uint8_t *base, int num_sms, SharedWs &w) {
  const Kv4Args &c = s.a.c;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t *p = base + at;
    at += up16(bytes);
    return p;
  };
  const size_t rows = (size_t)c.T * (s.a.Hq / c.Hkv), all = (size_t)c.T * s.a.Hq;
  w.own_len = reinterpret_cast<int32_t *>(take(4 * (size_t)c.B));
  w.own_table = reinterpret_cast<int32_t *>(take(4 * (size_t)c.B * c.cols));
  w.seq_group = reinterpret_cast<int32_t *>(take(4 * (size_t)c.B));
  w.len = reinterpret_cast<int32_t *>(take(4 * (size_t)s.groups));
  w.lead = reinterpret_cast<int32_t *>(take(4 * (size_t)s.groups));
  w.own = reinterpret_cast<float *>(take(4 * all * c.D));
  w.own_ml = reinterpret_cast<float *>(take(8 * all));
  w.pre = reinterpret_cast<float *>(take(4 * rows * c.Hkv * c.D));
  w.pre_ml = reinterpret_cast<float *>(take(8 * rows * c.Hkv));
  w.decode = take(kv4_decode_bytes(s.a, num_sms));
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
    int least = S, first = c.B;
    for (int i = start[g] + tid; i < start[g + 1]; i += kPlanThreads) {
      const int n = kv4_len(c, i);
      if (n > 0) {
        least = min(least, max(n - p.r + 1, 0));
        first = min(first, i);
      }
    }
    __shared__ int sl[kPlanThreads / 32], sf[kPlanThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
    }
    if ((tid & 31) == 0) {
      sl[tid >> 5] = least;
      sf[tid >> 5] = first;
    }
    __syncthreads();
    for (int i = 0; i < kPlanThreads / 32; ++i) {
      least = min(least, sl[i]);
      first = min(first, sf[i]);
    }
    lead = first < c.B ? first : -1;
    S = lead < 0 ? 0 : least / c.page_tokens * c.page_tokens;
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
    p.w.own_len[b] = len - skip;
    p.w.seq_group[b] = skip > 0 ? g : -1;
  }
  const int from = skip / c.page_tokens;
  for (int i = tid; i < c.cols; i += kPlanThreads)
    p.w.own_table[(size_t)b * c.cols + i] = from + i < c.cols ? c.table[(size_t)b * c.cols + from + i] : -1;
}

// A warp per row and KV head.
template <int D>
__global__ void __launch_bounds__(256) kv4_prefix_kernel(SharedKv4 p) {
  kv4_begin();
  const Kv4Args &c = p.s.a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  const int row = blockIdx.x * 8 + warp;
  __shared__ float qs[8][D];
  if (row >= p.rows) return;
  const int tok = row / p.G, b = tok / p.r, g = p.w.seq_group[b];
  if (g < 0) return;
  const int S = p.w.len[g], lead = p.w.lead[g];
  const uint16_t *q = p.s.a.q + (long long)tok * p.s.a.q_stride + (long long)(h * p.G + row - tok * p.G) * D;
  for (int i = lane; i < D; i += 32) qs[warp][i] = bf16_bits_to_f32(q[i]);
  __syncwarp();
  const float cs = p.s.a.sm_scale * c.ks * kLog2e;
  float m = -INFINITY, l = 0.0f, o[D / 32] = {};
  for (int pos0 = 0; pos0 < S; pos0 += 32) {
    const int pos = pos0 + lane;
    const uint8_t *grp = pos < S ? kv4_group<D>(c, lead, pos) : nullptr;
    if (grp) grp += h * kv4_head_bytes<D>(c);
    float z = 0.0f;
    for (int i = 0; i < D / 2 && grp; ++i) {
      const float2 k = __half22float2(e2m1x2_to_h2(grp[kv4_k_code<D>(pos & 15, i)]));
      const float s = e4m3_to_f32(grp[kv4_k_scale<D>(pos & 15, i / 8)]);
      z = fmaf(qs[warp][2 * i], k.x * s, z);
      z = fmaf(qs[warp][2 * i + 1], k.y * s, z);
    }
    z = pos < S ? z * cs : -INFINITY;
    float top = z;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    top = fmaxf(top, m);
    const float f = ex2(m - top), w = ex2(z - top);
    m = top;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= f;
    for (int j = 0; j < 32 && pos0 + j < S; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const uint8_t *gj = reinterpret_cast<const uint8_t *>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(grp), j));
      const int t = (pos0 + j) & 15;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int ch = i * 32 + lane;
        if (!gj) continue;
        const float2 v = __half22float2(e2m1x2_to_h2(gj[kv4_v_code<D>(t, ch / 2)]));
        o[i] = fmaf(wj, (ch & 1 ? v.y : v.x) * e4m3_to_f32(gj[kv4_v_scale<D>(t, ch / 16)]), o[i]);
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) p.w.pre[((size_t)h * D + i * 32 + lane) * p.rows + row] = o[i];
  if (lane == 0) reinterpret_cast<float2 *>(p.w.pre_ml)[(size_t)h * p.rows + row] = make_float2(m, l);
}

// A warp per row: the two parts joined.
template <int D>
__global__ void __launch_bounds__(256) kv4_merge_kernel(SharedKv4 p) {
  kv4_begin();
  const Kv4Args &c = p.s.a.c;
  const int lane = threadIdx.x & 31, h = blockIdx.y, row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  const int tok = row / p.G, b = tok / p.r;
  const long long out = (long long)tok * p.s.a.Hq + h * p.G + row - tok * p.G;
  const bool two = p.w.seq_group[b] >= 0;
  const float2 x = reinterpret_cast<const float2 *>(p.w.own_ml)[out];
  const float2 y = two ? reinterpret_cast<const float2 *>(p.w.pre_ml)[(size_t)h * p.rows + row] : make_float2(-INFINITY, 0.0f);
  const float m = fmaxf(x.x, y.x), safe = m == -INFINITY ? 0.0f : m;
  const float fx = ex2(x.x - safe), fy = ex2(y.x - safe), l = x.y * fx + y.y * fy;
  const float inv = l == 0.0f ? 0.0f : c.vs / l;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int ch = i * 64 + 2 * lane;
    const float2 o = *reinterpret_cast<const float2 *>(p.w.own + out * D + ch);
    float2 v = make_float2(0.0f, 0.0f);
    if (two) {
      const float *pre = p.w.pre + ((size_t)h * D + ch) * p.rows + row;
      v = make_float2(pre[0], pre[p.rows]);
    }
    *reinterpret_cast<uint32_t *>(p.s.a.out + out * D + ch) = bf16x2((o.x * fx + v.x * fy) * inv, (o.y * fx + v.y * fy) * inv);
  }
  if (p.s.a.lse && lane == 0) p.s.a.lse[out] = (m + log2f(l)) * 0.6931471805599453f;
}

template <int D>
cudaError_t launch_t(const SharedKv4 &p, int num_sms, cudaStream_t stream) {
  const Kv4Args &c = p.s.a.c;
  cudaError_t e = kv4_launch(kv4_shared_plan_kernel, c.B + p.s.groups, kPlanThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.rows + 7) / 8, c.Hkv);
  e = kv4_launch(kv4_prefix_kernel<D>, grid, 256, 0, stream, p);
  if (e != cudaSuccess) return e;
  Kv4AttnArgs own = p.s.a;
  own.c.kv_len = p.w.own_len;
  own.c.table = p.w.own_table;
  e = launch_kv4_decode(own, p.w.decode, num_sms, stream, p.w.own, p.w.own_ml);
  if (e != cudaSuccess) return e;
  return kv4_launch(kv4_merge_kernel<D>, grid, 256, 0, stream, p);
}

}  // namespace

size_t kv4_decode_shared_bytes(const Kv4SharedArgs &s, int num_sms) {
  SharedWs w;
  return s.a.c.T ? lay_out(s, nullptr, num_sms, w) : 0;
}

cudaError_t launch_kv4_decode_shared(const Kv4SharedArgs &s, void *workspace, int num_sms, cudaStream_t stream) {
  const int G = s.a.Hq / s.a.c.Hkv;
  SharedKv4 p{s, {}, s.a.c.T / s.a.c.B, G, s.a.c.T * G};
  lay_out(s, static_cast<uint8_t *>(workspace), num_sms, p.w);
  return s.a.c.D == 128 ? launch_t<128>(p, num_sms, stream) : launch_t<64>(p, num_sms, stream);
}

}  // namespace gdn
