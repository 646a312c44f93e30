// The 4-bit KV cache's data movement: new tokens into pages, tokens read back,
// pages copied and compacted.
#include "kv4.cuh"

namespace gdn {

namespace {

// New rows into their pages, or back. One CTA per 16-token group that the new
// rows touch and a few heads: its threads take one 16-element block of one token
// each (append: 32 bytes in, 8 code bytes out). The group's scales are gathered in
// shared memory and leave as 16-byte words where all of its tokens are new: a V
// scale is a byte 16 bytes from its neighbours in the token, and single bytes of
// 16 tokens cost more memory transactions than all the codes.
// Bound by the bytes: 4 d per token-head and K or V read or written in BF16, 9/16 d in 4 bits.
constexpr int kHeads = 8;  // of a CTA, at most

struct RowsArgs {
  Kv4Args a;
  uint16_t *k, *v;
  long long k_stride, v_stride;
  int heads;  // of a CTA
};

template <int D, bool READ>
__global__ void __launch_bounds__(256) kv4_rows_kernel(RowsArgs p) {
  constexpr int NB = D / 16, ITEMS = 2 * 16 * NB;  // of a head: K and V blocks of 16 tokens
  constexpr int U = 2;
  __shared__ int sb, sgroup;
  __shared__ __align__(16) uint8_t scales[kHeads * 2 * D];
  const Kv4Args &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {  // the sequence and its group: the blockIdx.x-th that new rows touch
    int base = 0, found = -1, group = 0;
    for (int b0 = 0; b0 < a.B && found < 0; b0 += 32) {
      int n = 0, g0 = 0;
      if (b0 + lane < a.B) {
        const Kv4Seq s = kv4_seq(a, b0 + lane);
        const int lo = max(0, s.len - (s.q1 - s.q0));
        g0 = lo >> 4;
        n = s.q1 > s.q0 && s.len > lo ? ((s.len - 1) >> 4) - g0 + 1 : 0;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, base + incl > (int)blockIdx.x);
      if (past) {
        const int l = __ffs(past) - 1;
        found = b0 + l;
        group = __shfl_sync(0xffffffffu, g0 - (base + incl - n), l) + (int)blockIdx.x;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      sb = found;
      sgroup = group;
    }
  }
  __syncthreads();
  const int b = sb;
  if (b < 0) return;
  const Kv4Seq s = kv4_seq(a, b);
  const int first = s.len - (s.q1 - s.q0), pos0 = sgroup * 16;  // the first new token; the group's
  const int t0 = max(0, max(first, 0) - pos0), t1 = min(16, s.len - pos0);  // the group's new tokens
  uint8_t *g = kv4_group<D>(a, b, pos0);
  if (!g) return;
  const int h0 = blockIdx.y * p.heads, hn = min(p.heads, a.Hkv - h0);
  const size_t head = kv4_head_bytes<D>(a);
  const float invk = inv6ts_of(a.ks), invv = inv6ts_of(a.vs);
  for (int i0 = tid; i0 < hn * ITEMS; i0 += 256 * U) {
    uint4 x[U][2];
    uint2 code[U];
    uint8_t sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 256 * u, blk = i % NB, t = i / NB % 16, is_v = i / (16 * NB) & 1, h = i / ITEMS;
      if (i >= hn * ITEMS || t < t0 || t >= t1) continue;
      if (READ) {
        const uint8_t *q = g + (h0 + h) * head;
        code[u] = *reinterpret_cast<const uint2 *>(q + (is_v ? kv4_v_code<D>(t, blk * 8) : kv4_k_code<D>(t, blk * 8)));
        sc[u] = q[is_v ? kv4_v_scale<D>(t, blk) : kv4_k_scale<D>(t, blk)];
      } else {
        const long long n = s.q0 + (pos0 + t - first);
        const uint4 *row = reinterpret_cast<const uint4 *>((is_v ? p.v + n * p.v_stride : p.k + n * p.k_stride) +
                                                           (h0 + h) * D + blk * 16);
        x[u][0] = row[0];
        x[u][1] = row[1];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 256 * u, blk = i % NB, t = i / NB % 16, is_v = i / (16 * NB) & 1, h = i / ITEMS;
      if (i >= hn * ITEMS || t < t0 || t >= t1) continue;
      const float ts = is_v ? a.vs : a.ks;
      if (READ) {
        __half2 e[8];
        e2m1x8_to_h2x4(code[u].x, *reinterpret_cast<__half2(*)[4]>(&e[0]));
        e2m1x8_to_h2x4(code[u].y, *reinterpret_cast<__half2(*)[4]>(&e[4]));
        const float f = e4m3_to_f32(sc[u]);
        uint32_t o[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const float2 y = __half22float2(e[m]);  // e2m1 x e4m3 is exact; one FP32 rounding by ts, one to BF16
          o[m] = f32_to_bf16_bits(y.x * f * ts) | (uint32_t)f32_to_bf16_bits(y.y * f * ts) << 16;
        }
        const long long n = s.q0 + (pos0 + t - first);
        uint4 *row = reinterpret_cast<uint4 *>((is_v ? p.v + n * p.v_stride : p.k + n * p.k_stride) + (h0 + h) * D + blk * 16);
        row[0] = make_uint4(o[0], o[1], o[2], o[3]);
        row[1] = make_uint4(o[4], o[5], o[6], o[7]);
      } else {
        float y[16];
        const uint32_t w[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          y[2 * m] = __uint_as_float(w[m] << 16);
          y[2 * m + 1] = __uint_as_float(w[m] & 0xFFFF0000u);
        }
        uint32_t lo, hi, scale;
        if (!quant_block16(y, ts, is_v ? invv : invk, lo, hi, scale)) flag_status(a.status, GDN_E_NONFINITE);
        *reinterpret_cast<uint2 *>(g + (h0 + h) * head + (is_v ? kv4_v_code<D>(t, blk * 8) : kv4_k_code<D>(t, blk * 8))) =
            make_uint2(lo, hi);
        scales[h * 2 * D + (is_v ? kv4_v_scale<D>(t, blk) : kv4_k_scale<D>(t, blk)) - 16 * D] = (uint8_t)scale;
      }
    }
  }
  if (READ) return;
  __syncthreads();
  if (t0 == 0 && t1 == 16) {
    for (int i = tid; i < hn * (2 * D / 16); i += 256) {
      const int h = i / (2 * D / 16), w = i % (2 * D / 16);
      reinterpret_cast<uint4 *>(g + (h0 + h) * head + 16 * D)[w] = reinterpret_cast<const uint4 *>(scales + h * 2 * D)[w];
    }
  } else {  // the other tokens' scales stay
    for (int i = tid; i < hn * ITEMS; i += 256) {
      const int blk = i % NB, t = i / NB % 16, is_v = i / (16 * NB) & 1, h = i / ITEMS;
      if (t < t0 || t >= t1) continue;
      const int at = is_v ? kv4_v_scale<D>(t, blk) : kv4_k_scale<D>(t, blk);
      (g + (h0 + h) * head)[at] = scales[h * 2 * D + at - 16 * D];
    }
  }
}

template <bool READ>
cudaError_t launch_rows(const Kv4Args &a, uint16_t *k, long long ks, uint16_t *v, long long vs, cudaStream_t stream) {
  if (a.T == 0 || a.B == 0) return cudaSuccess;
  // groups that n new rows touch: at most n, and (n + 30) / 16
  const long long groups = min((long long)a.T, (long long)a.T / 16 + 2LL * a.B);
  RowsArgs p{a, k, v, ks, vs, min(a.Hkv, kHeads)};
  while (p.heads > 1 && groups * ((a.Hkv + p.heads - 1) / p.heads) < 2 * 152) p.heads = (p.heads + 1) / 2;  // fill the SMs
  const dim3 grid((unsigned)groups, (unsigned)((a.Hkv + p.heads - 1) / p.heads));
  if (a.D == 128)
    kv4_rows_kernel<128, READ><<<grid, 256, 0, stream>>>(p);
  else
    kv4_rows_kernel<64, READ><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- pages
constexpr int kCopyChunk = 16384;  // bytes of one page and layer that one CTA moves: 4 x 16 bytes a thread

// n_dev (compaction): the number of copies comes from the plan, and the tables
// are rewritten by its map beside the copies.
__global__ void __launch_bounds__(256) copy_pages_kernel(Kv4PageArgs a, const int32_t *n_dev) {
  int n = a.n;
  if (n_dev) {
    pdl_wait();  // the plan is made
    n = *n_dev;
    const long long entries = (long long)a.rows * a.cols;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < entries; i += gridDim.x * 256LL) {
      const int p = a.table[i];
      a.tables_out[i] = p >= 0 && p < a.num_pages ? a.page_map[p] : -1;
    }
  }
  const int chunks = (int)((a.page_bytes + kCopyChunk - 1) / kCopyChunk);
  const long long total = (long long)n * a.layers * chunks;
  for (long long i = blockIdx.x; i < total; i += gridDim.x) {
    const int c = (int)(i % chunks);
    const long long j = i / chunks;
    const int l = (int)(j % a.layers), m = (int)(j / a.layers);
    const int s = a.src[m], d = a.dst[m];
    if (s < 0 || s >= a.num_pages || d < 0 || d >= a.num_pages) {
      if (threadIdx.x == 0) flag_status(a.status, GDN_E_RANGE);
      continue;
    }
    uint8_t *base = a.pages + l * a.layer_stride;
    const long long at = (long long)c * kCopyChunk;
    const uint4 *from = reinterpret_cast<const uint4 *>(base + s * a.page_bytes + at);
    uint4 *to = reinterpret_cast<uint4 *>(base + d * a.page_bytes + at);
    const int words = (int)(min((long long)kCopyChunk, a.page_bytes - at) / 16);
    uint4 x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int w = threadIdx.x + q * 256;
      if (w < words) x[q] = from[w];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int w = threadIdx.x + q * 256;
      if (w < words) to[w] = x[q];
    }
  }
}

// ---------------------------------------------------------------- compaction
// Workspace: [0] the number of moves, then the moved pages and their places.
struct CompactWs {
  int32_t *n_moves, *src, *dst;
};
CompactWs compact_ws(void *p, int num_pages) {
  int32_t *w = static_cast<int32_t *>(p);
  return {w, w + 4, w + 4 + (num_pages + 3) / 4 * 4};
}

// One CTA: a bitmap of the live pages in shared memory, its prefix counts, and
// from them every page's new id, a thread per page. With before(p) the live pages
// below p: a hole p < L is the (p - before(p))-th, a live p >= L the
// (before(p) - before(L))-th to move.
__global__ void __launch_bounds__(1024) compact_plan_kernel(Kv4PageArgs a, CompactWs w) {
  extern __shared__ uint32_t bits[];
  __shared__ int sums[32], prefix[1024], live_total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  const int words = (a.num_pages + 31) / 32;
  for (int i = tid; i < words; i += 1024) bits[i] = 0;
  __syncthreads();
  const long long entries = (long long)a.rows * a.cols;
  for (long long i = tid; i < entries; i += 4 * 1024) {
    int p[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) p[u] = i + u * 1024 < entries ? a.table[i + u * 1024] : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (p[u] >= a.num_pages) flag_status(a.status, GDN_E_RANGE);
      else if (p[u] >= 0) atomicOr(&bits[p[u] >> 5], 1u << (p[u] & 31));
    }
  }
  __syncthreads();
  // live pages before each thread's words
  const int per = (words + 1023) / 1024, w0 = min(tid * per, words), w1 = min(w0 + per, words);
  int mine = 0;
  for (int i = w0; i < w1; ++i) mine += __popc(bits[i]);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int x = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    sums[lane] = x;
    if (lane == 31) live_total = x;
  }
  __syncthreads();
  prefix[tid] = incl - mine + (warp ? sums[warp - 1] : 0);
  __syncthreads();
  const int L = live_total;
  auto before = [&](int p) {
    const int word = p >> 5;
    int t = word / per, n = prefix[t];
    for (int i = t * per; i < word; ++i) n += __popc(bits[i]);
    return n + __popc(bits[word] & ((1u << (p & 31)) - 1u));
  };
  const int bl = L < a.num_pages ? before(L) : L;
  for (int p = tid; p < a.num_pages; p += 1024) {
    const bool live = bits[p >> 5] >> (p & 31) & 1u;
    if (!live && p < L) w.dst[p - before(p)] = p;
    if (live && p >= L) w.src[before(p) - bl] = p;
  }
  if (tid == 0) {
    *w.n_moves = L - bl;
    *a.n_live = L;
  }
  __syncthreads();  // the lists are complete, and visible within this CTA
  for (int p = tid; p < a.num_pages; p += 1024) {
    const bool live = bits[p >> 5] >> (p & 31) & 1u;
    a.page_map[p] = !live ? -1 : p < L ? p : w.dst[before(p) - bl];
  }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Args &a, const uint16_t *k, long long k_stride, const uint16_t *v,
                              long long v_stride, cudaStream_t stream) {
  return launch_rows<false>(a, const_cast<uint16_t *>(k), k_stride, const_cast<uint16_t *>(v), v_stride, stream);
}
cudaError_t launch_kv4_read(const Kv4Args &a, uint16_t *k, uint16_t *v, cudaStream_t stream) {
  const long long stride = (long long)a.Hkv * a.D;
  return launch_rows<true>(a, k, stride, v, stride, stream);
}

cudaError_t launch_kv4_copy_pages(const Kv4PageArgs &a, cudaStream_t stream) {
  const long long total = (long long)a.n * a.layers * ((a.page_bytes + kCopyChunk - 1) / kCopyChunk);
  if (total == 0) return cudaSuccess;
  copy_pages_kernel<<<(unsigned)min(total, 152LL * 8), 256, 0, stream>>>(a, nullptr);
  return cudaGetLastError();
}

size_t kv4_compact_bytes(int num_pages) { return sizeof(int32_t) * (4 + 2 * (size_t)((num_pages + 3) / 4 * 4)); }

cudaError_t launch_kv4_compact(const Kv4PageArgs &a, cudaStream_t stream) {
  const CompactWs w = compact_ws(a.workspace, a.num_pages);
  const size_t smem = (size_t)(a.num_pages + 31) / 32 * 4;
  static bool allowed[64];
  cudaError_t e = kv4_allow_smem(compact_plan_kernel, 128 * 1024, allowed);
  if (e != cudaSuccess) return e;
  compact_plan_kernel<<<1, 1024, smem, stream>>>(a, w);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  Kv4PageArgs c = a;
  c.src = w.src;
  c.dst = w.dst;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(152 * 8, 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, copy_pages_kernel, c, (const int32_t *)w.n_moves);
}

}  // namespace gdn
