// The 4-bit KV cache's data movement: new tokens into pages, tokens read back,
// pages copied and compacted.
#include "kv4.cuh"

namespace gdn {

namespace {

// One thread per 16-element block of K or of V: 32 bytes in, 8 code bytes and
// one scale byte out.
template <int D, bool READ>
__global__ void __launch_bounds__(256) kv4_rows_kernel(Kv4Args a, uint16_t *k, long long k_stride, uint16_t *v,
                                                       long long v_stride) {
  constexpr int NB = D / 16;
  const long long total = (long long)a.T * a.Hkv * NB * 2;
  const float invk = inv6ts_of(a.ks), invv = inv6ts_of(a.vs);
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
    const int blk = (int)(i % NB);
    const long long j = i / NB;
    const int h = (int)(j % a.Hkv);
    const long long n2 = j / a.Hkv;
    const bool is_v = n2 >= a.T;
    const int n = (int)(is_v ? n2 - a.T : n2);
    const int b = kv4_seq_of(a, n);
    if (b < 0) continue;
    const Kv4Seq s = kv4_seq(a, b);
    const int pos = s.len - (s.q1 - s.q0) + (n - s.q0);
    if (n < s.q0 || n >= s.q1 || pos < 0) continue;
    uint8_t *g = kv4_group<D>(a, b, pos);
    if (!g) continue;
    g += h * kv4_head_bytes<D>(a);
    const int t = pos & 15;
    uint2 *codes = reinterpret_cast<uint2 *>(g + (is_v ? kv4_v_code<D>(t, blk * 8) : kv4_k_code<D>(t, blk * 8)));
    uint8_t *scale = g + (is_v ? kv4_v_scale<D>(t, blk) : kv4_k_scale<D>(t, blk));
    uint16_t *row = is_v ? v + n * v_stride : k + n * k_stride;
    row += h * D + blk * 16;
    const float ts = is_v ? a.vs : a.ks;
    if (READ) {
      const uint2 w = *codes;
      const float sc = e4m3_to_f32(*scale);
      __half2 e[8];
      e2m1x8_to_h2x4(w.x, *reinterpret_cast<__half2(*)[4]>(&e[0]));
      e2m1x8_to_h2x4(w.y, *reinterpret_cast<__half2(*)[4]>(&e[4]));
      uint32_t o[8];
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const float2 f = __half22float2(e[m]);  // e2m1 x e4m3 is exact; one FP32 rounding by ts, one to BF16
        o[m] = f32_to_bf16_bits(f.x * sc * ts) | (uint32_t)f32_to_bf16_bits(f.y * sc * ts) << 16;
      }
      reinterpret_cast<uint4 *>(row)[0] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4 *>(row)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
      float x[16];
      load_bf16x16(row, x);
      uint32_t lo, hi, sc;
      if (!quant_block16(x, ts, is_v ? invv : invk, lo, hi, sc)) flag_status(a.status, GDN_E_NONFINITE);
      *codes = make_uint2(lo, hi);
      *scale = (uint8_t)sc;
    }
  }
}

template <bool READ>
cudaError_t launch_rows(const Kv4Args &a, uint16_t *k, long long ks, uint16_t *v, long long vs, cudaStream_t stream) {
  const long long total = (long long)a.T * a.Hkv * (a.D / 16) * 2;
  if (total == 0 || a.B == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)min((total + 255) / 256, 152LL * 16);
  if (a.D == 128)
    kv4_rows_kernel<128, READ><<<blocks, 256, 0, stream>>>(a, k, ks, v, vs);
  else
    kv4_rows_kernel<64, READ><<<blocks, 256, 0, stream>>>(a, k, ks, v, vs);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- pages
constexpr int kCopyChunk = 16384;  // bytes of one page and layer that one CTA moves: 4 x 16 bytes a thread

__global__ void __launch_bounds__(256) copy_pages_kernel(Kv4PageArgs a, const int32_t *n_dev) {
  const int n = n_dev ? *n_dev : a.n;
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
// from them every page's new id. With before(p) the live pages below p: a hole
// p < L is the (p - before(p))-th, a live p >= L the (before(p) - before(L))-th
// to move.
__global__ void __launch_bounds__(1024) compact_plan_kernel(Kv4PageArgs a, CompactWs w) {
  extern __shared__ uint32_t bits[];
  __shared__ int sums[32], live_total, before_l;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = (a.num_pages + 31) / 32;
  for (int i = tid; i < words; i += 1024) bits[i] = 0;
  __syncthreads();
  const long long entries = (long long)a.rows * a.cols;
  for (long long i = tid; i < entries; i += 1024) {
    const int p = a.table[i];
    if (p >= a.num_pages) flag_status(a.status, GDN_E_RANGE);
    else if (p >= 0) atomicOr(&bits[p >> 5], 1u << (p & 31));
  }
  __syncthreads();
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
  const int first = incl - mine + (warp ? sums[warp - 1] : 0);  // live pages below word w0
  const int L = live_total;
  if (L == a.num_pages) {
    if (tid == 0) before_l = L;
  } else if ((L >> 5) >= w0 && (L >> 5) < w1) {
    int n = first;
    for (int i = w0; i < (L >> 5); ++i) n += __popc(bits[i]);
    before_l = n + __popc(bits[L >> 5] & ((1u << (L & 31)) - 1u));
  }
  __syncthreads();
  const int bl = before_l;
  int before = first;
  for (int i = w0; i < w1; ++i) {
    const uint32_t m = bits[i];
    for (int j = 0; j < 32; ++j) {
      const int p = i * 32 + j;
      if (p >= a.num_pages) break;
      const bool live = (m >> j) & 1u;
      if (!live && p < L) w.dst[p - before] = p;
      if (live && p >= L) w.src[before - bl] = p;
      before += live;
    }
  }
  if (tid == 0) {
    *w.n_moves = L - bl;
    *a.n_live = L;
  }
  __syncthreads();  // the lists are complete, and visible within this CTA
  before = first;
  for (int i = w0; i < w1; ++i) {
    const uint32_t m = bits[i];
    for (int j = 0; j < 32; ++j) {
      const int p = i * 32 + j;
      if (p >= a.num_pages) break;
      const bool live = (m >> j) & 1u;
      a.page_map[p] = !live ? -1 : p < L ? p : w.dst[before - bl];
      before += live;
    }
  }
}

__global__ void __launch_bounds__(256) remap_tables_kernel(Kv4PageArgs a) {
  const long long entries = (long long)a.rows * a.cols;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < entries; i += gridDim.x * 256LL) {
    const int p = a.table[i];
    a.tables_out[i] = p >= 0 && p < a.num_pages ? a.page_map[p] : -1;
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
  Kv4PageArgs c = a;
  c.src = w.src;
  c.dst = w.dst;
  copy_pages_kernel<<<152 * 8, 256, 0, stream>>>(c, w.n_moves);
  const long long entries = (long long)a.rows * a.cols;
  if (entries) remap_tables_kernel<<<(unsigned)min((entries + 255) / 256, 1024LL), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
