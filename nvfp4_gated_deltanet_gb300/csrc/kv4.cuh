// The paged 4-bit KV cache: its layout and the kernels' arguments.
#pragma once
#include "common.cuh"

namespace gdn {

constexpr int kKv4Group = 16;  // tokens of one head that lie together

// Where a group (16 tokens of one head, 18 d bytes) keeps token t. V's row
// order and swapped halves let lane (g, tq) of a warp MMA read 8 (d = 64: 4)
// code bytes of each of its four tokens 2tq, 2tq + 1, 2tq + 8, 2tq + 9 with the
// 32 lanes on 32 different banks, and their scales of one block as one word.
GDN_DEV int kv4_v_row(int t) { return (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3); }
template <int D>
GDN_DEV int kv4_k_code(int t, int i) { return t * (D / 2) + i; }  // i: byte of the row
template <int D>
GDN_DEV int kv4_v_code(int t, int i) {
  const int r = kv4_v_row(t);
  return 8 * D + r * (D / 2) + (D == 128 ? i ^ (((r >> 1) & 1) << 5) : i);
}
template <int D>
GDN_DEV int kv4_k_scale(int t, int b) { return 16 * D + t * (D / 16) + b; }
template <int D>
GDN_DEV int kv4_v_scale(int t, int b) { return 17 * D + b * 16 + ((t >> 1) & 3) * 4 + ((t & 1) | ((t >> 3) << 1)); }

struct Kv4Args {
  uint8_t *pages;
  int num_pages, page_tokens, Hkv, D;
  float ks, vs;
  const int32_t *kv_len, *table, *q_start;  // q_start null: T / B rows each
  int B, cols, T;
  int32_t *status;
  long long wait;  // budget of a wait on copies, SM cycles
  int zero_padding;  // kv4_batch::zero_padding; 0 without q_start
};
// The first padding row that is to be written (T where none is): past every row
// start, so that a bad one takes no rows from the other sequences. A whole warp.
GDN_DEV int kv4_padding(const Kv4Args &a, int lane) {
  if (!a.zero_padding) return a.T;
  int last = 0;
  for (int i = lane; i <= a.B; i += 32) {
    const int q = a.q_start[i];
    if (q <= a.T) last = max(last, q);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
  return last;
}

// A sequence's new rows [q0, q1) and its token count, checked: a bad entry
// flags GDN_E_RANGE and reads as an empty sequence.
struct Kv4Seq {
  int q0, q1, len;
};
GDN_DEV Kv4Seq kv4_seq(const Kv4Args &a, int b) {
  Kv4Seq s;
  if (a.q_start) {
    s.q0 = a.q_start[b];
    s.q1 = a.q_start[b + 1];
  } else {
    const int r = a.T / a.B;
    s.q0 = b * r;
    s.q1 = s.q0 + r;
  }
  s.len = a.kv_len[b];
  const bool bad_q = s.q0 < 0 || s.q1 < s.q0 || s.q1 > a.T;
  const bool bad_len = s.len < 0 || s.len > (long long)a.cols * a.page_tokens;
  if (bad_q || bad_len) flag_status(a.status, GDN_E_RANGE);
  if (bad_q) s.q0 = s.q1 = 0;
  if (bad_len) s.len = 0;
  return s;
}
// Sequence b's tokens, checked (kv4_seq without rows and without the flag).
GDN_DEV int kv4_len(const Kv4Args &a, int b) {
  const int n = a.kv_len[b];
  return n < 0 || n > (long long)a.cols * a.page_tokens ? 0 : n;
}
// The group that holds token `pos` of sequence b (head 0), or null for a bad page id.
template <int D>
GDN_DEV uint8_t *kv4_group(const Kv4Args &a, int b, int pos) {
  const int page = a.table[(size_t)b * a.cols + pos / a.page_tokens];
  if (page < 0 || page >= a.num_pages) {
    flag_status(a.status, GDN_E_RANGE);
    return nullptr;
  }
  return a.pages + ((size_t)page * a.Hkv * (a.page_tokens / 16) + (pos % a.page_tokens) / 16) * (18 * D);
}
// Bytes from one head's group to the next head's.
template <int D>
GDN_DEV size_t kv4_head_bytes(const Kv4Args &a) { return (size_t)(a.page_tokens / 16) * (18 * D); }

// ---------------------------------------------------------------- arithmetic of the attention kernels
GDN_DEV uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
// Eight E2M1 codes times a pair of scales
GDN_DEV void decode8(uint32_t w, __half2 s, uint32_t (&o)[4]) {
  __half2 h[4];
  e2m1x8_to_h2x4(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = h2u(__hmul2(h[i], s));
}

// Two floats rounded to BF16, the first in the low half
GDN_DEV uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// 2^x, to two units in the last place; 2^-inf = 0
GDN_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (x.lo, x.hi) * s + o
GDN_DEV float2 fma2(float2 x, float2 s, float2 o) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<unsigned long long *>(&r))
      : "l"(*reinterpret_cast<unsigned long long *>(&x)), "l"(*reinterpret_cast<unsigned long long *>(&s)),
        "l"(*reinterpret_cast<unsigned long long *>(&o)));
  return r;
}
GDN_DEV float2 add2(float2 x, float2 y) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long *>(&r))
      : "l"(*reinterpret_cast<unsigned long long *>(&x)), "l"(*reinterpret_cast<unsigned long long *>(&y)));
  return r;
}

// Let a kernel (one flag array each) have `bytes` of dynamic shared memory, once per device.
template <typename K>
cudaError_t kv4_allow_smem(K kernel, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

// Every kernel of the cache is launched so that it may begin while the one before
// it in the stream ends, and calls kv4_begin before it touches global memory: what
// earlier kernels wrote is there then, and only then may the next one begin. (The
// second kernel of a call reads the lengths, tables and queries before: its first
// has waited for them.) Call after call, 16 tokens appended and read take 6.6 us
// instead of 10.3, one decode of 131 tokens 5.5 instead of 8.2.
GDN_DEV void kv4_begin() {
  pdl_wait();
  pdl_launch_dependents();
}
template <typename... P, typename... A>
cudaError_t kv4_launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

cudaError_t launch_kv4_append(const Kv4Args &a, const uint16_t *k, long long k_stride, const uint16_t *v,
                              long long v_stride, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4Args &a, uint16_t *k, uint16_t *v, cudaStream_t stream);

struct Kv4AttnArgs {
  Kv4Args c;
  const uint16_t *q;
  long long q_stride;
  int Hq;
  float sm_scale;
  uint16_t *out;
  float *lse;  // or null
};
cudaError_t launch_kv4_decode(const Kv4AttnArgs &a, void *workspace, int num_sms, cudaStream_t stream);
size_t kv4_decode_bytes(const Kv4AttnArgs &a, int num_sms);  // its workspace
cudaError_t launch_kv4_prefill(const Kv4AttnArgs &a, long long total_kv, void *workspace, int num_sms,
                               cudaStream_t stream);
size_t kv4_prefill_bytes(const Kv4AttnArgs &a, long long total_kv);  // its workspace; 0: too large

struct Kv4PageArgs {
  uint8_t *pages;
  int layers, num_pages;
  long long layer_stride, page_bytes;
  const int32_t *src, *dst;
  int n;
  // compaction
  const int32_t *table;
  int rows, cols;
  int32_t *tables_out, *page_map, *n_live;
  void *workspace;
  int32_t *status;
};
cudaError_t launch_kv4_copy_pages(const Kv4PageArgs &a, cudaStream_t stream);
cudaError_t launch_kv4_compact(const Kv4PageArgs &a, cudaStream_t stream);
size_t kv4_compact_bytes(int num_pages);

}  // namespace gdn
