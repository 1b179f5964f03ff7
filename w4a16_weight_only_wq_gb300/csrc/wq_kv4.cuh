// wq_kv4.cuh -- layout and bounds of the 4-bit key/value cache, shared by the
// kernels that write and read it and (as plain host arithmetic) by the C ABI's
// wq_kv4_locate and wq_debug_kv4_sequence.  The layout is documented in
// include/wq.h.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>

#include "wq_internal.h"

namespace wq {

constexpr uint32_t kErrBounds = 7;  // mirrors WQ_ERR_DEVICE_BOUNDS

// Sizes of a cache's blocks: one head's slots of one page.
struct Kv4Layout {
  int page_shift;      // log2 of the page size
  int D, G;            // head dimension, scales per row
  int code_row;        // bytes of a row of codes, D / 2
  int64_t block;       // bytes of a block
  __host__ __device__ int page() const { return 1 << page_shift; }
  __host__ __device__ int64_t v_codes() const { return static_cast<int64_t>(code_row) << page_shift; }
  __host__ __device__ int64_t k_scales() const { return 2 * v_codes(); }
  __host__ __device__ int64_t v_scales() const { return k_scales() + (static_cast<int64_t>(2 * G) << page_shift); }
};

__host__ __device__ inline Kv4Layout kv4_layout(int page_size, int D, int group) {
  Kv4Layout l;
  l.page_shift = 0;
  while ((1 << l.page_shift) < page_size) ++l.page_shift;
  l.D = D;
  l.G = D / group;
  l.code_row = D / 2;
  l.block = (static_cast<int64_t>(D) + 4 * l.G) << l.page_shift;
  return l;
}

// Byte offset of a block, or -1 for a page or head outside the pool.
__host__ __device__ inline int64_t kv4_block_offset(int64_t page, int64_t num_pages, int head, int Hkv,
                                                    int64_t block) {
  if (page < 0 || page >= num_pages || head < 0 || head >= Hkv) return -1;
  return (page * Hkv + head) * block;
}

// Word and nibble of a dimension in a row of key codes / of value codes.
__host__ __device__ inline void kv4_key_nibble(int D, int dim, int* word, int* nibble) {
  const int w = dim >> 5, t = (dim >> 3) & 3, r = dim & 7;
  *word = t * (D >> 5) + w;
  *nibble = (r >> 1) + 4 * (r & 1);
}
__host__ __device__ inline void kv4_value_nibble(int D, int dim, int* word, int* nibble) {
  *word = (dim & 7) * (D >> 6) + (dim >> 6);
  *nibble = (dim >> 3) & 7;
}

// t / 7 without a division: a product with 1/7 and one correction by the
// remainder, which is exact.  For t from 2^-100 to 2^100 it is the quotient as
// IEEE division rounds it (the tests compare every mantissa).
__host__ __device__ inline float kv4_seventh(float t) {
#ifdef __CUDA_ARCH__
  const float q = __fmul_rn(t, 1.f / 7.f);
#else
  const float q = t * (1.f / 7.f);
#endif
  return fmaf(fmaf(-q, 7.f, t), 1.f / 7.f, q);
}

// One sequence's entries, clamped to what the call's buffers hold.
struct Kv4Seq {
  int64_t first, n, len;  // first new token, new tokens, cached tokens
  bool bad;               // something lay outside
};
__host__ __device__ inline Kv4Seq kv4_sequence(int64_t cu0, int64_t cu1, int64_t len, int64_t T,
                                               int64_t capacity) {
  Kv4Seq s;
  const int64_t c0 = cu0 < 0 ? 0 : cu0 > T ? T : cu0;
  const int64_t c1 = cu1 < c0 ? c0 : cu1 > T ? T : cu1;
  const int64_t l = len < 0 ? 0 : len > capacity ? capacity : len;
  s.first = c0;
  s.n = c1 - c0;
  s.len = l;
  s.bad = c0 != cu0 || c1 != cu1 || l != len;
  return s;
}

// A cache and a step's batch as the kernels take them.
struct Kv4Params {
  uint8_t* pool;
  const int32_t* page_table;
  const int32_t* cu_q;
  const int32_t* kv_len;
  int64_t num_pages, max_pages, T;
  int B, Hkv;
  Kv4Layout lay;
  uint32_t* err;
};
inline Kv4Params kv4_params(const Kv4Args& a) {
  Kv4Params p;
  p.pool = static_cast<uint8_t*>(a.pool);
  p.page_table = a.page_table;
  p.cu_q = a.cu_q;
  p.kv_len = a.kv_len;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.T = a.T;
  p.B = static_cast<int>(a.B);
  p.Hkv = a.Hkv;
  p.lay = kv4_layout(a.page_size, a.D, a.group);
  p.err = a.diag.err;
  return p;
}

// Token slots of one sequence's row of the page table.  Positions fit 31 bits.
__host__ __device__ inline int64_t kv4_capacity(int64_t max_pages, int page_shift) {
  const int64_t n = max_pages << page_shift;
  return n < (int64_t(1) << 30) ? n : int64_t(1) << 30;
}

#ifdef __CUDACC__
__device__ __forceinline__ Kv4Seq kv4_load_sequence(const Kv4Params& p, int b) {
  Kv4Seq s = kv4_sequence(__ldg(p.cu_q + b), __ldg(p.cu_q + b + 1), __ldg(p.kv_len + b), p.T,
                          kv4_capacity(p.max_pages, p.lay.page_shift));
  if (s.bad) atomicMax(p.err, kErrBounds);
  return s;
}
#endif

}  // namespace wq
