// wq_kv4_cache.cu -- the 4-bit key/value cache's writer and reader.
//
// Append: a new token's query and key heads are rotated by position, its key
// and value heads rounded to symmetric INT4 codes with one bf16 scale per
// group of dimensions, and written into the token's slot of its page.
//
//   pair (a, b) -> (a c - b s, a s + b c)
//   x = the exact rotated value rounded once to fp32
//   s = bf16(fp32(max|x| / 7)) (1 where that is 0),  q = clamp(rint(fp32(x / s)), -8, 7)
//
// the last line as wq_pack_symmetric rounds a weight.  The products of a bf16
// value and an fp32 cosine need 32 bits, so the key's two products and their
// sum carry an error term (two_prod / two_sum) and x is the correctly rounded
// sum: a code next to a rounding border does not depend on how the products
// were associated.  Queries are rounded to bf16 and take plain fp32.
//
// A CTA takes up to kMaxTokens consecutive tokens; where they go (sequence,
// slot, page) is looked up once for all of them while the first rows are in
// flight.  A row (head) takes D/8 lanes of 8 dimensions (16 bytes) each, a
// half-split rotation's partner dimensions come by shuffle, and one thread
// keeps its cosines for all the heads of a token that it walks.  Value words
// gather dimensions 8 apart, an 8 x 8 transpose of nibbles over 8 lanes
// (three shuffles).  Bound: bytes -- per token 2 D (Hq + 2 Hkv) read, 2 D Hq and the
// cache's D + 4 D/group per key/value head written.
//
// Measured (32 query and 8 key/value heads of 128): 8192 tokens: 63 us, 2.8 TB/s;
// 40 of them keys and values, about 500 instructions for two rows of 128 (the exact
// rotation, the codes, their transposition): 64% of the issue slots are taken while
// 41% of an SM's warps are resident, and a token's lookup and loads are waited for in
// the rest.  (Interleaved pairs 55 us; heads of 64: 43, of 256: 100.)  One token 5.1 us:
// a launch, the sequence's lookup and one row.  Reading back: 8192 tokens 16 us, 2.6
// TB/s (heads of 64: 12, of 256: 31), one 3.1 us.
#include "wq_device.cuh"
#include "wq_kv4.cuh"

namespace wq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;

// Nibble transpose over 8 lanes: lane i's nibble g becomes lane g's nibble i.
__device__ __forceinline__ uint32_t transpose_nibbles8(uint32_t x, int lane) {
  uint32_t y = __shfl_xor_sync(0xffffffffu, x, 4);
  x = (lane & 4) ? (x & 0xFFFF0000u) | (y >> 16) : (x & 0x0000FFFFu) | (y << 16);
  y = __shfl_xor_sync(0xffffffffu, x, 2);
  x = (lane & 2) ? (x & 0xFF00FF00u) | ((y >> 8) & 0x00FF00FFu) : (x & 0x00FF00FFu) | ((y & 0x00FF00FFu) << 8);
  y = __shfl_xor_sync(0xffffffffu, x, 1);
  x = (lane & 1) ? (x & 0xF0F0F0F0u) | ((y >> 4) & 0x0F0F0F0Fu) : (x & 0x0F0F0F0Fu) | ((y & 0x0F0F0F0Fu) << 4);
  return x;
}

// u v + w z rounded once to fp32 (up to a final double rounding of 2^-48):
// both products and the sum with their exact errors.
__device__ __forceinline__ float dot2_exact(float u, float v, float w, float z) {
  const float p = __fmul_rn(u, v), pe = __fmaf_rn(u, v, -p);
  const float q = __fmul_rn(w, z), qe = __fmaf_rn(w, z, -q);
  const float s = __fadd_rn(p, q), t = __fsub_rn(s, p);
  const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(s, t)), __fsub_rn(q, t));
  return __fadd_rn(s, __fadd_rn(e, __fadd_rn(pe, qe)));
}

// The same to fp32 accuracy, for the queries.
__device__ __forceinline__ float dot2_fast(float u, float v, float w, float z) {
  return __fmaf_rn(u, v, __fmul_rn(w, z));
}

// The 4-bit grid as defined, with IEEE divisions: the scale of a group whose
// largest |x| has the bits `top`, and a value's code in offset binary.
// (Out of line and by value, so that the eight stay in registers; one code a
// call.)
__device__ __noinline__ float scale_exact(uint32_t top) {
  const float scale = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 7.0f)));
  return scale == 0.f ? 1.f : scale;
}
__device__ __noinline__ uint32_t code_exact(float x, float scale) {
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(x, scale)), -8.f), 7.f)) + 8);
}
// The nibbles of a key word from those in order: even ones low, odd ones high.
__device__ __forceinline__ uint32_t key_word(uint32_t w) {
  uint32_t t = (w ^ (w >> 4)) & 0x00F000F0u;  // nibbles 0 2 1 3, 4 6 5 7
  w ^= t ^ (t << 4);
  return __byte_perm(w, 0, 0x3120);           // bytes 0 2, then 1 3
}
// Eight values' scale, and their codes as nibbles in order, without a
// division; false (for the whole warp) where a value
// lies so near a border between two codes, or the group so far from 1, that
// only the division decides.  max / 7 is the correctly rounded quotient
// (kv4_seventh); x times a reciprocal is off by 2^-21 of at most 7.03, so a code is
// sure unless the product comes within 1e-5 of a half.
__device__ __forceinline__ bool grid_fast(const float (&x)[8], uint32_t top, float& scale, uint32_t& word) {
  const float t = __uint_as_float(top);
  scale = t == 0.f ? 1.f : __bfloat162float(__float2bfloat16_rn(kv4_seventh(t)));
  bool unsure = t != 0.f && !(t > 0x1p-100f && t < 0x1p100f);
  const float inv = __fdividef(1.f, scale);
  constexpr float kRound = 12582912.f;  // 1.5 2^23: adding it rounds to an integer, in the low bits
  uint32_t w = 0;
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = __fmul_rn(x[i], inv), r = __fadd_rn(q, kRound);
    far = fmaxf(far, fabsf(__fsub_rn(q, __fsub_rn(r, kRound))));
    w |= (__float_as_uint(r) << (4 * i)) & (15u << (4 * i));
  }
  word = w ^ 0x88888888u;  // two's complement to offset binary
  unsure |= far > 0.49999f;
  return !__any_sync(0xffffffffu, unsure);
}

// Where a token of the batch goes.
struct Slot {
  int64_t pos;    // slot index in its sequence
  int64_t block;  // byte offset of head 0's block; -1: none; -2: the token belongs to no sequence
  int in_page;    // slot in the page
};
// Slots of tokens tok0 .. tok0 + n - 1 (n <= kMaxTokens); every thread of the
// CTA takes part and may read `slots` afterwards.
__device__ __forceinline__ void find_slots(const Kv4Params& p, int64_t tok0, int n, int* seqs, Slot* slots) {
  if (threadIdx.x < kMaxTokens) seqs[threadIdx.x] = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int64_t c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1);
    if (blockIdx.x == 0) kv4_load_sequence(p, b);  // records what does not fit, also of a sequence without new tokens
    for (int i = 0; i < n; ++i)
      if (c0 <= tok0 + i && tok0 + i < c1) atomicMax(seqs + i, b);
  }
  __syncthreads();
  if (threadIdx.x < n) {
    Slot s;
    s.pos = -1;
    s.block = -2;
    s.in_page = 0;
    const int b = seqs[threadIdx.x];
    if (b >= 0) {
      // a token's slot follows from the entries as they are: clamped ones would
      // move it onto a slot that is another token's
      const Kv4Seq q = kv4_load_sequence(p, b);
      s.pos = __ldg(p.kv_len + b) - (__ldg(p.cu_q + b + 1) - (tok0 + threadIdx.x));
      s.block = -1;
      if (s.pos >= 0 && s.pos < q.len) {
        const int64_t page = __ldg(p.page_table + b * p.max_pages + (s.pos >> p.lay.page_shift));
        s.block = kv4_block_offset(page, p.num_pages, 0, p.Hkv, p.lay.block);
        s.in_page = static_cast<int>(s.pos & (p.lay.page() - 1));
      }
      if (s.block < 0) atomicMax(p.err, kErrBounds);
    }
    slots[threadIdx.x] = s;
  }
  __syncthreads();
}

struct AppendParams {
  Kv4Params kv;
  Rows Q, Qo, K, V;
  int Hq;
  const float* rope;
  const int32_t* positions;
  int64_t max_pos;
  int rot_dim, group, tokens;  // tokens of a CTA
};

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo_to_f32(w[i]);
    x[2 * i + 1] = bf16_hi_to_f32(w[i]);
  }
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;                // lanes of a row
  constexpr int kRowsCta = kThreads / kLanes;  // rows in flight
  __shared__ int s_seq[kMaxTokens];
  __shared__ Slot s_slot[kMaxTokens];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.kv.T - tok0));
  const int lane = threadIdx.x & 31;
  const int L = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  const int half = p.rot_dim >> 1;
  const bool rotated = 8 * L < p.rot_dim;
  const bool second = 8 * L >= half;  // half-split: the pairs' second elements
  const int partner = INTERLEAVED ? lane : second ? lane - half / 8 : lane + half / 8;

  // A thread's rows: query heads r0, r0 + kRowsCta, .., then of the key and
  // value heads, taken as one list, the same.
  const int kv_rows = 2 * p.kv.Hkv;
  const __nv_bfloat16* q_src = static_cast<const __nv_bfloat16*>(p.Q.data) + tok0 * p.Q.token_stride + r0 * p.Q.head_stride + 8 * L;
  __nv_bfloat16* q_dst = static_cast<__nv_bfloat16*>(p.Qo.data) + tok0 * p.Qo.token_stride + r0 * p.Qo.head_stride + 8 * L;
  auto load_q = [&](int i, int step) -> uint4 {
    if (i >= n || r0 + step * kRowsCta >= p.Hq) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4*>(q_src + i * p.Q.token_stride + static_cast<int64_t>(step * kRowsCta) * p.Q.head_stride);
  };
  auto load_kv = [&](int i, int step) -> uint4 {
    const int r = r0 + step * kRowsCta;
    if (i >= n || r >= kv_rows) return make_uint4(0, 0, 0, 0);
    const bool v = r >= p.kv.Hkv;
    const Rows& m = v ? p.V : p.K;
    return *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(m.data) + (tok0 + i) * m.token_stride +
                                           (v ? r - p.kv.Hkv : r) * m.head_stride + 8 * L);
  };
  // in flight while the tokens' slots are looked up; later the next rows', and
  // the next token's, while one is worked on
  uint4 next_q = load_q(0, 0), next_kv = load_kv(0, 0);
  find_slots(p.kv, tok0, n, s_seq, s_slot);

  // the rotation of a lane's eight values; `other` holds the partners'
  float c[8], s[8];
  auto rotate = [&](float (&x)[8], const uint4& other, auto dot) {
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = dot(a, c[i], -b, s[i]);
        x[2 * i + 1] = dot(a, s[i], b, c[i]);
      }
    } else {
      float y[8];
      unpack_bf16x8(other, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = dot(x[i], c[i], y[i], s[i]);
    }
  };
  auto partners = [&](const uint4& raw) {  // lanes outside the rotation read a value they do not use
    uint4 other = raw;
    if (!INTERLEAVED && p.rot_dim > 0) {
      const int from = rotated ? partner : lane;
      other.x = __shfl_sync(0xffffffffu, raw.x, from);
      other.y = __shfl_sync(0xffffffffu, raw.y, from);
      other.z = __shfl_sync(0xffffffffu, raw.z, from);
      other.w = __shfl_sync(0xffffffffu, raw.w, from);
    }
    return other;
  };
  const int q_steps = (p.Hq + kRowsCta - 1) / kRowsCta, kv_steps = (kv_rows + kRowsCta - 1) / kRowsCta;
  for (int i = 0; i < n; ++i) {
    const int64_t tok = tok0 + i;
    const Slot slot = s_slot[i];
    const int64_t turn = p.positions != nullptr ? __ldg(p.positions + tok) : slot.pos;
    const bool turns = p.rot_dim == 0 || (turn >= 0 && turn < p.max_pos);
    const bool ok = slot.block >= 0 && turns;
    if (slot.block >= 0 && !turns && threadIdx.x == 0) atomicMax(p.kv.err, kErrBounds);
    // this thread's cosines and sines: of the pairs from 8 L (half-split, by
    // the pair's index; a first element's sine is taken with a minus, since it
    // becomes a c - b s and the second b c + a s) or 4 L (interleaved)
    if (ok && rotated) {
      const float* t = p.rope + turn * p.rot_dim + (INTERLEAVED ? 8 * L : 2 * (second ? 8 * L - half : 8 * L));
#pragma unroll
      for (int q = 0; q < (INTERLEAVED ? 2 : 4); ++q) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(t) + q);
        c[2 * q] = v.x;
        s[2 * q] = INTERLEAVED || second ? v.y : -v.y;
        c[2 * q + 1] = v.z;
        s[2 * q + 1] = INTERLEAVED || second ? v.w : -v.w;
      }
    }
    const bool known = slot.block != -2;  // (uniform) some sequence's token
    for (int step = 0; step < q_steps; ++step) {
      const uint4 raw = next_q;
      next_q = step + 1 == q_steps ? load_q(i + 1, 0) : load_q(i, step + 1);
      if (!known) continue;
      const uint4 other = partners(raw);
      const int r = r0 + step * kRowsCta;
      if (r >= p.Hq) continue;
      uint4 o = raw;
      if (!ok) {
        o = make_uint4(0, 0, 0, 0);
      } else if (rotated) {
        float x[8];
        unpack_bf16x8(raw, x);
        rotate(x, other, [](float u, float v, float w, float z) { return dot2_fast(u, v, w, z); });
        o = make_uint4(pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]), pack_bf16x2_rn(x[4], x[5]), pack_bf16x2_rn(x[6], x[7]));
      }
      *reinterpret_cast<uint4*>(q_dst + i * p.Qo.token_stride + static_cast<int64_t>(step * kRowsCta) * p.Qo.head_stride) = o;
    }
    for (int step = 0; step < kv_steps; ++step) {
      const uint4 raw = next_kv;
      next_kv = step + 1 == kv_steps ? load_kv(i + 1, 0) : load_kv(i, step + 1);
      if (!known) continue;
      const int r = r0 + step * kRowsCta;
      const bool is_v = r >= p.kv.Hkv;
      const uint4 other = __all_sync(0xffffffffu, is_v) ? raw : partners(raw);
      float x[8];
      unpack_bf16x8(raw, x);
      if (ok && rotated && !is_v)
        rotate(x, other, [](float u, float v, float w, float z) { return dot2_exact(u, v, w, z); });
      // ---- the 4-bit grid: the bits of |x| order as integers, NaN and inf on top
      uint32_t top = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(x[q]) & 0x7FFFFFFFu);
      for (int o = 1; o < p.group / 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool finite = top < 0x7F800000u;
      float scale;
      uint32_t word;
      if (!grid_fast(x, top, scale, word)) {
        scale = scale_exact(top);
        word = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) word |= (finite ? code_exact(x[q], scale) : 8u) << (4 * q);
      }
      if (__any_sync(0xffffffffu, is_v)) {
        const uint32_t vw = transpose_nibbles8(word, lane);
        word = is_v ? vw : key_word(word);
      } else {
        word = key_word(word);
      }
      if (!ok || r >= kv_rows) continue;
      uint8_t* blk = p.kv.pool + slot.block + (is_v ? r - p.kv.Hkv : r) * p.kv.lay.block;
      const int at = is_v ? (L & 7) * (D / 64) + (L >> 3) : (L & 3) * (D / 32) + (L >> 2);
      uint8_t* row = blk + (is_v ? p.kv.lay.v_codes() : 0) + slot.in_page * (D / 2);
      reinterpret_cast<uint32_t*>(row)[at] = word;
      if (8 * L % p.group == 0) {
        uint16_t* sc = reinterpret_cast<uint16_t*>(blk + (is_v ? p.kv.lay.v_scales() : p.kv.lay.k_scales())) +
                       slot.in_page * p.kv.lay.G + 8 * L / p.group;
        *sc = finite ? static_cast<uint16_t>(__float_as_uint(scale) >> 16) : static_cast<uint16_t>(0x7FC0);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const Kv4Params p, const Rows K, const Rows V, const int tokens) {
  constexpr int kLanes = D / 8;
  constexpr int kRowsCta = kThreads / kLanes;
  __shared__ int s_seq[kMaxTokens];
  __shared__ Slot s_slot[kMaxTokens];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int n = static_cast<int>(min(static_cast<int64_t>(tokens), p.T - tok0));
  const int lane = threadIdx.x & 31;
  const int L = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  find_slots(p, tok0, n, s_seq, s_slot);
  const int groups_shift = 31 - __clz(D / p.lay.G);  // log2 of the group
  const int steps = (2 * p.Hkv + kRowsCta - 1) / kRowsCta;
#pragma unroll 2
  for (int it = 0; it < n * steps; ++it) {
    const int i = it / steps, r = it % steps * kRowsCta + r0;
    const int64_t tok = tok0 + i;
    const Slot slot = s_slot[i];
    if (slot.block == -2) continue;  // (uniform)
    const bool is_v = r >= p.Hkv;
    const int h = is_v ? r - p.Hkv : r;
    const Rows& m = is_v ? V : K;
    uint32_t w = 0x88888888u;
    float scale = 0.f;
    if (r < 2 * p.Hkv && slot.block >= 0) {
      const uint8_t* blk = p.pool + slot.block + h * p.lay.block;
      const int word = is_v ? (L & 7) * (D / 64) + (L >> 3) : (L & 3) * (D / 32) + (L >> 2);
      w = reinterpret_cast<const uint32_t*>(blk + (is_v ? p.lay.v_codes() : 0) + slot.in_page * (D / 2))[word];
      scale = __uint_as_float(
          static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(
              blk + (is_v ? p.lay.v_scales() : p.lay.k_scales()))[slot.in_page * p.lay.G + (8 * L >> groups_shift)])
          << 16);
    }
    const uint32_t vw = transpose_nibbles8(w, lane);
    if (r >= 2 * p.Hkv || m.data == nullptr) continue;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t n = is_v ? vw >> (4 * i) : w >> (4 * ((i >> 1) + 4 * (i & 1)));
      x[i] = scale * static_cast<float>(static_cast<int>(n & 15u) - 8);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(m.data) + tok * m.token_stride + h * m.head_stride + 8 * L) =
        make_uint4(pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]), pack_bf16x2_rn(x[4], x[5]),
                   pack_bf16x2_rn(x[6], x[7]));
  }
}

// Tokens of a CTA: one while that leaves no SM with more than six CTAs (a
// decoding step's latency), else as many as keep six, up to kMaxTokens.  (Appending
// 8192 tokens: 1, 2, 4, 8 of a CTA take 74, 66, 63, 63 us.)
int tokens_of_cta(int64_t T, int num_sms) {
  const int64_t n = (T + 6 * num_sms - 1) / (6 * num_sms);
  return static_cast<int>(n < kMaxTokens ? n : kMaxTokens);
}

template <typename Kernel, typename... Args>
cudaError_t launch_tokens(Kernel kernel, int64_t ctas, int pdl, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Args& a, const Kv4AppendArgs& x, cudaStream_t stream) {
  AppendParams p;
  p.kv = kv4_params(a);
  p.Q = x.Q;
  p.Qo = x.Q_out;
  p.K = x.K;
  p.V = x.V;
  p.Hq = x.Hq;
  p.rope = x.rope;
  p.positions = x.positions;
  p.max_pos = x.max_pos;
  p.rot_dim = x.rot_dim;
  p.group = a.group;
  p.tokens = tokens_of_cta(a.T, a.num_sms);
  auto go = [&](auto kernel) { return launch_tokens(kernel, (a.T + p.tokens - 1) / p.tokens, a.pdl, stream, p); };
  if (a.D == 64) return x.interleaved ? go(kv4_append_kernel<64, true>) : go(kv4_append_kernel<64, false>);
  if (a.D == 128) return x.interleaved ? go(kv4_append_kernel<128, true>) : go(kv4_append_kernel<128, false>);
  return x.interleaved ? go(kv4_append_kernel<256, true>) : go(kv4_append_kernel<256, false>);
}

cudaError_t launch_kv4_read(const Kv4Args& a, Rows K, Rows V, cudaStream_t stream) {
  const Kv4Params p = kv4_params(a);
  const int n = tokens_of_cta(a.T, a.num_sms);
  auto go = [&](auto kernel) { return launch_tokens(kernel, (a.T + n - 1) / n, a.pdl, stream, p, K, V, n); };
  return a.D == 64 ? go(kv4_read_kernel<64>) : a.D == 128 ? go(kv4_read_kernel<128>) : go(kv4_read_kernel<256>);
}

}  // namespace wq
