// wq_logprobs.cu -- log probabilities of given tokens, with each row's
// entropy, the token's rank and the k largest logits, in one pass over them.
//
//   y_j = t x_j,  m = max y,  S = sum exp(y_j - m),  W = sum exp(y_j - m) (y_j - m)
//   logprob = y_tok - m - log S,   entropy = log S - W / S
//
// Bound: the logits' bytes, read once.  At 6.8 TB/s an SM receives 12 bf16
// logits a clock, 11 issue slots for each, so the inner loop is kept to the
// packed maximum of eight logits, and per logit one multiply-add, one clamp,
// one exponential and two accumulations; everything else hangs on the
// maximum of a thread's 32 logits of a tile and is rarely taken:
//  * a maximum far above the thread's reference moves it and rescales S and W;
//  * the rank counts logits only where the maximum passes the token's logit;
//  * a warp looks for alternatives only where it passes what is known to be
//    among the row's k best.
// (With a reference that followed each larger maximum of 8 logits, two steps of
// three took a branch, and 4096 x 248000 took 447 us at 82% of the issue slots.)
//
// Measured (bf16 but where said): 4096 x 248000, k = 1: 348 us, 5.8 TB/s, 84% of
// the issue slots (k = 0 307, 6.6 TB/s); 128 x 131071, k = 5: 23 us, 1.5 TB/s (k = 0 14: a launch, the
// first loads and the joins of three segments a row; the lists take the rest);
// 16 x 248000, k = 20: 16.5 us (k = 0 8.6); 1 x 32000 fp32, k = 0: 5.3 us; 2048 x 131071
// fp32: k = 0 166, 6.5 TB/s, k = 1 179, k = 5 211 (bf16 93, 114, 147).
//
// Alternatives: each warp keeps its k best in order, one a lane, as 64-bit
// keys (the logit's ordered bits, then the id's complement, so that equal
// logits go to the lowest id and the keys of a row are distinct); a candidate
// is placed with one vote and a shuffle.  A shared lower bound on the row's
// k-th best value discards the rest: at first the k-th largest of the 256
// threads' maxima over the CTA's first tiles (k threads hold a logit as large,
// and hardly more than k logits are), then the k-th best of the warps' lists,
// taken again after four rounds of tiles and whenever those have doubled, so
// that each doubling adds about k candidates to the CTA's.
//
// Few rows are split over CTAs (gridDim.x segments of a row); a segment's
// statistics and keys go to the workspace, and the last segment of a row to
// arrive joins them in segment order.
#include <cuda_bf16.h>

#include "wq_device.cuh"
#include "wq_internal.h"

namespace wq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxK = 32;
constexpr int kMaxSegments = 64;
constexpr int kPending = 256;                  // candidates of a warp on their way to its list
static_assert(kWarps * kPending <= kMaxSegments * kMaxK, "they share s_keys with the segments' keys");
constexpr int kVec = 8;                        // logits of one step of a thread
constexpr int kUnroll = 4;                     // steps in flight
constexpr int kTile = 32 * kVec * kUnroll;     // logits of a warp's tile
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// A segment's (warp's, thread's) statistics: the largest logit m, and with
// ref = max(m, low) c (c = t log2 e) the sums of e_j = 2^(c x_j - ref) and of
// e_j (c x_j - ref).  Logits at or below `low` = -1e38 / max(c, 1), where c x
// would leave fp32 (a mask of the type's lowest value, or -inf), count as
// `low`, which weighs nothing beside any other; a row with nothing above `low`
// gives each logit equal to its maximum the weight 1.
struct Partial {
  float m, s, w;
  int32_t rank;
};

struct Params {
  const void* logits;
  int64_t V, row_stride;
  const int64_t* tokens;
  const float* inv_temperature;
  int k;
  float* logprob;
  float* entropy;
  int32_t* rank;
  int32_t* top_ids;
  float* top_logprobs;
  uint32_t* arrived;    // [T]
  Partial* partials;    // [T][segments]
  uint64_t* keys;       // [T][segments][k]
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Bits of x that order as the values do; a NaN is above everything.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);  // -0 equals 0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o == 0xFFFFFFFFu ? 0x7FC00000u : (o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t make_key(float x, int64_t id) {
  return (static_cast<uint64_t>(ordered(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float*>(p);
  else return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16);
}

// A thread's running statistics and its warp's best keys.
struct State {
  float m, ref, limit, s, w;  // a logit above `limit` moves ref
  int rank;
  uint64_t mine;   // lane l: the warp's l-th best key (0: none yet)
  uint64_t kth;    // the k-th best (0 while there are fewer)
};

// Eight logits of a thread: their maximum (a NaN wins), and the values with
// everything below `low` raised to it (a NaN too).
template <typename T>
struct Loader;
template <>
struct Loader<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = ld_global_nc_v4(p);
    b = ld_global_nc_v4(p + 4);
  }
  __device__ __forceinline__ void none() { a = b = make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }  // -inf
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ float top() const {
    float x[8];
    get(x);
    return max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])), max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7])));
  }
  __device__ __forceinline__ void raised(float low, float (&x)[8]) const {
    get(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaxf(x[i], low);
  }
  __device__ __forceinline__ int above(float t) const {  // how many are greater than t, or a NaN
    float x[8];
    get(x);
    int n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) n += !(x[i] <= t);
    return n;
  }
};
template <>
struct Loader<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = ld_global_nc_v4(p); }
  __device__ __forceinline__ void none() { a = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }  // -inf
  __device__ __forceinline__ static void unpack(const uint32_t (&w)[4], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo_to_f32(w[i]);
      x[2 * i + 1] = bf16_hi_to_f32(w[i]);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    unpack(w, x);
  }
  __device__ __forceinline__ float top() const {  // two logits at a time
    const uint32_t m = bf16x2_max_nan(bf16x2_max_nan(a.x, a.y), bf16x2_max_nan(a.z, a.w));
    return max_nan(bf16_lo_to_f32(m), bf16_hi_to_f32(m));
  }
  __device__ __forceinline__ void raised(float low, float (&x)[8]) const {  // low is a bf16 number
    const uint32_t l = __float_as_uint(low) >> 16, ll = l | (l << 16);
    const uint32_t w[4] = {bf16x2_max(a.x, ll), bf16x2_max(a.y, ll), bf16x2_max(a.z, ll), bf16x2_max(a.w, ll)};
    unpack(w, x);
  }
  __device__ __forceinline__ int above(float t) const {  // t is a bf16 number
    const __nv_bfloat162 tt = __bfloat162bfloat162(__float2bfloat16_rn(t));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      bits |= __hgtu2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), tt) & (0x00010001u << i);
    return __popc(bits);
  }
};

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads)
token_logprobs_kernel(const Params p) {
  __shared__ float s_m[kWarps], s_s[kWarps], s_w[kWarps];
  __shared__ int s_rank[kWarps];
  __shared__ uint64_t s_keys[TOP ? kMaxSegments * kMaxK : 1];
  __shared__ __align__(16) uint32_t s_lane[TOP ? kThreads : 4];
  __shared__ uint32_t s_floor;  // ordered bits: a lower bound on the k-th best value
  __shared__ int s_last, s_count;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = gridDim.x, seg = blockIdx.x;
  const int64_t row = blockIdx.y;
  pdl_wait_primary();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  const float temp = p.inv_temperature != nullptr ? __ldg(p.inv_temperature + row) : 1.f;
  const float c = temp * kLog2e;
  const int64_t tok = __ldg(reinterpret_cast<const long long*>(p.tokens) + row);
  const bool has_tok = tok >= 0 && tok < p.V;
  const float xt = has_tok ? load1(x + tok) : INFINITY;  // (nothing ranks above)
  if (TOP && tid == 0) s_floor = 0;
  if (TOP) __syncthreads();

  // the segment's vectors of 8: the row from its first 16-byte aligned
  // element; the elements before and after belong to the first and last
  // segment
  const int64_t lead0 = ((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T);
  const int64_t lead = lead0 < p.V ? lead0 : p.V;
  const int nvec = static_cast<int>((p.V - lead) / kVec);
  const int tiles = (nvec + kTile / kVec - 1) / (kTile / kVec);
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * seg / S), t1 = static_cast<int>(static_cast<int64_t>(tiles) * (seg + 1) / S);

  // (the quotient cut to a bf16 number)
  const float low = __uint_as_float(__float_as_uint(-1e38f / fmaxf(c, 1.f)) & 0xFFFF0000u);
  State st;
  st.m = st.limit = -INFINITY;
  st.ref = low * c;
  const float margin = 8.f / c;
  st.s = st.w = 0.f;
  st.rank = 0;
  st.mine = st.kth = 0;
  const uint32_t k = static_cast<uint32_t>(p.k);

  // Candidates go through the warp's part of s_keys: lanes put theirs there,
  // then one loop places them in the list (one copy of its code).
  uint64_t* pend = s_keys + (TOP ? warp * kPending : 0);
  int pending = 0;
  auto offer = [&](float v, int64_t id, bool want) {
    const uint32_t bits = __ballot_sync(0xffffffffu, want);
    if (want) pend[pending + __popc(bits & ((1u << lane) - 1u))] = make_key(v, id);
    pending += __popc(bits);
  };
  auto place_pending = [&] {
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < pending; ++i) {
      const uint64_t cand = pend[i];
      if (cand <= st.kth) continue;  // (uniform)
      const int pos = __popc(__ballot_sync(0xffffffffu, st.mine > cand));
      const uint64_t up = __shfl_up_sync(0xffffffffu, st.mine, 1);
      if (lane == pos) st.mine = cand;
      else if (lane > pos) st.mine = up;
      st.kth = __shfl_sync(0xffffffffu, st.mine, k - 1);
    }
    pending = 0;
    __syncwarp();
  };
  // A tile's largest logit of a thread.  True: the tile's logits weigh (the
  // reference has moved if it had to: it stays 0 to 8, or 16, powers of two below
  // the maximum, so that few tiles move it, each a branch that 32 threads wait
  // for); false: none is above `low`, and those equal to the largest count.
  auto absorb = [&](float most) {
    if (fmaxf(most, st.m) <= low) {
      if (!(most <= st.m)) {
        st.s = st.w = 0.f;
        st.m = max_nan(st.m, most);
      }
      return false;
    }
    if (!(most <= st.limit)) {  // (or a NaN, which stays in m)
      const float ref = fmaxf(most, low) * c;
      const float d = most > low ? fmaxf(st.ref - ref, -1e30f) : -1e30f;
      const float f = exp2_approx(d);
      st.w = fmaf(st.s, d, st.w) * f;
      st.s *= f;
      st.ref = ref;
      st.limit = most + margin;
    }
    st.m = max_nan(st.m, most);
    return true;
  };
  // 8 logits of one thread, raised to `low`, into its sums of the tile (those are
  // added to the row's as wholes: beside a dominating logit, terms of 2^-24 of it
  // would be lost one by one)
  auto weigh = [&](const float (&v)[8], float& ts, float& tw) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = fmaf(v[i], c, -st.ref);
      const float e = exp2_approx(d);
      ts += e;
      tw = fmaf(e, d, tw);
    }
  };
  auto count = [&](const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) st.s += v[i] == st.m && v[i] != -INFINITY ? 1.f : 0.f;
  };

  // Raises the bound to the k-th largest of s_lane; the CTA has synchronised
  // after writing it.  One warp builds the value from its upper 16 bits down,
  // keeping a bit where k values reach it (two bits at a time took longer); the
  // lower bits (there are none in a bf16 logit's order) stay 0, still a bound.
  auto kth_of_lanes = [&] {
    if (warp == 0) {
      const uint4 u = *reinterpret_cast<const uint4*>(s_lane + 8 * lane), v = *reinterpret_cast<const uint4*>(s_lane + 8 * lane + 4);
      const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      uint32_t most = 0, least = 0xFFFFFFFFu, held = 0;  // of the lanes that hold a value
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        most = max(most, w[i]);
        least = min(least, w[i] - 1u);  // (0 becomes the largest)
        held += w[i] != 0;
      }
      most = __reduce_max_sync(0xffffffffu, most);
      least = __reduce_min_sync(0xffffffffu, least) + 1u;
      uint32_t t = 0;
      if (__reduce_add_sync(0xffffffffu, held) >= k) {
        // the bits that all values share are the k-th largest's too
        const int first = 31 - __clz(most ^ least);  // (-1: one value)
        t = first < 0 ? most : most & ~((2u << first) - 1u);
#pragma unroll 1
        for (uint32_t bit = first < 0 ? 0u : 1u << first; bit >= 0x10000u; bit >>= 1) {
          const uint32_t c = t | bit;
          uint32_t n = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) n += w[i] >= c;
          if (__reduce_add_sync(0xffffffffu, n) >= k) t = c;
        }
      }
      if (lane == 0) s_floor = max(s_floor, t);
    }
    __syncthreads();
  };

  // steps past the segment's last vector hold -inf, which weighs nothing
  Loader<T> raw[kUnroll];
  const T* const first = x + lead + static_cast<int64_t>(lane) * kVec;
  auto fetch = [&](int t) {
    const int left = t < t1 ? nvec - (t * (kTile / kVec) + lane) : 0;
    const T* src = first + static_cast<int64_t>(t) * kTile;
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      if (32 * q < left) raw[q].load(src + 32 * q * kVec);
      else raw[q].none();
    }
  };
  fetch(t0 + warp);
  if constexpr (TOP) {
    // the first bound: the k-th largest of the threads' maxima
    float top = raw[0].top();
#pragma unroll
    for (int q = 1; q < kUnroll; ++q) top = max_nan(top, raw[q].top());
    const uint32_t mine = (t0 + warp) * (kTile / kVec) + lane < nvec && t0 + warp < t1 ? ordered(top) : 0u;
    if (k == 1) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, mine);
      if (lane == 0) atomicMax(&s_floor, m);
      __syncthreads();
    } else {
      s_lane[tid] = mine;
      __syncthreads();
      kth_of_lanes();
    }
  }

  const int rounds = (t1 - t0 + kWarps - 1) / kWarps;  // every warp takes part in each
  int again = 4;  // the rounds after which the bound is next taken from the lists
                  // (the first bound does for a while: from 1, 128 rows with k = 5 took 30 us, not 27)
  for (int round = 0; round < rounds; ++round) {
    const int t = t0 + round * kWarps + warp;
    const int v0 = t * (kTile / kVec) + lane;
    Loader<T> cur[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) cur[q] = raw[q];
    fetch(t + kWarps);
    float most = cur[0].top();  // of this thread's tile
#pragma unroll
    for (int q = 1; q < kUnroll; ++q) most = max_nan(most, cur[q].top());
    float v[8];
    if (absorb(most)) {
      float ts = 0.f, tw = 0.f;
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        cur[q].raised(low, v);
        weigh(v, ts, tw);
      }
      st.s += ts;
      st.w += tw;
    } else {
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        cur[q].get(v);
        count(v);
      }
    }
    if (!(most <= xt)) {
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) st.rank += cur[q].above(xt);
    }
    if constexpr (TOP) {
      // what is known of the k-th best, as a value (no bound yet gives a NaN,
      // which nothing is below); later ids of a value that a full list holds
      // lose to it
      const float bound = from_ordered(*reinterpret_cast<volatile uint32_t*>(&s_floor));
      const bool full = st.kth != 0;
      const float bar = from_ordered(static_cast<uint32_t>(st.kth >> 32));
      const bool look = t < t1 && !(most < bound) && !(full && most <= bar);
      if (__any_sync(0xffffffffu, look)) {
        const uint64_t before = st.kth;
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
          cur[q].get(v);
          const bool live = look && v0 + 32 * q < nvec;
          if (!__any_sync(0xffffffffu, live && !(cur[q].top() < bound))) continue;
          const int64_t id0 = lead + static_cast<int64_t>(v0 + 32 * q) * kVec;
#pragma unroll
          for (int i = 0; i < 8; ++i) offer(v[i], id0 + i, live && !(v[i] < bound));
          if (pending > kPending - 256) place_pending();  // room for the next 256
        }
        place_pending();
        if (st.kth != before && lane == 0) atomicMax(&s_floor, static_cast<uint32_t>(st.kth >> 32));
      }
      if (round + 1 == again && round + 1 < rounds) {  // (uniform)
        again *= 2;
        if (k > 1) {
          // the k-th best of all lists (lanes from k on hold keys that were pushed
          // out of their list, or none: the bound is as true with them)
          s_lane[tid] = static_cast<uint32_t>(st.mine >> 32);
          __syncthreads();
          kth_of_lanes();
        }
      }
    }
  }
  // the row's ends: warp 0 of the first segment, warp 0 of the last
  auto ends = [&](int64_t id0, int n) {  // up to 7 elements, one a lane
    const bool live = lane < n;
    const float one = live ? load1(x + id0 + lane) : -INFINITY;
    if (live) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = -INFINITY;
      v[0] = one;
      if (absorb(one)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaxf(v[i], low);
        weigh(v, st.s, st.w);
      } else {
        count(v);
      }
      st.rank += !(one <= xt);
    }
    if constexpr (TOP) {
      offer(one, id0 + lane, live);
      place_pending();
    }
  };
  if (warp == 0 && seg == 0) ends(0, static_cast<int>(lead));
  if (warp == 0 && seg == S - 1) {
    const int64_t done = lead + static_cast<int64_t>(nvec) * kVec;
    ends(done, static_cast<int>(p.V - done));
  }
  if (st.m > low) {  // from here on relative to the maximum
    const float ref = st.m * c, d = st.ref - ref, f = exp2_approx(d);
    st.w = fmaf(st.s, d, st.w) * f;
    st.s *= f;
  }

  // ---- the warp's, then the CTA's statistics: sums relative to another
  // reference, d above it, shrink by 2^-d, and each e's exponent falls by d
  auto join = [&](float& m, float& s, float& w, float m2, float s2, float w2) {
    const float M = max_nan(m, m2), ref = fmaxf(M, low) * c;
    const float d1 = m == M ? 0.f : M > low ? fmaxf(fmaxf(m, low) * c - ref, -1e30f) : -1e30f;
    const float d2 = m2 == M ? 0.f : M > low ? fmaxf(fmaxf(m2, low) * c - ref, -1e30f) : -1e30f;
    const float f1 = exp2_approx(d1), f2 = exp2_approx(d2);
    w = fmaf(s, d1, w) * f1 + fmaf(s2, d2, w2) * f2;
    s = s * f1 + s2 * f2;
    m = M;
  };
  // lane 0 .. n - 1's (n a power of two; the others hold nothing), into every lane
  auto join_warp = [&](float& m, float& s, float& w, int& rank, int n) {
    for (int o = n / 2; o > 0; o >>= 1) {
      // both sides of a pair join the lower lane's to the upper one's, so all agree
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o),
                  w2 = __shfl_xor_sync(0xffffffffu, w, o);
      const bool up = lane & o;
      float ma = up ? m2 : m, sa = up ? s2 : s, wa = up ? w2 : w;
      join(ma, sa, wa, up ? m : m2, up ? s : s2, up ? w : w2);
      m = ma;
      s = sa;
      w = wa;
      rank += __shfl_xor_sync(0xffffffffu, rank, o);
    }
    m = __shfl_sync(0xffffffffu, m, 0);
    s = __shfl_sync(0xffffffffu, s, 0);
    w = __shfl_sync(0xffffffffu, w, 0);
    rank = __shfl_sync(0xffffffffu, rank, 0);
  };
  join_warp(st.m, st.s, st.w, st.rank, 32);
  if (lane == 0) {
    s_m[warp] = st.m;
    s_s[warp] = st.s;
    s_w[warp] = st.w;
    s_rank[warp] = st.rank;
  }
  if (TOP && tid == 0) s_count = 0;
  __syncthreads();
  if constexpr (TOP) {  // the lists' keys that the bound leaves
    if (st.mine != 0 && lane < k && static_cast<uint32_t>(st.mine >> 32) >= s_floor) s_keys[atomicAdd(&s_count, 1)] = st.mine;
    __syncthreads();
  }

  // the k best of n distinct keys in s_keys: a key's place is the number of
  // larger ones
  auto select = [&](int n, auto&& out) {
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = s_keys[i];
      uint32_t place = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) place += s_keys[j] > key;
      if (place < k) out(place, key);
    }
  };
  static_assert(kWarps == 8, "the shuffles below");
  const bool mine = lane < kWarps;
  float m = mine ? s_m[lane] : -INFINITY, s = mine ? s_s[lane] : 0.f, w = mine ? s_w[lane] : 0.f;
  int rank = mine ? s_rank[lane] : 0;
  join_warp(m, s, w, rank, kWarps);
  auto finish = [&](float M, float Sum, float Wsum, int Rank, int nkeys) {
    // base 2 to e; a row without a finite logit has no distribution
    const bool none = M == -INFINITY, nan = M != M || M == INFINITY;
    const float lse2 = log2f(Sum);  // relative to ref
    const float ref = fmaxf(M, low) * c;
    auto lp = [&](float v) {
      if (nan) return __uint_as_float(0x7FC00000u);
      if (none || v == -INFINITY) return -INFINITY;
      if (v <= low || M <= low) return (v - M) * temp - lse2 * kLn2;
      return fminf((fmaf(v, c, -ref) - lse2) * kLn2, 0.f);  // ref and the sum are rounded
    };
    if (tid == 0) {
      p.logprob[row] = has_tok ? lp(xt) : nan ? __uint_as_float(0x7FC00000u) : -INFINITY;
      p.entropy[row] = nan ? __uint_as_float(0x7FC00000u) : none ? 0.f : fmaxf((lse2 - Wsum / Sum) * kLn2, 0.f);
      p.rank[row] = !has_tok ? static_cast<int32_t>(p.V) : xt != xt ? 0 : Rank;
    }
    if constexpr (TOP)
      select(nkeys, [&](uint32_t place, uint64_t key) {
        const float v = from_ordered(static_cast<uint32_t>(key >> 32));
        p.top_ids[row * k + place] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
        p.top_logprobs[row * k + place] = lp(v);
      });
  };
  if (S == 1) {
    finish(m, s, w, rank, TOP ? s_count : 0);
    return;
  }
  // ---- several segments: the last to arrive joins them
  if (tid == 0) {
    Partial q;
    q.m = m;
    q.s = s;
    q.w = w;
    q.rank = rank;
    __stcg(reinterpret_cast<float4*>(p.partials + row * S + seg), *reinterpret_cast<const float4*>(&q));
  }
  if constexpr (TOP) {
    uint64_t* dst = p.keys + (row * S + seg) * k;
    if (tid < k) __stcg(reinterpret_cast<unsigned long long*>(dst + tid), 0ull);
    __syncthreads();
    select(s_count, [&](uint32_t place, uint64_t key) {
      __stcg(reinterpret_cast<unsigned long long*>(dst + place), static_cast<unsigned long long>(key));
    });
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    s_last = atomicAdd(p.arrived + row, 1u) == static_cast<uint32_t>(S - 1);
    if (s_last) p.arrived[row] = 0;
    s_count = 0;
    s_floor = 0;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  m = -INFINITY;
  s = w = 0.f;
  rank = 0;
  for (int i = lane; i < S; i += 32) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p.partials + row * S + i));
    join(m, s, w, v.x, v.y, v.z);
    rank += __float_as_int(v.w);
  }
  join_warp(m, s, w, rank, 32);
  if constexpr (TOP) {
    // a bound on the k-th best of the segments' keys, from the threads' largest
    const uint64_t* src = p.keys + row * S * k;
    uint32_t top = 0;
    for (int i = tid; i < S * static_cast<int>(k); i += kThreads)
      top = max(top, static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned long long*>(src + i)) >> 32));
    s_lane[tid] = top;
    __syncthreads();
    kth_of_lanes();
    const uint32_t floor_bits = s_floor;
    for (int i = tid; i < S * static_cast<int>(k); i += kThreads) {
      const uint64_t key = __ldcg(reinterpret_cast<const unsigned long long*>(src + i));
      if (key != 0 && static_cast<uint32_t>(key >> 32) >= floor_bits) s_keys[atomicAdd(&s_count, 1)] = key;
    }
    __syncthreads();
  }
  finish(m, s, w, rank, TOP ? s_count : 0);
}

// Segments of a row: as many CTAs as run at once, by their registers three per SM
// for bf16 logits and two for fp32 ones (128 rows of 131071, k = 5, two, three,
// four per SM: bf16 30, 30, 39 us, fp32 28, 41, 35; bf16 cut to 64 registers for
// four: 32), and at least two tiles a warp (joining two segments of one tile costs
// 2.4 us, a second tile 1 us).
int64_t most_segments(int64_t V) {
  const int64_t n = V / (2 * kWarps * kTile);
  return n < 1 ? 1 : n < kMaxSegments ? n : kMaxSegments;
}
int segments(int64_t T, int64_t V, int num_sms, bool f32) {
  const int64_t want = (f32 ? 2 : 3) * static_cast<int64_t>(num_sms) / T, most = most_segments(V);
  return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

// The workspace: the rows' arrival counters, then a call's partials, then its
// keys.  The counters' place does not depend on the call, so that what one call
// leaves behind them is never another's counter: rows are split only while two
// segments of each fit, so there are never more counters than this.
size_t counter_bytes(int num_sms) { return (static_cast<size_t>(3 * num_sms / 2) * 4 + 255) / 256 * 256; }
size_t segment_bytes(int k) { return sizeof(Partial) + 8 * static_cast<size_t>(k); }

}  // namespace

// For any call of up to T rows of up to V logits and up to k alternatives: where
// rows are split, there are at most 3 SMs segments in all.
size_t logprobs_workspace_bytes(int64_t T, int64_t V, int k, int num_sms) {
  const int64_t row = most_segments(V), all = 3 * static_cast<int64_t>(num_sms);
  const int64_t n = row == 1 ? 0 : T * row < all ? T * row : all;
  return counter_bytes(num_sms) + static_cast<size_t>(n) * segment_bytes(k);
}

size_t logprobs_workspace_needed(const LogprobsArgs& a) {
  const int S = segments(a.T, a.V, a.num_sms, a.f32);
  return S == 1 ? 0 : counter_bytes(a.num_sms) + static_cast<size_t>(a.T) * S * segment_bytes(a.k);
}

cudaError_t launch_token_logprobs(const LogprobsArgs& a, cudaStream_t stream) {
  const int S = segments(a.T, a.V, a.num_sms, a.f32);
  Params p;
  p.V = a.V;
  p.row_stride = a.row_stride;
  p.k = a.k;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = a.pdl ? 1 : 0;
  constexpr int64_t kMaxRows = 65535;  // of one launch: the grid's second dimension
  for (int64_t r = 0; r < a.T; r += kMaxRows) {
    const int64_t n = a.T - r < kMaxRows ? a.T - r : kMaxRows;
    p.logits = static_cast<const char*>(a.logits) + r * a.row_stride * (a.f32 ? 4 : 2);
    p.tokens = a.tokens + r;
    p.inv_temperature = a.inv_temperature == nullptr ? nullptr : a.inv_temperature + r;
    p.logprob = a.logprob + r;
    p.entropy = a.entropy + r;
    p.rank = a.rank + r;
    p.top_ids = a.top_ids == nullptr ? nullptr : a.top_ids + r * a.k;
    p.top_logprobs = a.top_logprobs == nullptr ? nullptr : a.top_logprobs + r * a.k;
    p.arrived = reinterpret_cast<uint32_t*>(ws) + r;
    p.partials = reinterpret_cast<Partial*>(ws + counter_bytes(a.num_sms)) + r * S;
    p.keys = reinterpret_cast<uint64_t*>(ws + counter_bytes(a.num_sms) + static_cast<size_t>(a.T) * S * sizeof(Partial)) + r * S * a.k;
    cfg.gridDim = dim3(static_cast<unsigned>(S), static_cast<unsigned>(n));
    cudaError_t e;
    if (a.f32)
      e = a.k > 0 ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<float, true>, p)
                  : cudaLaunchKernelEx(&cfg, token_logprobs_kernel<float, false>, p);
    else
      e = a.k > 0 ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<__nv_bfloat16, true>, p)
                  : cudaLaunchKernelEx(&cfg, token_logprobs_kernel<__nv_bfloat16, false>, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace wq
