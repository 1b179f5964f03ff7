// wq_kv4_split.cuh -- attention of a few query rows over the 4-bit cache: one
// new token per sequence, or a short block of drafted tokens.  Instantiated
// per head dimension in wq_kv4_split_d*.cu.
//
//   O_i = sum_j 2^(t_ij - m_i) v_j / sum_j 2^(t_ij - m_i),
//   t_ij = scale log2(e) sum_g s_jg sum_{d in g} q_id c_jd,   v_jd = s'_jg c'_jd
// with integer codes c, c' and the per-group scales s, s' of the cache.
//
// Bound: the cache's bytes.  At 6.8 TB/s an SM has to turn 47 codes a clock
// into operands, so the codes are never multiplied by a scale: both products
// run on the integer codes as fp16 (exact) with fp32 sums, the key scale
// multiplies a score and the value scale a weight.  Two or three integer
// operations make two operands.
//
//  * Rows.  The query rows of one key/value head (tokens x grouped heads) in
//    tiles of 8, or 16 for heads of 64 (8 NT).  Both products run transposed, on m16n8k16 with
//    n = 8 query rows: S^T = K Q^T (m = 16 keys), then O^T = V^T P^T (m = 16
//    dimensions, k = 16 keys), so eight rows waste nothing; the weights become
//    the second product's operand by an 8 x 8 transpose within the warp.
//  * Codes.  A granule is 16 consecutive keys, all of one page.  A thread's
//    key words (its quarter of the dimensions of keys g and g + 8) are 8 to 32
//    contiguous bytes; its value words hold dimension g of every eight, and a
//    byte permute of two keys' words pairs them for the transposed operand.
//    Each warp copies its own granules with 16-byte cp.async into a private
//    ring of kStages, so there is no barrier between warps while they stream;
//    rows are permuted within 128 bytes so that the fragment loads meet no
//    bank twice.
//  * Softmax in base 2 with one lazy reference R per row: weights are 2^(t - R)
//    and the sums of weights and of weighted values share it.  R follows the
//    largest product of a weight and its value scale, which is what fp16 has to
//    hold: when one passes 2^16, R is moved so that the largest lies at 2^10 to
//    2^11.  That is rare after a warp's first granule, so a granule takes one
//    vote instead of shuffles and a rescale of O, and products down to 2^-24 of
//    a row's largest keep fp16's 11 bits, however far its value scales are
//    apart.  Queries are normalised per row by a power of two (exact).
//  * Work.  The items (sequence, row tile, head) are laid end to end in units
//    of kUnit keys, and the CTAs take equal contiguous ranges of units, so a
//    ragged batch and a single long sequence load all SMs alike.  An item that
//    spans CTAs leaves partial (max, sum, O) rows in the workspace; the last
//    of its CTAs to arrive merges them in CTA order, so results do not depend
//    on timing.  The arrival counter belongs to the item's first CTA and is
//    reset by the merger.
//
// Measured (32 query and 8 key/value heads of 128): 64 sequences of 4096 at most,
// one token each: 53 us, 3.3 TB/s; one sequence of 131071: 46 us, 3.1 TB/s; one of
// 1000: 9.4 us.  What bounds it is not bytes (DRAM at half its rate) but about 400
// instructions for a granule of a head, dependent ones, in the sixteen warps an SM
// has registers for: they fill half of the issue slots.  For the short sequence it
// is the chain of a launch, the page lookup, a copy, the products and the join.
#pragma once

#include <atomic>
#include <mutex>
#include <type_traits>

#include "wq_device.cuh"
#include "wq_kv4.cuh"

namespace wq {
namespace kv4split {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = kWarps * 16;  // keys of a work unit, a granule per warp
constexpr int kStages = 4;          // granules in flight per warp
// CTAs of an SM, for the registers and the workspace: four of four warps.  Two
// of eight read one sequence of 131071 keys in 43 us instead of 46, having
// fewer partials to join, but a batch of 64 ragged ones in 58 instead of 53,
// since all of a CTA's warps wait where its range passes from item to item;
// a fifth CTA (96 registers, spilled) costs 5 us.
constexpr int kMaxCtasSm = 4;
constexpr int kMaxRows = 16;
constexpr float kPlace = 10.f;          // log2 of where R places a row's largest
constexpr float kNoRef = -1e30f;        // R of a row that has seen no key

struct Params {
  Kv4Params kv;
  Rows Q, O;
  int Hq, gq;          // query heads, and per key/value head
  float scale_log2;    // scale * log2(e)
  int window;          // 0: none
  float* partials;     // [2 * gridDim.x][rows][D + 4]
  uint32_t* arrived;   // [gridDim.x]
};

// ---------------------------------------------------------------- fp16 ---
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_half2_rn(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ uint32_t half2_max(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Whether one of two halves without sign is an infinity (a NaN loses against
// any number in half2_max, so it does not count).
__device__ __forceinline__ bool half2_is_over(uint32_t a) {
  return (a & 0xFFFFu) == 0x7C00u || (a >> 16) == 0x7C00u;
}
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of halves, row `lane / 4`, columns 2 (lane % 4) + {0, 1}, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// The same onto zeros, which need no registers.
__device__ __forceinline__ void mma_f16_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                   uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Nibbles i and i + 4 (i even: bits 0..3 of the halves, odd: bits 4..7) of x
// as the fp16 pair of their codes: 1024 + n (or 64 + n) by setting the
// exponent, minus 1032 (or 72) -- exact.
__device__ __forceinline__ uint32_t codes_low(uint32_t x) {
  return half2_sub(lop3_and_or(x, 0x000F000Fu, 0x64006400u), 0x64086408u);
}
__device__ __forceinline__ uint32_t codes_high(uint32_t x) {
  return half2_sub(lop3_and_or(x, 0x00F000F0u, 0x54005400u), 0x54805480u);
}

// 16-byte chunk (row, c) of a granule's codes in shared memory.  A row has
// C = D/32 chunks; the permutation spreads the rows one fragment load touches
// (keys 2t + e for the values, eight consecutive lanes' rows for the keys)
// over all banks.
//
// Two consequences keep the addresses in a few registers: row + 8 lies at a
// constant distance, kRow8, and row + 1 of an even row at the address with the
// bits kOdd flipped.
template <int D>
__device__ __forceinline__ int chunk_pos(int row, int c) {
  if constexpr (D == 64) return (row * 2 + c) ^ (((row >> 2) & 1) << 1);
  if constexpr (D == 128) return (row * 4 + c) ^ (((row >> 2) & 1) << 2) ^ (((row >> 1) & 1) << 1);
  return row * 8 + (c ^ (row & 1) ^ (((row >> 1) & 3) << 1));
}

// The exponent of |x| as a power of two, 2^floor(log2 |x|), within the
// normals; NaN and inf give 2^127.
__device__ __forceinline__ float pow2_floor(float x) {
  const uint32_t e = min(max((__float_as_uint(x) >> 23) & 0xFFu, 1u), 254u);
  return __uint_as_float(e << 23);
}

inline size_t kv4_counter_bytes(int num_sms) {
  return (static_cast<size_t>(num_sms) * kMaxCtasSm * 4 + 255) / 256 * 256;
}

inline Params make_params(const Kv4Args& a, const Kv4AttentionArgs& x) {
  Params p;
  p.kv = kv4_params(a);
  p.Q = x.Q;
  p.O = x.O;
  p.Hq = x.Hq;
  p.gq = x.Hq / a.Hkv;
  p.scale_log2 = x.scale * 1.44269504088896341f;
  p.window = static_cast<int>(x.window < (int64_t(1) << 30) ? x.window : int64_t(1) << 30);
  p.arrived = static_cast<uint32_t*>(x.workspace);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(x.workspace) + kv4_counter_bytes(a.num_sms));
  return p;
}

template <int D, int G>
struct Geometry {
  static constexpr int kCodes = 8 * D;          // bytes of a granule's key (or value) codes
  static constexpr int kScales = 32 * G;        // bytes of its key (or value) scales
  static constexpr int kStage = 2 * kCodes + 2 * kScales;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr uint32_t kRow8 = 8 * D / 2;                              // bytes from row to row + 8
  static constexpr uint32_t kOdd = D == 64 ? 32 : D == 128 ? 64 : 144;      // bits from an even row to the next
};
// The warps' partials of an item: O rows (padded by 4), reference and sum.  The
// same memory takes the factors of all CTAs' partials when they are joined.
constexpr int kMostCtas = 1024;
template <int D, int NT>
constexpr int merge_bytes() {
  constexpr int warps = kWarps * 8 * NT * (D + 4 + 2) * 4, ctas = 8 * NT * (kMostCtas + 1) * 4;
  return warps > ctas ? warps : ctas;
}
template <int D, int G, int NT>
constexpr int smem_bytes() {
  return (Geometry<D, G>::kRing > merge_bytes<D, NT>() ? Geometry<D, G>::kRing : merge_bytes<D, NT>()) + 128;
}

// The batch's work: sequence b has tiles(b) * Hkv items of units(b) units.
struct SeqWork {
  Kv4Seq s;
  int lo;       // first key any of its queries sees, down to a granule
  int units;
  int64_t items;
};
__device__ __forceinline__ SeqWork seq_work(const Params& p, int b, int rows_tile) {
  SeqWork w;
  w.s = kv4_load_sequence(p.kv, b);
  const int len = static_cast<int>(w.s.len);
  const int p0 = len - static_cast<int>(w.s.n);  // position of its first query (negative: sees nothing)
  w.lo = p.window > 0 && p0 - p.window + 1 > 0 ? (p0 - p.window + 1) & ~15 : 0;
  w.units = len > w.lo ? (len - w.lo + kUnit - 1) / kUnit : 1;
  w.items = (w.s.n * p.gq + rows_tile - 1) / rows_tile * p.kv.Hkv;
  return w;
}

// The item in work and the CTA's place in its units, kept by thread 0 in
// shared memory: the threads read what they need of it, and hold no registers
// for the rest while they stream.
struct Work {
  int64_t U, C;                // units in all, CTAs that have any
  int64_t u, u1;               // the CTA's next unit, and its end
  int64_t seq_start;           // unit where sequence b begins
  int64_t item_start, first;   // the item's first unit; its sequence's first token
  int b, h, rows, x0, x1, units;
  int len, lo, p0;             // cached tokens, first key, position of the sequence's first query
  int tok0, r0;                // the tile's first row: token tok0 of the sequence, head r0 of the group
  __device__ int64_t range_start(int64_t c) const { return U * c / C; }  // U < 2^45, C < 2^12
  __device__ int64_t cta_of(int64_t v) const {
    int64_t c = v * C / U;
    while (range_start(c + 1) <= v) ++c;
    return c;
  }
  // the item that holds unit u; false past the CTA's end
  __device__ bool next(const Params& p, int rows_tile) {
    if (u >= u1) return false;
    SeqWork sw = seq_work(p, b, rows_tile);
    while (u >= seq_start + sw.items * sw.units) {
      seq_start += sw.items * sw.units;
      sw = seq_work(p, ++b, rows_tile);
    }
    const int64_t item = (u - seq_start) / sw.units;
    item_start = seq_start + item * sw.units;
    units = sw.units;
    x0 = static_cast<int>(u - item_start);
    x1 = static_cast<int>(min(item_start + sw.units, u1) - item_start);
    h = static_cast<int>(item % p.kv.Hkv);
    const int64_t row0 = item / p.kv.Hkv * rows_tile;
    rows = static_cast<int>(min(sw.s.n * p.gq - row0, static_cast<int64_t>(rows_tile)));
    len = static_cast<int>(sw.s.len);
    lo = sw.lo;
    p0 = len - static_cast<int>(sw.s.n);
    first = sw.s.first;
    tok0 = static_cast<int>(row0 / p.gq);
    r0 = static_cast<int>(row0 % p.gq);
    u = item_start + x1;
    return true;
  }
};

template <int D, int G, int NT>
__global__ void __launch_bounds__(kThreads, kMaxCtasSm)
kv4_split_kernel(const Params p) {
  using Geo = Geometry<D, G>;
  constexpr int kRows = 8 * NT;
  static_assert(kRows <= kMaxRows, "the workspace's partials");
  constexpr int kKW = D / 32;                   // key words of a thread per key
  constexpr int kVW = D / 64;                   // value words of a thread per key
  constexpr int kGroupWords = kKW / G;          // key words of one group
  constexpr int kMT = D / 16;                   // 16-dimension tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[kThreads + 1];
  __shared__ Work wk;
  __shared__ int s_last, s_more, s_cf, s_cl;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  pdl_wait_primary();
  pdl_launch_dependents();

  // ---- this CTA's units: a scan of the sequences' units, a chunk a thread
  const int per = (p.kv.B + kThreads - 1) / kThreads;
  {
    int64_t sum = 0;
    for (int b = tid * per; b < min(p.kv.B, (tid + 1) * per); ++b) {
      const SeqWork w = seq_work(p, b, kRows);
      sum += w.items * w.units;
    }
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __shared__ int64_t s_warp[kWarps];
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int64_t base = 0;
    for (int w = 0; w < warp; ++w) base += s_warp[w];
    s_scan[tid + 1] = base + inc;
    if (tid == 0) s_scan[0] = 0;
    __syncthreads();
  }
  if (tid == 0) {
    wk.U = s_scan[kThreads];
    wk.C = wk.U < gridDim.x ? wk.U : gridDim.x;
    wk.u = wk.u1 = 0;
    if (blockIdx.x < wk.C) {
      wk.u = wk.range_start(blockIdx.x);
      wk.u1 = wk.range_start(blockIdx.x + 1);
      int lo = 0, hi = kThreads;  // the chunk with s_scan[lo] <= u < s_scan[lo + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s_scan[mid] <= wk.u) lo = mid; else hi = mid;
      }
      wk.b = lo * per;
      wk.seq_start = s_scan[lo];
    }
  }
  const uint32_t ring_s = smem_addr(smem + warp * kStages * Geo::kStage);
  // what a lane's addresses consist of
  const uint32_t page_mask = p.kv.lay.page() - 1;
  const uint32_t page_stride = static_cast<uint32_t>(p.kv.lay.block) * p.kv.Hkv;   // < 2^27
  const uint32_t v_codes = static_cast<uint32_t>(p.kv.lay.v_codes());
  const uint32_t scales_at = static_cast<uint32_t>(lane < 2 * G ? p.kv.lay.k_scales() : p.kv.lay.v_scales() - 32 * G);
  const uint32_t copy_at = chunk_pos<D>(lane / (D / 32), lane % (D / 32)) * 16;
  const uint32_t key_at = kKW == 2 ? chunk_pos<D>(g, t4 >> 1) * 16 + (t4 & 1) * 8 : chunk_pos<D>(g, t4 * (kKW / 4)) * 16;
  const uint32_t value_at = Geo::kCodes + (kVW == 1 ? chunk_pos<D>(2 * t4, g >> 2) * 16 + (g & 3) * 4
                                           : kVW == 2 ? chunk_pos<D>(2 * t4, g >> 1) * 16 + (g & 1) * 8
                                                      : chunk_pos<D>(2 * t4, g) * 16);
  const uint32_t scale_at = 2 * Geo::kCodes + g * 2 * G;

  while (true) {
    // ---- the item: a head and a tile of rows of a sequence, units [x0, x1)
    if (tid == 0) s_more = wk.next(p, kRows);
    __syncthreads();
    if (!s_more) break;
    const int len = wk.len;
    const int pos_first = wk.p0 + wk.tok0;
    const int pos_last = pos_first + (wk.r0 + wk.rows - 1) / p.gq;
    const int key0 = wk.lo + wk.x0 * kUnit + warp * 16;    // this warp's first granule
    const int ngran = wk.x1 - wk.x0;
    const int32_t* table = p.kv.page_table + wk.b * p.kv.max_pages;

    // ---- granule copies: a commit per granule, also for those past the end
    const uint8_t* head = p.kv.pool + p.kv.lay.block * wk.h + lane * 16;
    auto page_of = [&](int i) -> int {  // -1: not a page, -2: no granule
      const int key = key0 + i * kUnit;
      return i < ngran && key < len ? max(__ldg(table + (key >> p.kv.lay.page_shift)), -1) : -2;
    };
    auto issue = [&](int i, int page) {
      if (page != -2) {
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.kv.num_pages)) {
          // recorded; page 0 stands in, so nothing out of range is read
          if (lane == 0) atomicMax(p.kv.err, kErrBounds);
          page = 0;
        }
        const uint32_t slot = (key0 + i * kUnit) & page_mask;
        const uint8_t* blk = head + static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_stride;
        const uint8_t* kc = blk + slot * (D / 2);
        const uint8_t* vc = kc + v_codes;
        const uint32_t st = ring_s + (i % kStages) * Geo::kStage;
        constexpr int kCopies = D / 2 / 32;  // 16-byte chunks of a lane
#pragma unroll
        for (int q = 0; q < kCopies; ++q) {  // 512 bytes on: 8 rows of 64, or 4 of 128, whose chunks are permuted by 4 more
          const uint32_t at = st + ((D == 256 && (q & 1) ? copy_at ^ 64u : copy_at) + 512 * q);
          cp_async_16(at, kc + q * 512, 16);
          cp_async_16(at + Geo::kCodes, vc + q * 512, 16);
        }
        // lane * 16 is in the pointer: the value scales begin 32 G into the granule's
        if (lane < 4 * G) cp_async_16(st + 2 * Geo::kCodes + lane * 16, blk + scales_at + slot * 2 * G, 16);
      }
      cp_async_commit();
    };
    {
      int pg[kStages - 1];
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) pg[i] = page_of(i);
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) issue(i, pg[i]);
    }
    int next_page = page_of(kStages - 1);

    // ---- queries as B fragments: rows g (and g + 8), normalised per row
    uint32_t qa[2 * kKW][NT == 2 ? 4 : 2];
    float row_scale[NT][2];  // of rows 8 n + 2 t4 + {0, 1}
    int row_pos[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = g + 8 * i;
      const bool live = r < wk.rows;
      const int at = wk.r0 + (live ? r : 0);
      const int64_t tok = wk.first + wk.tok0 + at / p.gq;
      const int head_q = wk.h * p.gq + at % p.gq;
      const int pos = live ? pos_first + at / p.gq : -1;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.Q.data) + tok * p.Q.token_stride + head_q * p.Q.head_stride;
      uint4 raw[kKW];
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < kKW; ++w) {
        raw[w] = live ? *reinterpret_cast<const uint4*>(q + 32 * w + 8 * t4) : make_uint4(0, 0, 0, 0);
        const uint32_t e[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max((e[j] & 0x7FFFu), (e[j] >> 16) & 0x7FFFu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // |q| / norm < 2^13: products with codes and their sums stay far inside fp32
      const float norm = pow2_floor(fmaxf(__uint_as_float(top << 16), 1e-30f)) * 0x1p-12f;
      const float inv = 1.0f / norm;  // a power of two: exact
      const float rs = norm * p.scale_log2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        row_scale[i][e] = __shfl_sync(0xffffffffu, rs, 8 * t4 + 4 * e);
        row_pos[i][e] = __shfl_sync(0xffffffffu, pos, 8 * t4 + 4 * e);
      }
#pragma unroll
      for (int w = 0; w < kKW; ++w) {
        const uint32_t e[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          qa[2 * w + (j >> 1)][(j & 1) * NT + i] =
              pack_half2_rn(bf16_lo_to_f32(e[j]) * inv, bf16_hi_to_f32(e[j]) * inv);
      }
    }

    float ref[NT][2], l_sum[NT][2];
    float o[kMT][NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      ref[i][0] = ref[i][1] = kNoRef;
      l_sum[i][0] = l_sum[i][1] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;

    // One granule of keys kb .. kb + 15 at st in shared memory.  MASKED: not
    // every row sees all of them.
    auto granule = [&](uint32_t st, int kb, auto masked) {
      constexpr bool MASKED = decltype(masked)::value;
      // scales of this thread's keys g and g + 8
      constexpr int kSW = (G + 1) / 2;
      auto scale_words = [&](uint32_t (&v)[2][kSW], uint32_t a) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t at = a + 16 * x * G;
          if constexpr (G == 1) {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(at));
            v[x][0] = h;
          } else if constexpr (G == 2) {
            v[x][0] = ld_shared_u32(at);
          } else if constexpr (G == 4) {
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v[x][0]), "=r"(v[x][1]) : "r"(at));
          } else {
            const uint4 u = ld_shared_v4(at);
            v[x][0] = u.x;
            v[x][1] = u.y;
            v[x][2] = u.z;
            v[x][3] = u.w;
          }
        }
      };
      auto scale = [&](const uint32_t (&v)[2][kSW], int x, int q) {
        return (q & 1) ? bf16_hi_to_f32(v[x][q >> 1]) : bf16_lo_to_f32(v[x][q >> 1]);
      };
      uint32_t ks[2][kSW], kw[2][kKW];
      scale_words(ks, st + scale_at);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t at = st + key_at + x * Geo::kRow8;
        if constexpr (kKW == 2) {
          asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(kw[x][0]), "=r"(kw[x][1]) : "r"(at));
        } else {
#pragma unroll
          for (int c = 0; c < kKW / 4; ++c) {
            const uint4 v = ld_shared_v4(c ? st + (key_at ^ 16u) + x * Geo::kRow8 : at);
            kw[x][4 * c] = v.x;
            kw[x][4 * c + 1] = v.y;
            kw[x][4 * c + 2] = v.z;
            kw[x][4 * c + 3] = v.w;
          }
        }
      }
      // ---- scores: sc[n][2 x + e] of key kb + g + 8 x, row 8 n + 2 t4 + e
      float sc[NT][4];
#pragma unroll
      for (int q = 0; q < G; ++q) {
        float acc[NT][4], acc2[NT][4];  // two chains of products, for their latency
#pragma unroll
        for (int ww = 0; ww < kGroupWords; ++ww) {
          const int w = q * kGroupWords + ww;
          const uint32_t l0 = kw[0][w], l1 = kw[1][w], h0 = l0 >> 8, h1 = l1 >> 8;
          const uint32_t a0 = codes_low(l0), a1 = codes_low(l1), a2 = codes_high(l0), a3 = codes_high(l1);
          const uint32_t e0 = codes_low(h0), e1 = codes_low(h1), e2 = codes_high(h0), e3 = codes_high(h1);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (ww == 0) {
              mma_f16_16816_zero(acc[n], a0, a1, a2, a3, qa[2 * w][n], qa[2 * w][NT + n]);
              mma_f16_16816_zero(acc2[n], e0, e1, e2, e3, qa[2 * w + 1][n], qa[2 * w + 1][NT + n]);
            } else {
              mma_f16_16816(acc[n], a0, a1, a2, a3, qa[2 * w][n], qa[2 * w][NT + n]);
              mma_f16_16816(acc2[n], e0, e1, e2, e3, qa[2 * w + 1][n], qa[2 * w + 1][NT + n]);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = acc[n][e] + acc2[n][e], k = scale(ks, e >> 1, q);
            sc[n][e] = q == 0 ? a * k : fmaf(a, k, sc[n][e]);
          }
      }
      uint32_t vs[2][kSW];
      scale_words(vs, st + scale_at + Geo::kScales);
      // ---- weights, as fp16 products with each group's value scale
      float wt[NT][4], sum[NT][2];
      uint32_t wb[G][NT][2];  // rows in pairs of a key, until they are transposed
      uint32_t most = 0;
      bool seen[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = kb + g + 8 * (e >> 1), pos = row_pos[n][e & 1];
          seen[n][e] = !MASKED || (j <= pos && j < len && (p.window == 0 || j > pos - p.window));
        }
      auto weigh = [&] {
        most = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = exp2_approx(fmaf(sc[n][e], row_scale[n][e & 1], -ref[n][e & 1]));
            wt[n][e] = seen[n][e] ? w : 0.f;
          }
          sum[n][0] = wt[n][0] + wt[n][2];
          sum[n][1] = wt[n][1] + wt[n][3];
#pragma unroll
          for (int q = 0; q < G; ++q)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float w0 = wt[n][2 * x] * scale(vs, x, q), w1 = wt[n][2 * x + 1] * scale(vs, x, q);
              if (MASKED) {  // a key the row does not see adds nothing, whatever its scale
                w0 = seen[n][2 * x] ? w0 : 0.f;
                w1 = seen[n][2 * x + 1] ? w1 : 0.f;
              }
              wb[q][n][x] = pack_half2_rn(w0, w1);
              most = half2_max(most, wb[q][n][x] & 0x7FFF7FFFu);
            }
        }
      };
      weigh();
      bool over = half2_is_over(most);
#pragma unroll
      for (int n = 0; n < NT; ++n) over |= fmaxf(sum[n][0], sum[n][1]) > 0x1p105f;
      if (__any_sync(0xffffffffu, over)) {
        float sk[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          sk[x] = 0x1p-85f;  // holds a weight itself below 2^100
#pragma unroll
          for (int q = 0; q < G; ++q) sk[x] = fmaxf(sk[x], fabsf(scale(vs, x, q)));
          sk[x] = static_cast<float>(__float_as_uint(sk[x]) >> 23) - 127.f;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float top = kNoRef;
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (seen[n][2 * x + r]) top = fmaxf(top, sc[n][2 * x + r] * row_scale[n][r] + sk[x]);
            // the row's keys lie in the lanes of the same t4
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float moved = fmaxf(ref[n][r], top - kPlace);
            const float f = exp2_approx(ref[n][r] - moved);
            ref[n][r] = moved;
            l_sum[n][r] *= f;
            // O^T's columns are these rows too
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
              o[mt][n][r] *= f;
              o[mt][n][2 + r] *= f;
            }
          }
        weigh();
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        l_sum[n][0] += sum[n][0];
        l_sum[n][1] += sum[n][1];
#pragma unroll
        for (int q = 0; q < G; ++q) {
          wb[q][n][0] = transpose8(wb[q][n][0]);
          wb[q][n][1] = transpose8(wb[q][n][1]);
        }
      }
      // ---- O^T += V^T (w s')^T, a group of dimensions at a time
      uint32_t vw[4][kVW];  // keys 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t at = st + (y & 1 ? value_at ^ Geo::kOdd : value_at) + (y >> 1) * Geo::kRow8;
        if constexpr (kVW == 1) {
          vw[y][0] = ld_shared_u32(at);
        } else if constexpr (kVW == 2) {
          asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(vw[y][0]), "=r"(vw[y][1]) : "r"(at));
        } else {
          const uint4 v = ld_shared_v4(at);
          vw[y][0] = v.x;
          vw[y][1] = v.y;
          vw[y][2] = v.z;
          vw[y][3] = v.w;
        }
      }
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        constexpr int kTilesGroup = kMT / G;
        const int q = mt / kTilesGroup;
        // dimensions 16 mt + g and + 8: nibbles 2 (mt % 4) and + 1 of word mt / 4
        const int j = mt / 4;
        uint32_t z0 = __byte_perm(vw[0][j], vw[1][j], mt % 4 < 2 ? 0x5410 : 0x7632);
        uint32_t z1 = __byte_perm(vw[2][j], vw[3][j], mt % 4 < 2 ? 0x5410 : 0x7632);
        if (mt & 1) {
          z0 >>= 8;
          z1 >>= 8;
        }
        const uint32_t a0 = codes_low(z0), a1 = codes_high(z0), a2 = codes_low(z1), a3 = codes_high(z1);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16_16816(o[mt][n], a0, a1, a2, a3, wb[q][n][0], wb[q][n][1]);
      }
    };
    // granules that some row sees, and those that every row sees whole
    auto granules_to = [&](int key) { return key <= key0 ? 0 : min((key - key0 + kUnit - 1) / kUnit, ngran); };  // that begin before key
    const int end_seen = granules_to(min(len, pos_last + 1)), end_whole = granules_to(min(len, pos_first + 1) - 15);
    const int begin_seen = p.window > 0 ? granules_to(pos_first - p.window - 14) : 0;
    const int begin_whole = p.window > 0 ? granules_to(pos_last - p.window + 1) : 0;
#pragma unroll 1
    for (int i = 0; i < ngran; ++i) {
      __syncwarp();  // every lane is done with the stage that is refilled now
      issue(i + kStages - 1, next_page);
      next_page = page_of(i + kStages);
      cp_async_wait_group<kStages - 1>();
      __syncwarp();
      const uint32_t st = ring_s + (i % kStages) * Geo::kStage;
      if (i >= begin_whole && i < end_whole)
        granule(st, 0, std::false_type());
      else if (i >= begin_seen && i < end_seen)
        granule(st, key0 + i * kUnit, std::true_type());
    }
    cp_async_wait_all();
    __syncthreads();  // the rings are done; their memory takes the warps' partials

    // ---- merge the warps: rows of O, padded by 4 floats, then (max, sum)
    constexpr int kORow = D + 4;
    float* wo = reinterpret_cast<float*>(smem);
    float* wm = wo + kWarps * kRows * kORow;  // [warp][row]
    float* wl = wm + kWarps * kRows;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l_sum[n][r] += __shfl_xor_sync(0xffffffffu, l_sum[n][r], 4);
        l_sum[n][r] += __shfl_xor_sync(0xffffffffu, l_sum[n][r], 8);
        l_sum[n][r] += __shfl_xor_sync(0xffffffffu, l_sum[n][r], 16);
        if (g == 0) {
          wm[warp * kRows + 8 * n + 2 * t4 + r] = ref[n][r];
          wl[warp * kRows + 8 * n + 2 * t4 + r] = l_sum[n][r];
        }
      }
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 8 * n + 2 * t4 + (e & 1);
          if (r < wk.rows) wo[(warp * kRows + r) * kORow + 16 * mt + g + 8 * (e >> 1)] = o[mt][n][e];
        }
    }
    __syncthreads();
    const bool whole = wk.x0 == 0 && wk.x1 == wk.units;
    constexpr int kQuads = D / 4;
    auto out_row = [&](int r) {
      const int at = wk.r0 + r;
      return static_cast<__nv_bfloat16*>(p.O.data) + (wk.first + wk.tok0 + at / p.gq) * p.O.token_stride +
             (wk.h * p.gq + at % p.gq) * p.O.head_stride;
    };
    auto store = [&](int r, int c, float4 v, float L) {
      const float inv = L == 0.f ? 0.f : 1.f / L;  // a row without keys is 0; a NaN stays one
      st_global_v2(out_row(r) + 4 * c, pack_bf16x2_rn(v.x * inv, v.y * inv), pack_bf16x2_rn(v.z * inv, v.w * inv));
    };
    constexpr int kSlot = kRows * (D + 4);  // floats of a partial: rows of O, then (max, sum) pairs
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (wk.x0 == 0 ? 1 : 0);
    for (int q = tid; q < wk.rows * kQuads; q += kThreads) {
      const int r = q / kQuads, c = q % kQuads;
      float M = kNoRef;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * kRows + r]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        // a warp that saw nothing has sums of 0 (or a NaN, which stays)
        const float f = exp2_approx(wm[w * kRows + r] - M);
        const float4 y = *reinterpret_cast<const float4*>(wo + (w * kRows + r) * kORow + 4 * c);
        L += wl[w * kRows + r] * f;
        v.x += y.x * f;
        v.y += y.y * f;
        v.z += y.z * f;
        v.w += y.w * f;
      }
      if (whole) {
        store(r, c, v, L);
      } else {
        float* dst = p.partials + slot * kSlot;
        __stcg(reinterpret_cast<float4*>(dst + r * D + 4 * c), v);
        if (c == 0) __stcg(reinterpret_cast<float2*>(dst + kRows * D + 2 * r), make_float2(M, L));
      }
    }
    if (!whole) {
      // the CTAs of this item: from the one that holds its first unit to the
      // one that holds its last
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        s_cf = static_cast<int>(wk.cta_of(wk.item_start));
        s_cl = static_cast<int>(wk.cta_of(wk.item_start + wk.units - 1));
        s_last = atomicAdd(p.arrived + s_cf, 1u) == static_cast<uint32_t>(s_cl - s_cf);
        if (s_last) p.arrived[s_cf] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        // every partial's factor first (rows of the shared memory that the
        // warps' partials had), then sums whose loads do not wait for one another
        const int n = s_cl - s_cf + 1;
        float* fac = wo;                      // [row][n]
        float* sums = fac + kRows * n;        // [row]
        auto part = [&](int k) {
          return p.partials + (2 * static_cast<int64_t>(s_cf + k) + (k == 0 ? 1 : 0)) * kSlot;
        };
        for (int r = warp; r < wk.rows; r += kWarps) {
          float M = kNoRef;
          for (int k = lane; k < n; k += 32) M = fmaxf(M, __ldcg(part(k) + kRows * D + 2 * r));
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
          float L = 0.f;
          for (int k = lane; k < n; k += 32) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(k) + kRows * D + 2 * r));
            const float f = exp2_approx(ml.x - M);
            fac[r * n + k] = f;
            L += ml.y * f;
          }
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
          if (lane == 0) sums[r] = L;
        }
        __syncthreads();
        for (int q = tid; q < wk.rows * kQuads; q += kThreads) {
          const int r = q / kQuads, c = q % kQuads;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int k = 0; k < n; ++k) {
            const float f = fac[r * n + k];
            const float4 y = __ldcg(reinterpret_cast<const float4*>(part(k) + r * D + 4 * c));
            v.x += y.x * f;
            v.y += y.y * f;
            v.z += y.z * f;
            v.w += y.w * f;
          }
          store(r, c, v, sums[r]);
        }
      }
    }
    __syncthreads();  // the partials' memory becomes the rings again, and the item changes
  }
}

// CTAs that fit an SM, asked once per device and variant.
template <int D, int G, int NT>
struct Init {
  std::atomic<uint64_t> done{0};
  std::mutex mu;
  int ctas[64] = {};
  cudaError_t ensure(int device, int* per_sm) {
    const uint64_t bit = 1ull << (device & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
      std::lock_guard<std::mutex> lk(mu);
      if (!(done.load() & bit)) {
        constexpr int bytes = smem_bytes<D, G, NT>();
        cudaError_t e = cudaFuncSetAttribute(kv4_split_kernel<D, G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kv4_split_kernel<D, G, NT>, kThreads, bytes);
        if (e != cudaSuccess) return e;
        ctas[device & 63] = n < 1 ? 1 : n > kMaxCtasSm ? kMaxCtasSm : n;
        done.fetch_or(bit, std::memory_order_release);
      }
    }
    *per_sm = ctas[device & 63];
    return cudaSuccess;
  }
};

template <int D, int G, int NT>
cudaError_t launch_variant(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  static Init<D, G, NT> init;
  int per_sm = 1;
  cudaError_t e = init.ensure(a.device, &per_sm);
  if (e != cudaSuccess) return e;
  const Params p = make_params(a, x);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_sms * per_sm < kMostCtas ? a.num_sms * per_sm : kMostCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D, G, NT>();
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = a.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kv4_split_kernel<D, G, NT>, p);
}

}  // namespace kv4split
}  // namespace wq
