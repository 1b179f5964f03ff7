// wq_kv4_tile.cuh -- attention of many query rows over the 4-bit cache: blocks
// of drafted tokens with grouped heads, and chunks of a prompt.  Instantiated
// per head dimension in wq_kv4_tile_d*.cu.  The mathematics, the references
// of the softmax and the use of the workspace are those of wq_kv4_split.cuh;
// here both products run on the tensor cores from tensor memory.
//
// Bound: with 256 rows, the tensor cores -- a block of 128 keys takes two
// 128 x 128 x 128 products per 128 rows, 2,048 clocks for 256 rows, in which
// the SM's schedulers have 8,192 slots for 32,768 weights (about five
// instructions each) and 32,768 codes (about two each).
//
// Measured (32 query and 8 key/value heads of 128): 2048 tokens after 6144: 340 us,
// 708 TFLOP/s (with a window of 1024 keys 116, heads of 64 283); 8 blocks of 16 tokens
// after 16384 at most: 108 us.  A block of keys
// takes about 6,200 clocks for 256 rows: a stream's chain -- its softmax, 2,500
// clocks alone and about 4,000 beside the other stream's products, which take the
// shared memory's rate for their operands, and the eight warps of codes; then its
// two products, behind the other stream's in the tensor cores' queue -- is what is
// waited for (the tensor cores are busy 30% of the time, the issue slots 46%).  With
// 128 rows (a block in 3,700 clocks) the codes are: their 16 keys a warp are a chain
// of loads, scales, and stores of 3,000 clocks.
//
//  * Rows.  An item is a head's tile of 128 NT rows (tokens x grouped heads).
//    Two streams alternate on the tensor core so that one stream's softmax
//    runs under the other's products: with NT = 2 (more than 128 rows) the
//    tile's halves, with NT = 1 the same rows over even and over odd blocks of
//    keys, joined at the end of the item.
//    One thread of each stream issues the stream's products.
//  * Codes to operands.  Eight warps turn a block's codes into fp16 in shared
//    memory, once for all rows: keys as [key][dimension], values transposed as
//    [dimension][key], both in the 128-byte swizzle the tensor core reads.  A
//    warp owns 16 keys (one page).  Operands are codes times their scale, which
//    fp16 holds exactly (3 and 8 significant bits), relative to a power of two
//    for the warp's sixteen keys (or, for values of very different scales, for
//    each); that power multiplies scores and weights.  The next block's codes
//    wait in registers, the one after is on its way into L2.
//  * Softmax.  A thread owns a row (a lane of tensor memory); it reads the
//    scores in 32-column pieces, and writes the fp16 weights over them, from
//    where the second product reads them as its A operand.
//  * Work is spread over the CTAs as in the few-row kernel: equal contiguous
//    ranges of 128-key units, partial rows through the workspace, the last CTA
//    of an item joins them in order.
//  * Every wait is bounded; a wait that runs out ends all roles and is
//    recorded.
#pragma once

#include <atomic>
#include <mutex>

#include "wq_kv4_split.cuh"
#include "wq_tcgen05.cuh"

namespace wq {
namespace kv4tile {

using kv4split::exp2_approx;
using kv4split::kNoRef;
using kv4split::pack_half2_rn;
using kv4split::Params;
using kv4split::pow2_floor;

constexpr int kKeys = 128;              // keys of a block, and of a work unit
constexpr int kSoftWarps = 8;           // four per stream
constexpr int kCodeWarps = 8;           // 16 keys of a block each
constexpr int kThreads = (kSoftWarps + kCodeWarps) * 32;
constexpr int kFacRing = 4;             // blocks whose key factors are kept
constexpr uint32_t kSleepNs = 2000;     // longest sleep inside one try of a wait
// log2 of where a row's reference places its largest product of a weight and a
// value factor.  Lower than in the few-row kernel, since a move costs far more
// (0.14 moves a block and warp, with the reference placed at 2^10, made a chunk
// of 2048 tokens after 6144 take 584 us, none 411); 2^-20 of the largest is still
// held to 11 bits.
constexpr float kPlace = 6.f;
constexpr float kMostHalf = 65504.f;    // fp16's largest

// 1 / x of a normal power of two, without a division's chain.
__device__ __forceinline__ float pow2_inverse(float x) {
  const uint32_t b = __float_as_uint(x);
  return __uint_as_float(b == 254u << 23 ? 1u << 22 : (254u << 23) - b);  // (2^-127 is a subnormal)
}

struct TileParams {
  Params a;
  KernelDiag diag;
};

// Sixteen keys' common factors: of their scores (log2 e and the call's scale in
// it), and 2^v of their weights.
struct Granule {
  float k, v, v_inv, pad;  // v_inv = 2^-v
};

template <int D, int G, int NT>
struct Smem {
  static constexpr int kQ = 128 * D * 2;           // a tile's queries
  static constexpr int kBlock = kKeys * D * 2;     // a block's keys, or values
  static constexpr int kOffQ = 0;                  // (and, at an item's end, the factors of its partials)
  static constexpr int kOffK = kOffQ + 2 * kQ;
  static constexpr int kOffV = kOffK + 2 * kBlock;
  static constexpr int kOffFac = kOffV + 2 * kBlock;                   // [ring][key, value][128] fp32
  static constexpr int kOffGran = kOffFac + kFacRing * 2 * kKeys * 4;   // [ring][8] Granule
  static constexpr int kOffEven = kOffGran + kFacRing * 8 * 16;         // [ring][8] int
  static constexpr int kOffRat = kOffEven + kFacRing * 8 * 4;           // [block % 2][warp][2][16][G] fp16
  static constexpr int kOffBar = kOffRat + 2 * kCodeWarps * 2 * 16 * G * 2;
  static constexpr int kBars = 2 * 4 + 2 * 3;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kBytes = kOffMisc + 64 + 1024;             // + alignment
};

// ------------------------------------------------------------------ items ---
struct Item {
  int b, h, rows;
  int64_t row0;
  Kv4Seq s;
  int pos_first, pos_last, lo, units;
  int64_t start;  // its first unit
};

// The units of a sequence's row tile: the keys from the first that any of its
// rows sees to the last.
template <int kRows>
__device__ __forceinline__ void tile_range(const Params& p, const Kv4Seq& s, int64_t tile, Item* it) {
  const int64_t all = s.n * p.gq;
  it->row0 = tile * kRows;
  it->rows = static_cast<int>(min(all - it->row0, static_cast<int64_t>(kRows)));
  const int len = static_cast<int>(s.len), p0 = len - static_cast<int>(s.n);
  it->pos_first = p0 + static_cast<int>(it->row0 / p.gq);
  it->pos_last = p0 + static_cast<int>((it->row0 + it->rows - 1) / p.gq);
  const int hi = max(min(len, it->pos_last + 1), 0);
  it->lo = p.window > 0 ? max(it->pos_first - p.window + 1, 0) & ~15 : 0;
  it->units = hi > it->lo ? (hi - it->lo + kKeys - 1) / kKeys : 1;
}

// Walks the items from a given unit on.
template <int kRows>
struct Walk {
  const Params& p;
  Item it;
  int64_t tile, group_start;  // the tile's first unit (its heads follow one another)
  __device__ explicit Walk(const Params& q) : p(q) {}
  __device__ int64_t tiles() const { return (it.s.n * p.gq + kRows - 1) / kRows; }
  __device__ void open(int b, int64_t start) {
    it.b = b;
    it.s = kv4_load_sequence(p.kv, b);
    tile = 0;
    group_start = start;
    if (it.s.n > 0) tile_range<kRows>(p, it.s, 0, &it);
  }
  // the item that holds unit u (not before the one it stands on)
  __device__ void seek(int64_t u) {
    while (it.s.n == 0 || u >= group_start + static_cast<int64_t>(it.units) * p.kv.Hkv) {
      if (it.s.n > 0) group_start += static_cast<int64_t>(it.units) * p.kv.Hkv;
      if (it.s.n > 0 && tile + 1 < tiles())
        tile_range<kRows>(p, it.s, ++tile, &it);
      else
        open(it.b + 1, group_start);
    }
    it.h = static_cast<int>((u - group_start) / it.units);
    it.start = group_start + static_cast<int64_t>(it.h) * it.units;
  }
};

template <int kRows>
__device__ __forceinline__ int64_t seq_units(const Params& p, int b) {
  Item it;
  const Kv4Seq s = kv4_load_sequence(p.kv, b);
  const int64_t tiles = (s.n * p.gq + kRows - 1) / kRows;
  int64_t sum = 0;
  for (int64_t t = 0; t < tiles; ++t) {
    tile_range<kRows>(p, s, t, &it);
    sum += it.units;
  }
  return sum * p.kv.Hkv;
}

// A CTA that gives up in the item that holds unit u still counts as arrived at
// the one item that it has not reached and that others share, the last of its
// range: so the counters are zeros again when all CTAs are through.  `scan`: the
// units before each chunk of sequences.
template <int kRows, int kChunks>
static __device__ __noinline__ void arrive_at_last(const Params& p, const int64_t* scan, int64_t u) {
  const int64_t U = scan[kChunks], C = U < gridDim.x ? U : gridDim.x, cta = blockIdx.x;
  const int64_t u1 = U * (cta + 1) / C;  // where the CTA's range ends
  int lo = 0, hi = kChunks;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (scan[mid] < u1) lo = mid; else hi = mid;
  }
  Walk<kRows> walk(p);
  walk.open(lo * ((p.kv.B + kChunks - 1) / kChunks), scan[lo]);
  walk.seek(u1 - 1);
  const int64_t end = walk.it.start + walk.it.units;
  if (walk.it.start <= u || end <= u1) return;  // (has been reached; or is this CTA's alone)
  int64_t last = (end - 1) * C / U;  // the CTA that has the item's last unit
  while (U * (last + 1) / C < end) ++last;
  if (atomicAdd(p.arrived + cta, 1u) == static_cast<uint32_t>(last - cta)) p.arrived[cta] = 0;
}

// ------------------------------------------------------------ fp16 pairs ---
// Two fp32 numbers in one register pair, and their instructions.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // NaNs lose
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void half2_unpack(uint32_t a, float& lo, float& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(lo), "=f"(hi) : "r"(a));
}
// One lane of a whole warp, chosen the same for every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// 16 registers per thread -> 32 lanes x 16 consecutive TMEM columns.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Instruction descriptor, kind::f16: A, B fp16, D fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// ----------------------------------------------------- a block's softmax ---
// Waits for the loads before it, and hands their registers on: what uses them
// cannot be moved before the wait.
template <int N>
__device__ __forceinline__ void tmem_ld_wait_regs(uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 32, "");
  if constexpr (N == 8)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
  else
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// These two are rare and out of the block's loop; they are short loops because
// what costs them most is fetching their instructions.

// The reference that places the largest weight times value factor of a
// block's columns lo .. hi at 2^kPlace; kNoRef where there is none.
static __device__ __noinline__ float first_reference(uint32_t ts, const float* kfac, const float* vfac, float row_scale, int lo, int hi) {
  float top = kNoRef;
#pragma unroll 1
  for (int c = 0; c < kKeys; c += 8) {
    uint32_t raw[8];
    tmem_ld_32x32b_x8(ts + c, raw);
    tmem_ld_wait_regs(raw);
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      const float t = __uint_as_float(raw[y]) * kfac[c + y] * row_scale;
      const float v = fmaxf(fabsf(vfac[c + y]), 0x1p-85f);
      if (c + y >= lo && c + y <= hi) top = fmaxf(top, t + (static_cast<float>(__float_as_uint(v) >> 23) - 127.f));
    }
  }
  return fmaxf(floorf(top) - kPlace, kNoRef);
}
// What a row has so far times f, a power of two of 1 or less: the weights in
// `wcols` columns at ts and O's `ocols` at to.
static __device__ __noinline__ void shrink(uint32_t ts, int wcols, uint32_t to, int ocols, float f) {
  tmem_st_wait();  // the pieces' weights have been stored without a wait, and a load does not wait for stores
#pragma unroll 1
  for (int q = 0; q < wcols; q += 8) {
    uint32_t v[8];
    tmem_ld_32x32b_x8(ts + q, v);
    tmem_ld_wait_regs(v);
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      float x0, x1;
      half2_unpack(v[y], x0, x1);
      v[y] = pack_half2_rn(x0 * f, x1 * f);
    }
    tmem_st_32x32b_x8(ts + q, v);
  }
#pragma unroll 1
  for (int q = 0; q < ocols; q += 8) {
    uint32_t v[8];
    tmem_ld_32x32b_x8(to + q, v);
    tmem_ld_wait_regs(v);
#pragma unroll
    for (int y = 0; y < 8; ++y) v[y] = __float_as_uint(__uint_as_float(v[y]) * f);
    tmem_st_32x32b_x8(to + q, v);
  }
  tmem_st_wait();
}

// One row's block: scores from tensor memory (ts) to fp16 weights over them,
// in four pieces of 32 columns.
//
// EVEN: all columns count, and sixteen keys share their factors.  This is the
// usual block, and it reads next to nothing from shared memory: 64 loads of
// factors a row and block made it 1.7 times as slow under the other stream's
// scores, which read their operands from there at its full rate.
// Otherwise only the columns lo .. hi count, and each key has its own factors
// (kfac, vfac).  Scores are multiplied by row_scale.
//
// A weight that has left fp16 (or, where value factors are tiny, fp32's
// middle) moves the row's reference up and shrinks what the row has so far.
// Whether one has is asked a piece later, when the answer costs no wait: the
// scores of the piece are still there then, since piece c's weights take
// columns 16 c .. 16 c + 15 -- but for piece 0, which is asked at once.
template <int D, bool EVEN>
__device__ __forceinline__ void weigh_block(uint32_t ts, uint32_t to, const float* kfac, const float* vfac, const Granule* gran,
                                            float row_scale, int lo, int hi, bool has_o, float& ref, float& l) {
  if (__any_sync(0xffffffffu, ref == kNoRef)) {  // the first keys a row sees (O and the sum are 0 so far)
    const float r = first_reference(ts, kfac, vfac, row_scale, EVEN ? 0 : lo, EVEN ? kKeys - 1 : hi);
    if (ref == kNoRef) ref = r;
  }
  float sum_before = 0.f;
  bool over_before = false;
#pragma unroll 1
  for (int c = 0;;) {
    uint32_t w[16];
    float sum = 0.f;
    bool over = false;
    if (c < 4) {
      uint32_t raw[32];
      tmem_ld_32x32b_x32(ts + 32 * c, raw);
      // two columns to an instruction where there is one for them; the largest
      // weight by three-way maxima (a packed fp16 maximum takes five clocks)
      float most[2] = {0.f, 0.f};
      if constexpr (EVEN) {
        const float4 ga = *reinterpret_cast<const float4*>(gran + 2 * c), gb = *reinterpret_cast<const float4*>(gran + 2 * c + 1);
        tmem_ld_wait_regs(raw);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float k = (u ? gb.x : ga.x) * row_scale, nr = (u ? gb.y : ga.y) - ref;
          const uint64_t k2 = pair(k, k), nr2 = pair(nr, nr);
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int z = 8 * u; z < 8 * u + 8; ++z) {
            float t0, t1;
            unpair(fma2(pair(__uint_as_float(raw[2 * z]), __uint_as_float(raw[2 * z + 1])), k2, nr2), t0, t1);
            const float e0 = exp2_approx(t0), e1 = exp2_approx(t1);
            sums[z & 1] = add2(sums[z & 1], pair(e0, e1));
            w[z] = pack_half2_rn(e0, e1);
            most[z & 1] = max3(most[z & 1], e0, e1);
          }
          float s0, s1;
          unpair(add2(sums[0], sums[1]), s0, s1);
          sum = fmaf(s0 + s1, u ? gb.z : ga.z, sum);
        }
      } else {
        tmem_ld_wait_regs(raw);
        const uint64_t nr = pair(-ref, -ref), rs = pair(row_scale, row_scale);
        uint64_t sums[4] = {0, 0, 0, 0};
#pragma unroll
        for (int z = 0; z < 16; ++z) {
          const int j = 32 * c + 2 * z;
          const uint64_t kf = reinterpret_cast<const uint64_t*>(kfac)[j / 2], vf = reinterpret_cast<const uint64_t*>(vfac)[j / 2];
          const uint64_t x = pair(__uint_as_float(raw[2 * z]), __uint_as_float(raw[2 * z + 1]));
          float t0, t1, v0, v1;
          unpair(fma2(mul2(x, kf), rs, nr), t0, t1);
          const bool in0 = j >= lo && j <= hi, in1 = j + 1 >= lo && j + 1 <= hi;
          const uint64_t e = pair(in0 ? exp2_approx(t0) : 0.f, in1 ? exp2_approx(t1) : 0.f);
          sums[z & 3] = add2(sums[z & 3], e);
          unpair(mul2(e, vf), v0, v1);
          v0 = in0 ? v0 : 0.f;  // a hidden key adds nothing, whatever its factor
          v1 = in1 ? v1 : 0.f;
          w[z] = pack_half2_rn(v0, v1);
          most[z & 1] = max3(most[z & 1], v0, v1);
        }
        float s0, s1;
        unpair(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])), s0, s1);
        sum = s0 + s1;
      }
      over = fmaxf(most[0], most[1]) >= kMostHalf || sum > 0x1p105f;
    }
    if (__any_sync(0xffffffffu, c == 0 ? over : over_before)) {
      const int from = c == 0 ? 0 : c - 1;  // the piece that is over
      const float r =
          fmaxf(ref, first_reference(ts, kfac, vfac, row_scale, EVEN ? 32 * from : max(lo, 32 * from), EVEN ? kKeys - 1 : hi));
      if (__any_sync(0xffffffffu, r != ref)) {  // (else a score is not finite: nothing is left to move)
        const float f = exp2_approx(ref - r);   // a whole power of two
        shrink(ts, 16 * from, to, has_o ? D : 0, f);
        l *= f;
        ref = r;
        c = from;
        sum_before = 0.f;
        over_before = false;
        continue;
      }
    }
    l += sum_before;
    if (c == 4) break;
    tmem_st_32x32b_x16(ts + 16 * c, w);
    sum_before = sum;
    over_before = c != 0 && over;
    ++c;
  }
}

// Joins an item's partial rows, in order.  A warp takes 32 rows, a lane each,
// and 16 dimensions; the factors of the partials wait in `factors`.  Loads do not
// depend on one another: one partial after the other, a join of eight took 60 us.
// (Out of line, so that it does not cost the loop over blocks registers; with 32
// dimensions a task it still cost some, and a chunk 357 us instead of 340.)
template <int D>
constexpr int64_t kPartFloats = 256 * (D + 4);  // of one slot of the workspace

// A row's weighted sum from tensor memory to its place in the output, or, where
// there is none, to partial row `prow`: quads of dimensions [D/4][256], then
// reference and sum [256], so that with a lane a row every access of a warp is
// whole lines.  `any`: some block was summed (else the partial row is empty).
template <int D>
__device__ __noinline__ void store_row(uint32_t to, bool any, bool live, float ref, float sum, __nv_bfloat16* out, float* part, int prow) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t v[32];
    if (any) {
      tmem_ld_32x32b_x32(to + 32 * c, v);
      tmem_ld_wait_regs(v);
    } else {
#pragma unroll
      for (int y = 0; y < 32; ++y) v[y] = 0;
    }
    if (live && out != nullptr) {
#pragma unroll
      for (int y = 0; y < 4; ++y)
        st_global_v4(out + 32 * c + 8 * y, pack_bf16x2_rn(__uint_as_float(v[8 * y]) * inv, __uint_as_float(v[8 * y + 1]) * inv),
                     pack_bf16x2_rn(__uint_as_float(v[8 * y + 2]) * inv, __uint_as_float(v[8 * y + 3]) * inv),
                     pack_bf16x2_rn(__uint_as_float(v[8 * y + 4]) * inv, __uint_as_float(v[8 * y + 5]) * inv),
                     pack_bf16x2_rn(__uint_as_float(v[8 * y + 6]) * inv, __uint_as_float(v[8 * y + 7]) * inv));
    } else if (live) {
#pragma unroll
      for (int y = 0; y < 8; ++y)
        __stcg(reinterpret_cast<float4*>(part) + (8 * c + y) * 256 + prow,
               make_float4(__uint_as_float(v[4 * y]), __uint_as_float(v[4 * y + 1]), __uint_as_float(v[4 * y + 2]),
                           __uint_as_float(v[4 * y + 3])));
    }
  }
  if (live && out == nullptr) __stcg(reinterpret_cast<float2*>(part + 256 * D) + prow, make_float2(any ? ref : kNoRef, sum));
}

template <int D, int NT>
__device__ __noinline__ void join(const float* partials, int64_t cf, int parts, int rows, int64_t row0, __nv_bfloat16* out,
                                  int64_t token_stride, int64_t head_stride, int gq, float* factors) {
  constexpr int kAhead = D / 2;  // partials whose factors are held
  static_assert(kSoftWarps * kAhead * 32 * 4 <= 2 * 128 * D * 2, "the queries' place");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = (rows + 31) / 32;
  float* fk = factors + warp * kAhead * 32 + lane;
  int seen = -1;
  float M = kNoRef, sum = 0.f;
  for (int t = warp; t < blocks * (D / 16); t += kSoftWarps) {
    const int rb = t % blocks, qg = t / blocks, r = 32 * rb + lane;
    // partial x of the row (NT = 1: both streams' rows are partials)
    auto part_of = [&](int x) {
      const int64_t k = cf + (NT == 1 ? x >> 1 : x);
      return partials + (2 * k + (k == cf ? 1 : 0)) * kPartFloats<D>;
    };
    auto place = [&](int x) { return r + (NT == 1 ? 128 * (x & 1) : 0); };
    auto ref_sum = [&](int x) { return __ldcg(reinterpret_cast<const float2*>(part_of(x) + 256 * D) + place(x)); };
    const bool fresh = rb != seen;
    if (fresh) {
      M = kNoRef;
      sum = 0.f;
#pragma unroll 8
      for (int x = 0; x < parts; ++x) M = fmaxf(M, ref_sum(x).x);
      seen = rb;
    }
    float4 acc[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int from = 0; from < parts; from += kAhead) {
      const int end = min(parts, from + kAhead);
      if (fresh || parts > kAhead) {
#pragma unroll 8
        for (int x = from; x < end; ++x) {
          const float2 m2 = ref_sum(x);
          const float f = exp2_approx(m2.x - M);
          if (fresh) sum = fmaf(m2.y, f, sum);
          fk[(x - from) * 32] = f;
        }
      }
#pragma unroll 4
      for (int x = from; x < end; ++x) {
        const float4* src = reinterpret_cast<const float4*>(part_of(x)) + 4 * qg * 256 + place(x);
        const float f = fk[(x - from) * 32];
        float4 o[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) o[y] = __ldcg(src + y * 256);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          acc[y].x = fmaf(o[y].x, f, acc[y].x);
          acc[y].y = fmaf(o[y].y, f, acc[y].y);
          acc[y].z = fmaf(o[y].z, f, acc[y].z);
          acc[y].w = fmaf(o[y].w, f, acc[y].w);
        }
      }
    }
    if (r < rows) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      __nv_bfloat16* o = out + (row0 + r) / gq * token_stride + (row0 + r) % gq * head_stride + 16 * qg;
#pragma unroll
      for (int y = 0; y < 4; y += 2)
        st_global_v4(o + 4 * y, pack_bf16x2_rn(acc[y].x * inv, acc[y].y * inv), pack_bf16x2_rn(acc[y].z * inv, acc[y].w * inv),
                     pack_bf16x2_rn(acc[y + 1].x * inv, acc[y + 1].y * inv), pack_bf16x2_rn(acc[y + 1].z * inv, acc[y + 1].w * inv));
    }
  }
}

template <int D, int G, int NT>
__global__ void __launch_bounds__(kThreads, 1)
kv4_tile_kernel(const TileParams tp) {
  using S = Smem<D, G, NT>;
  constexpr int kRows = 128 * NT;
  constexpr uint32_t kTmemCols = 512;
  constexpr uint32_t kColO = 256;                 // S of stream s at 128 s, O at 256 + 128 s
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ int64_t s_scan[kThreads + 1];
  __shared__ int64_t s_warp[kThreads / 32];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_last, s_quit;
  const Params& p = tp.a;
  // (from lane 0, so that the compiler knows it the same in all lanes: the
  // products' operands then stay in uniform registers)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  volatile int* abort_flag = &s_abort;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* k_full = bars;          // [2] the block's keys are in shared memory
  uint64_t* k_empty = bars + 2;     // [2] every product that reads them is done
  uint64_t* v_full = bars + 4;      // [2]
  uint64_t* v_empty = bars + 6;     // [2]
  uint64_t* s_full = bars + 8;      // [stream] scores are in tensor memory
  uint64_t* o_done = bars + 10;     // [stream] the item's last weighted sum is done
  uint64_t* mma_done = bars + 12;   // [stream] everything issued is done (after giving up)
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], kCodeWarps);
      mbar_init(&k_empty[i], NT);   // from each stream that reads the block
      mbar_init(&v_full[i], kCodeWarps);
      mbar_init(&v_empty[i], NT);
      mbar_init(&s_full[i], 1);
      mbar_init(&o_done[i], 1);
      mbar_init(&mma_done[i], 1);
    }
    fence_mbar_init();
    s_abort = 0;
  }
  if (warp == kSoftWarps) {
    tmem_alloc(&s_tmem, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait_primary();
  pdl_launch_dependents();

  // ---- this CTA's units
  const int per = (p.kv.B + kThreads - 1) / kThreads;
  {
    int64_t inc = 0;
    for (int b = tid * per; b < min(p.kv.B, (tid + 1) * per); ++b) inc += seq_units<kRows>(p, b);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int64_t base = 0;
    for (int w = 0; w < warp; ++w) base += s_warp[w];
    s_scan[tid + 1] = base + inc;
    if (tid == 0) s_scan[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int64_t U = s_scan[kThreads];
  const int64_t C = U < gridDim.x ? U : gridDim.x;
  const int64_t cta = blockIdx.x;
  auto range_start = [&](int64_t c) { return U * c / C; };
  int64_t u0 = 0, u1 = 0;
  Walk<kRows> walk(p);
  if (cta < C) {
    u0 = range_start(cta);
    u1 = range_start(cta + 1);
    int lo = 0, hi = kThreads;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_scan[mid] <= u0) lo = mid; else hi = mid;
    }
    walk.open(lo * per, s_scan[lo]);
  }

  // lane 0 waits for its warp, so that a warp leaves its loop as a whole
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(smem_addr(bar), parity))) return true;
    int ok = 1;
    if (lane == 0) ok = role_wait(bar, parity, tp.diag, abort_flag, kSleepNs);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) mbar_try_wait(smem_addr(bar), parity);  // completes at once: makes the phase's writes visible
    return ok != 0;
  };
  // one arrival for a warp whose lanes have all done their part
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  const uint32_t sb = smem_addr(smem);

  if (warp < kSoftWarps) {
    // ================================================= softmax, one row a thread
    const int stream = warp >> 2, lane_row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * stream, to = tmem + lanes + kColO + 128 * stream;
    uint32_t n_s = 0, n_item = 0;     // score products, items seen by this stream
    const bool issuer = (warp & 3) == 0;  // one of its lanes issues the stream's products
    // ---- the products.  A thread's products run in the order it issues them,
    // so the next scores may go where the weights of the sum before them are.
    // The whole issuing warp calls these; one lane is elected for the products.
    constexpr uint32_t idesc_s = idesc_f16_f32(128, kKeys), idesc_o = idesc_f16_f32(128, D);
    const uint32_t d_s = tmem + 128 * stream, d_o = tmem + kColO + 128 * stream;
    const uint64_t q_desc = smem_desc_sw128(sb + S::kOffQ + (NT == 2 ? stream * S::kQ : 0));
    const uint64_t k_desc = smem_desc_sw128(sb + S::kOffK), v_desc = smem_desc_sw128(sb + S::kOffV);
    auto await = [&](uint64_t* bar, int64_t block) -> bool {  // block `block` of the CTA is in shared memory
      // test hook 2: a phase that never completes
      if (tp.diag.force_timeout == 2) return warp_wait(&mma_done[stream], 0);
      return warp_wait(&bar[block & 1], static_cast<uint32_t>((block >> 1) & 1));
    };
    // a block's place may be refilled: its products are known to be done (a
    // commit of their own would cost the tensor core about 150 clocks)
    auto release = [&](uint64_t* bar, int64_t block, bool alone) {
      if (lane != 0) return;
      mbar_arrive(&bar[block & 1]);
      if (NT == 2 && alone) mbar_arrive(&bar[block & 1]);  // the other stream has no rows
    };
    auto issue_scores = [&](int64_t block) {  // S = Q K^T
      if (!await(k_full, block)) return;
      const uint64_t kd = k_desc + __shfl_sync(0xffffffffu, static_cast<uint32_t>(block & 1) * (S::kBlock >> 4), 0);
      if (elect_one()) {
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_bf16(d_s, q_desc + (ks >> 2) * (16384 >> 4) + 2 * (ks & 3), kd + (ks >> 2) * ((kKeys * 128) >> 4) + 2 * (ks & 3),
                    idesc_s, ks != 0);
        umma_commit(&s_full[stream]);
      }
      __syncwarp();
    };
    auto issue_sum = [&](int64_t block, bool first, bool last) {  // O (+)= P V
      if (!await(v_full, block)) return;
      const uint64_t vd = v_desc + __shfl_sync(0xffffffffu, static_cast<uint32_t>(block & 1) * (S::kBlock >> 4), 0);
      const uint32_t add = __shfl_sync(0xffffffffu, first ? 0u : 1u, 0), done = __shfl_sync(0xffffffffu, last ? 1u : 0u, 0);
      if (elect_one()) {
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          umma_bf16_ts(d_o, d_s + 8 * ks, vd + (ks >> 2) * ((D * 128) >> 4) + 2 * (ks & 3), idesc_o, ks == 0 ? add : 1u);
        if (done) umma_commit(&o_done[stream]);
      }
      __syncwarp();
    };
    int64_t n_block = 0;              // blocks of the CTA so far (the factors' ring)
    bool ok = true;                   // no wait of this warp has given up
    int64_t u = u0;
    while (u < u1) {
      walk.seek(u);
      const Item& it = walk.it;
      const int x0 = static_cast<int>(u - it.start), x1 = static_cast<int>(min(it.start + it.units, u1) - it.start);
      const int n = x1 - x0;
      const int my = NT == 2 ? (it.rows > 128 * stream ? n : 0) : (n + 1 - stream) / 2;  // this stream's blocks
      const int row = NT == 2 ? 128 * stream + lane_row : lane_row;
      const bool live = row < it.rows;
      const int64_t R = it.row0 + (live ? row : 0);
      const int64_t tok = it.s.first + R / p.gq;
      const int head = it.h * p.gq + static_cast<int>(R % p.gq);
      const int len = static_cast<int>(it.s.len);
      const int p0 = len - static_cast<int>(it.s.n);
      const int pos = live ? p0 + static_cast<int>(R / p.gq) : -1;
      // ---- the row's query into shared memory
      // (NT = 1: both streams read the first tile, and both compute the norm)
      float row_scale;
      {
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.Q.data) + tok * p.Q.token_stride + head * p.Q.head_stride;
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = live ? *reinterpret_cast<const uint4*>(q + 8 * c) : make_uint4(0, 0, 0, 0);
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, max(e[j] & 0x7FFFu, (e[j] >> 16) & 0x7FFFu));
        }
        // fp16 holds the row normalised by a power of two, so that its largest
        // value is 2^12 or above: all bits of those down to 2^-26 of it.  (As they
        // are, values below 2^-14 would lose bits beside one of 2^-8.)
        const float big = __uint_as_float(top << 16);
        row_scale = pow2_floor(fmaxf(big, 1e-30f)) * 0x1p-12f;
        const float inv = 1.0f / row_scale;
        if (NT == 2 || stream == 0) {
          const uint32_t dst = sb + S::kOffQ + (NT == 2 ? stream * S::kQ : 0);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = live ? *reinterpret_cast<const uint4*>(q + 8 * c) : make_uint4(0, 0, 0, 0);
            const uint32_t e[4] = {v.x, v.y, v.z, v.w};
            uint32_t f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = pack_half2_rn(bf16_lo_to_f32(e[j]) * inv, bf16_hi_to_f32(e[j]) * inv);
            st_shared_v4(dst + (c >> 3) * 16384 + lane_row * 128 + (((c & 7) ^ (lane_row & 7)) << 4), f[0], f[1], f[2], f[3]);
          }
          fence_proxy_async_smem();
        }
      }
      // the stream's queries (NT = 1: both streams') are in place
      if (NT == 2)
        named_barrier_sync(2 + stream, 128);
      else
        named_barrier_sync(1, kSoftWarps * 32);
      const bool alone = it.rows <= 128;
      auto block_of = [&](int i) { return NT == 2 ? i : 2 * i + stream; };  // of the item's n
      if (issuer && ok && my > 0) issue_scores(n_block + block_of(0));
      const bool busy = __any_sync(0xffffffffu, live);  // else nobody reads what the products make of these rows
      // positions of the live rows of this warp's tile half, for the mask
      const int pf = NT == 2 && stream == 1 ? p0 + static_cast<int>((it.row0 + 128) / p.gq) : it.pos_first;
      const int pl = NT == 2 && stream == 0 && it.rows > 128 ? p0 + static_cast<int>((it.row0 + 127) / p.gq) : it.pos_last;

      float ref = live ? kNoRef : 0.f;  // (a row that is none asks for no reference)
      float L = 0.f;
      for (int i = 0; i < my; ++i) {  // (a warp that gave up still meets the barriers)
        const int blk = block_of(i);
        const int kb = it.lo + (x0 + blk) * kKeys;
        const float* kfac = reinterpret_cast<const float*>(smem + S::kOffFac) + ((n_block + blk) % kFacRing) * 2 * kKeys;
        const float* vfac = kfac + kKeys;
        if (ok) ok = warp_wait(&s_full[stream], n_s & 1);
        ++n_s;
        if (issuer && ok) {  // these scores, and the weighted sum issued before them, are done
          release(k_empty, n_block + blk, alone);
          if (i > 0) release(v_empty, n_block + block_of(i - 1), alone);
        }
        if (ok && busy) {
          tc_fence_after();
          const bool interior = kb + kKeys <= len && kb + kKeys - 1 <= pf && (p.window == 0 || kb > pl - p.window);
          // the columns lo .. hi of the block that this row sees
          const int hi = pos - kb, lo = p.window == 0 ? 0 : pos - p.window + 1 - kb;
          const int4* even = reinterpret_cast<const int4*>(smem + S::kOffEven) + ((n_block + blk) % kFacRing) * 2;
          const int4 ea = even[0], eb = even[1];
          const Granule* gran = reinterpret_cast<const Granule*>(smem + S::kOffGran) + ((n_block + blk) % kFacRing) * 8;
          if (interior && (ea.x & ea.y & ea.z & ea.w & eb.x & eb.y & eb.z & eb.w))
            weigh_block<D, true>(ts, to, kfac, vfac, gran, row_scale, lo, hi, i > 0, ref, L);
          else
            weigh_block<D, false>(ts, to, kfac, vfac, gran, row_scale, lo, hi, i > 0, ref, L);
          tmem_st_wait();
          tc_fence_before();
        }
        named_barrier_sync(2 + stream, 128);  // the stream's weights are in tensor memory
        if (issuer && ok) {
          issue_sum(n_block + blk, i == 0, i + 1 == my);
          if (i + 1 < my) issue_scores(n_block + block_of(i + 1));
        }
        __syncwarp();
      }
      // ---- the item's rows
      // ---- (a warp that gave up goes on to the barriers below, which the
      // others may already wait at; what it stores is undefined then)
      if (ok && my > 0) ok = warp_wait(&o_done[stream], n_item & 1);
      if (issuer && ok && my > 0) release(v_empty, n_block + block_of(my - 1), alone);
      if (my > 0) ++n_item;
      tc_fence_after();
      const bool whole = x0 == 0 && x1 == it.units;
      const bool direct = whole && (NT == 2 || n == 1);  // else there are partial rows to join
      if (my > 0 || (NT == 1 && !direct)) {
        float* part = p.partials + (2 * cta + (x0 == 0 ? 1 : 0)) * kPartFloats<D>;
        const int64_t R_ = it.row0 + row;
        store_row<D>(to, my > 0, live, ref, L,
                     direct ? static_cast<__nv_bfloat16*>(p.O.data) + (it.s.first + R_ / p.gq) * p.O.token_stride +
                                  (it.h * p.gq + R_ % p.gq) * p.O.head_stride
                            : nullptr,
                     part, 128 * stream + lane_row);
      }
      tc_fence_before();  // O has been read: the next item's products may overwrite it
      if (!direct) {
        auto cta_of = [&](int64_t v) {
          int64_t c = v * C / U;
          while (range_start(c + 1) <= v) ++c;
          return c;
        };
        const int64_t cf = whole ? cta : cta_of(it.start), cl = whole ? cta : cta_of(it.start + it.units - 1);
        __threadfence();
        named_barrier_sync(1, kSoftWarps * 32);
        if (tid == 0) {
          s_last = whole || atomicAdd(p.arrived + cf, 1u) == static_cast<uint32_t>(cl - cf);
          if (s_last && !whole) p.arrived[cf] = 0;
        }
        named_barrier_sync(1, kSoftWarps * 32);
        if (s_last) {
          __threadfence();
          join<D, NT>(p.partials, cf, static_cast<int>(cl - cf + 1) * (NT == 1 ? 2 : 1), it.rows, it.row0,
                      static_cast<__nv_bfloat16*>(p.O.data) + it.s.first * p.O.token_stride + it.h * p.gq * p.O.head_stride,
                      p.O.token_stride, p.O.head_stride, p.gq, reinterpret_cast<float*>(smem + S::kOffQ));
        }
      }
      // the item is over for both streams; all of them leave, or none
      named_barrier_sync(1, kSoftWarps * 32);
      if (tid == 0) s_quit = *abort_flag;
      named_barrier_sync(1, kSoftWarps * 32);
      if (s_quit) break;
      n_block += n;
      u = it.start + x1;
    }
    if (tid == 0 && u < u1) arrive_at_last<kRows, kThreads>(p, s_scan, u);
    // after giving up: let what was issued finish before tensor memory goes (a
    // commit counts its own thread's products, so the lane that issued them waits)
    if (issuer && __any_sync(0xffffffffu, *abort_flag)) {
      if (elect_one()) {
        umma_commit(&mma_done[stream]);
        KernelDiag d = tp.diag;
        if (d.wait_limit_ns < 1000000000ull) d.wait_limit_ns = 1000000000ull;
        mbar_wait_bounded(&mma_done[stream], 0, d);
      }
      __syncwarp();
    }
  } else {
    // ================================================= codes to operands
    const int cw = warp - kSoftWarps;   // keys 16 cw .. of every block
    constexpr int kKW = D / 32;         // key words of a thread per key
    static_assert(D == 64 || D == 128, "the value lanes below");
    // Registers of the next block: key codes of keys 8 x + its row (x = 0, 1),
    // value words of eight keys, the scales of one key or value row.
    struct Raw {
      uint32_t k[2][kKW], v[8];
      uint32_t sc[(G + 1) / 2];
    };
    // lanes of the key part: quarter t4 of row kr (and kr + 8); rows 4 apart in
    // a quarter-warp, whose chunks then fall on different banks
    const int t4 = lane & 3, kr = ((lane >> 2) & 1) * 4 + (lane >> 3);
    // lanes of the value part: dimension g of every eight, keys 8 oct ..; the
    // fourth choice is the word (D = 128) or the word's half (D = 64)
    const int vg = lane & 7, vsel = (lane >> 3) & 1, oct = lane >> 4;
    auto load = [&](Raw& r, const uint8_t* blk, int slot, bool have) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint8_t* a = blk + (slot + 8 * x + kr) * (D / 2) + t4 * (D / 8);
        if constexpr (kKW == 4) {
          const uint4 v = have ? __ldg(reinterpret_cast<const uint4*>(a)) : make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
          r.k[x][0] = v.x;
          r.k[x][1] = v.y;
          r.k[x][2] = v.z;
          r.k[x][3] = v.w;
        } else {
          const uint2 v = have ? __ldg(reinterpret_cast<const uint2*>(a)) : make_uint2(0x88888888u, 0x88888888u);
          r.k[x][0] = v.x;
          r.k[x][1] = v.y;
        }
      }
      const uint8_t* vb = blk + p.kv.lay.v_codes();
#pragma unroll
      for (int y = 0; y < 8; ++y)
        r.v[y] = have ? __ldg(reinterpret_cast<const uint32_t*>(vb + (slot + 8 * oct + y) * (D / 2)) +
                              (D == 128 ? 2 * vg + vsel : vg))
                      : 0x88888888u;
      // scales: lanes 0..15 key rows, 16..31 value rows
      const uint8_t* sp = blk + (lane < 16 ? p.kv.lay.k_scales() : p.kv.lay.v_scales()) + (slot + (lane & 15)) * 2 * G;
      if constexpr (G == 1)
        r.sc[0] = have ? __ldg(reinterpret_cast<const uint16_t*>(sp)) : 0u;
      else
#pragma unroll
        for (int q = 0; q < G / 2; ++q) r.sc[q] = have ? __ldg(reinterpret_cast<const uint32_t*>(sp) + q) : 0u;
    };

    // the walk of the blocks, one ahead of the block in work
    Walk<kRows> wb = walk;
    int64_t nu = u0;       // the unit of the block to fetch next
    int f_left = 0;        // this CTA's blocks of its item
    int f_len = 0, f_key = 0, f_hi = 0;
    const int32_t* table = nullptr;
    const uint8_t* f_head = nullptr;  // the item's head in page 0
    const uint32_t page_bytes = static_cast<uint32_t>(p.kv.Hkv) * static_cast<uint32_t>(p.kv.lay.block);  // (at most 2^26)
    const uint32_t pages = static_cast<uint32_t>(min(p.kv.num_pages, static_cast<int64_t>(INT32_MAX)));
    // pages of this warp's keys in the block to fetch and the two after it (-1
    // past the item's keys), looked up ahead of their use
    int p1 = -1, p2 = -1, p3 = -1;
    auto page_at = [&](int k) { return k < f_hi ? __ldg(table + (k >> p.kv.lay.page_shift)) : -1; };
    auto page_of = [&](int page) { return f_head + static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_bytes; };
    auto fetch = [&](Raw& r, int* key_out, int* len_out) {
      if (f_left == 0) {
        wb.seek(nu);
        f_left = static_cast<int>(min(min(wb.it.start + wb.it.units, u1) - nu, static_cast<int64_t>(INT32_MAX)));
        f_len = static_cast<int>(wb.it.s.len);
        f_key = wb.it.lo + static_cast<int>(nu - wb.it.start) * kKeys;
        f_hi = min(f_len, wb.it.lo + wb.it.units * kKeys);
        f_head = p.kv.pool + wb.it.h * p.kv.lay.block;
        table = p.kv.page_table + wb.it.b * p.kv.max_pages;
        p1 = page_at(f_key + 16 * cw);
        p2 = page_at(f_key + 16 * cw + kKeys);
        p3 = page_at(f_key + 16 * cw + 2 * kKeys);
      }
      const int k0 = f_key + 16 * cw;
      const bool have = k0 < f_hi;
      if (have && static_cast<uint32_t>(p1) >= pages) {  // recorded; page 0 stands in
        if (lane == 0) atomicMax(p.kv.err, kErrBounds);
        p1 = 0;
      }
      load(r, page_of(have ? p1 : 0), k0 & (p.kv.lay.page() - 1), have);
      // two blocks on, into L2
      if (static_cast<uint32_t>(p3) < pages) {
        const uint8_t* b2 = page_of(p3);
        const int in_page = (k0 + 2 * kKeys) & (p.kv.lay.page() - 1);
        constexpr int kLines = 16 * (D / 2) / 128;  // lines of 16 keys' codes
        if (lane < 2 * kLines) {
          const uint8_t* l = b2 + in_page * (D / 2) + (lane < kLines ? 0 : p.kv.lay.v_codes()) + (lane % kLines) * 128;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(l));
        } else if (lane < 2 * kLines + 2) {
          const uint8_t* l = b2 + (lane == 2 * kLines ? p.kv.lay.k_scales() : p.kv.lay.v_scales()) + in_page * 2 * G;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(l));
        }
      }
      p1 = p2;
      p2 = p3;
      p3 = page_at(k0 + 3 * kKeys);
      *key_out = f_key;
      *len_out = f_len;
      f_key += kKeys;
      ++nu;
      --f_left;
    };

    Raw next;
    int next_key = 0, next_len = 0;
    if (u0 < u1) fetch(next, &next_key, &next_len);
    // a block's keys go ahead of the values of the block before it: those wait
    // for a weighted sum, these only for scores
    uint32_t values[8];
    for (int64_t i = 0; i <= u1 - u0; ++i) {
      const Raw cur = next;
      if (i < u1 - u0) {
      const int slot = static_cast<int>(i & 1);
      const uint32_t parity = static_cast<uint32_t>((i >> 1) & 1);
      float* fac = reinterpret_cast<float*>(smem + S::kOffFac) + (i % kFacRing) * 2 * kKeys;
      // the block after this one is fetched while this one is worked on
      const int key = next_key, klen = next_len;
      if (i + 1 < u1 - u0) fetch(next, &next_key, &next_len);
      // ---- scales.  A code (three significant bits) times a bf16 scale
      // (eight) is exact in fp16's eleven, so operands are scaled codes; what
      // fp16's range needs is a power of two, one for the sixteen keys (and one
      // for their values) while their scales lie within 2^12 of one another,
      // else one a key.
      __half* rat = reinterpret_cast<__half*>(smem + S::kOffRat) + (slot * kCodeWarps + cw) * 2 * 16 * G;
      {
        const int r = lane & 15;
        const bool in = key + 16 * cw + r < klen;
        float s[G], top = 0.f, least = INFINITY;
        bool good = true;
#pragma unroll
        for (int q = 0; q < G; ++q) {
          s[q] = __uint_as_float(q & 1 ? cur.sc[q / 2] & 0xFFFF0000u : cur.sc[q / 2] << 16);
          good &= fabsf(s[q]) < INFINITY;
          top = fmaxf(top, fabsf(s[q]));
          if (s[q] != 0.f) least = fminf(least, fabsf(s[q]));
        }
        const bool use = in && good;
        float all = use ? top : 0.f, low = use ? least : INFINITY;  // of the sixteen keys or values
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
          all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, d));
          low = fminf(low, __shfl_xor_sync(0xffffffffu, low, d));
        }
        const bool near_ = low * 0x1p12f >= all;
        const float common = all == 0.f ? 1.f : pow2_floor(all);
        const float f = near_ || top == 0.f ? common : pow2_floor(top);
        const float inv = use ? pow2_inverse(f) : 0.f;
        // keys by row, then group; values by group, then key
#pragma unroll
        for (int q = 0; q < G; ++q)
          rat[lane < 16 ? r * G + q : 16 * G + q * 16 + r] = __float2half_rn(use ? s[q] * inv : 0.f);
        // a scale that is not a number makes the whole key one, by its factor
        const float own = !in ? 0.f : good ? f : __uint_as_float(0x7FC00000u);
        const bool even = __all_sync(0xffffffffu, near_ && (good || !in));
        if (!warp_wait(&k_empty[slot], parity ^ 1)) break;
        fac[(lane < 16 ? 0 : kKeys) + 16 * cw + r] = lane < 16 ? own * p.scale_log2 : own;
        const float log2_common = static_cast<float>(__float_as_uint(common) >> 23) - 127.f;
        float* gr = reinterpret_cast<float*>(smem + S::kOffGran) + ((i % kFacRing) * 8 + cw) * 4;
        if (lane == 0) {
          gr[0] = common * p.scale_log2;
          reinterpret_cast<int*>(smem + S::kOffEven)[(i % kFacRing) * 8 + cw] = even;
        }
        if (lane == 16) {
          gr[1] = log2_common;
          gr[2] = pow2_inverse(common);
        }
        __syncwarp();
      }
      // ---- keys
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int kk = 8 * x + kr;              // of the warp's 16
        const int row = 16 * cw + kk;
        const uint32_t base = sb + S::kOffK + slot * S::kBlock + row * 128;
        uint32_t ratio[G];
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const uint32_t h = *reinterpret_cast<const uint16_t*>(rat + kk * G + q);
          ratio[q] = h | (h << 16);
        }
#pragma unroll
        for (int w = 0; w < kKW; ++w) {
          const uint32_t a = cur.k[x][w], b = a >> 8;
          uint32_t c0 = kv4split::codes_low(a), c1 = kv4split::codes_high(a), c2 = kv4split::codes_low(b), c3 = kv4split::codes_high(b);
          const uint32_t r = ratio[w / (kKW / G)];
          c0 = half2_mul(c0, r);
          c1 = half2_mul(c1, r);
          c2 = half2_mul(c2, r);
          c3 = half2_mul(c3, r);
          const int ch = 4 * w + t4;            // 16-byte chunk of the row
          st_shared_v4(base + (ch >> 3) * (kKeys * 128) + (((ch & 7) ^ (row & 7)) << 4), c0, c1, c2, c3);
        }
      }
      fence_proxy_async_smem();
      warp_arrive(&k_full[slot]);
      }
      // ---- values, transposed: eight keys of a dimension are one chunk
      if (i > 0) {
        const int slot = static_cast<int>((i - 1) & 1);
        if (!warp_wait(&v_empty[slot], static_cast<uint32_t>(((i - 1) >> 1) & 1) ^ 1)) break;
        const __half* rat = reinterpret_cast<const __half*>(smem + S::kOffRat) + (slot * kCodeWarps + cw) * 2 * 16 * G;
        uint32_t out[8][4];  // [nibble][key pair]
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t lo = __byte_perm(values[2 * y], values[2 * y + 1], 0x5410);
          const uint32_t hi = __byte_perm(values[2 * y], values[2 * y + 1], 0x7632);
          out[0][y] = kv4split::codes_low(lo);
          out[1][y] = kv4split::codes_high(lo);
          out[2][y] = kv4split::codes_low(lo >> 8);
          out[3][y] = kv4split::codes_high(lo >> 8);
          out[4][y] = kv4split::codes_low(hi);
          out[5][y] = kv4split::codes_high(hi);
          out[6][y] = kv4split::codes_low(hi >> 8);
          out[7][y] = kv4split::codes_high(hi >> 8);
        }
        const int chunk = 2 * cw + oct;         // 8-key chunk of the block, 0..15
        const uint32_t base = sb + S::kOffV + slot * S::kBlock + (chunk >> 3) * (D * 128);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int d = (D == 128 ? 64 * vsel : 0) + 8 * n + vg;
          // dimensions 64 j + 8 n: the group is that over the group's size
          const int q = (D == 128 ? 64 * vsel + 8 * n : 8 * n) * G / D;
          const uint4 r = *reinterpret_cast<const uint4*>(rat + 16 * G + q * 16 + 8 * oct);
          out[n][0] = half2_mul(out[n][0], r.x);
          out[n][1] = half2_mul(out[n][1], r.y);
          out[n][2] = half2_mul(out[n][2], r.z);
          out[n][3] = half2_mul(out[n][3], r.w);
          if (D == 128 || vsel == (n >> 2))     // D = 64: a lane stores half of its word
            st_shared_v4(base + d * 128 + (((chunk & 7) ^ (d & 7)) << 4), out[n][0], out[n][1], out[n][2], out[n][3]);
        }
        fence_proxy_async_smem();
        warp_arrive(&v_full[slot]);
      }
#pragma unroll
      for (int y = 0; y < 8; ++y) values[y] = cur.v[y];
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int G, int NT>
cudaError_t launch_variant(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};  // devices whose shared-memory limit is set
  const uint64_t bit = 1ull << (a.device & 63);
  constexpr int bytes = Smem<D, G, NT>::kBytes;
  static_assert(bytes + 6144 <= 232448, "shared memory of one CTA, the static part with it");
  if (!(done.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kv4_tile_kernel<D, G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
  }
  TileParams p;
  p.a = kv4split::make_params(a, x);
  p.diag.err = a.diag.err;
  p.diag.wait_limit_ns = a.diag.wait_limit_ns;
  p.diag.force_timeout = a.diag.force_timeout;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = a.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kv4_tile_kernel<D, G, NT>, p);
}

}  // namespace kv4tile
}  // namespace wq
