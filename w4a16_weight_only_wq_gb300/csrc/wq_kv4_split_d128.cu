// wq_kv4_split_d128.cu -- the few-row attention over the 4-bit cache, heads of 128.
#include "wq_kv4_split.cuh"

namespace wq {

cudaError_t launch_kv4_split_d128(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  using namespace kv4split;
  const int G = a.D / a.group;
  // Tiles of 8 rows only: the accumulators of 16 rows of 128 dimensions do not fit a
  // thread's 128 registers beside the rest.  (16 rows in one tile of 16, spilled,
  // against two of 8, which read the codes twice, us: 64 sequences of 4096 230 / 129; 8
  // of 16384 119 / 72; 8 of 1024 26 / 21; one of 131071 129 / 71.)
  if (G == 1) return launch_variant<128, 1, 1>(a, x, stream);
  if (G == 2) return launch_variant<128, 2, 1>(a, x, stream);
  if (G == 4) return launch_variant<128, 4, 1>(a, x, stream);
  return cudaErrorNotSupported;
}

size_t kv4_workspace_bytes(int D, int num_sms) {
  using namespace kv4split;
  // partial rows: two slots for each CTA of the few-row kernel (16 rows at most), or of the many-row kernel (one, 256 rows)
  const size_t few = static_cast<size_t>(2 * kMaxCtasSm) * num_sms * kMaxRows, many = D == 256 ? 0 : static_cast<size_t>(2) * num_sms * 256;
  return kv4_counter_bytes(num_sms) + (few > many ? few : many) * (D + 4) * 4;
}

cudaError_t launch_kv4_attention(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  // More than 32 rows of a head and sequence (64, for heads of 64) go to the many-row
  // kernel, which reads the codes once for up to 256 rows where this one reads them
  // once for 8 (or 16).  us, few-row kernel / many-row, 32 query and 8 key/value heads:
  //   heads of 128, rows     24           32           40
  //   8 sequences of 16384   99 / 125     123 / 122    150 / 130
  //   64 of 4096             184 / 258    240 / 258    292 / 268
  //   8 of 1024              22 / 39      23 / 39      25 / 43
  //   one of 131071          101 / 139    119 / 128    149 / 162
  //   (group 32: 32 rows 141 / 128, 275 / 270, 25 / 39, 136 / 132)
  //   heads of 64, rows      32           48           64
  //   8 sequences of 16384   66 / 108     90 / 108     113 / 108
  //   32 of 4096             68 / 118     93 / 118     120 / 119
  //   8 of 1024              21 / 34      23 / 34      28 / 35
  //   one of 16384           27 / 42      24 / 43      31 / 43
  // (The many-row kernel's chain for a block hardly shrinks with rows or dimensions.)
  // A few short sequences, or one, do better here with more rows too; how long they
  // are is not known to the host.
  const int64_t rows = a.max_q * (x.Hq / a.Hkv);  // of one head of a sequence, at most
  if (a.D == 64 && rows > 64) return launch_kv4_tile_d64(a, x, stream);
  if (a.D == 128 && rows > 32) return launch_kv4_tile_d128(a, x, stream);
  if (a.D == 64) return launch_kv4_split_d64(a, x, stream);
  if (a.D == 128) return launch_kv4_split_d128(a, x, stream);
  return launch_kv4_split_d256(a, x, stream);
}

}  // namespace wq
