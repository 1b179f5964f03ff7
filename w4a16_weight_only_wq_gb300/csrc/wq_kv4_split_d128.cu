// wq_kv4_split_d128.cu -- the few-row attention over the 4-bit cache, heads of 128.
#include "wq_kv4_split.cuh"

namespace wq {

cudaError_t launch_kv4_split_d128(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  using namespace kv4split;
  const int G = a.D / a.group;
  // A tile of 8 rows where no sequence has more, else 16: one tile of 16
  // reads the codes once where two of 8 read them twice.
  const bool small = a.max_q * (x.Hq / a.Hkv) <= 8;
  if (G == 1) return small ? launch_variant<128, 1, 1>(a, x, stream) : launch_variant<128, 1, 2>(a, x, stream);
  if (G == 2) return small ? launch_variant<128, 2, 1>(a, x, stream) : launch_variant<128, 2, 2>(a, x, stream);
  if (G == 4) return small ? launch_variant<128, 4, 1>(a, x, stream) : launch_variant<128, 4, 2>(a, x, stream);
  return cudaErrorNotSupported;
}

size_t kv4_workspace_bytes(int D, int num_sms) {
  using namespace kv4split;
  // partial rows: two slots for each CTA of the few-row kernel (16 rows), or of the many-row kernel (one, 256 rows)
  const size_t few = static_cast<size_t>(2 * kMaxCtasSm) * num_sms * kMaxRows, many = D == 256 ? 0 : static_cast<size_t>(2) * num_sms * 256;
  return kv4_counter_bytes(num_sms) + (few > many ? few : many) * (D + 4) * 4;
}

cudaError_t launch_kv4_attention(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  // More than 16 rows of a head and sequence (64, for heads of 64) go to the many-row
  // kernel, which reads the codes once for up to 256 rows where this one reads them
  // once for 16.  Heads of 128 (32 query and 8 key/value heads), us at 32 / 64 / 128
  // rows, few-row kernel against many-row: 8 sequences of 16384: 223 / 424 / 826
  // against 122 / 126 / 140; 32 of 4096: 217 / 415 / 834 against 138 / 144 / 161; 8 of
  // 1024: 31 / 46 / 65 against 40 / 46 / 55; one of 16384: 46 / 63 / 98 against 46 / 60
  // / 89; 16 rows 119 against 20 rows 125.  (Of a few short sequences the few-row
  // kernel does better up to 64 rows, by 10 us; how long they are is not known here.)
  // Heads of 64, at 32 / 48 / 64 rows: 8 of 16384: 66 / 90 / 113 against 108 / 108 /
  // 108; 32 of 4096: 68 / 93 / 120 against 118 / 118 / 119; 8 of 1024: 21 / 23 / 28
  // against 34 / 34 / 35; one of 16384: 27 / 24 / 31 against 42 / 43 / 43: the many-row
  // kernel's chain for a block hardly shrinks with the dimensions.
  const int64_t rows = a.max_q * (x.Hq / a.Hkv);  // of one head of a sequence, at most
  if (a.D == 64 && rows > 64) return launch_kv4_tile_d64(a, x, stream);
  if (a.D == 128 && rows > 16) return launch_kv4_tile_d128(a, x, stream);
  if (a.D == 64) return launch_kv4_split_d64(a, x, stream);
  if (a.D == 128) return launch_kv4_split_d128(a, x, stream);
  return launch_kv4_split_d256(a, x, stream);
}

}  // namespace wq
