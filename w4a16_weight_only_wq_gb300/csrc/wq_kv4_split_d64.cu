// wq_kv4_split_d64.cu -- the few-row attention over the 4-bit cache, heads of 64.
#include "wq_kv4_split.cuh"

namespace wq {

cudaError_t launch_kv4_split_d64(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  using namespace kv4split;
  const int G = a.D / a.group;
  // A tile of 8 rows where no sequence has more, else 16: one tile of 16 reads the
  // codes once where two of 8 read them twice.  (us with tiles of 8 / 16: 8 rows, 64
  // sequences of 4096 54 / 67, 8 of 16384 32 / 38; 16 rows 92 / 72 and 50 / 41, one of
  // 131071 48 / 44.)
  const bool small = a.max_q * (x.Hq / a.Hkv) <= 8;
  if (G == 1) return small ? launch_variant<64, 1, 1>(a, x, stream) : launch_variant<64, 1, 2>(a, x, stream);
  if (G == 2) return small ? launch_variant<64, 2, 1>(a, x, stream) : launch_variant<64, 2, 2>(a, x, stream);
  return cudaErrorNotSupported;
}

}  // namespace wq
