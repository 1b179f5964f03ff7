// wq_kv4_tile_d64.cu -- the many-row attention over the 4-bit cache, heads of 64.
#include "wq_kv4_tile.cuh"

namespace wq {

cudaError_t launch_kv4_tile_d64(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  using namespace kv4tile;
  const int G = a.D / a.group;
  // One tile of 128 rows where no sequence has more, else two.  (Measured for
  // heads of 128, in wq_kv4_tile_d128.cu.)
  const bool one = a.max_q * (x.Hq / a.Hkv) <= 128;
  if (G == 1) return one ? launch_variant<64, 1, 1>(a, x, stream) : launch_variant<64, 1, 2>(a, x, stream);
  if (G == 2) return one ? launch_variant<64, 2, 1>(a, x, stream) : launch_variant<64, 2, 2>(a, x, stream);
  return cudaErrorNotSupported;
}

}  // namespace wq
