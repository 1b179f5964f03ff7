// wq_kv4_tile_d64.cu -- the many-row attention over the 4-bit cache, heads of 64.
#include "wq_kv4_tile.cuh"

namespace wq {

cudaError_t launch_kv4_tile_d64(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  using namespace kv4tile;
  const int G = a.D / a.group;
  // One tile of 128 rows where no sequence has more, else two.  (us with one / two
  // tiles, 32 query and 8 key/value heads; 100 rows: 8
  // sequences of 16384: 114 / 135; 32 of 4096: 128 / 141; 8 of 1024: 40 / 35.  256 rows:
  // 200 / 162; 240 / 173; 41 / 46.  A few short sequences go the other way; how long
  // they are is not known here.)
  const bool one = a.max_q * (x.Hq / a.Hkv) <= 128;
  if (G == 1) return one ? launch_variant<64, 1, 1>(a, x, stream) : launch_variant<64, 1, 2>(a, x, stream);
  if (G == 2) return one ? launch_variant<64, 2, 1>(a, x, stream) : launch_variant<64, 2, 2>(a, x, stream);
  return cudaErrorNotSupported;
}

}  // namespace wq
