// wq_kv4_tile_d128.cu -- the many-row attention over the 4-bit cache, heads of 128.
#include "wq_kv4_tile.cuh"

namespace wq {

cudaError_t launch_kv4_tile_d128(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  using namespace kv4tile;
  const int G = a.D / a.group;
  // One tile of 128 rows where no sequence has more, else two.  (us with one / two
  // tiles, 32 query and 8 key/value heads; 64 rows: 8 sequences of 16384: 126 / 151; 32
  // of 4096: 144 / 160; 8 of 1024: 46 / 39.  256 rows: 230 / 188; 301 / 204; 53 / 56.  A
  // few short sequences go the other way; how long they are is not known here.)
  const bool one = a.max_q * (x.Hq / a.Hkv) <= 128;
  if (G == 1) return one ? launch_variant<128, 1, 1>(a, x, stream) : launch_variant<128, 1, 2>(a, x, stream);
  if (G == 2) return one ? launch_variant<128, 2, 1>(a, x, stream) : launch_variant<128, 2, 2>(a, x, stream);
  if (G == 4) return one ? launch_variant<128, 4, 1>(a, x, stream) : launch_variant<128, 4, 2>(a, x, stream);
  return cudaErrorNotSupported;
}

}  // namespace wq
