// wq_kv4_tile_d128.cu -- the many-row attention over the 4-bit cache, heads of 128.
#include "wq_kv4_tile.cuh"

namespace wq {

cudaError_t launch_kv4_tile_d128(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  using namespace kv4tile;
  const int G = a.D / a.group;
  // One tile of 128 rows where no sequence has more, else two. (Two tiles, the
  // second empty, at 64 rows of 128: 8 sequences of 16384 take 204 us instead of 140,
  // 32 of 4096 216 instead of 157; one tile at 256 rows: 256 us instead of 203, 318
  // instead of 217; all before the joins took 16 dimensions a task, which saved 10%.)
  const bool one = a.max_q * (x.Hq / a.Hkv) <= 128;
  if (G == 1) return one ? launch_variant<128, 1, 1>(a, x, stream) : launch_variant<128, 1, 2>(a, x, stream);
  if (G == 2) return one ? launch_variant<128, 2, 1>(a, x, stream) : launch_variant<128, 2, 2>(a, x, stream);
  if (G == 4) return one ? launch_variant<128, 4, 1>(a, x, stream) : launch_variant<128, 4, 2>(a, x, stream);
  return cudaErrorNotSupported;
}

}  // namespace wq
