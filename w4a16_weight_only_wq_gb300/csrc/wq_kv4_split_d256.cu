// wq_kv4_split_d256.cu -- the few-row attention over the 4-bit cache, heads of 256.
#include "wq_kv4_split.cuh"

namespace wq {

cudaError_t launch_kv4_split_d256(const Kv4Args& a, const Kv4AttentionArgs& x, cudaStream_t stream) {
  using namespace kv4split;
  const int G = a.D / a.group;
  // us: 64 sequences of 4096, one token each 158; one of 131071 92; 256 tokens after
  // 16128 950, a window of 1024 of 8192 keys 94 (32 query and 8 key/value heads).
  // Tiles of 8 rows only: 16 rows of 256 dimensions take 128 accumulators a
  // thread, more than fit beside the rest.
  if (G == 2) return launch_variant<256, 2, 1>(a, x, stream);
  if (G == 4) return launch_variant<256, 4, 1>(a, x, stream);
  if (G == 8) return launch_variant<256, 8, 1>(a, x, stream);
  return cudaErrorNotSupported;
}

}  // namespace wq
