// Single-token attention over the paged cache at head_dim 256.
#include "decode.cuh"

namespace fa {
cudaError_t launch_decode_d256(const DecodeParams& p, const decode::Call& c, const decode::Launch& lc, cudaStream_t s) {
  return p.kv.e4m3 ? decode::launch_dim<256, true>(p, c, lc, s) : decode::launch_dim<256, false>(p, c, lc, s);
}
}  // namespace fa
