// Single-token attention over the paged cache at head_dim 128.
#include "decode.cuh"

namespace fa {
cudaError_t launch_decode_d128(const DecodeParams& p, const decode::Call& c, const decode::Launch& lc, cudaStream_t s) {
  return p.kv.e4m3 ? decode::launch_dim<128, true>(p, c, lc, s) : decode::launch_dim<128, false>(p, c, lc, s);
}
}  // namespace fa
