// Single-token attention over the paged cache at head_dim 128.
#include "decode.cuh"

namespace fa {
cudaError_t launch_decode_d128(const DecodeParams& p, const decode::Launch& lc, cudaStream_t s) {
  return p.kv.e4m3 ? decode::launch_rows<128, true>(p, lc, s) : decode::launch_rows<128, false>(p, lc, s);
}
}  // namespace fa
