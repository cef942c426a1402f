// Dispatch of single-token attention over the paged cache by head_dim, and its
// workspace (the kernels are in decode.cuh, one translation unit per head_dim).
#include "decode.cuh"

namespace fa {

cudaError_t launch_decode_d64(const DecodeParams& p, const decode::Launch& lc, cudaStream_t s);
cudaError_t launch_decode_d128(const DecodeParams& p, const decode::Launch& lc, cudaStream_t s);
cudaError_t launch_decode_d256(const DecodeParams& p, const decode::Launch& lc, cudaStream_t s);

namespace {

// The G query heads of a key/value head in chunks of at most 8 * max NH heads
// (the registers allow 32, at head_dim 256 16), as equal as can be.
decode::Launch split_heads(int heads, int heads_kv, int head_dim) {
  const int G = heads / heads_kv, most = head_dim == 256 ? 16 : 32;
  decode::Launch lc;
  lc.chunks = (G + most - 1) / most;
  lc.rows = (G + lc.chunks - 1) / lc.chunks;
  lc.chunks = (G + lc.rows - 1) / lc.rows;
  lc.group = 1;
  lc.blocks = 0;
  return lc;
}

}  // namespace

size_t decode_workspace_bytes(int batch, int heads, int heads_kv, int head_dim) {
  if (batch == 0) return 0;
  const decode::Launch lc = split_heads(heads, heads_kv, head_dim);
  const int group = lc.rows > 16 ? 1 : heads_kv % 4 == 0 ? 4 : heads_kv % 2 == 0 ? 2 : 1;
  const size_t blocks = lc.chunks > decode::kMaxBlocks ? lc.chunks : decode::kMaxBlocks;
  const size_t bytes =
      blocks * (sizeof(decode::Cut) + 2 * decode::part_floats(group * lc.rows, head_dim) * sizeof(float));
  return (bytes + 255) / 256 * 256;
}

cudaError_t launch_decode(const DecodeParams& p, cudaStream_t s) {
  const decode::Launch lc = split_heads(p.heads, p.kv.heads_kv, p.kv.head_dim);
  if (p.kv.head_dim == 64) return launch_decode_d64(p, lc, s);
  if (p.kv.head_dim == 128) return launch_decode_d128(p, lc, s);
  return launch_decode_d256(p, lc, s);
}

}  // namespace fa
