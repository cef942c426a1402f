// Dispatch of single-token attention over the paged cache by head_dim (the
// kernels are in decode.cuh, one translation unit per head_dim; what is
// launched is worked out in decode_shape.h).
#include "decode.cuh"

namespace fa {

cudaError_t launch_decode_d64(const DecodeParams& p, const decode::Call& c, const decode::Launch& lc, cudaStream_t s);
cudaError_t launch_decode_d128(const DecodeParams& p, const decode::Call& c, const decode::Launch& lc, cudaStream_t s);
cudaError_t launch_decode_d256(const DecodeParams& p, const decode::Call& c, const decode::Launch& lc, cudaStream_t s);

size_t decode_workspace_bytes(int batch, int heads, int heads_kv, int head_dim) {
  return decode::workspace_bytes(batch, heads, heads_kv, head_dim);
}

cudaError_t launch_decode(const DecodeParams& p, const Device& dev, cudaStream_t s) {
  decode::Launch lc = decode::split_heads(p.heads, p.kv.heads_kv, p.kv.head_dim, p.kv.e4m3);
  lc.device = dev.id;
  const decode::Call c{p.batch, p.heads, p.kv.heads_kv, p.kv.head_dim, p.kv.e4m3 != 0, p.max_pages * p.kv.page_size,
                       p.window, dev.sms};
  if (p.kv.head_dim == 64) return launch_decode_d64(p, c, lc, s);
  if (p.kv.head_dim == 128) return launch_decode_d128(p, c, lc, s);
  return launch_decode_d256(p, c, lc, s);
}

}  // namespace fa
