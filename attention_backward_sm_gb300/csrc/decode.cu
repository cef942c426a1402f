// Dispatch of single-token attention over the paged cache by head_dim, and its
// workspace (the kernels are in decode.cuh, one translation unit per head_dim).
#include "decode.cuh"

namespace fa {

cudaError_t launch_decode_d64(const DecodeParams& p, const decode::Launch& lc, cudaStream_t s);
cudaError_t launch_decode_d128(const DecodeParams& p, const decode::Launch& lc, cudaStream_t s);
cudaError_t launch_decode_d256(const DecodeParams& p, const decode::Launch& lc, cudaStream_t s);

namespace {

// The G query heads of a key/value head in chunks, as equal as can be, each of
// which reads the keys (the second and later ones mostly from the L2).  A chunk
// holds at most what the registers hold: 32 heads at head_dim 64, 24 (e4m3)
// or 16 at 128, 16 at 256.  32 requests of 8192 keys, 8 key/value heads, one
// chunk against two: d = 64, 256 query heads, bf16 129 and 161 us, e4m3 97 and
// 110; d = 128, 192 query heads, e4m3 138 and 185, but 256 query heads 310
// and 189 (spilled registers); bf16, 64 requests, 32 heads on one: 34.5 and
// 30.6 (half the warps).
decode::Launch split_heads(int heads, int heads_kv, int head_dim, bool e4m3) {
  const int G = heads / heads_kv, most = head_dim == 64 ? 32 : head_dim == 128 && e4m3 ? 24 : 16;
  decode::Launch lc;
  lc.chunks = (G + most - 1) / most;
  lc.rows = (G + lc.chunks - 1) / lc.chunks;
  lc.chunks = (G + lc.rows - 1) / lc.rows;
  lc.group = 1;
  lc.blocks = 0;
  lc.tile_shift = 0;
  lc.by_unit = 0;
  lc.sms = 0;
  lc.device = 0;
  return lc;
}

size_t workspace_bytes(const decode::Launch& lc, int heads_kv, int head_dim) {
  const int group = lc.rows > 16 ? 1 : heads_kv % 4 == 0 ? 4 : heads_kv % 2 == 0 ? 2 : 1;
  const size_t blocks = lc.chunks > decode::kMaxBlocks ? lc.chunks : decode::kMaxBlocks;
  return blocks * (sizeof(decode::Cut) + 2 * decode::part_floats(group * lc.rows, head_dim) * sizeof(float));
}

}  // namespace

size_t decode_workspace_bytes(int batch, int heads, int heads_kv, int head_dim) {
  if (batch == 0) return 0;
  const size_t a = workspace_bytes(split_heads(heads, heads_kv, head_dim, false), heads_kv, head_dim);
  const size_t b = workspace_bytes(split_heads(heads, heads_kv, head_dim, true), heads_kv, head_dim);
  return ((a > b ? a : b) + 255) / 256 * 256;
}

cudaError_t launch_decode(const DecodeParams& p, cudaStream_t s) {
  decode::Launch lc = split_heads(p.heads, p.kv.heads_kv, p.kv.head_dim, p.kv.e4m3);
  static std::atomic<int> sms[64];   // of each device, once asked
  cudaError_t e = cudaGetDevice(&lc.device);
  if (e != cudaSuccess) return e;
  const bool listed = lc.device >= 0 && lc.device < 64;
  lc.sms = listed ? sms[lc.device].load(std::memory_order_relaxed) : 0;
  if (lc.sms == 0) {
    e = cudaDeviceGetAttribute(&lc.sms, cudaDevAttrMultiProcessorCount, lc.device);
    if (e != cudaSuccess) return e;
    if (listed) sms[lc.device].store(lc.sms, std::memory_order_relaxed);
  }
  if (p.kv.head_dim == 64) return launch_decode_d64(p, lc, s);
  if (p.kv.head_dim == 128) return launch_decode_d128(p, lc, s);
  return launch_decode_d256(p, lc, s);
}

}  // namespace fa
