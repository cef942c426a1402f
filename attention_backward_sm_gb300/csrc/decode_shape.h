// What a decode call launches, from its sizes: the shape of the tiles, the
// number of blocks, what they leave in the workspace.  Host code and constants
// without CUDA, so that the choices can be checked without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <type_traits>

namespace fa {
namespace decode {

constexpr int kMaxSms = 152;   // of a GB300; a launch's blocks are at most what it holds
// Tiles per block from which on runs are cut by cost (Runs in decode.cuh).
constexpr int kManyTiles = 4;

// A call's sizes.
struct Call {
  int batch;
  int heads;
  int heads_kv;
  int head_dim;
  bool e4m3;
  int keys;      // max_pages * page_size
  int window;
  int sms;       // of the device
};

// NH: groups of 8 query heads per key/value head; HW: key/value heads per tile.
template <int D, bool E4M3, int NH, int HW>
struct Shape {
  static constexpr int kElem = E4M3 ? 1 : 2;
  static constexpr int kRowBytes = D * kElem;
  static constexpr int kRowsPerTile =   // heads x keys
      E4M3 && (D == 64 || (D == 256 && NH > 1)) ? 128 : 64;
  static constexpr int kTile = kRowsPerTile / HW;                    // keys
  static constexpr int kHeadBytes = kTile * kRowBytes;
  static constexpr int kTileBytes = kRowsPerTile * kRowBytes;        // of K, and of V
  static constexpr int kStageBytes = 2 * kTileBytes;
  // Blocks per SM: what shared memory (the ring of stages) and registers
  // (fragments of O and Q) leave room for.
  static constexpr int kBlocksPerSm = kStageBytes >= 65536 || (kStageBytes >= 32768 && NH > 2) ? 1
                                      : kStageBytes >= 32768 || NH > 2                         ? 2
                                      : NH > 1 || E4M3                                         ? 3
                                                                                               : 4;
  static constexpr int kStages = kStageBytes < 65536 && kBlocksPerSm == 1 ? 5 : 3;
  static constexpr int kRowWarps = kStageBytes >= 65536 && E4M3 ? 8 : 4;   // warps over a tile's rows
  static constexpr int kKeyWarps = kRowWarps / HW;
  static constexpr int kKeys = kTile / kKeyWarps;                          // of a warp
  // Warps over the same rows, each with a part of O's columns (and all of the
  // scores), where 4 warps would be all that an SM runs.
  static constexpr int kSplit = kRowWarps == 4 && kBlocksPerSm == 1 ? 2 : 1;
  // Weights of the second product as two 16-bit numbers.  Beside e4m3 values
  // only for up to 8 heads of up to 128: 128 requests of 1k to 16k keys, 32 / 8
  // heads of 128, 229 -> 231 us and the error of o 1.681e-3 -> 1.669e-3 (that of
  // its rounding); but 32 requests of 8192 keys, 8 key/value heads: 16 query heads
  // each of 128, 105 -> 118; 32 of 64, 98 -> 132; 8 of 256, 92 -> 101.
  static constexpr bool kTwoParts = !E4M3 || (NH == 1 && D <= 128);
  static constexpr int kThreads = kRowWarps * kSplit * 32;
  static constexpr int kHeads = 8 * NH;
  static constexpr int kOffsets = kStages + 1;               // tiles whose row offsets are kept
  // Key warps' O are joined in the stage just consumed, so many heads at a time.
  static constexpr int kJoinFit = kStageBytes / (kRowWarps * D * 4) / 8 * 8;
  static constexpr int kJoinHeads = kJoinFit < kHeads ? kJoinFit : kHeads;
  static constexpr int kSeenWords = (kTile + 31) / 32;
  static constexpr int kOffOffsets = kStages * kStageBytes;
  static constexpr int kOffSeen = kOffOffsets + kOffsets * kTile * 8;
  static constexpr int kOffJoin = kOffSeen + kOffsets * kSeenWords * 4;
  static constexpr int kOffScan = kOffJoin + (kKeyWarps > 1 ? 2 * kRowWarps * kHeads * 4 : 0);
  static constexpr int kOffZero = (kOffScan + kThreads / 32 * 4 + 44 + 15) / 16 * 16;   // 16 zero bytes
  static constexpr int kOffQ = kOffZero + 16;   // query rows of kStages units
  static_assert(kJoinHeads >= 8, "join buffer");
  static_assert(kTile == 16 || kTile == 32 || kTile == 64 || kTile == 128, "tile_shift");
  static_assert(kKeys == 16 || kKeys == 32, "a word of seen keys");
  static_assert(kTile <= kThreads && kTile % 16 == 0, "a thread per key looks up its page");
  static constexpr int smem(int rows) { return kOffQ + kStages * HW * rows * D * 2; }
  static constexpr bool fits(int rows) {
    return smem(rows) <= 227 * 1024 && kBlocksPerSm * (smem(rows) + 1024) <= 228 * 1024;
  }
  static_assert(HW > 1 || fits(kHeads), "shared memory");
};

// A unit that the end of a run cuts, entered by the run it starts in: runs
// [this one, last] hold its partial results, this one's in slot `slot`, the
// others' in slot 0.  (With at most half as many units as blocks, by_unit, the
// combine kernel has a block per unit, which works this out from the lengths
// instead.)
struct Cut {
  int unit;    // b * (heads_kv / HW) + head group, or -1: none
  int last;
  int slot;
  int pad;
};

struct Launch {
  int rows;        // query heads of a key/value head per chunk (at most 8 NH)
  int chunks;      // chunks of the G query heads of a key/value head
  int group;       // key/value heads per tile
  int blocks;      // blocks per chunk
  int tile_shift;  // log2 of the keys per tile
  int by_unit;     // combine goes by units, not by cuts
  int joined;      // a combine kernel follows (host only, like the next)
  int device;
};

#ifdef __CUDACC__
__host__ __device__
#endif
inline size_t part_floats(int rows, int d) {
  return (static_cast<size_t>(rows) * (d + 2) + 3) / 4 * 4;   // 16-byte aligned
}

// The G query heads of a key/value head in chunks, as equal as can be, each of
// which reads the keys (the second and later ones mostly from the L2).  A chunk
// holds at most what the registers hold: 32 heads at head_dim 64, 24 (e4m3)
// or 16 at 128, 16 at 256.  32 requests of 8192 keys, 8 key/value heads, one
// chunk against two: d = 64, 256 query heads, bf16 129 and 161 us, e4m3 97 and
// 110; d = 128, 192 query heads, e4m3 138 and 185, but 256 query heads 310
// and 189 (spilled registers); bf16, 64 requests, 32 heads on one: 34.5 and
// 30.6 (half the warps).
inline Launch split_heads(int heads, int heads_kv, int head_dim, bool e4m3) {
  const int G = heads / heads_kv, most = head_dim == 64 ? 32 : head_dim == 128 && e4m3 ? 24 : 16;
  Launch lc = {};
  lc.chunks = (G + most - 1) / most;
  lc.rows = (G + lc.chunks - 1) / lc.chunks;
  lc.chunks = (G + lc.rows - 1) / lc.rows;
  return lc;
}

// What the longest stretch of keys that a request can see comes to in tiles.
inline long long tiles_of(const Call& c, int tile) {
  const int n = c.window > 0 && c.window < c.keys ? c.window : c.keys;
  return n > tile ? (n + static_cast<long long>(tile) - 1) / tile : 1;
}

// Whether tiles of HW key/value heads are taken: where their queries fit
// beside the ring of stages, and either blocks have enough tiles (12 at least,
// were every request as long as the table allows) for the longer DRAM pieces to
// matter more than the more numerous partial results per unit, or units are
// many and of one or two tiles, so that few are cut and what counts is their
// number.  4 heads against 1, on one GPU: 128 requests of 1k to 16k keys, 32 / 8
// heads, d = 128, e4m3: 221 and 254 us; 189 requests of 2 keys, 16 heads of 64,
// e4m3: 7.4 and 14.6 us.  The table's width decides, the lengths are not known
// here: one request of 1k keys, bf16, 5.4 us with a table of its length, 5.6 with
// one of 8k keys (a head per tile), 5.9 with one of 32k (four).
template <int D, bool E4M3, int NH, int HW>
bool take_group(const Call& c, const Launch& lc) {
  using Sh = Shape<D, E4M3, NH, HW>;
  const long long units = static_cast<long long>(c.batch) * (c.heads_kv / HW), resident = Sh::kBlocksPerSm * c.sms;
  return c.heads_kv % HW == 0 && Sh::fits(lc.rows) &&
         (tiles_of(c, Sh::kTile) * units >= 12 * resident || (units >= resident && tiles_of(c, Sh::kTile) <= 2));
}

// f(NH), as an integral constant, for so many query heads per chunk.
template <int D, bool E4M3, class F>
auto with_rows(int rows, F f) {
  using std::integral_constant;
  if (rows <= 8) return f(integral_constant<int, 1>());
  if constexpr (D == 64)
    if (rows > 24) return f(integral_constant<int, 4>());
  if constexpr (D == 64 || (D == 128 && E4M3))
    if (rows > 16) return f(integral_constant<int, 3>());
  return f(integral_constant<int, 2>());
}

// f(NH, HW), as integral constants, with the shape that a call takes.
template <int D, bool E4M3, class F>
auto with_shape(const Call& c, const Launch& lc, F f) {
  using std::integral_constant;
  return with_rows<D, E4M3>(lc.rows, [&](auto nh) {
    constexpr int NH = decltype(nh)::value;
    if constexpr (NH <= 2) {   // more than 16 query heads on a key/value head: one of those at a time
      if (take_group<D, E4M3, NH, 4>(c, lc)) return f(nh, integral_constant<int, 4>());
      if (take_group<D, E4M3, NH, 2>(c, lc)) return f(nh, integral_constant<int, 2>());
    }
    return f(nh, integral_constant<int, 1>());
  });
}

// The blocks of a chunk that are resident at once, of all chunks together.
template <class Sh>
int resident_blocks(const Launch& lc, int sms) {
  const int blocks = Sh::kBlocksPerSm * (sms < kMaxSms ? sms : kMaxSms) / lc.chunks;
  return blocks > 1 ? blocks : 1;
}

// At most one block per tile, at most the blocks that are resident at once.
template <class Sh, int HW>
void set_blocks(const Call& c, Launch& lc) {
  lc.group = HW;
  const long long unit_tiles = tiles_of(c, Sh::kTile);
  const long long units = static_cast<long long>(c.batch) * (c.heads_kv / HW), tiles = unit_tiles * units;
  const int blocks = resident_blocks<Sh>(lc, c.sms);
  lc.blocks = tiles < blocks ? static_cast<int>(tiles) : blocks;
  lc.by_unit = 2 * units <= lc.blocks;
  lc.tile_shift = Sh::kTile == 16 ? 4 : Sh::kTile == 32 ? 5 : Sh::kTile == 64 ? 6 : 7;
  lc.joined = unit_tiles > 1;   // units of one tile are never cut
}

// Bytes of the workspace of a shape, if calls of these heads can take it.
template <int D, bool E4M3, int NH, int HW>
size_t shape_bytes(const Launch& lc, int heads_kv) {
  using Sh = Shape<D, E4M3, NH, HW>;
  if (heads_kv % HW != 0 || (HW > 1 && !Sh::fits(lc.rows))) return 0;
  const size_t blocks = static_cast<size_t>(resident_blocks<Sh>(lc, kMaxSms)) * lc.chunks;
  return blocks * (sizeof(Cut) + 2 * part_floats(HW * lc.rows, D) * sizeof(float));
}
template <int D, bool E4M3>
size_t cache_bytes(int heads, int heads_kv) {
  const Launch lc = split_heads(heads, heads_kv, D, E4M3);
  return with_rows<D, E4M3>(lc.rows, [&](auto nh) {
    constexpr int NH = decltype(nh)::value;
    size_t most = shape_bytes<D, E4M3, NH, 1>(lc, heads_kv);
    if constexpr (NH <= 2) {
      const size_t two = shape_bytes<D, E4M3, NH, 2>(lc, heads_kv), four = shape_bytes<D, E4M3, NH, 4>(lc, heads_kv);
      most = most > two ? most : two;
      most = most > four ? most : four;
    }
    return most;
  });
}

// Bytes that are enough for any lengths, table and cache of either type.
inline size_t workspace_bytes(int batch, int heads, int heads_kv, int head_dim) {
  if (batch == 0) return 0;
  const size_t a = head_dim == 64    ? cache_bytes<64, false>(heads, heads_kv)
                   : head_dim == 128 ? cache_bytes<128, false>(heads, heads_kv)
                                     : cache_bytes<256, false>(heads, heads_kv);
  const size_t b = head_dim == 64    ? cache_bytes<64, true>(heads, heads_kv)
                   : head_dim == 128 ? cache_bytes<128, true>(heads, heads_kv)
                                     : cache_bytes<256, true>(heads, heads_kv);
  return ((a > b ? a : b) + 255) / 256 * 256;
}

}  // namespace decode
}  // namespace fa
