// How finely fa_extend counts the costs of a call, from its sizes (plain C++).
#pragma once

namespace fa {
namespace extend {

// Units of a call, at most: tiles of rows of a key/value head, of the requests that
// can have any.  Their costs (kUnitMost at most for each, and 3 for every 2^cost_shift
// keys) are summed in 32 bits.
constexpr int kUnitMost = 32;
constexpr long long kMostCost = 1ll << 30;
constexpr long long kMostUnits = kMostCost / kUnitMost;
inline long long most_units(long long num_tokens, long long batch, int heads, int heads_kv, int head_dim) {
  const long long rows = head_dim == 256 ? 128 : 256;
  return (num_tokens * (heads / heads_kv) / rows + (batch < num_tokens ? batch : num_tokens)) * heads_kv;
}

// Keys that cost 1, log 2: a block's (2^block_bits), or as many as keep the sum of the
// costs of any lengths below kMostCost (keys: what the last row of a unit sees, at most).
// For fewer units than kMostUnits, so that there is such a number.
inline int cost_shift(long long units, long long keys, int block_bits) {
  int shift = block_bits;
  while (units >= kMostCost / (3 * (keys >> shift) + kUnitMost)) ++shift;
  return shift;
}

}  // namespace extend
}  // namespace fa
