// What a call of fa_extend launches, from its sizes, and its workspace.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "extend_shape.h"
#include "paged.h"

namespace fa {

struct ExtendParams {
  CUtensorMap tm_k;         // with box_rows
  CUtensorMap tm_v;
  CUtensorMap tm_q;         // with q_boxes
  PagedCache kv;
  const uint16_t* q;        // [num_tokens, heads, d], rows q_row_stride elements apart
  long long q_row_stride;
  const int32_t* table;     // [batch, max_pages], rows table_stride entries apart
  long long table_stride;
  const int32_t* seq_lens;
  const int32_t* cu_new;
  uint16_t* o;              // [num_tokens, heads, d]
  float* lse;               // [num_tokens, heads] or nullptr
  void* work;
  FastDiv page_div;         // by kv.page_size
  FastDiv group_div;        // by heads / heads_kv
  int max_pages;
  int batch;
  int num_tokens;
  int heads;
  int window;
  float scale;
  // set by launch_extend, like the tensor maps:
  int box_rows;             // keys of a TMA box, 0: none
  int q_boxes;
  int cost_shift;           // keys that cost 1, log 2
  int tile_keys16;          // rows of a tile / group, in 16ths
  int tile_tokens;          // tokens that a tile's rows belong to, at most
};

namespace extend {

constexpr int kMaxSms = 152;

template <int D>
struct Shape {
  static constexpr int kTiles = D == 256 ? 1 : 2;        // of 128 query rows
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kKeys = D == 256 ? 64 : 128;      // of a block
};

// A unit whose first blocks a run ends with: the rows' place and the last run
// that has a piece of it.  Runs (this, last] hold theirs in slot 0, this one in
// slot 1.
struct Cut {
  int row_end;    // rows of the request (tokens * group), 0: nothing is cut
  int row_first;  // first row of the unit
  int token0;     // row of q and o of the request's first token
  int head_kv;
  int last;
  int pad[3];
};

// Partial results: [runs][2 slots] of [d / 4][rows] four values each, then
// [rows] references and [rows] sums.
inline __host__ __device__ size_t part_floats(int rows, int d) { return static_cast<size_t>(rows) * (d + 2); }

inline size_t workspace_bytes(int head_dim) {
  const int rows = head_dim == 256 ? 128 : 256;
  return kMaxSms * (sizeof(Cut) + 2 * part_floats(rows, head_dim) * sizeof(float));
}

}  // namespace extend

cudaError_t launch_extend(const ExtendParams& p, const Device& dev, cudaStream_t s);
int extend_read_and_clear_status(cudaStream_t s, int* status);
cudaError_t extend_status_word(int** word);

}  // namespace fa
