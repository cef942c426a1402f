// Attention of one new token per request over a paged key/value cache.
//
// For request b, query head h (key/value head h / G, G = heads / heads_kv)
// and the visible cached keys j in [max(0, len - window), len):
//     x_j = scale * q . k_j,  o = sum_j exp(x_j) v_j / sum_j exp(x_j),
//     lse = ln sum_j exp(x_j)
// Keys whose block-table entry is not a page of the cache are not seen; a
// row that sees no key gets o = 0, lse = -inf.
//
// The call has to read every visible key and value once and does 2 G
// operations per cached bf16 byte: it is bound by HBM.  So
//   * the G query heads of a key/value head share one pass over its keys.  They
//     are the columns of 16 x 8 tensor-core products S^T = K Q^T, O^T += V^T P^T
//     (keys and dimensions in the rows, so that few heads waste little), which
//     keeps the arithmetic far below the time of the loads;
//   * a tile is some keys of HW neighbouring key/value heads (4, 2 or 1), a
//     warp per head.  In the packed layout a slot's heads lie side by side, and
//     read together they are long pieces of DRAM rows (e4m3, d = 64: 256 bytes
//     instead of 64); the heads also share the work of finding the rows.  With
//     fewer heads than warps the warps share the keys and are joined where a
//     unit ends;
//   * the tiles of all (request, head group) units, in order, are cut into
//     runs of equal cost, one per resident block.  Ragged lengths, one long request
//     and many short ones all load every SM alike, and a unit that lies in
//     several runs leaves at most one partial result per run, which
//     combine_kernel joins (fixed order: same bits on every call).  The host
//     needs no lengths.
//   * K and V rows come through cp.async into a ring of kStages tiles (any
//     page size and strides; a TMA box would tie the tile to the page), the
//     block-table entries one tile further ahead.
// Each warp keeps a running reference and sum for its keys.
//
// Measured (GPU time, bytes that have to be read over it): 64 requests of 256
// to 8192 keys, 32 / 8 heads of 128, bf16: 96 us, 6.3 TB/s; 4 of 65536 to
// 131072: 222 us, 7.0 TB/s (of a copy's 6.7); 128 of 1024 to 16384, e4m3: 231
// us, 6.3 TB/s; one of 1024: 5.4 us, of which 0.6 are its bytes: two launches,
// the lengths, the table, the keys and the partial results are read one after
// the other.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "decode_shape.h"
#include "internal.h"
#include "paged.h"
#include "sm103.cuh"

namespace fa {
namespace decode {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A warp's reference for the exponents moves only when a score exceeds it by
// more than kSlack (units of log 2): weights are at most 2^kSlack, and the
// maximum over the warp is taken a few times per unit instead of every tile.
constexpr float kSlack = 8.f;

// Workspace: [blocks] cuts, then partial results [blocks][2 slots]: [HW][rows]
// of D sums of p v, then [HW][rows] references and [HW][rows] sums of p.
__device__ __forceinline__ float* parts_of(float* work, size_t blocks) {
  return reinterpret_cast<float*>(reinterpret_cast<Cut*>(work) + blocks);
}

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;   // fewer source bytes than 16: the rest is zero-filled
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// Transposes an 8 x 8 matrix of 16-bit elements held two per lane.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// c += a b, 16 x 8 x 16, fp32 accumulate; operands bf16 or fp16.
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two 8-bit values to two halves (exact), from bits 0-15 or 16-31.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
// Byte offset of 16-byte piece c of row r in a tile whose rows are RB bytes,
// so that eight consecutive rows' pieces c lie in different banks.
template <int RB>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  if constexpr (RB >= 128) return r * RB + ((c ^ (r & 7)) << 4);
  else return r * RB + ((c ^ ((r >> 1) & 3)) << 4);
}

// ------------------------------------------------------------------ partition
struct Lens {
  const int32_t* seq;
  int most;      // max_pages * page_size
  int window;
  __device__ __forceinline__ int len(int b) const { return min(max(*(seq + b), 0), most); }
  __device__ __forceinline__ int first(int len) const { return window > 0 ? max(0, len - window) : 0; }
  // A request without keys has one (empty) tile: its row is written too.
  template <int TILE>
  __device__ __forceinline__ int tiles(int len) const {
    return max(1, (len - first(len) + TILE - 1) / TILE);
  }
  __device__ __forceinline__ int tiles(int len, int tile_shift) const {
    return max(1, (len - first(len) + (1 << tile_shift) - 1) >> tile_shift);
  }
};

// The list of all tiles (requests in order, the head groups of each, the
// tiles of each) cut into `runs` runs of equal cost, one per block; with fewer
// tiles than blocks, as many runs as tiles.  From 4 tiles per block on, a tile costs 2 and the
// end of a unit (warps joined, rows written: 0.5 to 0.7 us beside 1 to 1.3 for
// a tile) 1, and a tile belongs to the run its start lies in; against equal
// numbers of tiles: 37 requests of 1 to 5000 keys, window 1024, 16 heads of
// 64, 14.9 and 15.9 us; 21 of 19 to 674, 128 / 16 heads of 256, 23.3 and 27.4.
// (Such runs are at least 8 long, so none is empty.)  With fewer tiles they
// count alike: whole tiles are all there is to share out
// (64 of 1 to 120, 32 / 8 heads of 128: 7.8 us, by cost 9.2).
struct Runs {
  int tile, end;   // costs
  int runs, base, rem;
  __device__ __forceinline__ Runs(int tiles, int units, int blocks) {
    const bool more = tiles >= kManyTiles * blocks;
    tile = more ? 2 : 1;
    end = more ? 1 : 0;
    const int total = at(tiles, units);
    runs = min(total, blocks);
    base = static_cast<unsigned>(total) / static_cast<unsigned>(runs);
    rem = total - base * runs;
  }
  // Where a tile with so many tiles and units (ended ones) before it starts.
  __device__ __forceinline__ int at(int tiles, int units) const { return tile * tiles + end * units; }
  // The tiles of a unit that start before place x of it.
  __device__ __forceinline__ int tiles_before(int x) const { return (x + end) >> end; }
  __device__ __forceinline__ int start(int c) const { return c * base + min(c, rem); }
  // The run that holds place x.
  __device__ __forceinline__ int of(int x) const {
    const int y = x - rem * (base + 1);
    return y < 0 ? static_cast<unsigned>(x) / static_cast<unsigned>(base + 1)
                 : rem + static_cast<unsigned>(y) / static_cast<unsigned>(base);
  }
};

// Tiles of all requests before those of this thread, of its own (requests
// [b0, b1)) and in all, by a scan over the block.  scan: a word per warp.
template <int TILE, int THREADS>
struct Scan {
  int b0, b1, before, mine, total;
  int len0;   // of request b0
  __device__ __forceinline__ Scan(const Lens& L, int batch, int groups, int* scan) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (batch + THREADS - 1) / THREADS;
    b0 = min(tid * per, batch);
    b1 = min(b0 + per, batch);
    mine = 0;
    len0 = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int len = L.len(b);
      if (b == b0) len0 = len;
      mine += L.tiles<TILE>(len);
    }
    mine *= groups;
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) upto += scan[w];
      total += scan[w];
    }
    before = upto - mine;
  }
  // The threads whose requests hold places x and y write to found[6] the first
  // tile that starts at x or later (request, head group, tile, the request's
  // length, the number of tiles before it) and the number of tiles before y.
  __device__ __forceinline__ void find(const Lens& L, const Runs& runs, int batch, int groups, int x, int y,
                                       int* found) const {
    int at = runs.at(before, b0 * groups), tiles_before = before;
    const int end = runs.at(before + mine, b1 * groups);
    if (x >= end || y < at) return;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int len = b == b0 ? len0 : L.len(b), nt = L.tiles<TILE>(len);
      const unsigned unit = runs.at(nt, 1), span = unit * groups;
      if (static_cast<unsigned>(x - at) < span) {
        int hk = static_cast<unsigned>(x - at) / unit, t = runs.tiles_before(x - at - hk * unit);
        found[4] = tiles_before + hk * nt + t;
        if (t == nt) {   // in the cost of the unit's end
          t = 0;
          ++hk;
        }
        const bool next = hk == groups;
        found[0] = next ? b + 1 : b;
        found[1] = next ? 0 : hk;
        found[2] = t;
        found[3] = next && b + 1 < batch ? L.len(b + 1) : len;
      }
      if (static_cast<unsigned>(y - at) < span) {
        const int hk = static_cast<unsigned>(y - at) / unit;
        found[5] = tiles_before + hk * nt + runs.tiles_before(y - at - hk * unit);
      }
      at += span;
      tiles_before += nt * groups;
    }
  }
};

// A place in the list of tiles: tile t of nt of (request b, head group hk).
template <int TILE>
struct Place {
  int b, hk, t, nt, first, len;
  __device__ __forceinline__ void request(const Lens& L, int length) {
    len = length;
    first = L.first(len);
    nt = L.tiles<TILE>(len);
  }
  __device__ __forceinline__ void next(const Lens& L, int batch, int groups) {
    if (++t < nt) return;
    t = 0;
    if (++hk < groups) return;
    hk = 0;
    if (++b < batch) request(L, L.len(b));
  }
};

// ------------------------------------------------------------------ main kernel
template <int D, bool E4M3, int NH, int HW>
__global__ void __launch_bounds__(Shape<D, E4M3, NH, HW>::kThreads, Shape<D, E4M3, NH, HW>::kBlocksPerSm)
    decode_kernel(const DecodeParams p, const Launch lc) {
  using S = Shape<D, E4M3, NH, HW>;
  constexpr int TILE = S::kTile, RB = S::kRowBytes, ST = S::kStages, kThreads = S::kThreads;
  constexpr int KW = S::kKeyWarps, HEADS = S::kHeads;
  constexpr int KT = S::kKeys / 16;  // a warp's keys, in rows of the products
  constexpr int DO = D / S::kSplit;  // columns of O of a warp
  constexpr float kShift = E4M3 ? 4.f : 0.f;   // of the weights' exponents
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t sbase = smem_u32(smem);
  long long* const offsets = reinterpret_cast<long long*>(smem + S::kOffOffsets);
  uint32_t* const seen = reinterpret_cast<uint32_t*>(smem + S::kOffSeen);
  int* const scan = reinterpret_cast<int*>(smem + S::kOffScan);   // [warps]
  int* const found = scan + kThreads / 32;                        // of the run: Scan::find's, and the end

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the warp's key/value head of a tile, its part of the keys, its first column of O
  const int hw = warp % HW, kwarp = warp / HW % KW, c0 = warp / S::kRowWarps * DO;
  const int G = p.heads / p.kv.heads_kv, groups = p.kv.heads_kv / HW;
  const int row0 = blockIdx.y * lc.rows;                 // first query head of this chunk within its group
  const int rows = min(lc.rows, G - row0);
  const int block = blockIdx.y * lc.blocks + blockIdx.x;
  const Lens L{p.seq_lens, p.max_pages * p.kv.page_size, p.window};

  pdl_wait();
  pdl_launch();
  if (tid == 0) *reinterpret_cast<uint4*>(smem + S::kOffZero) = make_uint4(0, 0, 0, 0);
  const int q_bytes = HW * lc.rows * D * 2;   // of one unit's queries

  // The run of this block: every block counts all tiles, then finds where
  // its share starts.
  const Scan<TILE, kThreads> tiles(L, p.batch, groups, scan);
  const Runs runs(tiles.total, p.batch * groups, lc.blocks);
  int4* const cuts = reinterpret_cast<int4*>(p.work) + blockIdx.y * lc.blocks;
  if (static_cast<int>(blockIdx.x) >= runs.runs) {
    if (tid == 0) cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  // For the end: in registers meanwhile it would take what a combine block
  // needs to be set up beside this one (16 requests of 128 keys: 6.4 -> 8.2 us).
  Runs* const runs_kept = reinterpret_cast<Runs*>(found + 6);
  if (tid == 0) {
    *runs_kept = runs;
    if (static_cast<int>(blockIdx.x) + 1 == runs.runs) found[5] = tiles.total;
  }
  tiles.find(L, runs, p.batch, groups, runs.start(blockIdx.x), runs.start(blockIdx.x + 1), found);
  __syncthreads();
  const int start = found[4], n = found[5] - start;   // tiles before this run's, and its own
  Place<TILE> here;   // the tile being computed
  here.b = found[0];
  here.hk = found[1];
  here.t = found[2];
  here.request(L, found[3]);
  Place<TILE> ahead = here;   // the next tile to load

  // Page of this thread's key of a tile, and from it the row's offset (bytes,
  // without the head's; top bit: not seen) and the tile's bits of seen keys.
  auto look_up = [&](const Place<TILE>& at) -> int {
    const int key = at.first + at.t * TILE + tid;
    if (tid >= TILE || key >= at.len) return -1;
    return *(p.table + at.b * p.table_stride + p.page_div.quotient(key));
  };
  auto store_offset = [&](const Place<TILE>& at, int page, int ring) {
    if (tid >= TILE) return;
    const int key = at.first + at.t * TILE + tid;
    const bool ok = key < at.len && page >= 0 && page < p.kv.num_pages;
    const int slot = key - p.page_div.quotient(key) * p.kv.page_size;
    offsets[ring * TILE + tid] =
        ok ? (page * p.kv.page_stride + slot * p.kv.slot_stride) * S::kElem : static_cast<long long>(1ull << 63);
    const uint32_t bits = __ballot_sync(TILE < 32 ? (1u << (TILE & 31)) - 1u : 0xffffffffu, ok);
    if (lane == 0) seen[ring * S::kSeenWords + warp] = bits;
  };
  // 16-byte pieces of a key's row of a tile (all heads), keys per pass
  constexpr int CPR = RB / 16, PIECES = HW * CPR, KPP = kThreads / PIECES;
  const int piece_head = tid % PIECES / CPR, piece = tid % CPR, key_in_pass = tid / PIECES;
  auto load_tile = [&](const Place<TILE>& at, int ring, int stage, int q_slot, bool with_q) {
    const long long head = (at.hk * HW + piece_head) * p.kv.head_stride * S::kElem + piece * 16;
    const unsigned char* const kb = static_cast<const unsigned char*>(p.kv.k) + head;
    const unsigned char* const vb = static_cast<const unsigned char*>(p.kv.v) + head;
    const uint32_t dst = sbase + stage * S::kStageBytes + piece_head * S::kHeadBytes;
    auto load_row = [&](int r) {
      const long long off = offsets[ring * TILE + r];
      const uint32_t to = dst + swizzled<RB>(r, piece);
      const bool ok = off >= 0;   // unseen rows are zero-filled: nothing is read
      const long long from = off & 0x7fffffffffffffffll;
      cp_async16(to, kb + from, ok);
      cp_async16(to + S::kTileBytes, vb + from, ok);
    };
    // Of a tile that is not full, rows are filled up to the end of the last
    // warp's share that has a key; warps without one skip the tile.
    const int keys = at.len - at.first - at.t * TILE;
    if (keys >= TILE) {
#pragma unroll
      for (int i = 0; i < (TILE + KPP - 1) / KPP; ++i)
        if (TILE % KPP == 0 || key_in_pass + i * KPP < TILE) load_row(key_in_pass + i * KPP);
    } else {
      const int end = (keys + S::kKeys - 1) / S::kKeys * S::kKeys;
#pragma unroll 1
      for (int r = key_in_pass; r < end; r += KPP) load_row(r);
    }
    if (with_q) {
      const uint16_t* const q = p.q + at.b * p.q_row_stride + (at.hk * HW * G + row0) * D;
      const uint32_t to = sbase + S::kOffQ + q_slot * q_bytes;
      // the warps of a head (warp % HW) load its rows
      // (Code that a short call runs once is kept short, here and below: the
      // call waits for its instructions, too.  Loops left to the compiler's
      // unrolling: +2 to 5 % for calls under 10 us.)
#pragma unroll 1
      for (int i = warp / HW * 32 + lane; i < rows * (D / 8); i += kThreads / HW) {
        const int c = i % (D / 8), r = i / (D / 8);
        cp_async16(to + hw * lc.rows * D * 2 + swizzled<D * 2>(r, c), q + (hw * G + r) * D + c * 8, true);
      }
    }
  };

  // Prologue: the first ST - 1 tiles are on their way before the loop.
  int q_load = 0;                 // query slot of the unit being loaded
  {
    Place<TILE> load = here;
    int pages[ST - 1];   // looked up together: one trip to memory
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
      pages[i] = -1;
      if (i < n) {
        pages[i] = look_up(ahead);
        ahead.next(L, p.batch, groups);
      }
    }
    Place<TILE> at = here;
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
      if (i < n) {
        store_offset(at, pages[i], i);
        at.next(L, p.batch, groups);
      }
    }
    __syncthreads();
    for (int i = 0; i < ST - 1; ++i) {
      if (i < n) {
        const bool with_q = i == 0 || load.t == 0;
        if (i > 0 && with_q) q_load = q_load + 1 == ST ? 0 : q_load + 1;
        load_tile(load, i, i, q_load, with_q);
        load.next(L, p.batch, groups);
      }
      cp_commit();
    }
  }
  int page_ahead = ST - 1 < n ? look_up(ahead) : -1;

  // Per lane (g, quad): keys or dimensions g and g + 8 of 16, heads 2 quad and
  // 2 quad + 1 of 8.
  uint32_t qf[NH][D / 16][2];               // Q^T fragments (e4m3: fp16, rescaled per head)
  float o[NH][DO / 16][4];
  float m[NH][2], l[NH][2], factor[NH][2];  // reference, this lane's sum, scores to units of log 2
  int stage = 0, ring = 0, q_slot = 0;
  int load_stage = ST - 1, load_ring = ST - 1;
  bool fresh = true, first_piece = true;
  const int g = lane >> 2, quad = lane & 3;

  for (int s = 0; s < n; ++s) {
    cp_wait<ST - 2>();
    const bool more = s + ST - 1 < n;
    if (more) store_offset(ahead, page_ahead, load_ring);
    __syncthreads();   // tile s has landed for every thread; tile s - 1's stage is free
    if (more) {
      const bool with_q = ahead.t == 0;
      if (with_q) q_load = q_load + 1 == ST ? 0 : q_load + 1;
      load_tile(ahead, load_ring, load_stage, q_load, with_q);
      ahead.next(L, p.batch, groups);
      if (s + ST < n) page_ahead = look_up(ahead);
      load_stage = load_stage + 1 == ST ? 0 : load_stage + 1;
      load_ring = load_ring + 1 == S::kOffsets ? 0 : load_ring + 1;
    }
    cp_commit();

    if (fresh) {
      fresh = false;
      const uint32_t qb = sbase + S::kOffQ + q_slot * q_bytes + hw * lc.rows * D * 2;
      const float scale = p.scale * kLog2e * (p.kv.k_scale ? *(p.kv.k_scale + here.hk * HW + hw) : 1.f);
#pragma unroll
      for (int i = 0; i < NH; ++i) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          m[i][c] = -INFINITY;
          l[i][c] = 0.f;
          factor[i][c] = scale;
        }
#pragma unroll
        for (int j = 0; j < DO / 16; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[i][j][c] = 0.f;
        if constexpr (!E4M3) {
          const int r = 8 * i + (lane & 7);
#pragma unroll
          for (int j = 0; j < D / 16; j += 2) {
            uint32_t b[4];
            ldsm4(b, r < rows ? qb + swizzled<D * 2>(r, 2 * j + (lane >> 3)) : sbase + S::kOffZero);
            qf[i][j][0] = b[0];
            qf[i][j][1] = b[1];
            qf[i][j + 1][0] = b[2];
            qf[i][j + 1][1] = b[3];
          }
        } else {
          // A lane's four bytes of a K row are four consecutive dimensions;
          // they serve as the products' k = 2 quad, + 1, + 8, + 9, and the query
          // is laid out alike.  It is held in fp16, which its bf16 values fit
          // once each row is scaled by a power of two that brings its largest
          // element to [2^14, 2^15): exact but for elements 2^-28 below it.
          float top = 0.f;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t a = qb + swizzled<D * 2>(8 * i + g, 2 * j + (quad >> 1)) + (quad & 1) * 8;
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(qf[i][j][0]), "=r"(qf[i][j][1])
                         : "r"(8 * i + g < rows ? a : sbase + S::kOffZero)
                         : "memory");
#pragma unroll
            for (int c = 0; c < 2; ++c)
              top = fmaxf(top, fmaxf(fabsf(bf_lo(qf[i][j][c])), fabsf(bf_hi(qf[i][j][c]))));
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = static_cast<int>(__float_as_uint(top) >> 23);
          const int up = e == 255 ? 127 : min(268 - max(e, 1), 253);   // biased exponent of the power
          const float f = __uint_as_float(static_cast<uint32_t>(up) << 23);
          const float back = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) qf[i][j][c] = pack_f16x2(bf_lo(qf[i][j][c]) * f, bf_hi(qf[i][j][c]) * f);
#pragma unroll
          for (int c = 0; c < 2; ++c) factor[i][c] *= __shfl_sync(0xffffffffu, back, (2 * quad + c) * 4);
        }
      }
    }

    const uint32_t kt = sbase + stage * S::kStageBytes + hw * S::kHeadBytes, vt = kt + S::kTileBytes;
    const int key0 = kwarp * S::kKeys;
    uint32_t bits = seen[ring * S::kSeenWords + (key0 >> 5)] >> (key0 & 31);
    if constexpr (S::kKeys == 16) bits &= 0xffffu;
    if (bits != 0u) {
      // S^T = K Q^T for the warp's keys; with few products at a time, in two
      // chains of half the dimensions each.
      constexpr int CH = NH * KT == 1 ? 2 : 1;
      float x[KT][NH][4], x2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int i = 0; i < NH; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[k][i][c] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; j += 2) {
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const int r = key0 + 16 * k + (lane & 15);
          uint32_t a0[4], a1[4];   // dimensions 16 j + [0, 16) and + [16, 32)
          if constexpr (!E4M3) {
            ldsm4(a0, kt + swizzled<RB>(r, 2 * j + (lane >> 4)));
            ldsm4(a1, kt + swizzled<RB>(r, 2 * j + 2 + (lane >> 4)));
          } else {
            uint32_t b[4];
            ldsm4(b, kt + swizzled<RB>(r, j + (lane >> 4)));
            a0[0] = e4m3_lo(b[0]);
            a0[1] = e4m3_lo(b[1]);
            a0[2] = e4m3_hi(b[0]);
            a0[3] = e4m3_hi(b[1]);
            a1[0] = e4m3_lo(b[2]);
            a1[1] = e4m3_lo(b[3]);
            a1[2] = e4m3_hi(b[2]);
            a1[3] = e4m3_hi(b[3]);
          }
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            mma<E4M3>(x[k][i], a0, qf[i][j][0], qf[i][j][1]);
            mma<E4M3>(CH == 2 ? x2 : x[k][i], a1, qf[i][j + 1][0], qf[i][j + 1][1]);
          }
        }
      }
      if constexpr (CH == 2) {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[0][0][c] += x2[c];
      }
      // Weights 2^(x factor - m + kShift), unseen keys 0.  In fp16 (e4m3 caches)
      // they carry 2^kShift so that none above 2^-18 of the reference is subnormal.
      bool keep = true;
      float y[KT][NH][4];
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int i = 0; i < NH; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            y[k][i][c] = fmaf(x[k][i][c], factor[i][c & 1], kShift - m[i][c & 1]);
            if (bits != (S::kKeys == 16 ? 0xffffu : 0xffffffffu) && !((bits >> (16 * k + 8 * (c >> 1) + g)) & 1u))
              y[k][i][c] = -INFINITY;
            keep = keep && y[k][i][c] <= kSlack + kShift;
          }
      if (!__all_sync(0xffffffffu, keep)) {
        // Some score is past the slack (the first tile always): new reference.
#pragma unroll
        for (int i = 0; i < NH; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = m[i][c];
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                if ((bits >> (16 * k + 8 * u + g)) & 1u) top = fmaxf(top, x[k][i][2 * u + c] * factor[i][c]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float f = top == m[i][c] ? 1.f : ex2_approx(m[i][c] - top);
            m[i][c] = top;
            l[i][c] *= f;
#pragma unroll
            for (int j = 0; j < DO / 16; ++j) {
              o[i][j][c] *= f;
              o[i][j][2 + c] *= f;
            }
            const float ref = kShift - (top == -INFINITY ? 0.f : top);
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                y[k][i][2 * u + c] = (bits >> (16 * k + 8 * u + g)) & 1u
                                         ? fmaf(x[k][i][2 * u + c], factor[i][c], ref) : -INFINITY;
          }
      }
      // P^T for the second product (the sums take it in 32 bits).  One 16-bit
      // number would put o further from the exact row than its own rounding
      // does (bf16: 1.4 times), so it is the sum of two: beside bf16 values its
      // upper half and the rest, rounded (2^-16 off); beside e4m3 values its
      // upper 11 bits and the rest in fp16 (2^-21 off), or one fp16 number
      // (2^-11 off) where kTwoParts says so.  Neither part of a bf16 weight is
      // negative, and with the lowest bit set (2^-23) the rest is not zero, so
      // that an infinite value stays infinite (inf (p - q) + inf q and
      // inf 0 would not).
      uint32_t pf[KT][NH][2], pr[KT][NH][2];
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) e[c] = ex2_approx(y[k][i][c]);
          l[i][0] += e[0] + e[2];
          l[i][1] += e[1] + e[3];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if constexpr (E4M3) {
              if constexpr (S::kTwoParts) {
                const float t0 = __uint_as_float(__float_as_uint(e[2 * u]) & 0xFFFFE000u);
                const float t1 = __uint_as_float(__float_as_uint(e[2 * u + 1]) & 0xFFFFE000u);
                pf[k][i][u] = transposed(pack_f16x2(t0, t1));
                pr[k][i][u] = transposed(pack_f16x2(e[2 * u] - t0, e[2 * u + 1] - t1));
              } else {
                pf[k][i][u] = transposed(pack_f16x2(e[2 * u], e[2 * u + 1]));
              }
            } else {
              const uint32_t b0 = __float_as_uint(e[2 * u]), b1 = __float_as_uint(e[2 * u + 1]);
              pf[k][i][u] = transposed(__byte_perm(b0, b1, 0x7632));
              pr[k][i][u] = transposed(pack_bf16x2(__uint_as_float(b0 | 1u) - __uint_as_float(b0 & 0xFFFF0000u),
                                                   __uint_as_float(b1 | 1u) - __uint_as_float(b1 & 0xFFFF0000u)));
            }
          }
        }
      // O^T += V^T P^T
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const int r = key0 + 16 * k;
        if constexpr (!E4M3) {
#pragma unroll
          for (int j = 0; j < DO / 16; ++j) {
            uint32_t a[4];
            ldsm4t(a, vt + swizzled<RB>(r + (lane & 7) + ((lane >> 4) << 3), c0 / 8 + 2 * j + ((lane >> 3) & 1)));
#pragma unroll
            for (int i = 0; i < NH; ++i) {
              mma<false>(o[i][j], a, pf[k][i][0], pf[k][i][1]);
              mma<false>(o[i][j], a, pr[k][i][0], pr[k][i][1]);
            }
          }
        } else {
          // Transposed as 16-bit units, a register holds two keys' bytes of two
          // neighbouring dimensions: rows g and g + 8 of the product are
          // dimensions 2 g and 2 g + 1.
#pragma unroll
          for (int j = 0; j < DO / 16; j += 2) {
            uint32_t b[4];
            ldsm4t(b, vt + swizzled<RB>(r + (lane & 15), c0 / 16 + j + (lane >> 4)));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t even = __byte_perm(b[2 * u], b[2 * u + 1], 0x6420);
              const uint32_t odd = __byte_perm(b[2 * u], b[2 * u + 1], 0x7531);
              const uint32_t a[4] = {e4m3_lo(even), e4m3_lo(odd), e4m3_hi(even), e4m3_hi(odd)};
#pragma unroll
              for (int i = 0; i < NH; ++i) {
                mma<true>(o[i][j + u], a, pf[k][i][0], pf[k][i][1]);
                if constexpr (S::kTwoParts) mma<true>(o[i][j + u], a, pr[k][i][0], pr[k][i][1]);
              }
            }
          }
        }
      }
    }

    const bool unit_done = here.t + 1 == here.nt;
    if (unit_done || s + 1 == n) {
      // This warp's sums; with several key warps, joined in the stage just
      // consumed, else written from the registers.
      const bool starts_here = here.t <= s;   // the unit's first tile is in this run
      const bool whole = unit_done && starts_here;
      const int slot = first_piece ? 0 : 1;
      const long long out_row = static_cast<long long>(here.b) * p.heads + here.hk * HW * G + row0;   // of the first head
      float* const part = parts_of(p.work, gridDim.x * gridDim.y) +
                          (static_cast<size_t>(block) * 2 + slot) * part_floats(HW * lc.rows, D);
#pragma unroll
      for (int i = 0; i < NH; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) l[i][c] += __shfl_xor_sync(0xffffffffu, l[i][c], off);
      if constexpr (KW == 1) {
        const float vs = p.kv.v_scale ? *(p.kv.v_scale + here.hk * HW + hw) : 1.f;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          float inv[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            inv[c] = l[i][c] == 0.f ? 0.f : __fdividef(vs, l[i][c]);
            const int row = 8 * i + 2 * quad + c;
            if (g == 0 && c0 == 0 && row < rows) {
              if (!whole) {
                part[HW * lc.rows * D + hw * lc.rows + row] = m[i][c] - kShift;
                part[HW * lc.rows * D + (HW + hw) * lc.rows + row] = l[i][c];
              } else if (p.lse) {
                p.lse[out_row + hw * G + row] =
                    l[i][c] == 0.f ? -INFINITY : (m[i][c] - kShift + __log2f(l[i][c])) * kLn2;
              }
            }
          }
          if (whole) {
            // transposed to heads in the lanes' rows
            const bool have = 8 * i + g < rows;
            uint16_t* const to = p.o + (out_row + hw * G + 8 * i + g) * D + c0;
#pragma unroll
            for (int j = 0; j < DO / 16; ++j) {
              const uint32_t t0 = transposed(pack_bf16x2(o[i][j][0] * inv[0], o[i][j][1] * inv[1]));
              const uint32_t t1 = transposed(pack_bf16x2(o[i][j][2] * inv[0], o[i][j][3] * inv[1]));
              if (have) {
                if constexpr (E4M3) {
                  *reinterpret_cast<uint2*>(to + 16 * j + 4 * quad) =
                      make_uint2(__byte_perm(t0, t1, 0x5410), __byte_perm(t0, t1, 0x7632));
                } else {
                  *reinterpret_cast<uint32_t*>(to + 16 * j + 2 * quad) = t0;
                  *reinterpret_cast<uint32_t*>(to + 16 * j + 8 + 2 * quad) = t1;
                }
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int row = 8 * i + 2 * quad + c;
              float* const to = part + (hw * lc.rows + row) * D + c0;
              if (row < rows) {
#pragma unroll
                for (int j = 0; j < DO / 16; ++j) {
                  if constexpr (E4M3) {
                    *reinterpret_cast<float2*>(to + 16 * j + 2 * g) = make_float2(o[i][j][c], o[i][j][2 + c]);
                  } else {
                    to[16 * j + g] = o[i][j][c];
                    to[16 * j + 8 + g] = o[i][j][2 + c];
                  }
                }
              }
            }
          }
        }
      } else {
        constexpr int JH = S::kJoinHeads;
        float* const join_m = reinterpret_cast<float*>(smem + S::kOffJoin);   // [HW][KW][HEADS]
        float* const join_l = join_m + S::kRowWarps * HEADS;
        float* const buf = reinterpret_cast<float*>(smem + stage * S::kStageBytes);   // [HW][KW][JH][D]
        const int at = hw * KW + kwarp;
#pragma unroll
        for (int i = 0; i < NH; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (g == 0) {
              join_m[at * HEADS + 8 * i + 2 * quad + c] = m[i][c];
              join_l[at * HEADS + 8 * i + 2 * quad + c] = l[i][c];
            }
#pragma unroll
        for (int h0 = 0; h0 < HEADS; h0 += JH) {
          if (h0 >= rows) break;
          __syncthreads();   // every warp has read the stage, or the heads joined before
          // groups of 8 columns of a head are swizzled by the head
#pragma unroll
          for (int i = h0 / 8; i < (h0 + JH < HEADS ? h0 + JH : HEADS) / 8; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float* const to = buf + (at * JH + 8 * i - h0 + 2 * quad + c) * D;
#pragma unroll
              for (int j = 0; j < DO / 16; ++j) {
                const int col = c0 + 16 * j;
                if constexpr (!E4M3) {
                  to[((((col >> 3) ^ quad) << 3) | g)] = o[i][j][c];
                  to[(((((col >> 3) + 1) ^ quad) << 3) | g)] = o[i][j][2 + c];
                } else {
                  *reinterpret_cast<float2*>(to + (((((col >> 3) + (g >> 2)) ^ quad) << 3) | ((g & 3) * 2))) =
                      make_float2(o[i][j][c], o[i][j][2 + c]);
                }
              }
            }
          __syncthreads();
          const int heads = min(rows - h0, JH);
          for (int i = tid / 16; i < HW * heads; i += kThreads / 16) {   // 16 threads per row
            const int h = HW == 1 ? 0 : i / heads, local = i - h * heads, row = h0 + local;
            float top = -INFINITY, sum = 0.f, f[KW];
#pragma unroll
            for (int w = 0; w < KW; ++w) top = fmaxf(top, join_m[(h * KW + w) * HEADS + row]);
#pragma unroll
            for (int w = 0; w < KW; ++w) {
              const float lw = join_l[(h * KW + w) * HEADS + row];
              f[w] = lw == 0.f ? 0.f : ex2_approx(join_m[(h * KW + w) * HEADS + row] - top);
              sum = fmaf(f[w], lw, sum);
            }
            top -= kShift;
            const float vs = p.kv.v_scale ? *(p.kv.v_scale + here.hk * HW + h) : 1.f;
            const float inv = sum == 0.f ? 0.f : __fdividef(vs, sum);
            const long long to = out_row + h * G + row;
#pragma unroll(KW > 4 ? 1 : D / 64)
            for (int c4 = tid % 16; c4 < D / 4; c4 += 16) {
              float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int w = 0; w < KW; ++w) {
                const float4 v = *reinterpret_cast<const float4*>(
                    buf + ((h * KW + w) * JH + local) * D + ((((c4 >> 1) ^ ((row >> 1) & 3)) << 3) | ((c4 & 1) << 2)));
                acc.x = fmaf(f[w], v.x, acc.x);
                acc.y = fmaf(f[w], v.y, acc.y);
                acc.z = fmaf(f[w], v.z, acc.z);
                acc.w = fmaf(f[w], v.w, acc.w);
              }
              if (whole) {
                uint2 out;
                out.x = pack_bf16x2(acc.x * inv, acc.y * inv);
                out.y = pack_bf16x2(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2*>(p.o + to * D + c4 * 4) = out;
              } else {
                *reinterpret_cast<float4*>(part + (h * lc.rows + row) * D + c4 * 4) = acc;
              }
            }
            if (tid % 16 == 0) {
              if (!whole) {
                part[HW * lc.rows * D + h * lc.rows + row] = top;
                part[HW * lc.rows * D + (HW + h) * lc.rows + row] = sum;
              } else if (p.lse) {
                p.lse[to] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
              }
            }
          }
        }
      }
      if (tid == 0 && s + 1 == n && !lc.by_unit) {
        const int unit = here.b * groups + here.hk, last_tile = start + s - here.t + here.nt - 1;
        reinterpret_cast<int4*>(p.work)[blockIdx.y * lc.blocks + blockIdx.x] = make_int4(
            starts_here && !unit_done ? unit : -1, runs_kept->of(runs_kept->at(last_tile, unit)), slot, 0);
      }
      fresh = true;
      first_piece = false;
      q_slot = q_slot + 1 == ST ? 0 : q_slot + 1;
    }
    here.next(L, p.batch, groups);
    stage = stage + 1 == ST ? 0 : stage + 1;
    ring = ring + 1 == S::kOffsets ? 0 : ring + 1;
  }
}

// ------------------------------------------------------------------ combine
// One block per (cut, query head of a head group, 4 COLS columns): joins the
// partial results of the runs the unit lies in, group g of its threads those
// of runs g, g + GROUPS, ... in one pass with a running maximum, then the
// groups in order.  Few runs: 128 columns (or all); many: 32 columns by 16
// groups.  Blocks are small so that they can wait beside the main kernel's;
// the lengths, which say what runs a unit lies in, were complete before that
// kernel let this one be set up, and are read meanwhile.
constexpr int kJoinThreads = 128;

// Sums relative to a reference, moved to a reference `up` that is no lower.
__device__ __forceinline__ void rescale(float& top, float up, float& sum, float4& acc) {
  const float keep = up == top ? 1.f : ex2_approx(top - up);
  top = up;
  sum *= keep;
  acc.x *= keep;
  acc.y *= keep;
  acc.z *= keep;
  acc.w *= keep;
}
// Adds a partial result whose reference is no higher.
__device__ __forceinline__ void add_part(float top, float& sum, float4& acc, float m, float l, const float4& v) {
  const float f = l == 0.f ? 0.f : ex2_approx(m - top);
  sum = fmaf(f, l, sum);
  acc.x = fmaf(f, v.x, acc.x);
  acc.y = fmaf(f, v.y, acc.y);
  acc.z = fmaf(f, v.z, acc.z);
  acc.w = fmaf(f, v.w, acc.w);
}

template <int D, int COLS>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const DecodeParams p, const Launch lc) {
  constexpr int GROUPS = kJoinThreads / COLS, WARPS = kJoinThreads / 32;
  __shared__ float s_top[WARPS], s_sum[WARPS];
  __shared__ float4 s_acc[WARPS][COLS];
  const int tid = threadIdx.x;
  const int local = blockIdx.y % (lc.group * lc.rows), chunk = blockIdx.y / (lc.group * lc.rows);
  const int head = local / lc.rows, row = local % lc.rows;   // of the group; of the head's chunk
  const int G = p.heads / p.kv.heads_kv, groups = p.kv.heads_kv / lc.group;
  int unit, run, last, first_slot;
  if (lc.by_unit) {
    // the tiles before this unit and in all
    __shared__ int s_before[kJoinThreads / 32], s_total[kJoinThreads / 32];
    unit = blockIdx.x;
    const Lens L{p.seq_lens, p.max_pages * p.kv.page_size, p.window};
    const int b = unit / groups;
    int before = 0, total = 0;
#pragma unroll 1
    for (int i = tid; i < p.batch; i += kJoinThreads) {
      const int nt = L.tiles(L.len(i), lc.tile_shift);
      total += nt;
      if (i < b) before += nt;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, off);
      total += __shfl_xor_sync(0xffffffffu, total, off);
    }
    if (tid % 32 == 0) {
      s_before[tid / 32] = before;
      s_total[tid / 32] = total;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      before += s_before[w];
      total += s_total[w];
    }
    const Runs runs(total * groups, p.batch * groups, lc.blocks);
    const int nt = L.tiles(L.len(b), lc.tile_shift), tiles_before = before * groups + (unit - b * groups) * nt;
    const int first = runs.at(tiles_before, unit);
    run = runs.of(first);
    last = runs.of(runs.at(tiles_before + nt - 1, unit));
    // slot 0 where the tile before, of another unit, is not in that run
    first_slot = first - runs.at(1, 1) < runs.start(run) ? 0 : 1;
  } else {
    pdl_wait();
    const int4 cut = *(reinterpret_cast<const int4*>(p.work) + chunk * lc.blocks + blockIdx.x);
    if (cut.x < 0) return;
    unit = cut.x;
    run = blockIdx.x;
    last = cut.y;
    first_slot = cut.z;
  }
  const int b = unit / groups, hk = unit % groups * lc.group + head;
  const int n = last - run + 1;
  const float* const parts = parts_of(p.work, static_cast<size_t>(lc.blocks) * lc.chunks);
  const int part_rows = lc.group * lc.rows;
  const size_t pf = part_floats(part_rows, D);
  const int col = blockIdx.z * COLS + tid % COLS, group = tid / COLS;
  const float vs = p.kv.v_scale ? *(p.kv.v_scale + hk) : 1.f;
  // Before any block ends: the next kernel waits for this one only.
  pdl_wait();
  if (last == run || chunk * lc.rows + row >= G) return;   // not cut; no such head
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int U = COLS == 8 ? 4 : 1;   // partial results in flight per thread
  for (int i0 = group; i0 < n; i0 += U * GROUPS) {
    float mi[U], li[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * GROUPS;
      mi[u] = -INFINITY;
      li[u] = 0.f;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const float* const part =
            parts + (static_cast<size_t>(chunk * lc.blocks + run + i) * 2 + (i == 0 ? first_slot : 0)) * pf;
        v[u] = *reinterpret_cast<const float4*>(part + local * D + col * 4);
        mi[u] = part[part_rows * D + local];
        li[u] = part[part_rows * D + part_rows + local];
      }
    }
    float up = top;
#pragma unroll
    for (int u = 0; u < U; ++u) up = fmaxf(up, mi[u]);
    rescale(top, up, sum, acc);
#pragma unroll
    for (int u = 0; u < U; ++u) add_part(top, sum, acc, mi[u], li[u], v[u]);
  }
  // the groups of a warp, then the warps
#pragma unroll
  for (int off = COLS; off < 32; off <<= 1) {
    const float mo = __shfl_xor_sync(0xffffffffu, top, off), lo = __shfl_xor_sync(0xffffffffu, sum, off);
    const float4 vo = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, off), __shfl_xor_sync(0xffffffffu, acc.y, off),
                                  __shfl_xor_sync(0xffffffffu, acc.z, off), __shfl_xor_sync(0xffffffffu, acc.w, off));
    rescale(top, fmaxf(top, mo), sum, acc);
    add_part(top, sum, acc, mo, lo, vo);
  }
  const int warp = tid / 32;
  if (tid % 32 < COLS) s_acc[warp][tid % 32] = acc;
  if (tid % 32 == 0) {
    s_top[warp] = top;
    s_sum[warp] = sum;
  }
  __syncthreads();
  if (tid >= COLS) return;
#pragma unroll
  for (int w = 1; w < WARPS; ++w) {
    rescale(top, fmaxf(top, s_top[w]), sum, acc);
    add_part(top, sum, acc, s_top[w], s_sum[w], s_acc[w][tid]);
  }
  const float inv = sum == 0.f ? 0.f : __fdividef(vs, sum);
  const long long at = static_cast<long long>(b) * p.heads + hk * G + chunk * lc.rows + row;
  uint2 out;
  out.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  out.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.o + at * D + col * 4) = out;
  if (p.lse && col == 0) p.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------ launch
template <int D, bool E4M3, int NH, int HW>
cudaError_t launch_shape(const DecodeParams& p, const Call& c, Launch lc, cudaStream_t s) {
  using Sh = Shape<D, E4M3, NH, HW>;
  static std::atomic<unsigned long long> done{0}, few_done{0}, many_done{0};
  auto* const kernel = decode_kernel<D, E4M3, NH, HW>;
  cudaError_t e = prepare_once(reinterpret_cast<const void*>(kernel), 227 * 1024, lc.device, done);
  if (e != cudaSuccess) return e;
  set_blocks<Sh, HW>(c, lc);
  e = launch_pdl(kernel, dim3(lc.blocks, lc.chunks), dim3(Sh::kThreads), Sh::smem(lc.rows), s, p, lc);
  if (e != cudaSuccess || !lc.joined) return e;
  const int units = p.batch * (p.kv.heads_kv / HW);
  dim3 grid(lc.by_unit ? units : lc.blocks, lc.chunks * HW * lc.rows, D == 256 ? 2 : 1);
  // A unit lies in about blocks / units runs (ragged lengths: some in several
  // times as many).
  const bool few = 8ll * units > lc.blocks;
  auto* const combine = few ? combine_kernel<D, (D < 128 ? D : 128) / 4> : combine_kernel<D, 8>;
  if (!few) grid.z = D / 32;
  e = prepare_once(reinterpret_cast<const void*>(combine), 0, lc.device, few ? few_done : many_done);
  if (e != cudaSuccess) return e;
  return launch_pdl(combine, grid, dim3(kJoinThreads), 0, s, p, lc);
}

template <int D, bool E4M3>
cudaError_t launch_dim(const DecodeParams& p, const Call& c, const Launch& lc, cudaStream_t s) {
  return with_shape<D, E4M3>(c, lc, [&](auto nh, auto hw) {
    return launch_shape<D, E4M3, decltype(nh)::value, decltype(hw)::value>(p, c, lc, s);
  });
}

}  // namespace decode
}  // namespace fa
