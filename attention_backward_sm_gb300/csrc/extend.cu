// Attention of several new tokens per request over a paged key/value cache.
//
// Request b has n new tokens (rows cu[b] to cu[b + 1] of q) whose keys and
// values are in the cache already, s keys in all.  New token i is at position
// p = s - n + i and sees the keys j in [max(0, p - window + 1), p]:
//     x_j = scale * q . k_j,  o = sum_j exp(x_j) v_j / sum_j exp(x_j),
//     lse = ln sum_j exp(x_j)
// Keys whose block-table entry is not a page of the cache are not seen; a row
// that sees no key gets o = 0, lse = -inf.
//
// Products.  The rows of a unit are the query heads of one key/value head for
// some consecutive tokens (row r is token r / G, head r % G, G = heads /
// heads_kv), 256 of them as two tiles of 128 (one tile at head_dim 256).  So a
// key is read once for all heads that share it, and a call of a few tokens per
// request (2 G rows) has the tensor work of one that has none to share.  Per
// block of 128 keys (64 at head_dim 256): S = Q K^T into tensor memory, softmax
// with a thread per row, P as 16-bit values over S, O += P V with P from tensor
// memory; tcgen05 throughout.  With P in bf16 o is 2.3e-3 from the 64-bit result
// where the rounding of o alone leaves 1.7e-3; a second number per weight, as decode
// has it, would take half the products' time again.  P in fp16 (8-bit caches) adds
// next to nothing.  Chunks of hundreds of tokens are bound by these
// products and the exponentials, short ones by HBM.
//
// Work.  The units of all requests (requests in order, key/value heads, tiles
// of rows) and their blocks of keys are laid out on a line by what they cost
// (keys seen, and what a unit's start and end take), and the line is cut into
// runs of equal length, one per SM: ragged lengths, one long document and a
// causal mask's short first rows all load every SM alike, and the host needs no
// lengths.  A unit that lies in several runs leaves partial
// results (at most two per run), which a second kernel joins in a fixed order.
// The costs are closed forms of a request's numbers, so that every block finds
// its run with one scan over the requests.
//
// Warps: per tile of 128 rows four for the softmax and the output, then four
// that load keys and values (beside an 8-bit cache they make fp16 of them, eight
// at head_dim 256), one that issues the products, one that walks along the run,
// tells the others what is next and starts the copies by TMA, two that load
// queries.
//   Two tiles: the products of one run while the softmax works on the other,
//   in the order P_A V, S_A (of the next block), P_B V, S_B.
//   One tile (at most 128 rows): two score buffers, S of the next block is
//   issued before P V of this one.
// The tensor core takes a block's products in the order they are issued, which
// is what lets S overwrite the P before it without waiting.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/fabwd.h"
#include "checks.h"
#include "extend.h"
#include "internal.h"
#include "paged.h"
#include "quantise.cuh"
#include "sm103.cuh"

namespace fa {

__device__ int g_extend_status = 0;

namespace extend {
namespace {

constexpr uint32_t TMEM_COLS = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's reference for the exponents moves where the weights of half a block add
// up to more than kMostSum, or one of them exceeds 2^kMostLog: fp16 weights have to stay
// in their type's range, and beside bf16 ones the fp32 sums of n weights times values
// have room for values up to 2^113 / n.
constexpr float kMostLog = 14.5f, kMostSum = 0x1p15f;
// fp16 weights (8-bit caches) are stored times 2^7: at most 2^15, and the
// smallest step 2^-24 counts 2^-31 beside the row's largest weight.
constexpr float kF16Shift = 7.f;
constexpr int kPieces = 4;     // pieces of the run that the walker is ahead
constexpr int kLeastRun = 4;   // costs
constexpr int kMarks = 8;      // blocks whose missing pages are kept
constexpr int kLag = 2;        // loads in flight behind the newest

struct Piece {
  int n;            // blocks of keys; 0: the run is over
  int kb0;          // the first one
  int b;            // request
  int head_kv;
  int key_lo;       // keys that any row of the unit sees: [key_lo, key_hi)
  int key_hi;
  int token0;       // row of q of the request's first token
  int row_first;    // first row of the unit in the request
  int rows;         // of the unit
  int pos0;         // position of the request's first token
  int part;         // 0: the whole unit; 1, 2: partial, to slot part - 1
  int pad;
};

// S_FULL and P_READY: of tile 0 (and the first score buffer of a single tile), of
// tile 1, and of a single tile's second buffer.  Waits are by parity, so a wait for
// a phase must neither come before the phase ahead of it has ended nor after the
// one behind it: tile 1's warps, which take no part in units of one tile, have
// barriers of their own, and so has the end of a piece (O_LAST; O_DONE is of every
// block).
enum { B_Q_FULL = 0, B_Q_EMPTY, B_Q_RAW, B_S_FULL, B_P_READY = B_S_FULL + 3, B_P_HALF = B_P_READY + 3, B_O_DONE = B_P_HALF + 2, B_O_LAST = B_O_DONE + 2,
       B_O_FREE = B_O_LAST + 2, B_PIECE_FULL = B_O_FREE + 2, B_PIECE_EMPTY = B_PIECE_FULL + kPieces, B_TEARDOWN = B_PIECE_EMPTY + kPieces,
       B_FULL };

template <int D, bool E4M3>
struct Layout {
  using S = Shape<D>;
  static constexpr int BK = S::kKeys;
  static constexpr uint32_t TILE_Q = 128 * D * 2;
  static constexpr uint32_t CHUNK_Q = 128 * 128;
  static constexpr uint32_t TILE_KV = BK * D * 2;
  static constexpr uint32_t CHUNK_KV = BK * 128;
  // Ring of key and value tiles; 8-bit caches: and one of rows as they are cached,
  // on their way.
  static constexpr int NS = E4M3 ? (D == 64 ? 6 : 3) : D == 64 ? 8 : 5;
  static constexpr int NR = E4M3 ? (D == 64 ? 6 : 4) : 0;
  static constexpr uint32_t TILE_RAW = BK * D;
  static constexpr uint32_t Q = 0;
  static constexpr uint32_t KV = S::kTiles * TILE_Q;
  static constexpr uint32_t RAW = KV + NS * TILE_KV;
  static constexpr uint32_t BARS = RAW + NR * TILE_RAW;
  static constexpr int NUM_BARS = B_FULL + 2 * NS + 2 * NR;
  static constexpr uint32_t MARKS = (BARS + NUM_BARS * 8 + 15) / 16 * 16;    // [kMarks][4] words, a bit per key
  static constexpr uint32_t PIECES = MARKS + kMarks * 16;
  static constexpr uint32_t QSCALE = PIECES + kPieces * sizeof(Piece);       // [2 pieces][rows] (8-bit caches)
  static constexpr uint32_t MISC = QSCALE + (E4M3 ? 2 * S::kRows * 4 : 0);
  static constexpr uint32_t BYTES = MISC + 16;
  static constexpr uint32_t COL_O = 2 * BK;              // after two score buffers
  static constexpr int LOAD_WARPS = E4M3 && S::kTiles == 1 ? 8 : 4;
  // Who makes fp16 of the queries of an 8-bit cache: the loading warps, or at heads of 64,
  // whose tiles of keys are the smallest, the query warps.  (4 chunks of 2048 over cached
  // rows, 32 / 8 heads of 128: 960 us, and 1166 by the query warps; 32 / 8 heads of 64: 811,
  // and 757 by the query warps; 64 requests of 1 to 8 tokens 124, and 105.)
  static constexpr bool LOADERS_CONVERT_Q = E4M3 && D > 64;
  static constexpr int WARPS = 4 * S::kTiles + LOAD_WARPS + 4;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int LOAD_WARP = 4 * S::kTiles;
  static constexpr int MMA_WARP = LOAD_WARP + LOAD_WARPS;
  static constexpr int WALK_WARP = MMA_WARP + 1;
  static constexpr int Q_WARP = WALK_WARP + 1;           // two
  // registers: 65536 / THREADS at launch
  static constexpr uint32_t REG_LAUNCH = 65536 / THREADS / 8 * 8;
  static constexpr uint32_t REG_SOFTMAX = S::kTiles == 2 ? 184 : 208;
  static constexpr uint32_t REG_OTHER = S::kTiles == 2 ? 72 : E4M3 ? 96 : 144;
  static_assert(S::kTiles * 128 * REG_SOFTMAX + (THREADS - S::kTiles * 128) * REG_OTHER <= REG_LAUNCH * THREADS,
                "register budget");
  static_assert(COL_O + S::kTiles * D <= TMEM_COLS, "tensor memory budget");
  static_assert(BYTES <= 232448, "shared memory budget");
  static_assert(E4M3 || NS > kLag + 1, "loads in flight");
  static_assert(2 * kMarks - NS - NR >= 2, "marks outlive their block");
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t tile) { return sw128_desc(tile, 16, 1024); }
__device__ __forceinline__ constexpr uint64_t step_kmajor(int t, uint32_t chunk) {
  return ((t >> 2) * chunk + (t & 3) * 32) >> 4;
}
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t tile, uint32_t chunk) { return sw128_desc(tile, chunk, 1024); }
__device__ __forceinline__ constexpr uint64_t step_mnmajor(int t) { return (t * 2048) >> 4; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;   // fewer source bytes than 16: the rest is zero-filled
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four 8-bit values to four halves (exact).
__device__ __forceinline__ uint2 e4m3x4_f16(uint32_t x) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(x));
  return r;
}
// ------------------------------------------------------------------ partition
// A request's numbers, and the cost of its units.  Tile x costs kUnitCost and
// kBlockCost (a last tile of at most 128 rows: kShortCost) for every 2^cost_shift
// keys that its last row sees (as if none were missing), summed over tiles in closed
// form: costs only share out the work, so they are rounded as suits, but every block
// has to come to the same ones.  Plain 32-bit integers, without a division: the walk
// to a block's run is on the way of short calls.
// A unit's start and end cost as much as two blocks of keys (one tile of rows: six):
// with a cost of 1 for them 64 requests of 1 to 8 tokens take 125 us instead of 105,
// 37 ragged ones with a window of 1024 113 instead of 83.  A block of one tile of rows
// where the unit has room for two: as much as one of two, the ragged ones take 112.
template <int D>
struct Request {
  using S = Shape<D>;
  static constexpr int kUnitCost = S::kTiles == 2 ? 6 : 12, kBlockCost = S::kTiles == 2 ? 3 : 2, kShortCost = 2;
  static constexpr int kRowBits = S::kRows == 256 ? 8 : 7;
  int token0, len, pos0, base, rows;   // rows: tokens * group
  int tiles;
  int ramp;   // tiles that see less than the window
  int most;   // with a window: what a tile costs at most
  int last_block, last;   // what a block of the last tile costs, and the tile
  int cost;   // of all tiles, for one key/value head
  __device__ __forceinline__ Request(const ExtendParams& p, int b, int group) {
    const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1];
    len = min(max(p.seq_lens[b], 0), p.max_pages * p.kv.page_size);
    token0 = min(max(c0, 0), p.num_tokens);
    const int end = min(max(c1, token0), p.num_tokens);
    const long long n = max(static_cast<long long>(c1) - c0, 0ll);
    pos0 = static_cast<int>(max(len - n, -static_cast<long long>(p.num_tokens) - 1));
    rows = (end - token0) * group;
    tiles = (rows + S::kRows - 1) >> kRowBits;
    base = max(pos0, 0);
    ramp = tiles;
    last_block = S::kTiles == 2 && rows - (tiles - 1) * S::kRows <= 128 ? kShortCost : kBlockCost;
    last = kUnitCost + last_block * ((base + end - token0) >> p.cost_shift);
    most = 0x7fffffff;
    if (p.window > 0) {
      const long long seen = static_cast<long long>(p.window) + p.tile_tokens;
      ramp = seen > base ? static_cast<int>(min(((seen - base) * group) >> kRowBits, static_cast<long long>(tiles))) : 0;
      const int blocks = 1 + static_cast<int>(min(seen, 0x7fffffffll) >> p.cost_shift);
      most = kUnitCost + kBlockCost * blocks;
      last = min(last, kUnitCost + last_block * blocks);
    }
    cost = tiles > 0 ? full(p, tiles - 1) + last : 0;
  }
  // Of the tiles before tile x.
  __device__ __forceinline__ int before(const ExtendParams& p, int x) const { return x == tiles ? cost : full(p, x); }
  __device__ __forceinline__ int full(const ExtendParams& p, int x) const {
    const long long y = min(x, ramp);   // the sum of base + (i + 1) rows / group over i < y, in 32nds
    const long long keys = y * base * 32 + y * (y + 1) * p.tile_keys16;
    return x * kUnitCost + static_cast<int>((kBlockCost * keys) >> (p.cost_shift + 5)) + (x - static_cast<int>(y)) * (most - kUnitCost);
  }
};

struct Runs {
  int base, rem, runs;
  __device__ __forceinline__ Runs(int total, int blocks) {
    runs = max(1, min(total / kLeastRun, blocks));
    base = static_cast<unsigned>(total) / static_cast<unsigned>(runs);
    rem = total - base * runs;
  }
  __device__ __forceinline__ int start(int r) const { return r * base + min(r, rem); }
  // The run that holds place x.
  __device__ __forceinline__ int of(int x) const {
    const int y = x - rem * (base + 1);
    return y < 0 ? static_cast<unsigned>(x) / static_cast<unsigned>(base + 1)
                 : rem + static_cast<unsigned>(y) / static_cast<unsigned>(base);
  }
};

// Workspace: [runs] cuts, then the partial results.
__device__ __forceinline__ float* parts_of(void* work, int runs) {
  return reinterpret_cast<float*>(static_cast<Cut*>(work) + runs);
}

// Tile e of a piece of n blocks, in the order in which the products take them: K0
// V0 K1 V1 ... for two tiles of rows, K0 K1 V0 K2 V1 ... for one.
__device__ __forceinline__ bool is_key(int e, int n, bool two) {
  return two ? !(e & 1) : e == 0 || ((e & 1) && e + 1 < 2 * n);
}
// Values of the block before the newest key's.
__device__ __forceinline__ bool is_old(int e, int n, bool two) { return !two && e + 1 < 2 * n; }

// Queries of an 8-bit cache from bf16 to fp16 in place, a row times a power of two that
// puts its largest value just below 2^15; scale has the power's inverse.  Warp w of
// `warps`, NB rows (or pairs, fours of them) in flight.
template <int D, int NB>
__device__ __forceinline__ void convert_queries(uint32_t q, float* scale, int rows, int w, int warps, int lane) {
  constexpr int QPR = D / 8, QPI = 32 / QPR;   // pieces per row, rows per step
  const int c = lane % QPR;
#pragma unroll 1
  for (int r0 = w * (NB * QPI); r0 < rows; r0 += warps * NB * QPI) {
    auto place = [&](int i) {
      const int rr = r0 + i * QPI + lane / QPR;
      return q + (rr >> 7) * (128 * D * 2) + (c >> 3) * (128 * 128) + (rr & 127) * 128 + (((c & 7) ^ (rr & 7)) << 4);
    };
    uint32_t words[NB][4], top[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(words[i][0]), "=r"(words[i][1]), "=r"(words[i][2]), "=r"(words[i][3])
                   : "r"(place(i))
                   : "memory");
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      top[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top[i] = max(top[i], max(words[i][e] << 16 & 0x7FFF0000u, words[i][e] & 0x7FFF0000u));
    }
#pragma unroll
    for (int x = QPR / 2; x > 0; x >>= 1)
#pragma unroll
      for (int i = 0; i < NB; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], x));
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      // exponent field of the factor: 127 + 14 - (top's - 127), kept a normal number
      const int ex = min(max(268 - static_cast<int>(top[i] >> 23), 1), 254);
      const float f = __uint_as_float(static_cast<uint32_t>(ex) << 23);
      uint32_t out[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = pack_f16x2(bf_lo(words[i][e]) * f, bf_hi(words[i][e]) * f);
      st_shared_v4(place(i), out[0], out[1], out[2], out[3]);
      if (c == 0) scale[r0 + i * QPI + lane / QPR] = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
    }
  }
}

// ------------------------------------------------------------------ main kernel
template <int D, bool E4M3>
__global__ void __launch_bounds__(Layout<D, E4M3>::THREADS, 1) extend_kernel(const __grid_constant__ ExtendParams p) {
  using L = Layout<D, E4M3>;
  using S = Shape<D>;
  constexpr int BK = L::BK, NS = L::NS, NR = E4M3 ? L::NR : 1, TILES = S::kTiles, ROWS = S::kRows;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = p.heads / p.kv.heads_kv;
  int* const status = &g_extend_status;
  volatile int* const abort = reinterpret_cast<volatile int*>(smem + L::MISC);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC + 4);
  Piece* const pieces = reinterpret_cast<Piece*>(smem + L::PIECES);
  uint32_t* const marks = reinterpret_cast<uint32_t*>(smem + L::MARKS);
  float* const q_scale = reinterpret_cast<float*>(smem + L::QSCALE);
  const uint32_t bars = sbase + L::BARS;
  auto bar = [&](int i) { return bars + 8u * i; };
  auto full = [&](int s) { return bars + 8u * (B_FULL + s); };
  auto empty = [&](int s) { return bars + 8u * (B_FULL + NS + s); };
  // of the ring of cached rows, where the walker fills it
  [[maybe_unused]] auto landed = [&](int s) { return bars + 8u * (B_FULL + 2 * NS + s); };
  [[maybe_unused]] auto taken = [&](int s) { return bars + 8u * (B_FULL + 2 * NS + NR + s); };

  if (sbase & 1023) {
    if (threadIdx.x == 0) atomicCAS(status, 0, 99);
    return;
  }
  const bool boxed = E4M3 && p.box_rows > 0;
  if (threadIdx.x == 0) {
    *abort = 0;
    mbar_init(bar(B_Q_FULL), L::LOADERS_CONVERT_Q ? L::LOAD_WARPS : 2);   // a lane of every warp, here and below
    mbar_init(bar(B_Q_RAW), 2);
    mbar_init(bar(B_Q_EMPTY), 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(B_S_FULL + i), 1);
      mbar_init(bar(B_P_READY + i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_P_HALF + i), 4);
      mbar_init(bar(B_O_DONE + i), 1);
      mbar_init(bar(B_O_LAST + i), 1);
      mbar_init(bar(B_O_FREE + i), 4);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(bar(B_PIECE_FULL + i), 1);
      mbar_init(bar(B_PIECE_EMPTY + i), 4 * TILES + L::LOAD_WARPS + 3);   // all warps but the walker
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), boxed ? 4 : L::LOAD_WARPS);
      mbar_init(empty(i), 1);
    }
    if constexpr (E4M3)
      for (int i = 0; i < NR; ++i) {
        mbar_init(landed(i), 1);
        mbar_init(taken(i), 4);
      }
    mbar_init(bar(B_TEARDOWN), 1);
    mbar_init_fence();
  }
  if (warp == L::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch();

  if (warp == L::WALK_WARP) {
    // ------------------------------------------------------------ walker
    setmaxnreg_to<L::REG_OTHER, L::REG_LAUNCH>();
    Cut cut = {};
    int count = 0;   // pieces
    const int spare = p.cost_shift - (BK == 128 ? 7 : 6);   // blocks that cost 1 together, log 2
    bool ok = true;
    // 8-bit caches in boxes: brings a piece's rows to the ring of cached rows, a lane
    // per box, and marks missing pages.
    [[maybe_unused]] int asked = 0, block = 0;   // tiles, blocks
    [[maybe_unused]] auto bring = [&](const Piece& u) {
      const int32_t* const table = p.table + u.b * p.table_stride;
      const bool two = TILES == 2 && u.rows > 128;
      const int boxes = BK / p.box_rows, last_page = u.key_hi > 0 ? p.page_div.quotient(u.key_hi - 1) : -1;
      int first_key = u.kb0 * BK + lane * p.box_rows;   // of this lane's box in the next block
      auto page_of = [&](int key) {
        const int pi = p.page_div.quotient(key);
        return lane < boxes && key + p.box_rows > u.key_lo && pi <= last_page ? table[pi] : -1;
      };
      int page = page_of(first_key), at_page[2] = {0, 0}, at_slot[2] = {0, 0};
#pragma unroll 1
      for (int e = 0; ok && e < 2 * u.n; ++e, ++asked) {
        const bool key = is_key(e, u.n, two);
        if (key) {
          at_page[1] = at_page[0];
          at_slot[1] = at_slot[0];
          const bool there = page >= 0 && page < p.kv.num_pages;
          at_page[0] = there ? page : p.kv.num_pages;   // past the last: reads as zeros
          at_slot[0] = first_key - p.page_div.quotient(first_key) * p.kv.page_size;
          const unsigned missing = __ballot_sync(0xffffffffu, lane < boxes && !there);
          if (lane < BK / 32) {   // a bit per key
            uint32_t word = 0;
            if (missing)
              for (int i = 0; i < 32; ++i) word |= (missing >> ((lane * 32 + i) / p.box_rows) & 1) << i;
            marks[(block % kMarks) * 4 + lane] = word;
          }
          __syncwarp();
          ++block;
          first_key += BK;
          page = page_of(first_key);
        }
        const int s = asked % NR;
        if (asked >= NR && !mbar_wait(taken(s), (asked / NR - 1) & 1, abort, status)) ok = false;
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (lane == 0) mbar_arrive_expect_tx(landed(s), BK * D);
        __syncwarp();
        const int old = !key && is_old(e, u.n, two);
        if (lane < boxes)
          tma_load_4d(sbase + L::RAW + s * L::TILE_RAW + lane * p.box_rows * D, key ? &p.tm_k : &p.tm_v, 0, u.head_kv,
                      old ? at_slot[1] : at_slot[0], old ? at_page[1] : at_page[0], landed(s));
        __syncwarp();
      }
    };
    auto emit = [&](const Piece& piece) {
      const int slot = count % kPieces;
      if (count >= kPieces && !mbar_wait(bar(B_PIECE_EMPTY + slot), (count / kPieces - 1) & 1, abort, status)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) {
        pieces[slot] = piece;
        mbar_arrive(bar(B_PIECE_FULL + slot));
      }
      __syncwarp();
      ++count;
      if constexpr (E4M3)
        if (p.box_rows > 0 && piece.n > 0) bring(piece);
    };
    // The line's length, then the request that this block's run starts in: 32
    // requests at a time.
    const int heads_kv = p.kv.heads_kv;
    int total = 0, mine = 0;   // mine: of this lane's request among the last 32
#pragma unroll 1
    for (int b = lane; b < p.batch; b += 32) total += mine = Request<D>(p, b, group).cost * heads_kv;
    total = __reduce_add_sync(0xffffffffu, total);
    const Runs runs(total, gridDim.x);
    const int run_start = static_cast<int>(blockIdx.x) < runs.runs ? runs.start(blockIdx.x) : total;
    const int run_end = run_start < total ? runs.start(blockIdx.x + 1) : total;
    if (run_start < total) {
      int b = 0, at = 0;   // the request and its place on the line
#pragma unroll 1
      for (int b32 = 0; b32 < p.batch; b32 += 32) {
        if (p.batch > 32) mine = b32 + lane < p.batch ? Request<D>(p, b32 + lane, group).cost * heads_kv : 0;
        else if (lane >= p.batch) mine = 0;
        int upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at + upto > run_start);
        if (past) {
          const int l = __ffs(past) - 1;
          b = b32 + l;
          at += __shfl_sync(0xffffffffu, upto - mine, l);
          break;
        }
        at += __shfl_sync(0xffffffffu, upto, 31);
      }
      while (ok && b < p.batch && at < run_end) {
        const Request<D> r(p, b, group);
        if (r.cost == 0) {
          ++b;
          continue;
        }
        int hk = 0, x = 0;
        if (run_start > at) {
          const int in = run_start - at;
          hk = static_cast<unsigned>(in) / static_cast<unsigned>(r.cost);
          const int rem = in - hk * r.cost;
          int hi = r.tiles;   // before(x) <= rem < before(hi)
          while (hi - x > 1) {
            const int mid = (x + hi) >> 1;
            if (r.before(p, mid) <= rem) x = mid;
            else hi = mid;
          }
        }
        bool in_run = true;
        for (; ok && in_run && hk < heads_kv; ++hk, x = 0) {
          for (; ok && x < r.tiles; ++x) {
            const int c = at + hk * r.cost + r.before(p, x);
            if (c >= run_end) {
              in_run = false;
              break;
            }
            const int w = r.before(p, x + 1) - r.before(p, x);
            Piece u;
            u.b = b;
            u.head_kv = hk;
            u.token0 = r.token0;
            u.row_first = x * ROWS;
            u.rows = min(ROWS, r.rows - u.row_first);
            u.pos0 = r.pos0;
            const int first = r.pos0 + p.group_div.quotient(u.row_first);
            const int last = r.pos0 + p.group_div.quotient(u.row_first + u.rows - 1);
            u.key_hi = max(last + 1, 0);
            u.key_lo = p.window > 0 ? min(max(max(first, 0) - p.window + 1, 0), u.key_hi) : 0;   // (tokens before 0 see nothing)
            const int kb = u.key_lo / BK;
            const int nblk = max(1, (u.key_hi + BK - 1) / BK - kb);   // a unit that sees nothing has one (masked) block
            // Block j starts at c + min(j cost >> spare, w - 1).  Those in [run_start, run_end):
            const int cost = x + 1 == r.tiles ? r.last_block : Request<D>::kBlockCost;
            auto first_from = [&](int place) { return min((((place - c) << spare) + cost - 1) / cost, nblk); };
            const int j0 = run_start <= c ? 0 : first_from(run_start);
            const int j1 = run_end >= c + w ? nblk : first_from(run_end);
            if (j1 <= j0) {
              // inside a unit, but none of its blocks starts here: no partial result
              if (j0 > 0 && j0 < nblk) {
                float* const l = parts_of(p.work, gridDim.x) +
                                 static_cast<size_t>(blockIdx.x) * 2 * part_floats(ROWS, D) + static_cast<size_t>(ROWS) * (D + 1);
                for (int i = lane; i < ROWS; i += 32) l[i] = 0.f;
              }
              continue;
            }
            u.kb0 = kb + j0;
            u.n = j1 - j0;
            u.part = j0 > 0 ? 1 : j1 < nblk ? 2 : 0;
            if (u.part == 2) {
              // the run in which the unit's last block starts
              cut.row_end = r.rows;
              cut.row_first = u.row_first;
              cut.token0 = r.token0;
              cut.head_kv = hk;
              cut.last = min(runs.of(c + min(((nblk - 1) * cost) >> spare, w - 1)), runs.runs - 1);
            }
            emit(u);
          }
        }
        at += r.cost * heads_kv;
        ++b;
      }
    }
    Piece over = {};
    if (ok) emit(over);
    if constexpr (E4M3)
      if (!ok) {   // after an abort, what has been asked for lands before the block ends
        volatile int no_abort = 0;
        for (int i = max(0, asked - NR); i < asked; ++i)
          mbar_wait(landed(i % NR), (i / NR) & 1, &no_abort, status, 100000000ull);
      }
    if (lane == 0) reinterpret_cast<Cut*>(p.work)[blockIdx.x] = cut;
  } else if (warp == L::MMA_WARP) {
    // ------------------------------------------------------------ products
    setmaxnreg_to<L::REG_OTHER, L::REG_LAUNCH>();
    constexpr uint32_t ID_S = E4M3 ? idesc_f16(128, BK, 0) : idesc_bf16(128, BK, 0, 0);
    constexpr uint32_t ID_O = E4M3 ? idesc_f16(128, D, 1) : idesc_bf16(128, D, 0, 1);
    int slot = 0, phase = 0;                    // of the ring of tiles
    int used[2] = {0, 0};                       // phases of P_HALF
    int used_all[2] = {0, 0}, used_odd = 0;     // of P_READY
    int freed[2] = {0, 0};                      // pieces of a tile
    auto next_slot = [&] {
      if (++slot == NS) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto issue_s = [&](int t, int buf, int at) {
      const uint64_t a0 = desc_kmajor(sbase + L::Q + t * L::TILE_Q), b0 = desc_kmajor(sbase + L::KV + at * L::TILE_KV);
#pragma unroll 4
      for (int k = 0; k < D / 16; ++k)
        mma_ss(tmem + buf * BK, a0 + step_kmajor(k, L::CHUNK_Q), b0 + step_kmajor(k, L::CHUNK_KV), ID_S, k > 0);
    };
    auto issue_pv = [&](int t, int buf, int at, int k0, int k1, bool more) {   // 16 keys each
      const uint64_t b0 = desc_mnmajor(sbase + L::KV + at * L::TILE_KV, L::CHUNK_KV);
#pragma unroll 4
      for (int k = k0; k < k1; ++k)
        mma_ts(tmem + L::COL_O + t * D, tmem + buf * BK + k * 8, b0 + step_mnmajor(k), ID_O, more | (k > 0));
    };
    bool ok = true;
    auto wait = [&](uint32_t b, int parity) {
      if (ok && !mbar_wait(b, parity & 1, abort, status)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    for (int count = 0; ok; ++count) {
      const int ps = count % kPieces;
      if (!wait(bar(B_PIECE_FULL + ps), count / kPieces)) break;
      const int n = pieces[ps].n;
      const bool two = TILES == 2 && pieces[ps].rows > 128;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PIECE_EMPTY + ps));
      if (n == 0) break;
      if (!wait(bar(B_Q_FULL), count) || !wait(full(slot), phase)) break;
      tc_fence_after();
      if (elect_one()) {
        issue_s(0, 0, slot);
        mma_commit(bar(B_S_FULL));
        if (two) {
          issue_s(1, 1, slot);
          mma_commit(bar(B_S_FULL + 1));
        }
        mma_commit(empty(slot));
        if (n == 1) mma_commit(bar(B_Q_EMPTY));
      }
      __syncwarp();
      next_slot();
      if (two) {
        for (int j = 0; ok && j < n; ++j) {
          if (!wait(full(slot), phase)) break;
          const int v_slot = slot;
          next_slot();
          for (int t = 0; t < 2; ++t) {
            if (!wait(bar(B_P_HALF + t), used[t])) break;
            if (j == 0 && freed[t] > 0 && !wait(bar(B_O_FREE + t), freed[t] - 1)) break;
            tc_fence_after();
            if (elect_one()) issue_pv(t, t, v_slot, 0, BK / 32, j > 0);
            __syncwarp();
            if (t == 0 && j + 1 < n && !wait(full(slot), phase)) break;
            if (!wait(bar(B_P_READY + t), used_all[t])) break;
            ++used[t];
            ++used_all[t];
            tc_fence_after();
            if (elect_one()) {
              issue_pv(t, t, v_slot, BK / 32, BK / 16, true);
              if (t == 1) mma_commit(empty(v_slot));
              mma_commit(bar(B_O_DONE + t));
              if (j + 1 == n) mma_commit(bar(B_O_LAST + t));
              if (j + 1 < n) {
                issue_s(t, t, slot);
                mma_commit(bar(B_S_FULL + t));
                if (t == 1) {
                  mma_commit(empty(slot));
                  if (j + 2 == n) mma_commit(bar(B_Q_EMPTY));
                }
              }
            }
            __syncwarp();
          }
          if (j + 1 < n) next_slot();
        }
        ++freed[0];
        ++freed[1];
      } else {
        for (int j = 0; ok && j < n; ++j) {
          if (j + 1 < n) {
            if (!wait(full(slot), phase)) break;
            tc_fence_after();
            if (elect_one()) {
              issue_s(0, (j + 1) & 1, slot);
              mma_commit(bar(B_S_FULL + (j & 1 ? 0 : 2)));
              mma_commit(empty(slot));
              if (j + 2 == n) mma_commit(bar(B_Q_EMPTY));
            }
            __syncwarp();
            next_slot();
          }
          const int buf = j & 1;
          if (!wait(full(slot), phase) || !wait(bar(B_P_READY + 2 * buf), buf ? used_odd : used_all[0])) break;
          if (j == 0 && freed[0] > 0 && !wait(bar(B_O_FREE), freed[0] - 1)) break;
          if (buf) ++used_odd;
          else ++used_all[0];
          tc_fence_after();
          if (elect_one()) {
            issue_pv(0, buf, slot, 0, BK / 16, j > 0);
            mma_commit(empty(slot));
            mma_commit(bar(B_O_DONE));
            if (j + 1 == n) mma_commit(bar(B_O_LAST));
          }
          __syncwarp();
          next_slot();
        }
        ++freed[0];
      }
    }
    // every product issued has to end before the block does, after an abort, too
    if (elect_one()) mma_commit(bar(B_TEARDOWN));
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait(bar(B_TEARDOWN), 0, &no_abort, status);
  } else if (warp >= L::LOAD_WARP && warp < L::MMA_WARP) {
    // ------------------------------------------------------------ loads
    setmaxnreg_to<L::REG_OTHER, L::REG_LAUNCH>();
    constexpr int RPW = BK / L::LOAD_WARPS;  // keys of a block per warp
    constexpr int CPR = D / 8;               // 16-byte pieces per row of a tile
    constexpr int RPI = 32 / CPR;            // rows a warp's instruction covers
    const int w = warp - L::LOAD_WARP;
    int slot = 0, phase = 1;                 // of the ring: the first pass finds every slot empty
    uint32_t pending[kLag] = {};             // barriers of the copies in flight, oldest last (0: none)
    int block = 0, raw_in = 0, raw_out = 0;  // blocks of keys so far; places in the ring of cached rows
    int tiles = 0;                           // so far
    bool ok = true;
    auto wait = [&](uint32_t b, int parity) {
      if (ok && !mbar_wait(b, parity & 1, abort, status)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    auto arrive = [&](uint32_t b) {          // this warp's part is there
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    // Copies of this warp have been issued (or, with 0, none); those kLag before them have landed.
    auto issued = [&](uint32_t b) {
      cp_commit();
      cp_wait<kLag>();
      if (pending[kLag - 1]) arrive(pending[kLag - 1]);
#pragma unroll
      for (int i = kLag - 1; i > 0; --i) pending[i] = pending[i - 1];
      pending[0] = b;
    };
    auto drain = [&] {
      cp_wait<0>();
#pragma unroll
      for (int i = kLag - 1; i >= 0; --i) {
        if (pending[i]) arrive(pending[i]);
        pending[i] = 0;
      }
    };
    auto next_slot = [&] {
      ++tiles;
      if (++slot == NS) {
        slot = 0;
        phase ^= 1;
      }
    };
    if (!E4M3 && p.box_rows > 0 && lane == 0) {
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
    }
    for (int count = 0; ok; ++count) {
      const int ps = count % kPieces;
      if (!wait(bar(B_PIECE_FULL + ps), count / kPieces)) break;
      const Piece u = pieces[ps];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PIECE_EMPTY + ps));
      if (u.n == 0) break;
      const int32_t* const table = p.table + u.b * p.table_stride;
      const int last_page = u.key_hi > 0 ? p.page_div.quotient(u.key_hi - 1) : -1;
      auto page_of = [&](int kb) {   // of this lane's key
        const int key = kb * BK + w * RPW + lane;
        const int pi = p.page_div.quotient(key);
        return pi <= last_page && lane < RPW ? table[pi] : -1;
      };
      int page = E4M3 && p.box_rows > 0 ? -1 : page_of(u.kb0);
      // Where this lane's key is (of the block at hand, and of the one before), and
      // which keys of the warp are there.
      int at_page[2] = {0, 0}, at_slot[2] = {0, 0};
      unsigned good[2] = {0, 0};
      auto locate = [&](int kb) {
        good[1] = good[0];
        at_page[1] = at_page[0];
        at_slot[1] = at_slot[0];
        const int key = kb * BK + w * RPW + lane;
        const bool in = lane < RPW && key >= u.key_lo && key < u.key_hi;
        const bool there = in && page >= 0 && page < p.kv.num_pages;
        at_page[0] = page;
        at_slot[0] = key - p.page_div.quotient(key) * p.kv.page_size;
        good[0] = __ballot_sync(0xffffffffu, there);
        const unsigned missing = __ballot_sync(0xffffffffu, in && !there);
        if (lane == 0) {   // RPW bits of the block's
          if constexpr (RPW == 32) marks[(block % kMarks) * 4 + w] = missing;
          else if constexpr (RPW == 16) reinterpret_cast<uint16_t*>(marks)[(block % kMarks) * 8 + w] = missing;
          else reinterpret_cast<uint8_t*>(marks)[(block % kMarks) * 16 + w] = missing;
        }
        ++block;
        page = page_of(kb + 1);
      };
      auto offset = [&](int old) {   // elements of the cache; of keys that are there
        return static_cast<long long>(old ? at_page[1] : at_page[0]) * p.kv.page_stride +
               (old ? at_slot[1] : at_slot[0]) * p.kv.slot_stride + u.head_kv * p.kv.head_stride;
      };
      const bool two = TILES == 2 && u.rows > 128;
      int located = 0;

      if constexpr (!E4M3) {
        for (int e = 0; ok && e < 2 * u.n; ++e) {
          const bool key = is_key(e, u.n, two);
          if (key) locate(u.kb0 + located++);
          const int old = !key && is_old(e, u.n, two);
          if (!wait(empty(slot), phase)) break;
          const uint32_t tile = sbase + L::KV + slot * L::TILE_KV;
          const unsigned have_rows = old ? good[1] : good[0];
          if (p.box_rows > 0 && (key || have_rows == (RPW == 32 ? 0xffffffffu : (1u << RPW) - 1))) {
            // Boxes of box_rows keys, a lane each.  Scores of keys that a row does not
            // see are replaced, so it does not matter what is read for them (pages
            // that are none read as zeros); their values have to be zeros.
            if (lane == 0) mbar_arrive_expect_tx(full(slot), RPW * D * 2);
            __syncwarp();
            if (lane < RPW && (lane & (p.box_rows - 1)) == 0) {
              const int pg = old ? at_page[1] : at_page[0], sl = old ? at_slot[1] : at_slot[0];
              const int in = pg >= 0 && pg < p.kv.num_pages ? pg : p.kv.num_pages;
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(tile + c * L::CHUNK_KV + (w * RPW + lane) * 128, key ? &p.tm_k : &p.tm_v, c * 64, u.head_kv, sl,
                            in, full(slot));
            }
            __syncwarp();
            issued(0);
          } else {
            const uint16_t* const from = static_cast<const uint16_t*>(key ? p.kv.k : p.kv.v);
            const long long mine = offset(old);
#pragma unroll 4
            for (int i = 0; i < RPW / RPI; ++i) {
              const int lr = i * RPI + lane / CPR, c = lane % CPR, rr = w * RPW + lr;
              const long long o = __shfl_sync(0xffffffffu, mine, lr);
              const bool have = have_rows >> lr & 1;
              cp_async16(tile + (c >> 3) * L::CHUNK_KV + rr * 128 + (((c & 7) ^ (rr & 7)) << 4),
                         have ? from + o + c * 8 : p.q, have);
            }
            issued(full(slot));
          }
          next_slot();
        }
        drain();   // the products to come wait for them, and these loads for the products
      } else {
        constexpr int CP8 = D / 16, RP8 = 32 / CP8;   // pieces per cached row, rows per step
        // N rows of a tile, from row0 on, from the ring of cached rows as fp16; zeros where
        // `have` says so (of values that no row sees, whatever is in their slots).
        auto convert = [&](auto rows, uint32_t raw, uint32_t tile, int row0, unsigned have) {
          constexpr int N = decltype(rows)::value, STEPS = N / RP8, NB = STEPS < 4 ? STEPS : 4;   // NB loads in flight
          const bool all = (~have & (0xffffffffu >> (32 - N))) == 0;
          const int c = 2 * (lane % CP8);
#pragma unroll 1
          for (int i0 = 0; i0 < STEPS; i0 += NB) {
            uint4 v[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i)
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                           : "r"(raw + row0 * D + ((i0 + i) * 32 + lane) * 16)
                           : "memory");
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              const int lr = (i0 + i) * RP8 + lane / CP8, rr = row0 + lr;
              if (!all && !(have >> lr & 1)) v[i] = make_uint4(0, 0, 0, 0);
              const uint2 a = e4m3x4_f16(v[i].x), b = e4m3x4_f16(v[i].y), f = e4m3x4_f16(v[i].z), g = e4m3x4_f16(v[i].w);
              const uint32_t row = tile + (c >> 3) * L::CHUNK_KV + rr * 128;
              st_shared_v4(row + (((c & 7) ^ (rr & 7)) << 4), a.x, a.y, b.x, b.y);
              st_shared_v4(row + ((((c & 7) + 1) ^ (rr & 7)) << 4), f.x, f.y, g.x, g.y);
            }
          }
        };
        // This warp's share of Q, which the query warps have brought
        auto convert_q = [&] {
          if constexpr (L::LOADERS_CONVERT_Q) {
            if (!wait(bar(B_Q_RAW), count)) return;
            convert_queries<D, 2>(sbase + L::Q, q_scale + (count & 1) * ROWS, u.rows, w, L::LOAD_WARPS, lane);
            arrive(bar(B_Q_FULL));
          }
        };
        if (boxed) {
          // The walker fills the ring; group `mine` of four warps takes every GROUPS-th tile:
          // a tile's waits and fences come half as often to each of two.  (With four warps in
          // all it does not pay: 64 requests of 1 to 8 tokens, 32 / 8 heads of 64, 108 us, and
          // 125 as two pairs; with eight, 24 chunks over heads of 256, 115 us and 99 in groups.)
          constexpr int N = BK / 4, GROUPS = L::LOAD_WARPS / 4;
          const int mine = w / 4, row0 = w % 4 * N;
          if (mine > 0) convert_q();
#pragma unroll 1
          for (int e = mine; ok && e < 2 * u.n; e += GROUPS) {
            const int i = tiles + e, at = i % NS, raw_at = i % NR;
            if (!wait(landed(raw_at), i / NR) || !wait(empty(at), i / NS + 1)) break;
            unsigned have = 0xffffffffu;
            if (!is_key(e, u.n, two)) {
              // rows [key_lo, key_hi) of this warp's, without missing pages
              const int j = two ? e / 2 : e + 1 == 2 * u.n ? u.n - 1 : e / 2 - 1, k0 = (u.kb0 + j) * BK + row0;
              const int a = min(max(u.key_lo - k0, 0), N), b = min(max(u.key_hi - k0, 0), N);
              have = a < b ? (0xffffffffu >> (32 - (b - a))) << a : 0u;
              have &= ~(marks[((block + j) % kMarks) * 4 + row0 / 32] >> row0 % 32);
            }
            convert(std::integral_constant<int, N>(), sbase + L::RAW + raw_at * L::TILE_RAW, sbase + L::KV + at * L::TILE_KV, row0, have);
            arrive(full(at));
            if (lane == 0) mbar_arrive(taken(raw_at));
            if (e == 0) convert_q();
          }
          tiles += 2 * u.n;
          block += u.n;
        } else {
          // Every thread copies the pieces that it later converts, NR tiles ahead.
          constexpr int N8 = RPW / RP8;   // steps
          const uint32_t raw = sbase + L::RAW + w * (RPW * D);
          int staged = 0;
          unsigned rows_in[NR];   // which rows of the tiles on their way are there, newest first
          auto stage = [&] {
            unsigned have_rows = 0;
            if (staged < 2 * u.n) {
              const int e = staged++;
              const bool key = is_key(e, u.n, two);
              if (key) locate(u.kb0 + located++);
              const int old = !key && is_old(e, u.n, two);
              have_rows = old ? good[1] : good[0];
              const uint32_t to = raw + raw_in * L::TILE_RAW + lane * 16;
              const uint8_t* const from = static_cast<const uint8_t*>(key ? p.kv.k : p.kv.v);
              const long long mine = offset(old);
#pragma unroll
              for (int i = 0; i < N8; ++i) {
                const int lr = i * RP8 + lane / CP8, c = lane % CP8;
                const long long o = __shfl_sync(0xffffffffu, mine, lr);
                const bool have = have_rows >> lr & 1;
                cp_async16(to + i * 512, have ? static_cast<const void*>(from + o + c * 16) : p.q, have);
              }
              raw_in = raw_in + 1 == NR ? 0 : raw_in + 1;
            }
            cp_commit();
#pragma unroll
            for (int i = NR - 1; i > 0; --i) rows_in[i] = rows_in[i - 1];
            rows_in[0] = have_rows;
          };
#pragma unroll 1
          for (int i = 0; i < NR; ++i) stage();
          convert_q();
#pragma unroll 1
          for (int e = 0; ok && e < 2 * u.n; ++e) {
            cp_wait<NR - 1>();
            if (!wait(empty(slot), phase)) break;
            convert(std::integral_constant<int, RPW>(), sbase + L::RAW + raw_out * L::TILE_RAW, sbase + L::KV + slot * L::TILE_KV,
                    w * RPW, rows_in[NR - 1]);
            arrive(full(slot));
            next_slot();
            raw_out = raw_out + 1 == NR ? 0 : raw_out + 1;
            stage();
          }
        }
      }
    }
    cp_wait<0>();
    if (!ok) {   // after an abort, what has been asked for lands before the block ends
      volatile int no_abort = 0;
      if constexpr (!E4M3)
        for (int i = max(0, tiles - NS); i < tiles; ++i)
          mbar_wait(full(i % NS), (i / NS) & 1, &no_abort, status, 100000000ull);
    }
  } else if (warp < 4 * TILES) {
    // ------------------------------------------------------------ softmax and output
    setmaxnreg_to<L::REG_SOFTMAX, L::REG_LAUNCH>();
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                 // row of the tile (TMEM lane)
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lane_addr + L::COL_O + t * D;
    constexpr float kShift = E4M3 ? kF16Shift : 0.f;
    // phases seen of S_FULL, of its third, of O_DONE, of O_LAST; blocks
    int s_used = 0, s_odd = 0, o_used = 0, done = 0, block = 0;
    // Rows that belong to no request, while there is nothing else to do.
    {
      const int first = min(max(p.cu_new[p.batch], 0), p.num_tokens);
      const long long n16 = static_cast<long long>(p.num_tokens - first) * p.heads * (D / 8);
#pragma unroll 1
      for (long long i = static_cast<long long>(blockIdx.x) * (128 * TILES) + threadIdx.x; i < n16;
           i += static_cast<long long>(gridDim.x) * (128 * TILES)) {
        const long long row = static_cast<long long>(first) * p.heads + i / (D / 8);
        *reinterpret_cast<uint4*>(p.o + row * D + i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
        if (p.lse && i % (D / 8) == 0) p.lse[row] = -INFINITY;
      }
    }
    bool ok = true;
    for (int count = 0; ok; ++count) {
      const int ps = count % kPieces;
      ok = mbar_wait(bar(B_PIECE_FULL + ps), (count / kPieces) & 1, abort, status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const Piece u = pieces[ps];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PIECE_EMPTY + ps));
      if (u.n == 0) break;
      const bool two = TILES == 2 && u.rows > 128;
      if (t == 1 && !two) {   // the first tile's warps take both score buffers
        block += u.n;
        continue;
      }
      const int row = u.row_first + t * 128 + r, tok = p.group_div.quotient(row);
      const bool valid = t * 128 + r < u.rows;
      const int pos = u.pos0 + tok;
      // Visible keys [lo, hi), and of the warp's rows the largest lo and the smallest
      // hi; rows past the unit's are computed like any and not written.
      const int hi = valid ? pos + 1 : 0x7fffffff;
      const int lo = valid && p.window > 0 ? max(max(pos, 0) - p.window + 1, 0) : 0;
      const int lo_most = __reduce_max_sync(0xffffffffu, lo), hi_least = __reduce_min_sync(0xffffffffu, hi);
      const float k_scale = E4M3 && p.kv.k_scale ? p.kv.k_scale[u.head_kv] : 1.f;
      float sl2 = 0.f;   // set once Q is there
      float m_used = -INFINITY, l_run = 0.f;
      for (int j = 0; j < u.n; ++j, ++block) {
        const bool odd = !two && (j & 1);
        const int which = odd ? 2 : t;   // barrier
        const uint32_t t_s = tmem + lane_addr + (odd ? 1 : t) * BK;
        if (!mbar_wait(bar(B_S_FULL + which), (odd ? s_odd : s_used) & 1, abort, status)) ok = false;
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (odd) ++s_odd;
        else ++s_used;
        tc_fence_after();
        float x[BK];
#pragma unroll
        for (int c = 0; c < BK / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(t_s + c * 32, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) x[c * 32 + e] = __uint_as_float(v[e]);
        }
        if (j == 0) {
          sl2 = p.scale * k_scale * kLog2e;
          if constexpr (E4M3) sl2 *= q_scale[(count & 1) * ROWS + t * 128 + r];
        }
        const uint4 missing = *reinterpret_cast<const uint4*>(marks + (block % kMarks) * 4);
        const int key0 = (u.kb0 + j) * BK;
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < BK; ++e) asm volatile("" : "+f"(x[e]));   // no use before the wait
        // a = x sl2 - ref; P = 2^a
        {
          const float ref = (m_used == -INFINITY ? 0.f : m_used) - kShift;
          const float2 mul = make_float2(sl2, sl2), sub = make_float2(-ref, -ref);
#pragma unroll
          for (int e = 0; e < BK; e += 2) {
            const float2 a = fma2(make_float2(x[e], x[e + 1]), mul, sub);
            x[e] = a.x;
            x[e + 1] = a.y;
          }
        }
        if (key0 < lo_most || key0 + BK > hi_least || (missing.x | missing.y | (BK == 128 ? missing.z | missing.w : 0u))) {
          const int c_lo = max(lo - key0, 0), c_hi = min(max(hi - key0, 0), BK);
          const uint32_t words[4] = {missing.x, missing.y, missing.z, missing.w};
#pragma unroll
          for (int c = 0; c < BK / 32; ++c) {
            // columns [c_lo, c_hi) but the missing ones, of these 32
            const int from = min(max(c_lo - 32 * c, 0), 32), to = min(max(c_hi - 32 * c, 0), 32);
            uint32_t seen = from < to ? (0xffffffffu >> (32 - (to - from))) << from : 0u;
            seen &= ~words[c];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[c * 32 + e] = seen >> e & 1 ? x[c * 32 + e] : -INFINITY;
          }
        }
        // The reference is that of the blocks before: floating-point weights may be
        // far above 1.  It moves only where a row has none yet and where its weights
        // would grow past kMostSum or 2^kMostLog: then, rarely, the largest a
        // is looked for and the first half is worked out again.  So the exponentials
        // wait for no maximum.
        float sum = 0.f;
        const float m_old = m_used;
        bool fresh = valid && m_used == -INFINITY;
        auto half = [&](auto h) {   // weights of half the block, into the place of the scores
          float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
          for (int c = decltype(h)::value * BK / 64; c < (decltype(h)::value + 1) * BK / 64; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 w = make_float2(ex2_approx(x[c * 32 + 2 * e]), ex2_approx(x[c * 32 + 2 * e + 1]));
              if (e & 1) sum1 = add2(sum1, w);
              else sum0 = add2(sum0, w);
              pk[e] = E4M3 ? pack_f16x2(w.x, w.y) : pack_bf16x2(w.x, w.y);
            }
            tmem_st16(t_s + c * 16, pk);
          }
          return (sum0.x + sum0.y) + (sum1.x + sum1.y);
        };
        float rest0 = x[BK / 2], rest1 = x[BK / 2 + 1];   // largest a of the second half
#pragma unroll
        for (int e = BK / 2 + 2; e < BK; e += 4) {
          rest0 = fmaxf(fmaxf(x[e], x[e + 1]), rest0);
          if (e + 2 < BK) rest1 = fmaxf(fmaxf(x[e + 2], x[e + 3]), rest1);
        }
        for (int round = 0;; ++round) {
          sum = half(std::integral_constant<int, 0>());
          const bool move = valid && (fresh || !(sum <= kMostSum) || fmaxf(rest0, rest1) > kMostLog);
          // (a reference in the 2^30s is off by more than the range allows for: a few rounds)
          if (!__any_sync(0xffffffffu, move) || round == 4) break;
          float top = x[0];
#pragma unroll
          for (int e = 1; e < BK - 1; e += 2) top = fmaxf(fmaxf(x[e], x[e + 1]), top);
          top = fmaxf(top, x[BK - 1]) - kShift;
          const float by = move && top > -INFINITY ? top : 0.f;
          if (move && top > -INFINITY) m_used = (m_used == -INFINITY ? 0.f : m_used) + top;
#pragma unroll
          for (int e = 0; e < BK; ++e) x[e] -= by;
          rest0 -= by;
          rest1 -= by;
          fresh = false;
        }
        const bool grow = m_used != m_old;
        const float alpha = grow ? ex2_approx(m_old - m_used) : 1.f;   // 0 from -inf
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
          if (!mbar_wait(bar(B_O_DONE + t), (o_used + j - 1) & 1, abort, status)) ok = false;
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t v[16];
            tmem_ld16(t_o + c * 16, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
            tmem_st16(t_o + c * 16, v);
          }
        }
        if (two) {   // the products of the first half's keys can start
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_P_HALF + t));
        }
        l_run = fmaf(l_run, alpha, sum + half(std::integral_constant<int, 1>()));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P_READY + which));
      }
      if (!ok) break;
      // ------------------------------------------------------------ output
      if (!mbar_wait(bar(B_O_LAST + t), done++ & 1, abort, status)) ok = false;
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      o_used += u.n;
      tc_fence_after();
      const float top = m_used - kShift;   // what l_run and O are relative to
      if (u.part == 0) {
        const float v_scale = E4M3 && p.kv.v_scale ? p.kv.v_scale[u.head_kv] : 1.f;
        const float inv = l_run == 0.f ? 0.f : v_scale / l_run;
        const long long out = static_cast<long long>(u.token0 + tok) * p.heads + u.head_kv * group + (row - tok * group);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(t_o + c * 32, v);
          tmem_ld_wait();
          if (valid) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pk[e] = l_run == 0.f ? 0u
                                   : pack_bf16x2(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
            uint4* const to = reinterpret_cast<uint4*>(p.o + out * D + c * 32);
#pragma unroll
            for (int g = 0; g < 4; ++g) to[g] = make_uint4(pk[4 * g], pk[4 * g + 1], pk[4 * g + 2], pk[4 * g + 3]);
          }
        }
        if (valid && p.lse) p.lse[out] = l_run == 0.f ? -INFINITY : (top + log2f(l_run)) * kLn2;
      } else {
        float* const part = parts_of(p.work, gridDim.x) +
                            (static_cast<size_t>(blockIdx.x) * 2 + u.part - 1) * part_floats(ROWS, D);
        const int at = t * 128 + r;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(t_o + c * 32, v);
          tmem_ld_wait();
          if (valid) {
#pragma unroll
            for (int g = 0; g < 8; ++g)
              *reinterpret_cast<uint4*>(part + (static_cast<size_t>(c * 8 + g) * ROWS + at) * 4) =
                  make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
          }
        }
        if (valid) {
          part[static_cast<size_t>(ROWS) * D + at] = top;
          part[static_cast<size_t>(ROWS) * (D + 1) + at] = l_run;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_O_FREE + t));
    }
  } else if (warp >= L::Q_WARP) {
    // ------------------------------------------------------------ queries
    setmaxnreg_to<L::REG_OTHER, L::REG_LAUNCH>();
    constexpr int CPR = D / 8;               // 16-byte pieces per row
    constexpr int RPI = 32 / CPR;            // rows a warp's instruction covers
    const int w = warp - L::Q_WARP;
    bool ok = true;
    int asked = 0;
    for (int count = 0; ok; ++count) {
      const int ps = count % kPieces;
      ok = mbar_wait(bar(B_PIECE_FULL + ps), (count / kPieces) & 1, abort, status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const Piece u = pieces[ps];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PIECE_EMPTY + ps));
      if (u.n == 0) break;
      const int tiles = TILES == 2 && u.rows > 128 ? 2 : 1;
      if (count > 0) {
        ok = mbar_wait(bar(B_Q_EMPTY), (count - 1) & 1, abort, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
      }
      const uint32_t q_there = bar(E4M3 ? B_Q_RAW : B_Q_FULL);   // queries to be made fp16 get there first
      if (p.q_boxes) {
        // 128 rows are whole tokens: a box of the group's heads for 128 / group tokens
        if (lane == 0) {
          if (w == 0) {
            mbar_arrive_expect_tx(q_there, tiles * L::TILE_Q);
            for (int t = 0; t < tiles; ++t)
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(sbase + L::Q + t * L::TILE_Q + c * L::CHUNK_Q, &p.tm_q, c * 64, u.head_kv * group,
                            u.token0 + p.group_div.quotient(u.row_first + t * 128), q_there);
          } else {
            mbar_arrive(q_there);
          }
        }
        asked = count + 1;
      }
#pragma unroll 1
      for (int r0 = w * 32; !p.q_boxes && r0 < u.rows; r0 += 64) {
        const int r = r0 + lane, row = u.row_first + r, tok = p.group_div.quotient(row);
        const long long from = (u.token0 + tok) * p.q_row_stride + (u.head_kv * group + row - tok * group) * D;
        const unsigned valid = __ballot_sync(0xffffffffu, r < u.rows);
#pragma unroll 4
        for (int i = 0; i < 32 / RPI; ++i) {
          const int lr = i * RPI + lane / CPR, c = lane % CPR, rr = r0 + lr;
          const long long o = __shfl_sync(0xffffffffu, from, lr);
          const bool have = valid >> lr & 1;
          const uint32_t dst = sbase + L::Q + (rr >> 7) * L::TILE_Q + (c >> 3) * L::CHUNK_Q + (rr & 127) * 128 +
                               (((c & 7) ^ (rr & 7)) << 4);
          cp_async16(dst, p.q + (have ? o + c * 8 : 0), have);
        }
      }
      if (!p.q_boxes) {
        cp_commit();
        cp_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_there);
      }
      if constexpr (E4M3 && !L::LOADERS_CONVERT_Q) {
        ok = mbar_wait(q_there, count & 1, abort, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        convert_queries<D, 4>(sbase + L::Q, q_scale + (count & 1) * ROWS, u.rows, w, 2, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_Q_FULL));
      }
    }
    if (!ok && asked > 0) {   // after an abort, what has been asked for lands before the block ends
      volatile int no_abort = 0;
      mbar_wait(bar(E4M3 ? B_Q_RAW : B_Q_FULL), (asked - 1) & 1, &no_abort, status, 100000000ull);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == L::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ join
// Block (run, 32 rows): joins the partial results of the unit that run `run`
// starts and later runs go on with.  A lane per row, a warp for some columns.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const ExtendParams p, int blocks) {
  constexpr int ROWS = Shape<D>::kRows, WARPS = kJoinThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, at = blockIdx.y * 32 + lane, run = blockIdx.x;
  pdl_wait();
  const Cut cut = reinterpret_cast<const Cut*>(p.work)[run];
  if (cut.row_first + static_cast<int>(blockIdx.y) * 32 >= cut.row_end) return;
  const bool valid = cut.row_first + at < cut.row_end;
  const float* const parts = parts_of(p.work, blocks);
  auto part = [&](int i) {   // of run `run + i`
    return parts + (static_cast<size_t>(run + i) * 2 + (i == 0 ? 1 : 0)) * part_floats(ROWS, D);
  };
  const int n = cut.last - run + 1;
  // kAhead partial results in flight, relative to a running maximum
  constexpr int kAhead = D == 256 ? 2 : 4, COLS = D / 4 / WARPS;
  float top = -INFINITY, sum = 0.f;
  float4 acc[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; valid && i0 < n; i0 += kAhead) {
    float m[kAhead], l[kAhead];
    float4 v[kAhead][COLS];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const float* const q = part(min(i0 + a, n - 1));
      m[a] = q[static_cast<size_t>(ROWS) * D + at];
      l[a] = i0 + a < n ? q[static_cast<size_t>(ROWS) * (D + 1) + at] : 0.f;
#pragma unroll
      for (int c = 0; c < COLS; ++c)
        v[a][c] = *reinterpret_cast<const float4*>(q + (static_cast<size_t>(c * WARPS + warp) * ROWS + at) * 4);
    }
    float up = top;
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (l[a] != 0.f) up = fmaxf(up, m[a]);
    const float keep = up == top ? 1.f : ex2_approx(top - up);
    top = up;
    sum *= keep;
#pragma unroll
    for (int c = 0; c < COLS; ++c) acc[c].x *= keep, acc[c].y *= keep, acc[c].z *= keep, acc[c].w *= keep;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (l[a] == 0.f) continue;   // nothing seen: what is there does not count
      const float f = ex2_approx(m[a] - top);
      sum = fmaf(f, l[a], sum);
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        acc[c].x = fmaf(f, v[a][c].x, acc[c].x);
        acc[c].y = fmaf(f, v[a][c].y, acc[c].y);
        acc[c].z = fmaf(f, v[a][c].z, acc[c].z);
        acc[c].w = fmaf(f, v[a][c].w, acc[c].w);
      }
    }
  }
  if (!valid) return;
  const int group = p.heads / p.kv.heads_kv, row = cut.row_first + at, tok = p.group_div.quotient(row);
  const long long out = static_cast<long long>(cut.token0 + tok) * p.heads + cut.head_kv * group + (row - tok * group);
  const float v_scale = p.kv.v_scale ? p.kv.v_scale[cut.head_kv] : 1.f;
  const float inv = sum == 0.f ? 0.f : v_scale / sum;
#pragma unroll
  for (int c = 0; c < COLS; ++c)
    *reinterpret_cast<uint2*>(p.o + out * D + (c * WARPS + warp) * 4) =
        make_uint2(pack_bf16x2(acc[c].x * inv, acc[c].y * inv), pack_bf16x2(acc[c].z * inv, acc[c].w * inv));
  if (p.lse && warp == 0) p.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// The cache as [pages, page_size, heads, d], boxes of rows slots by 64 values of a
// head, swizzled as the products read them, or (8-bit caches) by the whole head.
bool make_page_map(CUtensorMap* m, const PagedCache& c, const void* base, int rows) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  // strides of dimensions of one are never used, but have to be valid ones
  auto stride = [&](long long elements, int n) { return static_cast<cuuint64_t>(n > 1 ? (c.e4m3 ? 1 : 2) * elements : 16); };
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.heads_kv),
                              static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {stride(c.head_stride, c.heads_kv), stride(c.slot_stride, c.page_size),
                                 stride(c.page_stride, c.num_pages)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(c.e4m3 ? c.head_dim : 64), 1, static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  // What a miss brings into the L2: no more than a head's row, since the next head's is
  // read by another SM, much later (64 requests of 4 tokens over 8192 keys, 32 / 8 heads
  // of 64: 261 us with 256 bytes, 221 so).
  const int row = c.head_dim * (c.e4m3 ? 1 : 2);   // bytes
  const auto promotion = row >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                         : row >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                      : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  return enc(m, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
             dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             c.e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, promotion,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as [tokens, heads, d], boxes of 128 rows by 64 values.
bool make_query_map(CUtensorMap* m, const ExtendParams& p, int group) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.kv.head_dim), static_cast<cuuint64_t>(p.heads),
                              static_cast<cuuint64_t>(p.num_tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * p.kv.head_dim),
                                 static_cast<cuuint64_t>(2 * (p.num_tokens > 1 ? p.q_row_stride : p.heads * p.kv.head_dim))};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(128 / group)}, steps[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, steps,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E4M3>
cudaError_t launch_dim(ExtendParams p, const Device& dev, cudaStream_t s) {
  using L = Layout<D, E4M3>;
  using S = Shape<D>;
  const long long group = p.heads / p.kv.heads_kv;
  const long long keys = static_cast<long long>(p.max_pages) * p.kv.page_size + p.num_tokens;   // as the costs have it
  p.tile_keys16 = static_cast<int>(S::kRows * 16 / group);
  p.tile_tokens = static_cast<int>(S::kRows / group + 1);
  p.cost_shift = cost_shift(most_units(p.num_tokens, p.batch, p.heads, p.kv.heads_kv, D), keys, S::kKeys == 128 ? 7 : 6);
  // Boxes of the largest power of two that divides a page, up to a warp's keys (8-bit
  // caches: a block's).  Without boxes, 16 bytes a thread at a time: 64 requests of 1 to
  // 8 tokens 116 us instead of 105, chunks of 2048 985 instead of 909, 24 chunks over
  // e4m3 heads of 256 132 instead of 99.  Boxes of less than 8 rows would be smaller than
  // the swizzle's pattern.
  p.box_rows = 0;
  const long long most = std::max({p.kv.page_stride, p.kv.slot_stride, p.kv.head_stride});
  if (p.kv.page_size % 8 == 0 && p.max_pages > 0 && most < (1ll << 39)) {
    int rows = 8;
    while (rows < (E4M3 ? S::kKeys : S::kKeys / L::LOAD_WARPS) && p.kv.page_size % (2 * rows) == 0) rows *= 2;
    if (!make_page_map(&p.tm_k, p.kv, p.kv.k, rows) || !make_page_map(&p.tm_v, p.kv, p.kv.v, rows))
      return cudaErrorInvalidValue;
    p.box_rows = rows;
  }
  // Queries in boxes where 128 rows are whole tokens (37 ragged requests with a window of
  // 1024, 16 heads of 64: 94 us without, 83 with).
  p.q_boxes = 0;
  if (group <= 128 && (group & (group - 1)) == 0 && p.q_row_stride < (1ll << 39)) {
    if (!make_query_map(&p.tm_q, p, static_cast<int>(group))) return cudaErrorInvalidValue;
    p.q_boxes = 1;
  }
  static std::atomic<unsigned long long> done{0}, join_done{0};
  auto* const kernel = extend_kernel<D, E4M3>;
  cudaError_t e = prepare_once(reinterpret_cast<const void*>(kernel), L::BYTES, dev.id, done);
  if (e != cudaSuccess) return e;
  const int blocks = dev.sms < kMaxSms ? dev.sms : kMaxSms;
  e = launch_pdl(kernel, dim3(blocks), dim3(L::THREADS), L::BYTES, s, p);
  if (e != cudaSuccess) return e;
  // units of one block are never cut
  if (static_cast<long long>(p.max_pages) * p.kv.page_size <= L::BK) return e;
  e = prepare_once(reinterpret_cast<const void*>(join_kernel<D>), 0, dev.id, join_done);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_kernel<D>, dim3(blocks, Shape<D>::kRows / 32), dim3(kJoinThreads), 0, s, p, blocks);
}

}  // namespace
}  // namespace extend

cudaError_t launch_extend(const ExtendParams& p, const Device& dev, cudaStream_t s) {
  using namespace extend;
  if (p.kv.e4m3)
    return p.kv.head_dim == 64    ? launch_dim<64, true>(p, dev, s)
           : p.kv.head_dim == 128 ? launch_dim<128, true>(p, dev, s)
                                  : launch_dim<256, true>(p, dev, s);
  return p.kv.head_dim == 64    ? launch_dim<64, false>(p, dev, s)
         : p.kv.head_dim == 128 ? launch_dim<128, false>(p, dev, s)
                                : launch_dim<256, false>(p, dev, s);
}

cudaError_t extend_status_word(int** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_extend_status); }

int extend_read_and_clear_status(cudaStream_t s, int* status) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(status, g_extend_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_extend_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return static_cast<int>(e);
}

}  // namespace fa
