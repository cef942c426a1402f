// Paged key/value cache: C entry points (those of decode and extend, too), and
// the kernels that give new tokens their places in the cache (plan) and write
// them there (append).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/fabwd.h"
#include "checks.h"
#include "extend.h"
#include "internal.h"
#include "paged.h"
#include "quantise.cuh"

namespace {

using namespace fa;

// ---------------------------------------------------------------- plan
constexpr int kPlanMaxThreads = 1024;

struct PlanParams {
  int32_t* table;
  long long table_stride;
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* new_lens;
  const int32_t* free_pages;
  int num_free;
  const int32_t* free_start;
  int page_size;
  fa::FastDiv page_div;
  int batch;
  int num_tokens;
  int64_t* slots;
  int32_t* positions;
  int32_t* cu_new;
  int32_t* seq_lens_out;
  int32_t* free_next;
};

__device__ __forceinline__ int clamp_int(long long x) {
  return static_cast<int>(x > 0x7fffffffll ? 0x7fffffffll : x);
}

struct Request {
  int seq, fresh;     // tokens cached, tokens new
  int have, take;     // pages held, pages to take
};

__device__ __forceinline__ Request load_request(const PlanParams& p, int b) {
  Request r;
  r.seq = max(*(p.seq_lens + b), 0);
  r.fresh = max(*(p.new_lens + b), 0);
  const int after = clamp_int(static_cast<long long>(r.seq) + r.fresh);
  // ceil(n / page_size) of n >= 0
  const int have = r.seq ? p.page_div.quotient(r.seq - 1) + 1 : 0;
  const int need = after ? p.page_div.quotient(after - 1) + 1 : 0;
  r.have = min(have, p.max_pages);
  r.take = min(need, p.max_pages) - r.have;
  return r;
}

// Sums over the lanes up to and including this one.
__device__ __forceinline__ void warp_scan(long long& a, long long& b) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
    if (static_cast<int>(threadIdx.x & 31) >= off) {
      a += x;
      b += y;
    }
  }
}

// Every block sums the requests' new tokens and pages itself (a block scan
// over runs of consecutive requests, one run per thread), then places its
// own tokens; block 0 also writes what there is one of per request.  Nothing
// is passed between blocks, so one launch is enough.  Bound by launch and
// memory latency, that of the kernel's own instructions included, so its loops
// are not unrolled (3 to 5 % of the call): 64 requests 2.2 us, 2048 requests
// 4.5 us, 74k tokens of 32 prompts 2.4 us.
__global__ void __launch_bounds__(kPlanMaxThreads) plan_kernel(const PlanParams p) {
  __shared__ long long run_tok[kPlanMaxThreads + 1];   // new tokens before each thread's run
  __shared__ long long run_page[kPlanMaxThreads + 1];  // pages taken before it
  __shared__ long long warp_tok[32], warp_page[32];
  const int t = threadIdx.x, threads = blockDim.x, warp = t >> 5, lane = t & 31;
  fa::pdl_wait();
  const int per = (p.batch + threads - 1) / threads;
  const int b0 = min(t * per, p.batch), b1 = min(b0 + per, p.batch);
  const long long start = p.free_start ? max(*(p.free_start), 0) : 0;
  long long tok = 0, page = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const Request r = load_request(p, b);
    tok += r.fresh;
    page += r.take;
  }
  warp_scan(tok, page);
  if (lane == 31) {
    warp_tok[warp] = tok;
    warp_page[warp] = page;
  }
  __syncthreads();
  if (warp == 0) {
    long long a = lane < threads / 32 ? warp_tok[lane] : 0, c = lane < threads / 32 ? warp_page[lane] : 0;
    warp_scan(a, c);
    warp_tok[lane] = a;
    warp_page[lane] = c;
  }
  __syncthreads();
  if (warp > 0) {
    tok += warp_tok[warp - 1];
    page += warp_page[warp - 1];
  }
  run_tok[t + 1] = tok;
  run_page[t + 1] = page;
  if (t == 0) run_tok[0] = run_page[0] = 0;
  __syncthreads();
  if (blockIdx.x == 0) {
    long long at = run_tok[t];
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int seq = max(*(p.seq_lens + b), 0), fresh = max(*(p.new_lens + b), 0);
      p.cu_new[b] = clamp_int(at);
      p.seq_lens_out[b] = clamp_int(static_cast<long long>(seq) + fresh);
      at += fresh;
    }
    if (t == 0) {
      p.cu_new[p.batch] = clamp_int(run_tok[threads]);
      *p.free_next = clamp_int(start + run_page[threads]);
    }
  }
  const long long total = run_tok[threads];
#pragma unroll 1
  for (long long i = static_cast<long long>(blockIdx.x) * threads + t; i < p.num_tokens;
       i += static_cast<long long>(gridDim.x) * threads) {
    long long slot = -1;
    int pos = 0;
    if (i < total) {
      int lo = 0, hi = threads;   // run_tok[lo] <= i < run_tok[hi]
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (run_tok[mid] <= i) lo = mid;
        else hi = mid;
      }
      long long at = run_tok[lo], taken = start + run_page[lo];
      int b = min(lo * per, p.batch);
      Request r = load_request(p, b);
#pragma unroll 1
      while (at + r.fresh <= i) {
        at += r.fresh;
        taken += r.take;
        r = load_request(p, ++b);
      }
      const long long place = static_cast<long long>(r.seq) + (i - at);
      pos = clamp_int(place);
      const int pi = p.page_div.quotient(pos), in_page = pos - pi * p.page_size;
      if (pi < p.max_pages && place == pos) {
        int id;
        if (pi < r.have) {
          id = p.table[b * p.table_stride + pi];
        } else {
          const long long f = taken + (pi - r.have);
          id = f < p.num_free ? *(p.free_pages + f) : -1;
          if (in_page == 0) p.table[b * p.table_stride + pi] = id;
        }
        if (id >= 0) slot = static_cast<long long>(id) * p.page_size + in_page;
      }
    }
    p.slots[i] = slot;
    p.positions[i] = pos;
  }
  if (total <= p.num_tokens) return;
  // Pages whose first token is past num_tokens are taken, too: the entries
  // that no token above has written, page by page (batch * max_pages at most,
  // whatever the lengths).  Calls with slots for all tokens pay 0.06 us for it
  // (as a function of its own, 0.3 to 1.5 us).
  const long long pages = run_page[threads];
#pragma unroll 1
  for (long long i = static_cast<long long>(blockIdx.x) * threads + t; i < pages;
       i += static_cast<long long>(gridDim.x) * threads) {
    int lo = 0, hi = threads;   // run_page[lo] <= i < run_page[hi]
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (run_page[mid] <= i) lo = mid;
      else hi = mid;
    }
    long long at = run_tok[lo], taken = run_page[lo];
    int b = min(lo * per, p.batch);
    Request r = load_request(p, b);
#pragma unroll 1
    while (taken + r.take <= i) {
      at += r.fresh;
      taken += r.take;
      r = load_request(p, ++b);
    }
    const long long pi = r.have + (i - taken), f = start + i;
    if (at + pi * p.page_size - r.seq >= p.num_tokens)
      p.table[b * p.table_stride + pi] = f < p.num_free ? *(p.free_pages + f) : -1;
  }
}

// ---------------------------------------------------------------- append
constexpr int kAppendThreads = 256;

struct AppendParams {
  fa::PagedCache kv;
  const uint16_t* k;
  const uint16_t* v;
  long long k_row_stride;
  long long v_row_stride;
  const int64_t* slots;
  fa::FastDiv page_div;
  int num_tokens;
};

// Each thread keeps one place in the row (16 bytes of the cache, so one head and
// one scale) and takes ROWS rows at a time: their slots, then all their
// loads, then the stores, so that enough loads are in flight.  Bound by HBM;
// few tokens by latency, so they take one row per thread.
// 32768 rows of 8 heads of 128 (269 MB, bf16) 42.1 us; 8191 rows of 16 heads
// of 64 to e4m3 (50 MB) 10.8 us.
template <bool E4M3, int ROWS>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  fa::pdl_wait();
  constexpr int N = E4M3 ? 2 : 1;   // 16-byte pieces of input per thread and row: one piece of the cache
  const int per_head = p.kv.head_dim / (8 * N), per_row = p.kv.heads_kv * per_head;
  const int wide = min(per_row, kAppendThreads), rows_per_pass = kAppendThreads / wide;
  const int r0 = threadIdx.x / wide, c = blockIdx.y * kAppendThreads + threadIdx.x - r0 * wide;
  if (r0 >= rows_per_pass || c >= per_row) return;
  const int h = c / per_head;
  const long long column = h * p.kv.head_stride + (c - h * per_head) * (8 * N);
  const long long num_slots = static_cast<long long>(p.kv.num_pages) * p.kv.page_size;
  const Scale ks(E4M3 ? p.kv.k_scale : nullptr, h), vs(E4M3 ? p.kv.v_scale : nullptr, h);
  const uint16_t* const kc = p.k + c * (8 * N);
  const uint16_t* const vc = p.v + c * (8 * N);
  for (long long row = static_cast<long long>(blockIdx.x) * rows_per_pass * ROWS + r0; row < p.num_tokens;
       row += static_cast<long long>(gridDim.x) * rows_per_pass * ROWS) {
    long long at[ROWS];   // element of the cache, -1: skipped
    uint4 k[ROWS][N], v[ROWS][N];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const long long r = row + i * rows_per_pass;
      at[i] = r < p.num_tokens ? *(reinterpret_cast<const long long*>(p.slots) + r) : -1;
      if (at[i] >= num_slots) at[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (at[i] < 0) continue;
      const long long r = row + i * rows_per_pass;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        k[i][n] = ldg_stream(kc + r * p.k_row_stride + 8 * n);
        v[i][n] = ldg_stream(vc + r * p.v_row_stride + 8 * n);
      }
      const long long page = at[i] <= 0x7fffffffll ? p.page_div.quotient(static_cast<int>(at[i])) : at[i] / p.kv.page_size;
      at[i] = page * p.kv.page_stride + (at[i] - page * p.kv.page_size) * p.kv.slot_stride + column;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (at[i] < 0) continue;
      if constexpr (E4M3) {
        const uint2 k0 = quantise8(k[i][0], ks), k1 = quantise8(k[i][1], ks);
        const uint2 v0 = quantise8(v[i][0], vs), v1 = quantise8(v[i][1], vs);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.kv.k) + at[i]) = make_uint4(k0.x, k0.y, k1.x, k1.y);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.kv.v) + at[i]) = make_uint4(v0.x, v0.y, v1.x, v1.y);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.kv.k) + at[i]) = k[i][0];
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.kv.v) + at[i]) = v[i][0];
      }
    }
  }
}

int blocks_for(long long items, int threads, int most) {
  const long long want = (items + threads - 1) / threads, cap = most;
  return static_cast<int>(want < 1 ? 1 : (want > cap ? cap : want));
}

}  // namespace

extern "C" {

int fa_kv_plan(int32_t* block_table, long long table_stride, int max_pages, const int32_t* seq_lens,
               const int32_t* new_lens, const int32_t* free_pages, int num_free, const int32_t* free_start,
               int page_size, int batch, int num_tokens, int64_t* slots, int32_t* positions, int32_t* cu_new,
               int32_t* seq_lens_out, int32_t* free_next, fa_stream_t stream) {
  if (batch < 0 || num_tokens < 0 || num_free < 0 || max_pages < 0)
    return set_last_error(FA_ERR_INVALID_ARG, "batch, num_tokens, num_free and max_pages must be >= 0");
  if (page_size < 1) return set_last_error(FA_ERR_INVALID_ARG, "page_size must be >= 1, got %d", page_size);
  if (batch > 1 && table_stride < max_pages)
    return set_last_error(FA_ERR_INVALID_ARG, "table_stride must be at least max_pages (%d), got %lld", max_pages,
                          table_stride);
  if (!cu_new || !free_next || (batch > 0 && (!seq_lens || !new_lens || !seq_lens_out)) ||
      (batch > 0 && max_pages > 0 && !block_table) || (num_free > 0 && !free_pages) ||
      (num_tokens > 0 && (!slots || !positions)))
    return set_last_error(FA_ERR_INVALID_ARG, "a device pointer is NULL");
  if (batch > 0 && (seq_lens_out == seq_lens || seq_lens_out == new_lens))
    return set_last_error(FA_ERR_INVALID_ARG, "seq_lens_out must not be seq_lens or new_lens");
  if (free_next == free_start)
    return set_last_error(FA_ERR_INVALID_ARG, "free_next must not be free_start");
  const void* al[] = {block_table, seq_lens, new_lens, free_pages, free_start, positions, cu_new, seq_lens_out, free_next};
  for (const void* ptr : al)
    if (misaligned4(ptr)) return set_last_error(FA_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(slots) & 7u)
    return set_last_error(FA_ERR_INVALID_ARG, "slots must be 8-byte aligned");
  fa::Device dev;
  int rc = check_device(dev);
  if (rc) return rc;
  const PlanParams p{block_table,  table_stride, max_pages, seq_lens,
                     new_lens,     free_pages,   num_free,  free_start,
                     page_size,    fa::FastDiv(static_cast<uint32_t>(page_size)),
                     batch,        num_tokens,   slots,     positions,
                     cu_new,       seq_lens_out, free_next};
  // a thread per request, up to a block's most
  const int threads = batch <= 256 ? 256 : batch <= 512 ? 512 : kPlanMaxThreads;
  cudaError_t e = fa::launch_pdl(plan_kernel, dim3(blocks_for(num_tokens, threads, 2 * dev.sms)), dim3(threads), 0,
                                 reinterpret_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) return cuda_fail(e, "plan launch");
  return ok();
}

int fa_kv_append(const fa_bf16* k, const fa_bf16* v, long long k_row_stride, long long v_row_stride,
                 const int64_t* slots, int num_tokens, void* k_cache, void* v_cache, int kv_type,
                 const float* k_scale, const float* v_scale, long long page_stride, long long slot_stride,
                 long long head_stride, int num_pages, int page_size, int heads_kv, int head_dim,
                 fa_stream_t stream) {
  AppendParams p;
  p.kv = make_cache(k_cache, v_cache, kv_type, k_scale, v_scale, page_stride, slot_stride, head_stride, num_pages,
                    page_size, heads_kv, head_dim);
  int rc = check_cache(p.kv, kv_type);
  if (rc) return rc;
  if (num_tokens < 0) return set_last_error(FA_ERR_INVALID_ARG, "num_tokens must be >= 0, got %d", num_tokens);
  const long long row = static_cast<long long>(heads_kv) * head_dim;
  if (row > 65535ll * 64)
    return set_last_error(FA_ERR_UNSUPPORTED, "heads_kv * head_dim too large (%d * %d)", heads_kv, head_dim);
  if ((rc = check_row_stride("k_row_stride", k_row_stride, row, num_tokens))) return rc;
  if ((rc = check_row_stride("v_row_stride", v_row_stride, row, num_tokens))) return rc;
  if (num_tokens == 0 || num_pages == 0) return ok();
  if (!k || !v || !slots || !k_cache || !v_cache)
    return set_last_error(FA_ERR_INVALID_ARG, "a device pointer is NULL");
  if (misaligned16(k) || misaligned16(v))
    return set_last_error(FA_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(slots) & 7u)
    return set_last_error(FA_ERR_INVALID_ARG, "slots must be 8-byte aligned");
  fa::Device dev;
  if ((rc = check_device(dev))) return rc;
  p.k = k;
  p.v = v;
  p.k_row_stride = k_row_stride;
  p.v_row_stride = v_row_stride;
  p.slots = slots;
  p.num_tokens = num_tokens;
  p.page_div = fa::FastDiv(static_cast<uint32_t>(page_size));
  const int per_row = static_cast<int>(row / (p.kv.e4m3 ? 16 : 8));   // threads
  const int rows_per_pass = per_row < kAppendThreads ? kAppendThreads / per_row : 1;
  // several rows per thread where that still gives every SM two blocks
  const int most = p.kv.e4m3 ? 2 : 4;
  const int rows = static_cast<long long>(num_tokens) * per_row >= 2ll * kAppendThreads * dev.sms * most ? most : 1;
  const dim3 grid(blocks_for(num_tokens, rows_per_pass * rows, 64 * dev.sms), (per_row + kAppendThreads - 1) / kAppendThreads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void (*const kernel)(AppendParams) = p.kv.e4m3 ? (rows > 1 ? append_kernel<true, 2> : append_kernel<true, 1>)
                                                  : (rows > 1 ? append_kernel<false, 4> : append_kernel<false, 1>);
  cudaError_t e = fa::launch_pdl(kernel, grid, dim3(kAppendThreads), 0, s, p);
  if (e != cudaSuccess) return cuda_fail(e, "append launch");
  return ok();
}

size_t fa_decode_workspace_size(int batch, int heads, int heads_kv, int head_dim) {
  if (batch < 0 || heads_kv < 1 || heads < 1 || heads % heads_kv != 0) {
    set_last_error(FA_ERR_INVALID_ARG,
                   "need batch >= 0 and query heads (%d) a positive multiple of key/value heads (%d)", heads, heads_kv);
    return 0;
  }
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) {
    set_last_error(FA_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256, got %d", head_dim);
    return 0;
  }
  ok();
  return fa::decode_workspace_bytes(batch, heads, heads_kv, head_dim);
}

int fa_decode(const fa_bf16* q, long long q_row_stride, const void* k_cache, const void* v_cache, int kv_type,
              const float* k_scale, const float* v_scale, long long page_stride, long long slot_stride,
              long long head_stride, int num_pages, int page_size, const int32_t* block_table,
              long long table_stride, int max_pages, const int32_t* seq_lens, int batch, int heads, int heads_kv,
              int head_dim, int window, float scale, fa_bf16* o, float* lse, void* workspace,
              size_t workspace_bytes, fa_stream_t stream) {
  fa::DecodeParams p;
  p.kv = make_cache(k_cache, v_cache, kv_type, k_scale, v_scale, page_stride, slot_stride, head_stride, num_pages,
                    page_size, heads_kv, head_dim);
  int rc = check_cache(p.kv, kv_type);
  if (rc) return rc;
  if (batch < 0) return set_last_error(FA_ERR_INVALID_ARG, "batch must be >= 0, got %d", batch);
  if (heads < 1 || heads % heads_kv != 0)
    return set_last_error(FA_ERR_INVALID_ARG, "query heads (%d) must be a positive multiple of key/value heads (%d)",
                          heads, heads_kv);
  if (static_cast<long long>(heads) * head_dim > 65535 * 64)
    return set_last_error(FA_ERR_UNSUPPORTED, "heads * head_dim too large (%d * %d)", heads, head_dim);
  if (heads / heads_kv > 1024)
    return set_last_error(FA_ERR_UNSUPPORTED, "at most 1024 query heads per key/value head, got %d", heads / heads_kv);
  if (window < 0) return set_last_error(FA_ERR_INVALID_ARG, "window must be >= 0, got %d", window);
  if (!isfinite(scale)) return set_last_error(FA_ERR_INVALID_ARG, "scale must be finite");
  if (max_pages < 0) return set_last_error(FA_ERR_INVALID_ARG, "max_pages must be >= 0, got %d", max_pages);
  if (static_cast<long long>(max_pages) * page_size > 0x7fff0000ll)
    return set_last_error(FA_ERR_UNSUPPORTED, "a block table of %d pages of %d slots is too long", max_pages, page_size);
  // The kernels count with 32 bits the costs of tiles (64 keys of a head at
  // least, 2) and units (1).
  if ((static_cast<long long>(max_pages) * page_size / 64 + 1) * heads_kv > 0x7fffffffll / 3 / (batch > 0 ? batch : 1))
    return set_last_error(FA_ERR_UNSUPPORTED, "%d requests of %d pages of %d slots and %d heads are too many", batch,
                          max_pages, page_size, heads_kv);
  if (batch > 1 && table_stride < 0)
    return set_last_error(FA_ERR_INVALID_ARG, "table_stride must be >= 0, got %lld", table_stride);
  if ((rc = check_row_stride("q_row_stride", q_row_stride, static_cast<long long>(heads) * head_dim, batch))) return rc;
  if (batch == 0) return ok();
  if (!q || !o || !seq_lens || (max_pages > 0 && !block_table) || (max_pages > 0 && num_pages > 0 && (!k_cache || !v_cache)))
    return set_last_error(FA_ERR_INVALID_ARG, "a device pointer is NULL");
  if (misaligned16(q) || misaligned16(o)) return set_last_error(FA_ERR_INVALID_ARG, "q and o must be 16-byte aligned");
  if (misaligned4(block_table) || misaligned4(seq_lens) || misaligned4(lse))
    return set_last_error(FA_ERR_INVALID_ARG, "block_table, seq_lens and lse must be 4-byte aligned");
  // Blocks that share a row write o while others still read q.
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(o);
  const uintptr_t row = 2ull * heads * head_dim;
  const uintptr_t q_bytes = (batch - 1) * 2ull * (batch > 1 ? q_row_stride : 0) + row;
  if (q0 < o0 + batch * row && o0 < q0 + q_bytes)
    return set_last_error(FA_ERR_INVALID_ARG, "o must not overlap q");
  const size_t need = fa::decode_workspace_bytes(batch, heads, heads_kv, head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return set_last_error(FA_ERR_INVALID_ARG, "workspace of %zu bytes needed, got %zu", need, workspace_bytes);
  if (misaligned16(workspace)) return set_last_error(FA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  fa::Device dev;
  if ((rc = check_device(dev))) return rc;
  p.q = q;
  p.q_row_stride = q_row_stride;
  p.table = block_table;
  p.table_stride = table_stride;
  p.seq_lens = seq_lens;
  p.o = o;
  p.lse = lse;
  p.work = static_cast<float*>(workspace);
  p.page_div = fa::FastDiv(static_cast<uint32_t>(page_size));
  p.max_pages = num_pages > 0 ? max_pages : 0;   // without pages no key is seen
  p.batch = batch;
  p.heads = heads;
  p.window = window;
  p.scale = scale;
  cudaError_t e = fa::launch_decode(p, dev, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  return ok();
}

size_t fa_extend_workspace_size(int head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) {
    set_last_error(FA_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256, got %d", head_dim);
    return 0;
  }
  ok();
  return fa::extend::workspace_bytes(head_dim);
}

int fa_extend(const fa_bf16* q, long long q_row_stride, const void* k_cache, const void* v_cache, int kv_type,
              const float* k_scale, const float* v_scale, long long page_stride, long long slot_stride,
              long long head_stride, int num_pages, int page_size, const int32_t* block_table,
              long long table_stride, int max_pages, const int32_t* seq_lens, const int32_t* cu_new, int batch,
              int num_tokens, int heads, int heads_kv, int head_dim, int window, float scale, fa_bf16* o, float* lse,
              void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  fa::ExtendParams p;
  p.kv = make_cache(k_cache, v_cache, kv_type, k_scale, v_scale, page_stride, slot_stride, head_stride, num_pages,
                    page_size, heads_kv, head_dim);
  int rc = check_cache(p.kv, kv_type);
  if (rc) return rc;
  if (batch < 0 || num_tokens < 0)
    return set_last_error(FA_ERR_INVALID_ARG, "batch and num_tokens must be >= 0, got %d and %d", batch, num_tokens);
  if (heads < 1 || heads % heads_kv != 0)
    return set_last_error(FA_ERR_INVALID_ARG, "query heads (%d) must be a positive multiple of key/value heads (%d)",
                          heads, heads_kv);
  if (static_cast<long long>(heads) * head_dim > 65535 * 64)
    return set_last_error(FA_ERR_UNSUPPORTED, "heads * head_dim too large (%d * %d)", heads, head_dim);
  // Rows (tokens by heads) and the costs of units are counted with 32 bits; every block
  // looks at all requests (2^20 of them 8 ms) while others wait for it, 20 s at most.
  if (batch > 1 << 28 || static_cast<long long>(num_tokens) * heads > 0x7ff00000ll ||
      fa::extend::most_units(num_tokens, batch, heads, heads_kv, head_dim) >= fa::extend::kMostUnits)
    return set_last_error(FA_ERR_UNSUPPORTED, "%d tokens of %d requests and %d heads are too many", num_tokens, batch,
                          heads);
  if (window < 0) return set_last_error(FA_ERR_INVALID_ARG, "window must be >= 0, got %d", window);
  if (!isfinite(scale)) return set_last_error(FA_ERR_INVALID_ARG, "scale must be finite");
  if (max_pages < 0) return set_last_error(FA_ERR_INVALID_ARG, "max_pages must be >= 0, got %d", max_pages);
  if (static_cast<long long>(max_pages) * page_size > 0x7fff0000ll)
    return set_last_error(FA_ERR_UNSUPPORTED, "a block table of %d pages of %d slots is too long", max_pages, page_size);
  if (batch > 1 && table_stride < 0)
    return set_last_error(FA_ERR_INVALID_ARG, "table_stride must be >= 0, got %lld", table_stride);
  if ((rc = check_row_stride("q_row_stride", q_row_stride, static_cast<long long>(heads) * head_dim, num_tokens)))
    return rc;
  if (num_tokens == 0) return ok();
  if (!q || !o || !cu_new || (batch > 0 && !seq_lens) || (batch > 0 && max_pages > 0 && !block_table) ||
      (batch > 0 && max_pages > 0 && num_pages > 0 && (!k_cache || !v_cache)))
    return set_last_error(FA_ERR_INVALID_ARG, "a device pointer is NULL");
  if (misaligned16(q) || misaligned16(o)) return set_last_error(FA_ERR_INVALID_ARG, "q and o must be 16-byte aligned");
  if (misaligned4(block_table) || misaligned4(seq_lens) || misaligned4(cu_new) || misaligned4(lse))
    return set_last_error(FA_ERR_INVALID_ARG, "block_table, seq_lens, cu_new and lse must be 4-byte aligned");
  // Blocks write rows of o while others still read q.
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(o);
  const uintptr_t row = 2ull * heads * head_dim;
  const uintptr_t q_bytes = (num_tokens - 1) * 2ull * (num_tokens > 1 ? q_row_stride : 0) + row;
  if (q0 < o0 + num_tokens * row && o0 < q0 + q_bytes)
    return set_last_error(FA_ERR_INVALID_ARG, "o must not overlap q");
  const size_t need = fa::extend::workspace_bytes(head_dim);
  if (!workspace || workspace_bytes < need)
    return set_last_error(FA_ERR_INVALID_ARG, "workspace of %zu bytes needed, got %zu", need, workspace_bytes);
  if (misaligned16(workspace)) return set_last_error(FA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  fa::Device dev;
  if ((rc = check_device(dev))) return rc;
  p.q = q;
  p.q_row_stride = q_row_stride;
  p.table = block_table;
  p.table_stride = table_stride;
  p.seq_lens = seq_lens;
  p.cu_new = cu_new;
  p.o = o;
  p.lse = lse;
  p.work = workspace;
  p.page_div = fa::FastDiv(static_cast<uint32_t>(page_size));
  p.group_div = fa::FastDiv(static_cast<uint32_t>(heads / heads_kv));
  p.max_pages = num_pages > 0 ? max_pages : 0;   // without pages no key is seen
  p.batch = batch;
  p.num_tokens = num_tokens;
  p.heads = heads;
  p.window = window;
  p.scale = scale;
  cudaError_t e = fa::launch_extend(p, dev, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "extend launch");
  return ok();
}

}  // extern "C"
