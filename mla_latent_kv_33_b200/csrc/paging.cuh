// Paged-cache bookkeeping on the GPU: the block tables and slot maps of a
// step, built from the requests' lengths, and ready latent rows written into
// the cache by a slot map. (MLA walk-through, section 1 step 1, fixes what a
// cached row is; how pages are handed out is this library's own.)
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace page {

constexpr int PLAN_THREADS = 512;
constexpr int MAX_REQUESTS = 16384;  // three ints of shared memory per request

struct PlanParams {
  const int32_t *ctx_lens;       // [B] tokens already cached, the shared blocks' among them
  const int32_t *new_lens;       // [B], or NULL: one new token each
  const int32_t *free_blocks;    // [num_free]
  const int32_t *shared_blocks;  // [num_shared]
  int32_t *block_table;          // [B][max_blocks]
  int32_t *seq_lens, *row_start, *seq_idx, *positions, *used;
  int64_t *slots;
  int64_t num_blocks;
  int32_t B, T, num_free, num_shared, block_size, max_blocks;
};

// What request b asks for. A request with bad lengths (negative, shorter than
// the shared blocks, past its table row) keeps its place among the rows but
// takes no block.
struct Request {
  int32_t ctx;
  int64_t rows, need;
  bool bad;
};

__device__ __forceinline__ int64_t blocks_for(int64_t tokens, int bs) {
  // (a 64-bit division costs some hundred instructions: only past 2^31)
  return tokens <= INT32_MAX - bs ? (static_cast<int32_t>(tokens) + bs - 1) / bs : (tokens + bs - 1) / bs;
}

__device__ __forceinline__ Request request_of(const PlanParams &p, int b) {
  Request r;
  r.ctx = p.ctx_lens[b];
  const int32_t n = p.new_lens != nullptr ? p.new_lens[b] : 1;
  const int64_t seq = static_cast<int64_t>(r.ctx) + n;
  r.rows = n > 0 ? n : 0;
  r.bad = r.ctx < 0 || n < 0 || static_cast<int64_t>(r.ctx) < static_cast<int64_t>(p.num_shared) * p.block_size ||
          seq > static_cast<int64_t>(p.max_blocks) * p.block_size || seq > INT32_MAX;
  r.need = r.bad ? 0 : blocks_for(seq, p.block_size) - blocks_for(r.ctx, p.block_size);
  return r;
}

__device__ __forceinline__ int32_t sat32(int64_t x) { return x > INT32_MAX ? INT32_MAX : static_cast<int32_t>(x); }

// Last index b < B with a[b] <= x (a is non-decreasing and a[0] = 0 <= x).
__device__ __forceinline__ int last_le(const int32_t *a, int B, int32_t x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One launch. Every block scans the requests into shared memory (row offsets
// and free-list offsets: both lengths are loaded twice, 16 bytes per request from
// L2, a few hundred nanoseconds for a thousand requests), then takes its stride
// of the table entries and of the rows; an entry or row finds its request by
// bisection. Nothing is communicated between blocks, so there is no second
// launch, no atomic on memory and no order to depend on. Bound: latency (launch, one
// dependent chain of loads per phase); the traffic of a step is a few hundred
// KB at most. 64 requests with one token each take 4.3 us, 1024 requests with
// 33 thousand rows 6.6 us (per call in a graph).
//
// Both offsets are sums of the requests before b whether those could be
// planned or not, so "the pool is short" and "the row buffers are full" hold
// for every later request that needs a block or a row: the planned requests'
// blocks are exactly the first `used` entries of the free list.
__global__ void __launch_bounds__(PLAN_THREADS) k_batch_plan(const PlanParams p) {
  extern __shared__ int32_t plan_smem[];
  // exclusive sums of rows and needed blocks (saturated), and the context length, -1 for a request left out
  int32_t *row0 = plan_smem, *blk0 = plan_smem + p.B, *ctx = plan_smem + 2 * p.B;
  __shared__ int64_t wrow[PLAN_THREADS / 32], wblk[PLAN_THREADS / 32];
  __shared__ int32_t s_used;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) griddep_launch_dependents();
  griddep_wait();
  if (tid == 0) s_used = 0;
  const int per = (p.B + PLAN_THREADS - 1) / PLAN_THREADS;
  const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);
  int64_t rows = 0, need = 0;
  for (int b = lo; b < hi; ++b) {
    const Request r = request_of(p, b);
    rows += r.rows;
    need += r.need;
  }
  int64_t irow = rows, iblk = need;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, irow, o), c = __shfl_up_sync(0xffffffffu, iblk, o);
    if (lane >= o) {
      irow += a;
      iblk += c;
    }
  }
  if (lane == 31) {
    wrow[warp] = irow;
    wblk[warp] = iblk;
  }
  __syncthreads();
  int64_t total = 0;
  irow -= rows;
  iblk -= need;
  for (int w = 0; w < PLAN_THREADS / 32; ++w) {
    if (w < warp) {
      irow += wrow[w];
      iblk += wblk[w];
    }
    total += wrow[w];
  }
  // offsets of this thread's requests; block 0's first stride also writes the per-request outputs
  bool any_bad = false;
  int32_t used = 0;
  for (int b = lo; b < hi; ++b) {
    const Request r = request_of(p, b);
    row0[b] = sat32(irow);
    blk0[b] = sat32(iblk);
    const bool skip = r.bad || (r.need > 0 && iblk + r.need > p.num_free) || (r.rows > 0 && irow + r.rows > p.T);
    any_bad |= skip;
    ctx[b] = skip ? -1 : r.ctx;
    if (!skip && r.need > 0) used = static_cast<int32_t>(iblk + r.need);
    if (blockIdx.x == 0) {
      p.seq_lens[b] = skip ? 0 : r.ctx + static_cast<int32_t>(r.rows);
      p.row_start[b] = sat32(irow);
    }
    irow += r.rows;
    iblk += r.need;
  }
  if (used > 0) atomicMax(&s_used, used);
  if (any_bad && blockIdx.x == 0) dev_error(MLA_DEVERR_DATA);
  __syncthreads();
  const int32_t used_all = s_used;
  if (blockIdx.x == 0 && tid == 0) {
    p.row_start[p.B] = sat32(total);
    p.used[0] = used_all;
  }
  const int64_t gtid = static_cast<int64_t>(blockIdx.x) * PLAN_THREADS + tid;
  const int64_t gstride = static_cast<int64_t>(gridDim.x) * PLAN_THREADS;
  // the shared blocks, at the front of every planned request's table row
  const int64_t nsh = static_cast<int64_t>(p.B) * p.num_shared;
  for (int64_t e = gtid; e < nsh; e += gstride) {
    const int b = nsh <= INT32_MAX ? static_cast<int32_t>(e) / p.num_shared : static_cast<int>(e / p.num_shared);
    const int k = static_cast<int>(e - static_cast<int64_t>(b) * p.num_shared);
    if (ctx[b] < 0) continue;
    const int32_t blk = p.shared_blocks[k];
    if (blk < 0 || blk >= p.num_blocks) dev_error(MLA_DEVERR_DATA);  // (no new row lies on it to report it)
    p.block_table[static_cast<int64_t>(b) * p.max_blocks + k] = blk;
  }
  // the blocks handed out: entry e of the free list goes to the request whose offset range holds e
  for (int64_t e = gtid; e < used_all; e += gstride) {
    const int b = last_le(blk0, p.B, static_cast<int32_t>(e));
    if (ctx[b] < 0) continue;
    const int64_t k = blocks_for(ctx[b], p.block_size) + (e - blk0[b]);
    p.block_table[static_cast<int64_t>(b) * p.max_blocks + k] = p.free_blocks[e];
  }
  // rows. An entry that this launch writes is taken from the list it is
  // written from, not from the table, which another block may not have
  // written yet; entries between the two are the request's own and untouched.
  for (int64_t t = gtid; t < p.T; t += gstride) {
    int32_t sidx = -1, pos = 0;
    int64_t slot = -1;
    if (t < total) {
      const int b = last_le(row0, p.B, static_cast<int32_t>(t));
      if (ctx[b] >= 0) {
        sidx = b;
        pos = ctx[b] + static_cast<int32_t>(t - row0[b]);
        const int32_t k = pos / p.block_size, held = static_cast<int32_t>(blocks_for(ctx[b], p.block_size));
        const int32_t blk = k >= held ? p.free_blocks[blk0[b] + (k - held)]
                                      : (k < p.num_shared ? p.shared_blocks[k]
                                                          : p.block_table[static_cast<int64_t>(b) * p.max_blocks + k]);
        if (blk < 0 || blk >= p.num_blocks)
          dev_error(MLA_DEVERR_DATA);
        else
          slot = static_cast<int64_t>(blk) * p.block_size + (pos - k * p.block_size);
      }
    }
    p.seq_idx[t] = sidx;
    p.positions[t] = pos;
    p.slots[t] = slot;
  }
}

// cache row slots[t] = rows[t], `vec` words of type V per row; a negative slot
// is padding. Neighbouring threads copy neighbouring words of a row, four
// independent words each, so that enough 16-byte loads are in flight; the copy
// is bound by memory (each row read once and written once): 12289 rows of 1152
// bytes in 5.6 us per call in a graph, 5.0 TB/s.
template <typename V>
__global__ void __launch_bounds__(256) k_cache_write(const V *__restrict__ rows, const int64_t *__restrict__ slots,
                                                     V *__restrict__ cache, int64_t cache_rows, int64_t n, int vec) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  constexpr int U = 4;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i0 < n; i0 += U * stride) {
    V x[U];
    int64_t dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // words and slots are fetched together: neither waits for the other
      const int64_t i = i0 + u * stride;
      dst[u] = -1;
      if (i < n) {
        x[u] = rows[i];
        const int64_t t = n <= INT32_MAX ? static_cast<int32_t>(i) / vec : i / vec;
        dst[u] = slots[t];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * stride;
      if (dst[u] < 0) continue;
      const int64_t c = n <= INT32_MAX ? static_cast<int32_t>(i) % vec : i % vec;
      if (dst[u] >= cache_rows) {
        if (c == 0) dev_error(MLA_DEVERR_DATA);
        dst[u] = -1;
      } else {
        dst[u] = dst[u] * vec + c;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] >= 0) cache[dst[u]] = x[u];
  }
}

}  // namespace page
}  // namespace mla
