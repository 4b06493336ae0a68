// pages_sm100.cuh — sharing, freeing, handing out and compacting pages of a paged K/V cache on
// the device, for sm_100a.
//
// The block table is the only state: a page is in use while a row of the table refers to it,
// and free otherwise, so there is no reference count or free list to keep consistent.  Both
// operators are two kernels after one clearing of the marks, with the page numbers never leaving
// the device:
//   plan   the rows' pages set bits of a map over the pool (many CTAs, one row each); the CTA that
//          finishes last ranks the free pages (fork) or the moves (compact) with popcounts and
//          one block-wide scan.  Ranks make the result independent of the order of execution.
//          A small table is planned by one CTA, with the map in shared memory and nothing to clear;
//          where there is little to copy, its cluster does that too, in the same launch.
//   move   many CTAs write the table and copy pages with 16-byte loads and stores
// Integer work on a few KB is bound by the latency of the launches and of the scan: 4 rows of 70
// pages, one page copied, 8.3 us as one cluster, 10.2 as one planning CTA and a move kernel, 11.9 with the
// clearing and many planning CTAs.  The copies are bound by HBM (each byte read once and written once):
// 0.73 GB of pages moved take 260 us, 5.6 TB/s.  (Replayed graphs; called, the two take 12.5 and 262 us.)
#pragma once

#include "sm100_common.cuh"

namespace attn {

// Programmatic dependent launch: the dependent grid may be set up from here on; it waits for this
// grid's end (and its writes) in pdl_wait.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

constexpr int kMaxPools = 128;     // pools that share one block table (layers x K and V)
constexpr int kPagesThreads = 256;
constexpr int kPlanThreads = 512;

struct PagePools {
  uint8_t* base[kMaxPools];
  long long page_bytes;  // the same for every pool, a multiple of 16
  int n;
};

struct ForkArgs {
  const int32_t* table;     // [S, cols]
  const int32_t* seq_lens;  // [S]
  const int32_t* parents;   // [rows]
  const int32_t* add;       // [rows] or null
  int32_t* new_table;       // [rows, new_cols]
  int32_t* new_lens;        // [rows]
  int32_t* n_free;          // [1] or null
  // workspace
  int* n_done;              // [1] CTAs that have marked their row (cleared, as the next three)
  uint32_t* full_bits;      // [words] pages some row has as a full page
  uint32_t* part_bits;      // [words] pages some row has as its part-filled last page
  int* first_part;          // [num_pages] rows - i for the lowest row i with the page as its part-filled page
  int* free_list;           // [num_pages] free pages, ascending
  int* row_part;            // [rows] the row's part-filled page or -1
  int* row_fresh;           // [rows] fresh pages after the part-filled one
  int* row_rank;            // [rows] rank of the row's first page from the free list
  int* row_keep;            // [rows] 1: the row keeps its part-filled page in place
  int* n_list;              // [1] free pages
  int S, cols, rows, new_cols, page_size, num_pages;
};

// Barrier of the cluster's CTAs; what they wrote to global memory before it is visible after it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// True in every thread of the CTA that arrives last, with the others' writes visible to it.
__device__ __forceinline__ bool last_cta(int* n_done) {
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(n_done, 1) == (int)gridDim.x - 1;
  __syncthreads();
  __threadfence();
  return last != 0;
}

// Block-wide exclusive scan of two ints per thread (.x and .y apart); *total gets the sums.  sums:
// 16 pairs of shared memory.  Every thread of a block of kPlanThreads calls it.
__device__ __forceinline__ int2 pages_scan(int2 v, int2* sums, int2* total) {
  constexpr int W = kPlanThreads / 32;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y0 = __shfl_up_sync(0xffffffffu, x.x, o), y1 = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) {
      x.x += y0;
      x.y += y1;
    }
  }
  if (lane == 31) sums[w] = x;
  __syncthreads();
  int2 before = make_int2(x.x - v.x, x.y - v.y), all = make_int2(0, 0);
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const int2 s = sums[k];
    if (k < w) {
      before.x += s.x;
      before.y += s.y;
    }
    all.x += s.x;
    all.y += s.y;
  }
  *total = all;
  return before;
}

// Tables planned by one CTA: up to this many entries, rows and pages; and bytes that its cluster copies.
constexpr int kSmallEntries = 2048, kSmallForkRows = 32, kSmallCompactRows = 256, kSmallPages = 65536, kSmallCluster = 8;
constexpr long long kSmallForkBytes = 1ll << 20;     // every row's part-filled page
constexpr long long kSmallCompactBytes = 4ll << 20;  // what could move; most often half of it does

// ------------------------------------------------------------------ fork

// A new row's length, and what it takes over from its parent: {parent, full pages, part-filled last
// page (0 or 1), new length}.
__device__ __forceinline__ int4 fork_row(const ForkArgs& a, int i, bool* bad) {
  const int max_tokens = a.cols * a.page_size;
  int p = __ldg(&a.parents[i]), old_len = 0, new_len = 0;
  const int add = a.add != nullptr ? __ldg(&a.add[i]) : 0;
  *bad = p < -1 || p >= a.S;
  if (*bad) p = -1;
  if (p >= 0) {
    old_len = __ldg(&a.seq_lens[p]);
    if (old_len < 0 || old_len > max_tokens) {
      *bad = true;
      old_len = 0;
    }
    const long long want = (long long)old_len + add;
    if (want < 0 || want > (long long)a.new_cols * a.page_size) {
      *bad = true;
      new_len = old_len;
    } else {
      new_len = (int)want;
    }
  }
  const int kept = min(old_len, new_len);
  return make_int4(p, kept / a.page_size, kept % a.page_size != 0 ? 1 : 0, new_len);
}

// Entry j of new row i: the parent's page (marked in the maps) or -1.
__device__ __forceinline__ void fork_entry(const ForkArgs& a, int i, int j, int4 row, uint32_t* full, uint32_t* part,
                                           int* first_part) {
  int e = -1;
  if (j < row.y + row.z) {
    e = __ldg(&a.table[(size_t)row.x * a.cols + j]);
    if (e < 0 || e >= a.num_pages) {
      latch_status(ATTN_ERR_BAD_PAGE);
      e = -1;
    } else if (j < row.y) {
      atomicOr(&full[e >> 5], 1u << (e & 31));
    } else {
      atomicOr(&part[e >> 5], 1u << (e & 31));
      if (first_part != nullptr) atomicMax(&first_part[e], a.rows - i);
    }
    if (j == row.y) a.row_part[i] = e;
  }
  a.new_table[(size_t)i * a.new_cols + j] = e;
}

__device__ __forceinline__ void fork_row_done(const ForkArgs& a, int i, int4 row, bool bad) {
  if (bad) latch_status(ATTN_ERR_INVALID_ARG);
  if (row.z == 0) a.row_part[i] = -1;
  a.new_lens[i] = row.w;
  a.row_fresh[i] = (row.w + a.page_size - 1) / a.page_size - row.y - row.z;
}

// Lists the free pages that are needed, in ascending order, and gives each row its rank in that list.  lowest(i, e): row
// i is the lowest with the part-filled page e.  Such a page stays with the lowest row that has it,
// unless some row has it as a full page (that row's tokens must not be written over).
template <typename Lowest>
__device__ __forceinline__ void fork_rank(const ForkArgs& a, const volatile uint32_t* full, const volatile uint32_t* part,
                                          Lowest lowest, int2* sums) {
  const int tid = threadIdx.x;
  const int words = (a.num_pages + 31) / 32;
  const int wpt = (words + kPlanThreads - 1) / kPlanThreads;
  const int w0 = min(words, tid * wpt), w1 = min(words, w0 + wpt);
  auto free_bits = [&](int w) -> uint32_t {
    uint32_t f = ~(full[w] | part[w]);
    if (w == words - 1 && (a.num_pages & 31) != 0) f &= (1u << (a.num_pages & 31)) - 1u;
    return f;
  };
  const volatile int *row_part = a.row_part, *row_fresh = a.row_fresh;
  const int rpt = (a.rows + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(a.rows, tid * rpt), i1 = min(a.rows, i0 + rpt);
  int2 mine = make_int2(0, 0);  // free pages, pages needed
  for (int w = w0; w < w1; ++w) mine.x += __popc(free_bits(w));
  for (int i = i0; i < i1; ++i) {
    const int e = row_part[i];
    int keep = 0;
    if (e >= 0) {
      keep = lowest(i, e) && (full[e >> 5] >> (e & 31) & 1u) == 0;
      mine.y += 1 - keep;
    }
    a.row_keep[i] = keep;
    mine.y += row_fresh[i];
  }
  int2 total;
  int2 at = pages_scan(mine, sums, &total);
  // only the pages that rows will take: writing all 65 thousand of an empty pool took 34 us
  for (int w = w0; w < w1 && at.x < total.y; ++w)
    for (uint32_t f = free_bits(w); f != 0 && at.x < total.y; f &= f - 1) a.free_list[at.x++] = 32 * w + __ffs(f) - 1;
  for (int i = i0; i < i1; ++i) {
    a.row_rank[i] = at.y;
    at.y += row_fresh[i] + (row_part[i] >= 0 && !a.row_keep[i] ? 1 : 0);
  }
  if (tid == 0) {
    if (total.y > total.x) latch_status(ATTN_ERR_TOO_LARGE);
    *a.n_list = total.x;
    if (a.n_free != nullptr) *a.n_free = max(0, total.x - total.y);
  }
}

// One CTA per new row (one at least); the last one to finish ranks.
__global__ void __launch_bounds__(kPlanThreads) attn_pages_fork_plan_kernel(const __grid_constant__ ForkArgs a) {
  __shared__ int2 sums[kPlanThreads / 32];
  const int i = blockIdx.x;
  if (i < a.rows) {
    bool bad;
    const int4 row = fork_row(a, i, &bad);
    for (int j = threadIdx.x; j < a.new_cols; j += kPlanThreads)
      fork_entry(a, i, j, row, a.full_bits, a.part_bits, a.first_part);
    if (threadIdx.x == 0) fork_row_done(a, i, row, bad);
  }
  if (!last_cta(a.n_done)) return;
  const volatile int* first_part = a.first_part;
  fork_rank(a, a.full_bits, a.part_bits, [&](int r, int e) { return first_part[e] == a.rows - r; }, sums);
}

// Copies `bytes` (a multiple of 16) with the block's threads, part `part` of `parts`.
__device__ __forceinline__ void copy_bytes(uint8_t* dst, const uint8_t* src, long long bytes, int part, int parts) {
  const long long n = bytes / 16;
  const long long lo = n * part / parts, hi = n * (part + 1) / parts;
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  long long i = lo + threadIdx.x;
  for (; i + 3 * kPagesThreads < hi; i += 4 * kPagesThreads) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __ldcs(s + i + k * kPagesThreads);
#pragma unroll
    for (int k = 0; k < 4; ++k) __stcs(d + i + k * kPagesThreads, v[k]);
  }
  for (; i < hi; i += kPagesThreads) __stcs(d + i, __ldcs(s + i));
}

// Pieces of a page that a warp copies, all their loads in flight at once.
constexpr int kPieceBytes = 4096;

__device__ __forceinline__ void copy_piece(const PagePools& pools, int pool, int src, int dst, int piece) {
  const int lane = threadIdx.x & 31;
  const long long n = min((long long)kPieceBytes, pools.page_bytes - (long long)piece * kPieceBytes) / 16;
  uint8_t* base = pools.base[pool] + (long long)piece * kPieceBytes;
  const uint4* s = reinterpret_cast<const uint4*>(base + (size_t)src * pools.page_bytes);
  uint4* d = reinterpret_cast<uint4*>(base + (size_t)dst * pools.page_bytes);
  uint4 v[kPieceBytes / 512];
#pragma unroll
  for (int k = 0; k < kPieceBytes / 512; ++k)
    if (lane + 32 * k < n) v[k] = __ldcs(s + lane + 32 * k);
#pragma unroll
  for (int k = 0; k < kPieceBytes / 512; ++k)
    if (lane + 32 * k < n) __stcs(d + lane + 32 * k, v[k]);
}

__device__ __forceinline__ int pieces_of(const PagePools& pools) {
  return (int)((pools.page_bytes + kPieceBytes - 1) / kPieceBytes);
}

// A planned row's page to copy from (.x) and to (.y, -1: nothing to copy).
__device__ __forceinline__ int2 fork_copy(const ForkArgs& a, int i, int n_list) {
  const int rank = a.row_rank[i], e = a.row_part[i];
  return make_int2(e, e >= 0 && !a.row_keep[i] && rank < n_list ? a.free_list[rank] : -1);
}

// The entries of row i that come from the free pages.
__device__ __forceinline__ void fork_fresh(const ForkArgs& a, int i, int n_list, int thread, int threads) {
  const int rank = a.row_rank[i], fresh = a.row_fresh[i];
  const bool copies = a.row_part[i] >= 0 && !a.row_keep[i];
  const int first = (a.new_lens[i] + a.page_size - 1) / a.page_size - fresh;
  int32_t* row = a.new_table + (size_t)i * a.new_cols;
  if (copies && thread == 0) row[first - 1] = rank < n_list ? a.free_list[rank] : -1;
  const int r0 = rank + (copies ? 1 : 0);
  for (int j = thread; j < fresh; j += threads) row[first + j] = r0 + j < n_list ? a.free_list[r0 + j] : -1;
}

// CTA (row, pool x part).
__global__ void __launch_bounds__(kPagesThreads)
    attn_pages_fork_move_kernel(const __grid_constant__ ForkArgs a, const __grid_constant__ PagePools pools, int parts) {
  pdl_wait();
  const int i = blockIdx.x, n_list = *a.n_list;
  if (blockIdx.y == 0) fork_fresh(a, i, n_list, threadIdx.x, kPagesThreads);
  const int2 c = fork_copy(a, i, n_list);
  if (c.y < 0) return;
  for (int w = blockIdx.y; w < pools.n * parts; w += gridDim.y) {
    uint8_t* base = pools.base[w / parts];
    copy_bytes(base + (size_t)c.y * pools.page_bytes, base + (size_t)c.x * pools.page_bytes, pools.page_bytes, w % parts,
               parts);
  }
}

// A small table.  The first CTA plans with the maps in (dynamic) shared memory.  For `move` the grid is one
// cluster, whose other CTAs wait at its barrier, and all of them move; else it is that one CTA.
__global__ void __launch_bounds__(kPlanThreads)
    attn_pages_fork_small_kernel(const __grid_constant__ ForkArgs a, const __grid_constant__ PagePools pools, int move) {
  extern __shared__ uint32_t maps[];
  __shared__ int2 sums[kPlanThreads / 32];
  __shared__ int4 rows[kSmallForkRows];
  if (blockIdx.x == 0) {
    const int words = (a.num_pages + 31) / 32;
    uint32_t *full = maps, *part = maps + words;
    for (int w = threadIdx.x; w < 2 * words; w += kPlanThreads) maps[w] = 0;
    if (threadIdx.x < a.rows) {
      bool bad;
      const int4 row = fork_row(a, threadIdx.x, &bad);
      rows[threadIdx.x] = row;
      fork_row_done(a, threadIdx.x, row, bad);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.rows * a.new_cols; k += kPlanThreads) {
      const int i = k / a.new_cols;
      fork_entry(a, i, k % a.new_cols, rows[i], full, part, nullptr);
    }
    __syncthreads();  // orders the block's global writes of row_part before their reads, too
    const volatile int* row_part = a.row_part;
    if (threadIdx.x < a.rows) rows[threadIdx.x].x = row_part[threadIdx.x];
    __syncthreads();
    auto lowest = [&](int r, int e) {
      for (int k = 0; k < r; ++k)
        if (rows[k].x == e) return false;
      return true;
    };
    fork_rank(a, full, part, lowest, sums);
  }
  if (!move) return pdl_launch_dependents();
  cluster_barrier();
  const int warp = blockIdx.x * (kPlanThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kPlanThreads / 32);
  const int n_list = *a.n_list;
  for (int i = warp; i < a.rows; i += warps) fork_fresh(a, i, n_list, threadIdx.x & 31, 32);
  const int pieces = pieces_of(pools), each = pools.n * pieces;
  for (int k = warp; k < a.rows * each; k += warps) {
    const int2 c = fork_copy(a, k / each, n_list);
    if (c.y >= 0) copy_piece(pools, k % each / pieces, c.x, c.y, k % pieces);
  }
}

// ------------------------------------------------------------------ compact

struct CompactArgs {
  const int32_t* table;     // [S, cols]
  const int32_t* seq_lens;  // [S]
  int32_t* new_table;       // [S, cols]; may be table
  int32_t* page_map;        // [num_pages]
  int32_t* n_live;          // [1] or null
  // workspace
  int* n_done;              // [1] CTAs that have marked their row (cleared, as the next)
  uint32_t* bits;           // [words] pages in use
  int* prefix;              // [words] pages in use before the word
  int* src;                 // [num_pages] pages that move, ascending
  int* dst;                 // [num_pages] where they go, ascending
  int* counts;              // [2] pages in use, pages that move
  int S, cols, page_size, num_pages;
};

__device__ __forceinline__ int pages_of_row(const CompactArgs& a, int s, bool* bad) {
  const int len = __ldg(&a.seq_lens[s]);
  *bad = len < 0 || len > a.cols * a.page_size;
  return *bad ? 0 : (len + a.page_size - 1) / a.page_size;
}

// With n pages in use, page ids below n stay and the others move, in ascending order, into the free
// ids below n.  No page is both a source and a destination.  A mover's rank is the number of pages in
// use before it, less those that stay; a hole's is the number of free ids before it.
__device__ __forceinline__ void compact_rank(const CompactArgs& a, const volatile uint32_t* bits, int2* sums) {
  __shared__ int stay;
  const int tid = threadIdx.x;
  const int words = (a.num_pages + 31) / 32;
  const int wpt = (words + kPlanThreads - 1) / kPlanThreads;
  const int w0 = min(words, tid * wpt), w1 = min(words, w0 + wpt);
  if (tid == 0) stay = 0;
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
  int2 total;
  const int first = pages_scan(make_int2(mine, 0), sums, &total).x;
  const int live = total.x;
  auto below = [&](int w) -> uint32_t {  // mask of the word's ids below `live`
    const int d = live - 32 * w;
    return d >= 32 ? 0xffffffffu : (d <= 0 ? 0u : (1u << d) - 1u);
  };
  int before = first;
  for (int w = w0; w < w1; ++w) {
    const uint32_t b = bits[w];
    a.bits[w] = b;
    a.prefix[w] = before;
    if (live / 32 == w) stay = before + __popc(b & below(w));
    before += __popc(b);
  }
  if (tid == 0 && live / 32 == words) stay = live;  // every page of a pool of 32 k pages is in use
  __syncthreads();
  before = first;
  for (int w = w0; w < w1; ++w) {
    const uint32_t b = bits[w];
    int r = before - stay + __popc(b & below(w));
    for (uint32_t f = b & ~below(w); f != 0; f &= f - 1) a.src[r++] = 32 * w + __ffs(f) - 1;
    r = 32 * w - before;
    for (uint32_t f = ~b & below(w); f != 0; f &= f - 1) a.dst[r++] = 32 * w + __ffs(f) - 1;
    before += __popc(b);
  }
  if (tid == 0) {
    a.counts[0] = live;
    a.counts[1] = live - stay;
    if (a.n_live != nullptr) *a.n_live = live;
  }
}

__device__ __forceinline__ void compact_mark(const CompactArgs& a, int s, int j, uint32_t* bits) {
  const int e = a.table[(size_t)s * a.cols + j];
  if (e < 0 || e >= a.num_pages)
    latch_status(ATTN_ERR_BAD_PAGE);
  else
    atomicOr(&bits[e >> 5], 1u << (e & 31));
}

// One CTA per row (one at least) marks its pages; the last one to finish ranks.
__global__ void __launch_bounds__(kPlanThreads) attn_pages_compact_plan_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ int2 sums[kPlanThreads / 32];
  if (blockIdx.x < a.S) {
    bool bad;
    const int n = pages_of_row(a, blockIdx.x, &bad);
    if (bad && threadIdx.x == 0) latch_status(ATTN_ERR_INVALID_ARG);
    for (int j = threadIdx.x; j < n; j += kPlanThreads) compact_mark(a, blockIdx.x, j, a.bits);
  }
  if (!last_cta(a.n_done)) return;
  compact_rank(a, a.bits, sums);
}

// The new number of page e in use.  Movers are ranked by the pages in use before them: of those,
// live - n_move stay.
__device__ __forceinline__ int compact_to(const CompactArgs& a, int e, int live, int n_move) {
  if (e < live) return e;
  const int r = a.prefix[e >> 5] + __popc(a.bits[e >> 5] & ((1u << (e & 31)) - 1u)) - (live - n_move);
  return a.dst[r];
}

// Writes the table and the map, grid-stride.
__device__ __forceinline__ void compact_write(const CompactArgs& a, int live, int n_move) {
  const long long step = (long long)gridDim.x * blockDim.x;
  const long long t0 = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  for (long long i = t0; i < a.num_pages; i += step) {
    const int e = (int)i;
    const bool used = a.bits[e >> 5] >> (e & 31) & 1u;
    a.page_map[e] = used ? compact_to(a, e, live, n_move) : -1;
  }
  for (long long i = t0; i < (long long)a.S * a.cols; i += step) {
    bool bad;
    const int n = pages_of_row(a, (int)(i / a.cols), &bad);
    int to = -1;
    if (i % a.cols < n) {
      const int e = a.table[i];
      if (e >= 0 && e < a.num_pages) to = compact_to(a, e, live, n_move);
    }
    a.new_table[i] = to;
  }
}

__global__ void __launch_bounds__(kPagesThreads)
    attn_pages_compact_move_kernel(const __grid_constant__ CompactArgs a, const __grid_constant__ PagePools pools,
                                   int parts) {
  pdl_wait();
  const int live = a.counts[0], n_move = a.counts[1];
  compact_write(a, live, n_move);
  const long long work = (long long)n_move * pools.n * parts;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const int part = (int)(w % parts);
    const int pool = (int)(w / parts % pools.n);
    const int k = (int)(w / parts / pools.n);
    uint8_t* base = pools.base[pool];
    copy_bytes(base + (size_t)a.dst[k] * pools.page_bytes, base + (size_t)a.src[k] * pools.page_bytes,
               pools.page_bytes, part, parts);
  }
}

// A small table, as for the fork.
__global__ void __launch_bounds__(kPlanThreads)
    attn_pages_compact_small_kernel(const __grid_constant__ CompactArgs a, const __grid_constant__ PagePools pools,
                                    int move) {
  extern __shared__ uint32_t maps[];
  __shared__ int2 sums[kPlanThreads / 32];
  __shared__ int used[kSmallCompactRows];
  if (blockIdx.x == 0) {
    const int words = (a.num_pages + 31) / 32;
    for (int w = threadIdx.x; w < words; w += kPlanThreads) maps[w] = 0;
    if (threadIdx.x < a.S) {
      bool bad;
      used[threadIdx.x] = pages_of_row(a, threadIdx.x, &bad);
      if (bad) latch_status(ATTN_ERR_INVALID_ARG);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.S * a.cols; k += kPlanThreads)
      if (k % a.cols < used[k / a.cols]) compact_mark(a, k / a.cols, k % a.cols, maps);
    __syncthreads();
    compact_rank(a, maps, sums);
  }
  if (!move) return pdl_launch_dependents();
  cluster_barrier();
  const int live = a.counts[0], n_move = a.counts[1];
  compact_write(a, live, n_move);
  const int warp = blockIdx.x * (kPlanThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kPlanThreads / 32);
  const int pieces = pieces_of(pools), each = pools.n * pieces;
  for (int k = warp; k < n_move * each; k += warps)
    copy_piece(pools, k % each / pieces, a.src[k / each], a.dst[k / each], k % pieces);
}

}  // namespace attn
