// pages_sm100.cuh — sharing, freeing, handing out and compacting pages of a paged K/V cache on
// the device, for sm_100a.
//
// The block table is the only state: a page is in use while a row of the table refers to it,
// and free otherwise, so there is no reference count or free list to keep consistent.  Both
// operators are three steps on one stream, with the page numbers never leaving the device:
//   mark   the rows' pages set bits of a map over the pool (many CTAs, one row each)
//   scan   one CTA ranks the free pages (fork) or the moves (compact) with popcounts and one
//          block-wide scan; ranks make the result independent of the order of execution
//   move   many CTAs write the table and copy pages with 16-byte loads and stores
// Integer work on a few KB is bound by the latency of the launches and of the scan; the
// copies are bound by HBM (each byte read once and written once).
#pragma once

#include "sm100_common.cuh"

namespace attn {

constexpr int kMaxPools = 128;     // pools that share one block table (layers x K and V)
constexpr int kPagesThreads = 256;
constexpr int kScanThreads = 1024;

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
  uint32_t* full_bits;      // [words] pages some row has as a full page
  uint32_t* part_bits;      // [words] pages some row has as its part-filled last page
  int* first_part;          // [num_pages] lowest row with the page as its part-filled page
  int* free_list;           // [num_pages] free pages, ascending
  int* row_part;            // [rows] the row's part-filled page or -1; scan: | keep flag in row_keep
  int* row_fresh;           // [rows] fresh pages after the part-filled one
  int* row_rank;            // [rows] rank of the row's first page from the free list
  int* row_keep;            // [rows] 1: the row keeps its part-filled page in place
  int* n_list;              // [1] free pages
  int S, cols, rows, new_cols, page_size, num_pages;
};

// Block-wide exclusive scan of one int per thread; *total gets the sum.  sums: 32 ints of shared
// memory.  Every thread of a block of kScanThreads calls it.
__device__ __forceinline__ int pages_scan(int v, int* sums, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // an earlier scan's readers of sums are done
  if (lane == 31) sums[w] = x;
  __syncthreads();
  if (w == 0) {
    int t = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    sums[lane] = t;
  }
  __syncthreads();
  *total = sums[31];
  return (w > 0 ? sums[w - 1] : 0) + x - v;
}

// ------------------------------------------------------------------ fork

// One CTA per new row: its length, the entries it shares with its parent, and the marks.
__global__ void __launch_bounds__(kPagesThreads) attn_pages_fork_mark_kernel(const __grid_constant__ ForkArgs a) {
  const int i = blockIdx.x;
  const int max_tokens = a.cols * a.page_size;
  int p = __ldg(&a.parents[i]), old_len = 0, new_len = 0;
  bool bad = p < -1 || p >= a.S;
  if (bad) p = -1;
  if (p >= 0) {
    old_len = __ldg(&a.seq_lens[p]);
    if (old_len < 0 || old_len > max_tokens) {
      bad = true;
      old_len = 0;
    }
    const long long want = (long long)old_len + (a.add != nullptr ? __ldg(&a.add[i]) : 0);
    if (want < 0 || want > (long long)a.new_cols * a.page_size) {
      bad = true;
      new_len = old_len;
    } else {
      new_len = (int)want;
    }
  }
  const int kept = min(old_len, new_len);
  const int nfull = kept / a.page_size;
  const bool part = kept % a.page_size != 0;
  const int32_t* src = a.table + (size_t)max(p, 0) * a.cols;
  int32_t* dst = a.new_table + (size_t)i * a.new_cols;
  for (int j = threadIdx.x; j < a.new_cols; j += blockDim.x) {
    int e = -1;
    if (j < nfull + (part ? 1 : 0)) {
      e = __ldg(&src[j]);
      if (e < 0 || e >= a.num_pages) {
        latch_status(ATTN_ERR_BAD_PAGE);
        e = -1;
      } else if (j < nfull) {
        atomicOr(&a.full_bits[e >> 5], 1u << (e & 31));
      } else {
        atomicOr(&a.part_bits[e >> 5], 1u << (e & 31));
        atomicMin(&a.first_part[e], i);
      }
    }
    dst[j] = e;
    if (part && j == nfull) a.row_part[i] = e;
  }
  if (threadIdx.x == 0) {
    if (bad) latch_status(ATTN_ERR_INVALID_ARG);
    if (!part) a.row_part[i] = -1;
    a.new_lens[i] = new_len;
    a.row_fresh[i] = (new_len + a.page_size - 1) / a.page_size - nfull - (part ? 1 : 0);
  }
}

// One CTA: the free pages in ascending order, and which of them each row gets.
__global__ void __launch_bounds__(kScanThreads) attn_pages_fork_scan_kernel(const __grid_constant__ ForkArgs a) {
  __shared__ int sums[32];
  const int tid = threadIdx.x;
  const int words = (a.num_pages + 31) / 32;
  const int wpt = (words + kScanThreads - 1) / kScanThreads;
  auto free_bits = [&](int w) -> uint32_t {
    uint32_t f = ~(a.full_bits[w] | a.part_bits[w]);
    if (w == words - 1 && (a.num_pages & 31) != 0) f &= (1u << (a.num_pages & 31)) - 1u;
    return f;
  };
  int mine = 0;
  for (int w = tid * wpt; w < min(words, (tid + 1) * wpt); ++w) mine += __popc(free_bits(w));
  int n_free;
  int rank = pages_scan(mine, sums, &n_free);
  for (int w = tid * wpt; w < min(words, (tid + 1) * wpt); ++w) {
    uint32_t f = free_bits(w);
    while (f != 0) {
      const int b = __ffs(f) - 1;
      a.free_list[rank++] = 32 * w + b;
      f &= f - 1;
    }
  }
  // rows in order: a part-filled page stays with the lowest row that has it, unless some row has it
  // as a full page (that row's tokens must not be written over)
  const int rpt = (a.rows + kScanThreads - 1) / kScanThreads;
  int need = 0;
  for (int i = tid * rpt; i < min(a.rows, (tid + 1) * rpt); ++i) {
    const int e = a.row_part[i];
    int keep = 0;
    if (e >= 0) {
      keep = a.first_part[e] == i && (a.full_bits[e >> 5] >> (e & 31) & 1u) == 0;
      need += 1 - keep;
    }
    a.row_keep[i] = keep;
    need += a.row_fresh[i];
  }
  int total;
  int at = pages_scan(need, sums, &total);
  for (int i = tid * rpt; i < min(a.rows, (tid + 1) * rpt); ++i) {
    a.row_rank[i] = at;
    at += a.row_fresh[i] + (a.row_part[i] >= 0 && !a.row_keep[i] ? 1 : 0);
  }
  if (tid == 0) {
    if (total > n_free) latch_status(ATTN_ERR_TOO_LARGE);
    *a.n_list = n_free;
    if (a.n_free != nullptr) *a.n_free = max(0, n_free - total);
  }
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

// CTA (row, pool x part): the row's fresh entries (first CTA of a row) and its page copy.
__global__ void __launch_bounds__(kPagesThreads)
    attn_pages_fork_move_kernel(const __grid_constant__ ForkArgs a, const __grid_constant__ PagePools pools, int parts) {
  const int i = blockIdx.x;
  const int rank = a.row_rank[i], e = a.row_part[i], n_list = *a.n_list;
  const bool copies = e >= 0 && !a.row_keep[i];
  const int to = copies && rank < n_list ? a.free_list[rank] : -1;
  if (blockIdx.y == 0) {
    const int len = a.new_lens[i];
    const int fresh = a.row_fresh[i];
    const int first = (len + a.page_size - 1) / a.page_size - fresh;
    int32_t* row = a.new_table + (size_t)i * a.new_cols;
    if (copies && threadIdx.x == 0) row[first - 1] = to;
    const int r0 = rank + (copies ? 1 : 0);
    for (int j = threadIdx.x; j < fresh; j += blockDim.x) row[first + j] = r0 + j < n_list ? a.free_list[r0 + j] : -1;
  }
  if (to < 0) return;
  for (int w = blockIdx.y; w < pools.n * parts; w += gridDim.y) {
    uint8_t* base = pools.base[w / parts];
    copy_bytes(base + (size_t)to * pools.page_bytes, base + (size_t)e * pools.page_bytes, pools.page_bytes, w % parts,
               parts);
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

__global__ void __launch_bounds__(kPagesThreads) attn_pages_compact_mark_kernel(const __grid_constant__ CompactArgs a) {
  const int s = blockIdx.x;
  bool bad;
  const int n = pages_of_row(a, s, &bad);
  if (bad && threadIdx.x == 0) latch_status(ATTN_ERR_INVALID_ARG);
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int e = a.table[(size_t)s * a.cols + j];
    if (e < 0 || e >= a.num_pages)
      latch_status(ATTN_ERR_BAD_PAGE);
    else
      atomicOr(&a.bits[e >> 5], 1u << (e & 31));
  }
}

// One CTA: with n pages in use, page ids below n stay and the others move, in ascending order,
// into the free ids below n.  No page is both a source and a destination.
__global__ void __launch_bounds__(kScanThreads) attn_pages_compact_scan_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ int sums[32];
  const int tid = threadIdx.x;
  const int words = (a.num_pages + 31) / 32;
  const int wpt = (words + kScanThreads - 1) / kScanThreads;
  const int w0 = min(words, tid * wpt), w1 = min(words, (tid + 1) * wpt);
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += __popc(a.bits[w]);
  int live;
  int before = pages_scan(mine, sums, &live);
  auto below = [&](int w) -> uint32_t {  // mask of the word's ids below `live`
    const int d = live - 32 * w;
    return d >= 32 ? 0xffffffffu : (d <= 0 ? 0u : (1u << d) - 1u);
  };
  int movers = 0;
  for (int w = w0; w < w1; ++w) {
    a.prefix[w] = before;
    before += __popc(a.bits[w]);
    movers += __popc(a.bits[w] & ~below(w));
  }
  int n_move;
  int ms = pages_scan(movers, sums, &n_move);
  int holes = 0;
  for (int w = w0; w < w1; ++w) holes += __popc(~a.bits[w] & below(w));
  int n_holes;
  int hs = pages_scan(holes, sums, &n_holes);  // as many as movers
  for (int w = w0; w < w1; ++w) {
    for (uint32_t f = a.bits[w] & ~below(w); f != 0; f &= f - 1) a.src[ms++] = 32 * w + __ffs(f) - 1;
    for (uint32_t f = ~a.bits[w] & below(w); f != 0; f &= f - 1) a.dst[hs++] = 32 * w + __ffs(f) - 1;
  }
  if (tid == 0) {
    a.counts[0] = live;
    a.counts[1] = n_move;
    if (a.n_live != nullptr) *a.n_live = live;
  }
}

// The new number of page e in use.  Movers are ranked by the pages in use before them: of those,
// live - n_move stay.
__device__ __forceinline__ int compact_to(const CompactArgs& a, int e, int live, int n_move) {
  if (e < live) return e;
  const int r = a.prefix[e >> 5] + __popc(a.bits[e >> 5] & ((1u << (e & 31)) - 1u)) - (live - n_move);
  return a.dst[r];
}

// Grid-stride over the table, the map and the pages to move.
__global__ void __launch_bounds__(kPagesThreads)
    attn_pages_compact_move_kernel(const __grid_constant__ CompactArgs a, const __grid_constant__ PagePools pools,
                                   int parts) {
  const int live = a.counts[0], n_move = a.counts[1];
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

}  // namespace attn
