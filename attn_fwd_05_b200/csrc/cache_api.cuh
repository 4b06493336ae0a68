// cache_api.cuh — host side of the 4-bit cache and page entry points of include/attn_b200.h:
// argument checks, workspace layouts and launches.  Included by attn_b200.cu after attn_api.cu,
// whose helpers (aligned, sm_count, ensure_smem, launch_status, align256) it uses.
#pragma once

#include "decode_kv4_sm100.cuh"
#include "kv4_sm100.cuh"
#include "pages_sm100.cuh"

namespace {

// A buffer of a call: null or empty ones share no bytes with any other.
struct Span {
  const void* p;
  size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// Whether a written buffer shares bytes with one that is read, or with another that is written: the
// blocks of a call have no order in which the one would be done with before the other.
template <size_t W, size_t R>
bool any_overlap(const Span (&written)[W], const Span (&read)[R]) {
  for (size_t i = 0; i < W; ++i) {
    for (const Span& r : read)
      if (overlap(written[i], r)) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(written[i], written[j])) return true;
  }
  return false;
}

// n * each bytes, at most 2^62 (no address plus that wraps around).
size_t span_bytes(long long n, size_t each) {
  constexpr size_t kMost = size_t(1) << 62;
  return n > 0 && each > kMost / (size_t)n ? kMost : (size_t)std::max(n, 0ll) * each;
}

bool kv4_head_dim(int d) { return d == 64 || d == 128 || d == 256; }
bool cache_page_size(int p) { return p == 16 || p == 32 || p == 64; }

// Sizes shared by the entry points that read a table into a 4-bit pool.  Record numbers fit an int.
// Longest row of a table: lengths and what is rounded up from them then fit 32 bits.
constexpr long long kMaxTokens = 1ll << 30;

attn_status kv4_check(const void* pool, const int32_t* table, const int32_t* seq_lens, int page_size, int S, int Hkv,
                      int d, int num_pages, int max_pages) {
  if (S < 0 || Hkv <= 0 || num_pages < 0 || max_pages <= 0) return ATTN_ERR_INVALID_ARG;
  if (!kv4_head_dim(d) || !cache_page_size(page_size)) return ATTN_ERR_UNSUPPORTED;
  if (S == 0) return ATTN_OK;
  if (table == nullptr || seq_lens == nullptr || (num_pages > 0 && pool == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(seq_lens, 4) || (num_pages > 0 && !aligned(pool, 16))) return ATTN_ERR_ALIGNMENT;
  if ((long long)max_pages * page_size > kMaxTokens) return ATTN_ERR_INVALID_ARG;
  if (num_pages > 0x7fffffffLL / Hkv / (page_size / attn::kKv4Tok)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

Span kv4_pool_span(const void* pool, int page_size, int Hkv, int d, int num_pages) {
  return {pool, span_bytes(num_pages, attn_kv4_page_bytes(Hkv, page_size, d))};
}

template <int NG>
attn_status launch_append(const attn::Kv4AppendArgs& a, unsigned grid, cudaStream_t st) {
  attn::attn_kv4_append_kernel<NG><<<grid, attn::kKv4AppendThreads, 0, st>>>(a);
  return launch_status();
}

template <int NG>
attn_status launch_gather(const attn::Kv4GatherArgs& a, unsigned grid, cudaStream_t st) {
  attn::attn_kv4_gather_kernel<NG><<<grid, attn::kKv4GatherWarps * 32, 0, st>>>(a);
  return launch_status();
}

// Launches a kernel that may be set up while the kernel before it on the stream still runs; the
// kernel waits for that one's results itself (pdl_wait).
template <typename... P, typename... A>
attn_status launch_dependent(void (*k)(P...), dim3 grid, int threads, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr;
  std::memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...) == cudaSuccess ? launch_status() : ATTN_ERR_CUDA;
}

// Launches a grid of clusters of `cluster` CTAs.
template <typename... P, typename... A>
attn_status launch_cluster(void (*k)(P...), dim3 grid, int cluster, int threads, size_t smem, cudaStream_t st,
                           const A&... args) {
  cudaLaunchAttribute attr;
  std::memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...) == cudaSuccess ? launch_status() : ATTN_ERR_CUDA;
}

struct DecKv4Layout {
  size_t off_lse, off_o, total;
  long long warps;
};

// Query heads of a segment: 8 columns of an MMA, or 16 where a group has more than 8 heads and
// the accumulators leave room (16 rows of up to 8192 tokens, 8 groups of 16: 38.7 us instead of 42.2; 32 rows at
// d = 64: 46.2 instead of 56.3).
int kv4_head_tiles(int group, int d) { return group > 8 && d <= 128 ? 2 : 1; }

DecKv4Layout kv4_layout(int S, int group, int d) {
  DecKv4Layout L;
  const int nt = kv4_head_tiles(group, d);
  L.warps = (long long)sm_count() * (d * nt <= 64 ? 4 : (d * nt <= 128 ? 3 : 2)) * 4;
  L.off_lse = align256((size_t)(S + 2) * 8);
  L.off_o = L.off_lse + align256((size_t)L.warps * 2 * 8 * nt * 4);
  L.total = L.off_o + (size_t)L.warps * 2 * 8 * nt * d * 4;
  return L;
}

template <int D, int NT>
attn_status launch_decode_kv4(const attn::DecKv4Args& a, cudaStream_t st, int slot) {
  using C = attn::DecKv4Cfg<D, NT>;
  // Few short rows go out in one launch, a cluster a segment: 7.4 us instead of 10.6 for one row of 512
  // tokens with 8 KV heads, 13.4 instead of 16.9 for 8 rows of 2048.  Not with fewer than 4 CTAs a
  // segment (16 rows of 512: 14.6 against 13.5, with d = 256 19.3 against 19.4), and not for rows that
  // could be longer than 1024 tokens a CTA (one row of 16384: 20.8 against 19.5), where the even cut over
  // all SMs gains more than the launch.  The table's width bounds the lengths, which are on the device.
  const long long segments = (long long)a.S * a.Hkv * a.n_hg, resident = (long long)sm_count() * C::CTAS_PER_SM;
  int cluster = attn::kDecKv4MaxCluster;
  while (cluster > attn::kDecKv4MinCluster && segments * cluster > resident) cluster /= 2;
  if (segments * cluster <= resident && (long long)a.max_pages * a.page_size <= attn::kDecKv4ClusterTokens * cluster) {
    attn::DecKv4Args b = a;
    b.cluster = cluster;
    auto kc = attn::attn_decode_kv4_split_kernel<D, NT, true>;
    if (!ensure_smem(kc, C::SMEM, slot + 8)) return ATTN_ERR_CUDA;
    return launch_cluster(kc, dim3((unsigned)(segments * cluster)), cluster, C::THREADS, C::SMEM, st, b);
  }
  auto k = attn::attn_decode_kv4_split_kernel<D, NT, false>;
  if (!ensure_smem(k, C::SMEM, slot)) return ATTN_ERR_CUDA;
  // no more CTAs than the longest possible rows can feed
  const double units = ((double)a.max_pages * a.page_size + attn::kDecKv4Unit - 1) / attn::kDecKv4Unit;
  const double ctas = std::ceil(a.S * units * a.Hkv * a.n_hg / (C::WARPS * attn::kDecKv4MinUnits));
  const int grid = (int)std::max(1.0, std::min(ctas, (double)sm_count() * C::CTAS_PER_SM));
  k<<<(unsigned)grid, C::THREADS, C::SMEM, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (a.S * a.Hq <= 4 * sm_count())
    return launch_dependent(attn::attn_decode_kv4_merge_kernel<D, NT, 16>, dim3(a.S * a.Hq), 16 * 32, st, a);
  return launch_dependent(attn::attn_decode_kv4_merge_kernel<D, NT, 4>, dim3(a.S * a.Hq), 4 * 32, st, a);
}

struct PagesLayout {
  size_t off[8], zero_bytes, zero_first, total;
};

// Workspace of both page operators: counts, marks (cleared by the call) and lists.
PagesLayout pages_layout(int num_pages, int rows) {
  PagesLayout L;
  const size_t words = align256(((size_t)num_pages + 31) / 32 * 4), ids = align256((size_t)num_pages * 4),
               per_row = align256((size_t)rows * 4);
  const size_t sizes[8] = {words, words, ids, ids, per_row, per_row, per_row, per_row};
  size_t at = 256;  // counts
  for (int i = 0; i < 8; ++i) {
    L.off[i] = at;
    at += sizes[i];
  }
  L.zero_bytes = 256 + 2 * words;
  L.zero_first = L.zero_bytes + ids;
  L.total = at;
  return L;
}

attn_status pools_check(void* const* pools, int n_pools, size_t page_bytes, int num_pages, attn::PagePools* out) {
  if (n_pools < 0 || (n_pools > 0 && pools == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (n_pools > attn::kMaxPools) return ATTN_ERR_TOO_LARGE;
  if (page_bytes % 16 != 0 || page_bytes > (size_t(1) << 40)) return ATTN_ERR_INVALID_ARG;
  std::memset(out, 0, sizeof(*out));
  for (int i = 0; i < n_pools; ++i) {
    if (num_pages > 0 && page_bytes > 0 && pools[i] == nullptr) return ATTN_ERR_INVALID_ARG;
    if (!aligned(pools[i], 16)) return ATTN_ERR_ALIGNMENT;
    out->base[i] = static_cast<uint8_t*>(pools[i]);
  }
  out->n = page_bytes > 0 ? n_pools : 0;
  out->page_bytes = (long long)page_bytes;
  return ATTN_OK;
}

// Whether the workspace or a pool shares bytes with another buffer of a page operator.  Pools may be one and
// the same (its pages are then moved twice, to the same places), not parts of one another.
template <size_t W, size_t R>
bool pools_overlap(const attn::PagePools& pp, int num_pages, const Span& workspace, const Span (&written)[W],
                   const Span (&read)[R]) {
  for (const Span& w : written)
    if (overlap(workspace, w)) return true;
  for (const Span& r : read)
    if (overlap(workspace, r)) return true;
  const uint8_t* sorted[attn::kMaxPools];
  const size_t bytes = span_bytes(num_pages, (size_t)pp.page_bytes);
  for (int i = 0; i < pp.n; ++i) {
    const Span pool = {pp.base[i], bytes};
    if (overlap(pool, workspace)) return true;
    for (const Span& w : written)
      if (overlap(pool, w)) return true;
    for (const Span& r : read)
      if (overlap(pool, r)) return true;
    sorted[i] = pp.base[i];
  }
  std::sort(sorted, sorted + pp.n);
  for (int i = 1; i < pp.n; ++i)
    if (sorted[i] != sorted[i - 1] && overlap({sorted[i], bytes}, {sorted[i - 1], bytes})) return true;
  return false;
}

// CTAs that share one page copy: one for every 16 KB, up to 32.
int copy_parts(size_t page_bytes) {
  return (int)std::max<size_t>(1, std::min<size_t>(32, page_bytes / 16384));
}

// One CTA that plans saves the clearing and a launch, while it has few entries and rows to walk.  Fork /
// compact in microseconds against clearing and a CTA a row: 8 x 64 entries 6.5 / 7.6 against 9.6 / 12.3, 16
// x 128 8.8 / 11.3 against 10.7 / 12.3, 32 x 128 11.7 / 15.8 against 11.3 / 14.3; 256 x 8 19.9 / 10.1 against
// 11.5 / 12.3 (a fork compares the rows' part-filled pages with one another).
bool small_table(int rows, int max_rows, int cols, int num_pages) {
  return rows <= max_rows && (long long)rows * cols <= attn::kSmallEntries && num_pages <= attn::kSmallPages;
}

// Whether the planning launch also copies: at most `bytes`, for which the 8 CTAs of a cluster are enough (256
// pages of 16 KB that could move, 4 MB: 10.9 us against 12.3; of 32 KB: 16.2).
int small_move(double copies, const attn::PagePools& pp, long long bytes) {
  return copies * pp.n * (double)pp.page_bytes <= (double)bytes;
}

}  // namespace

extern "C" {

size_t attn_kv4_page_bytes(int Hkv, int page_size, int d) {
  if (Hkv <= 0 || !kv4_head_dim(d) || !cache_page_size(page_size)) return 0;
  return (size_t)Hkv * (page_size / attn::kKv4Tok) * attn::kv4_record_bytes(d);
}

attn_status attn_kv4_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, void* kv_pool,
                            const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_new, int page_size,
                            void* k_out, void* v_out, int num_seqs, int num_new, int Hkv, int d, int num_pages,
                            int max_pages_per_seq, void* stream) {
  const attn_status chk =
      kv4_check(kv_pool, block_table, seq_lens, page_size, num_seqs, Hkv, d, num_pages, max_pages_per_seq);
  if (chk != ATTN_OK) return chk;
  if (num_new < 0 || (num_seqs == 0 && num_new > 0)) return ATTN_ERR_INVALID_ARG;
  if (num_new == 0) return ATTN_OK;
  if (k == nullptr || v == nullptr || cu_new == nullptr) return ATTN_ERR_INVALID_ARG;
  if (k_stride < (int64_t)Hkv * d || v_stride < (int64_t)Hkv * d) return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_new, 4) || (k_out && !aligned(k_out, 16)) ||
      (v_out && !aligned(v_out, 16)) || k_stride % 8 != 0 || v_stride % 8 != 0)
    return ATTN_ERR_ALIGNMENT;
  // written rows may be the rows read (each lane writes what it has read), not others of them
  const size_t row = (size_t)Hkv * d * 2, out = (size_t)num_new * row;
  const Span in_k = {k, span_bytes(num_new - 1, (size_t)k_stride * 2) + row},
             in_v = {v, span_bytes(num_new - 1, (size_t)v_stride * 2) + row};
  const bool over_k = k_out == k && out == in_k.bytes, over_v = v_out == v && out == in_v.bytes;
  const Span written[] = {{k_out, out}, {v_out, out}, kv4_pool_span(kv_pool, page_size, Hkv, d, num_pages)};
  const Span read[] = {{block_table, span_bytes(num_seqs, (size_t)max_pages_per_seq * 4)},
                       {seq_lens, (size_t)num_seqs * 4},
                       {cu_new, ((size_t)num_seqs + 1) * 4}};
  if (any_overlap(written, read) || overlap(written[2], in_k) || overlap(written[2], in_v) ||
      (!over_k && overlap(written[0], in_k)) || overlap(written[0], in_v) || (!over_v && overlap(written[1], in_v)) ||
      overlap(written[1], in_k))
    return ATTN_ERR_INVALID_ARG;
  attn::Kv4AppendArgs a;
  std::memset(&a, 0, sizeof(a));
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.pool = static_cast<uint8_t*>(kv_pool);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.cu_new = cu_new;
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.S = num_seqs;
  a.T = num_new;
  a.Hkv = Hkv;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages_per_seq;
  // as many heads a warp as leave some 48 warps to every SM (both sides: the kernel's comment)
  const long long quads = (long long)(num_new >> 2) + 2ll * num_seqs;
  a.heads = (int)std::max(1ll, std::min<long long>(Hkv, quads * Hkv / (48ll * sm_count())));
  const int warps = attn::kKv4AppendThreads / 32;
  const long long grid = (quads * ((Hkv + a.heads - 1) / a.heads) + warps - 1) / warps;
  if (grid > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (d) {
    case 64: return launch_append<1>(a, (unsigned)grid, st);
    case 128: return launch_append<2>(a, (unsigned)grid, st);
    default: return launch_append<4>(a, (unsigned)grid, st);
  }
}

attn_status attn_kv4_gather(const void* kv_pool, const int32_t* block_table, const int32_t* seq_lens, int page_size,
                            void* k, void* v, int num_seqs, int Hkv, int N, int d, int num_pages,
                            int max_pages_per_seq, void* stream) {
  const attn_status chk =
      kv4_check(kv_pool, block_table, seq_lens, page_size, num_seqs, Hkv, d, num_pages, max_pages_per_seq);
  if (chk != ATTN_OK) return chk;
  if (N < 0 || N > kMaxTokens) return ATTN_ERR_INVALID_ARG;
  if (num_seqs == 0 || N == 0) return ATTN_OK;
  if (k == nullptr || v == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return ATTN_ERR_ALIGNMENT;
  // k may be v: a lane writes V's values after K's
  const size_t out = span_bytes((long long)num_seqs * Hkv, (size_t)N * d * 2);
  const Span written[] = {{k, out}, {k == v ? nullptr : v, out}};
  const Span read[] = {kv4_pool_span(kv_pool, page_size, Hkv, d, num_pages),
                       {block_table, span_bytes(num_seqs, (size_t)max_pages_per_seq * 4)},
                       {seq_lens, (size_t)num_seqs * 4}};
  if (any_overlap(written, read)) return ATTN_ERR_INVALID_ARG;
  attn::Kv4GatherArgs a;
  std::memset(&a, 0, sizeof(a));
  a.pool = static_cast<const uint8_t*>(kv_pool);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.k = static_cast<__nv_bfloat16*>(k);
  a.v = static_cast<__nv_bfloat16*>(v);
  a.S = num_seqs;
  a.Hkv = Hkv;
  a.N = N;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages_per_seq;
  // N may be larger than any row: the warps of records past a row's end return
  const long long nrec = ((long long)N + 15) / 16;
  const long long units = nrec * num_seqs;
  if (units > 0x7fffffffLL * attn::kKv4GatherWarps / Hkv) return ATTN_ERR_INVALID_ARG;
  const unsigned grid = (unsigned)((units * Hkv + attn::kKv4GatherWarps - 1) / attn::kKv4GatherWarps);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (d) {
    case 64: return launch_gather<1>(a, grid, st);
    case 128: return launch_gather<2>(a, grid, st);
    default: return launch_gather<4>(a, grid, st);
  }
}

size_t attn_decode_paged_kv4_workspace_size(int num_seqs, int Hq, int Hkv, int d) {
  if (num_seqs < 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 || !kv4_head_dim(d)) return 0;
  return kv4_layout(num_seqs, Hq / Hkv, d).total;
}

attn_status attn_decode_paged_kv4(const void* q, const void* kv_pool, const int32_t* block_table,
                                  const int32_t* seq_lens, int page_size, void* o, float* lse, int num_seqs, int Hq,
                                  int Hkv, int d, int num_pages, int max_pages_per_seq, float scale, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  const attn_status chk =
      kv4_check(kv_pool, block_table, seq_lens, page_size, num_seqs, Hkv, d, num_pages, max_pages_per_seq);
  if (chk != ATTN_OK) return chk;
  if (num_seqs == 0) return ATTN_OK;
  if (q == nullptr || o == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || (lse != nullptr && !aligned(lse, 4))) return ATTN_ERR_ALIGNMENT;
  if ((long long)num_seqs * Hq > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  // the units of all rows are counted in 32 bits
  if ((double)num_seqs * (((double)max_pages_per_seq * page_size) / attn::kDecKv4Unit + 1.0) > 2147483647.0)
    return ATTN_ERR_INVALID_ARG;
  const int group = Hq / Hkv;
  const DecKv4Layout L = kv4_layout(num_seqs, group, d);
  if (workspace == nullptr || workspace_bytes < L.total) return ATTN_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return ATTN_ERR_ALIGNMENT;
  const size_t rows = (size_t)num_seqs * Hq;
  const Span written[] = {{o, rows * d * 2}, {lse, rows * 4}, {workspace, L.total}};
  const Span read[] = {{q, rows * d * 2},
                       kv4_pool_span(kv_pool, page_size, Hkv, d, num_pages),
                       {block_table, span_bytes(num_seqs, (size_t)max_pages_per_seq * 4)},
                       {seq_lens, (size_t)num_seqs * 4}};
  if (any_overlap(written, read)) return ATTN_ERR_INVALID_ARG;
  attn::DecKv4Args a;
  std::memset(&a, 0, sizeof(a));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.pool = static_cast<const uint8_t*>(kv_pool);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.unit_prefix = reinterpret_cast<long long*>(ws);
  a.part_lse = reinterpret_cast<float*>(ws + L.off_lse);
  a.part_o = reinterpret_cast<float*>(ws + L.off_o);
  a.S = num_seqs;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = group;
  const int nt = kv4_head_tiles(group, d);
  a.n_hg = (group + 8 * nt - 1) / (8 * nt);
  a.page_size = page_size;
  a.lg_blocks = page_size == 16 ? 0 : (page_size == 32 ? 1 : 2);
  a.num_pages = num_pages;
  a.max_pages = max_pages_per_seq;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (d) {
    case 64: return nt == 1 ? launch_decode_kv4<64, 1>(a, st, 20) : launch_decode_kv4<64, 2>(a, st, 21);
    case 128: return nt == 1 ? launch_decode_kv4<128, 1>(a, st, 22) : launch_decode_kv4<128, 2>(a, st, 23);
    default: return launch_decode_kv4<256, 1>(a, st, 24);
  }
}

size_t attn_pages_workspace_size(int num_pages, int rows) {
  if (num_pages < 0 || rows < 0) return 0;
  return pages_layout(num_pages, rows).total;
}

attn_status attn_pages_fork(const int32_t* block_table, const int32_t* seq_lens, const int32_t* parents,
                            const int32_t* add_tokens, int32_t* new_table, int32_t* new_lens, int page_size,
                            void* const* pools, int n_pools, size_t page_bytes, int num_seqs, int max_pages_per_seq,
                            int new_rows, int new_max_pages, int num_pages, int32_t* n_free, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (num_seqs < 0 || new_rows < 0 || max_pages_per_seq <= 0 || new_max_pages < max_pages_per_seq || num_pages < 0 ||
      page_size <= 0)
    return ATTN_ERR_INVALID_ARG;
  if ((long long)new_max_pages * page_size > kMaxTokens) return ATTN_ERR_INVALID_ARG;
  if ((long long)new_rows * new_max_pages > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;  // pages are counted in 32 bits
  attn::PagePools pp;
  const attn_status chk = pools_check(pools, n_pools, page_bytes, num_pages, &pp);
  if (chk != ATTN_OK) return chk;
  if ((num_seqs > 0 && (block_table == nullptr || seq_lens == nullptr)) ||
      (new_rows > 0 && (parents == nullptr || new_table == nullptr || new_lens == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(parents, 4) || !aligned(add_tokens, 4) ||
      !aligned(new_table, 4) || !aligned(new_lens, 4) || !aligned(n_free, 4))
    return ATTN_ERR_ALIGNMENT;
  const PagesLayout L = pages_layout(num_pages, new_rows);
  const size_t per_row = (size_t)new_rows * 4;
  const Span written[] = {{new_table, span_bytes(new_rows, (size_t)new_max_pages * 4)}, {new_lens, per_row}, {n_free, 4}};
  const Span read[] = {{block_table, span_bytes(num_seqs, (size_t)max_pages_per_seq * 4)},
                       {seq_lens, (size_t)num_seqs * 4},
                       {parents, per_row},
                       {add_tokens, per_row}};
  if (any_overlap(written, read)) return ATTN_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < L.total) return ATTN_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return ATTN_ERR_ALIGNMENT;
  if (pools_overlap(pp, num_pages, {workspace, L.total}, written, read)) return ATTN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  attn::ForkArgs a;
  std::memset(&a, 0, sizeof(a));
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.parents = parents;
  a.add = add_tokens;
  a.new_table = new_table;
  a.new_lens = new_lens;
  a.n_free = n_free;
  a.n_done = reinterpret_cast<int*>(ws);
  a.n_list = reinterpret_cast<int*>(ws) + 1;
  a.full_bits = reinterpret_cast<uint32_t*>(ws + L.off[0]);
  a.part_bits = reinterpret_cast<uint32_t*>(ws + L.off[1]);
  a.first_part = reinterpret_cast<int*>(ws + L.off[2]);
  a.free_list = reinterpret_cast<int*>(ws + L.off[3]);
  a.row_part = reinterpret_cast<int*>(ws + L.off[4]);
  a.row_fresh = reinterpret_cast<int*>(ws + L.off[5]);
  a.row_rank = reinterpret_cast<int*>(ws + L.off[6]);
  a.row_keep = reinterpret_cast<int*>(ws + L.off[7]);
  a.S = num_seqs;
  a.cols = max_pages_per_seq;
  a.rows = new_rows;
  a.new_cols = new_max_pages;
  a.page_size = page_size;
  a.num_pages = num_pages;
  const int parts = copy_parts(page_bytes);
  if (small_table(new_rows, attn::kSmallForkRows, new_max_pages, num_pages)) {
    const int move = small_move(new_rows, pp, attn::kSmallForkBytes), ctas = move ? attn::kSmallCluster : 1;
    const attn_status planned = launch_cluster(attn::attn_pages_fork_small_kernel, dim3(ctas), ctas, attn::kPlanThreads,
                                               (size_t)((num_pages + 31) / 32) * 8, st, a, pp, move);
    if (planned != ATTN_OK || move) return planned;
  } else {
    if (cudaMemsetAsync(ws, 0, L.zero_first, st) != cudaSuccess) return ATTN_ERR_CUDA;
    attn::attn_pages_fork_plan_kernel<<<(unsigned)std::max(new_rows, 1), attn::kPlanThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  }
  if (new_rows == 0) return ATTN_OK;
  const dim3 grid((unsigned)new_rows, (unsigned)std::max(1, std::min(pp.n * parts, 1024)));
  return launch_dependent(attn::attn_pages_fork_move_kernel, grid, attn::kPagesThreads, st, a, pp, parts);
}

attn_status attn_pages_compact(const int32_t* block_table, const int32_t* seq_lens, int32_t* new_table,
                               int32_t* page_map, int page_size, void* const* pools, int n_pools, size_t page_bytes,
                               int num_seqs, int max_pages_per_seq, int num_pages, int32_t* n_live, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (num_seqs < 0 || max_pages_per_seq <= 0 || num_pages < 0 || page_size <= 0) return ATTN_ERR_INVALID_ARG;
  if ((long long)max_pages_per_seq * page_size > kMaxTokens) return ATTN_ERR_INVALID_ARG;
  attn::PagePools pp;
  const attn_status chk = pools_check(pools, n_pools, page_bytes, num_pages, &pp);
  if (chk != ATTN_OK) return chk;
  if ((num_seqs > 0 && (block_table == nullptr || seq_lens == nullptr || new_table == nullptr)) ||
      (num_pages > 0 && page_map == nullptr))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(new_table, 4) || !aligned(page_map, 4) ||
      !aligned(n_live, 4))
    return ATTN_ERR_ALIGNMENT;
  const PagesLayout L = pages_layout(num_pages, num_seqs);
  const size_t bytes = span_bytes(num_seqs, (size_t)max_pages_per_seq * 4);
  const Span written[] = {{new_table, bytes}, {page_map, (size_t)num_pages * 4}, {n_live, 4}};
  const Span read[] = {{block_table == new_table ? nullptr : block_table, bytes}, {seq_lens, (size_t)num_seqs * 4}};
  if (any_overlap(written, read)) return ATTN_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < L.total) return ATTN_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return ATTN_ERR_ALIGNMENT;
  if (pools_overlap(pp, num_pages, {workspace, L.total}, written, read)) return ATTN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  attn::CompactArgs a;
  std::memset(&a, 0, sizeof(a));
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.new_table = new_table;
  a.page_map = page_map;
  a.n_live = n_live;
  a.n_done = reinterpret_cast<int*>(ws);
  a.counts = reinterpret_cast<int*>(ws) + 1;
  a.bits = reinterpret_cast<uint32_t*>(ws + L.off[0]);
  a.prefix = reinterpret_cast<int*>(ws + L.off[1]);
  a.src = reinterpret_cast<int*>(ws + L.off[2]);
  a.dst = reinterpret_cast<int*>(ws + L.off[3]);
  a.S = num_seqs;
  a.cols = max_pages_per_seq;
  a.page_size = page_size;
  a.num_pages = num_pages;
  const int parts = copy_parts(page_bytes);
  // a page moves into a free one, so at most half of the pool moves
  const double moves = std::min((double)num_seqs * max_pages_per_seq, num_pages / 2.0);
  if (small_table(num_seqs, attn::kSmallCompactRows, max_pages_per_seq, num_pages)) {
    const int move = small_move(moves, pp, attn::kSmallCompactBytes), ctas = move ? attn::kSmallCluster : 1;
    const attn_status planned = launch_cluster(attn::attn_pages_compact_small_kernel, dim3(ctas), ctas, attn::kPlanThreads,
                                               (size_t)((num_pages + 31) / 32) * 4, st, a, pp, move);
    if (planned != ATTN_OK || move) return planned;
  } else {
    if (cudaMemsetAsync(ws, 0, L.zero_bytes, st) != cudaSuccess) return ATTN_ERR_CUDA;
    attn::attn_pages_compact_plan_kernel<<<(unsigned)std::max(num_seqs, 1), attn::kPlanThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  }
  return launch_dependent(attn::attn_pages_compact_move_kernel, dim3((unsigned)(sm_count() * 8)), attn::kPagesThreads,
                          st, a, pp, parts);
}

}  // extern "C"
