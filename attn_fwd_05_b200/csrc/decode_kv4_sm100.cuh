// decode_kv4_sm100.cuh — one decode step over a paged K/V cache held in 4 bits, for sm_100a.
//
// What is computed is attn_decode_paged's softmax(scale q K^T) V with K and V standing for the
// cache's values x = s c + m (kv4_sm100.cuh).  The step has to read d * 9/8 bytes per cached
// token and KV head, 3.6 times fewer than the bf16 cache, so the arithmetic on those bytes is
// what has to keep up with HBM, and the kernel is built around its instruction count:
//
//   * The codes are the A operand (16 rows) of m16n8k16 MMAs and up to 8 query heads of the KV
//     group the 8 columns: S^T = K q^T has 16 tokens as rows, O^T = V^T P^T 16 channels, so no
//     row of a product is padding.  The records hold the codes in that operand's order.
//   * A 4-bit code becomes an fp16 operand without a conversion: masked into the mantissa of
//     1024 it is 1024 + c (or 1024 + 16 c, one nibble further up), and one fp16 FMA makes c - 8
//     of it, exactly.  K's scale and minimum are applied to the fp32 products,
//         q . K_j = sum_y s_jy (q_y . (c - 8)_jy) + (m_jy + 8 s_jy) sum(q_y),
//     V's scale goes into the probabilities and its minimum into one sum per head and group,
//         O_y = sum_j (p_j s_jy) (c - 8)_jy + sum_j p_j (m_jy + 8 s_jy).
//     Centring the codes keeps the rounding of p s (fp16, 11 bits) multiplied by the small signed
//     code instead of by an offset that the second sum would have to cancel.
//   * fp16 range: q is scaled by a power of two per head (its bf16 significand fits fp16's);
//     p s is scaled by a power of two per head and channel group that follows the largest p s seen, not the
//     largest s: a token of a large scale and no weight would push the others into fp16's subnormals.
//   * P^T reaches the B operand's layout with two 8x8 transposes (movmatrix) per group.
//   * The running maximum is raised only when a log2 score passes it by more than 8: one vote per
//     32 tokens in place of shuffles and a rescale.  P stays below 2^8 in between.
//
// Work split: the 32-token units of all (sequence, KV head, head group) segments form one
// stream; every warp takes a contiguous range of it of equal cost, whatever the lengths, and runs alone:
// it fetches its records with 16-byte asynchronous copies into its own ring in shared memory and
// never waits for another warp.  A segment that lies inside one warp's range is finished there; the
// others leave partials (at most two per warp) that the merge kernel joins by log-sum-exp.  Few short
// rows take one launch in place of two: a cluster of CTAs per segment, which joins them itself.
//
// What bounds it: mostly issue slots.  A 16-token tile of 128 (64) channels costs a warp 336 (233) instructions, its
// share of a segment's start and end included, 16 (8) of them MMAs, each of which holds its scheduler's
// issue port for about 8 cycles, while HBM delivers a tile per scheduler every 400 cycles.  The counters
// show 61 % of the slots taken and the MMAs' hold is another 21 %; with 64 channels it is 60 % and 15 %, and the
// rest are the waits of short segments.  64 sequences of 512 to 32768 tokens, 64 query heads on 8, d = 128: 287
// to 299 us replayed (the GPU at its power limit), 317 us called, 4.2 TB/s of cache; the loads alone (no
// arithmetic) take 213 us.  Two rows of 131071 tokens: 79 us; 96 rows of up to 2048 tokens, 16 heads, d = 64:
// 43 us.  Tried and slower, when the first batch took 273 us: the conversion into 8-bit operands for e4m3 MMAs
// (this MMA becomes conversions and f16 MMAs on this GPU: 450 us), one CTA of 16 warps (no gain), and
// tcgen05 with the codes expanded into shared memory (709 us: write, expansion and the operand's read
// take 912 cycles of shared memory per 128 tokens, of which HBM delivers as many in 794).
#pragma once

#include "kv4_sm100.cuh"
#include "pages_sm100.cuh"

namespace attn {

struct DecKv4Args {
  const __nv_bfloat16* q;      // [S, Hq, d]
  const uint8_t* pool;         // [num_pages, Hkv, page_size / 16, record]
  const int32_t* block_table;  // [S, max_pages]
  const int32_t* seq_lens;     // [S]
  __nv_bfloat16* o;            // [S, Hq, d]
  float* lse;                  // [S, Hq] or null
  long long* unit_prefix;      // workspace: [S + 1] cost of the sequences before s, then that of a range
  float* part_o;               // workspace: [warps][2][8 NT][d]
  float* part_lse;             // workspace: [warps][2][8 NT], log2 units
  int S, Hq, Hkv, group, n_hg, page_size, lg_blocks, num_pages, max_pages;
  int cluster;  // CTAs of a segment (the form for few short rows)
  float scale_log2;
};

template <int D, int NT>
struct DecKv4Cfg {
  static constexpr int NG = D / kKv4Group;
  static constexpr int ROWS = 8 * NT;  // query heads of a segment
  static constexpr int REC = kv4_record_bytes(D);
  static constexpr int UNIT = 2 * REC;  // a unit of work: 32 tokens, two records
  static constexpr int WARPS = 4;
  // resident CTAs (one fewer: 337 us instead of 301 for the batch above, 43 instead of 40.6 at d = 64, 52 instead of
  // 44 at d = 256; one more, squeezed into 128 and 96 registers, gained nothing: 282 against 281, 43 against 41
  // before p s had a scale of its own per head)
  static constexpr int CTAS_PER_SM = D * NT <= 64 ? 4 : (D * NT <= 128 ? 3 : 2);
  // units in flight a warp, the one at work included: 18 KB and less (d = 256, 16 rows of up to 8192
  // tokens: 46 us with 3 and 44 with 2; d = 128: 301 with 3, 302 with 4)
  static constexpr int STAGES = D == 64 ? 4 : (D == 128 ? 3 : 2);
  static constexpr int SMEM = WARPS * STAGES * UNIT;
  static constexpr int THREADS = WARPS * 32;
};

constexpr int kDecKv4Unit = 2 * kKv4Tok;  // tokens of a unit
constexpr int kDecKv4MinUnits = 2;        // shortest range of a warp, in units (1 to 8 measure alike)
constexpr int kDecKv4SegCost = 2;         // what starting and ending a segment costs, in units
constexpr int kDecKv4MaxCluster = 8;      // most CTAs of a segment in the form for few short rows
constexpr int kDecKv4MinCluster = 4;      // fewer CTAs: two launches
constexpr int kDecKv4ClusterTokens = 1024;  // longest row it takes, per CTA of the cluster

// ------------------------------------------------------------------ fp16 and copy helpers

// c += a b on a 16x8x16 tile, fp16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c = a b, the first step of a product.
__device__ __forceinline__ void mma_16816_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                    uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Transposes an 8x8 matrix of 16-bit elements held by the warp (two neighbours of a row a lane).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
template <int N>  // N words, N = 1, 2 or 4
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
  }
}

// The parameter words [row g, row g + 8][group] of a lane's two tokens.
template <int NG>
__device__ __forceinline__ void lds_params(uint32_t addr, uint32_t (&p)[2 * NG]) {
  constexpr int PER = 2 * NG >= 4 ? 4 : 2 * NG;
#pragma unroll
  for (int o = 0; o < 2 * NG; o += PER) {
    uint32_t w[PER];
    lds_words<PER>(addr + o * 4, w);
#pragma unroll
    for (int j = 0; j < PER; ++j) p[o + j] = w[j];
  }
}

__device__ __forceinline__ void sts_word(uint32_t addr, uint32_t w) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(w) : "memory");
}

// Larger of two pairs of fp16 numbers; NaN where either is.
__device__ __forceinline__ uint32_t max_nan_f16x2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

// A pair of bf16 powers of two 2^-e (halves: two query heads), -120 <= e <= 120.
__device__ __forceinline__ int unit_exponent(uint32_t u, int half) { return 127 - (int)((u >> (16 * half + 7)) & 0xffu); }
__device__ __forceinline__ uint32_t unit_pair(int e0, int e1) {
  return (uint32_t)(127 - e0) << 7 | (uint32_t)(127 - e1) << 23;
}
constexpr int kDecKv4UnitMin = -120, kDecKv4UnitMax = 120;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The pairs (nibble i of the low half, nibble i of the high half) of a word as fp16 c - 8,
// i = 0..3.  1024 + c - 1032 and (1024 + 16 c) / 16 - 72 are exact.  (Integers as the mantissa bits of 1024, for
// 4-bit weights: Kim et al. 2022, "Who Says Elephants Can't Run".)
__device__ __forceinline__ void kv4_centred(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t w8 = w >> 8;
  uint32_t x0, x1, x2, x3;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(x0) : "r"(w));
  asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(x1) : "r"(w));
  asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(x2) : "r"(w8));
  asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(x3) : "r"(w8));
  constexpr uint32_t kOne = 0x3c003c00u, kM1032 = 0xe408e408u;       // 1, -1032
  constexpr uint32_t kSixteenth = 0x2c002c00u, kM72 = 0xd480d480u;  // 1/16, -72
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[0]) : "r"(x0), "r"(kOne), "r"(kM1032));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[1]) : "r"(x1), "r"(kSixteenth), "r"(kM72));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[2]) : "r"(x2), "r"(kOne), "r"(kM1032));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[3]) : "r"(x3), "r"(kSixteenth), "r"(kM72));
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of x >= 0, clamped to [low, top]; of 0 the lower end, of infinity and NaN (which any
// scaling keeps) the upper end.
__device__ __forceinline__ int exponent_of(float x, int low, int top) {
  return min(top, max(low, (int)((__float_as_uint(x) >> 23) & 0xffu) - 127));
}

__device__ __forceinline__ float max_over_rows(float x) {  // over the 8 rows of an MMA fragment column
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum_over_rows(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// ------------------------------------------------------------------ the work stream

__device__ __forceinline__ int kv4_seq_len(const DecKv4Args& a, int s) {  // 0 for a length out of range
  const int len = __ldg(&a.seq_lens[s]);
  return len < 0 || len > a.max_pages * a.page_size ? 0 : len;
}

// Units of sequence s.
__device__ __forceinline__ int kv4_units(const DecKv4Args& a, int s) {
  return (kv4_seq_len(a, s) + kDecKv4Unit - 1) / kDecKv4Unit;
}

// A position in the stream: unit t of segment c (KV head and head group) of sequence s.
struct Kv4Cursor {
  int s, c, t, nt;
  __device__ __forceinline__ void forward(const DecKv4Args& a, int n) {
    t += n;
    while (t >= nt && s < a.S) {
      t -= nt;
      if (++c == a.Hkv * a.n_hg) {
        c = 0;
        nt = 0;
        while (++s < a.S && nt == 0) nt = kv4_units(a, s);
        if (nt > 0) --s;  // the loop's last increment passed the sequence found
      }
    }
  }
};

// The ranges are cut by cost: a segment of nt units counts nt + kDecKv4SegCost, the surplus in front
// of its first unit (many short rows would otherwise make their warps the last to finish: 96 rows of
// up to 2048 tokens with 16 heads take 58 us without it and 40.6 with it).
//
// Finds the first units of this CTA's warps: first[w] = {s, c, t, units of the range} (0 units: no
// work).  Every thread of the block calls it.  CTA 0 also leaves the prefix of costs for the merge.
template <int WARPS>
__device__ __forceinline__ void kv4_plan(const DecKv4Args& a, int4* first, long long* warp_sums, long long* begins) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int C = a.Hkv * a.n_hg;
  const int per_thread = (a.S + WARPS * 32 - 1) / (WARPS * 32);
  const int s0 = min(a.S, tid * per_thread), s1 = min(a.S, s0 + per_thread);
  // two sums in one scan: units in the low 32 bits, rows with work above (both below 2^31)
  long long mine = 0;
  for (int s = s0; s < s1; ++s) {
    const int nt = kv4_units(a, s);
    mine += (long long)nt + (nt > 0 ? 1ll << 32 : 0ll);
    if (blockIdx.x == 0 && (__ldg(&a.seq_lens[s]) < 0 || __ldg(&a.seq_lens[s]) > a.max_pages * a.page_size))
      latch_status(ATTN_ERR_INVALID_ARG);
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[wid] = x;
  if (tid < WARPS) first[tid] = make_int4(0, 0, 0, 0);
  __syncthreads();
  long long before = x - mine, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < wid) before += warp_sums[w];
    total += warp_sums[w];
  }
  auto cost = [](long long v) { return (v & 0xffffffffll) + (v >> 32) * kDecKv4SegCost; };
  const long long T = cost(total) * C, warps = (long long)gridDim.x * WARPS;
  const long long per = max((T + warps - 1) / warps, (long long)kDecKv4MinUnits);
  if (tid <= WARPS) begins[tid] = (total & 0xffffffffll) * C;  // of ranges past the end
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    const int nt = kv4_units(a, s);
    if (blockIdx.x == 0) a.unit_prefix[s] = cost(before);
    const long long f0 = cost(before) * C;
    const int len = nt > 0 ? nt + kDecKv4SegCost : 0;
    const long long f1 = f0 + (long long)len * C;
    for (int w = 0; w <= WARPS; ++w) {
      const long long f = ((long long)blockIdx.x * WARPS + w) * per;
      if (f >= f0 && f < f1) {
        const int c = (int)((f - f0) / len), t = max(0, (int)((f - f0) % len) - kDecKv4SegCost);
        begins[w] = (before & 0xffffffffll) * C + (long long)c * nt + t;  // units before the range
        if (w < WARPS) first[w] = make_int4(s, c, t, 0);
      }
    }
    before += (long long)nt + (nt > 0 ? 1ll << 32 : 0ll);
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.unit_prefix[a.S] = cost(total);
    a.unit_prefix[a.S + 1] = per;
  }
  __syncthreads();
  if (tid < WARPS) first[tid].w = (int)(begins[tid + 1] - begins[tid]);
  __syncthreads();
}

// ------------------------------------------------------------------ joining partials

template <int D, int W>
struct Kv4JoinSmem {
  float m[W], l[W], o[W][D];
};

// The block's W warps join np partials, at(k) the row of partial k, by their log-sum-exp, and write query
// head `out` (a row of o and lse).  np = 0: an empty row.  The warps take every W-th partial.
template <int D, int W, typename At>
__device__ __forceinline__ void kv4_join(const DecKv4Args& a, int np, At at, size_t out, Kv4JoinSmem<D, W>& sh) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float M = -INFINITY;
  for (int k = threadIdx.x; k < np; k += W * 32) M = fmaxf(M, a.part_lse[at(k)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) sh.m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) M = fmaxf(M, sh.m[w]);
  const float u = M == -INFINITY ? 0.f : M;
  float acc[PER], L = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int k = warp; k < np; k += W) {
    const size_t pi = at(k);
    const float x = a.part_lse[pi], e = ex2(x - u);
    if (x == -INFINITY) continue;  // a warp without units: its O is not written
    const float* po = a.part_o + pi * D + lane * PER;
    L += e;
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const float2 v = *reinterpret_cast<const float2*>(po + i);
      acc[i] += e * v.x;
      acc[i + 1] += e * v.y;
    }
  }
  if (lane == 0) sh.l[warp] = L;
#pragma unroll
  for (int i = 0; i < PER; ++i) sh.o[warp][lane * PER + i] = acc[i];
  __syncthreads();
  if (warp == 0) {
    L = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      L += sh.l[w];
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] += sh.o[w][lane * PER + i];
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    __nv_bfloat16* dst = a.o + out * D + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; i += 2)
      *reinterpret_cast<uint32_t*>(dst + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0 && a.lse != nullptr) a.lse[out] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
  }
}

// ------------------------------------------------------------------ split kernel

// CLUSTER: the form for few short rows, in one launch.  A cluster of a.cluster CTAs has one segment,
// cut evenly over its warps, and joins their partials itself after a barrier.
template <int D, int NT, bool CLUSTER>
__global__ void __launch_bounds__(DecKv4Cfg<D, NT>::THREADS, DecKv4Cfg<D, NT>::CTAS_PER_SM)
    attn_decode_kv4_split_kernel(const __grid_constant__ DecKv4Args a) {
  using C = DecKv4Cfg<D, NT>;
  constexpr int NG = C::NG;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int4 first[C::WARPS];
  __shared__ long long warp_sums[C::WARPS], begins[C::WARPS + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;  // row and column pair of the MMA fragments
  const int wid = blockIdx.x * C::WARPS + warp;
  int4 f;
  if constexpr (CLUSTER) {
    const int k = blockIdx.x / a.cluster, C_ = a.Hkv * a.n_hg;
    f = make_int4(k / C_, k % C_, 0, 0);
    const int len = __ldg(&a.seq_lens[f.x]);
    if ((len < 0 || len > a.max_pages * a.page_size) && lane == 0) latch_status(ATTN_ERR_INVALID_ARG);
    const int nt = kv4_units(a, f.x), warps = a.cluster * C::WARPS, per = (nt + warps - 1) / warps;
    f.z = min(nt, wid % warps * per);
    f.w = min(per, nt - f.z);
    if (f.w == 0 && lane < C::ROWS) a.part_lse[(size_t)2 * wid * C::ROWS + lane] = -INFINITY;
  } else {
    kv4_plan<C::WARPS>(a, first, warp_sums, begins);
    pdl_launch_dependents();
    f = first[warp];
    if (f.w == 0) return;
  }
  const int n = f.w;
  const uint32_t ring = smem_u32(smem) + warp * (C::STAGES * C::UNIT);

  // ---- fetch side: lane l keeps the record number of tile l % 2 of unit l / 2 of the current
  // batch of 16 units (-1: past the row's end, or its page is out of range), and of the next
  // batch, whose table loads are then in flight long before they are needed
  Kv4Cursor fc{f.x, f.y, f.z, 0};
  fc.nt = kv4_units(a, fc.s);
  if (n > 0) fc.forward(a, lane >> 1);
  auto record_of = [&](int unit) -> int {
    if (unit >= n || fc.s >= a.S) return -1;
    const int tile = 2 * fc.t + (lane & 1);
    if (tile * kKv4Tok >= kv4_seq_len(a, fc.s)) return -1;
    const int page = __ldg(&a.block_table[(size_t)fc.s * a.max_pages + (tile >> a.lg_blocks)]);
    if (page < 0 || page >= a.num_pages) {
      latch_status(ATTN_ERR_BAD_PAGE);
      return -1;
    }
    return ((page * a.Hkv + fc.c / a.n_hg) << a.lg_blocks) + (tile & ((1 << a.lg_blocks) - 1));
  };
  int rec_cur = record_of(lane >> 1);
  int rec_next = -1;
  if (n > 16) {
    fc.forward(a, 16);
    rec_next = record_of(16 + (lane >> 1));
  }
  uint32_t good = 0;  // bits 2 (i % 16) + tile: fetched
  auto issue = [&](int issued, uint32_t in) {
    if (issued < n) {
      if ((issued & 15) == 0 && issued > 0) {
        rec_cur = rec_next;
        if (issued + 16 < n) {
          fc.forward(a, 16);
          rec_next = record_of(issued + 16 + (lane >> 1));
        }
      }
      const int b = 2 * (issued & 15);
      const int r0 = __shfl_sync(0xffffffffu, rec_cur, b), r1 = __shfl_sync(0xffffffffu, rec_cur, b + 1);
      good = (good & ~(3u << b)) | ((r0 >= 0 ? 1u : 0u) << b) | ((r1 >= 0 ? 2u : 0u) << b);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rec = x == 0 ? r0 : r1;
        if (rec >= 0) {
          kv4_fetch_record<C::REC>(in + x * C::REC, a.pool + (size_t)rec * C::REC, lane);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < C::STAGES - 1; ++i) issue(i, ring + i * C::UNIT);

  // ---- the current segment
  int cs = f.x, cc = f.y;  // sequence, and KV head and head group
  int left = kv4_seq_len(a, cs) - f.z * kDecKv4Unit;  // tokens of the row from the current unit on
  bool cut = f.z > 0;      // the segment began in an earlier warp's range
  uint32_t qf[NT][NG * 4][2];   // B fragments of q, scaled per head
  float qs[NT][NG][2];          // sum of the scaled q over a group, heads 2t and 2t + 1
  float fac[NT][2];             // what turns the product with the scaled q and K into a log2 score
  uint32_t kmul;                // what K's parameters are multiplied by: bf16 2^-h, and 8 times that above
  float m[NT][2];               // reference of the exponentials (log2 score)
  float l[NT][2];               // sum of exponentials (this lane's tokens)
  float zs[NT][NG][2];          // sum of p (m + 8 s) (this lane's tokens)
  float oc[NT][NG * 4][4];      // O^T / 2^es: rows 8g + 2mt (+1), heads 2t, 2t + 1
  uint32_t unit[NT][NG];        // 2^-es of heads 2t and 2t + 1, what p s is multiplied by
  auto head_of = [&](int c) -> int { return c / a.n_hg * a.group + c % a.n_hg * C::ROWS; };
  auto rows_of = [&](int c) -> int { return min(C::ROWS, a.group - c % a.n_hg * C::ROWS); };
  auto begin = [&]() {
    const int nrows = rows_of(cc), hq0 = head_of(cc);
    int e[NT], largest = -100;  // exponents of the largest elements
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint2 raw[NG * 4];
      uint32_t big = 0;  // magnitudes of bf16 values order like their bits
#pragma unroll
      for (int ks = 0; ks < NG * 4; ++ks) {
        // channels 64 y + 16 t + 4 (ks % 4) .. of head g
        raw[ks] = nt * 8 + g < nrows
                      ? __ldg(reinterpret_cast<const uint2*>(a.q + ((size_t)cs * a.Hq + hq0 + nt * 8 + g) * D +
                                                             16 * t + (ks >> 2) * 64 + (ks & 3) * 4))
                      : make_uint2(0, 0);
        big = max(big, max((raw[ks].x << 16) & 0x7fff0000u, raw[ks].x & 0x7fff0000u));
        big = max(big, max((raw[ks].y << 16) & 0x7fff0000u, raw[ks].y & 0x7fff0000u));
      }
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // largest element to [2^13, 2^14): fp16 then holds every element down to 2^-30 of it exactly
      e[nt] = exponent_of(__uint_as_float(big), -100, 127);
      largest = max(largest, e[nt]);
      const float down = pow2i(13 - e[nt]);
#pragma unroll
      for (int ks = 0; ks < NG * 4; ++ks) {
        qf[nt][ks][0] = pack_f16x2(bf16lo_to_f32(raw[ks].x) * down, bf16hi_to_f32(raw[ks].x) * down);
        qf[nt][ks][1] = pack_f16x2(bf16lo_to_f32(raw[ks].y) * down, bf16hi_to_f32(raw[ks].y) * down);
      }
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        float s4[4];
        mma_16816_f16_first(s4, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, qf[nt][4 * y][0], qf[nt][4 * y][1]);
#pragma unroll
        for (int ks = 1; ks < 4; ++ks)
          mma_16816_f16(s4, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, qf[nt][4 * y + ks][0],
                        qf[nt][4 * y + ks][1]);
        qs[nt][y][0] = s4[0];
        qs[nt][y][1] = s4[1];
        zs[nt][y][0] = zs[nt][y][1] = 0.f;
        unit[nt][y] = unit_pair(kDecKv4UnitMin, kDecKv4UnitMin);
      }
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < NG * 4; ++i) oc[nt][i][0] = oc[nt][i][1] = oc[nt][i][2] = oc[nt][i][3] = 0.f;
    }
    // K's parameters take the factor 2^-13 that q does not have, so that the products overflow only where q . K
    // does; where scale times q is past fp32 (and K small, if the scores are finite), the factor stays in q
    const bool far = __any_sync(0xffffffffu, exponent_of(a.scale_log2, -126, 127) + largest > 125);
    const int h = far ? 0 : 13;
    kmul = far ? kBf16One | kBf16Eight << 16 : (kBf16One | kBf16Eight << 16) - 0x06800680u;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        // this lane's e belongs to head g; the fragments of the products want heads 2t and 2t + 1.  Kept above 0,
        // where all scores are 0 to within 2^-21 anyway: -inf of a masked slot has to stay -inf.
        const int ex = __shfl_sync(0xffffffffu, e[nt], 8 * t + 4 * hh) - 13 + h;
        fac[nt][hh] = fminf(fmaxf(a.scale_log2 * pow2i(ex), __int_as_float(1)), 3.4028234663852886e38f);
      }
  };
  if (n > 0) begin();

  uint32_t out = ring;
  for (int i = 0; i < n; ++i) {
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();
    const uint32_t have = (good >> (2 * (i & 15))) & 3u;  // read before issue() reuses the bits
    // into the stage of unit i - 1, which every lane has left
    issue(i + C::STAGES - 1, out == ring ? ring + (C::STAGES - 1) * C::UNIT : out - C::UNIT);
    // ---- S^T = (c - 8) q^T of both tiles, scaled and shifted per group
    float x[2][NT][4];       // products: [tile][..][row g: heads 2t, 2t+1; row g + 8: ...]
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const uint32_t base = out + tile * C::REC;
      uint32_t kp[2 * NG];  // parameters of this lane's tokens: [row g, g + 8][group]
      lds_params<NG>(base + 1024 * NG + g * 8 * NG, kp);
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        const uint4 u = lds128(base + 512 * y + lane * 16);
        uint32_t lo[2][4], hi[2][4];  // [word][pair] of rows g and g + 8
        kv4_centred(u.x, lo[0]);
        kv4_centred(u.y, lo[1]);
        kv4_centred(u.z, hi[0]);
        kv4_centred(u.w, hi[1]);
        const float s0 = fma_bf16(kp[y], kmul, 0.f), s1 = fma_bf16(kp[NG + y], kmul, 0.f);
        const float z0 = fma_bf16(kp[y], kmul >> 16, fma_bf16(kp[y] >> 16, kmul, 0.f));
        const float z1 = fma_bf16(kp[NG + y], kmul >> 16, fma_bf16(kp[NG + y] >> 16, kmul, 0.f));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float c[4];
          float* xx = x[tile][nt];
          mma_16816_f16_first(c, lo[0][0], hi[0][0], lo[0][1], hi[0][1], qf[nt][4 * y][0], qf[nt][4 * y][1]);
#pragma unroll
          for (int ks = 1; ks < 4; ++ks)
            mma_16816_f16(c, lo[ks >> 1][2 * (ks & 1)], hi[ks >> 1][2 * (ks & 1)], lo[ks >> 1][2 * (ks & 1) + 1],
                          hi[ks >> 1][2 * (ks & 1) + 1], qf[nt][4 * y + ks][0], qf[nt][4 * y + ks][1]);
          if (y == 0) {
            xx[0] = fmaf(s0, c[0], z0 * qs[nt][y][0]);
            xx[1] = fmaf(s0, c[1], z0 * qs[nt][y][1]);
            xx[2] = fmaf(s1, c[2], z1 * qs[nt][y][0]);
            xx[3] = fmaf(s1, c[3], z1 * qs[nt][y][1]);
          } else {
            xx[0] = fmaf(s0, c[0], fmaf(z0, qs[nt][y][0], xx[0]));
            xx[1] = fmaf(s0, c[1], fmaf(z0, qs[nt][y][1], xx[1]));
            xx[2] = fmaf(s1, c[2], fmaf(z1, qs[nt][y][0], xx[2]));
            xx[3] = fmaf(s1, c[3], fmaf(z1, qs[nt][y][1], xx[3]));
          }
        }
      }
    }
    if (left < kDecKv4Unit || have != 3u) {
      // tokens past the row's end or on a page out of range: whatever their slots hold must
      // not reach a sum.  This lane's rows are tokens 4 (g/2) + g%2 and two further.
#pragma unroll
      for (int tile = 0; tile < 2; ++tile)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (tile * kKv4Tok + 4 * (g >> 1) + (g & 1) + 2 * r >= left || !((have >> tile) & 1u)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[tile][nt][2 * r] = x[tile][nt][2 * r + 1] = -INFINITY;
#pragma unroll
            for (int y = 0; y < NG; ++y) sts_word(out + tile * C::REC + 1088 * NG + ((2 * g + r) * NG + y) * 4, 0u);
          }
      __syncwarp();
    }
    // ---- references: raised when a score passes m by 8
    bool raise = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        top[nt][hh] = fmaxf(fmaxf(x[0][nt][hh], x[0][nt][2 + hh]), fmaxf(x[1][nt][hh], x[1][nt][2 + hh]));
        raise |= fmaf(top[nt][hh], fac[nt][hh], -m[nt][hh]) > 8.0f;
      }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float al[2];
        int less[2];  // 2^es falls with the weights seen so far, by whole powers of two
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float to = fmaxf(m[nt][hh], max_over_rows(top[nt][hh]) * fac[nt][hh]);
          al[hh] = to == -INFINITY ? 1.0f : ex2(m[nt][hh] - to);
          less[hh] = to == -INFINITY ? 0 : (int)fminf(ceilf(to - m[nt][hh]), 240.0f);
          m[nt][hh] = to;
          l[nt][hh] *= al[hh];
        }
#pragma unroll
        for (int y = 0; y < NG; ++y) {
          int es[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int was = unit_exponent(unit[nt][y], hh);
            es[hh] = max(kDecKv4UnitMin, was - less[hh]);
            const float down = al[hh] * pow2i(min(was - es[hh], 126));  // al is 0 where that is more than 126
            zs[nt][y][hh] *= al[hh];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              oc[nt][4 * y + mt][hh] *= down;
              oc[nt][4 * y + mt][2 + hh] *= down;
            }
          }
          unit[nt][y] = unit_pair(es[0], es[1]);
        }
      }
    }
    // ---- P, the sums of its lane's tokens, and p s / 2^es in fp16
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const float u = m[nt][hh] == -INFINITY ? 0.f : m[nt][hh];
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
          x[tile][nt][hh] = ex2(fmaf(x[tile][nt][hh], fac[nt][hh], -u));
          x[tile][nt][2 + hh] = ex2(fmaf(x[tile][nt][2 + hh], fac[nt][hh], -u));
        }
        l[nt][hh] += (x[0][nt][hh] + x[0][nt][2 + hh]) + (x[1][nt][hh] + x[1][nt][2 + hh]);
      }
    uint32_t ps[2][NG][NT][2];  // [tile][group][..][row g, g + 8]: heads 2t, 2t + 1
    uint32_t most = 0;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      uint32_t vp[2 * NG];
      lds_params<NG>(out + tile * C::REC + 1088 * NG + g * 8 * NG, vp);
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        const uint32_t w0 = vp[y], w1 = vp[NG + y];
        const float z0 = fma_bf16(w0, kBf16Eight, fma_bf16(w0 >> 16, kBf16One, 0.f));
        const float z1 = fma_bf16(w1, kBf16Eight, fma_bf16(w1 >> 16, kBf16One, 0.f));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float* p = x[tile][nt];
          const uint32_t u0 = unit[nt][y], u1 = u0 >> 16;
          zs[nt][y][0] = fmaf(p[0], z0, fmaf(p[2], z1, zs[nt][y][0]));
          zs[nt][y][1] = fmaf(p[1], z0, fmaf(p[3], z1, zs[nt][y][1]));
          float s0 = fma_bf16(w0, u0, 0.f), s1 = fma_bf16(w0, u1, 0.f), s2 = fma_bf16(w1, u0, 0.f), s3 = fma_bf16(w1, u1, 0.f);
          mul2(s0, s1, p[0], p[1]);
          mul2(s2, s3, p[2], p[3]);
          ps[tile][y][nt][0] = pack_f16x2(s0, s1);
          ps[tile][y][nt][1] = pack_f16x2(s2, s3);
          most = max_nan_f16x2(most, max_nan_f16x2(ps[tile][y][nt][0], ps[tile][y][nt][1]));
        }
      }
    }
    // A product of 2^15 or more (its half plus 0x0800 reaches the sign), or NaN, as 0 times an s / 2^es past fp32 is:
    // 2^es becomes a power of two at most the largest product p s of the unit, which leaves 15 powers of
    // two above it, and 14 below it before the fp16 steps grow.
    if (__any_sync(0xffffffffu, ((most + 0x08000800u) & 0x80008000u) != 0)) {
#pragma unroll
      for (int y = 0; y < NG; ++y)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[2][2][2], big[2] = {0.f, 0.f};  // p s: [tile][row g, g + 8][head]
#pragma unroll
          for (int tile = 0; tile < 2; ++tile) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              uint32_t vp[1];
              lds_words<1>(out + tile * C::REC + 1088 * NG + ((2 * g + r) * NG + y) * 4, vp);
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                w[tile][r][hh] = x[tile][nt][2 * r + hh] * bf16lo_to_f32(vp[0]);
                big[hh] = fmaxf(big[hh], w[tile][r][hh]);
              }
            }
          }
          int es[2];
          float up[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int was = unit_exponent(unit[nt][y], hh);
            es[hh] = max(was, exponent_of(max_over_rows(big[hh]), kDecKv4UnitMin, kDecKv4UnitMax));
            up[hh] = pow2i(-es[hh]);
            const float down = pow2i(max(was - es[hh], -126));
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              oc[nt][4 * y + mt][hh] *= down;
              oc[nt][4 * y + mt][2 + hh] *= down;
            }
          }
          unit[nt][y] = unit_pair(es[0], es[1]);
#pragma unroll
          for (int tile = 0; tile < 2; ++tile)
#pragma unroll
            for (int r = 0; r < 2; ++r) ps[tile][y][nt][r] = pack_f16x2(w[tile][r][0] * up[0], w[tile][r][1] * up[1]);
        }
    }
    // ---- O^T += (c - 8)^T (p s)^T
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const uint32_t base = out + tile * C::REC;
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          b[nt][0] = movmatrix_trans(ps[tile][y][nt][0]);
          b[nt][1] = movmatrix_trans(ps[tile][y][nt][1]);
        }
        const uint4 u = lds128(base + 512 * NG + 512 * y + 128 * t + 16 * (g ^ (2 * t)));
        uint32_t p01[4], p23[4];  // tokens b = 0, 1 and b = 2, 3: channels c of a half of the unit
        kv4_centred(u.x, p01);
        kv4_centred(u.z, p23);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_16816_f16(oc[nt][4 * y + mt], p01[2 * mt], p01[2 * mt + 1], p23[2 * mt], p23[2 * mt + 1], b[nt][0],
                          b[nt][1]);
        kv4_centred(u.y, p01);
        kv4_centred(u.w, p23);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_16816_f16(oc[nt][4 * y + 2 + mt], p01[2 * mt], p01[2 * mt + 1], p23[2 * mt], p23[2 * mt + 1],
                          b[nt][0], b[nt][1]);
      }
    }
    out = out + C::UNIT == ring + C::STAGES * C::UNIT ? ring : out + C::UNIT;

    // ---- end of the segment, or of this warp's range
    const bool end = left <= kDecKv4Unit;
    left -= kDecKv4Unit;
    if (end || i == n - 1) {
      const bool whole = !CLUSTER && end && !cut;
      const int nrows = rows_of(cc), hq0 = head_of(cc);
      const size_t prow = (size_t)(2 * wid + (CLUSTER || cut ? 0 : 1)) * C::ROWS;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float sum = sum_over_rows(l[nt][hh]);
          const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;  // NaN stays
          const float lse2 = sum != 0.0f ? m[nt][hh] + log2f(sum) : -INFINITY;
          const int row = nt * 8 + 2 * t + hh;
#pragma unroll
          for (int y = 0; y < NG; ++y) {
            const float z = sum_over_rows(zs[nt][y][hh]);
            const float up = pow2i(unit_exponent(unit[nt][y], hh));
            float v[8];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              v[2 * mt] = fmaf(oc[nt][4 * y + mt][hh], up, z) * inv;
              v[2 * mt + 1] = fmaf(oc[nt][4 * y + mt][2 + hh], up, z) * inv;
            }
            if (row < nrows) {
              const int ch = 64 * y + 8 * g;
              if (whole) {
                *reinterpret_cast<uint4*>(a.o + ((size_t)cs * a.Hq + hq0 + row) * D + ch) =
                    make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                               pack_bf16x2(v[6], v[7]));
              } else {
                float4* dst = reinterpret_cast<float4*>(a.part_o + (prow + row) * D + ch);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
              }
            }
          }
          if (g == 0 && row < nrows) {
            if (!whole)
              a.part_lse[prow + row] = lse2;
            else if (a.lse != nullptr)
              a.lse[(size_t)cs * a.Hq + hq0 + row] = lse2 * 0.6931471805599453f;
          }
        }
      if (i + 1 < n) {
        if (++cc == a.Hkv * a.n_hg) {
          cc = 0;
          do {  // a row with work follows, since the range goes on
            ++cs;
          } while (cs < a.S - 1 && kv4_seq_len(a, cs) == 0);
        }
        left = kv4_seq_len(a, cs);
        cut = false;
        begin();
      }
    }
  }
  cp_async_wait<0>();
  if constexpr (CLUSTER) {
    __shared__ Kv4JoinSmem<D, C::WARPS> sh;
    cluster_barrier();
    const int rank = blockIdx.x % a.cluster, nrows = rows_of(f.y);
    const int w0 = blockIdx.x / a.cluster * (a.cluster * C::WARPS);
    for (int row = rank; row < nrows; row += a.cluster) {
      auto at = [&](int k) -> size_t { return (size_t)2 * (w0 + k) * C::ROWS + row; };
      kv4_join<D, C::WARPS>(a, kv4_units(a, f.x) > 0 ? a.cluster * C::WARPS : 0, at,
                            (size_t)f.x * a.Hq + head_of(f.y) + row, sh);
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ merge kernel

// One CTA per (sequence, query head): joins the partials of a segment that more than one warp's
// range shares; writes the rows of empty sequences.  Few rows have many partials each (one per warp
// of the split kernel that had a part of the row) and get 16 warps; many rows have few each and
// get 4.  Measured on two rows of 131071 tokens (110 partials a head): 21 us with 4 warps, 9 us with 16.
template <int D, int NT, int W>
__global__ void __launch_bounds__(W * 32) attn_decode_kv4_merge_kernel(const __grid_constant__ DecKv4Args a) {
  using C = DecKv4Cfg<D, NT>;
  __shared__ Kv4JoinSmem<D, W> sh;
  const int s = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq;
  pdl_wait();
  const long long p0 = a.unit_prefix[s], p1 = a.unit_prefix[s + 1], per = a.unit_prefix[a.S + 1];
  const int nt = max(0, (int)(p1 - p0) - kDecKv4SegCost);
  const int in_kv = h % a.group;
  const int c = (h / a.group) * a.n_hg + in_kv / C::ROWS;
  const int row = in_kv % C::ROWS;
  // the costs of the segment's first unit and of the one after its last
  const long long f0 = p0 * (a.Hkv * a.n_hg) + (long long)c * (nt + kDecKv4SegCost) + kDecKv4SegCost, f1 = f0 + nt;
  const long long w0 = f0 / per;
  const int np = nt > 0 ? (int)((f1 - 1) / per - w0) + 1 : 0;
  if (np == 1) return;  // finished by the warp that had all of it
  // the first warp's partial is the one it ended its range with (slot 1), the others' began before them
  auto at = [&](int k) -> size_t { return (size_t)(2 * (w0 + k) + (k == 0 ? 1 : 0)) * C::ROWS + row; };
  kv4_join<D, W>(a, np, at, (size_t)s * a.Hq + h, sh);
}

}  // namespace attn
