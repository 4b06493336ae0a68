// kv4_sm100.cuh — the 4-bit paged K/V cache: record layout, the quantizing append and the
// gather back to bf16, for sm_100a.
//
// A cached value is x = s c + m with a 4-bit code c and, per token and group of 64 channels,
// a bf16 scale s and a bf16 minimum m.  Sixteen tokens of one KV head form a record of
// 1152 (d / 64) bytes that holds K and V, so that the decode pass fetches everything it needs
// of 16 tokens with one contiguous, 128-byte aligned read.  Inside a record the codes lie in
// the order in which the lanes of a warp-level MMA take them (see record offsets below):
// the decode kernel then reads every operand with conflict-free 16-byte shared-memory loads
// and spends no instruction on moving codes between lanes.
#pragma once

#include <cuda_fp16.h>

#include "sm100_common.cuh"

namespace attn {

constexpr int kKv4Tok = 16;        // tokens per record
constexpr int kKv4Group = 64;      // channels per scale
constexpr int kKv4GroupBytes = 1152;  // record bytes per channel group: 512 K + 512 V codes, 64 + 64 parameters

// Record offsets.  token = 4a + 2 b1 + b0, channel = 64 y + x, NG = d / 64 groups:
//   K codes   512 y + ((2a + b0) 4 + x/16) 16 + 8 b1 + 4 ((x/8) % 2): 8 channels a word, channel
//             j = x % 8 in nibble j/2 + 4 (j % 2), so that a masked word holds two
//             neighbouring channels in its two halves
//   V codes   512 NG + 512 y + 128 a + 16 ((x/8) ^ 2a) + 8 b1 + 4 ((x/4) % 2): 4 channels of two
//             tokens a word, token b0 in half b0, channel x % 4 in nibble x % 4 of the half
//   K params  1024 NG + 4 (((2a + b0) 2 + b1) NG + y): s in the low half, m in the high half
//   V params  1088 NG + the same
__host__ __device__ constexpr int kv4_record_bytes(int d) { return (d / kKv4Group) * kKv4GroupBytes; }

__device__ __forceinline__ int kv4_k_code_off(int y, int a, int b0, int b1, int j) {  // j = x / 8
  return 512 * y + ((2 * a + b0) * 4 + (j >> 1)) * 16 + 8 * b1 + 4 * (j & 1);
}
template <int NG>
__device__ __forceinline__ int kv4_v_unit_off(int y, int a, int j) {
  return 512 * NG + 512 * y + 128 * a + 16 * (j ^ (2 * a));
}
template <int NG>
__device__ __forceinline__ int kv4_param_off(int v, int a, int b0, int b1) {  // word of group 0
  return 1024 * NG + 64 * NG * v + 4 * (((2 * a + b0) * 2 + b1) * NG);
}

struct Kv4AppendArgs {
  const __nv_bfloat16* k;  // [T, Hkv, d], tokens k_stride elements apart
  const __nv_bfloat16* v;
  uint8_t* pool;               // [num_pages, Hkv, page_size / 16, record]
  const int32_t* block_table;  // [S, max_pages]
  const int32_t* seq_lens;     // [S], with the new tokens
  const int32_t* cu_new;       // [S + 1]
  __nv_bfloat16* k_out;        // [T, Hkv, d] or null
  __nv_bfloat16* v_out;
  long long k_stride, v_stride;
  int S, T, Hkv, page_size, num_pages, max_pages;
};

// One lane's 8 channels of a group whose 64 channels lie in 8 neighbouring lanes: the group's
// scale and minimum (packed s | m << 16) and the codes as floats in r[0..7].
//
// c = nearest integer to (x - m) / s, ties to even, of the exact quotient.  The fast path forms
// (x - m) * rcp(s): the subtraction is exact or off by 2^-24, the product by 2^-22 relative,
// so for quotients up to 15.1 the value is within 2^-17 of the exact one; a value that close to
// a border between two codes (k + 1/2) is redone in 64 bits, where the quotient of these
// 8-bit significands is never rounded onto or across a border.
__device__ __forceinline__ uint32_t kv4_quantize8(const uint4& x, float (&r)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
  const __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
  const __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  // (minimum, -maximum) in one word: a single minimum per shuffle serves both
  __nv_bfloat162 e = __halves2bfloat162(__hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn)),
                                        __hneg(__hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx))));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    uint32_t u = *reinterpret_cast<uint32_t*>(&e);
    u = __shfl_xor_sync(0xffffffffu, u, o);
    e = __hmin2_nan(e, *reinterpret_cast<__nv_bfloat162*>(&u));
  }
  const float lo = __low2float(e) + 0.0f;  // a zero minimum is stored as +0
  const float hi = 0.0f - __high2float(e);
  const float span = hi - lo;
  if (!(span <= 3.4028234663852886e38f)) {  // infinite or NaN values, or a range past fp32: the group is NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = 0.0f;
    return 0x7fc07fc0u;
  }
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(span, 15.0f));
  const float s = __bfloat162float(sb);
  float xv[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    xv[2 * i] = bf16lo_to_f32(w[i]);
    xv[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
  if (span == 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = 0.0f;
    return (uint32_t)__bfloat16_as_ushort(sb) | (__float_as_uint(lo) & 0xffff0000u);
  }
  bool redo = s < 7.7e-34f;  // 2^-110: rcp(s) may overflow
  if (!redo) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = (xv[i] - lo) * inv;
      r[i] = (u + 12582912.0f) - 12582912.0f;  // 1.5 * 2^23: round to the nearest integer
      far = fmaxf(far, fabsf(u - r[i]));
    }
    redo = far > 0.5f - 1.52587890625e-5f;  // 2^-16
  }
  if (redo) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double q = ((double)xv[i] - (double)lo) / (double)s;
      r[i] = q >= 0.0 ? (float)fmin(rint(q), 15.0) : 0.0f;  // 0 / 0 (the scale underflowed): code 0
    }
  }
  return (uint32_t)__bfloat16_as_ushort(sb) | (__float_as_uint(lo) & 0xffff0000u);
}

// Values s c + m of 8 codes, rounded to bf16.
__device__ __forceinline__ uint4 kv4_values8(const float (&r)[8], uint32_t sm) {
  const float s = bf16lo_to_f32(sm), m = bf16hi_to_f32(sm);
  return make_uint4(pack_bf16x2(fmaf(s, r[0], m), fmaf(s, r[1], m)), pack_bf16x2(fmaf(s, r[2], m), fmaf(s, r[3], m)),
                    pack_bf16x2(fmaf(s, r[4], m), fmaf(s, r[5], m)), pack_bf16x2(fmaf(s, r[6], m), fmaf(s, r[7], m)));
}

// Largest s in [0, S) with (cu[s] >> 2) + 2 s <= q: sequence s owns the quads from there on.
// Its n tokens touch at most n/4 + 2 aligned quads of positions, which is what the next
// sequence's first quad leaves room for.  32 probes a step, one per lane.
__device__ __forceinline__ int kv4_find_seq(const int32_t* cu, int S, long long q, int lane) {
  int lo = 0, n = S;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool below = lane * step < n && ((long long)(__ldg(&cu[at]) >> 2) + 2ll * at) <= q;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int k = m == 0 ? 0 : 31 - __clz(m);  // for an increasing cu the probes are true up to k
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// One warp per (aligned quad of positions, KV head): lane = 8 (token of the quad) + (8-channel
// chunk).  The reads are bf16 rows of 128 bytes a group; the quad's K codes and V codes are
// one 128-byte line a group each.
template <int NG>
__global__ void __launch_bounds__(256) attn_kv4_append_kernel(const __grid_constant__ Kv4AppendArgs a) {
  constexpr int D = NG * kKv4Group;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const long long q = unit / a.Hkv;
  const int h = (int)(unit % a.Hkv);
  if (q >= (a.T >> 2) + 2ll * a.S) return;
  const int s = kv4_find_seq(a.cu_new, a.S, q, lane);
  const int c0 = __ldg(&a.cu_new[s]), c1 = __ldg(&a.cu_new[s + 1]);
  const int n = c1 - c0, len = __ldg(&a.seq_lens[s]);
  const long long qs = (long long)(c0 >> 2) + 2ll * s;
  if (c0 < 0 || n < 0 || c1 > a.T || len < n || len > a.max_pages * a.page_size || (s == 0 && c0 != 0) ||
      (s == a.S - 1 && c1 != a.T)) {
    latch_status(ATTN_ERR_INVALID_ARG);
    return;
  }
  const int start = len - n;
  const long long quad = (start >> 2) + (q - qs);  // quad of positions
  if (q < qs || 4 * quad >= len) return;
  const int i = lane >> 3, j = lane & 7;
  const int pos = (int)(4 * quad) + i;
  const bool live = pos >= start && pos < len;
  const int page = __ldg(&a.block_table[(size_t)s * a.max_pages + (4 * quad) / a.page_size]);
  const int tok = c0 + (pos - start);
  const size_t head = (size_t)h * D + 8 * j;
  uint4 kx[NG], vx[NG];
#pragma unroll
  for (int y = 0; y < NG; ++y) {
    kx[y] = vx[y] = make_uint4(0, 0, 0, 0);
    if (live) {
      kx[y] = __ldg(reinterpret_cast<const uint4*>(a.k + (size_t)tok * a.k_stride + head + 64 * y));
      vx[y] = __ldg(reinterpret_cast<const uint4*>(a.v + (size_t)tok * a.v_stride + head + 64 * y));
    }
  }
  if (page < 0 || page >= a.num_pages) {
    latch_status(ATTN_ERR_BAD_PAGE);
    return;
  }
  const int blocks = a.page_size / kKv4Tok;
  const int in_page = (int)(4 * quad) % a.page_size;
  uint8_t* rec = a.pool + (((size_t)page * a.Hkv + h) * blocks + in_page / kKv4Tok) * kv4_record_bytes(D);
  const int ta = (in_page >> 2) & 3, b0 = i & 1, b1 = i >> 1;
  const bool pair_live = __shfl_xor_sync(0xffffffffu, live ? 1 : 0, 8) && live;
  uint32_t par = 0;  // the parameter word this lane stores: lanes 0.. of K's groups, lanes 4.. of V's
#pragma unroll
  for (int y = 0; y < NG; ++y) {
    float r[8];
    uint32_t sm = kv4_quantize8(kx[y], r);
    if (j == y) par = sm;
    // even channels into the low half, odd ones into the high half; both sums are below 2^16
    const float ev = r[0] + 16.0f * r[2] + 256.0f * r[4] + 4096.0f * r[6];
    const float od = r[1] + 16.0f * r[3] + 256.0f * r[5] + 4096.0f * r[7];
    const uint32_t kw = (uint32_t)ev | ((uint32_t)od << 16);
    if (live) {
      *reinterpret_cast<uint32_t*>(rec + kv4_k_code_off(y, ta, b0, b1, j)) = kw;
      if (a.k_out != nullptr)
        *reinterpret_cast<uint4*>(a.k_out + (size_t)tok * a.Hkv * D + head + 64 * y) = kv4_values8(r, sm);
    }
    sm = kv4_quantize8(vx[y], r);
    if (j == 4 + y) par = sm;
    const float c03 = r[0] + 16.0f * r[1] + 256.0f * r[2] + 4096.0f * r[3];
    const float c47 = r[4] + 16.0f * r[5] + 256.0f * r[6] + 4096.0f * r[7];
    const uint32_t vw = (uint32_t)c03 | ((uint32_t)c47 << 16);
    // a word holds both tokens of a pair: the even token's lane writes channels 0-3, the odd one's 4-7
    const uint32_t other = __shfl_xor_sync(0xffffffffu, vw, 8);
    uint8_t* unit_v = rec + kv4_v_unit_off<NG>(y, ta, j) + 8 * b1;
    if (pair_live) {
      *reinterpret_cast<uint32_t*>(unit_v + 4 * b0) = b0 == 0 ? __byte_perm(vw, other, 0x5410) : __byte_perm(other, vw, 0x7632);
    } else if (live) {
      *reinterpret_cast<uint16_t*>(unit_v + 2 * b0) = (uint16_t)(vw & 0xffffu);
      *reinterpret_cast<uint16_t*>(unit_v + 4 + 2 * b0) = (uint16_t)(vw >> 16);
    }
    if (live && a.v_out != nullptr)
      *reinterpret_cast<uint4*>(a.v_out + (size_t)tok * a.Hkv * D + head + 64 * y) = kv4_values8(r, sm);
  }
  if (live && (j & 3) < NG)
    *reinterpret_cast<uint32_t*>(rec + kv4_param_off<NG>(j >> 2, ta, b0, b1) + 4 * (j & 3)) = par;
}

struct Kv4GatherArgs {
  const uint8_t* pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  __nv_bfloat16* k;  // [S, Hkv, N, d]
  __nv_bfloat16* v;
  int S, Hkv, N, page_size, num_pages, max_pages;
};

// One warp per (record, sequence): lanes as in the append, four quads of tokens in turn.
template <int NG>
__global__ void __launch_bounds__(256) attn_kv4_gather_kernel(const __grid_constant__ Kv4GatherArgs a) {
  constexpr int D = NG * kKv4Group;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int nrec = (a.N + kKv4Tok - 1) / kKv4Tok;
  const int r0 = (int)(unit % nrec);
  const long long sh = unit / nrec;
  const int h = (int)(sh % a.Hkv);
  const long long sq = sh / a.Hkv;
  if (sq >= a.S) return;
  const int s = (int)sq;
  int len = __ldg(&a.seq_lens[s]);
  if (len < 0 || len > a.max_pages * a.page_size) {
    latch_status(ATTN_ERR_INVALID_ARG);
    return;
  }
  len = min(len, a.N);
  const int p0 = r0 * kKv4Tok;
  if (p0 >= len) return;
  const int page = __ldg(&a.block_table[(size_t)s * a.max_pages + p0 / a.page_size]);
  if (page < 0 || page >= a.num_pages) {
    latch_status(ATTN_ERR_BAD_PAGE);
    return;
  }
  const int blocks = a.page_size / kKv4Tok;
  const uint8_t* rec =
      a.pool + (((size_t)page * a.Hkv + h) * blocks + (p0 % a.page_size) / kKv4Tok) * kv4_record_bytes(D);
  const int i = lane >> 3, j = lane & 7, b0 = i & 1, b1 = i >> 1;
  const size_t row0 = ((size_t)s * a.Hkv + h) * a.N + p0 + i;
#pragma unroll
  for (int ta = 0; ta < 4; ++ta) {
    if (p0 + 4 * ta + i >= len) break;
    const size_t out = (row0 + 4 * ta) * D + 8 * j;
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      const uint32_t ksm = __ldg(reinterpret_cast<const uint32_t*>(rec + kv4_param_off<NG>(0, ta, b0, b1) + 4 * y));
      const uint32_t vsm = __ldg(reinterpret_cast<const uint32_t*>(rec + kv4_param_off<NG>(1, ta, b0, b1) + 4 * y));
      const uint32_t kw = __ldg(reinterpret_cast<const uint32_t*>(rec + kv4_k_code_off(y, ta, b0, b1, j)));
      const uint2 vu = __ldg(reinterpret_cast<const uint2*>(rec + kv4_v_unit_off<NG>(y, ta, j) + 8 * b1));
      const uint32_t vw = __byte_perm(vu.x, vu.y, b0 == 0 ? 0x5410 : 0x7632);  // channels 0-3 | 4-7 << 16
      float r[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        r[2 * c] = (float)((kw >> (4 * c)) & 15u);
        r[2 * c + 1] = (float)((kw >> (16 + 4 * c)) & 15u);
      }
      *reinterpret_cast<uint4*>(a.k + out + 64 * y) = kv4_values8(r, ksm);
#pragma unroll
      for (int c = 0; c < 8; ++c) r[c] = (float)((vw >> (4 * c)) & 15u);
      *reinterpret_cast<uint4*>(a.v + out + 64 * y) = kv4_values8(r, vsm);
    }
  }
}

}  // namespace attn
