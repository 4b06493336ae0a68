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
  int heads;  // KV heads a warp takes in turn
};
constexpr int kKv4AppendThreads = 128;

// a b + c with bf16 a and b (16-bit halves of a word, say) and fp32 c: one FMA, where widening
// a half first would cost an instruction of the half-rate integer pipe.
__device__ __forceinline__ float fma_bf16(uint32_t a, uint32_t b, float c) {
  float d;
  asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"((uint16_t)a), "h"((uint16_t)b), "f"(c));
  return d;
}
constexpr uint32_t kBf16One = 0x3f80u, kBf16Eight = 0x4100u;

__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("min.u16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

// Bits of |x| less one, for both bf16 halves of a word (0 becomes 0xffff).
__device__ __forceinline__ uint32_t magnitude_less_one(uint32_t w) {
  uint32_t c;
  asm("add.u16x2 %0, %1, %2;" : "=r"(c) : "r"(w & 0x7fff7fffu), "r"(0xffffffffu));
  return c;
}

// One lane's 8 channels of a group whose 64 channels lie in 8 neighbouring lanes: the group's
// scale and minimum, and the codes as floats.
//
// c = nearest integer to (x - m) / s, ties to even, of the exact quotient.  Values of few
// significant bits meet a border k + 1/2 between two codes often, so borders have to be exact on
// the fast path: u = x - m, a first quotient u * rcp(s), and one correction by its remainder
// give the quotient within half an ulp (2^-21 up to 16), and exactly where it is representable, as
// a border is.  That suffices while no |x| or |m| but 0 is below 2^-12 s: x and m are then
// multiples of 2^-20 s (8 significant bits), u needs fewer than 24 bits and is exact, and a
// quotient that is no border is at least 2^-20 away from one.  Other groups are redone in 64 bits.
//
// The scale's division by 15 is a product with 1/15 and one correction by its remainder, which
// gives the correctly rounded quotient for every 24-bit significand (checked exhaustively).
// Every lane runs the fast path; `rare` lanes are put right by kv4_quantize_rare, apart, so that the
// fast paths of K and V lie in one basic block.
struct Kv4Group {
  float r[8];      // codes
  uint32_t sm;     // s | m << 16
  float lo, span;  // minimum, fp32 range
  bool rare;
};

__device__ __forceinline__ Kv4Group kv4_quantize8(const uint4& x) {
  Kv4Group g;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
  const __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
  const __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  const __nv_bfloat162 least = __hmin2(__hmin2(__habs2(h[0]), __habs2(h[1])), __hmin2(__habs2(h[2]), __habs2(h[3])));
  // (minimum, -maximum) in one word: a single minimum per shuffle serves both
  const uint32_t mnw = *reinterpret_cast<const uint32_t*>(&mn), mxw = *reinterpret_cast<const uint32_t*>(&mx) ^ 0x80008000u;
  const uint32_t lows = __byte_perm(mnw, mxw, 0x5410), highs = __byte_perm(mnw, mxw, 0x7632);
  __nv_bfloat162 e = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&lows),
                                 *reinterpret_cast<const __nv_bfloat162*>(&highs));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    uint32_t u = *reinterpret_cast<uint32_t*>(&e);
    u = __shfl_xor_sync(0xffffffffu, u, o);
    e = __hmin2_nan(e, *reinterpret_cast<__nv_bfloat162*>(&u));
  }
  const uint32_t ew = *reinterpret_cast<const uint32_t*>(&e);
  g.lo = fma_bf16(ew, kBf16One, 0.0f);  // a zero minimum is stored as +0
  g.span = -fma_bf16(ew >> 16, kBf16One, g.lo) + 0.0f;
  float q15 = g.span * (1.0f / 15.0f);
  q15 = fmaf(fmaf(-15.0f, q15, g.span), 1.0f / 15.0f, q15);
  const uint32_t sb = __bfloat16_as_ushort(__float2bfloat16_rn(q15));
  const float s = __uint_as_float(sb << 16);
  g.sm = sb | (__float_as_uint(g.lo) & 0xffff0000u);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to the nearest integer, ties to even
    const float u0 = fma_bf16(w[i], kBf16One, -g.lo), u1 = fma_bf16(w[i] >> 16, kBf16One, -g.lo);
    float q0 = u0, q1 = u1, e0, e1;
    mul2(q0, q1, inv, inv);
    fma2(e0, e1, q0, q1, -s, -s, u0, u1);
    fma2(q0, q1, e0, e1, inv, inv, q0, q1);
    add2(q0, q1, kRound, kRound);
    add2(q0, q1, -kRound, -kRound);
    g.r[2 * i] = q0;
    g.r[2 * i + 1] = q1;
  }
  // 2^-100 <= span: neither q15's remainder nor rcp(s) leaves the normal numbers.  The least magnitude,
  // zeros included, settles the precondition above nearly always.
  const float tiny = s * 0.000244140625f;  // 2^-12 s
  g.rare = !(g.span >= 7.888609e-31f && g.span <= 3.4028234663852886e38f &&
             fminf(__low2float(least), __high2float(least)) >= tiny && fabsf(g.lo) >= tiny);
  return g;
}

// The groups the fast path does not settle: non-finite, constant or tiny ranges, zeros and values
// below 2^-12 s.
__device__ __forceinline__ void kv4_quantize_rare(const uint4& x, Kv4Group& g) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if (!(g.span <= 3.4028234663852886e38f)) {  // infinite or NaN values, or a range past fp32: the group is NaN
    g.sm = 0x7fc07fc0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) g.r[i] = 0.0f;
    return;
  }
  if (g.span == 0.0f) {  // a constant group, or a token that is not there
#pragma unroll
    for (int i = 0; i < 8; ++i) g.r[i] = 0.0f;
    return;
  }
  if (g.span < 7.888609e-31f)
    g.sm = (g.sm & 0xffff0000u) | __bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(g.span, 15.0f)));
  const float s = bf16lo_to_f32(g.sm);
  // magnitudes order like their bits; less one, a zero becomes the largest
  const uint32_t least = min_u16x2(min_u16x2(magnitude_less_one(w[0]), magnitude_less_one(w[1])),
                                   min_u16x2(magnitude_less_one(w[2]), magnitude_less_one(w[3])));
  const uint32_t tiny = __float_as_uint(s * 0.000244140625f) >> 16;
  if (g.span >= 7.888609e-31f && min(least & 0xffffu, least >> 16) >= tiny &&
      ((__float_as_uint(g.lo) >> 16) & 0x7fffu) - 1u >= tiny)
    return;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const uint32_t wi = i == 0 ? w[0] : (i == 1 ? w[1] : (i == 2 ? w[2] : w[3]));
    float c[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float xi = k == 0 ? bf16lo_to_f32(wi) : bf16hi_to_f32(wi);
      const double q = ((double)xi - (double)g.lo) / (double)s;
      c[k] = q >= 0.0 ? (float)fmin(rint(q), 15.0) : 0.0f;  // 0 / 0 (the scale underflowed): code 0
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
      if (n == i) {
        g.r[2 * n] = c[0];
        g.r[2 * n + 1] = c[1];
      }
  }
}

// Values s c + m of 8 codes, rounded to bf16.
__device__ __forceinline__ uint4 kv4_values8(const float (&r)[8], uint32_t sm) {
  const float s = bf16lo_to_f32(sm), m = bf16hi_to_f32(sm);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) fma2(v[2 * i], v[2 * i + 1], r[2 * i], r[2 * i + 1], s, s, m, m);
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// The same from a word of codes: pairs (nibble i of the low half, nibble i of the high half), i =
// 0..3, as bf16 integers.  A code masked into the mantissa of 128 is 128 + c; the subtraction is exact.
__device__ __forceinline__ void kv4_code_values(uint32_t w, uint32_t sm, float (&lo)[4], float (&hi)[4]) {
  const float m = bf16hi_to_f32(sm);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t c = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(c) : "r"(c), "r"(0x3f803f80u), "r"(0xc300c300u));
    lo[i] = fma_bf16(sm, c, m);
    hi[i] = fma_bf16(sm, c >> 16, m);
  }
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

// One warp per aligned quad of positions and `heads` KV heads: lane = 8 (token of the quad) +
// (8-channel chunk).  The reads are bf16 rows of 128 bytes a group; the quad's K codes and V codes
// are one 128-byte line a group each.  A call is bound by HBM (2 d bytes read and 9 d / 16
// written per token, head and tensor, and 2 d more where the values are written back) once every SM
// has enough loads in flight: a warp therefore takes several heads where there are warps to spare, since
// its chain of dependent loads (sequence, position, page) then serves all of them (108K tokens, 8
// heads, d = 128: 359 us with one head a warp, 272 with 2, 229 with 4, 216 with 8; a decode step of 64
// tokens 6.2 us with one and 14.4 with 8), and fetches the next head's rows while it works on one
// (without: 254).  Small blocks and a few spilled words leave room for 20 warps an SM instead of
// 16: 199 us, 5.6 TB/s (24 warps with 108 bytes spilled: 245); d = 256: 413 us instead of 505.  (Replayed
// graphs; called one after another the prompts take 212 us, the step 11.)
template <int NG>
__global__ void __launch_bounds__(kKv4AppendThreads, NG == 1 ? 6 : (NG == 2 ? 5 : 3))
    attn_kv4_append_kernel(const __grid_constant__ Kv4AppendArgs a) {
  constexpr int D = NG * kKv4Group;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int parts = (a.Hkv + a.heads - 1) / a.heads;
  const long long q = unit / parts;
  const int h0 = (int)(unit % parts) * a.heads, h1 = min(a.Hkv, h0 + a.heads);
  if (q >= (a.T >> 2) + 2ll * a.S) return;
  const int s = kv4_find_seq(a.cu_new, a.S, q, lane);
  const int c0 = __ldg(&a.cu_new[s]), c1 = __ldg(&a.cu_new[s + 1]);
  const int n = c1 - c0, len = __ldg(&a.seq_lens[s]);
  const long long qs = (long long)(c0 >> 2) + 2ll * s;
  if (c0 < 0 || n < 0 || c1 > a.T || len < n || len > a.max_pages * a.page_size || (s == 0 && c0 != 0)) {
    latch_status(ATTN_ERR_INVALID_ARG);
    return;
  }
  const int start = len - n;
  const long long quad = (start >> 2) + (q - qs);  // quad of positions
  if (n == 0 || q < qs || 4 * quad >= len) return;
  const int i = lane >> 3, j = lane & 7;
  const int pos = (int)(4 * quad) + i;
  const bool live = pos >= start && pos < len;
  const int page = __ldg(&a.block_table[(size_t)s * a.max_pages + (4 * quad) / a.page_size]);
  const int tok = c0 + (pos - start);
  const __nv_bfloat16* kp = a.k + (size_t)tok * a.k_stride + 8 * j;
  const __nv_bfloat16* vp = a.v + (size_t)tok * a.v_stride + 8 * j;
  uint4 kn[NG], vn[NG];
  auto fetch = [&](int h) {
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      kn[y] = vn[y] = make_uint4(0, 0, 0, 0);
      if (live) {
        kn[y] = __ldg(reinterpret_cast<const uint4*>(kp + (size_t)h * D + 64 * y));
        vn[y] = __ldg(reinterpret_cast<const uint4*>(vp + (size_t)h * D + 64 * y));
      }
    }
  };
  fetch(h0);
  if (page < 0 || page >= a.num_pages) {
    latch_status(ATTN_ERR_BAD_PAGE);
    return;
  }
  const int blocks = a.page_size / kKv4Tok;
  const int in_page = (int)(4 * quad) % a.page_size;
  uint8_t* rec = a.pool + (((size_t)page * a.Hkv + h0) * blocks + in_page / kKv4Tok) * kv4_record_bytes(D);
  const int ta = (in_page >> 2) & 3, b0 = i & 1, b1 = i >> 1;
  const bool pair_live = __shfl_xor_sync(0xffffffffu, live ? 1 : 0, 8) && live;
  size_t out = ((size_t)tok * a.Hkv + h0) * D + 8 * j;
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    uint4 kx[NG], vx[NG];
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      kx[y] = kn[y];
      vx[y] = vn[y];
    }
    if (h + 1 < h1) fetch(h + 1);
    uint32_t par = 0;  // the parameter word this lane stores: lanes 0.. of K's groups, lanes 4.. of V's
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      Kv4Group gk = kv4_quantize8(kx[y]), gv = kv4_quantize8(vx[y]);
      if (gk.rare) kv4_quantize_rare(kx[y], gk);
      if (gv.rare) kv4_quantize_rare(vx[y], gv);
      if (j == y) par = gk.sm;
      if (j == 4 + y) par = gv.sm;
      // even channels into the low half, odd ones into the high half; both sums are below 2^16,
      // and adding 2^23 leaves them in the low bits
      float ev = gk.r[6], od = gk.r[7];
      fma2(ev, od, ev, od, 16.0f, 16.0f, gk.r[4], gk.r[5]);
      fma2(ev, od, ev, od, 16.0f, 16.0f, gk.r[2], gk.r[3]);
      fma2(ev, od, ev, od, 16.0f, 16.0f, gk.r[0], gk.r[1]);
      add2(ev, od, 8388608.0f, 8388608.0f);
      const uint32_t kw = __byte_perm(__float_as_uint(ev), __float_as_uint(od), 0x5410);
      // channels (0, 1) + 256 (2, 3) and (4, 5) + 256 (6, 7)
      float p0 = gv.r[2], p1 = gv.r[3], p4 = gv.r[6], p5 = gv.r[7];
      fma2(p0, p1, p0, p1, 256.0f, 256.0f, gv.r[0], gv.r[1]);
      fma2(p4, p5, p4, p5, 256.0f, 256.0f, gv.r[4], gv.r[5]);
      const uint32_t vw = __byte_perm(__float_as_uint(fmaf(p1, 16.0f, p0) + 8388608.0f),
                                      __float_as_uint(fmaf(p5, 16.0f, p4) + 8388608.0f), 0x5410);
      // a word holds both tokens of a pair: the even token's lane writes channels 0-3, the odd one's 4-7
      const uint32_t other = __shfl_xor_sync(0xffffffffu, vw, 8);
      uint8_t* unit_v = rec + kv4_v_unit_off<NG>(y, ta, j) + 8 * b1;
      if (pair_live) {
        *reinterpret_cast<uint32_t*>(unit_v + 4 * b0) =
            b0 == 0 ? __byte_perm(vw, other, 0x5410) : __byte_perm(other, vw, 0x7632);
      } else if (live) {
        *reinterpret_cast<uint16_t*>(unit_v + 2 * b0) = (uint16_t)(vw & 0xffffu);
        *reinterpret_cast<uint16_t*>(unit_v + 4 + 2 * b0) = (uint16_t)(vw >> 16);
      }
      if (live) {
        *reinterpret_cast<uint32_t*>(rec + kv4_k_code_off(y, ta, b0, b1, j)) = kw;
        if (a.k_out != nullptr) *reinterpret_cast<uint4*>(a.k_out + out + 64 * y) = kv4_values8(gk.r, gk.sm);
        if (a.v_out != nullptr) *reinterpret_cast<uint4*>(a.v_out + out + 64 * y) = kv4_values8(gv.r, gv.sm);
      }
    }
    if (live && (j & 3) < NG)
      *reinterpret_cast<uint32_t*>(rec + kv4_param_off<NG>(j >> 2, ta, b0, b1) + 4 * (j & 3)) = par;
    rec += (size_t)blocks * kv4_record_bytes(D);
    out += D;
  }
}

struct Kv4GatherArgs {
  const uint8_t* pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  __nv_bfloat16* k;  // [S, Hkv, N, d]
  __nv_bfloat16* v;
  int S, Hkv, N, page_size, num_pages, max_pages;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Copies a record into shared memory with the lanes of a warp, 16 bytes each.
template <int REC>
__device__ __forceinline__ void kv4_fetch_record(uint32_t dst, const uint8_t* src, int lane) {
#pragma unroll
  for (int i = 0; i < REC / 512; ++i) cp_async16(dst + i * 512 + lane * 16, src + i * 512 + lane * 16);
  if constexpr (REC % 512 != 0) {
    constexpr int kAt = REC / 512 * 512;
    if (lane < (REC % 512) / 16) cp_async16(dst + kAt + lane * 16, src + kAt + lane * 16);
  }
}

constexpr int kKv4GatherWarps = 8;

// One warp per record: 16 positions of a sequence and a KV head.  The work is a copy (9 d / 8 bytes in
// and 4 d out per token and head), so what counts is loads in flight: a record comes in whole by
// 16-byte asynchronous copies, and the lanes take their codes from shared memory (lane = 8 (token of a
// quad) + (8-channel chunk), as in the append).  8 contexts of 15 to 16.4 thousand tokens, 8 heads, d =
// 128: 112 us, 5.9 TB/s; with all heads in turn in one warp, the next record on its way, 117 us.
template <int NG>
__global__ void __launch_bounds__(kKv4GatherWarps * 32)
    attn_kv4_gather_kernel(const __grid_constant__ Kv4GatherArgs a) {
  constexpr int D = NG * kKv4Group, REC = kv4_record_bytes(D);
  __shared__ __align__(128) uint8_t stage[kKv4GatherWarps][REC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = (long long)blockIdx.x * kKv4GatherWarps + warp;
  const int nrec = (a.N + kKv4Tok - 1) / kKv4Tok;
  const int h = (int)(unit % a.Hkv);
  const long long sr = unit / a.Hkv;
  const int r0 = (int)(sr % nrec);
  const long long sq = sr / nrec;
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
  const size_t at = ((size_t)page * a.Hkv + h) * (a.page_size / kKv4Tok) + (p0 % a.page_size) / kKv4Tok;
  const uint8_t* st = stage[warp];
  kv4_fetch_record<REC>(smem_u32(st), a.pool + at * REC, lane);
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
  const int i = lane >> 3, j = lane & 7, b0 = i & 1, b1 = i >> 1;
  const size_t row0 = ((size_t)s * a.Hkv + h) * a.N + p0 + i;
#pragma unroll
  for (int ta = 0; ta < 4; ++ta) {
    if (p0 + 4 * ta + i >= len) break;
    const size_t out = (row0 + 4 * ta) * D + 8 * j;
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      const uint32_t ksm = *reinterpret_cast<const uint32_t*>(st + kv4_param_off<NG>(0, ta, b0, b1) + 4 * y);
      const uint32_t vsm = *reinterpret_cast<const uint32_t*>(st + kv4_param_off<NG>(1, ta, b0, b1) + 4 * y);
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(st + kv4_k_code_off(y, ta, b0, b1, j));
      const uint2 vu = *reinterpret_cast<const uint2*>(st + kv4_v_unit_off<NG>(y, ta, j) + 8 * b1);
      float lo[4], hi[4];
      kv4_code_values(kw, ksm, lo, hi);  // channels 2i and 2i + 1
      __stcs(reinterpret_cast<uint4*>(a.k + out + 64 * y),
             make_uint4(pack_bf16x2(lo[0], hi[0]), pack_bf16x2(lo[1], hi[1]), pack_bf16x2(lo[2], hi[2]),
                        pack_bf16x2(lo[3], hi[3])));
      // this token's halves of the two words: channels i and 4 + i
      kv4_code_values(__byte_perm(vu.x, vu.y, b0 == 0 ? 0x5410 : 0x7632), vsm, lo, hi);
      __stcs(reinterpret_cast<uint4*>(a.v + out + 64 * y),
             make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]),
                        pack_bf16x2(hi[2], hi[3])));
    }
  }
}

}  // namespace attn
