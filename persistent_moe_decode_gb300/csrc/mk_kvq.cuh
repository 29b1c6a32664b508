// The 4-bit key/value cache: record layout, quantiser and the attention of one
// page, shared by the cache operators (mk_kvq.cu) and whatever else reads a
// page of it.
//
// A page of 16 tokens holds one record of 18 D bytes per KV head (D = 64 or
// 128, NG = D / 64 groups of 64 dims): key codes (8 D bytes), value codes
// (8 D), key scales (D), value scales (D).  A group is step * code + low.
//
// The orders inside a record are the tensor cores' own, so that a lane reads
// its fragments with one wide load and no shuffle:
//   keys    token t, column c (0..3): 8 NG bytes = dims 64 g + 16 c .. + 15 of
//           every group g, dim n at nibble n.  Lane (row, c) of the A operand
//           K[token][dim] takes one column; a 32-bit word masked to its nibbles
//           0 and 4 (1 and 5, ...) is a pair of adjacent k elements.
//   values  token pair t / 2, column c (0..7): 8 NG bytes = dims 64 g + 8 c ..
//           + 7 of both tokens; 16-bit unit t % 2 of word u holds dims
//           4 u .. 4 u + 3 of token t.  Masking a word gives one dim of two
//           consecutive tokens: a k pair of the A operand V^T[dim][token].
//   scales  token t, group g: (step, low) as two BF16 numbers in one word.
// A nibble masked in place is an FP16 subnormal, code * 2^-24 (or, four bits
// up, 16 code * 2^-24), an exact operand after half an instruction; with one
// more it is the FP16 integer code - 8 (16 (code - 8)).  No code is rounded.
#pragma once
#include <stdint.h>
#include <float.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mk_ptx.cuh"

namespace mk {

constexpr int kKvqPage = 16;    // tokens of a page
constexpr int kKvqGroup = 64;   // dims that share a scale

template <int D>
struct KvqRec {
  static constexpr int NG = D / kKvqGroup;
  static constexpr int kBytes = 18 * D;
  static constexpr int kVal = 8 * D, kKeyScale = 16 * D, kValScale = 17 * D;
  static __device__ __forceinline__ int key_word(int t, int wi, int g) {   // dims 64 g + 8 wi .. + 7
    return t * (D / 2) + (wi >> 1) * (8 * NG) + g * 8 + (wi & 1) * 4;
  }
  static __device__ __forceinline__ int val_half(int t, int wi, int g, int u) {   // dims 64 g + 8 wi + 4 u .. + 3
    return kVal + (t >> 1) * D + wi * (8 * NG) + g * 8 + u * 4 + (t & 1) * 2;
  }
};

// ---------------------------------------------------------------- quantiser

__device__ __forceinline__ float fmin_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct KvqScale {
  float low, step, inv;   // inv = 1 / step to 2^-23, 0 with step 0
  __device__ __forceinline__ uint32_t word() const {
    return (__float_as_uint(step) >> 16) | (__float_as_uint(low) & 0xffff0000u);
  }
};

// (step, low) of a group with minimum lo and maximum hi (NaN where the group
// holds one): low = the largest BF16 number <= lo, step = the smallest BF16
// number >= (hi - low) / 15, at least 2^-126, or 0 for a constant group.  The
// product with 1 / 15, cut to BF16, is that number or one of the two below it;
// 15 times a BF16 number is exact in fp32, so two comparisons settle it (a
// division took three times as long).  A span that is not finite makes the
// whole group NaN.  BF: lo is a BF16 number.
template <bool BF = false>
__device__ __forceinline__ KvqScale kvq_scale(float lo, float hi) {
  KvqScale s;
  uint32_t cut = __float_as_uint(lo);
  if constexpr (!BF) {
    cut &= 0xffff0000u;
    if (cut != __float_as_uint(lo) && lo < 0.f) cut += 0x10000u;
  }
  s.low = __uint_as_float(cut) + 0.f;      // -0 becomes +0
  const float span = hi - s.low;
  cut = __float_as_uint(span * (1.f / 15.f)) & 0xffff0000u;
  if (__uint_as_float(cut) * 15.f < span) cut += 0x10000u;
  if (__uint_as_float(cut) * 15.f < span) cut += 0x10000u;
  s.step = fmaxf(__uint_as_float(cut), 1.17549435e-38f);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.inv) : "f"(s.step));
  const bool bad = !(span <= FLT_MAX);     // NaN included; span >= 0
  if (span == 0.f || bad) s.step = s.inv = 0.f;
  if (bad) s.low = __uint_as_float(0x7fc00000u);
  return s;
}

// Codes of eight values, nibble i of the word that of x[i]: (x - low) / step to
// the nearest integer, ties to even, the difference rounded to fp32.  Adding
// 1.5 2^23 downwards leaves c, the floor of diff * inv, in the low mantissa
// bits.  The product is within 5e-6 of the quotient, so r = diff - c step is
// between 0 and step but for that error, and one FMA gives it exactly: c step
// has at most 12 bits, and r is a multiple of diff's last bit no larger than
// diff.  The code is c, or c + 1 where r is above half a step, or at it with an
// odd c.  With H = 2 / 2^exponent(step), v = (r - step / 2) H + 1/2 held to
// 0..1 is above, at or below 1/2 as r is above, at or below half a step (the
// least difference is 2^-24, which v shows), so adding v to 1.5 2^23 + c
// rounds to the code, ties included.  All this is arithmetic of the FMA pipe,
// two values an instruction where it can be; with comparisons and selections
// the integer pipe bound a 256K prefix at 157 us.  Eight patterns, shifted and
// added, leave the codes and one constant.
__device__ __forceinline__ uint32_t kvq_codes(const float* x, const KvqScale& s) {
  constexpr float kMagic = 12582912.f;     // 0x4b400000
  const float h = __uint_as_float(0x7f800000u - (__float_as_uint(s.step) & 0x7f800000u));
  const float b = fmaf(-0.5f * h, s.step, 0.5f);
  const float2 low = make_float2(-s.low, -s.low), inv = make_float2(s.inv, s.inv);
  const float2 magic = make_float2(kMagic, kMagic), neg_step = make_float2(-s.step, -s.step);
  uint32_t word = 0;
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    const float2 diff = __fadd2_rn(make_float2(x[i], x[i + 1]), low);
    const float2 t = __ffma2_rd(diff, inv, magic);
    const float2 c = __fadd2_rn(t, make_float2(-kMagic, -kMagic));
    const float2 r = __ffma2_rn(c, neg_step, diff);
    const float2 code = __fadd2_rn(t, make_float2(__saturatef(fmaf(r.x, h, b)), __saturatef(fmaf(r.y, h, b))));
    word = word * 16u + __float_as_uint(code.y);
    word = word * 16u + __float_as_uint(code.x);
  }
  return s.inv == 0.f ? 0u : word - 0x4b400000u * 0x11111111u;
}

// scale of a group whose values lie eight a thread in eight neighbouring
// threads, all of which (`mask`) call it; of BF16 pairs, minimum and negated
// maximum travel in one register
__device__ __forceinline__ KvqScale kvq_group_scale(const uint32_t (&w)[4], unsigned mask) {
  using B2 = __nv_bfloat162;
  const B2* v = reinterpret_cast<const B2*>(w);
  const B2 mn = __hmin2_nan(__hmin2_nan(v[0], v[1]), __hmin2_nan(v[2], v[3]));
  const B2 mx = __hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3]));
  B2 m = __halves2bfloat162(__hmin_nan(mn.x, mn.y), __hneg(__hmax_nan(mx.x, mx.y)));
#pragma unroll
  for (int sh = 1; sh < 8; sh <<= 1) {
    const uint32_t o = __shfl_xor_sync(mask, *reinterpret_cast<const uint32_t*>(&m), sh);
    m = __hmin2_nan(m, *reinterpret_cast<const B2*>(&o));
  }
  return kvq_scale<true>(__low2float(m), -__high2float(m));
}

// the same of fp32 values
__device__ __forceinline__ KvqScale kvq_group_scale(const float* x, unsigned mask) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; i++) {
    lo = fmin_nan(lo, x[i]);
    hi = fmax_nan(hi, x[i]);
  }
#pragma unroll
  for (int sh = 1; sh < 8; sh <<= 1) {
    lo = fmin_nan(lo, __shfl_xor_sync(mask, lo, sh));
    hi = fmax_nan(hi, __shfl_xor_sync(mask, hi, sh));
  }
  return kvq_scale(lo, hi);
}

// codes of dims 64 g + 8 wi .. + 7 of token t and, from one thread of the
// group, its scale into a record
template <int D>
__device__ __forceinline__ void kvq_store_row(uint8_t* rec, int t, int wi, int g, int val, uint32_t word,
                                              const KvqScale& s) {
  using R = KvqRec<D>;
  if (val) {
    *(uint16_t*)(rec + R::val_half(t, wi, g, 0)) = (uint16_t)word;
    *(uint16_t*)(rec + R::val_half(t, wi, g, 1)) = (uint16_t)(word >> 16);
  } else {
    *(uint32_t*)(rec + R::key_word(t, wi, g)) = word;
  }
  if (wi == 0) *(uint32_t*)(rec + (val ? R::kValScale : R::kKeyScale) + 4 * (t * R::NG + g)) = s.word();
}

// ---------------------------------------------------------------- attention

// D = A B, m16n8k16, FP16 in, fp32 out
__device__ __forceinline__ void mma_f16_first(float* d, const uint32_t* a, const uint32_t* b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}

// D += A B
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, const uint32_t* b) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// a + b, two FP16 numbers each, subnormals kept
__device__ __forceinline__ uint32_t add_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// One warp's share of the attention of up to 8 query heads to one KV head,
// page by page.
//   x_t  = scale sum_i q_i k_ti = f sum_g step_tg (sum_{i in g} q'_i code_ti)
//          + sum_g low_tg sq_g,   sq_g = scale sum_{i in g} q_i
//   out  = sum_t p_t v_t / sum_t p_t,  p_t = 2^x_t (x in units of log2)
//   sum_t p_t v_ti = sum_t (p_t step_tg) (code_ti - 8) + sum_t p_t mid_tg,
//          mid_tg = low_tg + 8 step_tg: the two parts have the size of the
//          values.  (With codes 0 .. 15 and low they are the size of the
//          group's range and cancel in a mean over many tokens: 8 % off at
//          256K tokens, measured.)
// S^T = K Q^T takes the page's 16 tokens as M and the heads as N, O^T = V^T
// W^T the dims as M, 16 dims a tile, so no row of M is padding.  The weight of
// a value code is w_tg = p_t step_tg sc_g with p_t = 2^(x_t - r).  The reference
// r and each group's power of two sc_g move only when a p or w passes 2^15
// (one vote a page), and then so that the largest seen is 2^8: FP16 holds 11
// bits of every weight down to 2^-22 of the largest, for all sizes of scores and
// steps that the fp32 numbers beside it hold.  p step and the sums of p mid are
// formed before the division by sum p, with p up to 2^15 in each of fewer than
// 2^31 tokens: values below 2^80 cannot overflow them.  Nor can keys below that,
// whose sum of products reaches 2^23 steps, or queries, whose factor f is up to
// 2^11 times scale |q|; scores themselves stay below 2^100.
// QT = 2 / PT = 2 split q and w into FP16 high and low halves (22 bits) for
// fp32 activations, with the key codes centred too.  With one half each w is
// rounded to 11 bits, an eighth of a BF16 result's own rounding, and BF16 q is
// exact.  The key codes are then subnormals: a product stands at up to 2^0 when it
// is aligned, and what lies below 2^-24 is cut off each of 17 addends in 4
// products a group, 2^-17.9 in all of sums that f = 2^11 scale |q| multiplies: a
// score is off by less than 2^-6 scale max |q| step a group, against half of scale
// |q_i| step in every dim that the codes' own rounding costs (centring them too
// takes 32 instructions more a page and head).  And o takes every page in the
// product itself, which cuts off where fp32 calls add with a rounding.
template <int D, int QT, int PT>
struct KvqAttn {
  using R = KvqRec<D>;
  static constexpr int NG = R::NG;
  static constexpr int NW = 2 * NG;        // code words of a lane per token / token pair
  static constexpr int NT = 2 * NW;        // k-steps of S = 16-dim tiles of O

  uint32_t q[QT][NT][2];
  float f[2], sq[NG][2];                   // heads 2 cq, 2 cq + 1
  float r[2], l[2], sc[NG][2], om[NG][2];
  float o[NT][4];

  // log2 of the largest weight after the references move, the limit before; sc's own limit and its exponent field
  static constexpr float kHead = 8.f, kTop = 32768.f, kScMax = 0x1p120f;
  static constexpr int kScMaxExp = 247;

  template <int N>
  static __device__ __forceinline__ void load_words(uint32_t* dst, const uint8_t* p) {
    if constexpr (N == 4) {
      const uint4 t = *(const uint4*)p;
      dst[0] = t.x, dst[1] = t.y, dst[2] = t.z, dst[3] = t.w;
    } else if constexpr (N == 2) {
      const uint2 t = *(const uint2*)p;
      dst[0] = t.x, dst[1] = t.y;
    } else {
      dst[0] = *(const uint32_t*)p;
    }
  }

  // Place of the record's 16-byte chunk c in a copy of it in shared memory: the
  // value chunks of four token pairs side by side, so that the eight lanes of
  // one 128-byte read (two columns, four pairs) take eight neighbouring chunks
  // and not eight that share their banks.
  static __device__ __forceinline__ int staged(int c) {
    constexpr int V0 = R::kVal / 16, V1 = R::kKeyScale / 16, W = D / 16;   // value chunks, chunks of a pair
    if (c < V0 || c >= V1) return c;
    const int v = c - V0, pair = v / W, col = v % W;
    return V0 + (pair / 4) * (4 * W) + col * 4 + pair % 4;
  }

  // keys of tokens gl, gl + 8 and their scales
  struct Keys {
    uint32_t w[2][NW], sc[2][NG];
  };
  static __device__ __forceinline__ void load_keys(Keys& k, const uint8_t* rec, int lane) {
#pragma unroll
    for (int e = 0; e < 2; e++) {
      load_words<NW>(k.w[e], rec + ((lane >> 2) + 8 * e) * (D / 2) + (lane & 3) * (8 * NG));
      load_words<NG>(k.sc[e], rec + R::kKeyScale + ((lane >> 2) + 8 * e) * (4 * NG));
    }
  }
  // values of token pairs cq, cq + 4; STAGED: of a copy in the order of staged()
  template <bool STAGED>
  static __device__ __forceinline__ void load_values(uint32_t (*v)[NW], const uint8_t* rec, int lane) {
    const int gl = lane >> 2, cq = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; e++)
      load_words<NW>(v[e], rec + R::kVal + e * 4 * D +
                               (STAGED ? (gl * NG / 2 * 4 + cq) * 16 + gl * NG % 2 * 8 : cq * D + gl * (8 * NG)));
  }

  // x[g][16]: dims 64 g + 16 cq .. + 15 of query head gl (zeros where there is
  // no such head); scale_log2 = softmax scale times log2 e
  __device__ __forceinline__ void init(const float (*x)[16], float scale_log2, int lane) {
    const int cq = lane & 3;
    float top = 0.f, sum[NG];
#pragma unroll
    for (int g = 0; g < NG; g++) {
      sum[g] = 0.f;
#pragma unroll
      for (int i = 0; i < 16; i++) {
        top = fmaxf(top, fabsf(x[g][i]));
        sum[g] += x[g][i];
      }
    }
#pragma unroll
    for (int sh = 1; sh < 4; sh <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
#pragma unroll
      for (int g = 0; g < NG; g++) sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], sh);
    }
    // a power of two takes the head's largest |q| to [2^13, 2^14), its 16th part
    // (below) to [2^9, 2^10): FP16, whose last bit is at 2^-24, then holds the 8
    // bits of every BF16 q exactly down to 2^-26 of it (2^-17 of 2^9)
    const int e = top == 0.f ? 0 : min(126, 13 + 127 - (int)(__float_as_uint(top) >> 23));
    const float up = __uint_as_float((uint32_t)(e + 127) << 23);
    const float fh = scale_log2 * (QT == 2 ? 1.f : 16777216.f) * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int g = 0; g < NG; g++)
#pragma unroll
      for (int s = 0; s < 4; s++)          // word s / 2, nibbles 2 (s & 1) and + 1
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
          const int i = (s >> 1) * 8 + (s & 1) * 2 + hf;
          const float w = hf ? up * 0.0625f : up;   // the nibble four bits up counts 16 times
          const float a = x[g][i] * w, b = x[g][i + 4] * w;
          const uint32_t hi = pack_h2(a, b);
          q[0][g * 4 + s][hf] = hi;
          if constexpr (QT == 2) {
            const float2 hv = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            q[1][g * 4 + s][hf] = pack_h2(a - hv.x, b - hv.y);
          }
        }
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int src = (2 * cq + h) * 4;
      f[h] = __shfl_sync(0xffffffffu, fh, src);
#pragma unroll
      for (int g = 0; g < NG; g++) {
        sq[g][h] = __shfl_sync(0xffffffffu, sum[g] * scale_log2, src);
        sc[g][h] = kScMax;
        om[g][h] = 0.f;
      }
      r[h] = -FLT_MAX;
      l[h] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < NT; t++) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
  }

  // codes less 8 as FP16 integers (16 times that four bits up), from 1024 + n
  // less 1032 (1152).  Integers and not subnormals: the tensor cores align
  // their sums to the exponent a subnormal stands for, 2^-14, and would drop
  // up to 10 bits of them.
  static __device__ __forceinline__ uint32_t centred(uint32_t w) {
    return add_h2((w & 0x000f000fu) | 0x64006400u, 0xe408e408u);
  }
  static __device__ __forceinline__ uint32_t centred16(uint32_t w) {
    return add_h2((w & 0x00f000f0u) | 0x64006400u, 0xe480e480u);
  }

  // o += tile times weights.  The tensor cores cut their fp32 sums off rather
  // than round them; for fp32 results a page's products are summed from zero
  // (low halves first) and added with a rounding add
  static __device__ __forceinline__ void add_tile(float* o, const uint32_t* c, const uint32_t (*b)[2]) {
    if constexpr (PT == 1) {
      mma_f16(o, c, b[0]);
    } else {
      float t[4];
      mma_f16_first(t, c, b[1]);
      mma_f16(t, c, b[0]);
#pragma unroll
      for (int e = 0; e < 4; e++) o[e] += t[e];
    }
  }

  // scores (in units of log2) of tokens gl, gl + 8 of a page for heads 2 cq,
  // 2 cq + 1
  __device__ __forceinline__ void scores(float (*x)[2], const uint8_t* rec, int lane) {
    constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u;
    Keys ky;
    load_keys(ky, rec, lane);
    float acc[NG][4];
#pragma unroll
    for (int g = 0; g < NG; g++) {
      [[maybe_unused]] float low[4];
#pragma unroll
      for (int w = 0; w < 2; w++) {
        const int j = 2 * g + w;
        const uint32_t a = ky.w[0][j], b = ky.w[1][j], a8 = a >> 8, b8 = b >> 8;
        if constexpr (QT == 2) {
          const uint32_t c0[4] = {centred(a), centred(b), centred16(a), centred16(b)};
          const uint32_t c1[4] = {centred(a8), centred(b8), centred16(a8), centred16(b8)};
          w == 0 ? mma_f16_first(low, c0, q[1][2 * j]) : mma_f16(low, c0, q[1][2 * j]);
          mma_f16(low, c1, q[1][2 * j + 1]);
          w == 0 ? mma_f16_first(acc[g], c0, q[0][2 * j]) : mma_f16(acc[g], c0, q[0][2 * j]);
          mma_f16(acc[g], c1, q[0][2 * j + 1]);
        } else {
          const uint32_t c0[4] = {a & M0, b & M0, a & M1, b & M1};
          const uint32_t c1[4] = {a8 & M0, b8 & M0, a8 & M1, b8 & M1};
          w == 0 ? mma_f16_first(acc[g], c0, q[0][2 * j]) : mma_f16(acc[g], c0, q[0][2 * j]);
          mma_f16(acc[g], c1, q[0][2 * j + 1]);
        }
      }
      if constexpr (QT == 2)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[g][e] += low[e];
    }
#pragma unroll
    for (int e = 0; e < 2; e++) {
      float2 dot, off;                     // both heads
#pragma unroll
      for (int g = 0; g < NG; g++) {
        const float st = bf16lo(ky.sc[e][g]);
        const float ba = QT == 2 ? fmaf(8.f, st, bf16hi(ky.sc[e][g])) : bf16hi(ky.sc[e][g]);
        const float2 step = make_float2(st, st), base = make_float2(ba, ba);
        const float2 s2 = make_float2(acc[g][2 * e], acc[g][2 * e + 1]), q2 = make_float2(sq[g][0], sq[g][1]);
        dot = g == 0 ? __fmul2_rn(step, s2) : __ffma2_rn(step, s2, dot);
        off = g == 0 ? __fmul2_rn(base, q2) : __ffma2_rn(base, q2, off);
      }
      const float2 v = __ffma2_rn(dot, make_float2(f[0], f[1]), off);
      x[e][0] = v.x;
      x[e][1] = v.y;
    }
  }

  // Tokens [0, valid[n]) of N pages (MASK; else all 16 of each); valid is the
  // same in every lane and may be 0 or less (a page that is not there; its
  // record is read but not used).  N = 2 gives the scheduler two independent
  // chains and one vote for both.
  template <int N, bool STAGED, bool MASK>
  __device__ __forceinline__ void pages(const uint8_t* const (&rec)[N], const int (&valid)[N], int lane) {
    const int gl = lane >> 2;
    float x[N][2][2];                      // [page][token gl / gl + 8][head]
#pragma unroll
    for (int n = 0; n < N; n++) scores(x[n], rec[n], lane);
    uint32_t vs[N][2][NG];                 // value scales of tokens gl, gl + 8
#pragma unroll
    for (int n = 0; n < N; n++) {
#pragma unroll
      for (int e = 0; e < 2; e++) load_words<NG>(vs[n][e], rec[n] + R::kValScale + (gl + 8 * e) * (4 * NG));
      if (MASK && valid[n] < kKvqPage) {
        // rows past the sequence may hold anything, NaN scales included
#pragma unroll
        for (int e = 0; e < 2; e++)
          if (gl + 8 * e >= valid[n]) {
            x[n][e][0] = x[n][e][1] = -INFINITY;
#pragma unroll
            for (int g = 0; g < NG; g++) vs[n][e][g] = 0u;
          }
      }
    }
    float p[N][2][2], top;
    uint32_t wt[PT][N][NG][2];             // weights of both heads, FP16 (high halves, low halves)
    auto weights = [&]() {
      top = 0.f;
#pragma unroll
      for (int n = 0; n < N; n++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const float2 u = __fadd2_rn(make_float2(x[n][e][0], x[n][e][1]), make_float2(-r[0], -r[1]));
          p[n][e][0] = ex2(u.x);
          p[n][e][1] = ex2(u.y);
          top = fmaxf(fmaxf(top, p[n][e][0]), p[n][e][1]);
#pragma unroll
          for (int g = 0; g < NG; g++) {
            const float st = bf16lo(vs[n][e][g]);
            const float2 wv = __fmul2_rn(__fmul2_rn(make_float2(p[n][e][0], p[n][e][1]), make_float2(st, st)), make_float2(sc[g][0], sc[g][1]));
            const float w0 = wv.x, w1 = wv.y;
            top = fmaxf(fmaxf(top, w0), w1);
            const uint32_t hi = pack_h2(w0, w1);
            wt[0][n][g][e] = hi;
            if constexpr (PT == 2) {
              const float2 hv = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              wt[1][n][g][e] = pack_h2(w0 - hv.x, w1 - hv.y);
            }
          }
        }
    };
    weights();
    if (__builtin_expect(__any_sync(0xffffffffu, top > kTop), 0)) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        float m = -INFINITY;
#pragma unroll
        for (int n = 0; n < N; n++) m = fmaxf(m, fmaxf(x[n][0][h], x[n][1][h]));
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, sh));
        const float rn = fmaxf(r[h], m - kHead);
        const float al = ex2(r[h] - rn), up = ex2(rn - r[h]);
        r[h] = rn;
        l[h] *= al;
#pragma unroll
        for (int g = 0; g < NG; g++) {
          om[g][h] *= al;
          float t = 0.f;
#pragma unroll
          for (int n = 0; n < N; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) t = fmaxf(t, ex2(x[n][e][h] - rn) * bf16lo(vs[n][e][g]));
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, sh));
          // at most what keeps the old weights where they were, and this page's within 2^8; a power of two (the
          // exponent alone), so that it rounds nothing, and its inverse is another exponent
          const float fit = __uint_as_float((uint32_t)min(kScMaxExp, 261 - (int)(__float_as_uint(t) >> 23)) << 23);
          float s = fminf(sc[g][h] * up, fit);
          s = __uint_as_float(__float_as_uint(s) & 0x7f800000u);
          const float be = al == 0.f ? 0.f : al * (s * __uint_as_float(0x7f000000u - __float_as_uint(sc[g][h])));
          sc[g][h] = s;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            o[4 * g + i][h] *= be;
            o[4 * g + i][2 + h] *= be;
          }
        }
      }
      weights();
    }
#pragma unroll
    for (int n = 0; n < N; n++) {
      const float2 p0 = make_float2(p[n][0][0], p[n][0][1]), p1 = make_float2(p[n][1][0], p[n][1][1]);
      const float2 ln = __fadd2_rn(make_float2(l[0], l[1]), __fadd2_rn(p0, p1));
      l[0] = ln.x;
      l[1] = ln.y;
#pragma unroll
      for (int g = 0; g < NG; g++) {
        const float m0 = fmaf(8.f, bf16lo(vs[n][0][g]), bf16hi(vs[n][0][g]));
        const float m1 = fmaf(8.f, bf16lo(vs[n][1][g]), bf16hi(vs[n][1][g]));
        const float2 t = __ffma2_rn(
            p1, make_float2(m1, m1), __ffma2_rn(p0, make_float2(m0, m0), make_float2(om[g][0], om[g][1])));
        om[g][0] = t.x;
        om[g][1] = t.y;
      }
    }
#pragma unroll
    for (int n = 0; n < N; n++) {
      uint32_t v[2][NW];
      load_values<STAGED>(v, rec[n], lane);
#pragma unroll
      for (int g = 0; g < NG; g++) {
        // W^T as the B operand: the score tiles [token][head] transposed
        uint32_t b[PT][2];
#pragma unroll
        for (int t = 0; t < PT; t++)
#pragma unroll
          for (int e = 0; e < 2; e++) b[t][e] = movm_trans(wt[t][n][g][e]);
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const int j = 2 * g + u;
          const uint32_t a = v[0][j], c = v[1][j], a8 = a >> 8, c8 = c >> 8;
          const uint32_t c0[4] = {centred(a), centred16(a), centred(c), centred16(c)};
          const uint32_t c1[4] = {centred(a8), centred16(a8), centred(c8), centred16(c8)};
          add_tile(o[2 * j], c0, b);
          add_tile(o[2 * j + 1], c1, b);
        }
      }
    }
  }

  // the warp's sums against r: l over all its tokens, and v[g][h][8] = dims
  // 64 g + 8 gl .. + 7 of head 2 cq + h
  __device__ __forceinline__ void finish(float (*v)[2][8]) {
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], sh);
#pragma unroll
        for (int g = 0; g < NG; g++) om[g][h] += __shfl_xor_sync(0xffffffffu, om[g][h], sh);
      }
#pragma unroll
    for (int g = 0; g < NG; g++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const float un = 1.f / sc[g][h];
#pragma unroll
        for (int t = 0; t < 4; t++) {      // tile t: dims 2 t and (16 times its codes) 2 t + 1
          v[g][h][2 * t] = fmaf(o[4 * g + t][h], un, om[g][h]);
          v[g][h][2 * t + 1] = fmaf(o[4 * g + t][2 + h] * 0.0625f, un, om[g][h]);
        }
      }
  }
};

}  // namespace mk
