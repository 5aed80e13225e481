// Sparse single-token decode over the 4-bit KV cache: the split form with its
// partials, and the whole step (select, attention, merge) in one launch.
//
// With a group's value s·code + m, the products split into an integer part and
// a part that needs only sums:
//   q·k  = Σ_j s_j (q_j · code_j) + Σ_j m_j (Σ q_j)        (j: groups of 32)
//   Σ p v = Σ_i (p_i s_ij) code_i + Σ_i p_i m_ij            (i: tokens)
// Codes are never converted to numbers. A nibble in the low byte of a 16-bit
// half is an fp16 subnormal: code · 2^-24 in bits 0..3, code · 2^-20 in bits
// 4..7. One AND makes an mma operand register out of a code word, and the
// powers of two are taken out of q and of the outputs, exactly.
//
//  - Logits: A = 16 tokens x 16 channels of codes, B = the G <= 8 query heads,
//    so S comes as tokens x heads. q is bf16 and becomes fp16 by a power of two
//    per head (its largest value lies in [2^15, 2^16): what falls below fp16's
//    range is under 2^-39 of that). Each group's product is scaled by s in
//    fp32. The minima are one bf16 mma against Σ q_j in three bf16 parts.
//  - P·V: A = 16 channels x 16 tokens of codes, B = P·s per group. P leaves
//    the first product as tokens x heads, and movmatrix transposes it into the
//    B layout. P (times 2^8) and P·s are rounded to fp16, 11 bits, against 8
//    if they were bf16. s enters fp16 by a subtraction from its exponent field;
//    the base `lo` of that field follows the largest step met, as the running
//    maximum of the softmax follows the logits. The minima part is fp32 FMAs.
//
// Every warp works alone on whole 64-token blocks: no block-wide barrier in
// its loop, its own ring of K and V records in shared memory (cp.async, no
// spin waits), its own running maximum. The warps' partials meet at the end.
#include <cooperative_groups.h>

#include "kv4.cuh"

namespace sas {

namespace cg = cooperative_groups;
using namespace kv4;

namespace {

constexpr int kWarps = 4;           // warps of a CTA
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;      // portable cluster size
constexpr int kMaxPicks = 255;      // one-launch form: picks of a row
constexpr int kWarpBlocks = 64;     // blocks of a warp: a row's 256 over the 4 warps of one CTA
constexpr float kPShift = -20.f;    // P is kept times 2^-20: sums of a million tokens of P·V stay in fp32's range
constexpr float kPToHalf = 268435456.f;  // and goes to the tensor cores times 2^8: 2^28
constexpr int kStepField = 17;      // exponent field that the largest step gets in fp16 when the base is set
constexpr int kStepLimit = 23;      // a step with this field (2^8) moves the base: P·s stays under 2^16

struct Kv4DecodeArgs {
  const uint16_t* q;
  Cache c;
  const int32_t* cache_len;
  const float* s;
  const int32_t* idx_in;   // split form: the picks and LSE(s)
  const float* lse_s_in;
  int32_t* idx_out;        // one-launch form, each may be null
  float* lse_s_out;
  float* o_part;           // split form
  float* lse_part;
  uint16_t* o;             // one-launch form
  float* lse_o;            // may be null
  int* err;
  int B, Hkv, G, Lmax, K, gate, gated, n_split;
  float scale;
};

__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_zero(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_zero(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t y;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }  // -126 <= e <= 127
__device__ __forceinline__ float exp2_approx(float x) {  // 2^x, relative error about 2^-22, 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // a NaN is passed over, as fmaxf does
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// One group's words of NG (2 or 4): an 8- or 16-byte vector of shared memory.
template <int NG>
struct Words {
  uint32_t w[NG];
};
template <int NG>
__device__ __forceinline__ Words<NG> lds_words(const uint8_t* p) {
  Words<NG> r;
  if (NG == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[NG > 2 ? 2 : 0] = v.z, r.w[NG > 2 ? 3 : 0] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  }
  return r;
}
// The bf16 of NG groups (a token's steps or minima), as NG/2 registers.
template <int NG>
__device__ __forceinline__ Words<NG / 2> lds_params(const uint8_t* p) {
  Words<NG / 2> r;
  if (NG == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[NG / 2 - 1] = v.y;
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}
template <int N>
__device__ __forceinline__ float bf16_of(const Words<N>& r, int j) {
  return (j & 1) ? hi_bf16(r.w[j >> 1]) : lo_bf16(r.w[j >> 1]);
}

// The query heads of a row as B fragments. In the layouts of mma m16n8k16 a
// lane is (g, t) = (lane / 4, lane % 4): it holds head g of B, and heads 2t and
// 2t + 1 of a result.
template <int D>
struct Query {
  static constexpr int NG = D / kGroup;
  uint32_t b[NG][2][2];  // channels 32 j + 8 t + {0, 4}, {1, 5}/16; {2, 6}, {3, 7}/16
  uint32_t sum[2];       // part t of Σ q_j (three bf16 parts, and 0), groups 0, 1 and 2, 3
  float2 f;              // logit (log2 units) = S · f for heads 2t and 2t + 1
  float2 over;           // factors of S before f where f alone would leave fp32's range (queries above 2^100)
  bool big;              // whether any head of the row has one

  // This lane's channels of head g, as they are in memory.
  static __device__ __forceinline__ void read(const uint16_t* q, int G, uint4 (&x)[NG]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < NG; ++j)
      x[j] = g < G ? *reinterpret_cast<const uint4*>(q + g * D + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
  }

  __device__ __forceinline__ void make(const uint4 (&x)[NG], float scale) {
    const int t = threadIdx.x & 3;
    uint32_t mx = 0;  // largest magnitude, as bf16 bits
#pragma unroll
    for (int j = 0; j < NG; ++j)
      mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x[j].x & 0x7fff7fffu, x[j].y & 0x7fff7fffu),
                                 __vmaxu2(x[j].z & 0x7fff7fffu, x[j].w & 0x7fff7fffu)));
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // Exponent of the largest. The factor 2^(15 - e) stays a normal number: a
    // row under 2^-112 is raised by 2^127 only, which is far enough.
    const int e = max(min(int(mx >> 7), 254) - 127, -112);
    const float2 up = make_float2(exp2_int(15 - e), exp2_int(11 - e));  // the odd channels go in divided by 16
    float part[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      float2 v[4], sm2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = mul_f32x2(make_float2(lo_bf16(w[i]), hi_bf16(w[i])), up);
        sm2 = add_f32x2(sm2, v[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b[j][i][0] = pack_f16x2(v[i].x, v[i + 2].x);
        b[j][i][1] = pack_f16x2(v[i].y, v[i + 2].y);
      }
      float sm = fmaf(sm2.y, 16.f, sm2.x);
      sm += __shfl_xor_sync(0xffffffffu, sm, 1);
      sm += __shfl_xor_sync(0xffffffffu, sm, 2);
      sm *= 5.9604644775390625e-8f;  // 2^-24, the codes' scale
      const float p0 = bf16_to_f32(__bfloat16_as_ushort(__float2bfloat16_rn(sm)));
      const float p1 = bf16_to_f32(__bfloat16_as_ushort(__float2bfloat16_rn(sm - p0)));
      part[j] = t == 0 ? p0 : t == 1 ? p1 : t == 2 ? (sm - p0) - p1 : 0.f;
    }
    sum[0] = pack_bf16x2(part[0], part[1]);
    sum[1] = NG == 4 ? pack_bf16x2(part[NG - 2], part[NG - 1]) : 0u;
    const int e0 = __shfl_sync(0xffffffffu, e, 8 * t), e1 = __shfl_sync(0xffffffffu, e, 8 * t + 4);
    const float c = scale * kLog2e * 512.f;  // 2^24 / 2^15
    // kept positive and finite for any softmax scale: masked logits are -inf · f
    f = make_float2(fminf(fmaxf(c * exp2_int(min(e0, 100)), 1.17549435e-38f), 3.402823466e38f),
                    fminf(fmaxf(c * exp2_int(min(e1, 100)), 1.17549435e-38f), 3.402823466e38f));
    over = make_float2(exp2_int(max(e0 - 100, 0)), exp2_int(max(e1 - 100, 0)));
    big = __any_sync(0xffffffffu, e > 100);
  }
};

// A warp's running state. Rows of `acc` are channels: acc[j][i] holds channel
// 32 j + 4 g + 2 i (elements 0, 1) and 16 times the one after it (elements 2,
// 3) of heads 2t (even elements) and 2t + 1. Every nibble is masked out for a
// row of its own. Whole bytes (x + 16 y, with x as the difference of two rows)
// save an AND per word, 44.9 us against 45.6 over the 2048 blocks of a row. But
// the tensor cores cut their sums off, and x has 17 times that error: on this
// row, whose outputs are small next to Σ p s code, o was off by 0.32 % against
// 0.17 %, the rounding to bf16.
template <int D>
struct State {
  static constexpr int NG = D / kGroup;
  float acc[NG][2][4];
  float2 accm[NG];    // Σ p m over this lane's tokens, heads 2t and 2t + 1
  float m[2], l[2];   // maximum (log2), and Σ p over this lane's tokens (p times 2^-20 throughout)
  float w[2];         // gate outside the softmax: acc and accm are to be multiplied by 2^w
  uint32_t lo;        // base of the steps' exponent field, as bf16 bits in both halves
  uint32_t lim;       // largest step bits below the limit, in both halves

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NG; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][0][i] = acc[j][1][i] = 0.f;
      accm[j] = make_float2(0.f, 0.f);
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    w[0] = w[1] = -INFINITY;
    lo = lim = 0u;
  }
};

// S of NT tiles of tokens from a K record. With FULL, all of them count;
// otherwise those past ntok become -inf.
template <int D, int NT, bool FULL>
__device__ __forceinline__ void score_block(const uint8_t* rec, const Query<D>& q, int ntok, float2 (&S)[NT][2]) {
  using F = Fmt<D>;
  constexpr int NG = F::NG;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (!FULL && 16 * i >= ntok) {
      S[i][0] = S[i][1] = make_float2(-INFINITY, -INFINITY);
      continue;
    }
    const uint8_t* tile = rec + i * F::kTileBytes;
    const Words<NG> w0 = lds_words<NG>(tile + F::k_word(g, t, 0)), w1 = lds_words<NG>(tile + F::k_word(g + 8, t, 0));
    const Words<NG / 2> s0 = lds_params<NG>(tile + F::k_step(g, 0)), s1 = lds_params<NG>(tile + F::k_step(g + 8, 0));
    const Words<NG / 2> m0 = lds_params<NG>(tile + F::min_at(g, 0)), m1 = lds_params<NG>(tile + F::min_at(g + 8, 0));
    float x[4];
    mma_bf16_zero(x, m0.w[0], m1.w[0], NG == 4 ? m0.w[NG / 2 - 1] : 0u, NG == 4 ? m1.w[NG / 2 - 1] : 0u, q.sum[0], q.sum[1]);
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      float c[4];
      const uint32_t a = w0.w[j], b = w1.w[j], a8 = a >> 8, b8 = b >> 8;
      mma_f16_zero(c, a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u, q.b[j][0][0], q.b[j][0][1]);
      mma_f16(c, a8 & 0x000f000fu, b8 & 0x000f000fu, a8 & 0x00f000f0u, b8 & 0x00f000f0u, q.b[j][1][0], q.b[j][1][1]);
      const float y0 = bf16_of(s0, j), y1 = bf16_of(s1, j);
      x[0] = fmaf(c[0], y0, x[0]);
      x[1] = fmaf(c[1], y0, x[1]);
      x[2] = fmaf(c[2], y1, x[2]);
      x[3] = fmaf(c[3], y1, x[3]);
    }
    if (q.big) {
      x[0] *= q.over.x, x[1] *= q.over.y, x[2] *= q.over.x, x[3] *= q.over.y;
    }
    if (!FULL && 16 * i + 16 > ntok) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = 16 * i + g + 8 * (e >> 1) < ntok ? x[e] : -INFINITY;
    }
    S[i][0] = make_float2(x[0], x[1]);
    S[i][1] = make_float2(x[2], x[3]);
  }
}

// The online softmax: S becomes p · 2^-20 with p = 2^(S f + lam - max), and the
// state is rescaled. (f > 0, so the largest logit is that of the largest S.)
//
// With OUT the gate lies outside the softmax: the sum is over 2^(S f - max), and
// S becomes 2^(S f - max + lam - w). The weights have a running maximum 2^w of
// their own, relative to the softmax's, because P has fp16's range and a row's
// mass may lie where its gates are small, or a caller's LSE make them large.
//
// Every S is taken relative to the block's largest before it is scaled: p is
// then at most 1 whatever the logits' size, as the range of fp16 needs it, and
// a token is weighed by its distance from the largest, not by a difference of
// two roundings of large numbers.
template <int D, int NT, bool OUT>
__device__ __forceinline__ void softmax_block(State<D>& st, const Query<D>& q, float lam, float2 (&S)[NT][2]) {
  float top[2], sub[2], al[2], out_sub[2], out_al[2];
  top[0] = fmaxf(S[0][0].x, S[0][1].x);
  top[1] = fmaxf(S[0][0].y, S[0][1].y);
#pragma unroll
  for (int i = 1; i < NT; ++i) {
    top[0] = max3(top[0], S[i][0].x, S[i][1].x);
    top[1] = max3(top[1], S[i][0].y, S[i][1].y);
  }
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) {
    top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
    top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float own = fmaf(top[h], h ? q.f.y : q.f.x, OUT ? 0.f : lam);  // the block's largest logit
    const float mx = fmaxf(st.m[h], own);
    const float ref = mx == -INFINITY ? 0.f : mx;  // nothing but masked tokens so far: every p is 0
    al[h] = exp2_approx(st.m[h] - ref);
    sub[h] = (own - ref) + kPShift;
    if (OUT) {
      const float was = st.w[h] + (st.m[h] - ref), here = (own - ref) + lam;
      st.w[h] = fmaxf(was, here);
      const float wref = st.w[h] == -INFINITY ? 0.f : st.w[h];
      out_al[h] = exp2_approx(was - wref);
      out_sub[h] = (here - wref) + kPShift;
    } else {
      out_al[h] = al[h];
    }
    top[h] = top[h] == -INFINITY ? 0.f : -top[h];
    st.m[h] = mx;
  }
  const float2 less = make_float2(top[0], top[1]);
  const float2 add = make_float2(sub[0], sub[1]);
  const float2 out_add = OUT ? make_float2(out_sub[0], out_sub[1]) : add;
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float2 d = add_f32x2(S[i][u], less);
      float2 z = fma_f32x2(d, q.f, add);
      z.x = exp2_approx(z.x);
      z.y = exp2_approx(z.y);
      sum = add_f32x2(sum, z);
      if (OUT) {
        z = fma_f32x2(d, q.f, out_add);
        z.x = exp2_approx(z.x);
        z.y = exp2_approx(z.y);
      }
      S[i][u] = z;
    }
  st.l[0] = fmaf(st.l[0], al[0], sum.x);
  st.l[1] = fmaf(st.l[1], al[1], sum.y);
  if (__any_sync(0xffffffffu, out_al[0] != 1.f || out_al[1] != 1.f)) {
#pragma unroll
    for (int j = 0; j < State<D>::NG; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        st.acc[j][0][e] *= out_al[e & 1];
        st.acc[j][1][e] *= out_al[e & 1];
      }
      st.accm[j].x *= out_al[0];
      st.accm[j].y *= out_al[1];
    }
  }
}

// O += P V from the block's V record.
template <int D, int NT, bool FULL>
__device__ __forceinline__ void value_block(const uint8_t* rec, State<D>& st, int ntok, const float2 (&p)[NT][2]) {
  using F = Fmt<D>;
  constexpr int NG = F::NG;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (!FULL && 16 * i >= ntok) break;
    const uint8_t* tile = rec + i * F::kTileBytes;
    uint32_t stp[NG][2];  // steps of tokens 2t, 2t + 1 and 2t + 8, 2t + 9
#pragma unroll
    for (int j = 0; j < NG; j += 2) {
      const uint4 v = *reinterpret_cast<const uint4*>(tile + F::kSteps + (t * NG + j) * 8);
      stp[j][0] = v.x, stp[j][1] = v.y, stp[j + 1][0] = v.z, stp[j + 1][1] = v.w;
    }
    const Words<NG> w0 = lds_words<NG>(tile + F::v_half(2 * t, g, 0)), w1 = lds_words<NG>(tile + F::v_half(8 + 2 * t, g, 0));
    Words<NG / 2> m0 = lds_params<NG>(tile + F::min_at(g, 0)), m1 = lds_params<NG>(tile + F::min_at(g + 8, 0));
    if (!FULL && 16 * i + 16 > ntok) {  // tokens past the end may hold anything: their p is 0, and their steps and minima are made 0
      const int r = ntok - 16 * i;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t keep = (8 * h + 2 * t < r ? 0xffffu : 0u) | (8 * h + 2 * t + 1 < r ? 0xffff0000u : 0u);
#pragma unroll
        for (int j = 0; j < NG; ++j) stp[j][h] &= keep;
      }
#pragma unroll
      for (int j = 0; j < NG / 2; ++j) {
        m0.w[j] = g < r ? m0.w[j] : 0u;
        m1.w[j] = g + 8 < r ? m1.w[j] : 0u;
      }
    }
    uint32_t mx = st.lim;
#pragma unroll
    for (int j = 0; j < NG; ++j) mx = __vimax3_u16x2(mx, stp[j][0], stp[j][1]);
    if (__any_sync(0xffffffffu, mx != st.lim)) {  // a step past the limit, or the first that is not 0: the base moves up
      const uint32_t top = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
      const int old = int((st.lo & 0xffffu) >> 7), now = max(old, int(top >> 7) - kStepField);
      const float f = exp2_approx(float(old - now));
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          st.acc[j][0][e] *= f;
          st.acc[j][1][e] *= f;
        }
      st.lo = uint32_t(now << 7) * 0x10001u;
      st.lim = uint32_t(((now + kStepLimit) << 7) - 1) * 0x10001u;
    }
    const float2 h0 = mul_f32x2(p[i][0], make_float2(kPToHalf, kPToHalf)), h1 = mul_f32x2(p[i][1], make_float2(kPToHalf, kPToHalf));
    const uint32_t p0 = transpose8x8(pack_f16x2(h0.x, h0.y)), p1 = transpose8x8(pack_f16x2(h1.x, h1.y));
    const uint32_t lo8 = 0u - 8u * st.lo;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      // (max(bits, lo) - lo) << 3 in both halves: the fp16 whose exponent field is the step's less lo's
      const uint32_t b0 = mul_f16x2(p0, __vmaxu2(stp[j][0], st.lo) * 8u + lo8);
      const uint32_t b1 = mul_f16x2(p1, __vmaxu2(stp[j][1], st.lo) * 8u + lo8);
      const uint32_t a = w0.w[j], b = w1.w[j], a8 = a >> 8, b8 = b >> 8;
      mma_f16(st.acc[j][0], a & 0x000f000fu, a & 0x00f000f0u, b & 0x000f000fu, b & 0x00f000f0u, b0, b1);
      mma_f16(st.acc[j][1], a8 & 0x000f000fu, a8 & 0x00f000f0u, b8 & 0x000f000fu, b8 & 0x00f000f0u, b0, b1);
      const float x0 = bf16_of(m0, j), x1 = bf16_of(m1, j);
      st.accm[j].x = fmaf(p[i][1].x, x1, fmaf(p[i][0].x, x0, st.accm[j].x));
      st.accm[j].y = fmaf(p[i][1].y, x1, fmaf(p[i][0].y, x0, st.accm[j].y));
    }
  }
}

// A warp's copy of END bytes, 512 per instruction, the offsets as immediates
// (address arithmetic per copy took a tenth of the loop's instructions).
template <int O, int END>
__device__ __forceinline__ void copy_lines(uint32_t dst, const uint8_t* src) {
  if constexpr (O + 512 <= END) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;\n" ::"r"(dst), "l"(src), "n"(O));
    copy_lines<O + 512, END>(dst, src);
  } else if constexpr (O < END) {
    if ((threadIdx.x & 31) * 16 < END - O)
      asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;\n" ::"r"(dst), "l"(src), "n"(O));
  }
}

// A warp's ring: the K record of a block in one slot, its V record in the other.
// Item 2 i is block i's K, item 2 i + 1 its V; a slot is refilled as soon as it
// has been used. Records are named by their number (-1: a block left out).
template <int D>
struct Ring {
  static constexpr int kRecord = Fmt<D>::kRecord;
  static constexpr int kBytes = 2 * kRecord;

  static __device__ __forceinline__ void issue(uint8_t* ring, const Cache& c, int item, int rec, int ntok) {
    const int lane = threadIdx.x & 31;
    const uint8_t* src = ((item & 1) ? c.v : c.k) + size_t(rec) * kRecord + lane * 16;
    const uint32_t dst = smem_u32(ring) + (item & 1) * kRecord + lane * 16;
    if (ntok == kBlock) {
      copy_lines<0, kRecord>(dst, src);
    } else {  // the tiles that hold tokens
      const int bytes = (ntok + kTile - 1) / kTile * Fmt<D>::kTileBytes;
#pragma unroll 1
      for (int o = 0; o + lane * 16 < bytes; o += 512) cp_async16(dst + o, src + o);
    }
  }
  // Item `item` of n blocks, as a copy group of its own.
  static __device__ __forceinline__ void step(uint8_t* ring, const Cache& c, const int* rec_s, int n, int ntok0, int item) {
    if (item < 2 * n) {
      const int rec = rec_s[item >> 1];
      if (rec >= 0) issue(ring, c, item, rec, item < 2 ? ntok0 : kBlock);
    }
    cp_async_commit();
  }
};

// A warp over its n blocks: records rec_s, gates lam_s (log2). The first block
// has ntok0 tokens, the others all. Both items of the first are under way. A
// block that is not full goes through a loop of single tiles, which keeps the
// code that a warp has to fetch small.
template <int D, bool OUT>
__device__ __forceinline__ void run_blocks(const Kv4DecodeArgs& a, State<D>& st, const Query<D>& q, uint8_t* ring,
                                           const int* rec_s, const float* lam_s, int n, int ntok0) {
  using R = Ring<D>;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int ntok = rec_s[i] < 0 ? 0 : i == 0 ? ntok0 : kBlock;
    const float lam = a.gated ? lam_s[i] : 0.f;
    if (ntok == kBlock) {
      float2 S[kTiles][2];
      cp_async_wait<1>();
      __syncwarp();
      score_block<D, kTiles, true>(ring, q, ntok, S);
      __syncwarp();
      R::step(ring, a.c, rec_s, n, ntok0, 2 * i + 2);
      softmax_block<D, kTiles, OUT>(st, q, lam, S);
      cp_async_wait<1>();
      __syncwarp();
      value_block<D, kTiles, true>(ring + R::kRecord, st, ntok, S);
    } else {
      cp_async_wait<0>();
      __syncwarp();
#pragma unroll 1
      for (int k = 0; k * kTile < ntok; ++k) {
        float2 S[1][2];
        const uint8_t* tile = ring + k * Fmt<D>::kTileBytes;
        score_block<D, 1, false>(tile, q, ntok - k * kTile, S);
        softmax_block<D, 1, OUT>(st, q, lam, S);
        value_block<D, 1, false>(tile + R::kRecord, st, ntok - k * kTile, S);
      }
      __syncwarp();
      R::step(ring, a.c, rec_s, n, ntok0, 2 * i + 2);
    }
    __syncwarp();
    R::step(ring, a.c, rec_s, n, ntok0, 2 * i + 3);
  }
  cp_async_wait<0>();
}

// The merge of a row's (or a split's) partials over CS CTAs. A warp's partial
// is G x D normalised outputs in units of 4 channels, with the maximum and the
// sum of every head. The units of the lanes g (channels 32 j + 4 g) are merged
// by CTA g % CS: the warps store them straight into its shared memory, so that
// one cluster barrier is enough and no CTA reads another's memory.
template <int D>
struct Merge {
  static constexpr int NG = D / kGroup;
  int CS, rank, GS, U;  // GS lanes g and U = G · NG · GS units per CTA
  float4* o;            // [warp of the cluster][head][group][lane g / CS]
  float2* ml;           // [warp of the cluster][8 heads]

  static __host__ __device__ constexpr int lanes(int CS) { return (7 + CS) / CS; }
  static __host__ __device__ constexpr int bytes(int G, int CS) { return CS * kWarps * (G * NG * lanes(CS) * 16 + 64); }
  static constexpr int max_bytes(int CS = kMaxCluster) {  // of G <= 8 and up to CS CTAs
    return CS == 1 ? bytes(8, 1) : max_bytes(CS - 1) > bytes(8, CS) ? max_bytes(CS - 1) : bytes(8, CS);
  }

  __device__ __forceinline__ Merge(uint8_t* smem, int G, int CS, int rank)
      : CS(CS), rank(rank), GS(lanes(CS)), U(G * NG * GS), o(reinterpret_cast<float4*>(smem)),
        ml(reinterpret_cast<float2*>(smem + CS * kWarps * U * 16)) {}

  template <bool CLUSTER, bool OUT>
  __device__ __forceinline__ void push(State<D>& st, int G) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, from = rank * kWarps + int(threadIdx.x >> 5);
    // the minima's sums over the lanes g: lane g gets the total of one (group,
    // head), and hands it to the others
    float am[2 * NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) am[2 * j] = st.accm[j].x, am[2 * j + 1] = st.accm[j].y;
#pragma unroll
    for (int x = 16, n = NG; n >= 1; x >>= 1, n >>= 1) {
      const bool up = (lane & x) != 0;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = up ? am[i] : am[n + i], keep = up ? am[n + i] : am[i];
        am[i] = keep + __shfl_xor_sync(0xffffffffu, give, x);
      }
    }
    if (NG == 2) am[0] += __shfl_xor_sync(0xffffffffu, am[0], 4);
    // 2^24 of the codes, 2^-28 of P, 2^-112 of the two exponents' biases
    const int lo_e = int((st.lo & 0xffffu) >> 7);
    const float f = exp2_int(min(lo_e, 200) - 116);
    if (lo_e > 200) {
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.acc[j][0][e] *= exp2_int(lo_e - 200), st.acc[j][1][e] *= exp2_int(lo_e - 200);
    }
    const int slot = g / CS, owner = g - slot * CS;
    float4* dst = o + from * U + 2 * t * NG * GS + slot;
    if (CLUSTER) dst = cg::this_cluster().map_shared_rank(dst, owner);
    float l[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] = st.l[h];
#pragma unroll
      for (int x = 4; x <= 16; x <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
      float inv = l[h] == 0.f ? 0.f : __fdividef(1.f, l[h]);
      if (OUT) inv *= exp2_approx(st.w[h]);
      const float f0 = inv * f, f1 = f0 * 0.0625f;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const int from_g = NG == 4 ? 2 * j + h : 2 * (2 * j + h);
        const float m = __shfl_sync(0xffffffffu, am[0], from_g * 4 + t) * inv;
        if (2 * t + h < G)
          dst[(h * NG + j) * GS] =
              make_float4(fmaf(st.acc[j][0][h], f0, m), fmaf(st.acc[j][0][2 + h], f1, m),
                          fmaf(st.acc[j][1][h], f0, m), fmaf(st.acc[j][1][2 + h], f1, m));
      }
    }
    if (g < CS) {
      float4* to = reinterpret_cast<float4*>(ml + from * 8 + 2 * t);
      if (CLUSTER) to = cg::this_cluster().map_shared_rank(to, g);
      *to = make_float4(st.m[0], l[0], st.m[1], l[1]);
    }
  }

  // As many lanes to a unit (1 to 8) as the CTA has; out(head, channel, outputs,
  // lse) stores it. A row whose sum is NaN in any partial is NaN. The loops are
  // not unrolled: the code runs once, and fetching it is part of its time.
  template <typename Out>
  __device__ __forceinline__ void run(Out out) const {
    const int n = CS * kWarps;
    int lanes = 8;
    while (lanes > 1 && lanes * U > kThreads) lanes >>= 1;
    const int sub = threadIdx.x & (lanes - 1), unit = int(threadIdx.x) / lanes, step = kThreads / lanes;
#pragma unroll 1
    for (int base = 0; base < U; base += step) {
      const int s = min(base + unit, U - 1), hj = s / GS, g = (s - hj * GS) * CS + rank;
      const int head = hj / NG;
      const float2* mh = ml + head;
      const float4* oh = o + s;
      float M = -INFINITY;
#pragma unroll 1
      for (int w = sub; w < n; w += lanes) M = fmaxf(M, mh[w * 8].x);
#pragma unroll 1
      for (int x = 1; x < lanes; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
      const float ref = M == -INFINITY ? 0.f : M;
      float den = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int w = sub; w < n; w += lanes) {
        const float2 p = mh[w * 8];
        const float4 y = oh[w * U];
        const float k = p.y * exp2_approx(p.x - ref);
        const bool any = p.y != 0.f;  // not a warp without tokens
        den += any ? k : 0.f;
        v.x = any ? fmaf(k, y.x, v.x) : v.x;
        v.y = any ? fmaf(k, y.y, v.y) : v.y;
        v.z = any ? fmaf(k, y.z, v.z) : v.z;
        v.w = any ? fmaf(k, y.w, v.w) : v.w;
      }
#pragma unroll 1
      for (int x = 1; x < lanes; x <<= 1) {
        den += __shfl_xor_sync(0xffffffffu, den, x);
        v.x += __shfl_xor_sync(0xffffffffu, v.x, x);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, x);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, x);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, x);
      }
      if (sub != 0 || g >= 8 || base + unit >= U) continue;
      const float inv = den == 0.f ? 0.f : __fdividef(1.f, den);
      out(head, 32 * (hj - head * NG) + 4 * g, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv),
          den == 0.f ? -INFINITY : (M + __log2f(den) - kPShift) * kLn2);
    }
  }
};

// The first barrier of a cluster (its CTAs have started: their memory may be
// written), and the second (what was written is there).
__device__ __forceinline__ void cluster_begin() { asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// One warp's Top-K of a score row, without a block-wide barrier: lane i holds
// the keys of blocks i, 32 + i, ... in registers. A bisection between the
// smallest and the largest key finds a threshold with n keys at or above it, in
// half a dozen counts of the row (quarter_keys). Where a tie is cut, it ends on
// the tied key.
template <int CAP>
struct Row {
  uint32_t key[CAP];  // orderable key + 1, 0 past the history

  __device__ __forceinline__ void read(const float* s, int NB) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < CAP; ++i) key[i] = 32 * i + lane < NB ? __float_as_uint(__ldg(s + 32 * i + lane)) : 0u;
  }
  __device__ __forceinline__ void make(int c) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < CAP; ++i) key[i] = 32 * i + lane < c ? score_key(__uint_as_float(key[i])) + 1u : 0u;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t k = 0;
#pragma unroll
    for (int i = 0; i < CAP; ++i) k = max(k, key[i]);
    return __reduce_max_sync(0xffffffffu, k);
  }
  // log Σ exp of the row's scores, as the select kernels take it
  __device__ __forceinline__ float lse(int c) const {
    const uint32_t k = top();
    const float mx = k <= 1u ? -INFINITY : key_score(k - 1u);
    if (mx == -INFINITY) return -INFINITY;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < CAP; ++i)
      if (32 * i < c && key[i] != 0u) sum += expf(key_score(key[i] - 1u) - mx);
    return mx + logf(warp_sum(sum));
  }
  // The n highest of the c blocks (ties to the lower block), ascending, to sel.
  __device__ __forceinline__ void select(int c, int n, int* sel) const {
    const int lane = threadIdx.x & 31;
    uint32_t thr = 1u, tied = 0u;  // taken: keys >= thr, and the first `need` that equal tied
    int need = 0;
    if (n < c) {
      uint32_t lo = 0xffffffffu, hi = top() + 1u;  // count(lo) > n > count(hi)
#pragma unroll
      for (int i = 0; i < CAP; ++i) lo = min(lo, key[i] - 1u);
      lo = __reduce_min_sync(0xffffffffu, lo) + 1u;
      int above = 0;  // count(hi)
#pragma unroll 1
      for (int round = 0;; ++round) {
        if (hi - lo <= 1u) {
          thr = hi;
          tied = lo;
          need = n - above;
          break;
        }
        uint32_t mid[3];
        quarter_keys(lo, hi, round, mid);
        int cnt[3] = {0, 0, 0};
#pragma unroll
        for (int i = 0; i < CAP; ++i)
          if (CAP <= 16 || 32 * i < c) {
#pragma unroll
            for (int u = 0; u < 3; ++u) cnt[u] += key[i] >= mid[u] ? 1 : 0;
          }
#pragma unroll
        for (int u = 0; u < 3; ++u) cnt[u] = __reduce_add_sync(0xffffffffu, cnt[u]);
        if (cnt[0] == n || cnt[1] == n || cnt[2] == n) {
          thr = cnt[0] == n ? mid[0] : cnt[1] == n ? mid[1] : mid[2];
          break;
        }
#pragma unroll
        for (int u = 0; u < 3; ++u)
          if (cnt[u] > n) lo = mid[u];
#pragma unroll
        for (int u = 2; u >= 0; --u)
          if (cnt[u] < n) {
            hi = mid[u];
            above = cnt[u];
          }
      }
    }
    const unsigned below = (1u << lane) - 1u;
    int base = 0;
    if (need == 0) {
#pragma unroll
      for (int i = 0; i < CAP; ++i) {
        const unsigned b = __ballot_sync(0xffffffffu, key[i] >= thr);
        if (key[i] >= thr) sel[base + __popc(b & below)] = 32 * i + lane;
        base += __popc(b);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < CAP; ++i) {
      const unsigned eq = __ballot_sync(0xffffffffu, key[i] == tied);
      const bool take = key[i] >= thr || (key[i] == tied && __popc(eq & below) < need);
      need -= min(need, __popc(eq));
      const unsigned b = __ballot_sync(0xffffffffu, take);
      if (take) sel[base + __popc(b & below)] = 32 * i + lane;
      base += __popc(b);
    }
  }
};

}  // namespace

// One CTA per (sequence, KV head, split), or a cluster of CS. The blocks of
// the split's run go round the cluster's warps.
//
// All 2048 blocks of 8 heads of d = 128 in 64 splits: 36.9 us, 4.5 TB/s of
// records. 1200 instructions a block, the integer pipe (ANDs, shifts, steps into
// fp16) busy half of the time, and 512 CTAs on 148 multiprocessors, 3 on some
// and 4 on others. 64 ragged rows, K = 64, in 9 splits: 14.2 us, most of it the
// way to the first block. 4 CTAs of 128 registers a multiprocessor, against 3
// of 168 in the one-launch form, whose registers the selection needs. At d = 128
// the bound of 128 spills 36 to 48 bytes a thread. Clusters
// past one wave of CTAs cost more than they even out (128K 45.8 -> 52.9 us for
// the step).
template <int D, bool CLUSTER, bool OUT>
__global__ void __launch_bounds__(kThreads, 4) kv4_decode_split_kernel(Kv4DecodeArgs a) {
  using R = Ring<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int rec_s[kWarps][kMaxDecodeBlocksPerSplit / kWarps];
  __shared__ float lam_s[kWarps][kMaxDecodeBlocksPerSplit / kWarps];
  const int CS = CLUSTER ? int(cg::this_cluster().num_blocks()) : 1;
  const int rank = CLUSTER ? int(cg::this_cluster().block_rank()) : 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = CS * kWarps, worker = warp * CS + rank;
  const int item = blockIdx.x / CS, split = item % a.n_split, bh = item / a.n_split, b = bh / a.Hkv, h = bh % a.Hkv;
  const int NB = a.Lmax / kBlock;
  uint8_t* ring = smem + warp * R::kBytes;
  if (CLUSTER) cluster_begin();
  griddep_launch_dependents();  // the merge kernel may begin its launch; it waits for this grid's writes
  griddep_wait();               // idx and lse_s come from the select kernel that precedes this one
  int L = a.cache_len[b];
  uint4 raw[D / kGroup];
  Query<D>::read(a.q + size_t(bh) * a.G * D, a.G, raw);
  if (L < 1 || L > a.Lmax) {
    if (tid == 0) raise_error(a.err, SAS_ERR_DEVICE_INDEX);
    L = max(1, min(L, a.Lmax));
  }
  const int c = (L - 1) / kBlock, nl = 1 + min(a.K, c);
  const int per = (nl + a.n_split - 1) / a.n_split;
  const int lo = min(split * per, nl), blocks = min(lo + per, nl) - lo;
  const int n = worker < blocks ? (blocks - 1 - worker) / W + 1 : 0;
  for (int k = lane; k < n; k += 32) {
    const int pos = lo + k * W + worker;
    int m = c;
    float lam = 0.f;
    if (pos > 0) {
      m = a.idx_in[size_t(bh) * a.K + pos - 1];
      if (m >= c) raise_error(a.err, SAS_ERR_DEVICE_INDEX);
      if (m < 0 || m >= c)
        m = -1;
      else if (a.gated)
        lam = gate_lam2(a.gate, a.s[size_t(bh) * NB + m], a.lse_s_in != nullptr ? a.lse_s_in[bh] : 0.f);
    }
    const int rec = m < 0 ? -1 : record_of(a.c, b, h, m, a.Hkv, NB, a.err);
    rec_s[warp][k] = rec;
    lam_s[warp][k] = rec < 0 ? 0.f : lam;
  }
  __syncwarp();
  const int ntok0 = lo == 0 && worker == 0 ? L - c * kBlock : kBlock;  // tokens of the warp's first block
  R::step(ring, a.c, rec_s[warp], n, ntok0, 0);
  R::step(ring, a.c, rec_s[warp], n, ntok0, 1);
  Query<D> q;
  q.make(raw, a.scale);
  State<D> st;
  st.clear();
  run_blocks<D, OUT>(a, st, q, ring, rec_s[warp], lam_s[warp], n, ntok0);
  const Merge<D> mg(CLUSTER ? smem + kWarps * R::kBytes : smem, a.G, CS, rank);
  if (CLUSTER) {
    cluster_begun();
    mg.template push<true, OUT>(st, a.G);
    cluster_sync();
  } else {
    __syncthreads();  // the rings are done with, and the partials take their place
    mg.template push<false, OUT>(st, a.G);
    __syncthreads();
  }
  mg.run([&](int head, int col, float4 o, float lse) {
    const size_t row = (size_t(bh) * a.G + head) * a.n_split + split;
    *reinterpret_cast<float4*>(a.o_part + row * D + col) = o;
    if (col == 0) a.lse_part[row] = lse;
  });
}

// One cluster per (sequence, KV head). In each CTA one warp selects the row's
// blocks, in registers, and another takes the row's LSE if it is needed; then
// every warp of the cluster takes every W-th block of the list [current block,
// picks...]. The CTAs' redundant selection is cheaper than a hand-over between
// them, a selection by every warp was not: three CTAs share a multiprocessor,
// and their instructions count.
//
// 128 rows, K = 16 of 511 blocks, d = 128: 12.2 us (the bf16 cache's step 19.7),
// 8 rows, K = 64 of 127: 9.7 us (15.0). It is a chain of latencies; alone, the
// picks are known after 3.6 us, the records after 4.4, the blocks done after
// 8.8, the partials merged after 11.6. Selecting nothing would save 0.2 us, for
// the rest is hidden by the other warps and the launches on either side.
// Clusters of 16 for few rows are slower (9.8 -> 10.7 us).
template <int D, int CAP, bool OUT>
__global__ void __launch_bounds__(kThreads, 3) kv4_decode_fused_kernel(Kv4DecodeArgs a) {
  using R = Ring<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int sel_s[kMaxPicks + 1];
  __shared__ int rec_s[kWarps][kWarpBlocks];
  __shared__ float lam_s[kWarps][kWarpBlocks];
  __shared__ float lse_s;
  const int CS = int(cg::this_cluster().num_blocks()), rank = int(cg::this_cluster().block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = CS * kWarps;
  // the selecting warp is the last: the first ones start on the current block
  const int worker = warp * CS + rank;
  const int bh = int(blockIdx.x) / CS, b = bh / a.Hkv, h = bh % a.Hkv;
  const int NB = a.Lmax / kBlock;
  uint8_t* ring = smem + warp * R::kBytes;
  const float* srow = a.s + size_t(bh) * NB;
  const bool soft = a.gate == SAS_GATE_LOG_SOFTMAX || a.gate == SAS_GATE_SOFTMAX_OUTSIDE;
  cluster_begin();
  griddep_launch_dependents();
  griddep_wait();
  int L = a.cache_len[b];
  Row<CAP> row;
  const bool selects = warp == kWarps - 1, sums = warp == kWarps - 2 && (soft || (rank == 0 && a.lse_s_out != nullptr));
  if (selects || sums) row.read(srow, NB);
  uint4 raw[D / kGroup];
  Query<D>::read(a.q + size_t(bh) * a.G * D, a.G, raw);
  if (a.c.table != nullptr && tid * 32 < NB)  // the row's pages, for the lookup of the picks
    asm volatile("prefetch.global.L1 [%0];\n" ::"l"(a.c.table + size_t(b) * NB + tid * 32));
  if (L < 1 || L > a.Lmax) {
    if (tid == 0) raise_error(a.err, SAS_ERR_DEVICE_INDEX);
    L = max(1, min(L, a.Lmax));
  }
  const int c = (L - 1) / kBlock, n_pick = min(a.K, c);
  const int n = worker <= n_pick ? (n_pick - worker) / W + 1 : 0;
  const bool has_cur = worker == 0;
  const int ntok0 = has_cur ? L - c * kBlock : kBlock;
  if (has_cur) {  // the current block needs no selection
    const int rec = record_of(a.c, b, h, c, a.Hkv, NB, a.err);
#pragma unroll
    for (int item = 0; item < 2; ++item) {
      if (rec >= 0) R::issue(ring, a.c, item, rec, ntok0);
      cp_async_commit();
    }
  }
  if (selects) {
    row.make(c);
    row.select(c, n_pick, sel_s);
  } else if (sums) {
    row.make(c);
    const float lse = row.lse(c);
    if (lane == 0) {
      lse_s = lse;
      if (rank == 0 && a.lse_s_out != nullptr) a.lse_s_out[bh] = lse;
    }
  }
  Query<D> q;
  if (!selects) q.make(raw, a.scale);
  __syncthreads();  // the picks and the LSE
  const float lse = soft ? lse_s : 0.f;
  for (int k = lane; k < n; k += 32) {
    const int pos = k * W + worker, m = pos > 0 ? sel_s[pos - 1] : c;
    const float sm = a.gated && pos > 0 ? __ldg(srow + m) : 0.f;
    const int rec = record_of(a.c, b, h, m, a.Hkv, NB, a.err);
    rec_s[warp][k] = rec;
    lam_s[warp][k] = a.gated && pos > 0 && rec >= 0 ? gate_lam2(a.gate, sm, lse) : 0.f;
  }
  __syncwarp();
  if (!has_cur) {
    R::step(ring, a.c, rec_s[warp], n, ntok0, 0);
    R::step(ring, a.c, rec_s[warp], n, ntok0, 1);
  }
  if (selects) q.make(raw, a.scale);
  if (rank == 0 && warp == 0 && a.idx_out != nullptr)
    for (int i = lane; i < a.K; i += 32) a.idx_out[size_t(bh) * a.K + i] = i < n_pick ? sel_s[i] : -1;
  State<D> st;
  st.clear();
  run_blocks<D, OUT>(a, st, q, ring, rec_s[warp], lam_s[warp], n, ntok0);
  const Merge<D> mg(smem + kWarps * R::kBytes, a.G, CS, rank);
  cluster_begun();
  mg.template push<true, OUT>(st, a.G);
  cluster_sync();
  mg.run([&](int head, int col, float4 o, float ls) {
    const size_t at = size_t(bh) * a.G + head;
    *reinterpret_cast<uint2*>(a.o + at * D + col) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    if (col == 0 && a.lse_o != nullptr) a.lse_o[at] = ls;
  });
}

static Kv4DecodeArgs kv4_decode_args(const Shape& sh, const uint16_t* q, const Cache& c, const int32_t* cl,
                                     const float* s, int* err) {
  Kv4DecodeArgs a = {};
  a.q = q;
  a.c = c;
  a.cache_len = cl;
  a.s = s;
  a.err = err;
  a.B = sh.B;
  a.Hkv = sh.Hkv;
  a.G = sh.G;
  a.Lmax = sh.N;
  a.K = sh.K;
  a.gate = sh.gate;
  a.gated = sh.gated;
  a.scale = sh.scale;
  return a;
}

// Launches `kern` on `items` clusters of cs CTAs, as a dependent launch. cs = 0:
// plain CTAs. The kernel's limit of dynamic shared memory belongs to the
// function, not to the launch: it is one constant per kernel, because a smaller
// one set by another thread's call would refuse this one.
static cudaError_t launch_ctas(void (*kern)(Kv4DecodeArgs), int items, int cs, int smem, int max_smem, cudaStream_t st,
                               const Kv4DecodeArgs& a) {
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(items) * max(cs, 1));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

static cudaError_t multiprocessors(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// Split form. The cluster size: the largest power of two that keeps every CTA
// resident at once (16 warps per SM), at most 8 and at most one warp per block
// of a split.
template <int D, bool OUT>
static cudaError_t launch_split(const Kv4DecodeArgs& a, cudaStream_t st) {
  constexpr int ring = kWarps * Ring<D>::kBytes, max_smem = ring + Merge<D>::max_bytes();
  int sms = 0;
  const cudaError_t e = multiprocessors(&sms);
  if (e != cudaSuccess) return e;
  const int items = a.B * a.Hkv * a.n_split, per = (a.K + a.n_split) / a.n_split;
  const int want = min(min(kMaxCluster, (per + kWarps - 1) / kWarps), sms * 4 / items);
  int cs = 1;
  while (cs * 2 <= want) cs *= 2;
  if (cs == 1) return launch_ctas(kv4_decode_split_kernel<D, false, OUT>, items, 0, max(ring, Merge<D>::bytes(a.G, 1)), max_smem, st, a);
  return launch_ctas(kv4_decode_split_kernel<D, true, OUT>, items, cs, ring + Merge<D>::bytes(a.G, cs), max_smem, st, a);
}

cudaError_t launch_decode_kv4(const Shape& sh, const uint16_t* q, const Cache& c, const int32_t* cl, const float* s,
                              const int32_t* idx, const float* lse_s, int n_split, float* o_part, float* lse_part,
                              int* err, cudaStream_t st) {
  Kv4DecodeArgs a = kv4_decode_args(sh, q, c, cl, s, err);
  a.idx_in = idx;
  a.lse_s_in = lse_s;
  a.n_split = n_split;
  a.o_part = o_part;
  a.lse_part = lse_part;
  if (sh.outside) return sh.d == 128 ? launch_split<128, true>(a, st) : launch_split<64, true>(a, st);
  return sh.d == 128 ? launch_split<128, false>(a, st) : launch_split<64, false>(a, st);
}

// One launch. The cluster size: as many CTAs per row as keep the grid in one
// wave of resident CTAs, at most 8 and at most one warp per block of the list.
template <int D, int CAP, bool OUT>
static cudaError_t launch_fused_as(const Kv4DecodeArgs& a, cudaStream_t st) {
  constexpr int ring = kWarps * Ring<D>::kBytes, max_smem = ring + Merge<D>::max_bytes();
  int sms = 0;
  const cudaError_t e = multiprocessors(&sms);
  if (e != cudaSuccess) return e;
  const int rows = a.B * a.Hkv;
  const int cs = max(1, min(min(kMaxCluster, (a.K + kWarps) / kWarps), sms * 3 / rows));
  return launch_ctas(kv4_decode_fused_kernel<D, CAP, OUT>, rows, cs, ring + Merge<D>::bytes(a.G, cs), max_smem, st, a);
}

template <int D, int CAP>
static cudaError_t launch_fused(const Kv4DecodeArgs& a, bool outside, cudaStream_t st) {
  return outside ? launch_fused_as<D, CAP, true>(a, st) : launch_fused_as<D, CAP, false>(a, st);
}

cudaError_t launch_decode_fused_kv4(const Shape& sh, const uint16_t* q, const Cache& c, const int32_t* cl,
                                    const float* s, int32_t* idx, float* lse_s, uint16_t* o, float* lse_o, int* err,
                                    cudaStream_t st) {
  Kv4DecodeArgs a = kv4_decode_args(sh, q, c, cl, s, err);
  a.idx_out = idx;
  a.lse_s_out = lse_s;
  a.o = o;
  a.lse_o = lse_o;
  // blocks of a row that the selecting warp's registers hold
  if (sh.NB <= 4 * 32) return sh.d == 128 ? launch_fused<128, 4>(a, sh.outside, st) : launch_fused<64, 4>(a, sh.outside, st);
  if (sh.NB <= 16 * 32) return sh.d == 128 ? launch_fused<128, 16>(a, sh.outside, st) : launch_fused<64, 16>(a, sh.outside, st);
  return sh.d == 128 ? launch_fused<128, 64>(a, sh.outside, st) : launch_fused<64, 64>(a, sh.outside, st);
}

}  // namespace sas
