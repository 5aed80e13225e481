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

#include "decode_select.cuh"
#include "kv4.cuh"

namespace sas {

namespace cg = cooperative_groups;
using namespace kv4;

namespace {

constexpr int kWarps = dec::kThreads / 32;  // warps of a fused CTA
constexpr int kSplitWarps = 4;              // warps of a split CTA
constexpr int kSlots = 2;                   // record slots of a warp's ring
constexpr int kMaxTasks = 256;      // blocks of one CTA's list (fused: the whole list of a row)
constexpr float kPShift = 8.f;      // P is kept times 2^8
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
  int B, Hkv, G, Lmax, K, gate, gated, outside, need_lse, n_split;
  float scale;
};

__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_zero(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
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
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d;}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5};\n"
      "add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float exp2_approx(float x) {  // 2^x, relative error about 2^-22, 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
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

  __device__ __forceinline__ void load(const uint16_t* q, int G, float scale) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint4 x[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j)
      x[j] = g < G ? *reinterpret_cast<const uint4*>(q + g * D + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
    uint32_t mx = 0;  // largest magnitude, as bf16 bits
#pragma unroll
    for (int j = 0; j < NG; ++j)
      mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x[j].x & 0x7fff7fffu, x[j].y & 0x7fff7fffu),
                                 __vmaxu2(x[j].z & 0x7fff7fffu, x[j].w & 0x7fff7fffu)));
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // exponent of the largest; a row of zeros or subnormals uses the smallest normal's
    const int e = min(max(int(mx >> 7), 1), 254) - 127;
    float part[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      float v[8];
      float sm = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // 2^(15 - e) in two factors, neither of which leaves fp32's range
        v[2 * i] = lo_bf16(w[i]) * ldexpf(1.f, -e) * 32768.f;
        v[2 * i + 1] = hi_bf16(w[i]) * ldexpf(1.f, -e) * 32768.f;
        sm += v[2 * i] + v[2 * i + 1];
      }
      b[j][0][0] = pack_f16x2(v[0], v[4]);
      b[j][0][1] = pack_f16x2(v[1] * 0.0625f, v[5] * 0.0625f);
      b[j][1][0] = pack_f16x2(v[2], v[6]);
      b[j][1][1] = pack_f16x2(v[3] * 0.0625f, v[7] * 0.0625f);
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
    f = make_float2(c * ldexpf(1.f, min(e0, 100)), c * ldexpf(1.f, min(e1, 100)));
    over = make_float2(ldexpf(1.f, max(e0 - 100, 0)), ldexpf(1.f, max(e1 - 100, 0)));
    big = __any_sync(0xffffffffu, e > 100);
  }
};

// A warp's running state. Rows of `acc` are channels: acc[j][i] holds channels
// 32 j + 4 g + 2 i (elements 0, 1) and + 1 (elements 2, 3, times 2^4) of heads
// 2t (even elements) and 2t + 1.
template <int D>
struct State {
  static constexpr int NG = D / kGroup;
  float acc[NG][2][4];
  float2 accm[NG];    // Σ p m over this lane's tokens, heads 2t and 2t + 1
  float m[2], l[2];   // maximum (log2), and Σ p 2^8 over this lane's tokens
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
    lo = lim = 0u;
  }
};

// S of a block's 64 tokens from its K record. With FULL, all of them count;
// otherwise those past ntok become -inf.
template <int D, bool FULL>
__device__ __forceinline__ void score_block(const uint8_t* rec, const Query<D>& q, int ntok, float2 (&S)[kTiles][2]) {
  using F = Fmt<D>;
  constexpr int NG = F::NG;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
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

// The online softmax: S becomes p · 2^8 with p = 2^(S f + lam - max), and the
// state is rescaled. (f > 0, so the largest logit is that of the largest S.)
template <int D>
__device__ __forceinline__ void softmax_block(State<D>& st, const Query<D>& q, float lam, float2 (&S)[kTiles][2]) {
  float top[2], sub[2], al[2];
  top[0] = fmaxf(S[0][0].x, S[0][1].x);
  top[1] = fmaxf(S[0][0].y, S[0][1].y);
#pragma unroll
  for (int i = 1; i < kTiles; ++i) {
    top[0] = fmaxf(top[0], fmaxf(S[i][0].x, S[i][1].x));
    top[1] = fmaxf(top[1], fmaxf(S[i][0].y, S[i][1].y));
  }
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) {
    top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
    top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float mx = fmaxf(st.m[h], fmaf(top[h], h ? q.f.y : q.f.x, lam));
    const float ref = mx == -INFINITY ? 0.f : mx;  // nothing but masked tokens so far: every p is 0
    al[h] = exp2_approx(st.m[h] - ref);
    sub[h] = lam - ref + kPShift;
    st.m[h] = mx;
  }
  const float2 add = make_float2(sub[0], sub[1]);
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float2 z = fma_f32x2(S[i][u], q.f, add);
      z.x = exp2_approx(z.x);
      z.y = exp2_approx(z.y);
      S[i][u] = z;
      sum = add_f32x2(sum, z);
    }
  st.l[0] = fmaf(st.l[0], al[0], sum.x);
  st.l[1] = fmaf(st.l[1], al[1], sum.y);
  if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
    for (int j = 0; j < State<D>::NG; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        st.acc[j][0][e] *= al[e & 1];
        st.acc[j][1][e] *= al[e & 1];
      }
      st.accm[j].x *= al[0];
      st.accm[j].y *= al[1];
    }
  }
}

// O += P V from the block's V record.
template <int D, bool FULL>
__device__ __forceinline__ void value_block(const uint8_t* rec, State<D>& st, int ntok, const float2 (&p)[kTiles][2]) {
  using F = Fmt<D>;
  constexpr int NG = F::NG;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
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
    const uint32_t p0 = transpose8x8(pack_f16x2(p[i][0].x, p[i][0].y)), p1 = transpose8x8(pack_f16x2(p[i][1].x, p[i][1].y));
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

// A warp's ring of records. Item 2 i is block i's K, item 2 i + 1 its V; an
// item's slot is refilled as soon as it has been used.
template <int D>
__device__ __forceinline__ void ring_issue(uint8_t* ring, const Cache& c, int item, int slot, int rec, int ntok) {
  using F = Fmt<D>;
  const int lane = threadIdx.x & 31;
  const uint8_t* src = ((item & 1) ? c.v : c.k) + size_t(rec) * F::kRecord + lane * 16;
  const uint32_t dst = smem_u32(ring) + slot * F::kRecord + lane * 16;
  if (ntok == kBlock) {
#pragma unroll
    for (int o = 0; o < F::kRecord; o += 512) cp_async16(dst + o, src + o);
  } else {  // the tiles that hold tokens
    const int bytes = (ntok + kTile - 1) / kTile * F::kTileBytes;
#pragma unroll 1
    for (int o = 0; o + lane * 16 < bytes; o += 512) cp_async16(dst + o, src + o);
  }
}

// Runs a warp over blocks first, first + W, ... < n of its CTA's list
// (records rec_s, -1 for a block that is left out; gates lam_s). The item
// numbered `issued` is the first that is not yet under way.
template <int D, int W>
__device__ __forceinline__ void run_blocks(const Kv4DecodeArgs& a, State<D>& st, const Query<D>& q, uint8_t* ring,
                                           const int* rec_s, const float* lam_s, int first, int n, int cur_at,
                                           int cur_ntok, int issued) {
  const int mine = n > first ? (n - 1 - first) / W + 1 : 0;
  auto issue = [&](int item, int slot) {
    if (item < 2 * mine) {
      const int at = first + (item >> 1) * W;
      const int rec = rec_s[at];
      if (rec >= 0) ring_issue<D>(ring, a.c, item, slot, rec, at == cur_at ? cur_ntok : kBlock);
    }
    cp_async_commit();
  };
  for (int k = issued; k < kSlots; ++k) issue(k, k);
  int slot = 0;
  auto next = [&] {
    slot = slot + 1 == kSlots ? 0 : slot + 1;
  };
  for (int i = 0; i < mine; ++i) {
    const int at = first + i * W;
    const int ntok = rec_s[at] < 0 ? 0 : at == cur_at ? cur_ntok : kBlock;
    const float lam = lam_s[at];
    float2 S[kTiles][2];
    cp_async_wait<kSlots - 1>();
    __syncwarp();
    const uint8_t* rec = ring + slot * Fmt<D>::kRecord;
    if (ntok == kBlock)
      score_block<D, true>(rec, q, ntok, S);
    else
      score_block<D, false>(rec, q, ntok, S);
    __syncwarp();
    issue(2 * i + kSlots, slot);
    next();
    softmax_block<D>(st, q, a.outside ? 0.f : lam, S);
    if (a.outside) {
      const float gw = exp2f(lam);
#pragma unroll
      for (int k = 0; k < kTiles; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u) S[k][u] = make_float2(S[k][u].x * gw, S[k][u].y * gw);
    }
    cp_async_wait<kSlots - 1>();
    __syncwarp();
    rec = ring + slot * Fmt<D>::kRecord;
    if (ntok == kBlock)
      value_block<D, true>(rec, st, ntok, S);
    else
      value_block<D, false>(rec, st, ntok, S);
    __syncwarp();
    issue(2 * i + 1 + kSlots, slot);
    next();
  }
  cp_async_wait<0>();
}

// A warp's partial in shared memory: per head D normalised outputs, then the
// maximum and the sum.
template <int D>
struct Partial {
  float o[8][D];
  float m[8], l[8];
};

template <int D>
__device__ __forceinline__ void store_partial(const State<D>& st, Partial<D>* out) {
  constexpr int NG = D / kGroup;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float f = exp2f(float(int((st.lo & 0xffffu) >> 7) - 112));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float l = st.l[h];
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      float am = h ? st.accm[j].y : st.accm[j].x;
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) am += __shfl_xor_sync(0xffffffffu, am, o);
      am *= inv;
      float4 v;
      v.x = fmaf(st.acc[j][0][h] * (inv * 16777216.f), f, am);
      v.y = fmaf(st.acc[j][0][2 + h] * (inv * 1048576.f), f, am);
      v.z = fmaf(st.acc[j][1][h] * (inv * 16777216.f), f, am);
      v.w = fmaf(st.acc[j][1][2 + h] * (inv * 1048576.f), f, am);
      *reinterpret_cast<float4*>(&out->o[2 * t + h][32 * j + 4 * g]) = v;
    }
    if (g == 0) {
      out->m[2 * t + h] = st.m[h];
      out->l[2 * t + h] = l;
    }
  }
}

// Output `col`, `col` + 1 of head g, merged from n partials. A row whose sum is
// NaN in any of them is NaN. Returns the sum relative to M (times 2^8).
template <int D, typename At>
__device__ __forceinline__ float merge_partials(At at, int n, int g, int col, float2& o, float& M) {
  M = -INFINITY;
  for (int r = 0; r < n; ++r) M = fmaxf(M, at(r)->m[g]);
  const float ref = M == -INFINITY ? 0.f : M;
  float den = 0.f;
  o = make_float2(0.f, 0.f);
  for (int r = 0; r < n; ++r) {
    const Partial<D>* p = at(r);
    const float l = p->l[g];
    const float w = l == 0.f ? 0.f : l * exp2f(p->m[g] - ref);
    const float2 v = *reinterpret_cast<const float2*>(&p->o[g][col]);
    den += w;
    o.x = l == 0.f ? o.x : fmaf(w, v.x, o.x);
    o.y = l == 0.f ? o.y : fmaf(w, v.y, o.y);
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  o.x *= inv;
  o.y *= inv;
  return den;
}
__device__ __forceinline__ float lse_of(float M, float den) {
  return den == 0.f ? -INFINITY : (M + log2f(den) - kPShift) * kLn2;
}

// Dynamic shared memory of a CTA of W warps: the rings, and the partials in their place.
template <int D, int W>
constexpr int smem_bytes() {
  constexpr int ring = W * kSlots * Fmt<D>::kRecord, part = W * int(sizeof(Partial<D>));
  return ring > part ? ring : part;
}

}  // namespace

// One CTA per (sequence, KV head, split), or a cluster of CS (CLUSTER) whose
// CTAs take every CS-th block of the split's run.
template <int D, bool CLUSTER>
__global__ void __launch_bounds__(32 * kSplitWarps, 16 / kSplitWarps) kv4_decode_split_kernel(Kv4DecodeArgs a) {
  using F = Fmt<D>;
  constexpr int W = kSplitWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int rec_s[kMaxDecodeBlocksPerSplit];
  __shared__ float lam_s[kMaxDecodeBlocksPerSplit];
  const int CS = CLUSTER ? int(cg::this_cluster().num_blocks()) : 1;
  const int rank = CLUSTER ? int(cg::this_cluster().block_rank()) : 0;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int item = blockIdx.x / CS, split = item % a.n_split, bh = item / a.n_split, b = bh / a.Hkv, h = bh % a.Hkv;
  const int NB = a.Lmax / kBlock;
  uint8_t* ring = smem + warp * kSlots * F::kRecord;
  griddep_launch_dependents();  // the merge kernel may begin its launch; it waits for this grid's writes
  griddep_wait();               // idx and lse_s come from the select kernel that precedes this one
  int L = a.cache_len[b];
  if (L < 1 || L > a.Lmax) {
    if (tid == 0) raise_error(a.err, SAS_ERR_DEVICE_INDEX);
    L = max(1, min(L, a.Lmax));
  }
  const int c = (L - 1) / kBlock, nl = 1 + min(a.K, c);
  const int per = (nl + a.n_split - 1) / a.n_split;
  const int lo = min(split * per, nl), n = min(lo + per, nl) - lo;
  const int nt = rank < n ? (n - 1 - rank) / CS + 1 : 0;
  if (tid < nt) {
    const int pos = lo + tid * CS + rank;
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
    rec_s[tid] = rec;
    lam_s[tid] = rec < 0 ? 0.f : lam;
  }
  Query<D> q;
  q.load(a.q + size_t(bh) * a.G * D, a.G, a.scale);
  State<D> st;
  st.clear();
  __syncthreads();
  run_blocks<D, W>(a, st, q, ring, rec_s, lam_s, warp, nt, lo == 0 && rank == 0 ? 0 : -1, L - c * kBlock, 0);
  __syncthreads();  // the rings are done with
  Partial<D>* part = reinterpret_cast<Partial<D>*>(smem);
  store_partial<D>(st, part + warp);
  if (CLUSTER)
    cg::this_cluster().sync();  // every partial of the cluster is in place
  else
    __syncthreads();
  for (int e = rank * 32 * W + tid; e < a.G * D / 2; e += CS * 32 * W) {
    const int g = 2 * e / D, col = 2 * e % D;
    float2 o;
    float M;
    const float den = merge_partials<D>(
        [&](int r) { return CLUSTER ? cg::this_cluster().map_shared_rank(part, r / W) + r % W : part + r; }, CS * W, g,
        col, o, M);
    const size_t row = (size_t(bh) * a.G + g) * a.n_split + split;
    *reinterpret_cast<float2*>(a.o_part + row * D + col) = o;
    if (col == 0) a.lse_part[row] = lse_of(M, den);
  }
  if (CLUSTER) cg::this_cluster().sync();  // no CTA leaves while another may still read its partials
}

// One cluster per (sequence, KV head): each CTA selects the row's blocks
// itself and takes every CS-th one.
template <int D>
__global__ void __launch_bounds__(dec::kThreads, 3) kv4_decode_fused_kernel(Kv4DecodeArgs a) {
  using F = Fmt<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int sel_s[dec::kFusedMaxK];
  __shared__ int rec_s[kMaxTasks];
  __shared__ float lam_s[kMaxTasks];
  __shared__ int xch_s[4], wtot_s[kWarps], napp_s;
  __shared__ float redf_s[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = int(blockIdx.x) / CS, b = bh / a.Hkv, h = bh % a.Hkv;
  const int NB = a.Lmax / kBlock;
  uint8_t* ring = smem + warp * kSlots * F::kRecord;
  // the keys lie in the rings of warps 1 to 3, behind warp 0's, which starts on the current block at once
  static_assert((kWarps - 1) * kSlots * F::kRecord >= dec::kFusedMaxNB * 4 + 768 * 4, "keys, histogram, picks, candidates");
  uint32_t* key_s = reinterpret_cast<uint32_t*>(smem + kSlots * F::kRecord);
  int* hist_s = reinterpret_cast<int*>(key_s + dec::kFusedMaxNB);
  int* app_s = hist_s + 256;
  uint32_t* cand_k = reinterpret_cast<uint32_t*>(app_s + 256);
  int* cand_m = app_s + 384;
  griddep_launch_dependents();
  if (tid == 0) napp_s = 0;
  griddep_wait();
  // the row's scores are read while the cache length is still in flight
  const float* srow = a.s + size_t(bh) * NB;
  for (int m = tid; m < NB - 1; m += dec::kThreads) key_s[m] = __float_as_uint(__ldg(srow + m));
  int L = a.cache_len[b];
  if (L < 1 || L > a.Lmax) {
    if (tid == 0) raise_error(a.err, SAS_ERR_DEVICE_INDEX);
    L = max(1, min(L, a.Lmax));
  }
  const int c = (L - 1) / kBlock, n = min(a.K, c), nl = 1 + n;
  const int nt = rank < nl ? (nl - 1 - rank) / CS + 1 : 0;  // list positions rank, rank + CS, ...
  int issued = 0;
  if (rank == 0 && warp == 0) {  // the current block needs no selection
    const int rec = record_of(a.c, b, h, c, a.Hkv, NB, a.err);
    if (lane == 0) {
      rec_s[0] = rec;
      lam_s[0] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (rec >= 0) ring_issue<D>(ring, a.c, k, k, rec, L - c * kBlock);
      cp_async_commit();
    }
    issued = 2;
  }
  float mx = -INFINITY;
  for (int m = tid; m < c; m += dec::kThreads) {  // each thread converts the scores it read
    const float v = __uint_as_float(key_s[m]);
    key_s[m] = score_key(v) + 1u;  // >= 1, so the threshold 1 takes every block
    mx = fmaxf(mx, v);
  }
  Query<D> q;
  q.load(a.q + size_t(bh) * a.G * D, a.G, a.scale);
  float lse = 0.f;
  if (a.need_lse) {  // LSE of the history scores, as the select kernels take it
    mx = warp_max(mx);
    if (lane == 0) redf_s[warp] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(redf_s[0], redf_s[1]), fmaxf(redf_s[2], redf_s[3]));
    __syncthreads();
    float sum = 0.f;
    if (mx != -INFINITY)
      for (int m = tid; m < c; m += dec::kThreads) sum += expf(__ldg(srow + m) - mx);
    sum = warp_sum(sum);
    if (lane == 0) redf_s[warp] = sum;
    __syncthreads();
    const float tot = (redf_s[0] + redf_s[1]) + (redf_s[2] + redf_s[3]);
    lse = (c == 0 || mx == -INFINITY) ? -INFINITY : mx + logf(tot);
  }
  __syncthreads();  // every key is in place
  int32_t* idx_row = (rank == 0 && a.idx_out != nullptr) ? a.idx_out + size_t(bh) * a.K : nullptr;
  // list position pos holds block m: this CTA's task, if it is
  auto place = [&](int pos, int m) {
    if (idx_row != nullptr) idx_row[pos - 1] = m;
    if (pos % CS == rank) {
      const int rec = record_of(a.c, b, h, m, a.Hkv, NB, a.err);
      rec_s[pos / CS] = rec;
      lam_s[pos / CS] = a.gated && rec >= 0 ? gate_lam2(a.gate, __ldg(srow + m), lse) : 0.f;
    }
  };
  if (n == c) {
    for (int m = tid; m < c; m += dec::kThreads) place(m + 1, m);
  } else {
    uint32_t thr = 1u;
    int need_eq = 0;
    if (!cta_select(key_s, c, n, hist_s, xch_s, app_s, &napp_s, cand_k, cand_m, &xch_s[3], thr, need_eq)) {
      __syncthreads();
      for (int i = tid; i < n; i += dec::kThreads) {
        const int v = app_s[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += app_s[j] < v ? 1 : 0;
        place(r + 1, v);
      }
    } else {
      // ties cut at the threshold, taken from the lowest block index: each thread
      // owns a contiguous run of blocks, and two block-wide scans place the picks
      const int per = (c + dec::kThreads - 1) / dec::kThreads;
      const int lo = min(c, tid * per), hi = min(c, lo + per);
      int eq = 0, tot = 0, take = 0;
      for (int m = lo; m < hi; ++m) eq += key_s[m] == thr ? 1 : 0;
      const int eq0 = cta_excl_sum(eq, wtot_s, tot);
      for (int m = lo, e = eq0; m < hi; ++m) {
        const bool is_eq = key_s[m] == thr;
        take += (key_s[m] > thr || (is_eq && e < need_eq)) ? 1 : 0;
        e += is_eq ? 1 : 0;
      }
      int pos = cta_excl_sum(take, wtot_s, tot);
      for (int m = lo, e = eq0; m < hi; ++m) {
        const bool is_eq = key_s[m] == thr;
        if (key_s[m] > thr || (is_eq && e < need_eq)) place(++pos, m);
        e += is_eq ? 1 : 0;
      }
    }
  }
  if (idx_row != nullptr)
    for (int i = n + tid; i < a.K; i += dec::kThreads) idx_row[i] = -1;
  if (rank == 0 && a.lse_s_out != nullptr && tid == 0) a.lse_s_out[bh] = lse;
  __syncthreads();  // the tasks are placed, and the keys' rings are free
  State<D> st;
  st.clear();
  run_blocks<D, kWarps>(a, st, q, ring, rec_s, lam_s, warp, nt, rank == 0 ? 0 : -1, L - c * kBlock, issued);
  __syncthreads();  // the rings are done with
  Partial<D>* part = reinterpret_cast<Partial<D>*>(smem);
  store_partial<D>(st, part + warp);
  cluster.sync();  // every partial of the cluster is in place
  for (int e = rank * dec::kThreads + tid; e < a.G * D / 2; e += CS * dec::kThreads) {
    const int g = 2 * e / D, col = 2 * e % D;
    float2 o;
    float M;
    const float den = merge_partials<D>(
        [&](int r) { return cluster.map_shared_rank(part, r / kWarps) + r % kWarps; }, CS * kWarps, g, col, o, M);
    const size_t row = size_t(bh) * a.G + g;
    *reinterpret_cast<uint32_t*>(a.o + row * D + col) = pack_bf16x2(o.x, o.y);
    if (col == 0 && a.lse_o != nullptr) a.lse_o[row] = lse_of(M, den);
  }
  cluster.sync();  // no CTA leaves while another may still read its partials
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
  a.outside = sh.outside;
  a.scale = sh.scale;
  return a;
}

// Launches `kern` on `items` clusters of cs CTAs, as a dependent launch.
static cudaError_t launch_clusters(void (*kern)(Kv4DecodeArgs), int items, int cs, int threads, int smem, cudaStream_t st,
                                   const Kv4DecodeArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(items) * cs);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

static cudaError_t multiprocessors(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// Split form. The cluster size: the largest power of two that keeps every CTA
// resident at once (16 warps per SM), at most 8 and at most half the blocks of
// a split.
template <int D>
static cudaError_t launch_split(const Kv4DecodeArgs& a, cudaStream_t st) {
  constexpr int W = kSplitWarps, smem = smem_bytes<D, W>();
  static_assert(smem <= 48 * 1024, "no opt-in needed");
  int sms = 0;
  const cudaError_t e = multiprocessors(&sms);
  if (e != cudaSuccess) return e;
  const int items = a.B * a.Hkv * a.n_split, per = (a.K + a.n_split) / a.n_split;
  const int want = min(min(dec::kMaxCluster, (per + W - 1) / W), sms * (16 / W) / items);
  int cs = 1;
  while (cs * 2 <= want) cs *= 2;
  if (cs == 1) return launch_pdl(kv4_decode_split_kernel<D, false>, dim3(items), dim3(32 * W), smem, st, a);
  return launch_clusters(kv4_decode_split_kernel<D, true>, items, cs, 32 * W, smem, st, a);
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
  const cudaError_t e = sh.d == 128 ? launch_split<128>(a, st) : launch_split<64>(a, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The cluster size: as many CTAs per row as keep the grid in one wave of
// resident CTAs, at most 8 and at most one per block of the list.
template <int D>
static cudaError_t launch_fused(const Kv4DecodeArgs& a, cudaStream_t st) {
  constexpr int smem = smem_bytes<D, kWarps>();
  static_assert(smem <= 48 * 1024, "no opt-in needed");
  int sms = 0;
  const cudaError_t e = multiprocessors(&sms);
  if (e != cudaSuccess) return e;
  const int rows = a.B * a.Hkv;
  const int cs = max(1, min(min(dec::kMaxCluster, a.K + 1), sms * 3 / rows));
  return launch_clusters(kv4_decode_fused_kernel<D>, rows, cs, dec::kThreads, smem, st, a);
}

cudaError_t launch_decode_fused_kv4(const Shape& sh, const uint16_t* q, const Cache& c, const int32_t* cl,
                                    const float* s, int32_t* idx, float* lse_s, uint16_t* o, float* lse_o, int* err,
                                    cudaStream_t st) {
  Kv4DecodeArgs a = kv4_decode_args(sh, q, c, cl, s, err);
  a.idx_out = idx;
  a.lse_s_out = lse_s;
  a.o = o;
  a.lse_o = lse_o;
  a.need_lse = (lse_s != nullptr || sh.gate == SAS_GATE_LOG_SOFTMAX || sh.gate == SAS_GATE_SOFTMAX_OUTSIDE) ? 1 : 0;
  const cudaError_t e = sh.d == 128 ? launch_fused<128>(a, st) : launch_fused<64>(a, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sas
