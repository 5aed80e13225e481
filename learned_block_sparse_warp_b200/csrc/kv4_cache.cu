// Writing the 4-bit KV cache, reading it back, and its block-mean keys.
//
// Write: a group of 32 channels x has minimum m and step
//   s = bf16((max − min) / 15),  code = floor((x − m) / s + 1/2),
// so that s·code + m is within s/2 of x ((max − m)/s is at most 15 (1 + 2^-8)).
// A step below 2^-126 is stored as 0 and every code with it. A group whose
// range is not a finite fp32 (a NaN, an infinity, or a range above the largest
// float) is stored as s = 0, m = NaN: it reads back as NaN, and attention rows
// that reach it become NaN.
//
// Read: bf16(s·code + m), one rounding. Means: Σ s·(code/64) + Σ m/64 in fp32.
//
// The read is bound by the bytes it moves. Write and means are bound by nothing
// alone: their integer instructions and the wait for their loads share the time
// (the figures are at the kernels). Write and read give a tile of 16 tokens to a warp, the means a
// record: enough independent 16-byte loads per lane that the few dependent ones
// before them (length, page) are hidden by the multiprocessor's other warps.
#include "kv4.cuh"

namespace sas {

using namespace kv4;

struct Kv4Args {
  Cache c;
  const int32_t* cache_len;
  const int32_t* new_len;  // null: n_tokens for every sequence
  int n_tokens, B, Hkv, Lmax;
  int* err;
};

// One group's parameters and the codes of this lane's two 8-channel chunks.
struct Quant16 {
  uint32_t word[2];  // nibble p: code of the chunk's channel p
  uint16_t s, m;     // bf16
};

__device__ __forceinline__ float2 dup2(float x) { return make_float2(x, x); }

__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two neighbouring lanes hold a group, 16 bf16 channels each. Every lane of the
// warp takes part. Sixteen channels a lane rather than eight, because the
// group's parameters cost as much as eight of its codes, and the arithmetic is
// most of a long write's instructions.
//
// The quotient (x − m)/s is formed as (x − m)·r with r = 1/s raised by 2^-20,
// which outweighs the reciprocal's error: a value half-way between two levels
// goes up, as in the definition. fma adds 1.5·2^23, so the code is in the low
// bits, rounded once. A value just under half-way may have gone up with them:
// its residue x − m − s·code is below −s/2, and such a code is taken down.
// x − m and the residue are rounded down. What they are compared with, half an
// odd multiple of s, is an fp32 number, so a difference that is not one (of
// values of very different sizes) stays on its side of it, and the codes are
// those of the exact x − m.
__device__ __forceinline__ Quant16 quantise16(const uint4 (&x)[2]) {
  constexpr float kMagic = 12582912.f;
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  __nv_bfloat162 mx = *reinterpret_cast<const __nv_bfloat162*>(&w[0]), mn = mx;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
    mx = __hmax2_nan(mx, v);
    mn = __hmin2_nan(mn, v);
  }
  // (max, −min) in one register: one shuffle serves both
  const uint32_t mxb = *reinterpret_cast<const uint32_t*>(&mx), mnb = *reinterpret_cast<const uint32_t*>(&mn) ^ 0x80008000u;
  const uint32_t lo2 = __byte_perm(mxb, mnb, 0x5410), hi2 = __byte_perm(mxb, mnb, 0x7632);
  __nv_bfloat162 e = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&lo2), *reinterpret_cast<const __nv_bfloat162*>(&hi2));
  uint32_t eb = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&e), 1);
  e = __hmax2_nan(e, *reinterpret_cast<const __nv_bfloat162*>(&eb));
  eb = *reinterpret_cast<const uint32_t*>(&e);
  const float hi = __uint_as_float(eb << 16), neg_lo = __uint_as_float(eb & 0xffff0000u);
  const float range = __fadd_rn(hi, neg_lo);
  const bool bad = !(range <= 3.402823466e38f);
  // range / 15, correctly rounded: the product with 1/15 is within an ulp, and a
  // step by its residue (Markstein 1990) rounds it while the residue is a normal
  // number
  float quot = __fmul_rn(range, 0.0666666701436042785644531f);
  quot = fmaf(fmaf(-15.f, quot, range), 0.0666666701436042785644531f, quot);
  if (range < 1e-25f) quot = __fdiv_rn(range, 15.f);
  const uint16_t sb = __bfloat16_as_ushort(__float2bfloat16_rn(quot));
  const bool flat = bad || sb < 0x80u;  // a step below 2^-126, or no range
  const float s = flat ? 0.f : bf16_to_f32(sb);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(s));
  r = flat ? 0.f : __fmul_rn(r, 1.00000095367431640625f);
  float least = 0.f;
  Quant16 q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t word = 0;
#pragma unroll
    for (int i = 4 * h + 3; i >= 4 * h; --i) {
      const float2 d = add_down_f32x2(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), dup2(neg_lo));
      const float2 c = fma_f32x2(d, dup2(r), dup2(kMagic));
      const float2 rest = fma_down_f32x2(add_f32x2(c, dup2(-kMagic)), dup2(-s), d);
      least = min3(least, rest.x, rest.y);
      word = word * 16u + __float_as_uint(c.y);
      word = word * 16u + __float_as_uint(c.x);
    }
    q.word[h] = word - 0x3f400000u;  // less what the eight 1.5·2^23 leave in it
  }
  if (least < -0.5f * s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t word = 0;
#pragma unroll
      for (int i = 4 * h + 3; i >= 4 * h; --i)
#pragma unroll
        for (int e = 1; e >= 0; --e) {
          const float d = __fadd_rd(__uint_as_float(e ? w[i] & 0xffff0000u : w[i] << 16), neg_lo);
          const float n = fmaf(d, r, kMagic) - kMagic;
          word = (word << 4) | (uint32_t(n) - (__fmaf_rd(n, -s, d) < -0.5f * s ? 1u : 0u));
        }
      q.word[h] = word;
    }
  }
  if (bad) q.word[0] = q.word[1] = 0u;
  q.s = flat ? uint16_t(0) : sb;
  const uint16_t mb = uint16_t(eb >> 16) ^ uint16_t(0x8000);
  q.m = bad ? uint16_t(0x7fc0u) : mb == 0x8000u ? uint16_t(0) : mb;  // −0 becomes +0
  return q;
}

// The tile of a warp: block m of sequence b and head h, and which of its 16
// tokens [r0, r1) are new. i0 is the row of k and v that token 0 of the tile
// would have.
struct Tile {
  int b, h, m, in_block, r0, r1, i0;
};

// Warp `item` of [bh][tile]. False where the window has no such tile.
__device__ __forceinline__ bool tile_of(const Kv4Args& a, unsigned item, unsigned per, Tile* t) {
  const unsigned bh = item / per;
  if (bh >= unsigned(a.B) * a.Hkv) return false;
  t->b = int(bh / a.Hkv);
  t->h = int(bh % a.Hkv);
  const Window w = window_of(a.cache_len, a.new_len, t->b, a.n_tokens, a.Lmax, a.err);
  const int tile = w.pos / kTile + int(item % per), first = tile * kTile;
  t->m = tile / kTiles;
  t->in_block = tile % kTiles;
  t->i0 = first - w.pos;
  t->r0 = max(-t->i0, 0);
  t->r1 = min(w.n - t->i0, kTile);
  return t->r0 < t->r1;
}

// 16-byte unit of a V tile's codes in the staging buffer: unit (u, g, t) holds
// the groups of one token pair. The order keeps the stores of one token pair in
// different banks.
template <int D>
__device__ __forceinline__ int stage_unit(int unit) {
  return D == 128 && unit < 64 ? unit ^ ((unit >> 3) & 3) : unit;
}

// Warps of a write CTA. The bound of 28 warps per multiprocessor (72 registers)
// measures best: writing 32K tokens and reading them back takes 56 us with it,
// 68 at the 91 registers of the unbounded kernel. The write alone takes 34 us,
// 5.2 TB/s, 0.79 of a copy's rate. Of what it does the integer pipe is busiest,
// at 66 % of its rate, 69 % of the cycles issue, and the loads of a tile are the
// largest stall.
constexpr int kWriteWarps = 4;

// A token's codes, step and minimum to their places in a tile in global memory.
template <int D>
__device__ __forceinline__ void store_token(uint8_t* tile, bool is_v, int r, int j, int hq, const Quant16& g) {
  using F = Fmt<D>;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int q = hq + 2 * u;
    if (is_v) {
      *reinterpret_cast<uint16_t*>(tile + F::v_half(r, 2 * q, j)) = uint16_t(g.word[u]);
      *reinterpret_cast<uint16_t*>(tile + F::v_half(r, 2 * q + 1, j)) = uint16_t(g.word[u] >> 16);
    } else {
      *reinterpret_cast<uint32_t*>(tile + F::k_word(r, q, j)) = g.word[u];
    }
  }
  if (hq == 0) {
    *reinterpret_cast<uint16_t*>(tile + (is_v ? F::v_step(r, j) : F::k_step(r, j))) = g.s;
    *reinterpret_cast<uint16_t*>(tile + F::min_at(r, j)) = g.m;
  }
}

// A warp per tile; blockIdx.y is 0 for K and 1 for V. D/16 lanes hold a token:
// lane (j, hq) has the chunks hq and hq + 2 of group j's four, so that each
// load fills 32-byte sectors.
template <int D>
__global__ void __launch_bounds__(32 * kWriteWarps, 28 / kWriteWarps) kv4_write_kernel(Kv4Args a, unsigned per, const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v) {
  using F = Fmt<D>;
  constexpr int LPR = D / 16, TPI = 32 / LPR, NI = kTile / TPI;
  __shared__ __align__(16) uint8_t stage_s[kWriteWarps][F::kTileBytes];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_v = blockIdx.y != 0;
  Tile t;
  if (!tile_of(a, blockIdx.x * (kWriteWarps) + warp, per, &t)) return;
  const int j = lane % LPR >> 1, hq = lane & 1, at = lane / LPR;
  const uint16_t* src = (is_v ? v : k) + (int64_t(t.b * a.Hkv + t.h) * a.n_tokens + t.i0) * D + 32 * j + 8 * hq;
  uint4 x[NI][2];
  if (t.r1 - t.r0 < kTile) {  // a part of the tile: the other tokens' bits stay as they are
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = i * TPI + at;
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (r >= t.r0 && r < t.r1) {
        x[i][0] = __ldcs(reinterpret_cast<const uint4*>(src + int64_t(r) * D));
        x[i][1] = __ldcs(reinterpret_cast<const uint4*>(src + int64_t(r) * D + 16));
      }
    }
    const int rec = record_of(a.c, t.b, t.h, t.m, a.Hkv, a.Lmax / kBlock, a.err);
    if (rec < 0) return;
    uint8_t* tile = (is_v ? a.c.v : a.c.k) + size_t(rec) * F::kRecord + t.in_block * F::kTileBytes;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (i * TPI + TPI <= t.r0 || i * TPI >= t.r1) continue;
      const Quant16 g = quantise16(x[i]);
      const int r = i * TPI + at;
      if (r >= t.r0 && r < t.r1) store_token<D>(tile, is_v, r, j, hq, g);
    }
    return;
  }
  src += at * D;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    x[i][0] = __ldcs(reinterpret_cast<const uint4*>(src + i * TPI * D));
    x[i][1] = __ldcs(reinterpret_cast<const uint4*>(src + i * TPI * D + 16));
  }
  const int rec = record_of(a.c, t.b, t.h, t.m, a.Hkv, a.Lmax / kBlock, a.err);
  if (rec < 0) return;
  uint8_t* tile = (is_v ? a.c.v : a.c.k) + size_t(rec) * F::kRecord + t.in_block * F::kTileBytes;
  // the whole tile: staged, so that it leaves in 16-byte stores
  uint8_t* stage = stage_s[warp];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = i * TPI + at;
    const Quant16 g = quantise16(x[i]);
    if (is_v) {  // a word holds two tokens: the even one's lane puts together the first chunk's, the odd one's the second's
      const bool odd = (r & 1) != 0;
      const uint32_t own = odd ? g.word[1] : g.word[0];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? g.word[0] : g.word[1], LPR);
      const uint32_t a0 = odd ? got : own, a1 = odd ? own : got;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int to = F::v_half(r & ~1, 2 * hq + 4 * (r & 1) + u, j);
        *reinterpret_cast<uint32_t*>(stage + stage_unit<D>(to >> 4) * 16 + (to & 15)) = __byte_perm(a0, a1, u ? 0x7632 : 0x5410);
      }
    } else {
      *reinterpret_cast<uint32_t*>(stage + F::k_word(r, hq, j)) = g.word[0];
      *reinterpret_cast<uint32_t*>(stage + F::k_word(r, hq + 2, j)) = g.word[1];
    }
    if (hq == 0) {
      *reinterpret_cast<uint16_t*>(stage + (is_v ? F::v_step(r, j) : F::k_step(r, j))) = g.s;
      *reinterpret_cast<uint16_t*>(stage + F::min_at(r, j)) = g.m;
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < (F::kTileBytes + 511) / 512; ++i) {
    const int unit = i * 32 + lane;
    if (unit < F::kTileBytes / 16)
      *reinterpret_cast<uint4*>(tile + unit * 16) =
          *reinterpret_cast<const uint4*>(stage + (is_v ? stage_unit<D>(unit) : unit) * 16);
  }
}

// Four registers (nibbles i and i + 4 of a word) as bf16 s·code + m: 128 + code
// is the bf16 with the code in its low bits, 128 comes off exactly, and the fma
// rounds once.
__device__ __forceinline__ void dequant8(uint32_t word, uint32_t s2, uint32_t m2, uint32_t (&r)[4]) {
  const uint32_t base = 0x43004300u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = ((word >> (4 * i)) & 0x000f000fu) | base;
    const __nv_bfloat162 n = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c), *reinterpret_cast<const __nv_bfloat162*>(&base));
    const __nv_bfloat162 y = __hfma2(n, *reinterpret_cast<const __nv_bfloat162*>(&s2), *reinterpret_cast<const __nv_bfloat162*>(&m2));
    r[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// N 32-bit words from a pointer aligned to all of them.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x, w[N > 1 ? 1 : 0] = x.y, w[N > 2 ? 2 : 0] = x.z, w[N > 3 ? 3 : 0] = x.w;
  } else if (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x, w[N > 1 ? 1 : 0] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// 64K tokens of 8 heads of d = 128 take 53 us, 6.6 TB/s: as fast as a copy.
// A warp per tile; blockIdx.y is 0 for K and 1 for V. A lane reads the words of
// one (token, t) of K or (g, token pair) of V and writes 16 or 2 x 8 bytes per
// group, so that four or eight lanes fill 64 bytes of an output row.
template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Args a, unsigned per, uint16_t* __restrict__ k,
                                                       uint16_t* __restrict__ v) {
  using F = Fmt<D>;
  constexpr int NG = F::NG;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const bool is_v = blockIdx.y != 0;
  uint16_t* dst = is_v ? v : k;
  if (dst == nullptr) return;
  Tile tl;
  if (!tile_of(a, blockIdx.x * 8 + (threadIdx.x >> 5), per, &tl)) return;
  const int rec = record_of(a.c, tl.b, tl.h, tl.m, a.Hkv, a.Lmax / kBlock, a.err);
  if (rec < 0) return;
  const uint8_t* tile = (is_v ? a.c.v : a.c.k) + size_t(rec) * F::kRecord + tl.in_block * F::kTileBytes;
  dst += (int64_t(tl.b * a.Hkv + tl.h) * a.n_tokens + tl.i0) * D;
  const int g = lane >> 2, t = lane & 3;
  if (is_v) {
    uint32_t w[2][NG], s[2 * NG], m[2][2][NG / 2];  // s: groups x token pairs; m: [pair][token of it]
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      load_words<NG>(tile + F::v_half(8 * u + 2 * t, g, 0), w[u]);
      load_words<NG / 2>(tile + F::min_at(8 * u + 2 * t, 0), m[u][0]);
      load_words<NG / 2>(tile + F::min_at(8 * u + 2 * t + 1, 0), m[u][1]);
    }
#pragma unroll
    for (int j = 0; j < NG; j += 2) {
      const uint4 y = *reinterpret_cast<const uint4*>(tile + F::kSteps + (t * NG + j) * 8);
      s[2 * j] = y.x, s[2 * j + 1] = y.y, s[2 * j + 2] = y.z, s[2 * j + 3] = y.w;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = 8 * u + 2 * t;
      const bool even = r >= tl.r0 && r < tl.r1, odd = r + 1 >= tl.r0 && r + 1 < tl.r1;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        uint32_t y[4];
        dequant8(w[u][j], s[2 * j + u], __byte_perm(m[u][0][j / 2], m[u][1][j / 2], (j & 1) ? 0x7632 : 0x5410), y);
        uint16_t* o = dst + r * D + 32 * j + 4 * g;
        if (even) __stcs(reinterpret_cast<uint2*>(o), make_uint2(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410)));
        if (odd) __stcs(reinterpret_cast<uint2*>(o + D), make_uint2(__byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632)));
      }
    }
  } else {
    uint32_t w[2][NG], s[2][NG / 2], m[2][NG / 2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      load_words<NG>(tile + F::k_word(8 * u + g, t, 0), w[u]);
      load_words<NG / 2>(tile + F::k_step(8 * u + g, 0), s[u]);
      load_words<NG / 2>(tile + F::min_at(8 * u + g, 0), m[u]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = 8 * u + g;
      const bool live = r >= tl.r0 && r < tl.r1;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const uint32_t sel = (j & 1) ? 0x3232 : 0x1010;
        uint32_t y[4];
        dequant8(w[u][j], __byte_perm(s[u][j / 2], 0, sel), __byte_perm(m[u][j / 2], 0, sel), y);
        if (live)
          __stcs(reinterpret_cast<uint4*>(dst + r * D + 32 * j + 8 * t),
                 make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410),
                            __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632)));
      }
    }
  }
}

// (x & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;\n" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  return y;
}

// 1/64 of nibbles 2 c and 2 c + 1 of a word as floats: the share of a mean, which
// keeps the sums of any finite keys in fp32's range. A nibble at bit p is left
// where it is: under the exponent of 2^(17 - p) it counts 1/64s, and 2^(17 - p)
// comes off exactly. Bits 20 and up are moved down by 12 first.
__device__ __forceinline__ float2 nibble_pair(uint32_t w, int c) {
  const uint32_t x = 2 * c >= 5 ? w >> 12 : w, y = 2 * c + 1 >= 5 ? w >> 12 : w;
  const int px = 8 * c - (2 * c >= 5 ? 12 : 0), py = 8 * c + 4 - (2 * c + 1 >= 5 ? 12 : 0);
  const uint32_t ex = uint32_t(127 + 17 - px) << 23, ey = uint32_t(127 + 17 - py) << 23;
  return add_f32x2(make_float2(__uint_as_float(and_or(x, 15u << px, ex)), __uint_as_float(and_or(y, 15u << py, ey))),
                   make_float2(-__uint_as_float(ex), -__uint_as_float(ey)));
}

// The mean key of a K record, by a warp. A lane sums the 8 tokens g, g + 8, ...
// of its t, 8 channels per group; the lanes of a t are then added pairwise, each
// keeping half of the channels.
template <int D>
__device__ __forceinline__ void mean_of(const uint8_t* rec, uint16_t* out) {
  using F = Fmt<D>;
  constexpr int NG = F::NG;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t w[2 * kTiles][NG], s[2 * kTiles][NG / 2], lo[2 * kTiles][NG / 2];
#pragma unroll
  for (int i = 0; i < 2 * kTiles; ++i) {
    const uint8_t* tile = rec + i / 2 * F::kTileBytes;
    const int r = g + 8 * (i & 1);
    load_words<NG>(tile + F::k_word(r, t, 0), w[i]);
    load_words<NG / 2>(tile + F::k_step(r, 0), s[i]);
    load_words<NG / 2>(tile + F::min_at(r, 0), lo[i]);
  }
  float2 acc[NG][4];  // channels 32 j + 8 t + {2 i, 2 i + 1}
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    float low = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 2 * kTiles; ++i) {
      const float sf = __uint_as_float((j & 1) ? s[i][j / 2] & 0xffff0000u : s[i][j / 2] << 16);
      low = fmaf(__uint_as_float((j & 1) ? lo[i][j / 2] & 0xffff0000u : lo[i][j / 2] << 16), 1.f / kBlock, low);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[j][c] = fma_f32x2(nibble_pair(w[i][j], c), dup2(sf), acc[j][c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[j][c] = add_f32x2(acc[j][c], dup2(low));
  }
  // lanes g and g ^ 4 swap halves of the groups, then g ^ 2 and g ^ 1 halves of what is left
  constexpr int N = NG * 8;
  float x[N];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) x[2 * i] = acc[i / 4][i % 4].x, x[2 * i + 1] = acc[i / 4][i % 4].y;
#pragma unroll
  for (int o = 16, n = N / 2; o >= 4; o >>= 1, n >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? x[i] : x[n + i], keep = up ? x[n + i] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  // this lane has the N/8 channels from N/8 · g of its t's list
  const int c0 = g * (N / 8), ch = 32 * (c0 / 8) + 8 * t + c0 % 8;
  if (NG == 4)
    *reinterpret_cast<uint2*>(out + ch) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  else
    *reinterpret_cast<uint32_t*>(out + ch) = pack_bf16x2(x[0], x[1]);
}

// Candidate block `item` of [bh][block]: its K record, or -1 where the new
// tokens have not completed it. row: its place among the means.
__device__ __forceinline__ int completed(const Kv4Args& a, unsigned item, unsigned per, size_t* row) {
  const unsigned bh = item / per;
  if (bh >= unsigned(a.B) * a.Hkv) return -1;
  const int b = int(bh / a.Hkv), h = int(bh % a.Hkv), NB = a.Lmax / kBlock;
  const Window wd = window_of(a.cache_len, a.new_len, b, a.n_tokens, a.Lmax, a.err);
  const int m = wd.pos / kBlock + int(item % per);
  if (wd.n == 0 || kBlock * (m + 1) > wd.pos + wd.n) return -1;
  *row = size_t(bh) * NB + m;
  return record_of(a.c, b, h, m, a.Hkv, NB, a.err);
}

constexpr int kMeanWarps = 4;

// One warp per candidate block. The record comes through shared memory, by ten
// copies a lane: 32768 records of d = 128 take 41 us so, 4.1 TB/s, against 51 us
// straight from global memory in registers and 42 us with a persistent grid and
// a ring of two records a warp; 8192 take 11 us. Neither a pipe nor DRAM is at
// its limit there: 980 instructions a record, half of them on the half-rate
// integer pipe, keep that 54 % busy and 61 % of the cycles issuing, DRAM is at
// 32 %, and the wait for the one record that a warp has is the largest stall.
template <int D>
__global__ void __launch_bounds__(32 * kMeanWarps, 28 / kMeanWarps) kv4_means_kernel(Kv4Args a, unsigned per, uint16_t* __restrict__ kmean) {
  constexpr int kRecord = Fmt<D>::kRecord;
  __shared__ __align__(16) uint8_t rec_s[kMeanWarps][kRecord];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  size_t row;
  const int rec = completed(a, blockIdx.x * kMeanWarps + warp, per, &row);
  if (rec < 0) return;
  const uint8_t* src = a.c.k + size_t(rec) * kRecord + lane * 16;
  const uint32_t dst = smem_u32(rec_s[warp]) + lane * 16;
#pragma unroll
  for (int o = 0; o < kRecord; o += 512) cp_async16(dst + o, src + o);
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
  mean_of<D>(rec_s[warp], kmean + row * D);
}

static Kv4Args kv4_args(const Shape& sh, const Cache& c, int n_tokens, const int32_t* cache_len,
                        const int32_t* new_len, int* err) {
  return {c, cache_len, new_len, n_tokens, sh.B, sh.Hkv, sh.N, err};
}

// The most 16-token tiles that n_tokens tokens can touch.
static unsigned tiles_of(int n_tokens) { return unsigned(n_tokens + kTile - 2) / kTile + 1; }

// CTAs of `warps` warps for `per` items of every sequence and head.
static bool kv4_grid(const Shape& sh, unsigned per, int warps, unsigned* ctas) {
  const uint64_t items = uint64_t(sh.B) * sh.Hkv * per;
  *ctas = unsigned((items + warps - 1) / warps);
  return items < (uint64_t(1) << 32) - 64;
}

cudaError_t launch_kv4_write(const Shape& sh, const Cache& c, int n_tokens, const uint16_t* k, const uint16_t* v,
                             const int32_t* cache_len, const int32_t* new_len, int* err, cudaStream_t st) {
  const Kv4Args a = kv4_args(sh, c, n_tokens, cache_len, new_len, err);
  const unsigned per = tiles_of(n_tokens);
  unsigned n;
  if (!kv4_grid(sh, per, kWriteWarps, &n)) return cudaErrorInvalidConfiguration;
  return launch_pdl(sh.d == 128 ? kv4_write_kernel<128> : kv4_write_kernel<64>, dim3(n, 2), dim3(32 * kWriteWarps), 0, st, a, per, k, v);
}

cudaError_t launch_kv4_read(const Shape& sh, const Cache& c, int n_tokens, uint16_t* k, uint16_t* v,
                            const int32_t* cache_len, const int32_t* new_len, int* err, cudaStream_t st) {
  const Kv4Args a = kv4_args(sh, c, n_tokens, cache_len, new_len, err);
  const unsigned per = tiles_of(n_tokens);
  unsigned n;
  if (!kv4_grid(sh, per, 8, &n)) return cudaErrorInvalidConfiguration;
  return launch_pdl(sh.d == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>, dim3(n, 2), dim3(256), 0, st, a, per, k, v);
}

cudaError_t launch_kv4_means(const Shape& sh, const Cache& c, int n_tokens, const int32_t* cache_len,
                             const int32_t* new_len, uint16_t* kmean, int* err, cudaStream_t st) {
  const Kv4Args a = kv4_args(sh, c, n_tokens, cache_len, new_len, err);
  const unsigned per = unsigned(n_tokens + kBlock - 1) / kBlock;  // the most blocks that n_tokens tokens can complete
  unsigned n;
  if (!kv4_grid(sh, per, kMeanWarps, &n)) return cudaErrorInvalidConfiguration;
  return launch_pdl(sh.d == 128 ? kv4_means_kernel<128> : kv4_means_kernel<64>, dim3(n), dim3(32 * kMeanWarps), 0, st, a, per, kmean);
}

}  // namespace sas
