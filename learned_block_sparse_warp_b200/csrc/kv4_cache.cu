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
// Read: bf16(s·code + m), one rounding. Means: (1/64) Σ (s·code + m) in fp32.
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

// One group's parameters and this lane's 8 codes.
struct Quant8 {
  uint32_t word;   // nibble p: code of the lane's channel p
  uint16_t s, m;   // bf16
};

// Four consecutive lanes hold a group, 8 bf16 channels each. Every lane of the
// warp takes part.
__device__ __forceinline__ Quant8 quantise8(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  __nv_bfloat162 mx = *reinterpret_cast<const __nv_bfloat162*>(&w[0]), mn = mx;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
    mx = __hmax2_nan(mx, v);
    mn = __hmin2_nan(mn, v);
  }
  // (max, −min) in one register: one shuffle serves both
  __nv_bfloat162 e = __halves2bfloat162(__hmax_nan(mx.x, mx.y), __hneg(__hmin_nan(mn.x, mn.y)));
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    const uint32_t u = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&e), o);
    e = __hmax2_nan(e, *reinterpret_cast<const __nv_bfloat162*>(&u));
  }
  const float hi = __bfloat162float(e.x), lo = -__bfloat162float(e.y);
  const float range = __fsub_rn(hi, lo);
  const bool bad = !(fabsf(range) <= 3.402823466e38f);
  __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(range, 15.f));
  float s = __bfloat162float(sb);
  if (bad || s < kMinStep) {
    s = 0.f;
    sb = __float2bfloat16_rn(0.f);
  }
  // 1/s raised by 2^-20, which outweighs its rounding: a value half-way
  // between two levels goes up, as in the definition. fma adds 1.5·2^23, so
  // the code is in the low bits, rounded once.
  const float inv = s > 0.f ? __fmul_rn(__fdiv_rn(1.f, s), 1.00000095367431640625f) : 0.f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xffff0000u);
    const uint32_t cb = __float_as_uint(fmaf(__fsub_rn(b, lo), inv, 12582912.f));
    const uint32_t ca = __float_as_uint(fmaf(__fsub_rn(a, lo), inv, 12582912.f));
    word = (word << 8) | ((cb & 15u) << 4) | (ca & 15u);
  }
  Quant8 q;
  q.word = bad ? 0u : word;
  q.s = __bfloat16_as_ushort(sb);
  q.m = bad ? uint16_t(0x7fc0u) : __bfloat16_as_ushort(__float2bfloat16_rn(__fadd_rn(lo, 0.f)));  // −0 becomes +0
  return q;
}

// D/8 lanes per token and KV head; blockIdx.y is 0 for K and 1 for V.
template <int D>
__global__ void __launch_bounds__(256) kv4_write_kernel(Kv4Args a, const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v) {
  using F = Fmt<D>;
  constexpr int LPR = D / 8;
  griddep_launch_dependents();
  griddep_wait();
  const int NB = a.Lmax / kBlock;
  const bool is_v = blockIdx.y != 0;
  const uint16_t* src = is_v ? v : k;
  uint8_t* dst = is_v ? a.c.v : a.c.k;
  const int l = threadIdx.x % LPR, j = l >> 2, q = l & 3;
  const int64_t rows = int64_t(a.B) * a.Hkv * a.n_tokens;
  for (int64_t r0 = int64_t(blockIdx.x) * (256 / LPR); r0 < rows; r0 += int64_t(gridDim.x) * (256 / LPR)) {
    const int64_t row = r0 + threadIdx.x / LPR;
    bool live = row < rows;
    uint4 x = make_uint4(0, 0, 0, 0);
    int b = 0, h = 0, pos = 0;
    if (live) {
      const int i = int(row % a.n_tokens), bh = int(row / a.n_tokens);
      b = bh / a.Hkv;
      h = bh % a.Hkv;
      const Window w = window_of(a.cache_len, a.new_len, b, a.n_tokens, a.Lmax, a.err);
      live = i < w.n;
      pos = w.pos + i;
      if (live) x = *reinterpret_cast<const uint4*>(src + row * D + 8 * l);
    }
    const Quant8 g = quantise8(x);
    if (!live) continue;
    const int rec = record_of(a.c, b, h, pos / kBlock, a.Hkv, NB, a.err);
    if (rec < 0) continue;
    uint8_t* tile = dst + size_t(rec) * F::kRecord + (pos % kBlock) / kTile * F::kTileBytes;
    const int r = pos % kTile;
    if (is_v) {
      *reinterpret_cast<uint16_t*>(tile + F::v_half(r, 2 * q, j)) = uint16_t(g.word);
      *reinterpret_cast<uint16_t*>(tile + F::v_half(r, 2 * q + 1, j)) = uint16_t(g.word >> 16);
    } else {
      *reinterpret_cast<uint32_t*>(tile + F::k_word(r, q, j)) = g.word;
    }
    if (q == 0) {
      *reinterpret_cast<uint16_t*>(tile + (is_v ? F::v_step(r, j) : F::k_step(r, j))) = g.s;
      *reinterpret_cast<uint16_t*>(tile + F::min_at(r, j)) = g.m;
    }
  }
}

// 8 values s·code + m of one word.
__device__ __forceinline__ void values8(uint32_t word, float s, float m, float* x) {
#pragma unroll
  for (int p = 0; p < 8; ++p) x[p] = fmaf(s, __uint_as_float(0x4b000000u | ((word >> (4 * p)) & 15u)) - 8388608.f, m);
}

template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Args a, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  using F = Fmt<D>;
  constexpr int LPR = D / 8;
  griddep_launch_dependents();
  griddep_wait();
  const int NB = a.Lmax / kBlock;
  const bool is_v = blockIdx.y != 0;
  uint16_t* dst = is_v ? v : k;
  const uint8_t* src = is_v ? a.c.v : a.c.k;
  if (dst == nullptr) return;
  const int l = threadIdx.x % LPR, j = l >> 2, q = l & 3;
  const int64_t rows = int64_t(a.B) * a.Hkv * a.n_tokens;
  for (int64_t row = int64_t(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR; row < rows;
       row += int64_t(gridDim.x) * (256 / LPR)) {
    const int i = int(row % a.n_tokens), bh = int(row / a.n_tokens);
    const int b = bh / a.Hkv, h = bh % a.Hkv;
    const Window w = window_of(a.cache_len, a.new_len, b, a.n_tokens, a.Lmax, a.err);
    if (i >= w.n) continue;
    const int pos = w.pos + i;
    const int rec = record_of(a.c, b, h, pos / kBlock, a.Hkv, NB, a.err);
    if (rec < 0) continue;
    const uint8_t* tile = src + size_t(rec) * F::kRecord + (pos % kBlock) / kTile * F::kTileBytes;
    const int r = pos % kTile;
    uint32_t word;
    if (is_v)
      word = uint32_t(*reinterpret_cast<const uint16_t*>(tile + F::v_half(r, 2 * q, j))) |
             uint32_t(*reinterpret_cast<const uint16_t*>(tile + F::v_half(r, 2 * q + 1, j))) << 16;
    else
      word = *reinterpret_cast<const uint32_t*>(tile + F::k_word(r, q, j));
    const float s = bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + (is_v ? F::v_step(r, j) : F::k_step(r, j))));
    const float m = bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + F::min_at(r, j)));
    float x[8];
    values8(word, s, m, x);
    *reinterpret_cast<uint4*>(dst + row * D + 8 * l) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
}

// One warp per (sequence, KV head, candidate block). D/8 lanes cover a token's
// words, so 32/(D/8) tokens are summed side by side.
template <int D>
__global__ void __launch_bounds__(256) kv4_means_kernel(Kv4Args a, uint16_t* __restrict__ kmean) {
  using F = Fmt<D>;
  constexpr int LPR = D / 8, TP = 32 / LPR;
  griddep_launch_dependents();
  griddep_wait();
  const int NB = a.Lmax / kBlock;
  const int per = (a.n_tokens + kBlock - 1) / kBlock;  // most blocks that n_tokens tokens can complete
  const int64_t items = int64_t(a.B) * a.Hkv * per;
  const int lane = threadIdx.x & 31, l = lane % LPR, j = l >> 2, q = l & 3;
  for (int64_t it = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items; it += int64_t(gridDim.x) * 8) {
    const int bh = int(it / per), b = bh / a.Hkv, h = bh % a.Hkv;
    const Window w = window_of(a.cache_len, a.new_len, b, a.n_tokens, a.Lmax, a.err);
    const int m = w.pos / kBlock + int(it % per);
    if (kBlock * (m + 1) > w.pos + w.n || w.n == 0) continue;
    const int rec = record_of(a.c, b, h, m, a.Hkv, NB, a.err);
    if (rec < 0) continue;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int tok = lane / LPR; tok < kBlock; tok += TP) {
      const uint8_t* tile = a.c.k + size_t(rec) * F::kRecord + tok / kTile * F::kTileBytes;
      const int r = tok % kTile;
      float x[8];
      values8(*reinterpret_cast<const uint32_t*>(tile + F::k_word(r, q, j)),
              bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + F::k_step(r, j))),
              bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + F::min_at(r, j))), x);
#pragma unroll
      for (int p = 0; p < 8; ++p) acc[p] += x[p];
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) acc[p] += __shfl_xor_sync(0xffffffffu, acc[p], o);
      acc[p] *= 1.f / kBlock;
    }
    if (lane < LPR)
      *reinterpret_cast<uint4*>(kmean + ((size_t(bh) * NB + m) * D + 8 * l)) = make_uint4(
          pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
  }
}

static Kv4Args kv4_args(const Shape& sh, const Cache& c, int n_tokens, const int32_t* cache_len,
                        const int32_t* new_len, int* err) {
  return {c, cache_len, new_len, n_tokens, sh.B, sh.Hkv, sh.N, err};
}

static unsigned kv4_grid(int64_t items, int per_cta) {
  const int64_t n = (items + per_cta - 1) / per_cta;
  return unsigned(n < 1 ? 1 : n > (1 << 30) ? (1 << 30) : n);
}

cudaError_t launch_kv4_write(const Shape& sh, const Cache& c, int n_tokens, const uint16_t* k, const uint16_t* v,
                             const int32_t* cache_len, const int32_t* new_len, int* err, cudaStream_t st) {
  const Kv4Args a = kv4_args(sh, c, n_tokens, cache_len, new_len, err);
  const dim3 grid(kv4_grid(int64_t(sh.B) * sh.Hkv * n_tokens, 256 / (sh.d / 8)), 2);
  const cudaError_t e = sh.d == 128 ? launch_pdl(kv4_write_kernel<128>, grid, dim3(256), 0, st, a, k, v)
                                    : launch_pdl(kv4_write_kernel<64>, grid, dim3(256), 0, st, a, k, v);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv4_read(const Shape& sh, const Cache& c, int n_tokens, uint16_t* k, uint16_t* v,
                            const int32_t* cache_len, const int32_t* new_len, int* err, cudaStream_t st) {
  const Kv4Args a = kv4_args(sh, c, n_tokens, cache_len, new_len, err);
  const dim3 grid(kv4_grid(int64_t(sh.B) * sh.Hkv * n_tokens, 256 / (sh.d / 8)), 2);
  const cudaError_t e = sh.d == 128 ? launch_pdl(kv4_read_kernel<128>, grid, dim3(256), 0, st, a, k, v)
                                    : launch_pdl(kv4_read_kernel<64>, grid, dim3(256), 0, st, a, k, v);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv4_means(const Shape& sh, const Cache& c, int n_tokens, const int32_t* cache_len,
                             const int32_t* new_len, uint16_t* kmean, int* err, cudaStream_t st) {
  const Kv4Args a = kv4_args(sh, c, n_tokens, cache_len, new_len, err);
  const dim3 grid(kv4_grid(int64_t(sh.B) * sh.Hkv * ((n_tokens + kBlock - 1) / kBlock), 8));
  const cudaError_t e = sh.d == 128 ? launch_pdl(kv4_means_kernel<128>, grid, dim3(256), 0, st, a, kmean)
                                    : launch_pdl(kv4_means_kernel<64>, grid, dim3(256), 0, st, a, kmean);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sas
