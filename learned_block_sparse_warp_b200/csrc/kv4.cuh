// The 4-bit KV cache's format, shared by the kernels that write it, read it
// back, summarise it and attend over it.
//
// A group is 32 channels of one token. It keeps its minimum m and a step s in
// bf16 and one 4-bit code per channel: value = s·code + m. A record is one
// 64-token block of one KV head, of K or of V: four tiles of 16 tokens, each
// 8 d bytes of codes followed by its steps and its minima (5 bits a value in
// all, 40 d bytes a record).
//
// The order inside a tile is that of the mma.sync m16n8k16 A fragments that
// read it, so a lane's operands are one 16-byte (d = 128) shared-memory load:
//  - K: the rows of A are tokens. A token's row is 4 chunks, one per lane t of
//    a quad; chunk t holds one word per group j, whose nibble p is channel
//    32 j + 8 t + p.
//  - V: the rows of A are channels and its k index runs over tokens, two to a
//    register. Word (u, g, t, j) holds tokens 8u + 2t (low half) and
//    8u + 2t + 1 (high half); nibble p of a half is channel 32 j + 4 g + p.
//    Tokens never share a 16-bit half, so a token is written without reading.
//  - K steps, K minima and V minima are [token][group]. V steps are
//    [t][group][i], token 8 (i / 2) + 2 t + i % 2: the four a lane multiplies.
#pragma once

#include "common.cuh"

namespace sas {
namespace kv4 {

constexpr int kGroup = 32;                 // channels that share a step and a minimum
constexpr int kTile = 16;                  // tokens per tile
constexpr int kTiles = kBlock / kTile;     // tiles per record
constexpr float kMinStep = 1.17549435e-38f;  // 2^-126: smaller steps are stored as 0

template <int D>
struct Fmt {
  static constexpr int NG = D / kGroup;             // groups per token
  static constexpr int kCodes = 8 * D;              // code bytes of a tile
  static constexpr int kSteps = kCodes;             // byte offset of a tile's steps
  static constexpr int kMins = kCodes + 2 * kTile * NG;  // and of its minima
  static constexpr int kTileBytes = 10 * D;
  static constexpr int kRecord = kTiles * kTileBytes;
  // byte offsets inside a tile; r is the token of the tile
  static __host__ __device__ constexpr int k_word(int r, int t, int j) { return r * (D / 2) + t * 4 * NG + 4 * j; }
  static __host__ __device__ constexpr int k_step(int r, int j) { return kSteps + 2 * (r * NG + j); }
  static __host__ __device__ constexpr int v_half(int r, int g, int j) {
    return (r >> 3) * 128 * NG + (4 * g + ((r & 7) >> 1)) * 4 * NG + 4 * j + 2 * (r & 1);
  }
  static __host__ __device__ constexpr int v_step(int r, int j) {
    return kSteps + 2 * ((((r & 7) >> 1) * NG + j) * 4 + 2 * (r >> 3) + (r & 1));
  }
  static __host__ __device__ constexpr int min_at(int r, int j) { return kMins + 2 * (r * NG + j); }
};

// The cache as the kernels see it.
struct Cache {
  uint8_t* k;
  uint8_t* v;
  const int32_t* table;  // page of block m of sequence b at table[b * NB + m]; null for the dense cache
  int n_pages;
};

// Record of block m of sequence b, KV head h: dense [B, Hkv, NB] or paged
// [n_pages, Hkv]. A page outside the pool raises SAS_ERR_DEVICE_INDEX and
// returns -1.
__device__ __forceinline__ int record_of(const Cache& c, int b, int h, int m, int Hkv, int NB, int* err) {
  if (c.table == nullptr) return (b * Hkv + h) * NB + m;
  const int pg = c.table[size_t(b) * NB + m];
  if (pg < 0 || pg >= c.n_pages) {
    raise_error(err, SAS_ERR_DEVICE_INDEX);
    return -1;
  }
  return pg * Hkv + h;
}

// The new tokens of a sequence: `n` of them, the first at position `pos`.
// Lengths that break 0 <= n <= n_tokens, n <= L <= Lmax raise
// SAS_ERR_DEVICE_INDEX and give n = 0.
struct Window {
  int pos, n;
};
__device__ __forceinline__ Window window_of(const int32_t* cache_len, const int32_t* new_len, int b, int n_tokens,
                                            int Lmax, int* err) {
  const int L = cache_len[b];
  const int n = new_len != nullptr ? new_len[b] : n_tokens;
  if (n < 0 || n > n_tokens || L < n || L > Lmax) {
    raise_error(err, SAS_ERR_DEVICE_INDEX);
    return {0, 0};
  }
  return {L - n, n};
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
// The same, rounded down.
__device__ __forceinline__ float2 fma_down_f32x2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};\n"
      "fma.rm.f32x2 d, a, b, c; mov.b64 {%0, %1}, d;}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add_down_f32x2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rm.f32x2 d, a, b; mov.b64 {%0, %1}, d;}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

}  // namespace kv4
}  // namespace sas
