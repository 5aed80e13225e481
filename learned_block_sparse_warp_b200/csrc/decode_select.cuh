// Top-K selection of one score row inside a 128-thread decode CTA, shared by the
// one-launch decode kernels over the bf16 and the 4-bit cache.
#pragma once

#include "common.cuh"

namespace sas {

namespace dec {
constexpr int kThreads = 128;
constexpr int kMaxTasks = kMaxDecodeBlocksPerSplit;  // task slots per chunk of items (2 CTAs per SM at d = 128)
constexpr int kFusedMaxK = 255;     // the fused step keeps the whole selected list in shared memory
constexpr int kFusedMaxNB = 2048;   // and the row's keys (4 bytes each) in one ring stage
constexpr int kMaxCluster = 8;      // portable cluster size
}  // namespace dec

// Exclusive sum over the 128 threads of the CTA (tot gets the total). Contains
// two __syncthreads; wtot holds 4 ints of shared memory.
__device__ __forceinline__ int cta_excl_sum(int v, int* wtot, int& tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += u;
  }
  if (lane == 31) wtot[warp] = incl;
  __syncthreads();
  int before = incl - v;
  tot = 0;
#pragma unroll
  for (int w = 0; w < dec::kThreads / 32; ++w) {
    before += (w < warp) ? wtot[w] : 0;
    tot += wtot[w];
  }
  __syncthreads();
  return before;
}

// One 8-bit radix pass over the keys of key[0, c) whose bits above `shift + 8`
// equal prefix's: fixes the digit at which the count from the top bin reaches
// need. xch gets the digit, the number still needed within its bin, and the
// bin's count. (Plain shared atomics: aggregating equal digits within a warp
// first, by match.any, measured slower on sm_100a.)
__device__ inline void cta_radix_pass(const uint32_t* key, int c, int pass, uint32_t prefix, int need, int* hist, int* xch) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int shift = 24 - 8 * pass;
  for (int i = tid; i < 256; i += dec::kThreads) hist[i] = 0;
  __syncthreads();
  for (int m = tid; m < c; m += dec::kThreads) {
    const uint32_t k = key[m];
    if (pass == 0 || ((k ^ prefix) >> (shift + 8)) == 0u) atomicAdd(&hist[(k >> shift) & 255u], 1);
  }
  __syncthreads();
  if (tid < 32) {  // lane owns bins [8 lane, 8 lane + 8); counts run from the top bin down
    int cnt[8], own = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      cnt[u] = hist[8 * lane + u];
      own += cnt[u];
    }
    int incl = own;  // own plus every lane above
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_down_sync(0xffffffffu, incl, off);
      if (lane + off < 32) incl += u;
    }
    int acc = incl - own;  // keys in bins above this lane's
    if (acc < need && need <= incl) {
#pragma unroll
      for (int u = 7; u >= 0; --u) {
        if (acc + cnt[u] >= need) {
          xch[0] = 8 * lane + u;
          xch[1] = need - acc;
          xch[2] = cnt[u];
          break;
        }
        acc += cnt[u];
      }
    }
  }
  __syncthreads();
}

// The n largest of key[0, c) in shared memory (0 < n < c), ties to the lowest
// index. The first 8-bit radix pass fixes the leading byte of the n-th largest
// key. When at most 128 keys share that byte (the usual case: scores spread
// over several exponents), those candidates are ranked against each other
// directly, one per thread, and the picks (every key with a larger leading
// byte, and the candidates ranked below the number still needed) are appended
// to app in any order. Otherwise three more passes find the exact threshold;
// the picks are appended likewise unless a tie is cut at it, in which case
// the function returns true with the threshold and the number of its equals
// to take, and the caller places the picks in index order.
__device__ inline bool cta_select(const uint32_t* key, int c, int n, int* hist, int* xch, int* app, int* napp,
                           uint32_t* cand_k, int* cand_m, int* ncand, uint32_t& thr, int& need_eq) {
  const int tid = threadIdx.x;
  if (tid == 0) *ncand = 0;
  cta_radix_pass(key, c, 0, 0u, n, hist, xch);
  const uint32_t d0 = uint32_t(xch[0]);
  const int need1 = xch[1], cnt0 = xch[2];
  if (cnt0 <= dec::kThreads) {
    for (int m = tid; m < c; m += dec::kThreads) {
      const uint32_t k = key[m], top = k >> 24;
      if (top > d0) {
        app[atomicAdd(napp, 1)] = m;
      } else if (top == d0) {
        const int s = atomicAdd(ncand, 1);
        cand_k[s] = k;
        cand_m[s] = m;
      }
    }
    __syncthreads();
    if (tid < cnt0) {
      const uint32_t k = cand_k[tid];
      const int mi = cand_m[tid];
      int r = 0;  // candidates ahead of this one: larger keys, and equal keys at lower indexes
#pragma unroll 8
      for (int j = 0; j < cnt0; ++j) {
        const uint32_t kj = cand_k[j];
        r += (kj > k || (kj == k && cand_m[j] < mi)) ? 1 : 0;
      }
      if (r < need1) app[atomicAdd(napp, 1)] = mi;
    }
    return false;
  }
  uint32_t prefix = d0 << 24;
  int need = need1;
#pragma unroll 1
  for (int pass = 1; pass < 4; ++pass) {
    cta_radix_pass(key, c, pass, prefix, need, hist, xch);
    prefix |= uint32_t(xch[0]) << (24 - 8 * pass);
    need = xch[1];
  }
  thr = prefix;
  need_eq = need;
  if (need_eq != xch[2]) return true;  // a tie is cut at the threshold
  for (int m = tid; m < c; m += dec::kThreads)
    if (key[m] >= thr) app[atomicAdd(napp, 1)] = m;
  return false;
}

}  // namespace sas
