// Sparse single-token decode over the 4-bit KV cache: the split form with its
// partials, and the whole step (select, attention) in one launch.
#include "decode_select.cuh"
#include "kv4.cuh"

namespace sas {

using namespace kv4;

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

template <int D>
struct SimpleState {
  float acc[8 * D / dec::kThreads];  // outputs e = tid + 128 i of the G x D tile
};

// One block: dequantise K, score, online softmax, dequantise V, accumulate.
template <int D>
__device__ void simple_block(const Kv4DecodeArgs& a, SimpleState<D>& st, int rec, int ntok, float lam, float gw,
                             const float* q_s, float (*kv_s)[D + 1], float (*sc)[kBlock], float* m_s, float* l_s,
                             float* al_s) {
  using F = Fmt<D>;
  const int tid = threadIdx.x;
  for (int e = tid; e < kBlock * D; e += dec::kThreads) {
    const int tok = e / D, c = e % D, j = c / 32, r = tok % kTile;
    const uint8_t* tile = a.c.k + size_t(rec) * F::kRecord + tok / kTile * F::kTileBytes;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + F::k_word(r, c % 32 / 8, j));
    const float s = bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + F::k_step(r, j)));
    const float m = bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + F::min_at(r, j)));
    kv_s[tok][c] = tok < ntok ? fmaf(s, float((w >> (4 * (c % 8))) & 15u), m) : 0.f;
  }
  __syncthreads();
  for (int e = tid; e < a.G * kBlock; e += dec::kThreads) {
    const int g = e / kBlock, tok = e % kBlock;
    float z = 0.f;
    for (int c = 0; c < D; ++c) z = fmaf(q_s[g * D + c], kv_s[tok][c], z);
    sc[g][tok] = tok < ntok ? z * a.scale * kLog2e + lam : -INFINITY;
  }
  __syncthreads();
  if (tid < a.G) {
    float mx = m_s[tid];
    for (int t = 0; t < kBlock; ++t) mx = fmaxf(mx, sc[tid][t]);
    const float al = m_s[tid] == -INFINITY ? 0.f : exp2f(m_s[tid] - mx);
    float sum = 0.f;
    for (int t = 0; t < kBlock; ++t) {
      const float p = sc[tid][t] == -INFINITY ? 0.f : exp2f(sc[tid][t] - mx);
      sum += p;
      sc[tid][t] = p * gw;
    }
    m_s[tid] = mx;
    l_s[tid] = l_s[tid] * al + sum;
    al_s[tid] = al;
  }
  for (int e = tid; e < kBlock * D; e += dec::kThreads) {
    const int tok = e / D, c = e % D, j = c / 32, r = tok % kTile;
    const uint8_t* tile = a.c.v + size_t(rec) * F::kRecord + tok / kTile * F::kTileBytes;
    const uint32_t w = *reinterpret_cast<const uint16_t*>(tile + F::v_half(r, c % 32 / 4, j));
    const float s = bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + F::v_step(r, j)));
    const float m = bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + F::min_at(r, j)));
    kv_s[tok][c] = tok < ntok ? fmaf(s, float((w >> (4 * (c % 4))) & 15u), m) : 0.f;
  }
  __syncthreads();
  for (int i = 0; i < 8 * D / dec::kThreads; ++i) {
    const int e = tid + dec::kThreads * i, g = e / D, c = e % D;
    if (g < a.G) {
      float x = st.acc[i] * al_s[g];
      for (int t = 0; t < ntok; ++t) x = fmaf(sc[g][t], kv_s[t][c], x);
      st.acc[i] = x;
    }
  }
  __syncthreads();
}

template <int D, bool FUSED>
__global__ void __launch_bounds__(dec::kThreads) kv4_decode_kernel(Kv4DecodeArgs a) {
  __shared__ float kv_s[kBlock][D + 1], q_s[8 * D], sc[8][kBlock], m_s[8], l_s[8], al_s[8];
  __shared__ int sel_s[dec::kFusedMaxK];
  __shared__ uint32_t cand_k[128];
  __shared__ int cand_m[128], hist_s[256], app_s[256], xch_s[4], wtot_s[4], napp_s;
  __shared__ float redf_s[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ns = FUSED ? 1 : a.n_split;
  const int split = blockIdx.x % ns, bh = blockIdx.x / ns, b = bh / a.Hkv, h = bh % a.Hkv;
  const int NB = a.Lmax / kBlock;
  griddep_launch_dependents();
  griddep_wait();
  int L = a.cache_len[b];
  if (L < 1 || L > a.Lmax) {
    if (tid == 0) raise_error(a.err, SAS_ERR_DEVICE_INDEX);
    L = max(1, min(L, a.Lmax));
  }
  const int c = (L - 1) / kBlock, n = min(a.K, c);
  const float* srow = a.s + size_t(bh) * NB;
  float lse = 0.f;
  if (FUSED) {
    uint32_t* key_s = reinterpret_cast<uint32_t*>(&kv_s[0][0]);
    float mx = -INFINITY;
    for (int m = tid; m < c; m += dec::kThreads) {
      key_s[m] = score_key(srow[m]) + 1u;
      mx = fmaxf(mx, srow[m]);
    }
    mx = warp_max(mx);
    if (lane == 0) redf_s[warp] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(redf_s[0], redf_s[1]), fmaxf(redf_s[2], redf_s[3]));
    __syncthreads();
    float sum = 0.f;
    if (mx != -INFINITY)
      for (int m = tid; m < c; m += dec::kThreads) sum += expf(srow[m] - mx);
    sum = warp_sum(sum);
    if (lane == 0) redf_s[warp] = sum;
    if (tid == 0) napp_s = 0;
    __syncthreads();
    lse = (c == 0 || mx == -INFINITY) ? -INFINITY : mx + logf((redf_s[0] + redf_s[1]) + (redf_s[2] + redf_s[3]));
    uint32_t thr = 1u;
    int need_eq = 0;
    bool tie = false;
    if (n == c) {
      for (int m = tid; m < c; m += dec::kThreads) app_s[m] = m;
    } else if (n > 0) {
      tie = cta_select(key_s, c, n, hist_s, xch_s, app_s, &napp_s, cand_k, cand_m, &xch_s[3], thr, need_eq);
    }
    __syncthreads();
    if (n > 0 && !tie) {
      for (int i = tid; i < n; i += dec::kThreads) {
        const int v = app_s[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += app_s[j] < v ? 1 : 0;
        sel_s[r] = v;
      }
    } else if (n > 0 && tid == 0) {
      int pos = 0, eq = 0;
      for (int m = 0; m < c; ++m) {
        const bool is_eq = key_s[m] == thr;
        if (key_s[m] > thr || (is_eq && eq < need_eq)) sel_s[pos++] = m;
        eq += is_eq ? 1 : 0;
      }
    }
    __syncthreads();
    if (a.idx_out != nullptr)
      for (int i = tid; i < a.K; i += dec::kThreads) a.idx_out[size_t(bh) * a.K + i] = i < n ? sel_s[i] : -1;
    if (a.lse_s_out != nullptr && tid == 0) a.lse_s_out[bh] = lse;
  } else if (a.gated && a.lse_s_in != nullptr) {
    lse = a.lse_s_in[bh];
  }
  SimpleState<D> st;
  for (int i = 0; i < 8 * D / dec::kThreads; ++i) st.acc[i] = 0.f;
  for (int e = tid; e < a.G * D; e += dec::kThreads) q_s[e] = bf16_to_f32(a.q[size_t(bh) * a.G * D + e]);
  if (tid < 8) {
    m_s[tid] = -INFINITY;
    l_s[tid] = 0.f;
  }
  __syncthreads();
  const int nl = 1 + n, per = (nl + ns - 1) / ns;
  const int lo = min(split * per, nl), hi = min(lo + per, nl);
  for (int pos = lo; pos < hi; ++pos) {
    int m = c, ntok = L - c * kBlock;
    float lam = 0.f;
    if (pos > 0) {
      m = FUSED ? sel_s[pos - 1] : a.idx_in[size_t(bh) * a.K + pos - 1];
      ntok = kBlock;
      if (m >= c && tid == 0) raise_error(a.err, SAS_ERR_DEVICE_INDEX);
      if (m < 0 || m >= c) continue;
      if (a.gated) lam = gate_lam2(a.gate, srow[m], lse);
    }
    const int rec = record_of(a.c, b, h, m, a.Hkv, NB, a.err);
    if (rec < 0) continue;
    simple_block<D>(a, st, rec, ntok, a.outside ? 0.f : lam, a.outside ? exp2f(lam) : 1.f, q_s, kv_s, sc, m_s, l_s,
                    al_s);
  }
  for (int i = 0; i < 8 * D / dec::kThreads; ++i) {
    const int e = tid + dec::kThreads * i, g = e / D, col = e % D;
    if (g >= a.G) continue;
    const float l = l_s[g], val = l > 0.f || l != l ? st.acc[i] / l : 0.f;
    const float ls = l > 0.f || l != l ? (m_s[g] + log2f(l)) * kLn2 : -INFINITY;
    const size_t row = size_t(bh) * a.G + g;
    if (FUSED) {
      a.o[row * D + col] = __bfloat16_as_ushort(__float2bfloat16_rn(val));
      if (col == 0 && a.lse_o != nullptr) a.lse_o[row] = ls;
    } else {
      a.o_part[(row * ns + split) * D + col] = val;
      if (col == 0) a.lse_part[row * ns + split] = ls;
    }
  }
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

cudaError_t launch_decode_kv4(const Shape& sh, const uint16_t* q, const Cache& c, const int32_t* cl, const float* s,
                              const int32_t* idx, const float* lse_s, int n_split, float* o_part, float* lse_part,
                              int* err, cudaStream_t st) {
  Kv4DecodeArgs a = kv4_decode_args(sh, q, c, cl, s, err);
  a.idx_in = idx;
  a.lse_s_in = lse_s;
  a.n_split = n_split;
  a.o_part = o_part;
  a.lse_part = lse_part;
  const dim3 grid(unsigned(sh.B) * sh.Hkv * n_split);
  const cudaError_t e = sh.d == 128 ? launch_pdl(kv4_decode_kernel<128, false>, grid, dim3(dec::kThreads), 0, st, a)
                                    : launch_pdl(kv4_decode_kernel<64, false>, grid, dim3(dec::kThreads), 0, st, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_decode_fused_kv4(const Shape& sh, const uint16_t* q, const Cache& c, const int32_t* cl,
                                    const float* s, int32_t* idx, float* lse_s, uint16_t* o, float* lse_o, int* err,
                                    cudaStream_t st) {
  Kv4DecodeArgs a = kv4_decode_args(sh, q, c, cl, s, err);
  a.idx_out = idx;
  a.lse_s_out = lse_s;
  a.o = o;
  a.lse_o = lse_o;
  const dim3 grid(unsigned(sh.B) * sh.Hkv);
  const cudaError_t e = sh.d == 128 ? launch_pdl(kv4_decode_kernel<128, true>, grid, dim3(dec::kThreads), 0, st, a)
                                    : launch_pdl(kv4_decode_kernel<64, true>, grid, dim3(dec::kThreads), 0, st, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sas
