// C entry points of the 4-bit KV cache: argument checks and dispatch. Their
// contracts are in include/sas.h.
#include "kv4.cuh"

namespace sas {
sas_status check_params(const sas_params* p, Shape* sh);
int* error_word();
bool decode_fused_fits(const Shape& sh);
cudaError_t launch_kv4_write(const Shape& sh, const kv4::Cache& c, int n_tokens, const uint16_t* k, const uint16_t* v,
                             const int32_t* cache_len, const int32_t* new_len, int* err, cudaStream_t st);
cudaError_t launch_kv4_read(const Shape& sh, const kv4::Cache& c, int n_tokens, uint16_t* k, uint16_t* v,
                            const int32_t* cache_len, const int32_t* new_len, int* err, cudaStream_t st);
cudaError_t launch_kv4_means(const Shape& sh, const kv4::Cache& c, int n_tokens, const int32_t* cache_len,
                             const int32_t* new_len, uint16_t* kmean, int* err, cudaStream_t st);
cudaError_t launch_decode_kv4(const Shape& sh, const uint16_t* q, const kv4::Cache& c, const int32_t* cl,
                              const float* s, const int32_t* idx, const float* lse_s, int n_split, float* o_part,
                              float* lse_part, int* err, cudaStream_t st);
cudaError_t launch_decode_fused_kv4(const Shape& sh, const uint16_t* q, const kv4::Cache& c, const int32_t* cl,
                                    const float* s, int32_t* idx, float* lse_s, uint16_t* o, float* lse_o, int* err,
                                    cudaStream_t st);
}  // namespace sas

using sas::Shape;

namespace {

bool ok_opt(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void* p) { return p != nullptr && ok_opt(p); }
sas_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SAS_OK : SAS_ERR_CUDA; }

// Parameters and cache of a call. need_k / need_v: the sides the call touches.
sas_status check_cache(const sas_params* p, const sas_kv4_cache* c, bool need_k, bool need_v, Shape* sh,
                       sas::kv4::Cache* out) {
  const sas_status r = sas::check_params(p, sh);
  if (r != SAS_OK) return r;
  if (c == nullptr || !ok_opt(c->k) || !ok_opt(c->v) || !ok_opt(c->block_table)) return SAS_ERR_INVALID_ARG;
  if ((need_k && c->k == nullptr) || (need_v && c->v == nullptr)) return SAS_ERR_INVALID_ARG;
  if (c->block_table != nullptr &&
      (c->n_pages < 1 || int64_t(c->n_pages) * sh->Hkv > (int64_t(1) << 31) / sas::kBlock))
    return SAS_ERR_INVALID_ARG;
  *out = {c->k, c->v, c->block_table, c->n_pages};
  return SAS_OK;
}

bool ok_tokens(const Shape& sh, int n_tokens, const int32_t* cache_len, const int32_t* new_len) {
  return n_tokens >= 1 && n_tokens <= sh.N && ok_ptr(cache_len) && ok_opt(new_len);
}

}  // namespace

extern "C" {

sas_status sas_kv4_write(const sas_params* p, const sas_kv4_cache* cache, int n_tokens, const sas_bf16* k,
                         const sas_bf16* v, const int32_t* cache_len, const int32_t* new_len, void* stream) {
  Shape sh;
  sas::kv4::Cache c;
  const sas_status r = check_cache(p, cache, true, true, &sh, &c);
  if (r != SAS_OK) return r;
  if (!ok_tokens(sh, n_tokens, cache_len, new_len) || !ok_ptr(k) || !ok_ptr(v)) return SAS_ERR_INVALID_ARG;
  return from_cuda(sas::launch_kv4_write(sh, c, n_tokens, k, v, cache_len, new_len, sas::error_word(),
                                         static_cast<cudaStream_t>(stream)));
}

sas_status sas_kv4_read(const sas_params* p, const sas_kv4_cache* cache, int n_tokens, sas_bf16* k, sas_bf16* v,
                        const int32_t* cache_len, const int32_t* new_len, void* stream) {
  Shape sh;
  sas::kv4::Cache c;
  const sas_status r = check_cache(p, cache, k != nullptr, v != nullptr, &sh, &c);
  if (r != SAS_OK) return r;
  if (!ok_tokens(sh, n_tokens, cache_len, new_len) || !ok_opt(k) || !ok_opt(v) || (k == nullptr && v == nullptr))
    return SAS_ERR_INVALID_ARG;
  return from_cuda(sas::launch_kv4_read(sh, c, n_tokens, k, v, cache_len, new_len, sas::error_word(),
                                        static_cast<cudaStream_t>(stream)));
}

sas_status sas_kv4_block_mean_keys(const sas_params* p, const sas_kv4_cache* cache, int n_tokens,
                                   const int32_t* cache_len, const int32_t* new_len, sas_bf16* kmean, void* stream) {
  Shape sh;
  sas::kv4::Cache c;
  const sas_status r = check_cache(p, cache, true, false, &sh, &c);
  if (r != SAS_OK) return r;
  if (!ok_tokens(sh, n_tokens, cache_len, new_len) || !ok_ptr(kmean)) return SAS_ERR_INVALID_ARG;
  return from_cuda(sas::launch_kv4_means(sh, c, n_tokens, cache_len, new_len, kmean, sas::error_word(),
                                         static_cast<cudaStream_t>(stream)));
}

sas_status sas_decode_kv4(const sas_params* p, const sas_bf16* q, const sas_kv4_cache* cache,
                          const int32_t* cache_len, const float* s, const int32_t* idx, const float* lse_s,
                          int n_split, float* o_part, float* lse_part, void* stream) {
  Shape sh;
  sas::kv4::Cache c;
  const sas_status r = check_cache(p, cache, true, true, &sh, &c);
  if (r != SAS_OK) return r;
  if (sh.G > 8) return SAS_ERR_UNSUPPORTED;
  if (!ok_ptr(q) || !ok_ptr(cache_len) || !ok_ptr(idx) || !ok_ptr(o_part) || !ok_ptr(lse_part))
    return SAS_ERR_INVALID_ARG;
  if (sh.gated && (!ok_ptr(s) || !ok_opt(lse_s))) return SAS_ERR_INVALID_ARG;
  if ((sh.gate == SAS_GATE_LOG_SOFTMAX || sh.gate == SAS_GATE_SOFTMAX_OUTSIDE) && lse_s == nullptr)
    return SAS_ERR_INVALID_ARG;
  if (n_split < 1 || n_split > sh.K + 1 || n_split > 65535) return SAS_ERR_INVALID_ARG;
  if ((sh.K + n_split) / n_split > sas::kMaxDecodeBlocksPerSplit) return SAS_ERR_UNSUPPORTED;
  if (int64_t(sh.B) * sh.Hkv * n_split > (int64_t(1) << 31) - 1) return SAS_ERR_UNSUPPORTED;
  return from_cuda(sas::launch_decode_kv4(sh, q, c, cache_len, sh.gated ? s : nullptr, idx,
                                          sh.gated ? lse_s : nullptr, n_split, o_part, lse_part, sas::error_word(),
                                          static_cast<cudaStream_t>(stream)));
}

sas_status sas_decode_fused_kv4(const sas_params* p, const sas_bf16* q, const sas_kv4_cache* cache,
                                const int32_t* cache_len, const float* s, int32_t* idx, float* lse_s, sas_bf16* o,
                                float* lse_o, void* stream) {
  Shape sh;
  sas::kv4::Cache c;
  const sas_status r = check_cache(p, cache, true, true, &sh, &c);
  if (r != SAS_OK) return r;
  if (!sas::decode_fused_fits(sh)) return SAS_ERR_UNSUPPORTED;
  if (!ok_ptr(q) || !ok_ptr(cache_len) || !ok_ptr(s) || !ok_ptr(o) || !ok_opt(idx) || !ok_opt(lse_s) || !ok_opt(lse_o))
    return SAS_ERR_INVALID_ARG;
  return from_cuda(sas::launch_decode_fused_kv4(sh, q, c, cache_len, s, idx, lse_s, o, lse_o, sas::error_word(),
                                                static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
