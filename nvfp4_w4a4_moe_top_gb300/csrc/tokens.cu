// C ABI of the operators at the token ends (declared in include/moe_tokens.h):
// argument checks on the host and the launches.
#include "kernels.cuh"
#include "tokens.cuh"

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool req(const void* p, uintptr_t n) { return p != nullptr && aligned(p, n); }
inline bool opt(const void* p, uintptr_t n) { return aligned(p, n); }

int finish(int rc) {
  const cudaError_t e = cudaGetLastError();
  return rc == 0 && e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Rows ld >= d elements apart whose offsets stay far inside 64 bits.
bool rows_ok(int64_t ld, int rows, int d) { return ld >= d && ld <= (int64_t(1) << 46) / (rows > 0 ? rows : 1); }
bool type_ok(int dtype) { return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F32; }

bool embed_shape(int T, int V, int d) {
  return T >= 0 && V >= 1 && V <= MOE_EMBED_MAX_V && d >= 8 && d <= MOE_EMBED_MAX_D && d % 8 == 0;
}
bool finite(float x) { return x - x == 0.0f; }
constexpr int kMaxBackwardT = 1 << 24;

}  // namespace

extern "C" {

int moe_embed_tokens(const int32_t* ids, const void* table, int dtype, int64_t ldt, int T, int V, int d, float scale,
                     uint16_t* out, int64_t ldo, int* status, void* stream) {
  if (!type_ok(dtype) || !embed_shape(T, V, d) || !rows_ok(ldt, V, d) || ldt % 8 != 0 || !rows_ok(ldo, T, d) ||
      ldo % 8 != 0 || !finite(scale))
    return MOE_ERR_SHAPE;
  if (!opt(status, 4) || (T > 0 && (!req(ids, 4) || !req(table, 16) || !req(out, 16)))) return MOE_ERR_POINTER;
  const int rc = moe::check_device();
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  const moe::EmbedArgs a = {ids, table, dtype, ldt, T, V, d, scale, out, ldo, status};
  return finish(moe::launch_embed_tokens(a, (cudaStream_t)stream));
}

size_t moe_embed_tokens_backward_workspace_bytes(int T, int V, int d) {
  if (!embed_shape(T, V, d) || T > kMaxBackwardT) return 0;
  return moe::embed_tokens_backward_ws(T, V, d);
}

int moe_embed_tokens_backward(const uint16_t* dy, int64_t ldy, const int32_t* ids, int T, int V, int d, float scale,
                              int accumulate, float* dtable, void* ws, size_t ws_bytes, int* status, void* stream) {
  if (!embed_shape(T, V, d) || T > kMaxBackwardT || !rows_ok(ldy, T, d) || ldy % 8 != 0 || !finite(scale) ||
      (accumulate != 0 && accumulate != 1))
    return MOE_ERR_SHAPE;
  if (!req(dtable, 16) || !opt(status, 4) || !opt(ws, 16) || (T > 0 && (!req(dy, 16) || !req(ids, 4) || !ws)))
    return MOE_ERR_POINTER;
  if (T > 0 && ws_bytes < moe::embed_tokens_backward_ws(T, V, d)) return MOE_ERR_WORKSPACE;
  const int rc = moe::check_device();
  if (rc != MOE_OK) return rc;
  if (T == 0)
    return finish(accumulate || cudaMemsetAsync(dtable, 0, (size_t)V * d * 4, (cudaStream_t)stream) == cudaSuccess ? 0
                                                                                                               : -1);
  const moe::EmbedBwdArgs a = {dy, ldy, ids, T, V, d, scale, accumulate, dtable, static_cast<char*>(ws), status};
  return finish(moe::launch_embed_tokens_backward(a, (cudaStream_t)stream));
}

int moe_sample_tokens(const void* logits, int dtype, int64_t ld, int T, int V, const float* inv_temperature,
                      const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* tokens,
                      float* logprob, float* kept_logprob, int* status, void* stream) {
  if (!type_ok(dtype) || T < 0 || V < 1 || V > MOE_SAMPLE_MAX_V || !rows_ok(ld, T, V)) return MOE_ERR_SHAPE;
  if (!opt(inv_temperature, 4) || !opt(top_k, 4) || !opt(top_p, 4) || !opt(min_p, 4) || !opt(logprob, 4) ||
      !opt(kept_logprob, 4) || !opt(status, 4))
    return MOE_ERR_POINTER;
  if (T > 0 && (!req(logits, dtype == MOE_DTYPE_BF16 ? 2 : 4) || !req(u, 4) || !req(tokens, 4))) return MOE_ERR_POINTER;
  const int rc = moe::check_device();
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  const moe::SampleArgs a = {logits, dtype, ld, T,      V,       inv_temperature, top_k,
                             top_p,  min_p, u,  tokens, logprob, kept_logprob,    status};
  return finish(moe::launch_sample_tokens(a, (cudaStream_t)stream));
}

}  // extern "C"
