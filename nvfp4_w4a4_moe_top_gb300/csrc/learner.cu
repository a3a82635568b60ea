// C ABI of the learner operators (declared in include/moe_learner.h):
// argument checks on the host and the launches.
#include "kernels.cuh"
#include "learner.cuh"

bool moe::allow_smem(const void* kernel, int bytes, int most) {
  return bytes <= 16 * 1024 ||  // with the kernel's static share, within the 48 KB that need no asking
         (bytes <= most &&
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess);
}

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool req(const void* p, uintptr_t n) { return p != nullptr && aligned(p, n); }
inline bool opt(const void* p, uintptr_t n) { return aligned(p, n); }

int finish(int rc) {
  const cudaError_t e = cudaGetLastError();
  return rc == 0 && e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Rows ld >= V elements apart whose offsets stay far inside 64 bits.
bool rows_ok(int64_t ld, int T, int V) { return ld >= V && ld <= (int64_t(1) << 46) / (T > 0 ? T : 1); }

bool norm_shape(int T, int d) { return T >= 0 && d >= 16 && d <= 16384 && d % 16 == 0; }

// T, V, row strides, type and temperature of a logits call.
bool logits_shape(int dtype, int64_t ld, int T, int V, float inv_t) {
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) return false;
  if (T < 0 || V < 1 || V > (1 << 30) || !rows_ok(ld, T, V)) return false;
  return inv_t >= 1e-6f && inv_t <= 1e6f;  // false for NaN
}
uintptr_t esize(int dtype) { return dtype == MOE_DTYPE_BF16 ? 2 : 4; }

int distill(const void* logits, int dtype, int64_t ld, int T, int V, const int32_t* teacher_ids,
            const float* teacher_logits, const float* teacher_lse, int K, float inv_temperature, float* loss,
            float* stats_out, const float* stats, const float* g, void* dlogits, int64_t ldd, int* status,
            void* stream) {
  moe::DistillArgs a = {logits,          dtype, ld,        T,     V, teacher_ids, teacher_logits, teacher_lse, K,
                        inv_temperature, loss,  stats_out, stats, g, dlogits,     ldd,            status};
  const int rc = moe::check_device();
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  return finish(moe::launch_distill(a, (cudaStream_t)stream));
}

// The checks that the distillation entry points share.
int distill_check(const void* logits, int dtype, int64_t ld, int T, int V, const int32_t* teacher_ids,
                  const float* teacher_logits, const float* teacher_lse, int K, float inv_temperature, int* status) {
  if (!logits_shape(dtype, ld, T, V, inv_temperature) || V > MOE_DISTILL_MAX_V || K < 1 || K > MOE_DISTILL_MAX_K)
    return MOE_ERR_SHAPE;
  if (!opt(teacher_lse, 4) || !opt(status, 4)) return MOE_ERR_POINTER;
  if (T > 0 && (!req(logits, esize(dtype)) || !req(teacher_ids, 4) || !req(teacher_logits, 4))) return MOE_ERR_POINTER;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_mx8_sf_bytes(int64_t rows, int d) {
  if (rows < 0 || d < 128 || d % 128 != 0) return 0;
  return (size_t)((rows + 127) / 128) * (size_t)(d / 128) * 512;
}

int moe_add_rmsnorm(const uint16_t* x, int64_t ldx, const uint16_t* res, int64_t ldr, const uint16_t* w, float eps,
                    int T, int d, uint16_t* h, uint16_t* y, uint8_t* y8, uint8_t* y8_sf, float* rstd, int* status,
                    void* stream) {
  if (!norm_shape(T, d) || !rows_ok(ldx, T, d) || ldx % 8 != 0 || (res && (!rows_ok(ldr, T, d) || ldr % 8 != 0)) ||
      !(eps >= 0.0f) || !(eps <= 1e30f) || (y8 && d % 128 != 0))
    return MOE_ERR_SHAPE;
  if (!opt(res, 16) || !opt(h, 16) || !opt(y, 16) || !opt(y8, 16) || !opt(y8_sf, 16) || !opt(rstd, 4) ||
      !opt(status, 4) || (y8 == nullptr) != (y8_sf == nullptr))
    return MOE_ERR_POINTER;
  if (T > 0 && (!req(x, 16) || !req(w, 16) || (res && !h))) return MOE_ERR_POINTER;
  const int rc = moe::check_device();
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  const moe::NormArgs a = {x, ldx, res, ldr, w, eps, T, d, h, y, y8, y8_sf, rstd, status};
  return finish(moe::launch_add_rmsnorm(a, (cudaStream_t)stream));
}

size_t moe_add_rmsnorm_backward_workspace_bytes(int T, int d) {
  if (!norm_shape(T, d)) return 0;
  return moe::add_rmsnorm_backward_ws(T, d);
}

int moe_add_rmsnorm_backward(const uint16_t* dy, const uint16_t* dh, const uint16_t* h, const float* rstd,
                             const uint16_t* w, int T, int d, uint16_t* dx, float* dw, void* ws, size_t ws_bytes,
                             int* status, void* stream) {
  if (!norm_shape(T, d)) return MOE_ERR_SHAPE;
  if (!opt(dh, 16) || !opt(dw, 4) || !opt(ws, 16) || !opt(status, 4)) return MOE_ERR_POINTER;
  if (T > 0 && (!req(dy, 16) || !req(h, 16) || !req(rstd, 4) || !req(w, 16) || !req(dx, 16) || (dw && !ws)))
    return MOE_ERR_POINTER;
  if (dw && ws_bytes < moe::add_rmsnorm_backward_ws(T, d)) return MOE_ERR_WORKSPACE;
  const int rc = moe::check_device();
  if (rc != MOE_OK) return rc;
  if (T == 0)
    return finish(dw && cudaMemsetAsync(dw, 0, (size_t)d * 4, (cudaStream_t)stream) != cudaSuccess ? -1 : 0);
  const moe::NormBwdArgs a = {dy, dh, h, rstd, w, T, d, dx, dw, static_cast<float*>(ws), status};
  return finish(moe::launch_add_rmsnorm_backward(a, (cudaStream_t)stream));
}

int moe_token_logprobs(const void* logits, int dtype, int64_t ld, int T, int V, const int32_t* targets,
                       float inv_temperature, int n_top, float* logprob, float* entropy, float* stats,
                       int32_t* top_ids, float* top_logprob, int* status, void* stream) {
  if (!logits_shape(dtype, ld, T, V, inv_temperature) || n_top < 0 || n_top > MOE_LOGPROBS_MAX_TOP)
    return MOE_ERR_SHAPE;
  if (!opt(targets, 4) || !opt(logprob, 4) || !opt(entropy, 4) || !opt(stats, 4) || !opt(top_ids, 4) ||
      !opt(top_logprob, 4) || !opt(status, 4))
    return MOE_ERR_POINTER;
  if (T > 0 && (!req(logits, esize(dtype)) || (logprob && !targets) || (n_top > 0 && (!top_ids || !top_logprob))))
    return MOE_ERR_POINTER;
  const int rc = moe::check_device();
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  const moe::LogprobArgs a = {logits, dtype,   ld,    T,       V,           targets, inv_temperature,
                              n_top,  logprob, entropy, stats, top_ids, top_logprob, status};
  return finish(moe::launch_token_logprobs(a, (cudaStream_t)stream));
}

int moe_token_logprobs_backward(const void* logits, int dtype, int64_t ld, int T, int V, const int32_t* targets,
                                float inv_temperature, const float* stats, const float* entropy,
                                const float* g_logprob, const float* g_entropy, void* dlogits, int64_t ldd,
                                int* status, void* stream) {
  if (!logits_shape(dtype, ld, T, V, inv_temperature) || !rows_ok(ldd, T, V) ||
      (dlogits == logits && dlogits && ldd != ld))
    return MOE_ERR_SHAPE;
  if (!opt(targets, 4) || !opt(entropy, 4) || !opt(g_logprob, 4) || !opt(g_entropy, 4) || !opt(status, 4))
    return MOE_ERR_POINTER;
  if (T > 0 && (!req(logits, esize(dtype)) || !req(dlogits, esize(dtype)) || !req(stats, 4) ||
                (!g_logprob && !g_entropy) || (g_logprob && !targets) || (g_entropy && !entropy)))
    return MOE_ERR_POINTER;
  const int rc = moe::check_device();
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  const moe::LogprobBwdArgs a = {logits, dtype,   ld,        T,         V,       targets, inv_temperature,
                                 stats,  entropy, g_logprob, g_entropy, dlogits, ldd,     status};
  return finish(moe::launch_token_logprobs_backward(a, (cudaStream_t)stream));
}

int moe_distill_topk(const void* logits, int dtype, int64_t ld, int T, int V, const int32_t* teacher_ids,
                     const float* teacher_logits, const float* teacher_lse, int K, float inv_temperature, float* loss,
                     float* stats, int* status, void* stream) {
  const int rc =
      distill_check(logits, dtype, ld, T, V, teacher_ids, teacher_logits, teacher_lse, K, inv_temperature, status);
  if (rc != MOE_OK) return rc;
  if (!opt(stats, 16) || (T > 0 && !req(loss, 4))) return MOE_ERR_POINTER;
  return distill(logits, dtype, ld, T, V, teacher_ids, teacher_logits, teacher_lse, K, inv_temperature, loss, stats,
                 nullptr, nullptr, nullptr, 0, status, stream);
}

int moe_distill_topk_backward(const void* logits, int dtype, int64_t ld, int T, int V, const int32_t* teacher_ids,
                              const float* teacher_logits, const float* teacher_lse, int K, float inv_temperature,
                              const float* stats, const float* g, void* dlogits, int64_t ldd, int* status,
                              void* stream) {
  const int rc =
      distill_check(logits, dtype, ld, T, V, teacher_ids, teacher_logits, teacher_lse, K, inv_temperature, status);
  if (rc != MOE_OK) return rc;
  if (!rows_ok(ldd, T, V) || (dlogits == logits && dlogits && ldd != ld)) return MOE_ERR_SHAPE;
  if (T > 0 && (!req(dlogits, esize(dtype)) || !req(stats, 16) || !req(g, 4))) return MOE_ERR_POINTER;
  return distill(logits, dtype, ld, T, V, teacher_ids, teacher_logits, teacher_lse, K, inv_temperature, nullptr,
                 nullptr, stats, g, dlogits, ldd, status, stream);
}

int moe_distill_topk_train(const void* logits, int dtype, int64_t ld, int T, int V, const int32_t* teacher_ids,
                           const float* teacher_logits, const float* teacher_lse, int K, float inv_temperature,
                           const float* g, float* loss, void* dlogits, int64_t ldd, int* status, void* stream) {
  const int rc =
      distill_check(logits, dtype, ld, T, V, teacher_ids, teacher_logits, teacher_lse, K, inv_temperature, status);
  if (rc != MOE_OK) return rc;
  if (!rows_ok(ldd, T, V) || (dlogits == logits && dlogits && ldd != ld)) return MOE_ERR_SHAPE;
  if (T > 0 && (!req(dlogits, esize(dtype)) || !req(loss, 4) || !req(g, 4))) return MOE_ERR_POINTER;
  return distill(logits, dtype, ld, T, V, teacher_ids, teacher_logits, teacher_lse, K, inv_temperature, loss, nullptr,
                 nullptr, g, dlogits, ldd, status, stream);
}

}  // extern "C"
