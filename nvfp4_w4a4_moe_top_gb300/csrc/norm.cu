// Residual add + RMS norm with BF16 and block-scaled 8-bit outputs, and its
// gradient.
#include "learner.cuh"

namespace moe {

constexpr int kNmThreads = 256, kNmWarps = kNmThreads / 32;
constexpr int kNmBwdBlocks = 304;

// Scale byte of a block from its largest magnitude: the smallest power of two
// S with amax / S <= 448 = 0.875 * 2^9, as its exponent + 127.
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  // amax = 2^(e - 127) (1 + f): S = 2^(e - 127 - 8), one more where 1 + f > 1.75
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 0);
}
// 1 / 2^(byte - 127)
__device__ __forceinline__ float mx_scale_inv(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__global__ void __launch_bounds__(kNmThreads) add_rmsnorm_kernel(NormArgs a) {
  __shared__ float red[kNmWarps];
  const int64_t t = blockIdx.x;
  const uint16_t* x = a.x + t * a.ldx;
  const uint16_t* rs = a.res ? a.res + t * a.ldr : nullptr;
  extern __shared__ float hrow[];
  float ss = 0.0f;
  bool bad = false;
  for (int i = threadIdx.x; i < a.d; i += kNmThreads) {
    uint32_t hb = x[i];
    if (rs) hb = f32_to_bf16_bits(bf16_bits_to_f32(hb) + bf16_bits_to_f32(rs[i]));
    const float h = bf16_bits_to_f32(hb);
    if (a.h) a.h[t * a.d + i] = (uint16_t)hb;
    bad |= !is_finite_f32(h);
    hrow[i] = h;
    ss = fmaf(h, h, ss);
  }
  if (bad) set_status(a.status, MOE_STATUS_NONFINITE_X);
  ss = block_sum<kNmWarps>(ss, red);
  const float rstd = 1.0f / sqrtf(ss / (float)a.d + a.eps);
  if (threadIdx.x == 0 && a.rstd) a.rstd[t] = rstd;
  for (int i0 = 0; i0 < a.d; i0 += kNmThreads) {
    const int i = i0 + threadIdx.x;
    const float y = i < a.d ? hrow[i] * rstd * bf16_bits_to_f32(a.w[i]) : 0.0f;
    if (a.y && i < a.d) a.y[t * a.d + i] = (uint16_t)f32_to_bf16_bits(y);
    if (a.y8) {
      const float amax = warp_max(fabsf(y));
      const uint32_t sb = mx_scale_byte(amax);
      if (i < a.d) {
        a.y8[t * a.d + i] = (uint8_t)(e4m3x2_hw(y * mx_scale_inv(sb), 0.0f) & 0xFFu);
        if ((threadIdx.x & 31) == 0) a.sf[sf_tile_offset(t, i >> 5, a.d >> 7)] = (uint8_t)sb;
      }
    }
  }
}

__global__ void __launch_bounds__(kNmThreads) add_rmsnorm_backward_kernel(NormBwdArgs a) {
  __shared__ float red[kNmWarps];
  constexpr int kMax = 16384 / kNmThreads;
  float dw[kMax];
  for (int k = 0; k < kMax; ++k) dw[k] = 0.0f;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const float r = a.rstd[t];
    float c = 0.0f;
    for (int k = 0, i = threadIdx.x; i < a.d; ++k, i += kNmThreads) {
      const float n = bf16_bits_to_f32(a.h[t * a.d + i]) * r, dy = bf16_bits_to_f32(a.dy[t * a.d + i]);
      c = fmaf(dy * bf16_bits_to_f32(a.w[i]), n, c);
      dw[k] = fmaf(dy, n, dw[k]);
    }
    c = block_sum<kNmWarps>(c, red) / (float)a.d;
    for (int i = threadIdx.x; i < a.d; i += kNmThreads) {
      const float n = bf16_bits_to_f32(a.h[t * a.d + i]) * r, dy = bf16_bits_to_f32(a.dy[t * a.d + i]);
      float v = r * (dy * bf16_bits_to_f32(a.w[i]) - n * c);
      if (a.dh) v += bf16_bits_to_f32(a.dh[t * a.d + i]);
      a.dx[t * a.d + i] = (uint16_t)f32_to_bf16_bits(v);
    }
  }
  if (a.dw)
    for (int k = 0, i = threadIdx.x; i < a.d; ++k, i += kNmThreads) a.part[(int64_t)blockIdx.x * a.d + i] = dw[k];
}

__global__ void __launch_bounds__(kNmThreads) add_rmsnorm_dw_kernel(const float* part, int nb, int d, float* dw) {
  const int i = blockIdx.x * kNmThreads + threadIdx.x;
  if (i >= d) return;
  float s = 0.0f;
  for (int b = 0; b < nb; ++b) s += part[(int64_t)b * d + i];
  dw[i] = s;
}

// host launchers
size_t add_rmsnorm_backward_ws(int T, int d) { return (size_t)(T < kNmBwdBlocks ? T : kNmBwdBlocks) * d * 4; }

int launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  const int smem = a.d * 4;
  if (cudaFuncSetAttribute(add_rmsnorm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536) != cudaSuccess)
    return -1;
  add_rmsnorm_kernel<<<dim3((unsigned)a.T), kNmThreads, smem, s>>>(a);
  return 0;
}
int launch_add_rmsnorm_backward(const NormBwdArgs& a, cudaStream_t s) {
  const int nb = a.T < kNmBwdBlocks ? a.T : kNmBwdBlocks;
  add_rmsnorm_backward_kernel<<<dim3((unsigned)nb), kNmThreads, 0, s>>>(a);
  if (a.dw) add_rmsnorm_dw_kernel<<<dim3((unsigned)((a.d + 255) / 256)), kNmThreads, 0, s>>>(a.part, nb, a.d, a.dw);
  return 0;
}

}  // namespace moe
