// Device helpers of the learner operators (norm.cu, logprob.cu, distill.cu):
// rows of logits of any alignment, and softmax statistics about a running
// maximum.
#pragma once

#include "../../include/moe_learner.h"
#include "common.cuh"
#include "kernels.cuh"

namespace moe {

// ---- arguments of the launches ----
struct NormArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* res;
  int64_t ldr;
  const uint16_t* w;
  float eps;
  int T, d;
  uint16_t* h;
  uint16_t* y;
  uint8_t* y8;
  uint8_t* sf;
  float* rstd;
  int* status;
};
struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* dh;
  const uint16_t* h;
  const float* rstd;
  const uint16_t* w;
  int T, d;
  uint16_t* dx;
  float* dw;
  float* part;  // dw of each block, [blocks][d]
};
struct LogprobArgs {
  const void* logits;
  int dtype;
  int64_t ld;
  int T, V;
  const int32_t* targets;
  float inv_t;
  int n_top;
  float* logprob;
  float* entropy;
  float* stats;
  int32_t* top_ids;
  float* top_logprob;
  int* status;
};
struct LogprobBwdArgs {
  const void* logits;
  int dtype;
  int64_t ld;
  int T, V;
  const int32_t* targets;
  float inv_t;
  const float* stats;
  const float* entropy;
  const float* g_logprob;
  const float* g_entropy;
  void* dlogits;
  int64_t ldd;
  int* status;
};
// loss NULL: the gradient from `stats`; dlogits NULL: the loss alone.
struct DistillArgs {
  const void* logits;
  int dtype;
  int64_t ld;
  int T, V;
  const int32_t* teacher_ids;
  const float* teacher_logits;
  const float* teacher_lse;
  int K;
  float inv_t;
  float* loss;
  float* stats_out;
  const float* stats;
  const float* g;
  void* dlogits;
  int64_t ldd;
  int* status;
};
int launch_add_rmsnorm(const NormArgs& a, cudaStream_t s);
size_t add_rmsnorm_backward_ws(int T, int d);
int launch_add_rmsnorm_backward(const NormBwdArgs& a, cudaStream_t s);
int launch_token_logprobs(const LogprobArgs& a, cudaStream_t s);
int launch_token_logprobs_backward(const LogprobBwdArgs& a, cudaStream_t s);
int launch_distill(const DistillArgs& a, cudaStream_t s);

constexpr float kLowest = -3.402823466e+38f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7FFFFFFFu); }

// Larger of two floats, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// 2^x, results below 2^-126 flushed to zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row of V elements as `head` elements up to the first 16-byte boundary,
// `nvec` vectors of 16 bytes, and `tail` elements after them.
template <typename E>
struct Row {
  static constexpr int kVec = 16 / (int)sizeof(E);
  const E* p;
  int head, nvec, tail;
  __device__ __forceinline__ Row(const E* row, int V) : p(row) {
    const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(E));
    head = mis == 0 ? 0 : min(V, kVec - mis);
    nvec = (V - head) / kVec;
    tail = V - head - nvec * kVec;
  }
  __device__ __forceinline__ const uint4* vec() const { return reinterpret_cast<const uint4*>(p + head); }
  __device__ __forceinline__ int tail_start() const { return head + nvec * kVec; }
};

__device__ __forceinline__ float to_f32(uint16_t b) { return bf16_bits_to_f32(b); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(float v, uint16_t& o) { o = (uint16_t)f32_to_bf16_bits(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }

// The elements of a 16-byte vector.
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// Softmax statistics of a set of logits: m their maximum (kLowest for none
// but -inf, NaN with a NaN), s = sum 2^((x - m) c), and with ENT e = sum
// 2^((x - m) c) (x - m), where c = inv_temperature log2(e).  The differences
// are formed before the product, so that logits of any finite size (masks at
// the type's lowest value among them) give finite exponents; x - m is held at
// -1e30 at least where it multiplies a weight, so that -inf gives 0 and not
// NaN.
template <bool ENT>
struct Soft {
  float m = kLowest, s = 0.0f, e = 0.0f;
  __device__ __forceinline__ void rescale(float nm, float c) {
    const float d = m - nm;
    const float f = exp2_fast(d * c);
    if (ENT) e = f * (e + s * fmaxf(d, -1e30f));
    s *= f;
    m = nm;
  }
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N], float c) {
    float nm = m;
#pragma unroll
    for (int i = 0; i < N; ++i) nm = max_nan(nm, x[i]);
    rescale(nm, c);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = x[i] - nm;
      const float w = exp2_fast(d * c);
      s += w;
      if (ENT) e = fmaf(w, fmaxf(d, -1e30f), e);
    }
  }
  __device__ __forceinline__ void merge(const Soft& o, float c) {
    const float nm = max_nan(m, o.m);
    Soft b = o;
    rescale(nm, c);
    b.rescale(nm, c);
    s += b.s;
    e += b.e;
  }
  __device__ __forceinline__ Soft shfl_xor(int o) const {
    Soft b;
    b.m = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    b.s = __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (ENT) b.e = __shfl_xor_sync(0xFFFFFFFFu, e, o);
    return b;
  }
  __device__ __forceinline__ void warp_merge(float c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      // both lanes of a pair merge in the same order, so all lanes agree
      const Soft b = shfl_xor(o);
      if (threadIdx.x & o) {
        Soft t = b;
        t.merge(*this, c);
        *this = t;
      } else {
        merge(b, c);
      }
    }
  }
  // Merged over the block's NW warps; every thread gets the result.
  template <int NW>
  __device__ __forceinline__ void block_merge(float c, Soft* red) {
    warp_merge(c);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = *this;
    __syncthreads();
    Soft b;
    if ((threadIdx.x & 31) < NW) b = red[threadIdx.x & 31];
    b.warp_merge(c);
    *this = b;
    __syncthreads();
  }
};

// Sum over the block's NW warps in a fixed order; every thread gets it.
template <int NW>
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < NW ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  return v;
}

// Order of the alternatives: larger logit first, then the lower id.
// -0 and +0 are equal.
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t id) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)o << 32) | (0xFFFFFFFFu - id);
}
__device__ __forceinline__ float rank_logit(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int rank_id(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

}  // namespace moe
