// Log-probabilities of given tokens with entropy and top alternatives, and
// their gradient.
#include "learner.cuh"

namespace moe {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;

template <typename E, bool ENT>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_kernel(LogprobArgs a) {
  __shared__ Soft<ENT> red[kLpWarps];
  __shared__ uint64_t kred[kLpWarps];
  const int64_t t = blockIdx.x;
  const E* row = static_cast<const E*>(a.logits) + t * a.ld;
  const Row<E> r(row, a.V);
  const float c = a.inv_t * kLog2e;
  Soft<ENT> acc;
  for (int i = threadIdx.x; i < r.nvec; i += kLpThreads) {
    float x[Row<E>::kVec];
    unpack(__ldcs(r.vec() + i), x);
    acc.add(x, c);
  }
  if ((int)threadIdx.x < r.head) {
    const float x[1] = {to_f32(row[threadIdx.x])};
    acc.add(x, c);
  }
  if ((int)threadIdx.x < r.tail) {
    const float x[1] = {to_f32(row[r.tail_start() + threadIdx.x])};
    acc.add(x, c);
  }
  acc.template block_merge<kLpWarps>(c, red);
  const bool bad = !(acc.m <= 3.402823466e+38f);  // NaN or +inf
  const bool none = acc.s == 0.0f;
  const float l = logf(acc.s);
  if (threadIdx.x == 0) {
    if (bad) set_status(a.status, MOE_STATUS_NONFINITE_LOGITS);
    const float nan = quiet_nan();
    if (a.logprob) {
      const int y = a.targets[t];
      if (y >= a.V) set_status(a.status, MOE_STATUS_BAD_TOKEN);
      float lp = 0.0f;
      if (y >= 0 && y < a.V) lp = bad ? nan : none ? neg_inf() : (to_f32(row[y]) - acc.m) * a.inv_t - l;
      a.logprob[t] = lp;
    }
    if (ENT) a.entropy[t] = bad ? nan : none ? 0.0f : l - a.inv_t * (acc.e / acc.s);
    if (a.stats) {
      a.stats[2 * t] = bad ? nan : none ? neg_inf() : acc.m;
      a.stats[2 * t + 1] = bad ? nan : none ? 0.0f : l;
    }
  }
  // alternatives: n_top passes, each for the first key after the one before
  uint64_t last = ~0ull;
  for (int j = 0; j < a.n_top; ++j) {
    uint64_t best = 0;
    for (int i = threadIdx.x; i < a.V && !bad; i += kLpThreads) {
      const float x = to_f32(row[i]);
      const uint64_t k = x == neg_inf() ? 0 : rank_key(x, (uint32_t)i);
      if (k < last && k > best) best = k;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
    if ((threadIdx.x & 31) == 0) kred[threadIdx.x >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kLpWarps; ++w) best = max(best, kred[w]);
    __syncthreads();
    if (threadIdx.x == 0) {
      a.top_ids[t * a.n_top + j] = best ? rank_id(best) : -1;
      a.top_logprob[t * a.n_top + j] =
          bad ? quiet_nan() : best ? (rank_logit(best) - acc.m) * a.inv_t - l : neg_inf();
    }
    last = best ? best : 1;  // 1: nothing follows
  }
}

// One block per row: d_v = inv_t (p_v (A + B (ln p_v + H)) + g 1[v = target])
// with A = -g, B = -g_ent.
template <typename E>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_backward_kernel(LogprobBwdArgs a) {
  const int64_t t = blockIdx.x;
  const E* row = static_cast<const E*>(a.logits) + t * a.ld;
  E* out = static_cast<E*>(a.dlogits) + t * a.ldd;
  const int y = a.targets ? a.targets[t] : -1;
  if (y >= a.V && threadIdx.x == 0) set_status(a.status, MOE_STATUS_BAD_TOKEN);
  const bool has = y >= 0 && y < a.V;
  const float g = has && a.g_logprob ? a.g_logprob[t] : 0.0f;
  const float ge = a.g_entropy ? a.g_entropy[t] : 0.0f;
  const float m = a.stats[2 * t], l = a.stats[2 * t + 1];
  const bool zero = m == neg_inf() || (g == 0.0f && ge == 0.0f);
  const float H = a.g_entropy ? a.entropy[t] : 0.0f;
  const float A = -g - ge * H;
  for (int i = threadIdx.x; i < a.V; i += kLpThreads) {
    float v = 0.0f;
    if (!zero) {
      const float lp = fmaxf((to_f32(row[i]) - m) * a.inv_t, -1e30f) - l;
      v = exp2_fast(lp * kLog2e) * (A - ge * lp);
      if (i == y) v += g;
      v *= a.inv_t;
      if (!(m <= 3.402823466e+38f)) v = quiet_nan();
    }
    from_f32(v, out[i]);
  }
}

// host launchers
int launch_token_logprobs(const LogprobArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.T);
  if (a.dtype == MOE_DTYPE_BF16) {
    if (a.entropy) token_logprobs_kernel<uint16_t, true><<<grid, kLpThreads, 0, s>>>(a);
    else token_logprobs_kernel<uint16_t, false><<<grid, kLpThreads, 0, s>>>(a);
  } else {
    if (a.entropy) token_logprobs_kernel<float, true><<<grid, kLpThreads, 0, s>>>(a);
    else token_logprobs_kernel<float, false><<<grid, kLpThreads, 0, s>>>(a);
  }
  return 0;
}
int launch_token_logprobs_backward(const LogprobBwdArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.T);
  if (a.dtype == MOE_DTYPE_BF16) token_logprobs_backward_kernel<uint16_t><<<grid, kLpThreads, 0, s>>>(a);
  else token_logprobs_backward_kernel<float><<<grid, kLpThreads, 0, s>>>(a);
  return 0;
}

}  // namespace moe
