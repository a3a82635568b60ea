// Log-probabilities of given tokens with entropy and top alternatives, and
// their gradient.
#include "learner.cuh"

namespace moe {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;
constexpr int kLpBatch = 4;     // 16-byte loads a thread has in flight
constexpr int kLpPending = 64;  // candidates a warp holds before it sorts them

__device__ __forceinline__ bool finite_max(float m) { return m <= 3.402823466e+38f; }  // not NaN, not +inf

// The alternatives of a block's part of the row, from the threads' maxima: the
// n-th largest of them is a lower bound of the n-th largest logit, so only the
// threads that reach it (about n of them) hold candidates, and only their
// vectors are read again (from L2).  Each warp takes its own threads one by
// one, a vector per lane; candidates wait in shared memory until there are 32
// to sort into the warp's list.  Returns the block's list in warp 0.
template <typename E>
struct TopShared {
  uint64_t lists[kLpWarps][32];
  uint32_t vals[kLpWarps][32];
  uint64_t pending[kLpWarps][kLpPending];
  uint32_t bound;
};

template <typename E>
__device__ __forceinline__ uint64_t block_top(const Row<E>& r, int v0, int v1, bool ends, float tmax, int n,
                                              TopShared<E>& sh) {
  constexpr int N = Row<E>::kVec;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mine = rank_value(tmax);
  const uint32_t top = block_list_merge<kLpWarps>(list_sort(mine), sh.vals);
  if (warp == 0 && lane == n - 1) sh.bound = top;
  __syncthreads();
  const uint32_t bound = sh.bound;

  uint64_t list = 0, least = (uint64_t)bound << 32;  // keys below `least` cannot enter
  uint64_t* pend = sh.pending[warp];
  int held = 0;
  auto flush = [&](int k) {  // sort the first k <= 32 pending keys into the list
    __syncwarp();
    const uint64_t key = lane < k ? pend[lane] : 0;
    const uint64_t rest = lane + 32 < held ? pend[lane + 32] : 0;
    __syncwarp();
    if (lane + 32 < held) pend[lane] = rest;
    held = held > 32 ? held - 32 : 0;
    list = list_merge(list, list_sort(key));
    const uint64_t nth = __shfl_sync(0xFFFFFFFFu, list, n - 1);
    least = max(least, nth);
    __syncwarp();
  };
  auto offer = [&](float x, int id, bool valid) {
    const uint64_t key = rank_key(x, (uint32_t)id);
    const bool in = valid && x != neg_inf() && key >= least;
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
    if (who == 0) return;
    if (in) pend[held + __popc(who & ((1u << lane) - 1))] = key;
    held += __popc(who);
    if (held >= 32) flush(32);
  };
  uint32_t hot = __ballot_sync(0xFFFFFFFFu, mine >= bound);
  while (hot) {
    const int h = __ffs(hot) - 1;
    hot &= hot - 1;
    for (int i0 = v0 + warp * 32 + h; i0 < v1; i0 += 32 * kLpThreads) {
      const int i = i0 + lane * kLpThreads;
      const bool valid = i < v1;
      float x[N];
      unpack(__ldg(r.vec() + (valid ? i : i0)), x);
#pragma unroll
      for (int e = 0; e < N; ++e) offer(x[e], r.head + i * N + e, valid);
    }
  }
  if (warp == 0 && ends) {  // the elements outside the vectors
    const bool a = lane < r.head, b = lane < r.tail;
    offer(a ? to_f32(r.p[lane]) : 0.0f, lane, a);
    offer(b ? to_f32(r.p[r.tail_start() + lane]) : 0.0f, r.tail_start() + lane, b);
  }
  if (held) flush(held);
  return block_list_merge<kLpWarps>(list, sh.lists);
}

// One row per cluster of gridDim.x blocks, each a contiguous part of its
// vectors.  A thread keeps its own running maximum and sums (one pass, no
// exchange until the end); the parts meet in the cluster's first block through
// distributed shared memory.
template <typename E, bool ENT, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 2) token_logprobs_kernel(LogprobArgs a) {
  __shared__ Soft<ENT> red[kLpWarps];
  __shared__ Soft<ENT> part;
  __shared__ uint64_t plist[32];
  const int nb = gridDim.x, rank = blockIdx.x;
  const int64_t t = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  if (t >= a.T) return;  // the whole cluster
  const E* row = static_cast<const E*>(a.logits) + t * a.ld;
  const Row<E> r(row, a.V);
  const int v0 = (int)((int64_t)r.nvec * rank / nb), v1 = (int)((int64_t)r.nvec * (rank + 1) / nb);
  const float c = a.inv_t * kLog2e;
  Soft<ENT> acc;
  const uint4* vec = r.vec();
  int i = v0 + threadIdx.x;
  for (; i + (kLpBatch - 1) * kLpThreads < v1; i += kLpBatch * kLpThreads) {
    uint4 v[kLpBatch];
#pragma unroll
    for (int u = 0; u < kLpBatch; ++u) v[u] = TOP ? __ldg(vec + i + u * kLpThreads) : __ldcs(vec + i + u * kLpThreads);
    acc.add_batch(v, c, E());
  }
  for (; i < v1; i += kLpThreads) {
    const uint4 v[1] = {__ldg(vec + i)};
    acc.add_batch(v, c, E());
  }
  if (rank == 0) {
    if ((int)threadIdx.x < r.head) {
      const float x[1] = {to_f32(row[threadIdx.x])};
      acc.add(x, c);
    }
    if ((int)threadIdx.x < r.tail) {
      const float x[1] = {to_f32(row[r.tail_start() + threadIdx.x])};
      acc.add(x, c);
    }
  }
  const float tmax = acc.m;
  acc.template block_merge<kLpWarps>(c, red);
  uint64_t list = 0;
  if (TOP) {
    __shared__ TopShared<E> top;
    if (finite_max(acc.m) && acc.s > 0.0f) list = block_top(r, v0, v1, rank == 0, tmax, a.n_top, top);
  }
  if (nb > 1) {
    if (threadIdx.x == 0) part = acc;
    if (TOP && threadIdx.x < 32) plist[threadIdx.x] = list;
    cluster_arrive();
    cluster_wait();
    if (rank == 0 && threadIdx.x < 32) {
      for (int b = 1; b < nb; ++b) {
        Soft<ENT> o;
        o.m = cluster_load_f32(&part.m, b);
        o.s = cluster_load_f32(&part.s, b);
        if (ENT) o.e = cluster_load_f32(&part.e, b);
        acc.merge(o, c);
        if (TOP) {
          const uint32_t* p = reinterpret_cast<const uint32_t*>(&plist[threadIdx.x]);
          const uint64_t lo = cluster_load(p, b), hi = cluster_load(p + 1, b);
          list = list_merge(list, lo | (hi << 32));
        }
      }
    }
    cluster_arrive();  // the other blocks' shared memory is read no more
    cluster_wait();
  }
  if (rank != 0 || threadIdx.x >= 32) return;
  const bool bad = !finite_max(acc.m), none = acc.s == 0.0f;
  const float l = logf(acc.s), nan = quiet_nan();
  if (threadIdx.x == 0) {
    if (bad) set_status(a.status, MOE_STATUS_NONFINITE_LOGITS);
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
  if (TOP && (int)threadIdx.x < a.n_top) {
    if (bad) list = 0;
    a.top_ids[t * a.n_top + threadIdx.x] = list ? rank_id(list) : -1;
    a.top_logprob[t * a.n_top + threadIdx.x] =
        bad ? nan : list ? (rank_logit(list) - acc.m) * a.inv_t - l : neg_inf();
  }
}

// d_v = inv_t (p_v (A - g_ent ln p_v) + g 1[v = target]), A = -g - g_ent H.
// blockIdx.x a part of the row.
constexpr int kLbThreads = 256;
constexpr int kLbBatch = 4;

template <typename E>
__global__ void __launch_bounds__(kLbThreads) token_logprobs_backward_kernel(LogprobBwdArgs a) {
  constexpr int N = Row<E>::kVec;
  const int64_t t = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  if (t >= a.T) return;
  const E* row = static_cast<const E*>(a.logits) + t * a.ld;
  E* out = static_cast<E*>(a.dlogits) + t * a.ldd;
  const int y = a.targets ? a.targets[t] : -1;
  if (y >= a.V && threadIdx.x == 0 && blockIdx.x == 0) set_status(a.status, MOE_STATUS_BAD_TOKEN);
  const bool has = y >= 0 && y < a.V;
  const float g = has && a.g_logprob ? a.g_logprob[t] * a.inv_t : 0.0f;
  const float ge = a.g_entropy ? a.g_entropy[t] * a.inv_t : 0.0f;
  const float m = a.stats[2 * t], l = a.stats[2 * t + 1];
  const bool zero = m == neg_inf() || (g == 0.0f && ge == 0.0f);
  const float A = -g - (a.g_entropy ? ge * a.entropy[t] : 0.0f);
  // -inf gives p = 0 times a finite number; a NaN row's l makes all its values NaN
  auto grad = [&](float x) {
    const float lp = fmaxf((x - m) * a.inv_t, -1e30f) - l;
    return exp2_fast(lp * kLog2e) * fmaf(-ge, lp, A);
  };
  const Row<E> r(row, a.V);
  if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
    const int nb = gridDim.x, b = blockIdx.x;
    const int v0 = (int)((int64_t)r.nvec * b / nb), v1 = (int)((int64_t)r.nvec * (b + 1) / nb);
    uint4* ov = reinterpret_cast<uint4*>(out + r.head);
    const int yv = has && y >= r.head ? (y - r.head) / N : -1, ye = (y - r.head) % N;
    auto store = [&](const uint4& v, int i) {
      float x[N];
      unpack(v, x);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = grad(x[e]);
      if (i == yv) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e == ye) x[e] += g;
      }
      __stcs(ov + i, pack(x));
    };
    int i = v0 + threadIdx.x;
    if (zero) {
      for (; i < v1; i += kLbThreads) __stcs(ov + i, make_uint4(0u, 0u, 0u, 0u));
    } else {
      for (; i + (kLbBatch - 1) * kLbThreads < v1; i += kLbBatch * kLbThreads) {
        uint4 v[kLbBatch];
#pragma unroll
        for (int u = 0; u < kLbBatch; ++u) v[u] = __ldcs(r.vec() + i + u * kLbThreads);
#pragma unroll
        for (int u = 0; u < kLbBatch; ++u) store(v[u], i + u * kLbThreads);
      }
      for (; i < v1; i += kLbThreads) store(__ldcs(r.vec() + i), i);
    }
    if (b == 0) {
      const int k = threadIdx.x < (unsigned)r.head ? (int)threadIdx.x
                                                   : r.tail_start() + (int)threadIdx.x - r.head;
      if ((int)threadIdx.x < r.head + r.tail) {
        const float v = zero ? 0.0f : grad(to_f32(row[k])) + (k == y ? g : 0.0f);
        from_f32(v, out[k]);
      }
    }
  } else {  // rows of different alignment: element by element
    const int64_t per = (a.V + gridDim.x - 1) / gridDim.x, k0 = per * blockIdx.x;
    const int64_t k1 = k0 + per < a.V ? k0 + per : a.V;
    for (int64_t k = k0 + threadIdx.x; k < k1; k += kLbThreads) {
      const float v = zero ? 0.0f : grad(to_f32(row[k])) + (k == y ? g : 0.0f);
      from_f32(v, out[k]);
    }
  }
}

// host launchers
int launch_token_logprobs(const LogprobArgs& a, cudaStream_t s) {
  // Blocks per row: one where the rows alone fill two blocks per SM, else as
  // many (up to 8, a portable cluster) as do, while each keeps a batch of
  // loads per thread.
  const int64_t nvec = (int64_t)a.V * (a.dtype == MOE_DTYPE_BF16 ? 2 : 4) / 16;
  int nb = 1;
  while (nb < 8 && (int64_t)a.T * nb < 304 && nvec / (nb * 2) >= kLpThreads) nb *= 2;
  const unsigned gy = a.T < 65535 ? a.T : 65535, gz = (a.T + gy - 1) / gy;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nb, gy, gz);
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = nb;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = nb > 1 ? 1 : 0;
  const bool ent = a.entropy != nullptr, top = a.n_top > 0;
  void (*f)(LogprobArgs);
  if (a.dtype == MOE_DTYPE_BF16)
    f = ent ? (top ? token_logprobs_kernel<uint16_t, true, true> : token_logprobs_kernel<uint16_t, true, false>)
            : (top ? token_logprobs_kernel<uint16_t, false, true> : token_logprobs_kernel<uint16_t, false, false>);
  else
    f = ent ? (top ? token_logprobs_kernel<float, true, true> : token_logprobs_kernel<float, true, false>)
            : (top ? token_logprobs_kernel<float, false, true> : token_logprobs_kernel<float, false, false>);
  return cudaLaunchKernelEx(&cfg, f, a) == cudaSuccess ? 0 : -1;
}
int launch_token_logprobs_backward(const LogprobBwdArgs& a, cudaStream_t s) {
  const int64_t nvec = (int64_t)a.V * (a.dtype == MOE_DTYPE_BF16 ? 2 : 4) / 16;
  const int64_t per = kLbThreads * kLbBatch * 2;
  const unsigned nb = (unsigned)(nvec < per ? 1 : (nvec + per - 1) / per);
  const unsigned gy = a.T < 65535 ? a.T : 65535, gz = (a.T + gy - 1) / gy;
  const dim3 grid(nb, gy, gz);
  if (a.dtype == MOE_DTYPE_BF16) token_logprobs_backward_kernel<uint16_t><<<grid, kLbThreads, 0, s>>>(a);
  else token_logprobs_backward_kernel<float><<<grid, kLbThreads, 0, s>>>(a);
  return 0;
}

}  // namespace moe
