// Distillation from a teacher's top logits: loss and gradient.
#include "learner.cuh"

namespace moe {

constexpr int kDsThreads = 512, kDsWarps = kDsThreads / 32;

// The teacher's entry of one thread (j = threadIdx.x < K): id < 0 where there
// is none.
struct Entry {
  int id;
  float a;
};

// Row scalars of the teacher.
struct Teacher {
  float q, lq;  // this thread's entry (q = 0 where there is none)
  float r, Q;   // mass off the list; total mass
};

// Reads entry j of row t and drops bad ids and repeats (the first stays).
// ids: shared, MOE_DISTILL_MAX_K ints.
__device__ __forceinline__ Entry load_entry(const DistillArgs& a, int64_t t, int* ids) {
  Entry en = {-1, 0.0f};
  const int j = threadIdx.x;
  if (j < a.K) {
    en.id = a.teacher_ids[t * a.K + j];
    en.a = a.teacher_logits[t * a.K + j];
    ids[j] = en.id;
  }
  __syncthreads();
  if (j < a.K && en.id >= 0) {
    bool ok = en.id < a.V;
    for (int i = 0; i < j && ok; ++i) ok = ids[i] != en.id;
    if (!ok) {
      set_status(a.status, MOE_STATUS_BAD_TOKEN);
      en.id = -1;
    } else if (!(en.a <= 3.402823466e+38f)) {
      set_status(a.status, MOE_STATUS_NONFINITE_LOGITS);
      en.a = quiet_nan();
    }
  }
  return en;
}

template <int NW>
__device__ __forceinline__ Teacher teacher_mass(const DistillArgs& a, int64_t t, const Entry& en, float* red,
                                                Soft<false>* sred) {
  Teacher T;
  const bool live = en.id >= 0;
  if (a.teacher_lse) {
    const float L = a.teacher_lse[t];
    if (!(fabsf(L) <= 3.402823466e+38f) && threadIdx.x == 0) set_status(a.status, MOE_STATUS_NONFINITE_LOGITS);
    T.lq = en.a * a.inv_t - L;
    T.q = live ? expf(T.lq) : 0.0f;
    const float sum = block_sum<NW>(T.q, red);
    T.r = max_nan(1.0f - sum, 0.0f);
    T.Q = T.r > 0.0f ? 1.0f : sum;
  } else {
    const float c = a.inv_t * kLog2e;
    Soft<false> acc;
    if (live) {
      const float x[1] = {en.a};
      acc.add(x, c);
    }
    acc.template block_merge<NW>(c, sred);
    T.lq = (en.a - acc.m) * a.inv_t - logf(acc.s);
    T.q = live && acc.s > 0.0f ? expf(T.lq) : 0.0f;
    if (live && !(acc.m <= 3.402823466e+38f)) T.q = T.lq = quiet_nan();
    T.r = 0.0f;
    T.Q = acc.s > 0.0f || !(acc.m <= 3.402823466e+38f) ? 1.0f : 0.0f;
  }
  return T;
}

struct DsShared {
  int ids[MOE_DISTILL_MAX_K];
  Soft<false> sred[kDsWarps];
  float red[kDsWarps];
};

// LOSS: the statistics and the loss; GRAD: the gradient, from the statistics
// just computed or (without LOSS) the stored ones.
template <typename E, bool LOSS, bool GRAD>
__global__ void __launch_bounds__(kDsThreads) distill_kernel(DistillArgs a) {
  extern __shared__ uint32_t listed[];  // one bit per id of the row
  __shared__ DsShared sh;
  const int64_t t = blockIdx.x;
  const E* row = static_cast<const E*>(a.logits) + t * a.ld;
  const float c = a.inv_t * kLog2e;
  for (int i = threadIdx.x; i < (a.V + 31) / 32; i += kDsThreads) listed[i] = 0;
  const Entry en = load_entry(a, t, sh.ids);
  const bool live = en.id >= 0;
  if (live) atomicOr(&listed[en.id >> 5], 1u << (en.id & 31));
  const float xs = live ? to_f32(row[en.id]) : 0.0f;
  const Teacher T = teacher_mass<kDsWarps>(a, t, en, sh.red, sh.sred);
  __syncthreads();

  float m, l, mt, lt;
  if (LOSS) {
    Soft<false> tail;
    for (int i = threadIdx.x; i < a.V; i += kDsThreads)
      if (!(listed[i >> 5] >> (i & 31) & 1)) {
        const float x[1] = {to_f32(row[i])};
        tail.add(x, c);
      }
    Soft<false> all;
    if (live) {
      const float x[1] = {xs};
      all.add(x, c);
    }
    tail.template block_merge<kDsWarps>(c, sh.sred);
    all.template block_merge<kDsWarps>(c, sh.sred);
    all.merge(tail, c);
    m = all.m, mt = tail.m;
    l = logf(all.s), lt = logf(tail.s);
    if (all.s == 0.0f) m = neg_inf(), l = 0.0f;
    if (tail.s == 0.0f) mt = neg_inf(), lt = 0.0f;
    if (!(all.m <= 3.402823466e+38f)) {
      m = l = mt = lt = quiet_nan();
      if (threadIdx.x == 0) set_status(a.status, MOE_STATUS_NONFINITE_LOGITS);
    }
  } else {
    const float4 st = *reinterpret_cast<const float4*>(a.stats + 4 * t);
    m = st.x, l = st.y, mt = st.z, lt = st.w;
  }
  const bool none = m == neg_inf();
  const float lp = (xs - m) * a.inv_t - l;                                             // ln p of this entry
  const float ls = mt == neg_inf() ? neg_inf() : (mt - m) * a.inv_t + lt - l;  // ln of the mass off the list
  if (LOSS) {
    float part = 0.0f;
    if (live && !(T.q == 0.0f)) part = none ? -neg_inf() : T.q * (T.lq - lp);
    float loss = block_sum<kDsWarps>(part, sh.red);
    if (!(T.r == 0.0f)) loss += none ? -neg_inf() : T.r * (logf(T.r) - ls);
    if (threadIdx.x == 0) {
      a.loss[t] = m == m ? loss : quiet_nan();
      if (a.stats_out) *reinterpret_cast<float4*>(a.stats_out + 4 * t) = make_float4(m, l, mt, lt);
    }
  }
  if (GRAD) {
    E* out = static_cast<E*>(a.dlogits) + t * a.ldd;
    const float g = a.g[t] * a.inv_t;
    const float off = mt == neg_inf() ? 0.0f : g * (expf(ls) * T.Q - T.r);
    for (int i = threadIdx.x; i < a.V; i += kDsThreads) {
      const float x = to_f32(row[i]);
      if (listed[i >> 5] >> (i & 31) & 1) continue;
      from_f32(none || mt == neg_inf() ? 0.0f : off * expf((x - mt) * a.inv_t - lt), out[i]);
    }
    if (live) from_f32(none ? 0.0f : g * (expf(lp) * T.Q - T.q), out[en.id]);
  }
}

// host launchers
template <typename E>
static int launch_distill_of(const DistillArgs& a, cudaStream_t s) {
  const int smem = (a.V + 31) / 32 * 4;
  void (*f)(DistillArgs) = a.loss ? (a.dlogits ? distill_kernel<E, true, true> : distill_kernel<E, true, false>)
                                  : distill_kernel<E, false, true>;
  if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -1;
  f<<<dim3((unsigned)a.T), kDsThreads, smem, s>>>(a);
  return 0;
}
int launch_distill(const DistillArgs& a, cudaStream_t s) {
  return a.dtype == MOE_DTYPE_BF16 ? launch_distill_of<uint16_t>(a, s) : launch_distill_of<float>(a, s);
}

}  // namespace moe
