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
  int* status;
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
// Lets a kernel use `bytes` of dynamic shared memory on the current device.
// `most` is what its largest launch needs: the limit is the kernel's own, not
// the launch's, so every call sets that one value, and a thread with a small
// launch takes nothing from another thread's large one.
bool allow_smem(const void* kernel, int bytes, int most);

int launch_add_rmsnorm(const NormArgs& a, cudaStream_t s);
size_t add_rmsnorm_backward_ws(int T, int d);
int launch_add_rmsnorm_backward(const NormBwdArgs& a, cudaStream_t s);
int launch_token_logprobs(const LogprobArgs& a, cudaStream_t s);
int launch_token_logprobs_backward(const LogprobBwdArgs& a, cudaStream_t s);
int launch_distill(const DistillArgs& a, cudaStream_t s);

// A launch whose grid may be set up while the stream's kernel before it ends,
// where that begins with begin_kernel as all kernels launched here do (after
// any other kernel, or a copy, it starts as launches do), in clusters of
// `cluster` blocks along x.
template <typename... P, typename... A>
int launch_kernel(void (*f)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, f, P(args)...) == cudaSuccess ? 0 : -1;
}
// First in every kernel, before any access to global memory: lets the next
// launch be set up once all of this grid runs, and waits until what the stream
// ran before is complete and visible.  Small calls in a row save most of a
// launch's latency.  What the kernels before may have written is then read by
// plain loads: a load through the read-only path might be moved ahead of the
// wait.
__device__ __forceinline__ void begin_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr float kLowest = -3.402823466e+38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The larger magnitude of each half, NaN if either is; the sign is of no use.
__device__ __forceinline__ uint32_t max_abs_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---- thread-block clusters: a row's blocks exchange their parts ----
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The 4 bytes at shared address p of block `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_load(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float cluster_load_f32(const float* p, uint32_t rank) {
  return __uint_as_float(cluster_load(p, rank));
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
  // The vectors; on a 16-byte boundary also where there are none.
  __device__ __forceinline__ const uint4* vec() const {
    return reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p + head) & ~(uintptr_t)15);
  }
  __device__ __forceinline__ int tail_start() const { return head + nvec * kVec; }
  // First vector of part `rank` of 2^shift parts; part 2^shift is the end.
  __device__ __forceinline__ int part(int rank, int shift) const {
    const int per = (nvec >> shift) + ((nvec & ((1 << shift) - 1)) != 0);
    return min(rank * per, nvec);
  }
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
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  return make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]), bf16x2_rn(x[6], x[7]));
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// Order of the alternatives: larger logit first, then the lower id.
// -0 and +0 are equal, and max_nan's NaN is above all numbers.
__device__ __forceinline__ uint32_t rank_value(float x) {
  uint32_t b = __float_as_uint(x);
  if (b == 0x80000000u) b = 0u;
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t id) {
  return ((uint64_t)rank_value(x) << 32) | (0xFFFFFFFFu - id);
}
__device__ __forceinline__ float rank_logit(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int rank_id(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

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
};

// Softmax statistics of a stream of logits, in base 2 about an integer shift:
// m the maximum, M >= ceil(m c) an integer, s = sum 2^(x c - M), and with ENT
// e = sum 2^(x c - M) (x c - M).  The exponent is one FMA, rounded once
// whatever the size of x c, and changing the shift multiplies by a power of
// two.  M stays at -2^20 or above, so parts of a row that hold only masks
// (-inf or the type's lowest value) add zeros.  Rows whose own maximum leaves
// |m c| above 2^20 need the differences formed first (Soft): see shift_ok.
// BF16 pairs are held at -2^100 at least for ENT, so that a zero weight meets
// a finite exponent.
constexpr float kShiftLimit = 1048576.0f;  // 2^20

template <bool ENT>
struct Run {
  float m = kLowest, M = -kShiftLimit, s = 0.0f, e = 0.0f;
  // Whether the sums may be used, for the row's c (m is the row's maximum).
  __device__ __forceinline__ bool shift_ok(float c) const { return fabsf(m * c) <= kShiftLimit; }
  __device__ __forceinline__ void shift(float nM) {
    const float d = M - nM;
    const float f = exp2_fast(d);
    if (ENT) e = f * fmaf(s, d, e);
    s *= f;
    M = nM;
  }
  __device__ __forceinline__ float raise(float x, float c) {
    m = max_nan(m, x);
    shift(fmaxf(ceilf(m * c), -kShiftLimit));
    return x;
  }
  static __device__ __forceinline__ void step(uint64_t x, uint64_t c2, uint64_t nM2, uint64_t& s2, uint64_t& e2) {
    const uint64_t t = fma_f32x2(x, c2, nM2);
    float a, b;
    unpack2(t, a, b);
    const uint64_t w = f32x2_pack(exp2_fast(a), exp2_fast(b));
    s2 = add_f32x2(s2, w);
    if (ENT) e2 = fma_f32x2(w, t, e2);
  }
  __device__ __forceinline__ void take(const uint64_t (&s2)[2], const uint64_t (&e2)[2]) {
    float a, b;
    unpack2(add_f32x2(s2[0], s2[1]), a, b);
    s += a + b;
    if (ENT) {
      unpack2(add_f32x2(e2[0], e2[1]), a, b);
      e += a + b;
    }
  }
  // A batch of 16-byte vectors of BF16 (or FP32) logits: one maximum and one
  // shift for the batch, then packed arithmetic on pairs.  Returns the maximum.
  template <int U>
  __device__ __forceinline__ float add(const uint4 (&v)[U], float c, uint16_t) {
    uint32_t w[4 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[4 * u] = v[u].x, w[4 * u + 1] = v[u].y, w[4 * u + 2] = v[u].z, w[4 * u + 3] = v[u].w;
    uint32_t mx[4] = {w[0], w[1], w[2], w[3]};
#pragma unroll
    for (int i = 4; i < 4 * U; ++i) mx[i & 3] = max_nan_bf16x2(mx[i & 3], w[i]);
    const uint32_t mp = max_nan_bf16x2(max_nan_bf16x2(mx[0], mx[1]), max_nan_bf16x2(mx[2], mx[3]));
    const float top = raise(max_nan(bf16_lo(mp), bf16_hi(mp)), c);
    const uint64_t nM2 = f32x2_pack(-M, -M), c2 = f32x2_pack(c, c);
    uint64_t s2[2] = {0ull, 0ull}, e2[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) {
      const uint32_t p = ENT ? max_nan_bf16x2(w[i], 0xF180F180u) : w[i];  // -2^100
      step(f32x2_pack(bf16_lo(p), bf16_hi(p)), c2, nM2, s2[i & 1], e2[i & 1]);
    }
    take(s2, e2);
    return top;
  }
  template <int U>
  __device__ __forceinline__ float add(const uint4 (&v)[U], float c, float) {
    float x[4 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[4 * u] = __uint_as_float(v[u].x), x[4 * u + 1] = __uint_as_float(v[u].y);
      x[4 * u + 2] = __uint_as_float(v[u].z), x[4 * u + 3] = __uint_as_float(v[u].w);
    }
    return add(x, c);
  }
  template <int N>
  __device__ __forceinline__ float add(const float (&x)[N], float c) {
    float mx[2] = {x[0], x[N - 1]};
#pragma unroll
    for (int i = 1; i < N - 1; ++i) mx[i & 1] = max_nan(mx[i & 1], x[i]);
    const float top = raise(max_nan(mx[0], mx[1]), c);
    const uint64_t nM2 = f32x2_pack(-M, -M), c2 = f32x2_pack(c, c);
    uint64_t s2[2] = {0ull, 0ull}, e2[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float a = x[i], b = i + 1 < N ? x[i + 1] : neg_inf();
      step(ENT ? f32x2_pack(fmaxf(a, -0x1p100f), fmaxf(b, -0x1p100f)) : f32x2_pack(a, b), c2, nM2, s2[i / 2 & 1],
           e2[i / 2 & 1]);
    }
    take(s2, e2);
    return top;
  }
  // Merged over lanes 0 .. N - 1, N a power of two (the other lanes' parts are
  // empty): the largest shift first, so that each part is scaled once.  Every
  // lane gets m and M, lanes 0 .. N - 1 the sums.
  template <int N>
  __device__ __forceinline__ void warp_merge() {
    const int top = __reduce_max_sync(0xFFFFFFFFu, (int)M);
    m = rank_logit((uint64_t)__reduce_max_sync(0xFFFFFFFFu, rank_value(m)) << 32);
    shift((float)top);
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (ENT) e += __shfl_xor_sync(0xFFFFFFFFu, e, o);
    }
  }
};

// `count` vectors of a part of a row, from vec.
struct Part {
  const uint4* vec;
  int count;
};

// cp_async16 with an L2 cache policy.
__device__ __forceinline__ void cp_async16_hint(uint32_t dst, const void* src, bool valid, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0), "l"(policy)
               : "memory");
}

// A sequence of row parts read by TH threads (thread k takes the vectors k, k
// + TH, ..) through a ring of slots of the thread's own in shared memory: D
// groups of U asynchronous 16-byte copies in flight, across the ends of rows,
// and no barrier between threads.  part(t) names row t's part; each part comes
// PASSES times before the next.
template <int TH, int U, int D, int PASSES, typename E, typename P>
struct Stream {
  P part;
  uint4* ring;  // this thread's first slot; slots `stride` apart
  int stride, k;
  int64_t T, step;
  // next group to fetch: of row t, from vector i
  int64_t t;
  Part cur;
  int i, pass, fill, use;
  uint64_t keep, drop;  // L2 policies of a pass that comes again, and of the last

  __device__ __forceinline__ Stream(P p, uint4* ring_, int stride_, int k_, int64_t t0, int64_t step_, int64_t T_)
      : part(p), ring(ring_), stride(stride_), k(k_), T(T_), step(step_), t(t0), i(0), pass(0), fill(0), use(0) {
    if (PASSES > 1) keep = l2_evict_last(), drop = l2_evict_first();
    if (t < T) cur = part(t);
#pragma unroll
    for (int g = 0; g < D; ++g) fetch();
  }
  static __device__ __forceinline__ uint4 none(uint16_t) {
    return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
  }
  static __device__ __forceinline__ uint4 none(float) {
    return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  }
  __device__ __forceinline__ void fetch() {
    if (t < T) {
      uint4* slot = ring + fill * U * stride;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = i + u * TH + k;
        const bool in = at < cur.count;
        if (PASSES > 1)
          cp_async16_hint(smem_u32(slot + u * stride), cur.vec + (in ? at : 0), in, pass + 1 < PASSES ? keep : drop);
        else
          cp_async16(smem_u32(slot + u * stride), cur.vec + (in ? at : 0), in);
      }
      fill = fill + 1 == D ? 0 : fill + 1;
      i += U * TH;
      if (i >= cur.count) {
        i = 0;
        if (PASSES > 1 && pass + 1 < PASSES) {
          ++pass;
        } else {
          pass = 0;
          t += step;
          if (t < T) cur = part(t);
        }
      }
    }
    cp_async_commit();
  }
  // The next pass over a part of `count` vectors in groups of U: pre(slot, g)
  // on the group's slots, then f(v, g) on its vectors; each slot refilled after
  // it.  Places past the end hold -inf; an empty part is one group of such.
  template <typename P2, typename F>
  __device__ __forceinline__ void row(int count, P2 pre, F f) {
    const int n = count > U * TH ? (count + U * TH - 1) / (U * TH) : 1;
    for (int g = 0; g < n; ++g) {
      asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
      uint4* slot = ring + use * U * stride;
      use = use + 1 == D ? 0 : use + 1;
      pre(slot, g);
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = slot[u * stride];
      const int j = g * U * TH + k;
      if ((g + 1) * U * TH > count) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j + u * TH >= count) v[u] = none(E());
      }
      f(v, g);
      fetch();  // into the slots just read
    }
  }
};

// ---- lists of 32 keys held by a warp, lane i the i-th largest ----
template <typename K>
__device__ __forceinline__ K order_step(K v, int j, bool desc) {
  const K p = __shfl_xor_sync(0xFFFFFFFFu, v, j);
  return (((threadIdx.x & j) == 0) == desc) ? max(v, p) : min(v, p);
}
template <typename K>
__device__ __forceinline__ K list_sort(K v) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) v = order_step(v, j, (threadIdx.x & 31 & k) == 0);
  return v;
}
// The 32 largest of two sorted lists, sorted (a bitonic sequence, cleaned).
template <typename K>
__device__ __forceinline__ K list_merge(K a, K b) {
  K v = max(a, __shfl_sync(0xFFFFFFFFu, b, 31 - (int)(threadIdx.x & 31)));
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) v = order_step(v, j, true);
  return v;
}
}  // namespace moe
