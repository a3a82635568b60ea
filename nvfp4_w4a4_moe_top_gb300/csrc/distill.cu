// Distillation from a teacher's top logits: loss and gradient.  With the
// teacher's q over a list of ids and r off it, the student's p and s = sum of p
// off the list:
//   loss = sum q (ln q - ln p) + r (ln r - ln s)
//   d loss / dz = p - q on the list, p - r p / s off it.
// p / s = e^(z - lse of the part off the list), so neither s nor the quotient
// comes from a difference, and both keep their precision when s is small.
#include "learner.cuh"

namespace moe {

constexpr int kDsU = 4, kDsD = 2;  // vectors per group of copies, groups in flight
constexpr int kDsMaxThreads = 1024;
constexpr int kDsTurns = 4;  // resident grids of rows per launch at most (see kLpTurns)

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// The row's list in shared memory: ids (-1: no entry), the teacher's logits,
// the student's logits.
struct DsList {
  int id[MOE_DISTILL_MAX_K];
  float a[MOE_DISTILL_MAX_K];
  float x[MOE_DISTILL_MAX_K];
};

// The teacher's side of a row, by one warp: ln q_j = (a_j - base) inv_t - shift
// (q = 0 where there is no entry), r its mass off the list, Q = sum q + r.
struct Teacher {
  float base, shift, r, Q;
  __device__ __forceinline__ float lq(float a, float inv_t) const { return (a - base) * inv_t - shift; }
};
__device__ __forceinline__ Teacher teacher_side(const DsList& li, int K, float inv_t, bool has_lse, float lse,
                                                int* status) {
  const int lane = threadIdx.x & 31;
  Teacher T;
  bool bad = false;
  if (has_lse) {
    T.base = 0.0f;
    T.shift = lse;
    bad = !(fabsf(T.shift) <= 3.402823466e+38f);
    float sum = 0.0f;
    for (int j = lane; j < K; j += 32)
      if (li.id[j] >= 0) {
        bad |= !(li.a[j] <= 3.402823466e+38f);
        sum += expf(T.lq(li.a[j], inv_t));
      }
    sum = warp_sum(sum);
    // Where the list holds all of the teacher's mass, 1 - sum is what FP32 leaves
    // of it: each q is off by the roundings of its exponent (a inv_t, lse and
    // their difference, some 2^-24 (|a inv_t| + 2 |lse|), and |a inv_t| is near
    // |lse| where q weighs) and by its own and the sum's.  A rest within that
    // is none: as mass it would meet a student with the same mask and make the
    // loss infinite.  60000 random lists of 1 to 256, |lse| up to 1000: at most
    // 0.6 of the limit.
    const float rest = 1.0f - sum;
    T.r = rest <= 0x1p-23f * (8.0f + 2.0f * fabsf(lse)) ? 0.0f : rest;
    T.Q = T.r > 0.0f ? 1.0f : sum;
  } else {
    float m = kLowest;
    for (int j = lane; j < K; j += 32)
      if (li.id[j] >= 0) {
        bad |= !(li.a[j] <= 3.402823466e+38f);
        m = max_nan(m, li.a[j]);
      }
    m = warp_max_nan(m);
    float sum = 0.0f;
    for (int j = lane; j < K; j += 32)
      if (li.id[j] >= 0) sum += expf((li.a[j] - m) * inv_t);
    sum = warp_sum(sum);
    T.base = m;
    T.shift = logf(sum);
    T.r = 0.0f;
    T.Q = sum == 0.0f ? 0.0f : 1.0f;
  }
  if (bad) set_status(status, MOE_STATUS_NONFINITE_LOGITS);
  if (__any_sync(0xFFFFFFFFu, bad)) T.shift = T.Q = quiet_nan();
  return T;
}
__device__ __forceinline__ float teacher_q(const Teacher& T, const DsList& li, int j, float inv_t) {
  return li.id[j] < 0 || T.Q == 0.0f ? 0.0f : expf(T.lq(li.a[j], inv_t));
}

// The listed elements of a vector in shared memory become -inf; bit e of
// `bits`: element e.
__device__ __forceinline__ void drop_listed(uint4* v, uint32_t bits, uint16_t) {
  for (; bits; bits &= bits - 1) reinterpret_cast<uint16_t*>(v)[__ffs(bits) - 1] = 0xFF80u;
}
__device__ __forceinline__ void drop_listed(uint4* v, uint32_t bits, float) {
  for (; bits; bits &= bits - 1) reinterpret_cast<uint32_t*>(v)[__ffs(bits) - 1] = 0xFF800000u;
}
// Bits of the listed elements of vector i of the row (kVec bits each, vector 0
// after a place for the elements before it).
__device__ __forceinline__ uint32_t listed_bits(const uint32_t* bits, int i, uint16_t) {
  return reinterpret_cast<const uint8_t*>(bits)[i + 1];
}
__device__ __forceinline__ uint32_t listed_bits(const uint32_t* bits, int i, float) {
  return reinterpret_cast<const uint8_t*>(bits)[(i + 1) >> 1] >> ((i + 1 & 1) * 4) & 15u;
}

// Rows in turn, TH threads (one block) per row, or per part of a row: of
// gridDim.x parts, which with SUMS form a cluster.  SUMS: the row's sums,
// loss and statistics; GRAD: its gradient, from the sums or (without SUMS) the
// stored statistics.  A bit per id marks the listed ones, whose elements leave
// the stream of the sums, so that the mass off the list is summed by itself.
// With both, the stream brings each part twice; the second time it comes from
// L2, which holds the rows that the resident blocks work on (first pass with
// the evict-last policy, second with evict-first: 454 -> 372 us).
// 4096 x 131072 BF16, 64 listed: loss 155 us (1.0 of the measured copy rate),
// gradient 328 (0.96), both 371 (0.85 of one read and one write; DRAM moves just
// those, and no exponentials in the second pass change nothing: the third trip
// between L2 and the SMs is what it waits for).  Parts kept in shared memory
// between the passes, in clusters of 2 to 8, took 650 to 1120 us: with one row
// per SM nothing is fetched while a row's sums meet.
template <typename E, bool SUMS, bool GRAD, int TH>
__global__ void __launch_bounds__(TH, TH == 32 ? 24 : kDsMaxThreads / TH) distill_kernel(DistillArgs a) {
  constexpr int N = Row<E>::kVec, NW = TH / 32;
  extern __shared__ uint4 ring[];
  __shared__ DsList list;
  __shared__ Run<false> red[NW];
  __shared__ Run<false> cpart;
  __shared__ Soft<false> sred[NW];
  __shared__ float coef[2];
  __shared__ bool diff;
  __shared__ int dup;
  const int nb = gridDim.x, lg = 31 - __clz(nb), rank = blockIdx.x;  // nb: a power of two
  const int k = threadIdx.x, lane = k & 31;
  const int64_t t0 = blockIdx.y, step = gridDim.y;
  const float c = a.inv_t * kLog2e;
  const E* logits = static_cast<const E*>(a.logits);
  uint32_t* bits = reinterpret_cast<uint32_t*>(ring + TH * kDsU * kDsD);
  begin_kernel();
  for (int i = k; i < (a.V + 2 * N + 31) / 32; i += TH) bits[i] = 0u;
  if (k == 0) dup = 0;
  auto part = [&](int64_t t) {
    const Row<E> r(logits + t * a.ld, a.V);
    const int v0 = r.part(rank, lg), v1 = r.part(rank + 1, lg);
    return Part{r.vec() + v0, v1 - v0};
  };
  Stream<TH, kDsU, kDsD, SUMS && GRAD ? 2 : 1, E, decltype(part)> stream(part, ring + k, TH, k, t0, step, a.T);
  __syncthreads();
  // the next row's entry of this thread (all of them where TH >= K)
  int nid = -1;
  float na = 0.0f;
  if (k < a.K && t0 < a.T) nid = a.teacher_ids[t0 * a.K + k], na = a.teacher_logits[t0 * a.K + k];
  for (int64_t t = t0; t < a.T; t += step) {
    const E* row = logits + t * a.ld;
    const Row<E> r(row, a.V);
    const int v0 = r.part(rank, lg), v1 = r.part(rank + 1, lg), count = v1 - v0;
    auto bit_of = [&](int id) { return id - r.head + N; };
    const float g_row = GRAD && k < 32 ? a.g[t] : 0.0f, lse_row = a.teacher_lse && k < 32 ? a.teacher_lse[t] : 0.0f;
    float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!SUMS && k < 32) st = *reinterpret_cast<const float4*>(a.stats + 4 * t);
    // ---- the list: range, repeats (the first stays), bits ----
    float xs = 0.0f;
    for (int j = k; j < a.K; j += TH) {
      int id = j == k ? nid : a.teacher_ids[t * a.K + j];
      list.a[j] = j == k ? na : a.teacher_logits[t * a.K + j];
      if (id >= a.V) {
        set_status(a.status, MOE_STATUS_BAD_TOKEN);
        id = -1;
      }
      list.id[j] = id;
      if (id >= 0) {
        const float x = to_f32(row[id]);
        if (j == k) xs = x;
        else list.x[j] = x;
        const int b = bit_of(id);
        if (atomicOr(&bits[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u) dup = 1;
      }
    }
    __syncthreads();
    if (dup) {  // rare: every repeat loses its entry
      bool again[MOE_DISTILL_MAX_K / 32];
#pragma unroll
      for (int e = 0; e < MOE_DISTILL_MAX_K / 32; ++e) {
        const int j = k + e * TH;
        again[e] = false;
        if (j < a.K && list.id[j] >= 0)
          for (int i = 0; i < j; ++i) again[e] |= list.id[i] == list.id[j];
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < MOE_DISTILL_MAX_K / 32; ++e) {
        if (again[e]) {
          set_status(a.status, MOE_STATUS_BAD_TOKEN);
          list.id[k + e * TH] = -1;
        }
      }
      if (k == 0) dup = 0;
      __syncthreads();
    }
    auto listed = [&](int i) { return (bits[bit_of(i) >> 5] >> (bit_of(i) & 31) & 1u) != 0u; };
    const int edge = k < r.head ? k : r.tail_start() + k - r.head;  // this thread's element outside the vectors
    const bool has_edge = rank == 0 && k < r.head + r.tail;
    // One warp works on the list: the teacher's side now, the row's statistics
    // (maximum and ln-sum of the row, m, l, and off the list, mt, lt) where the
    // sums end, and the loss and the gradient on the list beside the gradient
    // off it, which is coef[0] times 2^(x c - coef[1]), or 2^((x - coef[1]) c)
    // with `diff`.  Weight 0 (a masked row) gives zeros and no product with
    // what the row's numbers give, which may be NaN.
    Teacher T;
    float m = 0.0f, l = 0.0f, mt = 0.0f, lt = 0.0f;
    if (k < 32)
      T = teacher_side(list, a.K, a.inv_t, a.teacher_lse != nullptr, lse_row, rank == 0 ? a.status : nullptr);
    auto weights = [&](float rescale, float shift) {
      const float ls = (mt - m) * a.inv_t + lt - l;  // ln of the mass off the list
      if (lane == 0) {
        coef[0] = mt == neg_inf() || g_row == 0.0f ? 0.0f : g_row * a.inv_t * (expf(ls) * T.Q - T.r) * rescale;
        coef[1] = shift;
      }
    };
    if (SUMS) {
      Run<false> acc;
      // the listed elements of a group (in the thread's own slots) leave it
      auto drop = [&](uint4* slot, int g) {
        const int i = g * kDsU * TH + k;
        uint32_t b[kDsU], any = 0;
#pragma unroll
        for (int u = 0; u < kDsU; ++u) {
          b[u] = i + u * TH < count ? listed_bits(bits, v0 + i + u * TH, E()) : 0u;
          any |= b[u];
        }
        if (any) {
#pragma unroll
          for (int u = 0; u < kDsU; ++u) drop_listed(slot + u * TH, b[u], E());
        }
      };
      stream.row(count, drop, [&](const uint4 (&v)[kDsU], int) { acc.add(v, c, E()); });
      if (has_edge && !listed(edge)) {
        const float x[1] = {to_f32(row[edge])};
        acc.add(x, c);
      }
      if (k < a.K) list.x[k] = xs;
      acc.template warp_merge<32>();
      if (lane == 0) red[k >> 5] = acc;
      __syncthreads();
      // from the part off the list
      auto finish = [&](float mt_, float lt_, float rescale, float shift) {
        mt = mt_, lt = lt_;
        const bool empty = mt == neg_inf();
        m = empty ? kLowest : mt;
        bool any = !empty;
        for (int j = lane; j < a.K; j += 32)
          if (list.id[j] >= 0) {
            m = max_nan(m, list.x[j]);
            any |= list.x[j] != neg_inf();
          }
        m = warp_max_nan(m);
        any = __any_sync(0xFFFFFFFFu, any);
        float s = 0.0f;
        for (int j = lane; j < a.K; j += 32)
          if (list.id[j] >= 0) s += exp2_fast((list.x[j] - m) * c);
        s = warp_sum(s);
        if (!empty) s += exp2_fast((mt - m) * c) * expf(lt);
        l = logf(s);
        const bool bad = !(m <= 3.402823466e+38f);
        if (!any) m = neg_inf(), l = 0.0f;
        if (bad) m = l = mt = lt = quiet_nan();
        if (GRAD) weights(rescale, shift);
      };
      if (k < 32) {
        acc = Run<false>();
        if (lane < NW) acc = red[lane];
        acc.template warp_merge<32>();
        if (lane == 0) cpart = acc;
      }
      if (nb > 1) {
        cluster_arrive();
        cluster_wait();
        if (k < 32) {
          acc = Run<false>();
          if (lane < nb) {
            acc.m = cluster_load_f32(&cpart.m, lane);
            acc.M = cluster_load_f32(&cpart.M, lane);
            acc.s = cluster_load_f32(&cpart.s, lane);
          }
          acc.template warp_merge<32>();
        }
        cluster_arrive();  // this block has read the others' parts; waited for before cpart is written again
      }
      if (k < 32) {
        acc.s = __shfl_sync(0xFFFFFFFFu, acc.s, 0);
        const bool differ = acc.m <= 3.402823466e+38f && !acc.shift_ok(c);
        if (lane == 0) diff = differ;
        if (!differ) finish(acc.m, kLn2 * (log2f(acc.s) - fmaf(acc.m, c, -acc.M)), 1.0f / acc.s, acc.M);
      }
      __syncthreads();
      if (diff) {  // masks at extreme values, or nothing off the list: differences first
        Soft<false> all;
        for (int i = k; i < a.V; i += TH)
          if (!listed(i)) {
            const float x[1] = {to_f32(row[i])};
            all.add(x, c);
          }
        all.warp_merge(c);
        if (lane == 0) sred[k >> 5] = all;
        if (nb > 1) {  // no block writes (dlogits may be the logits) before all have read the row
          cluster_wait();
          cluster_arrive();
          cluster_wait();
          cluster_arrive();
        }
        __syncthreads();
        if (k < 32) {
          all = Soft<false>();
          if (lane < NW) all = sred[lane];
          all.warp_merge(c);
          const float lt = all.s == 0.0f ? 0.0f : logf(all.s);
          finish(all.s == 0.0f ? neg_inf() : all.m, lt, expf(-lt), all.m);
        }
        __syncthreads();
      }
    } else {
      if (k < a.K) list.x[k] = xs;
      if (k < 32) {
        m = st.x, l = st.y, mt = st.z, lt = st.w;
        if (lane == 0) diff = true;
        weights(expf(-lt), mt);
      }
      __syncthreads();
    }
    if (k < 32) {
      const bool none = m == neg_inf(), bad = m != m;
      float part = 0.0f;
      for (int j = lane; j < a.K; j += 32) {
        const float q = teacher_q(T, list, j, a.inv_t), lp = (list.x[j] - m) * a.inv_t - l;
        if (SUMS && list.id[j] >= 0 && !(q == 0.0f)) part += none ? -neg_inf() : q * (T.lq(list.a[j], a.inv_t) - lp);
        if (GRAD) list.a[j] = none || g_row == 0.0f ? 0.0f : g_row * a.inv_t * (expf(lp) * T.Q - q);
      }
      if (SUMS) {
        part = warp_sum(part);
        const float ls = mt == neg_inf() ? neg_inf() : (mt - m) * a.inv_t + lt - l;
        if (!(T.r == 0.0f)) part += none ? -neg_inf() : T.r * (logf(T.r) - ls);
        if (bad || T.Q != T.Q) part = quiet_nan();
        if (lane == 0 && rank == 0) {
          if (bad) set_status(a.status, MOE_STATUS_NONFINITE_LOGITS);
          a.loss[t] = part;
          if (a.stats_out) *reinterpret_cast<float4*>(a.stats_out + 4 * t) = make_float4(m, l, mt, lt);
        }
      }
    }
    // the bits of this row go; the next row's entry comes
    const int64_t tn = t + step;
    if (k < a.K && tn < a.T) nid = a.teacher_ids[tn * a.K + k], na = a.teacher_logits[tn * a.K + k];
    for (int j = k; j < a.K; j += TH)
      if (list.id[j] >= 0) bits[bit_of(list.id[j]) >> 5] = 0u;
    if (GRAD) {
      const float w = coef[0], shift = coef[1];
      const bool by_diff = diff;
      E* out = static_cast<E*>(a.dlogits) + t * a.ldd;
      const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
      auto grad = [&](float x) {
        return w == 0.0f ? 0.0f : w * exp2_fast(by_diff ? (x - shift) * c : fmaf(x, c, -shift));
      };
      const uint64_t c2 = f32x2_pack(c, c), s2 = f32x2_pack(-shift, -shift), w2 = f32x2_pack(w, w);
      auto put = [&](const uint4& v, int i) {  // vector i of the row
        float x[N];
        unpack(v, x);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const uint64_t xe = f32x2_pack(x[e], x[e + 1]);
          float lo, hi;
          unpack2(by_diff ? mul_f32x2(add_f32x2(xe, s2), c2) : fma_f32x2(xe, c2, s2), lo, hi);
          unpack2(mul_f32x2(f32x2_pack(exp2_fast(lo), exp2_fast(hi)), w2), x[e], x[e + 1]);
        }
        if (w == 0.0f) {  // also where nothing is off the list, and the shift no number
#pragma unroll
          for (int e = 0; e < N; ++e) x[e] = 0.0f;
        }
        if (same) {
          __stcs(reinterpret_cast<uint4*>(out + r.head) + i, pack(x));
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) from_f32(x[e], out[r.head + (int64_t)i * N + e]);
        }
      };
      stream.row(count, [](uint4*, int) {}, [&](const uint4 (&v)[kDsU], int g) {
#pragma unroll
        for (int u = 0; u < kDsU; ++u) {
          const int i = g * kDsU * TH + u * TH + k;
          if (i < count) put(v[u], v0 + i);
        }
      });
      if (has_edge) from_f32(grad(to_f32(row[edge])), out[edge]);
      __syncthreads();
      // ids of this block's part, over what the stream wrote there
      const int lo = rank == 0 ? 0 : r.head + v0 * N, hi = rank == nb - 1 ? r.tail_start() : r.head + v1 * N;
      for (int j = k; j < a.K; j += TH) {
        const int id = list.id[j];
        if (id >= 0 && ((id >= lo && id < hi) || (rank == 0 && id >= r.tail_start()))) from_f32(list.a[j], out[id]);
      }
    }
    if (SUMS && nb > 1) cluster_wait();
    __syncthreads();
  }
}

// host launchers
template <typename E, bool SUMS, bool GRAD>
static void (*distill_of(int th))(DistillArgs) {
  return th == 32     ? distill_kernel<E, SUMS, GRAD, 32>
         : th == 128  ? distill_kernel<E, SUMS, GRAD, 128>
         : th == 256  ? distill_kernel<E, SUMS, GRAD, 256>
         : th == 512  ? distill_kernel<E, SUMS, GRAD, 512>
                      : distill_kernel<E, SUMS, GRAD, SUMS && GRAD ? 1024 : 512>;
}
template <typename E>
static int launch_distill_of(const DistillArgs& a, cudaStream_t s) {
  const int64_t nvec = (int64_t)a.V / Row<E>::kVec;
  const bool sums = a.loss != nullptr, grad = a.dlogits != nullptr;
  auto bits_of = [](int V) { return (V + 2 * Row<E>::kVec + 31) / 32 * 4; };
  const int sms = gemm_num_ctas(), bits = bits_of(a.V), bits_1024 = 80 * 1024;
  const int most = bits <= bits_1024 ? 1024 : 512;  // threads whose ring fits beside the bits
  // Few rows: more blocks per row until there is one for each SM.
  int nb = 1;
  while (nb < 8 && (int64_t)a.T * nb < sms && nvec / (nb * 2) >= 512) nb *= 2;
  // The gradient alone exchanges nothing: parts of 2048 vectors or more until
  // the last of 16 rounds per SM weighs little (1024 x 100003 BF16: 72 -> 68 us;
  // 500 x 100000 FP32: 76 -> 65).
  if (!sums)
    while (nb < 8 && (int64_t)a.T * nb < 16 * sms && nvec / (nb * 2) >= 2048) nb *= 2;
  const int64_t part = nvec / nb;
  // Threads per row: as few as hide a row's ends (list, sums, loss) behind
  // other rows.  Loss, BF16: 6000 x 8192 27 us with 32 and 34 with 128; 16384 x
  // 32768 175 with 128 and 213 with 256; 4096 x 131072 166 and 153.  Gradient:
  // 6000 x 8192 38 with 32 and 41 with 128; 6000 x 16384 71 and 64.  The step:
  // 6000 x 8192 51 and 56, 6000 x 16384 93 and 84; its 1024 threads per SM work
  // on rows that L2 has to hold between the passes: 80 MB of it (4096 x 131072:
  // 372 with 512, 455 with 256).
  int th = part <= (grad ? 1024 : 2048) ? 32 : part <= 8192 ? 128 : 256;
  if (sums && grad && th > 32) th = part <= 3072 ? 128 : part <= 8192 ? 256 : part <= 16384 ? 512 : 1024;
  if (bits > 40 * 1024 && th < 256) th = 256;
  // More while all rows have them at once, 128 also in two rounds (the step, 600
  // x 16384: 23 us with 32 threads, 11 with 256; 2000 x 16384: 43 and 33 with 128;
  // the loss, 600 x 16384: 11 and 7); very short rows only where SMs would be
  // left idle (the step, 4 x 4096: 9.1 us with 32, 5.6 with 256; 2000 x 2000:
  // 11.2 and 13.1 with 128).
  auto more = [](int n) { return n == 32 ? 128 : 2 * n; };
  const int64_t rows = (int64_t)a.T * nb, room = (int64_t)sms * kDsMaxThreads;
  while (th < 512 && part > (th == 32 && rows > 2 * sms ? 512 : 2 * th) &&
         rows * more(th) <= (th == 32 ? 2 * room : room))
    th = more(th);
  if (th > most) th = most;
  const int ring = th * kDsU * kDsD * 16, smem = ring + bits;
  const int smem_most = ring + (th == 1024 ? bits_1024 : bits_of(MOE_DISTILL_MAX_V));
  int fit = 227 * 1024 / (smem + 5 * 1024);
  if (fit > kDsMaxThreads / th) fit = kDsMaxThreads / th;
  if (fit < 1) fit = 1;
  const int64_t grid = (int64_t)sms * fit / nb * kDsTurns;
  auto f = !sums  ? distill_of<E, false, true>(th)
           : grad ? distill_of<E, true, true>(th)
                  : distill_of<E, true, false>(th);
  if (!allow_smem((const void*)f, smem, smem_most)) return -1;
  return launch_kernel(f, dim3(nb, (unsigned)(a.T < grid ? a.T : grid)), th, smem, sums ? nb : 1, s, a);
}
int launch_distill(const DistillArgs& a, cudaStream_t s) {
  return a.dtype == MOE_DTYPE_BF16 ? launch_distill_of<uint16_t>(a, s) : launch_distill_of<float>(a, s);
}

}  // namespace moe
