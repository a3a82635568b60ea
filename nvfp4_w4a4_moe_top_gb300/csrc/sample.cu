// The draw of a token from each row of logits: temperature, top-k, top-p,
// min-p, and the inverse of the distribution function at a given number u.
//
// Weights are 64-bit fixed-point numbers, w = 2^s at the row's maximum, s such
// that a row's sum stays below 2^63.  Sums of them are the same in any order:
// threads and atomics add them as they come, and the result is one.
#include "exp_table.cuh"
#include "tokens.cuh"

namespace moe {

constexpr int kSaU = 4;       // vectors read together
constexpr int kSaRuns = 8;    // runs of a thread at most
constexpr int kSaBins = 2048;
constexpr float kMinExponent = -42.0f;  // weights below 2^-42 count as 0

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) { return __shfl_xor_sync(0xFFFFFFFFu, v, o); }
__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += shfl_xor64(v, o);
  return v;
}

template <int TH>
struct SampleShared {
  static constexpr int NW = TH / 32;
  uint64_t exp2[64];                // 2^(j/64) 2^62
  uint64_t part[kSaRuns + 2][NW];   // sums of the runs by warp; the row's ends
  uint64_t pre[kSaRuns + 3];        // what comes before each of them
  uint64_t scan[NW];
  uint64_t list[TH];
  uint64_t mass[kSaBins];
  uint32_t count[kSaBins];
  float wmax[NW];
  uint64_t target;
  // results that one thread finds for all
  uint64_t key, incl;
  uint32_t found, bin_count, listed;
  int bin;
  int id;
  float x;
};

// Weights of a row: 2^((x - m) c) for logits x about the maximum m.
struct Weights {
  float m, ch, cl;  // c = inv_temperature log2(e) = ch + cl
  int s;
  const uint64_t* exp2;
  // To about 2^-38: the exponent is formed from the exact difference x - m as a
  // pair of floats and split into a multiple of 1/64, whose power is read from a
  // table, and a rest r, for which the series of 2^r - 1 has four terms.  The
  // largest term is a pair of floats again, and the product with the table's
  // entry and the sum are integers.
  __device__ __forceinline__ uint64_t operator()(float x) const {
    const float d = x - m;
    const float p = __fmul_rn(d, ch);  // a product of its own: never part of an FMA
    if (!(p >= kMinExponent - 1.0f)) return 0;  // -inf and a difference beyond the range among them
    const float b = d - x, lost = (x - (d - b)) + (-m - b);  // x - m = d + lost
    const float e = fmaf(lost, ch, fmaf(d, cl, fmaf(d, ch, -p)));
    if ((p - kMinExponent) + e < 0.0f) return 0;
    const float z = p + 196608.0f;  // 1.5 2^17: steps of 1/64
    const int i = __float_as_int(z) - __float_as_int(196608.0f);
    const float r0 = p - (z - 196608.0f);
    const float r = r0 + e, rl = (r0 - r) + e;
    const float a = __fmul_rn(r, 0.693147182464599609375f);  // ln 2, and what it leaves below
    const float al = fmaf(r, -1.904654299957768e-9f, fmaf(rl, 0.69314718f, fmaf(r, 0.693147182464599609375f, -a)));
    const float tail = r * r * fmaf(r, fmaf(r, 0.00961812911f, 0.0555041087f), 0.240226507f);
    const int q = __float2int_rn(a * 0x1p38f) + __float2int_rn((al + tail) * 0x1p38f);
    const uint64_t t = exp2[i & 63];
    const uint64_t w = t + (uint64_t)(((int64_t)q * (int64_t)(t >> 32)) >> 6);
    const int down = 62 - s - (i >> 6);
    return (w + (1ull << (down - 1))) >> down;
  }
};

// A row's elements in the order of the ids: the elements in front of the
// vectors, the vectors in runs, the elements after them.  Run q of thread k:
// the vectors (q per + j) TH + k, j < per; of all threads: `per` TH vectors.
template <typename E, int TH>
struct SampleRow {
  Row<E> r;
  int per, runs;
  __device__ __forceinline__ SampleRow(const E* row, int V) : r(row, V) {
    const int n = (r.nvec + TH - 1) / TH;  // vectors of a thread
    per = kSaU;
    while (per * kSaRuns < n) per *= 2;
    runs = (n + per - 1) / per;
  }
  // f(x, id) on the elements of vector i
  template <typename F>
  __device__ __forceinline__ void vector(const uint4& v, int i, F f) const {
    constexpr int N = Row<E>::kVec;
    float x[N];
    unpack(v, x);
#pragma unroll
    for (int e = 0; e < N; ++e) f(x[e], r.head + i * N + e);
  }
  // f(x, id) on this thread's elements of run q
  template <typename F>
  __device__ __forceinline__ void run(int q, F f) const {
    for (int j = 0; j < per; j += kSaU) {
      const int i0 = (q * per + j) * TH + (int)threadIdx.x;
      if (i0 >= r.nvec) break;
      uint4 v[kSaU];
#pragma unroll
      for (int u = 0; u < kSaU; ++u) v[u] = r.vec()[min(i0 + u * TH, r.nvec - 1)];
#pragma unroll
      for (int u = 0; u < kSaU; ++u)
        if (i0 + u * TH < r.nvec) vector(v[u], i0 + u * TH, f);
    }
  }
  // f(x, id) on this thread's elements outside the vectors
  template <typename F>
  __device__ __forceinline__ void front(F f) const {
    if ((int)threadIdx.x < r.head) f(to_f32(r.p[threadIdx.x]), (int)threadIdx.x);
  }
  template <typename F>
  __device__ __forceinline__ void back(F f) const {
    const int id = r.tail_start() + (int)threadIdx.x;
    if ((int)threadIdx.x < r.tail) f(to_f32(r.p[id]), id);
  }
  template <typename F>
  __device__ __forceinline__ void all(F f) const {
    front(f);
    for (int q = 0; q < runs; ++q) run(q, f);
    back(f);
  }
};

// Exclusive sum over the block's threads, and the total.  Ends with a barrier
// before `scan` may be used again.
template <int TH>
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t& total, SampleShared<TH>& sh) {
  constexpr int NW = TH / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) sh.scan[warp] = incl;
  __syncthreads();
  uint64_t before = incl - v;
  total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const uint64_t s = sh.scan[w];
    before += w < warp ? s : 0;
    total += s;
  }
  __syncthreads();
  return before;
}

// The first id up to which the sum of f(x, id), a whole number, is above
// target(sum over the row); sh.id and sh.x.  Returns the sum over the row.
template <typename E, int TH, typename F, typename G>
__device__ __forceinline__ uint64_t pick(const SampleRow<E, TH>& row, F f, G target_of, SampleShared<TH>& sh) {
  constexpr int NW = TH / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t v = 0;
  auto add = [&](float x, int id) { v += f(x, id); };
  for (int q = 0; q < row.runs; ++q) {
    v = 0;
    row.run(q, add);
    v = warp_sum64(v);
    if (lane == 0) sh.part[q + 1][warp] = v;
  }
  if (warp == 0) {
    v = 0;
    row.front(add);
    v = warp_sum64(v);
    if (lane == 0) sh.part[0][0] = v;
    v = 0;
    row.back(add);
    v = warp_sum64(v);
    if (lane == 0) sh.part[row.runs + 1][0] = v;
  }
  __syncthreads();
  if (warp == 0) {
    uint64_t sum = 0;
    for (int e = 0; e < row.runs + 2; ++e) {
      const int n = e == 0 || e == row.runs + 1 ? 1 : NW;
      v = warp_sum64(lane < n ? sh.part[e][lane] : 0);
      if (lane == 0) sh.pre[e] = sum;
      sum += v;
    }
    if (lane == 0) {
      sh.pre[row.runs + 2] = sum;
      const uint64_t t = target_of(sum);
      sh.target = t < sum ? t : sum - 1;  // sum > 0
    }
  }
  __syncthreads();
  const uint64_t total = sh.pre[row.runs + 2], target = sh.target;
  int e = 0;
  while (e < row.runs + 1 && sh.pre[e + 1] <= target) ++e;
  uint64_t left = target - sh.pre[e];
  // walks the elements of one part of the row in order
  bool done = false;
  auto walk = [&](float x, int id) {
    const uint64_t w = f(x, id);
    if (!done && w > left) {
      done = true;
      sh.id = id;
      sh.x = x;
    }
    left -= w;
  };
  if (e == 0 || e == row.runs + 1) {
    if (threadIdx.x == 0) {
      const int i0 = e == 0 ? 0 : row.r.tail_start(), n = e == 0 ? row.r.head : row.r.tail;
      for (int i = 0; i < n && !done; ++i) walk(to_f32(row.r.p[i0 + i]), i0 + i);
    }
  } else {  // thread k takes `per` vectors in a row
    const int i0 = ((e - 1) * TH + (int)threadIdx.x) * row.per, i1 = min(i0 + row.per, row.r.nvec);
    v = 0;
    for (int i = i0; i < i1; ++i) row.vector(row.r.vec()[i], i, add);
    uint64_t sum;
    const uint64_t before = block_scan<TH>(v, sum, sh);
    if (before <= left && left < before + v) {
      left -= before;
      for (int i = i0; i < i1 && !done; ++i) row.vector(row.r.vec()[i], i, walk);
    }
  }
  __syncthreads();
  return total;
}

// Bins of the distance below the row's maximum in the order of rank_value: by
// 1/64 of a power of two over sixteen of them, then by half of one.
__device__ __forceinline__ int first_bin(uint32_t d) {
  return d < (1u << 27) ? (int)(d >> 17) : 1024 + (int)((d - (1u << 27)) >> 22);
}
__device__ __forceinline__ uint32_t first_bin_start(int b) {
  return b < 1024 ? (uint32_t)b << 17 : (1u << 27) + ((uint32_t)(b - 1024) << 22);
}

// The last element of the shortest leading part, in the order of the keys and
// of the keys >= least, that holds `target` elements (COUNT) or weight: its key
// in sh.key, the weight up to and with it in sh.incl.  False if all together do
// not.  target >= 1.
template <bool COUNT, typename E, int TH>
__device__ __forceinline__ bool select(const SampleRow<E, TH>& row, const Weights& weight, uint64_t target,
                                       uint64_t least, SampleShared<TH>& sh) {
  constexpr int PER = kSaBins / TH;
  const uint32_t top = rank_value(weight.m);
  uint32_t d0 = 0, d1 = 0xFFFFFFFFu;  // distances in question
  uint64_t base_n = 0, base_w = 0;    // elements before them, and their weight
  for (int level = 0;; ++level) {
    int shift = 0;
    while (((d1 - d0) >> shift) >= (uint32_t)kSaBins) ++shift;
    for (int b = threadIdx.x; b < kSaBins; b += TH) sh.count[b] = 0, sh.mass[b] = 0;
    if (threadIdx.x == 0) sh.found = 0, sh.listed = 0;
    __syncthreads();
    row.all([&](float x, int id) {
      const uint64_t key = rank_key(x, (uint32_t)id);
      const uint32_t d = top - (uint32_t)(key >> 32);
      if (x == neg_inf() || key < least || d < d0 || d > d1) return;
      const int b = level == 0 ? first_bin(d) : (int)((d - d0) >> shift);
      atomicAdd(&sh.count[b], 1u);
      const uint64_t w = weight(x);
      if (w) atomicAdd((unsigned long long*)&sh.mass[b], (unsigned long long)w);
    });
    __syncthreads();
    uint64_t n = 0, w = 0, total;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += sh.count[threadIdx.x * PER + i], w += sh.mass[threadIdx.x * PER + i];
    uint64_t n0 = base_n + block_scan<TH>(n, total, sh), w0 = base_w + block_scan<TH>(w, total, sh);
    if (COUNT ? n0 < target && target <= n0 + n : w0 < target && target <= w0 + w) {
      for (int i = 0;; ++i) {
        const int b = threadIdx.x * PER + i;
        const uint32_t bn = sh.count[b];
        const uint64_t bw = sh.mass[b];
        if (COUNT ? target <= n0 + bn : target <= w0 + bw) {
          sh.found = 1, sh.bin = b, sh.bin_count = bn;
          sh.key = n0, sh.incl = w0;
          break;
        }
        n0 += bn, w0 += bw;
      }
    }
    __syncthreads();
    if (!sh.found) return false;
    const int bin = sh.bin;
    const uint32_t in = sh.bin_count;
    base_n = sh.key, base_w = sh.incl;
    if (level == 0) {
      d0 = first_bin_start(bin);
      d1 = bin + 1 < kSaBins ? first_bin_start(bin + 1) - 1 : 0xFFFFFFFFu;
    } else {
      const uint32_t start = d0 + ((uint32_t)bin << shift), rest = d1 - start, width = (1u << shift) - 1;
      d0 = start;
      d1 = start + min(rest, width);
    }
    __syncthreads();
    if (in <= (uint32_t)TH) {  // few: sorted
      row.all([&](float x, int id) {
        const uint64_t key = rank_key(x, (uint32_t)id);
        const uint32_t d = top - (uint32_t)(key >> 32);
        if (x != neg_inf() && key >= least && d >= d0 && d <= d1) sh.list[atomicAdd(&sh.listed, 1u)] = key;
      });
      __syncthreads();
      const uint64_t key = threadIdx.x < in ? sh.list[threadIdx.x] : 0;
      int place = 0;
      for (uint32_t j = 0; j < in; ++j) place += sh.list[j] > key;
      __syncthreads();
      if (threadIdx.x < in) sh.list[place] = key;
      __syncthreads();
      const uint64_t mine = threadIdx.x < in ? sh.list[threadIdx.x] : 0;
      const uint64_t mw = threadIdx.x < in ? weight(rank_logit(mine)) : 0;
      const uint64_t before = base_w + block_scan<TH>(mw, total, sh);
      if (threadIdx.x < in &&
          (COUNT ? base_n + threadIdx.x + 1 == target : before < target && target <= before + mw))
        sh.key = mine, sh.incl = before + mw;
      __syncthreads();
      return true;
    }
    if (d0 == d1) {  // ties: the first of them in the order of the ids
      const uint32_t value = top - d0;
      const uint64_t w1 = weight(rank_logit((uint64_t)value << 32));
      const uint64_t take = COUNT ? target - base_n : (target - base_w + w1 - 1) / w1;
      pick<E, TH>(row, [&](float x, int id) {
        return (uint64_t)(x != neg_inf() && rank_value(x) == value && rank_key(x, (uint32_t)id) >= least);
      }, [&](uint64_t) { return take - 1; }, sh);
      if (threadIdx.x == 0) sh.key = rank_key(sh.x, (uint32_t)sh.id), sh.incl = base_w + take * w1;
      __syncthreads();
      return true;
    }
  }
}

template <typename E, int TH>
__global__ void __launch_bounds__(TH) sample_tokens_kernel(SampleArgs a) {
  constexpr int NW = TH / 32;
  extern __shared__ char smem[];
  SampleShared<TH>& sh = *reinterpret_cast<SampleShared<TH>*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < 64)
    sh.exp2[threadIdx.x] = (uint64_t)__float2ll_rn(kExp2Tab[threadIdx.x][0] * 0x1p62f) +
                           (uint64_t)__float2ll_rn(kExp2Tab[threadIdx.x][1] * 0x1p62f);
  begin_kernel();
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const SampleRow<E, TH> row(static_cast<const E*>(a.logits) + t * a.ld, a.V);
    const float inv_t = a.inv_t ? a.inv_t[t] : 1.0f, u = a.u[t];
    const float top_p = a.top_p ? a.top_p[t] : 1.0f, min_p = a.min_p ? a.min_p[t] : 0.0f;
    const int top_k = a.top_k ? a.top_k[t] : 0;
    float m = neg_inf();
    row.all([&](float x, int) { m = max_nan(m, x); });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    __syncthreads();
    if (lane == 0) sh.wmax[warp] = m;
    __syncthreads();
    m = sh.wmax[0];
    for (int w = 1; w < NW; ++w) m = max_nan(m, sh.wmax[w]);
    const bool params = inv_t >= 1e-6f && inv_t <= 1e6f && u >= 0.0f && u < 1.0f && top_p == top_p && min_p == min_p;
    if (!params || !(m <= 3.402823466e+38f) || m == neg_inf()) {
      if (threadIdx.x == 0) {
        const bool none = params && m == neg_inf();
        a.tokens[t] = -1;
        if (a.logprob) a.logprob[t] = none ? neg_inf() : quiet_nan();
        if (a.kept_logprob) a.kept_logprob[t] = none ? neg_inf() : quiet_nan();
        if (!params) set_status(a.status, MOE_STATUS_BAD_SAMPLING);
        if (!(m <= 3.402823466e+38f)) set_status(a.status, MOE_STATUS_NONFINITE_LOGITS);
      }
      continue;
    }
    Weights weight;
    const double c = (double)inv_t * 1.4426950408889634;
    weight.m = m, weight.ch = (float)c, weight.cl = (float)(c - (double)weight.ch);
    weight.s = min(52, 63 - (32 - __clz(a.V - 1)));
    weight.exp2 = sh.exp2;
    uint64_t sum = 0, total;
    row.all([&](float x, int) { sum += weight(x); });
    block_scan<TH>(sum, total, sh);
    uint64_t least = 0, mass = total;  // kept: keys from least on
    if (top_k > 0 && top_k < a.V && select<true, E, TH>(row, weight, (uint64_t)top_k, least, sh))
      least = sh.key, mass = sh.incl;
    __syncthreads();
    if (top_p < 1.0f) {
      const uint64_t target = max(1ull, (unsigned long long)__double2ull_ru((double)fmaxf(top_p, 0.0f) * (double)mass));
      if (select<false, E, TH>(row, weight, target, least, sh)) least = max(least, sh.key);
      __syncthreads();
    }
    if (min_p > 0.0f) {
      // the smallest float x with (x - m) inv_t >= ln min_p
      const double edge = (double)m + log((double)fminf(min_p, 1.0f)) / (double)inv_t;
      least = max(least, (uint64_t)rank_value(__double2float_ru(edge)) << 32);
    }
    mass = pick<E, TH>(row, [&](float x, int id) {
      return x != neg_inf() && rank_key(x, (uint32_t)id) >= least ? weight(x) : 0;
    }, [&](uint64_t sum) { return __double2ull_rd((double)u * (double)sum); }, sh);
    if (threadIdx.x == 0) {
      const float z = (sh.x - m) * inv_t, unit = ldexpf(1.0f, -weight.s);
      const uint64_t one = 1ull << weight.s;
      a.tokens[t] = sh.id;
      if (a.logprob) a.logprob[t] = z - log1pf((float)(total - one) * unit);
      if (a.kept_logprob) a.kept_logprob[t] = z - log1pf((float)(mass - one) * unit);
    }
    __syncthreads();
  }
}

int launch_sample_tokens(const SampleArgs& a, cudaStream_t s) {
  constexpr int TH = 512;
  const int64_t most = (int64_t)gemm_num_ctas() * 2 * 8;
  const int smem = (int)sizeof(SampleShared<TH>);
  auto f = a.dtype == MOE_DTYPE_BF16 ? sample_tokens_kernel<uint16_t, TH> : sample_tokens_kernel<float, TH>;
  if (!allow_smem((const void*)f, smem, smem)) return -1;
  return launch_kernel(f, (unsigned)(a.T < most ? a.T : most), TH, smem, 1, s, a);
}

}  // namespace moe
