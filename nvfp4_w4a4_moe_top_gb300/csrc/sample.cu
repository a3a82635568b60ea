// The draw of a token from each row of logits: temperature, top-k, top-p,
// min-p, and the inverse of the distribution function at a given number u.
// One read of the logits is the bound: four operations and one exponential per
// element.  What is kept is little for most rows, and found from the maxima of
// short runs; the rest of the work then touches a few hundred elements.
//
// Weights are w = 2^((x - m) c) about the row's maximum m, as 64-bit fixed-point
// numbers of unit 2^-s, s such that a row's sum stays below 2^63.  Sums of them
// are the same in any order: threads and atomics add them as they come, and the
// result is one.
//
// There are two kinds of weights.  Weights from FP32 exponentials make sums with
// a relative error below delta (see row_delta); a decision that is nearer to its
// border than that is made again with weights to about 2^-37.
#include "exp_table.cuh"
#include "tokens.cuh"

namespace moe {

constexpr int kSaU = 4;     // vectors read together
constexpr int kSaD = 2;     // groups of them on the way
constexpr int kSaRuns = 8;  // runs of a thread at most
constexpr int kSaBins = 2048;
constexpr int kSaNear = 1024;  // bins of the sixteen powers of two below the maximum
constexpr float kMinExponent = -42.0f;  // weights below 2^-42 count as 0

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// total p for 0 <= p < 1, rounded down or up to a whole number.
template <bool UP>
__device__ __forceinline__ uint64_t part_of(uint64_t total, float p) {
  const uint32_t bits = __float_as_uint(p);
  const int down = 126 - (int)(bits >> 23);  // p = mantissa 2^-24 2^-down
  if (!(p >= 0x1p-63f)) return UP && p > 0.0f && total > 0 ? 1 : 0;  // total < 2^63
  const uint64_t a = (uint64_t)((bits & 0x7FFFFFu) | 0x800000u) << 40, hi = __umul64hi(total, a);
  const bool rest = (total * a | (hi & ((1ull << down) - 1))) != 0;
  return (hi >> down) + (UP && rest ? 1 : 0);
}

template <int TH>
struct SampleShared {
  static constexpr int NW = TH / 32, kList = TH < 1024 ? 2 * TH : TH;
  uint64_t exp2[64];               // 2^(j/64) 2^62
  uint64_t part[kSaRuns + 2][NW];  // sums of the runs by warp; the row's ends
  uint64_t pre[kSaRuns + 3];       // what comes before each of them
  uint64_t scan[2][NW];
  float wmax[NW];
  float edge[2];  // ln(min_p) / inv_temperature, a pair
  // results that one thread finds for all
  uint64_t target, key, incl, before, after, base_n, base_w;
  uint32_t found, listed;
  int bin, sure_bin, id, kept;
  float x;
};
// What shares its memory with the ring that the logits come through.
template <int TH>
struct SampleWork {
  uint64_t list[SampleShared<TH>::kList], weight[SampleShared<TH>::kList];
  uint32_t lo[kSaBins], hi[kSaBins];
};
template <int TH>
constexpr int kSaRing = TH * kSaU * kSaD * 16;
template <int TH>
constexpr int kSaSmem = (kSaRing<TH> > (int)sizeof(SampleWork<TH>) ? kSaRing<TH> : (int)sizeof(SampleWork<TH>)) +
                        TH * kSaRuns * 8 + (int)sizeof(SampleShared<TH>);

__device__ __forceinline__ void add64(uint32_t* lo, uint32_t* hi, uint64_t v) {
  const uint32_t l = (uint32_t)v, was = atomicAdd(lo, l);
  const uint32_t h = (uint32_t)(v >> 32) + (was + l < was);
  if (h) atomicAdd(hi, h);
}

// Weights of a row: 2^((x - m) c) for logits x about the maximum m.
struct Weights {
  float m, ch, cl;  // c = inv_temperature log2(e) = ch + cl
  int s;
  const uint64_t* exp2;
  // From an FP32 exponential.
  __device__ __forceinline__ float ratio(float x) const {
    const float t = (x - m) * ch;
    return t >= kMinExponent ? exp2_fast(t) : 0.0f;
  }
  static __device__ __forceinline__ uint64_t mantissa(float w) { return (__float_as_uint(w) & 0x7FFFFFu) | 0x800000u; }
  __device__ __forceinline__ uint64_t fast(float x) const {
    const float w = ratio(x);  // in [0, 1]
    return w > 0.0f ? mantissa(w) << (s - 23) >> (127 - (int)(__float_as_uint(w) >> 23)) : 0;
  }
  // To about 2^-37: the exponent is formed from the exact difference x - m as a
  // pair of floats and split into a multiple of 1/64, whose power is read from a
  // table, and a rest r, for which the series of 2^r - 1 has four terms.  The
  // largest term is a pair of floats again, and the product with the table's
  // entry and the sum are integers.
  __device__ __forceinline__ uint64_t exact(float x) const {
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
  template <bool EXACT>
  __device__ __forceinline__ uint64_t of(float x) const {
    return EXACT ? exact(x) : fast(x);
  }
};

// A bound of the relative error of sums of fast weights, of a row whose V
// weights sum to S >= 1.  A weight 2^-t, t >= 0, is off by the exponential's
// 2^-22, by less than 3 2^-24 t ln 2 from the roundings of its exponent (the
// difference, c, the product), and by the additions: 18 2^-24 at most (10 in a
// batch, one per batch of a run), and the change from the batches' shift to m,
// 2^-21.  The mean of t over the weights is at most (S - 1) / S log2(V / (S -
// 1)), its value where all but the first are equal.
__device__ __forceinline__ float row_delta(float S, int V) {
  const float rest = fmaxf(S - 1.0f, 1e-12f);
  return 0x1p-19f + 0x1p-22f * (rest / S * log2f((float)V / rest) + 1.0f);
}

// A row's elements in the order of the ids: the elements in front of the
// vectors, the vectors in runs, the elements after them.  Run q of thread k:
// the vectors (q per + j) TH + k, j < per; of all threads: `per` TH vectors.
// high: this thread's runs' maxima, TH apart.
template <typename E, int TH>
struct SampleRow {
  Row<E> r;
  const float* high;
  int per, runs;
  __device__ __forceinline__ SampleRow(const E* row, int V, const float* h) : r(row, V), high(h) {
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
  // Runs without a logit of rank `least` are skipped.
  __device__ __forceinline__ bool has(int q, uint32_t least) const { return rank_value(high[q * TH]) >= least; }
  template <typename F>
  __device__ __forceinline__ void all(uint32_t least, F f) const {
    front(f);
    for (int q = 0; q < runs; ++q)
      if (has(q, least)) run(q, f);
    back(f);
  }
};

// Exclusive sum over the block's threads, and the total.  `turn` changes from
// call to call: one barrier is then enough.
template <int TH>
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t& total, SampleShared<TH>& sh, int& turn) {
  constexpr int NW = TH / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) sh.scan[turn][warp] = incl;
  __syncthreads();
  uint64_t w = lane < NW ? sh.scan[turn][lane] : 0;
  turn ^= 1;
  total = warp_sum64(w);
  return incl - v + warp_sum64(lane < warp ? w : 0);
}

// The first id up to which the sum of whole numbers over the row is above
// target(sum over the row): sh.id, sh.x, and the sum before and with it,
// sh.before, sh.after.  own(q): this thread's sum of run q; f(x, id) one
// element's.  sh.id = -1 where the elements of the run do not reach what its
// sum says (fast weights).  Returns the sum over the row.
template <typename E, int TH, typename S, typename F, typename G>
__device__ __forceinline__ uint64_t pick(const SampleRow<E, TH>& row, S own, F f, G target_of, SampleShared<TH>& sh,
                                         int& turn) {
  constexpr int NW = TH / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t v = 0;
  auto add = [&](float x, int id) { v += f(x, id); };
  for (int q = 0; q < row.runs; ++q) {
    v = warp_sum64(own(q));
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
      sh.id = -1;
    }
  }
  __syncthreads();
  const uint64_t total = sh.pre[row.runs + 2], target = sh.target;
  int e = 0;
  while (e < row.runs + 1 && sh.pre[e + 1] <= target) ++e;
  const uint64_t first = sh.pre[e];
  uint64_t left = target - first;
  // walks the elements of one part of the row in order
  bool done = false;
  auto walk = [&](float x, int id) {
    const uint64_t w = f(x, id);
    if (!done && w > left) {
      done = true;
      sh.id = id;
      sh.x = x;
      sh.before = target - left;
      sh.after = target - left + w;
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
    const uint64_t before = block_scan<TH>(v, sum, sh, turn);
    if (before <= left && left < before + v) {
      left -= before;
      for (int i = i0; i < i1 && !done; ++i) row.vector(row.r.vec()[i], i, walk);
    }
  }
  __syncthreads();
  return total;
}
// The same with the runs' sums from their elements; runs without a logit of
// rank `least` add nothing.
template <typename E, int TH, typename F, typename G>
__device__ __forceinline__ uint64_t pick_all(const SampleRow<E, TH>& row, uint32_t least, F f, G target_of,
                                             SampleShared<TH>& sh, int& turn) {
  return pick<E, TH>(row, [&](int q) {
    uint64_t v = 0;
    if (row.has(q, least)) row.run(q, [&](float x, int id) { v += f(x, id); });
    return v;
  }, f, target_of, sh, turn);
}

// Bins of the distance below the row's maximum in the order of rank_value: by
// 1/64 of a power of two over sixteen of them, then by half of one.
__device__ __forceinline__ int first_bin(uint32_t d) {
  return d < (1u << 27) ? (int)(d >> 17) : kSaNear + (int)((d - (1u << 27)) >> 22);
}
__device__ __forceinline__ uint32_t first_bin_start(int b) {
  return b < kSaNear ? (uint32_t)b << 17 : (1u << 27) + ((uint32_t)(b - kSaNear) << 22);
}

// n distinct keys, descending, in list (room for kList).
template <int TH>
__device__ __forceinline__ void sort_list(uint64_t* list, int n) {
  const int k = threadIdx.x;
  if (n <= 256 && n <= TH) {  // each key's place by counting the larger ones
    const uint64_t key = k < n ? list[k] : 0;
    int place = 0;
    if (k < ((n + 31) & ~31))
      for (int j = 0; j < n; ++j) place += list[j] > key;
    __syncthreads();
    if (k < n) list[place] = key;
    __syncthreads();
    return;
  }
  int size = 64;
  while (size < n) size *= 2;
  for (int i = n + k; i < size; i += TH) list[i] = 0;
  __syncthreads();
  for (int w = 2; w <= size; w *= 2)
    for (int j = w / 2; j > 0; j /= 2) {
      for (int i = k; i < size / 2; i += TH) {
        const int a = (i / j) * 2 * j + (i & (j - 1)), b = a + j;
        const uint64_t x = list[a], y = list[b];
        if ((x < y) == ((a & w) == 0)) list[a] = y, list[b] = x;
      }
      __syncthreads();
    }
}

// Sums of the n weights up to and with each, in their place; returns their sum.
template <int TH>
__device__ __forceinline__ void sum_list(uint64_t* weight, int n, SampleShared<TH>& sh, int& turn) {
  constexpr int PER = SampleShared<TH>::kList / TH;
  uint64_t w[PER], v = 0, total;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = (int)threadIdx.x * PER + i;
    v += j < n ? weight[j] : 0;
    w[i] = v;
  }
  const uint64_t before = block_scan<TH>(v, total, sh, turn);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = (int)threadIdx.x * PER + i;
    if (j < n) weight[j] = before + w[i];
  }
  __syncthreads();
}

// The last element of the shortest leading part, in the order of the keys and
// of the keys >= least, that holds `target` elements (COUNT) or weight: its key
// in sh.key, the weight up to and with it in sh.incl, what comes before it in
// sh.before.  False if all together do not.  target >= 1.  With fast weights
// sh.sure_bin is the first bin of distances whose elements may or may not be in
// that part, given an error `err` of the weights.
template <bool COUNT, bool EXACT, typename E, int TH>
__device__ __noinline__ bool select(const SampleRow<E, TH>& row, const Weights& weight, uint64_t target,
                                    uint64_t least, uint32_t skip, uint64_t err, SampleShared<TH>& sh,
                                    SampleWork<TH>& work, int& turn) {
  constexpr int PER = kSaBins / TH, kList = SampleShared<TH>::kList;
  const uint32_t top = rank_value(weight.m);
  const int up = COUNT || EXACT ? 0 : weight.s - 31;  // unit of the bins' weights: 2^-31 for fast ones
  uint32_t d0 = 0, d1 = 0xFFFFFFFFu;  // distances in question
  uint64_t base_n = 0, base_w = 0;    // elements (COUNT) or weight before them
  for (int level = 0;; ++level) {
    int shift = 0;
    while (((d1 - d0) >> shift) >= (uint32_t)kSaBins) ++shift;
    for (int b = threadIdx.x; b < kSaBins; b += TH) work.lo[b] = 0, work.hi[b] = 0;
    if (threadIdx.x == 0) sh.found = 0, sh.listed = 0;
    __syncthreads();
    row.all(skip, [&](float x, int id) {
      const uint64_t key = rank_key(x, (uint32_t)id);
      const uint32_t d = top - (uint32_t)(key >> 32);
      if (x == neg_inf() || key < least || d < d0 || d > d1) return;
      const int b = level == 0 ? first_bin(d) : (int)((d - d0) >> shift);
      if (COUNT) {
        atomicAdd(&work.lo[b], 1u);
      } else if (EXACT) {
        const uint64_t w = weight.exact(x);
        if (w) add64(&work.lo[b], &work.hi[b], w);
      } else {
        const float w = weight.ratio(x);
        const uint32_t v = (uint32_t)Weights::mantissa(w) << 8 >> min(31, 127 - (int)(__float_as_uint(w) >> 23));
        if (w > 0.0f && v) {
          const uint32_t was = atomicAdd(&work.lo[b], v);
          if (was + v < was) atomicAdd(&work.hi[b], 1u);
        }
      }
    });
    __syncthreads();
    auto bin = [&](int b) { return ((uint64_t)work.hi[b] << 32 | work.lo[b]) << up; };
    uint64_t n = 0, total;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += bin(threadIdx.x * PER + i);
    uint64_t n0 = (COUNT ? base_n : base_w) + block_scan<TH>(n, total, sh, turn);
    const uint64_t low = target > err ? target - err : 0;  // what is certainly in the part
    if (!COUNT && level == 0 && n0 < low && low <= n0 + n) {
      uint64_t c = n0;
      int i = 0;
      while (i < PER - 1 && c + bin(threadIdx.x * PER + i) < low) c += bin(threadIdx.x * PER + i++);
      sh.sure_bin = threadIdx.x * PER + i;
    }
    if (!COUNT && level == 0 && threadIdx.x == 0 && low == 0) sh.sure_bin = 0;
    if (n0 < target && target <= n0 + n) {
      int i = 0;
      while (i < PER - 1 && n0 + bin(threadIdx.x * PER + i) < target) n0 += bin(threadIdx.x * PER + i++);
      sh.found = 1, sh.bin = threadIdx.x * PER + i;
      sh.base_n = n0;
    }
    __syncthreads();
    if (!sh.found) return false;
    const int b = sh.bin;
    (COUNT ? base_n : base_w) = sh.base_n;
    if (level == 0) {
      d0 = first_bin_start(b);
      d1 = b + 1 < kSaBins ? first_bin_start(b + 1) - 1 : 0xFFFFFFFFu;
    } else {
      const uint32_t start = d0 + ((uint32_t)b << shift), rest = d1 - start, width = (1u << shift) - 1;
      d0 = start;
      d1 = start + min(rest, width);
    }
    // the elements of the bin, if they are few
    row.all(skip, [&](float x, int id) {
      const uint64_t key = rank_key(x, (uint32_t)id);
      const uint32_t d = top - (uint32_t)(key >> 32);
      if (x != neg_inf() && key >= least && d >= d0 && d <= d1) {
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < (uint32_t)kList) work.list[at] = key;
      }
    });
    __syncthreads();
    const int in = (int)sh.listed;
    if (in <= kList) {
      sort_list<TH>(work.list, in);
      if constexpr (COUNT) {
        if (threadIdx.x == 0) sh.key = work.list[target - base_n - 1];
      } else {
        for (int j = threadIdx.x; j < in; j += TH) work.weight[j] = weight.exact(rank_logit(work.list[j]));
        __syncthreads();
        sum_list<TH>(work.weight, in, sh, turn);
        // the first that reaches the target; the last where the fast weights of
        // the bins reached it and these do not
        for (int j = threadIdx.x; j < in; j += TH) {
          const uint64_t before = base_w + (j ? work.weight[j - 1] : 0), incl = base_w + work.weight[j];
          if (before < target && (target <= incl || j == in - 1))
            sh.key = work.list[j], sh.incl = incl, sh.before = before;
        }
      }
      __syncthreads();
      return true;
    }
    if (d0 == d1) {  // ties: the first of them in the order of the ids
      const uint32_t value = top - d0;
      const uint64_t w1 = COUNT ? 1 : max(1ull, (unsigned long long)weight.exact(rank_logit((uint64_t)value << 32)));
      uint64_t take = COUNT ? target - base_n : (target - base_w + w1 - 1) / w1;
      take = max(1ull, min((unsigned long long)take, (unsigned long long)in));
      pick_all<E, TH>(row, skip, [&](float x, int id) {
        return (uint64_t)(x != neg_inf() && rank_value(x) == value && rank_key(x, (uint32_t)id) >= least);
      }, [&](uint64_t) { return take - 1; }, sh, turn);
      if (threadIdx.x == 0) {
        sh.key = rank_key(sh.x, (uint32_t)sh.id);
        sh.incl = base_w + take * w1, sh.before = sh.incl - w1;
      }
      __syncthreads();
      return true;
    }
  }
}

struct Filters {
  float inv_t, u, top_p, min_p;
  int top_k;  // 0: off
};
struct Drawn {
  int id;
  float x;
  uint64_t total, kept;  // weight of the row and of what is kept
};

// A row whose kept elements are too many for a list.  False where fast weights
// leave the decision open.
template <bool EXACT, typename E, int TH>
__device__ __noinline__ bool draw_many(const SampleRow<E, TH>& row, const Weights& weight, const Filters& a, int V,
                                       uint64_t total, uint64_t err, uint64_t edge, uint32_t skip, Drawn& out,
                                       SampleShared<TH>& sh, SampleWork<TH>& work, int& turn) {
  uint64_t least = 0, mass = total, sum;  // kept: keys from least on
  if (EXACT && a.top_k == 0 && a.top_p < 1.0f) {
    mass = 0;
    row.all(0, [&](float x, int) { mass += weight.exact(x); });
    block_scan<TH>(mass, sum, sh, turn);
    mass = out.total = sum;
  }
  if (a.top_k > 0 && select<true, EXACT, E, TH>(row, weight, (uint64_t)a.top_k, 0, skip, 0, sh, work, turn))
    least = sh.key;
  uint32_t sure = 0xFFFFFFFFu;  // elements nearer to the maximum than this are kept for certain
  if (a.top_p < 1.0f) {
    if (a.top_k > 0) {
      uint64_t v = 0;
      row.all(max(skip, (uint32_t)(least >> 32)),
              [&](float x, int id) { v += rank_key(x, (uint32_t)id) >= least ? weight.of<EXACT>(x) : 0; });
      block_scan<TH>(v, mass, sh, turn);
    }
    const uint64_t target = max(1ull, (unsigned long long)part_of<true>(mass, fmaxf(a.top_p, 0.0f)));
    // the sums of the bins, of unit 2^-31, lose less than one unit per element
    const uint64_t open = EXACT ? 0 : 2 * err + ((uint64_t)V << (weight.s - 31));
    if (select<false, EXACT, E, TH>(row, weight, target, least, skip, open, sh, work, turn)) {
      least = max(least, sh.key);
      const uint64_t w = sh.incl - sh.before;
      if (!EXACT && (target - sh.before <= open || sh.incl < target + open)) {
        // whether a few elements next to the border are kept is open: harmless
        // where they weigh no more than the error, unless one of them is drawn
        if (w > open) return false;
        sure = first_bin_start(sh.sure_bin);
        err += 4 * open;
      }
    }
    __syncthreads();
  }
  least = max(least, edge);
  out.kept = pick_all<E, TH>(row, max(skip, (uint32_t)(least >> 32)), [&](float x, int id) {
    return x != neg_inf() && rank_key(x, (uint32_t)id) >= least ? weight.of<EXACT>(x) : 0;
  }, [&](uint64_t all) { return part_of<false>(all, a.u); }, sh, turn);
  out.id = sh.id, out.x = sh.x;
  if (EXACT) return true;
  if (sh.id < 0 || rank_value(weight.m) - rank_value(sh.x) >= sure) return false;
  return (sh.before == 0 || sh.target - sh.before > err) && (sh.after >= out.kept || sh.after - sh.target > err);
}

template <typename E, int TH>
__global__ void __launch_bounds__(TH, 1024 / TH) sample_tokens_kernel(SampleArgs a) {
  constexpr int NW = TH / 32, kList = SampleShared<TH>::kList;
  extern __shared__ uint4 smem[];
  uint4* ring = smem;
  SampleWork<TH>& work = *reinterpret_cast<SampleWork<TH>*>(smem);
  SampleShared<TH>& sh = *reinterpret_cast<SampleShared<TH>*>(reinterpret_cast<char*>(smem) + kSaSmem<TH> -
                                                             sizeof(SampleShared<TH>));
  float* highs = reinterpret_cast<float*>(reinterpret_cast<char*>(smem) + kSaSmem<TH> - sizeof(SampleShared<TH>) -
                                          TH * kSaRuns * 8) + threadIdx.x;
  float* sums = highs + TH * kSaRuns;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < 64)
    sh.exp2[threadIdx.x] = (uint64_t)__float2ll_rn(kExp2Tab[threadIdx.x][0] * 0x1p62f) +
                           (uint64_t)__float2ll_rn(kExp2Tab[threadIdx.x][1] * 0x1p62f);
  begin_kernel();
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* logits = static_cast<const E*>(a.logits) + t * a.ld;
    const SampleRow<E, TH> row(logits, a.V, highs);
    Filters fl;
    fl.inv_t = a.inv_t ? a.inv_t[t] : 1.0f, fl.u = a.u[t];
    fl.top_p = a.top_p ? a.top_p[t] : 1.0f, fl.min_p = a.min_p ? a.min_p[t] : 0.0f;
    fl.top_k = a.top_k ? a.top_k[t] : 0;
    if (fl.top_k < 0 || fl.top_k >= a.V) fl.top_k = 0;
    const bool params = fl.inv_t >= 1e-6f && fl.inv_t <= 1e6f && fl.u >= 0.0f && fl.u < 1.0f && fl.top_p == fl.top_p &&
                        fl.min_p == fl.min_p;
    // ---- one pass: maximum and sum of each run ----
    Weights weight;
    weight.ch = __fmul_rn(fl.inv_t, kLog2e);
    weight.cl = fmaf(fl.inv_t, 1.92596303e-8f, fmaf(fl.inv_t, kLog2e, -weight.ch));  // log2(e) = kLog2e + 1.93e-8
    weight.s = min(52, 63 - (32 - __clz(a.V - 1)));
    weight.exp2 = sh.exp2;
    const float c = weight.ch;
    float m = neg_inf();
    {
      auto part = [&](int64_t) { return Part{row.r.vec(), row.r.nvec}; };
      Stream<TH, kSaU, kSaD, 1, E, decltype(part)> stream(part, ring + threadIdx.x, TH, threadIdx.x, t, 1, t + 1);
      if (fl.min_p > 0.0f && threadIdx.x == TH - 1) {
        const double e = log((double)fminf(fl.min_p, 1.0f)) / (double)fl.inv_t;
        sh.edge[0] = (float)e;
        sh.edge[1] = (float)(e - (double)(float)e);
      }
      Run<false> acc;
      float high = neg_inf();
      int q = 0, left = row.per / kSaU;
      stream.row(row.r.nvec, [](uint4*, int) {}, [&](const auto& v, int) {
        high = max_nan(high, acc.add(v, c, E()));
        if (q < kSaRuns) highs[q * TH] = high, sums[q * TH] = acc.s;
        if (--left == 0) {
          m = max_nan(m, high);
          ++q, left = row.per / kSaU, high = neg_inf(), acc = Run<false>();
        }
      });
      m = max_nan(m, high);
      cp_async_wait_all();
    }
    row.front([&](float x, int) { m = max_nan(m, x); });
    row.back([&](float x, int) { m = max_nan(m, x); });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane == 0) sh.wmax[warp] = m;
    __syncthreads();
    m = lane < NW ? sh.wmax[lane] : neg_inf();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (!params || !(m <= 3.402823466e+38f) || m == neg_inf()) {
      if (threadIdx.x == 0) {
        const bool none = params && m == neg_inf();
        a.tokens[t] = -1;
        if (a.logprob) a.logprob[t] = none ? neg_inf() : quiet_nan();
        if (a.kept_logprob) a.kept_logprob[t] = none ? neg_inf() : quiet_nan();
        if (!params) set_status(a.status, MOE_STATUS_BAD_SAMPLING);
        if (!(m <= 3.402823466e+38f)) set_status(a.status, MOE_STATUS_NONFINITE_LOGITS);
      }
      __syncthreads();
      continue;
    }
    weight.m = m;
    // the runs' sums from their own shifts to the maximum
    const float mc = __fmul_rn(m, c), M = fmaxf(ceilf(mc), -kShiftLimit);
    const float to_m = exp2_fast((M - mc) - fmaf(m, c, -mc));
    auto run_sum = [&](int q) {
      const float h = fmaxf(highs[q * TH], kLowest), shift = fmaxf(ceilf(h * c), -kShiftLimit) - M;
      const float w = sums[q * TH] * exp2_fast(shift) * to_m;
      return (uint64_t)__float2ull_rn(ldexpf(w, weight.s));
    };
    const bool shift_ok = fabsf(mc) <= kShiftLimit;
    const bool filtered = fl.top_k > 0 || fl.top_p < 1.0f || fl.min_p > 0.0f;
    uint64_t edge = 0;  // keys below have less than min_p
    if (fl.min_p > 0.0f) {  // the smallest float that is not below m + ln(min_p) / inv_temperature
      const float e = sh.edge[0], v = m + e, b = v - m, lost = (m - (v - b)) + (e - b);
      const float up = __fadd_ru(v, lost + sh.edge[1]);
      edge = (uint64_t)rank_value(up >= -3.402823466e+38f ? up : kLowest) << 32;  // also where the sum is out of range
    }
    Drawn out;
    uint64_t sum = 0, err = 0;
    if (shift_ok) {
      if (filtered) {
        for (int q = 0; q < row.runs; ++q) sum += run_sum(q);
        row.front([&](float x, int) { sum += weight.fast(x); });
        row.back([&](float x, int) { sum += weight.fast(x); });
        block_scan<TH>(sum, out.total, sh, turn);
      } else {
        out.total = out.kept =
            pick<E, TH>(row, run_sum, [&](float x, int) { return weight.fast(x); },
                        [&](uint64_t all) { return part_of<false>(all, fl.u); }, sh, turn);
        out.id = sh.id, out.x = sh.x;
      }
      const float S = (float)out.total * ldexpf(1.0f, -weight.s);
      err = (uint64_t)((float)out.total * row_delta(S, a.V));
    } else {
      row.all(0, [&](float x, int) { sum += weight.exact(x); });
      block_scan<TH>(sum, out.total, sh, turn);
    }
    bool done = false;
    if (!filtered) {
      done = shift_ok && sh.id >= 0 && (sh.before == 0 || sh.target - sh.before > err) &&
             (sh.after >= out.total || sh.after - sh.target > err);
    } else {
      // ---- a lower bound of what is kept, from the runs' maxima ----
      const uint32_t top = rank_value(m);
      uint32_t skip = (uint32_t)(edge >> 32);
      const bool by_count = fl.top_k > 0, by_mass = !by_count && fl.top_p < 1.0f;
      if (by_count && fl.top_p < 1.0f) skip = 0;  // all of the top_k count for top_p
      if (threadIdx.x == 0) sh.found = 0, sh.listed = 0;
      bool few = true;
      if (by_count || by_mass) {
        for (int b = threadIdx.x; b < kSaNear; b += TH) work.lo[b] = 0, work.hi[b] = 0;
        __syncthreads();
        auto offer = [&](float x) {
          const uint32_t d = top - rank_value(x);
          if (d >= 1u << 27 || x == neg_inf()) return;
          if (by_count) atomicAdd(&work.lo[d >> 17], 1u);
          else add64(&work.lo[d >> 17], &work.hi[d >> 17], weight.fast(x));
        };
        for (int q = 0; q < row.runs; ++q) offer(highs[q * TH]);
        row.front([&](float x, int) { offer(x); });
        row.back([&](float x, int) { offer(x); });
        __syncthreads();
        constexpr int PER = kSaNear / TH;
        uint64_t n = 0, all;
        auto bin = [&](int i) {
          const int b = threadIdx.x * PER + i;
          return (uint64_t)work.hi[b] << 32 | work.lo[b];
        };
#pragma unroll
        for (int i = 0; i < PER; ++i) n += bin(i);
        uint64_t need = fl.top_k;
        if (by_mass) need = part_of<true>(out.total, fmaxf(fl.top_p, 0.0f)), need += (need >> 14) + 1;  // the weights' errors
        uint64_t n0 = block_scan<TH>(n, all, sh, turn);
        if (n0 < need && need <= n0 + n) {
          int i = 0;
          while (i < PER - 1 && n0 + bin(i) < need) n0 += bin(i++);
          sh.found = 1, sh.bin = threadIdx.x * PER + i;
        }
        __syncthreads();
        if (sh.found) skip = max(skip, top - min(top, ((uint32_t)(sh.bin + 1) << 17) - 1));
        else few = skip > 0;  // min_p's bound alone
      } else {
        __syncthreads();
      }
      // ---- the elements from there on, if they are few ----
      if (few) {
        row.all(skip, [&](float x, int id) {
          if (rank_value(x) >= skip && x != neg_inf()) {
            const uint32_t at = atomicAdd(&sh.listed, 1u);
            if (at < (uint32_t)kList) work.list[at] = rank_key(x, (uint32_t)id);
          }
        });
        __syncthreads();
        few = sh.listed <= (uint32_t)kList;
      }
      if (few) {
        int n = (int)sh.listed;
        sort_list<TH>(work.list, n);
        if (fl.top_k > 0) n = min(n, fl.top_k);
        for (int j = threadIdx.x; j < n; j += TH) work.weight[j] = weight.exact(rank_logit(work.list[j]));
        __syncthreads();
        sum_list<TH>(work.weight, n, sh, turn);
        if (fl.top_p < 1.0f) {
          uint64_t mass = by_count ? work.weight[n - 1] : out.total, near = by_count ? 0 : err;
          for (;;) {
            const uint64_t target = max(1ull, (unsigned long long)part_of<true>(mass, fmaxf(fl.top_p, 0.0f)));
            const uint64_t all = work.weight[n - 1];  // below the target where min_p ends the list before top_p does
            if (threadIdx.x == 0) sh.kept = n, sh.found = near && all < target && target - all <= near;
            __syncthreads();
            for (int j = threadIdx.x; j < n; j += TH) {
              const uint64_t before = j ? work.weight[j - 1] : 0, incl = work.weight[j];
              if (before < target && target <= incl) {
                sh.kept = j + 1;
                sh.found = near && ((j && target - before <= near) || incl - target < near);
              }
            }
            __syncthreads();
            if (!sh.found) break;
            // too close for the fast sum of the row
            sum = 0;
            row.all(0, [&](float x, int) { sum += weight.exact(x); });
            block_scan<TH>(sum, mass, sh, turn);
            out.total = mass, near = 0;
          }
          n = sh.kept;
        }
        if (edge) {
          __syncthreads();
          for (int j = threadIdx.x; j < n; j += TH)
            if (work.list[j] >= edge && (j == n - 1 || work.list[j + 1] < edge)) sh.kept = j + 1;
          __syncthreads();
          n = sh.kept;
        }
        out.kept = work.weight[n - 1];
        const uint64_t target = part_of<false>(out.kept, fl.u);
        if (n <= 256 && n <= TH) {  // each by the weight of the lower ids
          if ((int)threadIdx.x < ((n + 31) & ~31)) {
            const int j = threadIdx.x;
            const uint32_t mine = j < n ? (uint32_t)work.list[j] : 0;  // larger for lower ids
            uint64_t before = 0, last = 0;
            for (int i = 0; i < n; ++i) {
              const uint64_t upto = work.weight[i];
              if ((uint32_t)work.list[i] > mine) before += upto - last;
              last = upto;
            }
            if (j < n) {
              const uint64_t w = work.weight[j] - (j ? work.weight[j - 1] : 0);
              if (before <= target && target < before + w) sh.id = rank_id(work.list[j]), sh.x = rank_logit(work.list[j]);
            }
          }
          __syncthreads();
        } else {  // sorted by id
          constexpr int PER = kList / TH;
          uint64_t mine[PER], w[PER];
          uint32_t value[PER];
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int j = threadIdx.x + i * TH;
            mine[i] = j < n ? work.list[j] : 0;
            w[i] = j < n ? work.weight[j] - (j ? work.weight[j - 1] : 0) : 0;
            value[i] = (uint32_t)(mine[i] >> 32);
          }
          __syncthreads();
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int j = threadIdx.x + i * TH;
            if (j < n) work.list[j] = mine[i] << 32 | (uint32_t)j, work.weight[j] = w[i], work.lo[j] = value[i];
          }
          __syncthreads();
          sort_list<TH>(work.list, n);
          uint64_t own = 0, all;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int j = threadIdx.x * PER + i;
            w[i] = j < n ? work.weight[(uint32_t)work.list[j]] : 0;
            own += w[i];
          }
          uint64_t before = block_scan<TH>(own, all, sh, turn);
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int j = threadIdx.x * PER + i;
            if (before <= target && target < before + w[i]) {
              sh.id = rank_id(work.list[j] >> 32);
              sh.x = rank_logit((uint64_t)work.lo[(uint32_t)work.list[j]] << 32);
            }
            before += w[i];
          }
          __syncthreads();
        }
        out.id = sh.id, out.x = sh.x;
        done = true;
      } else if (shift_ok) {
        done = draw_many<false, E, TH>(row, weight, fl, a.V, out.total, err, edge, skip, out, sh, work, turn);
        __syncthreads();
        if (!done)
          draw_many<true, E, TH>(row, weight, fl, a.V, out.total, 0, edge, skip, out, sh, work, turn), done = true;
      }
    }
    if (!done) {  // fast weights leave it open, or are out of range
      __syncthreads();
      draw_many<true, E, TH>(row, weight, fl, a.V, out.total, 0, edge, 0, out, sh, work, turn);
      if (!filtered) out.total = out.kept;
    }
    if (threadIdx.x == 0) {
      const float z = (out.x - m) * fl.inv_t, unit = ldexpf(1.0f, -weight.s);
      const int64_t one = int64_t(1) << weight.s;
      a.tokens[t] = out.id;
      if (a.logprob) a.logprob[t] = z - log1pf((float)((int64_t)out.total - one) * unit);
      if (a.kept_logprob) a.kept_logprob[t] = z - log1pf((float)((int64_t)out.kept - one) * unit);
    }
    __syncthreads();
  }
}

template <int TH>
static int launch_sample(const SampleArgs& a, cudaStream_t s) {
  const int64_t most = (int64_t)gemm_num_ctas() * (1024 / TH) * 8;
  auto f = a.dtype == MOE_DTYPE_BF16 ? sample_tokens_kernel<uint16_t, TH> : sample_tokens_kernel<float, TH>;
  if (!allow_smem((const void*)f, kSaSmem<TH>, kSaSmem<TH>)) return -1;
  return launch_kernel(f, (unsigned)(a.T < most ? a.T : most), TH, kSaSmem<TH>, 1, s, a);
}
int launch_sample_tokens(const SampleArgs& a, cudaStream_t s) { return launch_sample<512>(a, s); }

}  // namespace moe
