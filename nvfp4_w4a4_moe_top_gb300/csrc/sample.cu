// The draw of a token from each row of logits: temperature, top-k, top-p,
// min-p, and the inverse of the distribution function at a given number u.
// One read of the logits is the bound: four operations and one exponential per
// element.  What is kept is little for most rows, and found from the maxima of
// short runs; the rest of the work then touches a few hundred elements.
//
// Weights are w = 2^((x - m) c) about the row's maximum m, as 64-bit fixed-point
// numbers of unit 2^-s, s such that a row's sum is 2^63 at most (of equal logits; a
// sum of FP32 parts may be off it by a part of 2^-18, and fits 64 bits without a
// sign).  Sums of them are the same in any order: threads and atomics add them as
// they come, and the result is one.
//
// A token is one or another, so a decision is only taken where it is certain.
// Weights from FP32 exponentials make sums with a bounded relative error
// (sum_error).  A row with a decision that is nearer to its border than that, and a
// row that keeps too many elements for a list, stays open and is decided by
// weights to 2^-34, whose own error is below what 64-bit floating-point sums of so
// many elements show.  How often: rows of 131072 ids without filters, one in 200
// where the weight lies in a few ids, one in six where it lies in 40000; with a top_k
// beyond the list (1536, or 1024 for 128 threads) every row that min_p does not
// shorten, peaked or not: 2048 x 131072 with top-k 5000 961 us, with top-p too 985.
//
//   sample_tokens_kernel  rows by a block each; marks open rows in tokens
//   sample_open_kernel    the open rows, by eight blocks each or one
//   sample_open_short_kernel  the same for up to kShortV ids
//   sample_few_kernel     all of it for few rows, a cluster per row
//
// Times (BF16, 131072 ids, us; HBM's floor 79 for 2048 rows, 20 for 512): 2048 rows
// whose weight lies in few ids 113 without filters, 125 with top-k 50, 107 with
// min-p; 2048 rows of which one in ten stays open, with top-p 0.95, 274 (150 and 120
// for the two launches); 512 rows without filters 35, and 37 for the second launch
// where it has a row to decide, 3 where it has none; 2 rows with top-p 11.
#include "exp_table.cuh"
#include "tokens.cuh"

namespace moe {

constexpr int kSaU = 4;     // vectors read together
constexpr int kSaD = 2;     // groups of them on the way
constexpr int kSaRuns = 8;  // runs of a thread at most
constexpr int kSaNear = 1024;  // bins of the sixteen powers of two below the maximum
constexpr float kMinExponent = -42.0f;  // weights below 2^-42 count as 0
// In tokens: left to the second launch, kOpen - (ceil(log2(the row's weight)) + 64
// times the bits of its maximum, if they are 16).
constexpr int kOpen = -2;
template <typename E>
__device__ __forceinline__ int open_flag(int log_s, float m) {
  return kOpen - (log_s + (sizeof(E) == 2 ? (int)(__float_as_uint(m) >> 16) * 64 : 0));
}

// In parts of 27 bits, 32 of which add up in a word.
__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
  constexpr uint32_t k27 = (1u << 27) - 1;
  const uint32_t a = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)v & k27);
  const uint32_t b = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)(v >> 27) & k27);
  const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)(v >> 54));
  return a + ((uint64_t)b << 27) + ((uint64_t)c << 54);
}

// total p for 0 <= p < 1, rounded down or up to a whole number.
template <bool UP>
__device__ __forceinline__ uint64_t part_of(uint64_t total, float p) {
  const uint32_t bits = __float_as_uint(p);
  const int down = 126 - (int)(bits >> 23);  // p = mantissa 2^-24 2^-down
  if (!(p >= 0x1p-63f)) return UP && p > 0.0f && total > 0 ? 1 : 0;  // a part of 2^63, or little more
  const uint64_t a = (uint64_t)((bits & 0x7FFFFFu) | 0x800000u) << 40, hi = __umul64hi(total, a);
  const bool rest = (total * a | (hi & ((1ull << down) - 1))) != 0;
  return (hi >> down) + (UP && rest ? 1 : 0);
}

// w as a fixed-point number of unit 2^-s, 43 <= s <= 52, 0 <= w < 2^(64 - s).
__device__ __forceinline__ uint64_t fixed(float w, int s) {
  const int e = (int)(__float_as_uint(w) >> 23) - 127;
  const uint64_t v = ((__float_as_uint(w) & 0x7FFFFFu) | 0x800000u);
  return e < -s ? 0 : e + s >= 23 ? v << (e + s - 23) : v >> (23 - e - s);
}

template <int TH>
struct SampleShared {
  static constexpr int NW = TH / 32;
  static constexpr int kList = TH < 256 ? 1024 : 1536;  // weighed elements: a longer top_k leaves the row open
  uint64_t exp2[64];               // 2^(j/64) 2^62
  uint64_t part[kSaRuns + 2][NW];  // sums of the runs by warp; the row's ends
  uint64_t sums[kSaRuns + 2];      // of all warps
  uint64_t scan[2][NW];
  float wmax[NW];
  float edge[2];  // ln(min_p) / inv_temperature, a pair
  // results that one thread finds for all
  uint64_t target, before, after, left;
  uint32_t found, listed, hot;
  int bin, id, kept, at;
  float x;
};
// What shares its memory with the ring that the logits come through.
template <int TH>
struct SampleWork {
  static constexpr int kHot = TH * kSaRuns, kListed = TH < 256 ? 1024 : 2048;
  uint64_t list[kListed], weight[SampleShared<TH>::kList];
  union {
    struct {
      uint32_t lo[kSaNear], hi[kSaNear];
    };
    uint32_t hot[kHot];      // thread, run << 16
    uint64_t group[kSaNear]; // sums of 32 vectors of one run, of 2^15 vectors at most
  };
};
template <int TH>
constexpr int kSaRing = TH * kSaU * kSaD * 16;
template <int TH>
constexpr int kSaSmem = (kSaRing<TH> > (int)sizeof(SampleWork<TH>) ? kSaRing<TH> : (int)sizeof(SampleWork<TH>)) +
                        TH * kSaRuns * 8 + (int)sizeof(SampleShared<TH>);

// Blocks of an SM, as many as its shared memory holds.
template <int TH>
constexpr int kSaBlocks = TH == 128 ? 6 : 1024 / TH;

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
  __device__ __forceinline__ uint64_t fast(float x) const {
    const float w = ratio(x);  // in [0, 1]
    return fixed(w, s);
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
};

// Bounds of the relative error of a row's sums of V weights with sum S >= 1.  The
// exponential is off by 2^-22 of itself.  A weight 2^-t, t >= 0, is off by t ln 2
// times each relative error of its exponent: 2^-24 for each rounding (one in the
// pass over the row, the difference and the product in a weight by itself), and
// the part of c that ch leaves out.  (t up to 1 larger in the pass, whose weights
// are about the shift.)  The mean of t over the weights is at most (S - 1) / S
// log2(V / (S - 1)), its value where all but the first are equal.  `adds`: the
// FP32 additions that an element goes through.
__device__ __forceinline__ float sum_error(float S, int V, const float cl_over_ch, int roundings, int adds) {
  const float rest = fmaxf(S - 1.0f, 1e-12f);
  const float t = __fdividef(rest, S) * __log2f(__fdividef((float)V, rest)) + 1.01f;
  return 0x1p-22f + 0x1p-24f * (float)adds + 0.7f * t * (0x1p-24f * (float)roundings + cl_over_ch);
}
// The error of a sum W of n weights by themselves, to add to sum_error's of the row:
// their t is their own, at most log2(n / W) on average, as a part of light weights
// has a larger one than its row.  3 additions in a vector; the last 2^-22 is of the
// factor that brings the pass's sums, which say where the part begins, to the maximum.
__device__ __forceinline__ float part_error(float W, int n, const float cl_over_ch) {
  const float t = __log2f(__fdividef((float)n, fmaxf(W, 1e-12f))) + 1.01f;
  return W * (0x1p-21f + 0x1p-24f * 3.0f + 0.7f * t * (0x1p-23f + cl_over_ch));
}

// Maximum and sum of a run in the pass over the row: about its own integer
// shift, as Run's (learner.cuh), with four sums of pairs for a batch of vectors,
// so that an element goes through few additions.
struct RunSum {
  float m = neg_inf(), M = -kShiftLimit, s = 0.0f;
  static __device__ __forceinline__ float shift_of(float m, float c) {
    return fmaxf(ceilf(fmaxf(m, kLowest) * c), -kShiftLimit);
  }
  __device__ __forceinline__ void raise(float x, float c) {
    m = max_nan(m, x);
    const float n = shift_of(m, c);
    s *= exp2_fast(M - n);
    M = n;
  }
  template <int N>
  __device__ __forceinline__ void take(const uint64_t (&x)[N], float c) {
    const uint64_t nM2 = f32x2_pack(-M, -M), c2 = f32x2_pack(c, c);
    uint64_t w[4] = {0ull, 0ull, 0ull, 0ull}, none[1] = {0ull};
#pragma unroll
    for (int i = 0; i < N; ++i) Run<false>::step(x[i], c2, nM2, w[i & 3], none[0]);
    float a, b;
    unpack2(add_f32x2(add_f32x2(w[0], w[1]), add_f32x2(w[2], w[3])), a, b);
    s += a + b;
  }
  template <int U>
  __device__ __forceinline__ void add(const uint4 (&v)[U], float c, uint16_t) {
    uint32_t w[4 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[4 * u] = v[u].x, w[4 * u + 1] = v[u].y, w[4 * u + 2] = v[u].z, w[4 * u + 3] = v[u].w;
    uint32_t mx[4] = {w[0], w[1], w[2], w[3]};
#pragma unroll
    for (int i = 4; i < 4 * U; ++i) mx[i & 3] = max_nan_bf16x2(mx[i & 3], w[i]);
    const uint32_t mp = max_nan_bf16x2(max_nan_bf16x2(mx[0], mx[1]), max_nan_bf16x2(mx[2], mx[3]));
    raise(max_nan(bf16_lo(mp), bf16_hi(mp)), c);
    uint64_t x[4 * U];
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) x[i] = f32x2_pack(bf16_lo(w[i]), bf16_hi(w[i]));
    take(x, c);
  }
  template <int U>
  __device__ __forceinline__ void add(const uint4 (&v)[U], float c, float) {
    uint64_t x[2 * U];
    float mx = neg_inf();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float a = __uint_as_float(v[u].x), b = __uint_as_float(v[u].y), d = __uint_as_float(v[u].z),
                  e = __uint_as_float(v[u].w);
      mx = max_nan(mx, max_nan(max_nan(a, b), max_nan(d, e)));
      x[2 * u] = f32x2_pack(a, b), x[2 * u + 1] = f32x2_pack(d, e);
    }
    raise(mx, c);
    take(x, c);
  }
};

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
  __device__ __forceinline__ bool has(int q, uint32_t least) const { return least == 0 || rank_value(high[q * TH]) >= least; }
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

// The part of the row with the target: e = 0 the elements before the vectors, 1
// + q run q, then the elements after them.  Finds in it the first id up to which
// the sum of f(x, id) is above `left`; `first`: the sum before the part.  sh.id
// (-1 if the elements do not reach it), sh.x, and the sum over the row before and
// with that element, sh.before, sh.after.
// (-1 too if the sums of vectors and the elements differ.)  of_vector: the sum of
// f over the elements of a vector.
template <typename E, int TH, typename F, typename H>
__device__ __forceinline__ void pick_in(const SampleRow<E, TH>& row, int e, uint64_t left, uint64_t first, F f,
                                        H of_vector, SampleShared<TH>& sh, uint64_t* group, int& turn) {
  constexpr int NW = TH / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto walk = [&](float x, int id, uint64_t& before, bool& done) {
    const uint64_t w = f(x, id);
    if (!done && before + w > left) {
      done = true;
      sh.id = id, sh.x = x;
      sh.before = first + before, sh.after = first + before + w;
    }
    before += w;
  };
  if (threadIdx.x == 0) sh.id = -1, sh.at = -1;
  if (e == 0 || e == row.runs + 1) {
    if (threadIdx.x == 0) {
      const int i0 = e == 0 ? 0 : row.r.tail_start(), n = e == 0 ? row.r.head : row.r.tail;
      uint64_t before = 0;
      bool done = false;
      for (int i = 0; i < n && !done; ++i) walk(to_f32(row.r.p[i0 + i]), i0 + i, before, done);
    }
    __syncthreads();
    return;
  }
  // sums of 32 vectors in a row, then the vectors, then the elements
  const int start = (e - 1) * row.per * TH;
  for (int j = 0; j < row.per; j += kSaU) {
    uint4 v[kSaU];
    const int i0 = start + j * TH + (int)threadIdx.x;
#pragma unroll
    for (int u = 0; u < kSaU; ++u) v[u] = row.r.vec()[min(i0 + u * TH, row.r.nvec - 1)];
#pragma unroll
    for (int u = 0; u < kSaU; ++u) {
      const uint64_t w = warp_sum64(i0 + u * TH < row.r.nvec ? of_vector(v[u]) : 0);
      if (lane == 0) group[(j + u) * NW + warp] = w;
    }
  }
  __syncthreads();
  const int n = row.per * NW, each = (n + TH - 1) / TH, g0 = (int)threadIdx.x * each;
  uint64_t sum = 0, total;
  for (int g = g0; g < min(g0 + each, n); ++g) sum += group[g];
  uint64_t before = block_scan<TH>(sum, total, sh, turn);
  if (before <= left && left < before + sum) {
    int g = g0;
    while (before + group[g] <= left) before += group[g++];
    sh.at = g, sh.left = before;
  }
  __syncthreads();
  if (warp == 0 && sh.at >= 0) {
    const int i = start + sh.at * 32 + lane;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    uint64_t w = 0;
    if (i < row.r.nvec) {
      v = row.r.vec()[i];
      row.vector(v, i, [&](float x, int id) { w += f(x, id); });
    }
    uint64_t incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t m = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += m;
    }
    uint64_t b = sh.left + incl - w;
    if (b <= left && left < b + w) {
      bool done = false;
      row.vector(v, i, [&](float x, int id) { walk(x, id, b, done); });
    }
  }
  __syncthreads();
}

// sh.part summed over the warps; the row's sum.  After the barrier that follows
// the last of sh.part.
template <typename E, int TH>
__device__ __forceinline__ uint64_t sum_parts(const SampleRow<E, TH>& row, SampleShared<TH>& sh) {
  constexpr int NW = TH / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = warp; e < row.runs + 2; e += NW) {
    const int n = e == 0 || e == row.runs + 1 ? 1 : NW;
    const uint64_t v = warp_sum64(lane < n ? sh.part[e][lane] : 0);
    if (lane == 0) sh.sums[e] = v;
  }
  __syncthreads();
  uint64_t total = 0;
  for (int e = 0; e < row.runs + 2; ++e) total += sh.sums[e];
  return total;
}

// The part with the target, from sh.sums.
template <typename E, int TH>
__device__ __forceinline__ int find_part(const SampleRow<E, TH>& row, uint64_t target, uint64_t& first,
                                         const SampleShared<TH>& sh) {
  int e = 0;
  first = 0;
  while (e < row.runs + 1 && first + sh.sums[e] <= target) first += sh.sums[e++];
  return e;
}

// The ends of the row into sh.part, by the first warp.
template <typename E, int TH, typename F>
__device__ __forceinline__ void sum_ends(const SampleRow<E, TH>& row, F f, SampleShared<TH>& sh) {
  if (threadIdx.x >= 32) return;
  uint64_t a = 0, b = 0;
  if (row.r.head) row.front([&](float x, int id) { a = f(x, id); });
  if (row.r.tail) row.back([&](float x, int id) { b = f(x, id); });
  if (row.r.head) a = warp_sum64(a);
  if (row.r.tail) b = warp_sum64(b);
  if (threadIdx.x == 0) sh.part[0][0] = a, sh.part[row.runs + 1][0] = b;
}

// The first id up to which the sum of f over the row is above part u of all of
// it, as pick_in gives it, with the target in sh.target.  sh.part has the runs'
// sums.  group: room for the sums within a run, in use by nobody.  Returns the sum
// over the row, which is not 0.
template <typename E, int TH, typename F, typename H>
__device__ __forceinline__ uint64_t pick(const SampleRow<E, TH>& row, float u, F f, H of_vector, SampleShared<TH>& sh,
                                         uint64_t* group, int& turn) {
  sum_ends<E, TH>(row, f, sh);
  __syncthreads();
  const uint64_t total = sum_parts<E, TH>(row, sh);
  const uint64_t target = min((unsigned long long)part_of<false>(total, u), (unsigned long long)total - 1);
  uint64_t first;
  const int e = find_part<E, TH>(row, target, first, sh);
  if (threadIdx.x == 0) sh.target = target;
  pick_in<E, TH>(row, e, target - first, first, f, of_vector, sh, group, turn);
  return total;
}

// n distinct keys, descending, in list (room for the next power of two).
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

// Sums of the n <= LIST weights up to and with each, in their place.
template <int LIST, int TH>
__device__ __forceinline__ void sum_list(uint64_t* weight, int n, SampleShared<TH>& sh, int& turn) {
  constexpr int PER = (LIST + TH - 1) / TH;
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

struct Filters {
  float inv_t, u, top_p, min_p;
  int top_k;  // 0: off
};
struct Drawn {
  int id;
  float x;
  uint64_t total, kept;  // weight of the row and of what is kept
};

// A row's numbers, and whether they are in range.
__device__ __forceinline__ Filters filters_of(const SampleArgs& a, int64_t t, bool& good) {
  Filters f;
  f.inv_t = a.inv_t ? a.inv_t[t] : 1.0f, f.u = a.u[t];
  f.top_p = a.top_p ? a.top_p[t] : 1.0f, f.min_p = a.min_p ? a.min_p[t] : 0.0f;
  f.top_k = a.top_k ? a.top_k[t] : 0;
  if (f.top_k < 0 || f.top_k >= a.V) f.top_k = 0;
  good = f.inv_t >= 1e-6f && f.inv_t <= 1e6f && f.u >= 0.0f && f.u < 1.0f && f.top_p == f.top_p && f.min_p == f.min_p;
  return f;
}
// ln(min_p) / inv_temperature as a pair.
__device__ __forceinline__ void min_p_edge(const Filters& f, float (&edge)[2]) {
  const double e = log((double)fminf(f.min_p, 1.0f)) / (double)f.inv_t;
  edge[0] = (float)e;
  edge[1] = (float)(e - (double)(float)e);
}
// The key from which on logits have min_p: of the smallest float that is not
// below m + ln(min_p) / inv_temperature.
__device__ __forceinline__ uint64_t min_p_key(float m, const float (&edge)[2]) {
  const float v = m + edge[0], b = v - m, lost = (m - (v - b)) + (edge[0] - b);
  const float up = __fadd_ru(v, lost + edge[1]);
  return (uint64_t)rank_value(up >= -3.402823466e+38f ? up : kLowest) << 32;  // also where the sum is out of range
}
__device__ __forceinline__ Weights weights_of(float inv_t, float m, int V, const uint64_t* exp2) {
  Weights w;
  w.m = m;
  w.ch = __fmul_rn(inv_t, kLog2e);
  w.cl = fmaf(inv_t, 1.92596303e-8f, fmaf(inv_t, kLog2e, -w.ch));  // log2(e) = kLog2e + 1.93e-8
  w.s = min(52, 63 - (32 - __clz(V - 1)));
  w.exp2 = exp2;
  return w;
}
template <int TH>
__device__ __forceinline__ void load_exp2(SampleShared<TH>& sh) {
  if (threadIdx.x < 64)
    sh.exp2[threadIdx.x] = (uint64_t)__float2ll_rn(kExp2Tab[threadIdx.x][0] * 0x1p62f) +
                           (uint64_t)__float2ll_rn(kExp2Tab[threadIdx.x][1] * 0x1p62f);
}
__device__ __forceinline__ void put_drawn(const SampleArgs& a, int64_t t, const Drawn& d, float inv_t, float m, int s) {
  const float z = (d.x - m) * inv_t, unit = ldexpf(1.0f, -s);
  const uint64_t one = uint64_t(1) << s;  // the rest, below 0 where a sum of FP32 parts is below 1
  a.tokens[t] = d.id;
  if (a.logprob) a.logprob[t] = z - log1pf((float)(int64_t)(d.total - one) * unit);
  if (a.kept_logprob) a.kept_logprob[t] = z - log1pf((float)(int64_t)(d.kept - one) * unit);
}

// The end of a row, from its runs' maxima and sums.  Without filters the runs' sums
// give the run with the token, which is read again (from L2).  With filters the
// maxima bound what is kept from below: at least top_k of them, or maxima with
// top_p of the weight, reach a value, so only runs whose maximum reaches it are read
// again, and what they hold from there on is listed, sorted, and weighed exactly;
// only the row's sum, which top_p alone needs, is then of FP32 weights.  The
// barriers and dependent reads of all this take 5 to 10 us, which other blocks'
// reads cover.  Returns 0 with the token and its numbers written, or what marks the
// row as open.  own: this thread's maximum; highs, sums: its runs', TH apart.
template <typename E, int TH>
__device__ __forceinline__ int end_row(const SampleArgs& a, int64_t t, const SampleRow<E, TH>& row, const Filters& fl,
                                       bool params, Weights weight, float own, const float* highs, const float* sums,
                                       SampleShared<TH>& sh, SampleWork<TH>& work, int& turn) {
  constexpr int NW = TH / 32, kList = SampleShared<TH>::kList;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float c = weight.ch;
  float m = own;
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
    return 0;
  }
  weight.m = m;
  // the runs' sums from their own shifts to the maximum, of unit 2^-s
  const float mc = __fmul_rn(m, c), M = fmaxf(ceilf(mc), -kShiftLimit), cl_ch = fabsf(weight.cl) / weight.ch;
  const float to_m = exp2_fast((M - mc) - fmaf(m, c, -mc));
  auto run_float = [&](int q) {  // at most 2^10
    return sums[q * TH] * exp2_fast(RunSum::shift_of(highs[q * TH], c) - M) * to_m;
  };
  const bool shift_ok = fabsf(mc) <= kShiftLimit;
  const bool filtered = fl.top_k > 0 || fl.top_p < 1.0f || fl.min_p > 0.0f;
  uint64_t edge = 0;  // keys below have less than min_p
  if (fl.min_p > 0.0f) edge = min_p_key(m, sh.edge);
  Drawn out;
  uint64_t sum = 0, err;  // err: of sums of the pass
  const float unit = ldexpf(1.0f, -weight.s);
  int e = 0;  // the part of the row with the token
  if (filtered && !shift_ok) {  // the pass's weights are out of range
    row.all(0, [&](float x, int) { sum += weight.fast(x); });
    block_scan<TH>(sum, out.total, sh, turn);
  } else if (filtered) {
    float w = 0.0f;
    for (int q = 0; q < row.runs; ++q) w += run_float(q);
    sum = fixed(w, weight.s);
    row.front([&](float x, int) { sum += weight.fast(x); });
    row.back([&](float x, int) { sum += weight.fast(x); });
    block_scan<TH>(sum, out.total, sh, turn);
  }
  if (!filtered) {
    // the warp's sums of the eight runs: lane l ends with run l / 4's
    float w[kSaRuns];
#pragma unroll
    for (int q = 0; q < kSaRuns; ++q) {
      w[q] = 0.0f;
      if (q < row.runs) {
        if (shift_ok) w[q] = run_float(q);
        else row.run(q, [&](float x, int) { w[q] += weight.ratio(x); });
      }
    }
#pragma unroll
    for (int h = 4, o = 16; h > 0; h /= 2, o /= 2)
#pragma unroll
      for (int q = 0; q < h; ++q) {
        const float keep = lane & o ? w[q + h] : w[q], give = lane & o ? w[q] : w[q + h];
        w[q] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
      }
    w[0] += __shfl_xor_sync(0xFFFFFFFFu, w[0], 2);
    w[0] += __shfl_xor_sync(0xFFFFFFFFu, w[0], 1);
    if ((lane & 3) == 0 && lane / 4 < row.runs) sh.part[lane / 4 + 1][warp] = fixed(w[0], weight.s);
    out.total = out.kept = pick<E, TH>(row, fl.u, [&](float x, int) { return weight.fast(x); }, [&](const uint4& v) {
      constexpr int N = Row<E>::kVec;
      float x[N];
      unpack(v, x);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = weight.ratio(x[e]);
#pragma unroll
      for (int h = N / 2; h > 0; h /= 2)
#pragma unroll
        for (int e = 0; e < h; ++e) x[e] += x[e + h];
      return fixed(x[0], weight.s);
    }, sh, work.group, turn);
    out.id = sh.id, out.x = sh.x;
    uint64_t first;
    e = find_part<E, TH>(row, sh.target, first, sh);
  }
  {
    // in the pass 3 additions per sum of pairs, 3 to join them, one per batch of
    // a run, a product with to_m; then 5 over the warp, or, with the filters, 8
    // for the thread's runs, and to_m's own error, which is otherwise the same
    // for all.  Where the range of the pass is exceeded, as many as a run has
    // elements, and 5 over the warp.
    const float S = (float)out.total * unit;
    err = shift_ok ? (uint64_t)((float)out.total * sum_error(S, a.V, cl_ch, 1, 7 + row.per / kSaU + (filtered ? 12 : 5)))
                   : (uint64_t)((float)out.total * sum_error(S, a.V, cl_ch, 2, filtered ? 0 : row.per * Row<E>::kVec + 5));
    err += (uint64_t)a.V << (weight.s - 42);  // weights below 2^-42, which the pass adds
    // The elements before and after the vectors are weights by themselves: one rounding
    // more, 0.7 2^-24 w t each, and w t is 0.531 at most; and without to_m.
    err += (uint64_t)(row.r.head + row.r.tail) * (3ull << (weight.s - 27));
    if (!filtered) {
      err += (sh.sums[0] + sh.sums[row.runs + 1]) >> 22;
      err += (uint64_t)ldexpf(part_error((float)sh.sums[e] * unit, min(a.V, row.per * TH * Row<E>::kVec), cl_ch), weight.s);
    }
  }
  const int open = open_flag<E>(64 - __clzll((long long)out.total) - weight.s, m);
  bool done = false;
  if (!filtered) {
    // In front of it there is nothing where `before` is 0; behind it there may be ids
    // where `after` is the row's sum, which rounds light ones away.
    done = sh.id >= 0 && (sh.before == 0 || sh.target - sh.before > err) &&
           sh.after > sh.target && sh.after - sh.target > err;
  } else {
    // ---- a lower bound of what is kept, from the maxima ----
    const uint32_t top = rank_value(m);
    uint32_t skip = (uint32_t)(edge >> 32);
    const bool by_count = fl.top_k > 0, by_mass = !by_count && fl.top_p < 1.0f;
    if (by_count && fl.top_p < 1.0f) skip = 0;  // all of the top_k count for top_p
    if (threadIdx.x == 0) sh.found = 0, sh.listed = 0, sh.hot = 0;
    bool few = true;
    // by all elements where the maxima are fewer than top_k
    for (bool whole = false; by_count || by_mass; whole = true) {
      for (int b = threadIdx.x; b < kSaNear; b += TH) work.lo[b] = 0, work.hi[b] = 0;
      __syncthreads();
      auto offer = [&](float x, uint64_t w) {
        const uint32_t d = top - rank_value(x);
        if (d >= 1u << 27 || x == neg_inf()) return;
        if (by_count) atomicAdd(&work.lo[d >> 17], 1u);
        else add64(&work.lo[d >> 17], &work.hi[d >> 17], w);
      };
      if (whole) {
        row.all(0, [&](float x, int) { offer(x, 0); });
      } else if (by_count && fl.top_k <= TH / 4) {
        offer(own, 0);
      } else if (by_count) {
        for (int q = 0; q < row.runs; ++q) offer(highs[q * TH], 0);
      } else {
        // the weights that matter: all others together are below a quarter of
        // what top_p leaves out
        const float least = (1.0f - fl.top_p) * (float)out.total * unit * 0.25f / (float)(TH * kSaRuns);
        auto heavy = [&](float x) {
          const float w = weight.ratio(x);
          if (w >= least) offer(x, fixed(w, weight.s));
        };
        for (int q = 0; q < row.runs; ++q) heavy(highs[q * TH]);
        row.front([&](float x, int) { heavy(x); });
        row.back([&](float x, int) { heavy(x); });
      }
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
      // (work.lo is read no more: the list of runs shares its memory)
      if (sh.found) skip = max(skip, top - min(top, ((uint32_t)(sh.bin + 1) << 17) - 1));
      else if (by_count && !whole && fl.top_k <= kList) continue;
      else few = skip > 0;  // min_p's bound alone
      break;
    }
    __syncthreads();
    // ---- the elements from there on, if they are few ----
    if (few) {
      auto offer = [&](float x, int id) {
        if (rank_value(x) >= skip && x != neg_inf()) {
          const uint32_t at = atomicAdd(&sh.listed, 1u);
          if (at < (uint32_t)SampleWork<TH>::kListed) work.list[at] = rank_key(x, (uint32_t)id);
        }
      };
      // the runs that have any, read by all threads together
      constexpr int kHot = SampleWork<TH>::kHot;
      if (rank_value(own) >= skip)
        for (int q = 0; q < row.runs; ++q)
          if (row.has(q, skip)) {
            const uint32_t at = atomicAdd(&sh.hot, 1u);
            if (at < (uint32_t)kHot) work.hot[at] = threadIdx.x | (uint32_t)q << 16;
          }
      __syncthreads();
      few = sh.hot <= (uint32_t)kHot;
      if (few) {
        const int items = (int)sh.hot * row.per;
        for (int j = threadIdx.x; j < items; j += TH) {
          const uint32_t who = work.hot[j / row.per];
          const int i = ((int)(who >> 16) * row.per + j % row.per) * TH + (int)(who & 0xFFFFu);
          if (i < row.r.nvec) row.vector(row.r.vec()[i], i, offer);
        }
        row.front(offer);
        row.back(offer);
      }
      __syncthreads();
      few &= sh.listed <= (uint32_t)SampleWork<TH>::kListed && (sh.listed <= (uint32_t)kList || (by_count && fl.top_k <= kList));
    }
    if (few) {
      int n = (int)sh.listed;
      sort_list<TH>(work.list, n);
      if (fl.top_k > 0) n = min(n, fl.top_k);
      for (int j = threadIdx.x; j < n; j += TH) work.weight[j] = weight.exact(rank_logit(work.list[j]));
      __syncthreads();
      sum_list<kList, TH>(work.weight, n, sh, turn);
      if (fl.top_p < 1.0f) {
        const uint64_t mass = by_count ? work.weight[n - 1] : out.total, near = by_count ? 0 : err;
        {
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
        }
        if (sh.found) {  // too close for the fast sum of the row
          __syncthreads();
          return open;
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
      if (n <= 128) {  // each by the weight of the lower ids
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
      } else {  // by the weights of 1024 ranges of ids, then within one
        const int shift = max(0, 32 - __clz(a.V - 1) - 10);
        for (int b = threadIdx.x; b < kSaNear; b += TH) work.lo[b] = work.hi[b] = 0;
        if (threadIdx.x == 0) sh.listed = 0;
        __syncthreads();
        auto weight_of = [&](int j) { return work.weight[j] - (j ? work.weight[j - 1] : 0); };
        for (int j = threadIdx.x; j < n; j += TH) {
          const int b = rank_id(work.list[j]) >> shift;
          add64(&work.lo[b], &work.hi[b], weight_of(j));
        }
        __syncthreads();
        constexpr int PER = kSaNear / TH;
        uint64_t own = 0, all;
        auto bin = [&](int i) {
          const int b = threadIdx.x * PER + i;
          return (uint64_t)work.hi[b] << 32 | work.lo[b];
        };
#pragma unroll
        for (int i = 0; i < PER; ++i) own += bin(i);
        uint64_t before = block_scan<TH>(own, all, sh, turn);
        if (before <= target && target < before + own) {
          int i = 0;
          while (before + bin(i) <= target) before += bin(i++);
          sh.bin = threadIdx.x * PER + i, sh.left = before;
        }
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += TH)
          if (rank_id(work.list[j]) >> shift == sh.bin)
            work.group[atomicAdd(&sh.listed, 1u)] = work.list[j] << 32 | (uint32_t)j;  // larger for lower ids
        __syncthreads();
        const int in = (int)sh.listed;
        for (int i = threadIdx.x; i < in; i += TH) {
          const uint64_t mine = work.group[i];
          uint64_t b = sh.left;
          for (int k = 0; k < in; ++k)
            if (work.group[k] > mine) b += weight_of((int)(uint32_t)work.group[k]);
          const int j = (int)(uint32_t)mine;
          if (b <= target && target < b + weight_of(j)) sh.id = rank_id(work.list[j]), sh.x = rank_logit(work.list[j]);
        }
        __syncthreads();
      }
      out.id = sh.id, out.x = sh.x;
      done = true;
    }
  }
  if (done && threadIdx.x == 0) put_drawn(a, t, out, fl.inv_t, m, weight.s);
  __syncthreads();
  return done ? 0 : open;
}

// A row per block at a time.  The logits come through a ring of asynchronous copies
// per thread (64 KB on the way per SM); each thread keeps maximum and sum of up to
// eight runs of its vectors, so that nothing of the row but these needs to stay.
// HBM's share: 2048 x 131072 with min-p 107 us, 0.74 of the measured copy rate; what
// is missing are the ends of rows (a launch of 1216 rows issues in 57% of its slots,
// 80 instructions per vector of 8).  Two and three times the bytes on the way, runs
// of other lengths, a prefetch of the row that comes next into L2, and the end of a row as a function of its own (its call takes
// registers from the pass) were slower.
template <typename E, int TH>
__global__ void __launch_bounds__(TH, kSaBlocks<TH>) sample_tokens_kernel(SampleArgs a) {
  extern __shared__ uint4 smem[];
  uint4* ring = smem;
  SampleWork<TH>& work = *reinterpret_cast<SampleWork<TH>*>(smem);
  SampleShared<TH>& sh = *reinterpret_cast<SampleShared<TH>*>(reinterpret_cast<char*>(smem) + kSaSmem<TH> -
                                                             sizeof(SampleShared<TH>));
  float* highs = reinterpret_cast<float*>(reinterpret_cast<char*>(smem) + kSaSmem<TH> - sizeof(SampleShared<TH>) -
                                          TH * kSaRuns * 8) + threadIdx.x;
  float* sums = highs + TH * kSaRuns;
  load_exp2(sh);
  begin_kernel();
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* logits = static_cast<const E*>(a.logits) + t * a.ld;
    const SampleRow<E, TH> row(logits, a.V, highs);
    bool params;
    const Filters fl = filters_of(a, t, params);
    // ---- one pass: maximum and sum of each run ----
    const Weights weight = weights_of(fl.inv_t, 0.0f, a.V, sh.exp2);
    const float c = weight.ch;
    float m = neg_inf();
    {
      auto part = [&](int64_t) { return Part{row.r.vec(), row.r.nvec}; };
      Stream<TH, kSaU, kSaD, 1, E, decltype(part)> stream(part, ring + threadIdx.x, TH, threadIdx.x, t, 1, t + 1);
      if (fl.min_p > 0.0f && threadIdx.x == TH - 1) min_p_edge(fl, sh.edge);
      RunSum acc;
      int q = 0, left = row.per / kSaU;
      stream.row(row.r.nvec, [](uint4*, int) {}, [&](const auto& v, int) {
        acc.add(v, c, E());
        highs[q * TH] = acc.m, sums[q * TH] = acc.s;
        if (--left == 0) {
          m = max_nan(m, acc.m);
          q = min(q + 1, kSaRuns - 1), left = row.per / kSaU, acc = RunSum();
        }
      });
      m = max_nan(m, acc.m);
      cp_async_wait_all();
    }
    row.front([&](float x, int) { m = max_nan(m, x); });
    row.back([&](float x, int) { m = max_nan(m, x); });
    const int open = end_row<E, TH>(a, t, row, fl, params, weight, m, highs, sums, sh, work, turn);
    if (open && threadIdx.x == 0) a.tokens[t] = open;
  }
}

// 4 bytes to shared address p of block `rank` of the cluster.
__device__ __forceinline__ void cluster_store(const void* p, uint32_t rank, uint32_t v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// ---- rows that are left open: a team of blocks per row, a part of it each, and
// weights to 2^-34.  The team is a cluster of eight blocks, or, where there are many
// open rows, one block: eight are sooner done with one row, but wait for one
// another.  The sums are whole numbers, so the results are the same. ----
// Sizes of a team's work: threads of a block, bins, listed elements, groups of 32
// vectors, and blocks.
template <int THREADS, int BINS, int LIST, int GROUPS, int TEAM>
struct TeamSizes {
  static constexpr int kThreads = THREADS, kWarps = THREADS / 32, kBins = BINS, kList = LIST, kGroups = GROUPS;
  static constexpr int kTeam = TEAM, kTeamLog = TEAM == 8 ? 3 : 0;
  static constexpr int kNear = BINS / 2, kNearShift = BINS == 4096 ? 16 : 18;  // kNear << kNearShift = 2^27
  static constexpr bool kValues = BINS == 4096;                                // a bin per BF16 value
  static_assert(kNear << kNearShift == 1 << 27, "sixteen powers of two");
};
using LongTeam = TeamSizes<512, 4096, 2048, 1024, 8>;  // groups: (2^20 / 4 / 8) / 32
// Rows of up to kShortV ids, by one small block: many rows on the way, which wait
// for their own barriers only.
using ShortTeam = TeamSizes<128, 1024, 512, 64, 1>;
constexpr int kShortV = 8192;
constexpr int kTeamU = 4;          // vectors read together
constexpr int kClaimed = -(1 << 30);  // in tokens: an open row that a block works on

template <typename C>
struct TeamWork {
  uint64_t power[1024];             // 2^(j/1024) 2^62
  union {
    struct {
      uint64_t list[C::kList], weight[C::kList];
    };
    uint64_t table[C::kBins];      // BF16: the weight of each bin's one value
  };
  uint64_t group[C::kGroups + 2];  // the elements before the vectors, 32 vectors in a row each, the elements after
  uint64_t ties[C::kGroups + 2];
  uint32_t lo[C::kBins], hi[C::kBins];
  uint64_t box[2][2];               // what the blocks tell one another, in turn
  int64_t claimed;                  // a row that a block takes
  int flag, first;
  uint32_t row[2], first_row[2];    // the cluster's next row and its first one: number, flag
  uint32_t rows;                    // open rows that it counted
  uint64_t base, key, incl;
  int edge;
};

// Shared memory of a block that works on few rows.
struct FewWork {
  SampleShared<LongTeam::kThreads> sh;
  union {
    TeamWork<LongTeam> team;
    struct {
      SampleWork<LongTeam::kThreads> work;
      float highs[LongTeam::kThreads * kSaRuns], sums[LongTeam::kThreads * kSaRuns];
    };
  };
  uint32_t open;
};

// Bins of the ranks at and below the row's maximum's, `top`: by 1/128 (1/32) of a
// power of two over sixteen of them, then one bin down to -2^-10, then by 1/64
// (1/16) of a power of two over 32 of them, and the rest.
constexpr uint32_t kNegative = 0x7FFFFFFFu - 0x3A800000u;  // rank of -2^-10
template <typename C>
__device__ __forceinline__ int first_bin(uint32_t top, uint32_t rank) {
  const uint32_t d = top - rank;
  if (d < 1u << 27) return (int)(d >> C::kNearShift);
  return rank >= kNegative ? C::kNear : min(C::kBins - 1, C::kNear + 1 + (int)((kNegative - 1 - rank) >> (C::kNearShift + 1)));
}
// First distance below `top` that is not in a bin before b.
template <typename C>
__device__ __forceinline__ uint32_t first_bin_start(uint32_t top, int b) {
  if (b <= C::kNear) return (uint32_t)b << C::kNearShift;
  const int64_t d = (int64_t)top - (int64_t)kNegative + 1 + ((int64_t)(b - C::kNear - 1) << (C::kNearShift + 1));
  return b >= C::kBins ? 0xFFFFFFFFu : (uint32_t)max((long long)d, 1ll << 27);
}

// A block's part of a row, ids from id0 on, and what the block and its team know.
template <typename E, typename C>
struct Team {
  Row<E> r;
  int id0, rank, size, turn, scan_turn, groups;
  Weights weight;
  SampleShared<C::kThreads>& sh;
  TeamWork<C>& work;

  // Weights to 2^-34 as Weights::exact, but with the powers of 2^(1/1024): the
  // rest's series has three terms, and its one FP32 number is good to 2^-35.  A
  // function object, so that loops keep its numbers in registers.
  struct Exact {
    float m, ch, cl;
    int s;
    const uint64_t* power;
    __device__ __forceinline__ uint64_t operator()(float x) const;
  };
  __device__ __forceinline__ Exact exact_weights() const {
    return {weight.m, weight.ch, weight.cl, weight.s, work.power};
  }
  // f(x, id) on this thread's elements of the part; after(x, n, id) behind each n
  // elements from id on; end(group) behind each group of this warp, in step
  template <typename F, typename G, typename H>
  __device__ __forceinline__ void each(F f, G end, H after) const {
    constexpr int N = Row<E>::kVec;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Row<E> r = this->r;
    const int id0 = this->id0, groups = this->groups;
    for (int g0 = warp; g0 < groups; g0 += kTeamU * C::kWarps) {
      uint4 v[kTeamU];
#pragma unroll
      for (int u = 0; u < kTeamU; ++u) v[u] = r.vec()[min((g0 + u * C::kWarps) * 32 + lane, r.nvec - 1)];
#pragma unroll
      for (int u = 0; u < kTeamU; ++u) {
        const int g = g0 + u * C::kWarps, i = g * 32 + lane;
        if (g >= groups) break;
        if (i < r.nvec) {
          float x[N];
          unpack(v[u], x);
#pragma unroll
          for (int k = 0; k < N; ++k) f(x[k], id0 + r.head + i * N + k);
          after(x, N, id0 + r.head + i * N);
        }
        end(g + 1);
      }
    }
    if (warp == 0) {
      float x[N];
      if (lane < r.head) {
        x[0] = to_f32(r.p[lane]);
        f(x[0], id0 + lane);
        after(x, 1, id0 + lane);
      }
      end(0);
      if (lane < r.tail) {
        const int id = r.tail_start() + lane;
        x[0] = to_f32(r.p[id]);
        f(x[0], id0 + id);
        after(x, 1, id0 + id);
      }
      end(groups + 1);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each(f, [](int) {}, [](const auto&, int, int) {});
  }
  // The largest of this thread's elements.
  __device__ __forceinline__ float high() const {
    float m = neg_inf();
    if constexpr (sizeof(E) == 4) {
      each([&](float x, int) { m = fmaxf(m, x); });
    } else {
      uint32_t w = 0xFF80FF80u;
      for (int i0 = threadIdx.x; i0 < r.nvec; i0 += kTeamU * C::kThreads) {
        uint4 v[kTeamU];
#pragma unroll
        for (int u = 0; u < kTeamU; ++u) v[u] = r.vec()[min(i0 + u * C::kThreads, r.nvec - 1)];
#pragma unroll
        for (int u = 0; u < kTeamU; ++u)
          w = max_nan_bf16x2(w, max_nan_bf16x2(max_nan_bf16x2(v[u].x, v[u].y), max_nan_bf16x2(v[u].z, v[u].w)));
      }
      m = fmaxf(bf16_lo(w), bf16_hi(w));
      if ((int)threadIdx.x < r.head) m = fmaxf(m, to_f32(r.p[threadIdx.x]));
      if ((int)threadIdx.x < r.tail) m = fmaxf(m, to_f32(r.p[r.tail_start() + threadIdx.x]));
    }
    return m;
  }
  // f's sums into the groups
  template <typename F, typename H>
  __device__ __forceinline__ void sums(F f, H after) const {
    uint64_t v = 0;
    uint64_t* group = work.group;
    each([&](float x, int id) { v += f(x, id); }, [&](int g) {
      v = warp_sum64(v);
      if ((threadIdx.x & 31) == 0) group[g] = v;
      v = 0;
    }, after);
    __syncthreads();
  }
  template <typename F>
  __device__ __forceinline__ void sums(F f) const {
    sums(f, [](const auto&, int, int) {});
  }
  __device__ __forceinline__ uint64_t scan(uint64_t v, uint64_t& total) {
    return block_scan<C::kThreads>(v, total, sh, scan_turn);
  }
  __device__ __forceinline__ void sync() const {
    if (C::kTeam == 1 || size == 1) {
      __syncthreads();
    } else {
      cluster_arrive();
      cluster_wait();
    }
  }
  // Two numbers of each block: lane r of every warp gets rank r's (0 from lane 8
  // on).  A barrier of the team.
  __device__ __forceinline__ void share(uint64_t a, uint64_t b, uint64_t& va, uint64_t& vb) {
    const int lane = threadIdx.x & 31;
    uint64_t* box = work.box[turn];
    if (threadIdx.x == 0) box[0] = a, box[1] = b;
    sync();
    va = vb = 0;
    if (C::kTeam == 1 || size == 1) {
      if (lane == 0) va = box[0], vb = box[1];
    } else if (lane < C::kTeam) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(box);
      va = cluster_load(p, lane) | (uint64_t)cluster_load(p + 1, lane) << 32;
      vb = cluster_load(p + 2, lane) | (uint64_t)cluster_load(p + 3, lane) << 32;
    }
    turn ^= 1;
  }
  // The groups' sums over the team, and this block's and those before it.
  __device__ __forceinline__ uint64_t total(uint64_t& mine, uint64_t& before) { return total(work.group, mine, before); }
  __device__ __forceinline__ uint64_t total(const uint64_t* group, uint64_t& mine, uint64_t& before) {
    uint64_t v = 0, all, none;
    for (int g = threadIdx.x; g < groups + 2; g += C::kThreads) v += group[g];
    scan(v, mine);
    share(mine, 0, all, none);
    before = warp_sum64((int)(threadIdx.x & 31) < rank ? all : 0);
    return warp_sum64(all);
  }
  // The first id up to which the sum of f is above target, with the groups' sums
  // given: true for the block that has it, sh.id (within the row) and sh.x.
  template <typename F>
  __device__ __forceinline__ bool find(uint64_t target, uint64_t mine, uint64_t before, F f) {
    return find(work.group, target, mine, before, f);
  }
  template <typename F>
  __device__ __forceinline__ bool find(const uint64_t* group, uint64_t target, uint64_t mine, uint64_t before, F f) {
    if (target < before || target >= before + mine) return false;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = groups + 2;
    const int each = (n + C::kThreads - 1) / C::kThreads, g0 = (int)threadIdx.x * each;
    const uint64_t left = target - before;
    uint64_t sum = 0, all;
    for (int g = g0; g < min(g0 + each, n); ++g) sum += group[g];
    uint64_t b = scan(sum, all);
    if (b <= left && left < b + sum) {
      int g = g0;
      while (b + group[g] <= left) b += group[g++];
      sh.at = g, sh.left = b;
    }
    __syncthreads();
    if (warp == 0) {
      constexpr int N = Row<E>::kVec;
      const int g = sh.at, i = (g - 1) * 32 + lane;
      float x[N];
      int id = id0, k = 0;  // this lane's first id, and how many
      if (g == 0 || g == groups + 1) {
        id += (g ? r.tail_start() : 0) + lane;
        k = lane < (g ? r.tail : r.head) ? 1 : 0;
        if (k) x[0] = to_f32(r.p[id - id0]);
      } else if (i < r.nvec) {
        id += r.head + i * N;
        k = N;
        unpack(r.vec()[i], x);
      }
      uint64_t w = 0;
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < k) w += f(x[e], id + e);
      uint64_t incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t m = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += m;
      }
      uint64_t at = sh.left + incl - w;
      if (at <= left && left < at + w) {
        bool done = false;
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e < k && !done) {
            at += f(x[e], id + e);
            if (at > left) done = true, sh.id = id + e, sh.x = x[e];
          }
      }
    }
    __syncthreads();
    return true;
  }
  // The blocks' lists together in the first block's; counts: each block's, by lane.
  __device__ __forceinline__ void gather(uint64_t counts) {
    int at = (int)__shfl_sync(0xFFFFFFFFu, counts, 0);
    for (int q = 1; q < size; ++q) {
      const int n = (int)__shfl_sync(0xFFFFFFFFu, counts, q);
      for (int j = threadIdx.x; j < n; j += C::kThreads) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(&work.list[j]);
        work.list[at + j] = cluster_load(p, q) | (uint64_t)cluster_load(p + 1, q) << 32;
      }
      at += n;
    }
    __syncthreads();
  }
  // In the first block: the first of the n listed keys, in their order, with
  // which `base` and the weights reach target: work.key and the sum, work.incl; 0
  // if none does, or base alone.
  __device__ __forceinline__ void reach(int n, uint64_t base, uint64_t target) {
    const Exact exact = exact_weights();
    sort_list<C::kThreads>(work.list, n);
    for (int j = threadIdx.x; j < n; j += C::kThreads) work.weight[j] = exact(rank_logit(work.list[j]));
    if (threadIdx.x == 0) work.key = work.incl = 0;
    __syncthreads();
    sum_list<C::kList, C::kThreads>(work.weight, n, sh, scan_turn);
    for (int j = threadIdx.x; j < n; j += C::kThreads) {
      const uint64_t before = base + (j ? work.weight[j - 1] : 0), upto = base + work.weight[j];
      if (before < target && target <= upto) work.key = work.list[j], work.incl = upto;
    }
    __syncthreads();
  }
  __device__ __forceinline__ void list(float x, int id) {
    const uint32_t at = atomicAdd(&sh.listed, 1u);
    if (at < (uint32_t)C::kList) work.list[at] = rank_key(x, (uint32_t)id);
  }
  __device__ __forceinline__ void clear(bool both) {
    for (int b = threadIdx.x; b < C::kBins; b += C::kThreads) {
      work.lo[b] = 0;
      if (both) work.hi[b] = 0;
    }
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
  }
  // The bins' sums over the team, each block a slice of them; what comes before a
  // thread's bins, and the sum of all.  Barriers of the team.
  __device__ __forceinline__ uint64_t slice(bool both, uint64_t& sum) {
    sync();
    const int each = C::kBins / size / C::kThreads, b0 = (rank * C::kThreads + (int)threadIdx.x) * each;
    uint64_t n = 0, mine, all, none;
    for (int i = 0; i < each; ++i) n += bin(b0 + i, both);
    uint64_t before = scan(n, mine);
    share(mine, 0, all, none);
    before += warp_sum64((int)(threadIdx.x & 31) < rank ? all : 0);
    sum = warp_sum64(all);
    return before;
  }
  __device__ __forceinline__ uint64_t bin(int b, bool both) const {
    if (C::kTeam == 1 || size == 1) return work.lo[b] + (both ? (uint64_t)work.hi[b] << 32 : 0);
    uint64_t n = 0;
#pragma unroll
    for (int q = 0; q < C::kTeam; ++q) {
      n += cluster_load(&work.lo[b], q);
      if (both) n += (uint64_t)cluster_load(&work.hi[b], q) << 32;
    }
    return n;
  }
  // The bin in which the sum over the bins, `before` in front of this thread's,
  // reaches target (1 .. the sum): true for its thread.
  __device__ __forceinline__ bool bin_at(uint64_t target, uint64_t before, bool both, int& b, uint64_t& at) const {
    const int each = C::kBins / size / C::kThreads, b0 = (rank * C::kThreads + (int)threadIdx.x) * each;
    at = before;
    if (target <= at) return false;
    for (b = b0; b < b0 + each; ++b) {
      const uint64_t n = bin(b, both);
      if (target <= at + n) return true;
      at += n;
    }
    return false;
  }

  // The last element of the shortest leading part, in the order of the keys and
  // of the keys >= least, that holds `target` elements (COUNT) or weight: its key,
  // and the weight up to and with it.  False if all together do not.
  template <bool COUNT>
  __device__ __noinline__ bool select(uint64_t target, uint64_t least, uint64_t& key_out, uint64_t& incl_out) {
    const uint32_t top = rank_value(weight.m);
    const Exact exact = exact_weights();
    uint32_t *lo = work.lo, *hi = work.hi;
    uint32_t d0 = 0, d1 = 0xFFFFFFFFu;
    uint64_t base = 0, all, none;  // elements or weight before these distances
    for (int level = 0;; ++level) {
      int shift = 0;
      while (((d1 - d0) >> shift) >= (uint32_t)C::kBins) ++shift;
      clear(true);
      each([&](float x, int id) {
        const uint64_t key = rank_key(x, (uint32_t)id);
        const uint32_t d = top - (uint32_t)(key >> 32);
        if (x == neg_inf() || key < least || d < d0 || d > d1) return;
        const int b = level == 0 ? first_bin<C>(top, top - d) : (int)((d - d0) >> shift);
        if (COUNT) {
          atomicAdd(&lo[b], 1u);
        } else {
          const uint64_t w = exact(x);
          if (w) add64(&lo[b], &hi[b], w);
        }
      });
      uint64_t sum, at;
      const uint64_t n0 = slice(true, sum) + base;
      if (threadIdx.x == 0) sh.found = 0;
      __syncthreads();
      int its;
      if (bin_at(target, n0, true, its, at)) sh.found = 1 + its, work.base = at;
      __syncthreads();
      share(sh.found, sh.found ? work.base : 0, all, none);
      const int bin = (int)warp_sum64(all) - 1;
      if (bin < 0) return false;
      base = warp_sum64(none);
      if (level == 0) {
        d0 = first_bin_start<C>(top, bin);
        d1 = bin + 1 < C::kBins ? first_bin_start<C>(top, bin + 1) - 1 : 0xFFFFFFFFu;
      } else {
        const uint32_t start = d0 + ((uint32_t)bin << shift), rest = d1 - start, width = (1u << shift) - 1;
        d0 = start;
        d1 = start + min(rest, width);
      }
      each([&](float x, int id) {
        const uint64_t key = rank_key(x, (uint32_t)id);
        const uint32_t d = top - (uint32_t)(key >> 32);
        if (x != neg_inf() && key >= least && d >= d0 && d <= d1) list(x, id);
      });
      __syncthreads();
      share(sh.listed, 0, all, none);
      const uint64_t in = warp_sum64(all);
      if (in <= (uint64_t)C::kList) {  // the first block decides
        uint64_t key = 0, incl = 0;
        if (rank == 0) {
          gather(all);
          if (COUNT) {
            sort_list<C::kThreads>(work.list, (int)in);
            key = work.list[target - base - 1];
          } else {
            reach((int)in, base, target);
            key = work.key, incl = work.incl;
          }
        }
        share(key, incl, all, none);
        key_out = warp_sum64(all), incl_out = warp_sum64(none);
        return true;
      }
      if (d0 == d1) {  // ties: the first of them in the order of the ids
        const uint32_t value = top - d0;
        const uint64_t w1 = COUNT ? 1 : exact(rank_logit((uint64_t)value << 32)), take = (target - base + w1 - 1) / w1;
        auto tie = [&](float x, int id) {
          return (uint64_t)(x != neg_inf() && rank_value(x) == value && rank_key(x, (uint32_t)id) >= least);
        };
        sums(tie);
        uint64_t mine, before;
        total(mine, before);
        const uint64_t key = find(take - 1, mine, before, tie) ? rank_key(sh.x, (uint32_t)sh.id) : 0;
        share(key, 0, all, none);
        key_out = warp_sum64(all), incl_out = base + take * w1;
        return true;
      }
    }
  }

  // The draw with top_p alone: a histogram of rounded weights says near which
  // values the kept part ends; one pass then sums the weights above them and all
  // weights, and lists the elements in between.  False, without a result, where
  // these are too many or the end is not among them.  log_s: of the row's weight.
  __device__ __forceinline__ bool draw_top_p(const Filters& fl, int V, int log_s, Drawn& out, bool& owner) {
    const float scale = ldexpf(1.0f, 31 - log_s), m = weight.m, ch = weight.ch;
    const Exact exact = exact_weights();
    uint32_t* lo = work.lo;
    // Bins of the FP32 exponent, which never rises where the logit falls: equal
    // logits share a bin, and a bin's logits are above the next one's.
    auto bin_of = [](float t) {
      return min((uint32_t)(__float_as_int(fmaf(t, -(C::kBins - 1) / 42.0f, 12582912.0f)) - 0x4B400000), (uint32_t)C::kBins - 1);
    };
    clear(false);
    each([&](float x, int) {
      const float t = __fmul_rn(x - m, ch);
      const uint32_t v = __float2uint_rn(t >= kMinExponent ? exp2_fast(t) * scale : 0.0f);
      if (v) atomicAdd(&lo[bin_of(t)], v);
    });
    uint64_t sum, all, none, ignored;
    const uint64_t n0 = slice(false, sum);
    // off by half a unit per element, and the error of FP32 weights
    const uint64_t mid = part_of<false>(sum, fmaxf(fl.top_p, 0.0f)), slack = (uint64_t)V / 2 + (sum >> 17) + 1;
    const uint64_t low = mid > slack ? mid - slack : 1, high = min((unsigned long long)(mid + slack), (unsigned long long)sum);
    if (threadIdx.x == 0) work.key = work.incl = 0;
    __syncthreads();
    int its;
    if (bin_at(low, n0, false, its, ignored)) work.key = 1 + its;
    if (bin_at(high, n0, false, its, ignored)) work.incl = 1 + its;
    __syncthreads();
    share(work.key, work.incl, all, none);
    const int b0 = (int)warp_sum64(all) - 1, b1 = (int)warp_sum64(none) - 1;
    if (b0 < 0 || b1 < b0) return false;
    uint64_t S = 0;
    uint32_t near = 0;  // a bit per element that is to be listed, the last one lowest
    sums([&](float x, int) {
      const uint32_t b = bin_of(__fmul_rn(x - m, ch));
      const uint64_t w = exact(x);
      S += w;
      near = near << 1 | (b - (uint32_t)b0 <= (uint32_t)(b1 - b0) ? 1u : 0u);
      return b < (uint32_t)b0 ? w : 0;
    }, [&](const auto& x, int n, int id) {
      if (near) {
        constexpr int N = Row<E>::kVec;
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (k < n && near >> (n - 1 - k) & 1) list(x[k], id + k);
        near = 0;
      }
    });
    const int listed = (int)sh.listed;
    uint64_t part;
    scan(S, part);
    share(part, (uint64_t)listed, all, none);
    S = warp_sum64(all);
    if (warp_sum64(none) > (uint64_t)C::kList) return false;
    uint64_t mine, before;
    const uint64_t base = total(mine, before);
    const uint64_t target = max(1ull, (unsigned long long)part_of<true>(S, fmaxf(fl.top_p, 0.0f)));
    uint64_t key = 0, kept = 0;
    // the own list, before the first block mixes it with the others'
    constexpr int PER = C::kList / C::kThreads;
    uint64_t own[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) own[i] = (int)threadIdx.x + i * C::kThreads < listed ? work.list[threadIdx.x + i * C::kThreads] : 0;
    if (rank == 0) {
      __syncthreads();
      gather(none);
      reach((int)warp_sum64(none), base, target);
      key = work.key, kept = work.incl;
    }
    share(key, kept, all, none);
    key = warp_sum64(all), kept = warp_sum64(none);
    if (key == 0) return false;
    // the kept ones of the list join their groups
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (own[i] >= key) {
        const int at = rank_id(own[i]) - id0, v = at - r.head;
        const int g = at < r.head ? 0 : at >= r.tail_start() ? groups + 1 : 1 + v / (32 * Row<E>::kVec);
        uint32_t* p = reinterpret_cast<uint32_t*>(&work.group[g]);
        add64(p, p + 1, exact(rank_logit(own[i])));
      }
    __syncthreads();
    out.total = S;
    out.kept = total(mine, before);
    owner = find(part_of<false>(out.kept, fl.u), mine, before, [&](float x, int id) {
      return x != neg_inf() && rank_key(x, (uint32_t)id) >= key ? exact(x) : 0;
    });
    return true;
  }

  // ---- BF16: a bin per value ----
  // One histogram of whole numbers then gives every filter's end with exact
  // weights, and a table of 4096 weights replaces their evaluation per element
  // (2048 open rows of 131072 with top-p 1012 us, 1222 without this; 512 without
  // filters 120 and 155).
  // The 16 bits in the order of the values, by distance below the maximum's: 2048
  // values (sixteen powers of two), one bin for all down to -2^-10, 2046 values (16
  // powers of two) below that, and a bin for the rest.
  static constexpr int kMid = C::kNear, kLast = C::kBins - 1;
  struct Bins {
    uint32_t top;      // rank of the maximum, in both halves
    int below;         // distance of a value below -2^-10, less its bin; 0 under a
                       // negative maximum, where the bins go on to kLast
    uint32_t low, off; // below + kMid and below, in both halves
    __device__ __forceinline__ static uint32_t rank(uint32_t pair) {
      uint32_t sign;
      asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(sign) : "r"(pair));  // each half its sign bit
      return pair ^ (sign | 0x80008000u);
    }
    __device__ __forceinline__ Bins(float m) {
      const uint32_t t = rank_value(m) >> 16;  // of 0, not -0
      top = t << 16 | t;
      below = max(0, (int)t - 0x457F - kMid);  // -2^-10 has rank 0x457F and lies in bin kMid
      low = (uint32_t)(below + kMid) * 0x10001u, off = (uint32_t)below * 0x10001u;
    }
    // Of a pair of values: the bins of the first part up to kMid, and of the second
    // from kMid on.
    __device__ __forceinline__ uint32_t pair(uint32_t values) const {
      const uint32_t d = top - rank(values);  // no half borrows: the maximum is at the top
      return __vminu2(d, kMid * 0x10001u) + __vminu2(__vmaxu2(d, low) - off, kLast * 0x10001u) - kMid * 0x10001u;
    }
    __device__ __forceinline__ int of(float x) const {
      const uint32_t v = __float_as_uint(x) >> 16;
      const uint32_t t = top & 0xFFFFu, r = rank(v) & 0xFFFFu;
      return t < r ? 0 : (int)(pair(v | v << 16) & 0xFFFFu);  // -0 under 0 is above it in rank
    }
    // The value of a bin that has one.
    __device__ __forceinline__ float value(int b) const {
      const int r = (int)(top & 0xFFFFu) - (b < kMid ? b : b + below);
      if (r <= 0x7F) return neg_inf();  // none
      const uint32_t bits = r & 0x8000 ? (uint32_t)r ^ 0x8000u : ~(uint32_t)r & 0xFFFFu;
      return __uint_as_float(bits << 16);
    }
  };
  // f(bin) on this thread's elements, end(group) as in each; and several(x, bin) on
  // the elements of the bins of several values, which are few: a vector is looked
  // through only where it has one.
  template <typename F, typename S, typename G>
  __device__ __forceinline__ void each_bin(const Bins& bins, F f, S several, G end) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Row<E> r = this->r;
    const int groups = this->groups;
    auto one = [&](uint32_t bits) {
      const float x = __uint_as_float(bits << 16);
      const int b = bins.of(x);
      f(b);
      if (b == kMid || b == kLast) several(x, b);
    };
    for (int g0 = warp; g0 < groups; g0 += kTeamU * C::kWarps) {
      uint4 v[kTeamU];
#pragma unroll
      for (int u = 0; u < kTeamU; ++u) v[u] = r.vec()[min((g0 + u * C::kWarps) * 32 + lane, r.nvec - 1)];
#pragma unroll
      for (int u = 0; u < kTeamU; ++u) {
        const int g = g0 + u * C::kWarps;
        if (g >= groups) break;
        if (g * 32 + lane < r.nvec) {
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          bool any = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t pair = bins.pair(w[k]);
            const int a = (int)(pair & 0xFFFFu), b = (int)(pair >> 16);
            f(a);
            f(b);
            any |= a == kMid || a == kLast || b == kMid || b == kLast;
          }
          if (any) {
            uint64_t lo = w[0] | (uint64_t)w[1] << 32, hi = w[2] | (uint64_t)w[3] << 32;
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              const float x = __uint_as_float((uint32_t)lo << 16);
              const int b = bins.of(x);
              if (b == kMid || b == kLast) several(x, b);
              lo = lo >> 16 | hi << 48, hi >>= 16;
            }
          }
        }
        end(g + 1);
      }
    }
    if (warp == 0) {
      if (lane < r.head) one(r.p[lane]);
      end(0);
      if (lane < r.tail) one(r.p[r.tail_start() + lane]);
      end(groups + 1);
    }
  }
  // The bin in which the sum over the bins of n(b) reaches target, with what comes
  // before it: shared with the team.  `before`: in front of this thread's bins.
  template <typename N>
  __device__ __forceinline__ int reach_bin(uint64_t target, uint64_t before, N n, uint64_t& at) {
    const int each = C::kBins / size / C::kThreads, b0 = (rank * C::kThreads + (int)threadIdx.x) * each;
    if (threadIdx.x == 0) work.key = work.incl = 0;
    __syncthreads();
    for (int b = b0; b < b0 + each && before < target; ++b) {
      const uint64_t v = n(b);
      if (target <= before + v) work.key = 1 + b, work.incl = before;
      before += v;
    }
    __syncthreads();
    uint64_t all, none;
    share(work.key, work.incl, all, none);
    at = warp_sum64(none);
    return (int)warp_sum64(all) - 1;
  }

  // All filters from one histogram of the values, whose weights are exact.  False,
  // without a result, where what is kept ends in a bin of several values.
  __device__ __noinline__ bool draw_bf16(const Filters& fl, int V, Drawn& out, bool& owner) {
    const bool filtered = fl.top_k > 0 || fl.top_p < 1.0f || fl.min_p > 0.0f;
    const Exact exact = exact_weights();
    const Bins bins(weight.m);
    // 0 and -0, which are equal, and -inf lie in bins of several values but below
    // a maximum of less than 2^-95 or of the lowest values
    const uint32_t first_rank = bins.top & 0xFFFFu;
    if (first_rank - 0x8000u < (uint32_t)C::kBins || first_rank < 0x80u + C::kBins) return false;
    uint64_t* table = work.table;
    for (int b = threadIdx.x; b < C::kBins; b += C::kThreads)
      table[b] = b == kMid || b == kLast ? 0 : exact(bins.value(b));
    int last = C::kBins;       // kept are the elements of the bins before `last`
    uint64_t take = 0, all, none;  // and the first `take` of it
    if (filtered) {
      uint32_t* lo = work.lo;
      uint64_t mid = 0, rest = 0;  // weights of the bins of several values
      clear(false);
      uint32_t masked = 0;
      each_bin(bins, [&](int b) { atomicAdd(&lo[b], 1u); }, [&](float x, int b) {
        const uint64_t w = exact(x);
        (b == kMid ? mid : rest) += w;
        masked += x == neg_inf();
      }, [](int) {});
      __syncthreads();
      if (masked) atomicSub(&lo[kLast], masked);
      uint64_t a, b;
      scan(mid, a);
      scan(rest, b);
      share(a, b, all, none);
      mid = warp_sum64(all), rest = warp_sum64(none);
      const int each = C::kBins / size / C::kThreads, b0 = (rank * C::kThreads + (int)threadIdx.x) * each;
      auto number = [&](int at) { return bin(at, false); };
      auto mass = [&](int at) { return at == kMid ? mid : at == kLast ? rest : table[at] * bin(at, false); };
      uint64_t n = 0, w = 0, mine_n, mine_w;
      for (int at = b0; at < b0 + each; ++at) n += number(at), w += mass(at);
      uint64_t n0 = scan(n, mine_n), w0 = scan(w, mine_w);
      share(mine_n, mine_w, all, none);
      const int lane = threadIdx.x & 31;
      n0 += warp_sum64(lane < rank ? all : 0), w0 += warp_sum64(lane < rank ? none : 0);
      uint64_t kept = out.total = warp_sum64(none), at;
      if (fl.top_k > 0) {
        const int found = reach_bin((uint64_t)fl.top_k, n0, number, at);
        if (found == kMid || found == kLast) return false;
        if (found >= 0) {
          last = found, take = (uint64_t)fl.top_k - at;
          if (fl.top_p < 1.0f) {  // the weight up to there
            if (threadIdx.x == 0) work.incl = 0;
            __syncthreads();
            if (found >= b0 && found < b0 + each) {
              uint64_t before = w0;
              for (int k = b0; k < found; ++k) before += mass(k);
              work.incl = before;
            }
            __syncthreads();
            share(work.incl, 0, all, none);
            kept = warp_sum64(all) + take * table[found];
          }
        }
      }
      if (fl.top_p < 1.0f) {
        const uint64_t target = max(1ull, (unsigned long long)part_of<true>(kept, fmaxf(fl.top_p, 0.0f)));
        const int found = reach_bin(target, w0, mass, at);
        if (found == kMid || found == kLast || found < 0) return false;
        last = found, take = (target - at + table[found] - 1) / table[found];
      }
      if (fl.min_p > 0.0f) {  // the first bin below the edge
        if (threadIdx.x == 0) min_p_edge(fl, sh.edge), work.edge = C::kBins;
        __syncthreads();
        const uint32_t edge = (uint32_t)(min_p_key(weight.m, sh.edge) >> 32);
        for (int k = threadIdx.x; k < C::kBins; k += C::kThreads)
          if (k != kMid && k != kLast && rank_value(bins.value(k)) < edge) {
            atomicMin(&work.edge, k);
            break;
          }
        __syncthreads();
        const int first = work.edge;
        // among the values of the one bin, or those of the other where they count
        if (first == C::kBins && last == C::kBins && rest) return false;
        if (first < last || (first == last && take > 0)) {
          if (first == kMid + 1) return false;
          last = first, take = 0;
        }
        __syncthreads();
      }
    }
    // weights before `last`, and elements of it
    uint64_t v = 0;
    uint32_t ties = 0;
    __syncthreads();
    each_bin(bins, [&](int b) {
      v += b < last ? table[b] : 0;
      ties += b == last ? 1 : 0;
    }, [&](float x, int b) { v += b < last ? exact(x) : 0; }, [&](int g) {
      v = warp_sum64(v);
      ties = __reduce_add_sync(0xFFFFFFFFu, ties);
      if ((threadIdx.x & 31) == 0) work.group[g] = v, work.ties[g] = ties;
      v = 0, ties = 0;
    });
    __syncthreads();
    uint64_t mine, before, key = 0;
    if (take > 0) {
      total(work.ties, mine, before);
      const int n = groups + 2, each = (n + C::kThreads - 1) / C::kThreads, g0 = (int)threadIdx.x * each;
      uint64_t sum = 0, part;
      for (int g = g0; g < min(g0 + each, n); ++g) sum += work.ties[g];
      uint64_t at = scan(sum, part) + before;
      for (int g = g0; g < min(g0 + each, n) && at < take; at += work.ties[g++])
        work.group[g] += table[last] * min((unsigned long long)work.ties[g], (unsigned long long)(take - at));
      __syncthreads();
      if (find(work.ties, take - 1, mine, before, [&](float x, int) { return (uint64_t)(bins.of(x) == last); }))
        key = rank_key(sh.x, (uint32_t)sh.id);
      share(key, 0, all, none);
      key = warp_sum64(all);
    }
    out.kept = total(mine, before);
    if (!filtered) out.total = out.kept;
    owner = find(min((unsigned long long)part_of<false>(out.kept, fl.u), (unsigned long long)out.kept - 1), mine, before,
                 [&](float x, int id) -> uint64_t {
                   const int b = bins.of(x);
                   if (b == kMid || b == kLast) return b < last ? exact(x) : 0;
                   return b < last || (b == last && take > 0 && rank_key(x, (uint32_t)id) >= key) ? table[b] : 0;
                 });
    return true;
  }

  __device__ __forceinline__ bool draw(const Filters& fl, int V, int log_s, Drawn& out) {
    const bool filtered = fl.top_k > 0 || fl.top_p < 1.0f || fl.min_p > 0.0f;
    const Exact exact = exact_weights();
    bool owner;
    if constexpr (sizeof(E) == 2 && C::kValues) {
      if (draw_bf16(fl, V, out, owner)) return owner;
    }
    if (fl.top_k == 0 && fl.top_p < 1.0f && !(fl.min_p > 0.0f) && draw_top_p(fl, V, log_s, out, owner)) return owner;
    uint64_t least = 0, key, incl, mine, before, S = 0;
    if (fl.top_k > 0 && select<true>((uint64_t)fl.top_k, 0, key, incl)) least = key;
    if (fl.top_p < 1.0f) {
      sums([&](float x, int id) { return rank_key(x, (uint32_t)id) >= least ? exact(x) : 0; });
      const uint64_t mass = total(mine, before);
      const uint64_t target = max(1ull, (unsigned long long)part_of<true>(mass, fmaxf(fl.top_p, 0.0f)));
      if (select<false>(target, least, key, incl)) least = max(least, key);
    }
    if (fl.min_p > 0.0f) {
      if (threadIdx.x == 0) min_p_edge(fl, sh.edge);
      __syncthreads();
      least = max(least, min_p_key(weight.m, sh.edge));
    }
    auto kept = [&](float x, int id) { return x != neg_inf() && rank_key(x, (uint32_t)id) >= least ? exact(x) : 0; };
    sums([&](float x, int id) {
      const uint64_t w = exact(x);
      S += w;
      return x != neg_inf() && rank_key(x, (uint32_t)id) >= least ? w : 0;
    });
    out.kept = out.total = total(mine, before);
    if (filtered) {
      uint64_t part, all, none;
      scan(S, part);
      share(part, 0, all, none);
      out.total = warp_sum64(all);
    }
    const uint64_t target = part_of<false>(out.kept, fl.u);
    return find(min((unsigned long long)target, (unsigned long long)out.kept - 1), mine, before, kept);
  }
};

// Without branches, so that the weights of a vector are formed side by side: an
// exponent out of range is held at -44, where only its own bits are used, and the
// result dropped.
template <typename E, typename C>
__device__ __forceinline__ uint64_t Team<E, C>::Exact::operator()(float x) const {
  const float d = x - m;
  const float p0 = __fmul_rn(d, ch), p = fmaxf(p0, -44.0f);
  const float b = d - x, lost = (x - (d - b)) + (-m - b);
  const float e = fmaf(lost, ch, fmaf(d, cl, fmaf(d, ch, -p0)));
  const float z = p + 12288.0f;  // 1.5 2^13: steps of 1/1024
  const int i = __float_as_int(z) - __float_as_int(12288.0f);
  const float q = (p - (z - 12288.0f)) + e;
  const int n = __float2int_rn(q * fmaf(q, fmaf(q, 0x1p40f * 0.0555041087f, 0x1p40f * 0.240226507f), 0x1p40f * 0.69314718f));
  const uint64_t t = power[i & 1023];
  const uint64_t w = (t + (uint64_t)(((int64_t)n * (int64_t)(t >> 32)) >> 8)) >> (62 - s - (i >> 10));
  return (p0 - kMinExponent) + e >= 0.0f ? w : 0;
}

// The powers of 2^(1/1024) for exact weights.
template <typename C>
__device__ __forceinline__ void load_powers(SampleShared<C::kThreads>& sh, TeamWork<C>& work) {
  load_exp2(sh);
  __syncthreads();
  Weights one;  // 2^(j / 1024 - 1), of unit 2^-61
  one.m = 1024.0f, one.ch = 0x1p-10f, one.cl = 0.0f, one.s = 61, one.exp2 = sh.exp2;
  for (int j = threadIdx.x; j < 1024; j += C::kThreads) work.power[j] = one.exact((float)j) << 2;
  __syncthreads();
}

// An open row's token by its team of `size` blocks.
template <typename E, typename C>
__device__ __forceinline__ void open_row(const SampleArgs& a, int64_t t, int flag, int rank, int size, int& turn,
                                         int& scan_turn, SampleShared<C::kThreads>& sh, TeamWork<C>& work) {
  [[maybe_unused]] const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lg = size == 1 ? 0 : C::kTeamLog;
  const int log_s = (kOpen - flag) & 63;
  const E* logits = static_cast<const E*>(a.logits) + t * a.ld;
  const Row<E> whole(logits, a.V);
  const int v0 = whole.part(rank, lg), v1 = whole.part(rank + 1, lg);
  const int id0 = rank == 0 ? 0 : whole.head + v0 * Row<E>::kVec;
  const int id1 = rank == size - 1 ? a.V : whole.head + v1 * Row<E>::kVec;
  const Row<E> r(logits + id0, id1 - id0);
  Team<E, C> team = {r, id0, rank, size, turn, scan_turn, (r.nvec + 31) / 32, Weights(), sh, work};
  bool params;
  const Filters fl = filters_of(a, t, params);
  // the row's maximum, a number
  uint32_t top;
  if constexpr (sizeof(E) == 2) {
    top = rank_value(__uint_as_float((uint32_t)((kOpen - flag) >> 6) << 16));
  } else {
    const float high = team.high();
    top = __reduce_max_sync(0xFFFFFFFFu, rank_value(high));
    if (lane == 0) sh.scan[0][warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xFFFFFFFFu, lane < C::kWarps ? (uint32_t)sh.scan[0][lane] : 0u);
    __syncthreads();
    uint64_t all, none;
    team.share(top, 0, all, none);
    top = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)all);
  }
  team.weight = weights_of(fl.inv_t, rank_logit((uint64_t)top << 32), a.V, sh.exp2);
  team.weight.s = min(52, 62 - log_s);  // as fine as the row's own sum allows
  Drawn out;
  if (team.draw(fl, a.V, log_s, out) && threadIdx.x == 0) {
    out.id = sh.id, out.x = sh.x;
    put_drawn(a, t, out, fl.inv_t, team.weight.m, team.weight.s);
  }
  __syncthreads();
  scan_turn = team.scan_turn;
  turn = team.turn;
}

// Few rows: a cluster of eight blocks per row, each of which reads one of the runs
// that a block's threads have; the first block ends the row, and if it stays open
// all eight decide it at once.
template <typename E, int BLOCKS>
__global__ void __launch_bounds__(LongTeam::kThreads, BLOCKS) sample_few_kernel(SampleArgs a) {
  using C = LongTeam;
  constexpr int TH = C::kThreads;
  static_assert(C::kTeam == kSaRuns, "a run per block");
  extern __shared__ uint4 smem[];
  FewWork& few = *reinterpret_cast<FewWork*>(smem);
  TeamWork<C>& work = few.team;
  SampleShared<C::kThreads>& sh = few.sh;
  const int rank = (int)blockIdx.x % C::kTeam;
  const int64_t t = blockIdx.x / C::kTeam;
  float *highs = few.highs + threadIdx.x, *sums = few.sums + threadIdx.x;
  int turn = 0, team_turn = 0;
  load_exp2(sh);
  cluster_arrive();  // all blocks run: their shared memory may be written
  cluster_wait();
  begin_kernel();
  const SampleRow<E, TH> row(static_cast<const E*>(a.logits) + t * a.ld, a.V, highs);
  bool params;
  const Filters fl = filters_of(a, t, params);
  const Weights weight = weights_of(fl.inv_t, 0.0f, a.V, sh.exp2);
  if (rank < row.runs) {
    RunSum acc;
    for (int j = 0; j < row.per; j += kSaU) {
      const int i0 = (rank * row.per + j) * TH + (int)threadIdx.x;
      uint4 v[kSaU];
#pragma unroll
      for (int u = 0; u < kSaU; ++u) {
        v[u] = Stream<TH, 1, 1, 1, E, int>::none(E());
        if (i0 + u * TH < row.r.nvec) v[u] = row.r.vec()[i0 + u * TH];
      }
      acc.add(v, weight.ch, E());
    }
    cluster_store(&highs[rank * TH], 0, __float_as_uint(acc.m));
    cluster_store(&sums[rank * TH], 0, __float_as_uint(acc.s));
  }
  if (rank == 0 && fl.min_p > 0.0f && threadIdx.x == TH - 1) min_p_edge(fl, sh.edge);
  cluster_arrive();
  cluster_wait();
  if (rank == 0) {
    float m = neg_inf();
    for (int q = 0; q < row.runs; ++q) m = max_nan(m, highs[q * TH]);
    row.front([&](float x, int) { m = max_nan(m, x); });
    row.back([&](float x, int) { m = max_nan(m, x); });
    const int open = end_row<E, TH>(a, t, row, fl, params, weight, m, highs, sums, sh, few.work, turn);
    if (threadIdx.x < C::kTeam) cluster_store(&few.open, threadIdx.x, (uint32_t)open);
  }
  cluster_arrive();
  cluster_wait();
  if (few.open) {
    load_powers(sh, work);
    open_row<E, C>(a, t, (int)few.open, rank, C::kTeam, team_turn, turn, sh, work);
  }
  cluster_arrive();  // no block ends while another reads its shared memory
  cluster_wait();
}

__device__ __forceinline__ bool is_open(int token) { return token <= kOpen && token > kClaimed; }

// The next open row from place `seen` to `end` of the rows taken in turn from
// `start` on, or -1; taken by marking its token, so that no other block has it.
template <typename C>
__device__ __noinline__ int64_t claim(const SampleArgs& a, int64_t start, int64_t& seen, int64_t end, int& flag,
                                      TeamWork<C>& work) {
  constexpr int kEach = 4;
  while (seen < end) {
    int token[kEach], mine = kEach;
    auto row = [&](int i) {
      const int64_t t = seen + i * C::kThreads + threadIdx.x + start;
      return t >= a.T ? t - a.T : t;
    };
#pragma unroll
    for (int i = 0; i < kEach; ++i) token[i] = seen + i * C::kThreads + threadIdx.x < end ? __ldcg(&a.tokens[row(i)]) : 0;
#pragma unroll
    for (int i = kEach - 1; i >= 0; --i)
      if (is_open(token[i])) mine = i;
    if (threadIdx.x == 0) work.first = kEach * C::kThreads;
    if (!__syncthreads_or(mine < kEach)) {
      seen += kEach * C::kThreads;
      continue;
    }
    const int place = mine * C::kThreads + (int)threadIdx.x;
    if (mine < kEach) atomicMin(&work.first, place);
    __syncthreads();
    if (place == work.first) {
      const int64_t t = row(mine);
      const int was = mine == 0 ? token[0] : mine == 1 ? token[1] : mine == 2 ? token[2] : token[3];
      work.claimed = atomicCAS(&a.tokens[t], was, kClaimed) == was ? t : -1;
      work.flag = was;
    }
    __syncthreads();
    const int64_t got = work.claimed;
    flag = work.flag;
    __syncthreads();
    if (got >= 0) return got;
  }
  return -1;
}
// How far a block that works alone looks: past its own share of the rows, so that
// it has work where others have much, but not at all rows.
__device__ __forceinline__ int64_t claim_window(int T, int blocks) {
  const int64_t share = ((int64_t)T + blocks - 1) / blocks;
  return min((long long)T, max(4ll * share, 4096ll));
}

// Open rows, taken by marking their tokens.  Few are decided by eight blocks each,
// one after the other within a cluster; their time is the chain of the cluster's
// barriers (a launch for one row with top-p some 45 us, half of the stalls at barriers).
// Many are decided by one block each, two per SM, bound by instructions (52 per
// element: 2048 open rows of 131072 BF16 ids with top-p 972 us).  Among these are
// spills: two blocks of 512 threads leave a thread 64 registers, which the ways to
// decide a row exceed (BF16 560 bytes stored and 832 loaded, FP32 168 and 316; short
// BF16 rows 132 and 248, few BF16 rows by two blocks per SM 68 and 164).  With nothing
// open the launch costs 3 us behind the first.
template <typename E>
__global__ void __launch_bounds__(LongTeam::kThreads, 2) sample_open_kernel(SampleArgs a) {
  using C = LongTeam;
  extern __shared__ uint4 smem[];
  TeamWork<C>& work = *reinterpret_cast<TeamWork<C>*>(smem);
  SampleShared<C::kThreads>& sh = *reinterpret_cast<SampleShared<C::kThreads>*>(&work + 1);
  const int rank_in_cluster = (int)blockIdx.x % C::kTeam;
  const int64_t teams = gridDim.x / C::kTeam, cluster = blockIdx.x / C::kTeam;
  int turn = 0, scan_turn = 0;
  cluster_arrive();  // all blocks run: their shared memory may be written
  cluster_wait();
  begin_kernel();
  // Alone where there are more open rows than two per team, and where a block's
  // groups have room for a row.  The count may be short of rows that others have
  // taken; any mode is right.
  const int64_t start = (int64_t)a.T * (cluster * C::kTeam) / gridDim.x;
  const bool room = a.V / Row<E>::kVec <= C::kGroups * 32;
  int rows = 0;
  if (rank_in_cluster == 0) {
    constexpr int kEach = 8, kBatch = kEach * C::kThreads;
    int token[kEach];
    int64_t from = 0;
    for (; from < a.T && rows <= 2 * teams; from += kBatch) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int64_t t = from + i * C::kThreads + threadIdx.x;
        token[i] = t < a.T ? __ldcg(&a.tokens[t]) : 0;
        n += is_open(token[i]);
      }
      n = __reduce_add_sync(0xFFFFFFFFu, n);
      if ((threadIdx.x & 31) == 0) sh.scan[0][threadIdx.x >> 5] = n;
      __syncthreads();
      for (int w = 0; w < C::kWarps; ++w) rows += (int)sh.scan[0][w];
      __syncthreads();
    }
    // not alone: the first open row of the last tokens read, from `start` on
    if (rows > 0 && !(rows > 2 * teams && room)) {
      uint32_t near = 0xFFFFFFFFu;
      int was = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int64_t t = from - kBatch + i * C::kThreads + threadIdx.x;
        const uint32_t d = (uint32_t)(t >= start ? t - start : t - start + a.T);
        if (is_open(token[i]) && d < near) near = d, was = token[i];
      }
      const uint32_t least = __reduce_min_sync(0xFFFFFFFFu, near);
      if ((threadIdx.x & 31) == 0) sh.scan[0][threadIdx.x >> 5] = least;
      if (threadIdx.x == 0) work.claimed = -1;
      __syncthreads();
      const uint32_t first =
          __reduce_min_sync(0xFFFFFFFFu, (uint32_t)sh.scan[0][(threadIdx.x & 31) % C::kWarps]);
      if (near == first && is_open(was)) {
        int64_t t = start + first;
        if (t >= a.T) t -= a.T;
        if (atomicCAS(&a.tokens[t], was, kClaimed) == was) work.claimed = t, work.flag = was;
      }
      __syncthreads();
      if (threadIdx.x < C::kTeam) {
        cluster_store(&work.first_row[0], threadIdx.x, (uint32_t)work.claimed);
        cluster_store(&work.first_row[1], threadIdx.x, (uint32_t)work.flag);
      }
    }
    if (threadIdx.x < C::kTeam) cluster_store(&work.rows, threadIdx.x, (uint32_t)rows);
  }
  cluster_arrive();
  cluster_wait();
  rows = (int)work.rows;
  if (rows == 0) return;
  load_powers(sh, work);
  // The first block takes a row and tells the others: a barrier per row.  A cluster
  // that counts no more open rows than there are clusters takes one only, where all
  // blocks look through all rows.  None is left over: the cluster that counted first
  // counted all, before any was taken, and goes on until there are none if they were
  // more; if they were not, a cluster that took none has seen all of them taken.
  const bool alone = rows > 2 * teams && room;
  const bool one = rows <= teams && claim_window(a.T, gridDim.x) == a.T;
  int64_t seen = 0, t = (int)work.first_row[0];
  int flag = (int)work.first_row[1];
  auto next = [&]() {  // the cluster's next row
    if (rank_in_cluster == 0) {
      t = claim(a, start, seen, a.T, flag, work);
      if (threadIdx.x < C::kTeam) {
        cluster_store(&work.row[0], threadIdx.x, (uint32_t)t);
        cluster_store(&work.row[1], threadIdx.x, (uint32_t)flag);
      }
    }
    cluster_arrive();
    cluster_wait();
    t = (int)work.row[0], flag = (int)work.row[1];
  };
  if (alone) {  // every block for itself
    const int64_t own = (int64_t)a.T * blockIdx.x / gridDim.x, end = claim_window(a.T, gridDim.x);
    seen = 0;
    while ((t = claim(a, own, seen, end, flag, work)) >= 0)
      open_row<E, C>(a, t, flag, 0, 1, turn, scan_turn, sh, work);
    return;
  }
  for (;;) {
    if (t < 0) next();
    if (t < 0) break;
    open_row<E, C>(a, t, flag, rank_in_cluster, C::kTeam, turn, scan_turn, sh, work);
    if (one) break;
    t = -1;
  }
  cluster_arrive();  // no block ends while another reads its shared memory
  cluster_wait();
}

// The same for short rows, a block each.
template <typename E>
__global__ void __launch_bounds__(ShortTeam::kThreads, 8) sample_open_short_kernel(SampleArgs a) {
  using C = ShortTeam;
  extern __shared__ uint4 smem[];
  TeamWork<C>& work = *reinterpret_cast<TeamWork<C>*>(smem);
  SampleShared<C::kThreads>& sh = *reinterpret_cast<SampleShared<C::kThreads>*>(&work + 1);
  bool ready = false;
  int turn = 0, scan_turn = 0, flag = 0;
  begin_kernel();
  const int64_t start = (int64_t)a.T * blockIdx.x / gridDim.x;
  const int64_t end = claim_window(a.T, gridDim.x);
  int64_t seen = 0;
  for (int64_t t; (t = claim(a, start, seen, end, flag, work)) >= 0;) {
    if (!ready) load_powers(sh, work), ready = true;
    open_row<E, C>(a, t, flag, 0, 1, turn, scan_turn, sh, work);
  }
}

// Clusters of eight blocks of kernel F that run at once on the current device, which
// is less than its blocks would suggest (a cluster lies within a part of the chip: of
// 152 SMs' 19 with one block per SM 15, of 38 with two 36); the answer is kept per
// host thread.
template <auto F>
static int clusters_at_once(int threads, int smem) {
  thread_local int cached_dev = -1, cached = 0;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev == cached_dev) return cached;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(8);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 8;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (!allow_smem((const void*)F, smem, smem) || cudaOccupancyMaxActiveClusters(&n, F, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  cached_dev = dev, cached = n;
  return n;
}

// 1 where the rows are too many.
template <typename E>
static int launch_few(const SampleArgs& a, cudaStream_t s) {
  constexpr int smem = (int)sizeof(FewWork);
  auto f = sample_few_kernel<E, 1>;
  if (a.T > clusters_at_once<sample_few_kernel<E, 1>>(LongTeam::kThreads, smem)) {
    if (a.T >= clusters_at_once<sample_few_kernel<E, 2>>(LongTeam::kThreads, smem)) return 1;
    f = sample_few_kernel<E, 2>;
  }
  if (!allow_smem((const void*)f, smem, smem)) return -1;
  return launch_kernel(f, (unsigned)(a.T * LongTeam::kTeam), LongTeam::kThreads, smem, LongTeam::kTeam, s, a);
}

template <int TH>
static int launch_sample(const SampleArgs& a, cudaStream_t s) {
  const int64_t most = (int64_t)gemm_num_ctas() * kSaBlocks<TH> * 8;
  auto f = a.dtype == MOE_DTYPE_BF16 ? sample_tokens_kernel<uint16_t, TH> : sample_tokens_kernel<float, TH>;
  // Where there is an SM for each row, shared memory for no second block: blocks of
  // a launch that is set up early would otherwise lie two in an SM (152 x 131072 with
  // min-p 19.5 us, 22.8 without).
  constexpr int kAlone = 120 * 1024;
  static_assert(TH != 512 || kSaSmem<TH> <= kAlone, "a block's own share");
  const int smem = TH == 512 && a.T <= gemm_num_ctas() ? kAlone : kSaSmem<TH>;
  if (!allow_smem((const void*)f, smem, TH == 512 ? kAlone : kSaSmem<TH>)) return -1;
  return launch_kernel(f, (unsigned)(a.T < most ? a.T : most), TH, smem, 1, s, a);
}
int launch_sample_tokens(const SampleArgs& a, cudaStream_t s) {
  const bool bf = a.dtype == MOE_DTYPE_BF16;
  const int sms = gemm_num_ctas();
  // A cluster per row where all run at once, one block per SM, or, up to one row
  // less, two, whose registers are half as many, which costs each row 2 us.  With
  // top-p, 131072 ids: 15 rows 11.9 us; 16 rows 14.5 and, in two launches, 18; 32 flat
  // rows 59 and 78; as many rows as clusters, 36, were slower so (21.4 and 18.1).
  static_assert(LongTeam::kTeam == 8, "as clusters_at_once has it");
  const int few = bf ? launch_few<uint16_t>(a, s) : launch_few<float>(a, s);
  if (few <= 0) return few;
  // Threads per row.  What a row's end costs is barriers and dependent loads, so
  // many rows are done by small blocks, whose ends the others cover; 512 threads
  // where all rows have such a block at once (no filter, BF16, one in six rows flat:
  // 512 x 131072 44 us with 256 threads, 51 with 512, 304 x 131072 30 and 27; 12000 x
  // 12000 177 with 128, 238 with 256; 3000 x 32768 96 and 105; 2048 x 131072 117 with
  // 256, 133 with 128).
  const int64_t nvec = (int64_t)a.V * (bf ? 2 : 4) / 16;
  const int rc = nvec <= 1024 || (nvec <= 4096 && a.T > 2 * sms) ? launch_sample<128>(a, s)
                 : a.T <= 2 * sms                                ? launch_sample<512>(a, s)
                                                                 : launch_sample<256>(a, s);
  if (rc != 0) return rc;
  if (a.V <= kShortV) {
    using C = ShortTeam;
    constexpr int smem = (int)(sizeof(TeamWork<C>) + sizeof(SampleShared<C::kThreads>));
    auto f = bf ? sample_open_short_kernel<uint16_t> : sample_open_short_kernel<float>;
    if (!allow_smem((const void*)f, smem, smem)) return -1;
    return launch_kernel(f, (unsigned)(a.T < 8 * sms ? a.T : 8 * sms), C::kThreads, smem, 1, s, a);
  }
  using C = LongTeam;
  constexpr int smem = (int)(sizeof(TeamWork<C>) + sizeof(SampleShared<C::kThreads>));
  auto f = bf ? sample_open_kernel<uint16_t> : sample_open_kernel<float>;
  if (!allow_smem((const void*)f, smem, smem)) return -1;
  // Not all that run at once: the last ones find their places late (nothing open, 152
  // rows, 1 us less with 32 clusters than with 36).
  const int n = bf ? clusters_at_once<sample_open_kernel<uint16_t>>(C::kThreads, smem)
                   : clusters_at_once<sample_open_kernel<float>>(C::kThreads, smem);
  const int teams = n > 1 ? n - n / 8 : 1;
  return launch_kernel(f, (unsigned)((a.T < teams ? a.T : teams) * C::kTeam), C::kThreads, smem, C::kTeam, s, a);
}

}  // namespace moe
