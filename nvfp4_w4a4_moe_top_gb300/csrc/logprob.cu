// Log-probabilities of given tokens with entropy and top alternatives, and
// their gradient.  With z = x inv_t about the row's maximum m and l = ln sum
// e^(z - m):  ln p = z - m - l,  H = l - sum p (z - m),
//   d ln p_y / dz = 1[v = y] - p,  dH / dz = -p (ln p + H).
// Both are bound by HBM: one read of the logits (forward), one read and one
// write (gradient), at some seven operations and one exponential per element.
#include "learner.cuh"

namespace moe {

constexpr int kLpThreads = 256;
constexpr int kLpU = 4;  // vectors per group of copies
constexpr int kLpBlocksPerSm = 3;
// Groups in flight: 64 KB of ring per block, or 48 KB and the 16 KB of maxima
// that the alternatives need.
template <bool TOP>
constexpr int kLpD = TOP ? 3 : 4;
// Maxima kept per thread: with more of them the runs that are read again are
// shorter (20 alternatives, BF16: 10000 x 16384 97 us with 8, 76 with 16; 8000 x
// 24000 114 and 87; 4096 x 131072 191 and 185).
constexpr int kLpSlots = 16;
// Resident grids of rows per launch at most: blocks that end early make room
// for others (one grid of blocks that take all rows in turn waits for the
// slowest SM: 4096 rows of 131072, 178 us against 158).  With no more rows than
// that each group has one row, and the other blocks of its SM cover its end;
// beyond it a group takes several and fetches the next while it ends one.
constexpr int kLpTurns = 8;
template <bool TOP>
constexpr int kLpSmem = kLpThreads * (kLpU * kLpD<TOP> * 16 + (TOP ? kLpSlots * 4 : 0));

__device__ __forceinline__ bool finite_max(float m) { return m <= 3.402823466e+38f; }  // not NaN, not +inf

// Barrier of the TH threads of a row.
template <int TH>
__device__ __forceinline__ void group_sync() {
  if (TH == 32) __syncwarp();
  else if (TH == kLpThreads) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"((int)threadIdx.x / TH + 1), "n"(TH) : "memory");
}

// The alternatives of a part of a row, read by TH threads.  A value that n
// threads' maxima reach is a lower bound of the n-th largest logit.  Each
// thread also keeps the maxima of up to kLpSlots runs of its vectors, so that
// only the runs that reach the bound (little more than n) are read again, from
// L2, by all threads together; a run of nothing but -inf reaches no bound, so
// rows that leave fewer than n ids unmasked are as fast (2 x 131072 BF16 with 5
// ids left, 20 alternatives: 7.3 us; 4096 rows 169 us; through the lists below
// 24 and 764).  The few logits at or above the bound (ties among them) are
// listed, and each finds its place by counting the larger ones: no sorting, and
// no order of atomics in the result.  More runs or candidates than fit (long
// ties) go through sorted lists of 32 per warp instead (list_top).
template <int TH>
struct TopShared {
  static constexpr int NW = TH / 32, kCap = TH < 128 ? 128 : 256, kHot = TH < 64 ? 64 : TH;
  uint64_t cand[kCap];
  uint32_t vals[2][NW];
  int hot[kHot];  // thread * kLpSlots + slot
  int nhot, ncand;
};

// A lower bound, reached by at least n of the threads, of the threads' maxima
// (as rank_value): the n-th largest for one warp; else "k warps reach it with
// j threads each", k j >= n, for the two smallest j that allow it.  Part 1,
// before the group_sync: each warp's (j + 1)-th largest maximum, j = j0, j0 +
// 1.
template <int TH>
__device__ __forceinline__ uint32_t top_bound1(uint32_t mine, int n, TopShared<TH>& sh) {
  if (TH == 32) return __shfl_sync(0xFFFFFFFFu, list_sort(mine), n - 1);
  constexpr int NW = TH / 32;
  const int j0 = (n - 1) / NW, warp = (threadIdx.x & (TH - 1)) >> 5;
  uint32_t v = mine, last = 0;
  for (int j = 0; j <= j0 + 1; ++j) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, v);
    if ((int)(threadIdx.x & 31) == __ffs(__ballot_sync(0xFFFFFFFFu, v == top)) - 1) v = 0;
    if (j == j0) last = top;
    if (j == j0 + 1 && (threadIdx.x & 31) < 2) sh.vals[threadIdx.x & 1][warp] = threadIdx.x & 1 ? top : last;
  }
  return 0;
}
template <int TH>
__device__ __forceinline__ uint32_t top_bound2(uint32_t bound, int n, const TopShared<TH>& sh) {
  if (TH == 32) return bound;
  constexpr int NW = TH / 32;
  const int lane = threadIdx.x & 31, j = (n - 1) / NW + 1 + lane / NW;  // threads per warp, lanes below 2 NW
  const int k = (n + j - 1) / j;                                        // warps needed
  const uint32_t* vals = sh.vals[lane / NW & 1];
  const uint32_t v = vals[lane % NW];
  int reach = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) reach += vals[w] >= v;
  return __reduce_max_sync(0xFFFFFFFFu, lane < 2 * NW && reach >= k ? v : 0u);
}

// The alternatives of a part that has any number of candidates (ties): its
// vectors read again by all warps, each with a list of the 32 largest that it
// fills 32 candidates at a time; keys below the n-th largest so far are dropped
// at once, so that of equal logits only the first are sorted.  The group's list
// goes to sh.cand, zeros after the last.  4096 x 131072 BF16 with 5 ids that
// are not at the lowest value, 20 alternatives: 447 us (one candidate load at a
// time, tested element by element: 803; four loads at a time: 392, but the
// kernel then spills registers and rows without ties take 5% longer).
template <int TH, typename E>
__device__ __noinline__ void list_top(const Row<E>& r, int v0, int v1, bool ends, uint32_t bound, int n,
                                      float* slots, TopShared<TH>& sh) {
  constexpr int N = Row<E>::kVec, NW = TH / 32;
  static_assert(kLpSlots >= 6, "the slots hold 96 keys per warp");
  const int lane = threadIdx.x & 31, warp = (threadIdx.x & (TH - 1)) >> 5;
  uint64_t list = 0, least = (uint64_t)bound << 32;  // keys below `least` cannot enter
  // the warps' slots, no longer needed, take up to 64 pending keys and a list
  auto keys = [&](int w, int i) -> uint64_t& {
    return reinterpret_cast<uint64_t*>(slots + (w - warp) * 32 - lane + (i >> 4) * kLpThreads)[i & 15];
  };
  auto pend = [&](int i) -> uint64_t& { return keys(warp, i); };
  int held = 0;
  auto flush = [&]() {  // sorts up to 32 pending keys into the list
    __syncwarp();
    const uint64_t key = lane < held ? pend(lane) : 0;
    const uint64_t rest = lane + 32 < held ? pend(lane + 32) : 0;
    __syncwarp();
    if (lane + 32 < held) pend(lane) = rest;
    held = held > 32 ? held - 32 : 0;
    list = list_merge(list, list_sort(key));
    least = max(least, __shfl_sync(0xFFFFFFFFu, list, n - 1));
    __syncwarp();
  };
  auto offer = [&](float x, int id, bool valid) {
    const uint64_t key = rank_key(x, (uint32_t)id);
    const bool in = valid && x != neg_inf() && key >= least;
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
    if (who == 0) return;
    if (in) pend(held + __popc(who & ((1u << lane) - 1))) = key;
    held += __popc(who);
    if (held >= 32) flush();
  };
  constexpr int B = 2;
  for (int i0 = v0 + warp * 32; i0 < v1; i0 += TH * B) {
    uint4 v[B];
#pragma unroll
    for (int u = 0; u < B; ++u) v[u] = r.vec()[min(i0 + u * TH + lane, v1 - 1)];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int i = i0 + u * TH + lane;
      float x[N], high = neg_inf();
      unpack(v[u], x);
#pragma unroll
      for (int e = 0; e < N; ++e) high = fmaxf(high, x[e]);
      if (!__any_sync(0xFFFFFFFFu, i < v1 && rank_key(high, (uint32_t)(r.head + i * N)) >= least)) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) offer(x[e], r.head + i * N + e, i < v1);
    }
  }
  if (warp == 0 && ends) {  // the elements outside the vectors
    const bool a = lane < r.head, b = lane < r.tail;
    offer(a ? to_f32(r.p[lane]) : 0.0f, lane, a);
    offer(b ? to_f32(r.p[r.tail_start() + lane]) : 0.0f, r.tail_start() + lane, b);
  }
  if (held) flush();
#pragma unroll
  for (int m = NW / 2; m > 0; m >>= 1) {
    if (warp >= m && warp < 2 * m) keys(warp, 64 + lane) = list;
    group_sync<TH>();
    if (warp < m) list = list_merge(list, keys(warp + m, 64 + lane));
  }
  if (warp == 0) sh.cand[lane] = list;
}

// The candidates of the part into sh.cand; returns their number (keys of 0
// count for nothing).  `mine`: the thread's maximum; slots: those of its runs,
// each of U << shift vectors; bound1: top_bound1's.  Called by all TH threads
// after a group_sync that follows top_bound1 and the last use of sh.ncand.
template <int TH, typename E>
__device__ __forceinline__ int group_top(const Row<E>& r, int v0, int v1, bool ends, float mine, uint32_t bound1,
                                         float* slots, int shift, int n, TopShared<TH>& sh) {
  constexpr int N = Row<E>::kVec;
  const int k = threadIdx.x & (TH - 1);
  const int run = kLpU << shift, used = ((v1 - v0 + TH - 1) / TH + run - 1) / run;  // vectors in a run; runs
  if (TH == 32 && n > 8) {  // the lanes' maxima bound little: with each lane's second run
    float a = kLowest, b = kLowest;
    for (int q = 0; q < used; ++q) {
      const float x = slots[q * kLpThreads];
      b = fmaxf(b, fminf(a, x));
      a = fmaxf(a, x);
    }
    bound1 = __shfl_sync(0xFFFFFFFFu, list_merge(list_sort(rank_value(a)), list_sort(rank_value(b))), n - 1);
  }
  const uint32_t bound = top_bound2<TH>(bound1, n, sh);
  const float fb = rank_logit((uint64_t)bound << 32);
  if (mine >= fb)
    for (int q = 0; q < used; ++q)
      if (slots[q * kLpThreads] >= fb) {
        const int at = atomicAdd(&sh.nhot, 1);
        if (at < TopShared<TH>::kHot) sh.hot[at] = q << 16 | k;
      }
  if (k == 0) sh.ncand = 0;
  group_sync<TH>();
  auto offer = [&](float x, int id) {
    if (x >= fb && x != neg_inf()) {
      const int at = atomicAdd(&sh.ncand, 1);
      if (at < TopShared<TH>::kCap) sh.cand[at] = rank_key(x, (uint32_t)id);
    }
  };
  const int nhot = sh.nhot;
  if (nhot <= TopShared<TH>::kHot) {
    const int items = nhot * run;
    for (int q = k; q < items; q += TH) {
      const int who = sh.hot[q / kLpU >> shift];
      const int i = v0 + (who & 0xFFFF) + ((who >> 16) * run + (q & (run - 1))) * TH;
      if (i < v1) {
        float x[N];
        unpack(r.vec()[i], x);
        uint32_t in = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) in |= (x[e] >= fb ? 1u : 0u) << e;
        if (in) {
          int at = atomicAdd(&sh.ncand, __popc(in));
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (in >> e & 1) {
              if (at < TopShared<TH>::kCap) sh.cand[at] = rank_key(x[e], (uint32_t)(r.head + i * N + e));
              ++at;
            }
        }
      }
    }
    if (ends) {
      if (k < r.head) offer(to_f32(r.p[k]), k);
      if (k < r.tail) offer(to_f32(r.p[r.tail_start() + k]), r.tail_start() + k);
    }
  }
  group_sync<TH>();
  const int c = sh.ncand;
  if (k == 0) sh.nhot = 0;
  if (nhot <= TopShared<TH>::kHot && c <= TopShared<TH>::kCap) return c;
  list_top<TH>(r, v0, v1, ends, bound, n, slots, sh);
  group_sync<TH>();
  return 32;
}

// put(place, key) for each of the n largest of the keys cand[0..c) of a group:
// a key's place is the number of larger ones.
template <int TH, typename F>
__device__ __forceinline__ void place_top(const uint64_t* cand, int c, int n, F put) {
  constexpr int KC = TopShared<TH>::kCap / TH;  // keys of a thread at most
  const int k = threadIdx.x & (TH - 1);
  uint64_t key[KC];
  int larger[KC];
#pragma unroll
  for (int q = 0; q < KC; ++q) key[q] = k + q * TH < c ? cand[k + q * TH] : 0, larger[q] = 0;
  for (int j = 0; j < c; j += 8) {  // the array is a multiple of 8
    uint64_t o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) o[u] = j + u < c ? cand[j + u] : 0;
#pragma unroll
    for (int q = 0; q < KC; ++q)
      if (q == 0 || c > q * TH) {
#pragma unroll
        for (int u = 0; u < 8; ++u) larger[q] += o[u] > key[q];
      }
  }
#pragma unroll
  for (int q = 0; q < KC; ++q)
    if (key[q] != 0 && larger[q] < n) put(larger[q], key[q]);
}

// The same from nb sorted lists of 32, list b at lists + 32 b (zeros after the
// last key): thread 32 b + i places the i-th key of list b, by its place there
// and a binary search of each other list.
template <typename F>
__device__ __forceinline__ void place_lists(const uint64_t* lists, int nb, int n, F put) {
  const int b = threadIdx.x >> 5, i = threadIdx.x & 31;
  if (b >= nb || i >= n) return;
  const uint64_t key = lists[32 * b + i];
  int larger = i;
#pragma unroll
  for (int o = 0; o < 8; ++o) {  // nb <= 8
    if (o < nb && o != b) {
      int at = 0;  // keys of list o known to be larger
#pragma unroll
      for (int w = 32; w > 0; w >>= 1)
        if (at + w <= 32 && lists[32 * o + at + w - 1] > key) at += w;
      larger += at;
    }
  }
  if (key != 0 && larger < n) put(larger, key);
}

// TH threads per row (or, for a cluster of nb = gridDim.x blocks, per part of
// a row), the blocks taking rows in turn.  A thread keeps its own running
// maximum and sums over its vectors; the threads meet at the row's end, with
// the next row's vectors, if they have one, on their way.  The parts of a
// cluster meet in its first block through distributed shared memory.
// 4096 x 131072 BF16 with entropy: 157 us, 6.83 TB/s, 1.0 of the measured copy
// rate (loads into registers in batches of four, two blocks per SM: 234 us,
// waiting for them; the ring keeps 64 KB per block on the way).  With 20
// alternatives 185 us: what a row's end waits for, its barriers and the second
// read of the candidates, is then no longer hidden.
template <typename E, bool ENT, bool TOP, int TH>
__global__ void __launch_bounds__(kLpThreads, kLpBlocksPerSm) token_logprobs_kernel(LogprobArgs a) {
  constexpr int NW = TH / 32, NG = kLpThreads / TH;
  extern __shared__ uint4 ring[];
  __shared__ Run<ENT> red[2][kLpThreads / 32];
  __shared__ Run<ENT> cpart;
  __shared__ uint64_t clist[32];
  __shared__ TopShared<TH> tops[TOP ? NG : 1];
  const int nb = TH < kLpThreads ? 1 : gridDim.x, rank = TH < kLpThreads ? 0 : blockIdx.x;
  const int lg = TH < kLpThreads ? 0 : 31 - __clz(nb);  // nb is a power of two
  const int group = threadIdx.x / TH, k = threadIdx.x & (TH - 1), lane = threadIdx.x & 31;
  TopShared<TH>& top = tops[TOP ? group : 0];
  begin_kernel();
  const int64_t t0 = (int64_t)blockIdx.y * NG + group, step = (int64_t)gridDim.y * NG;
  const float c = a.inv_t * kLog2e;
  const E* logits = static_cast<const E*>(a.logits);
  auto part = [&](int64_t t) {
    const Row<E> r(logits + t * a.ld, a.V);
    const int v0 = r.part(rank, lg), v1 = r.part(rank + 1, lg);
    return Part{r.vec() + v0, v1 - v0};
  };
  if (TOP && k == 0) top.nhot = 0;
  // Runs of 2^shift groups per slot, enough for the longest part.
  float* slots = reinterpret_cast<float*>(ring + kLpThreads * kLpU * kLpD<TOP>) + threadIdx.x;
  const int groups = (a.V / Row<E>::kVec / nb + kLpU * TH) / (kLpU * TH), runs = (groups + kLpSlots - 1) / kLpSlots;
  const int shift = runs <= 1 ? 0 : 32 - __clz(runs - 1);
  Stream<TH, kLpU, kLpD<TOP>, 1, E, decltype(part)> stream(part, ring + threadIdx.x, kLpThreads, k, t0, step, a.T);
  int odd = 0, ynext = a.logprob && k == 0 && rank == 0 && t0 < a.T ? a.targets[t0] : -1;
  for (int64_t t = t0; t < a.T; t += step, odd ^= 1) {
    const E* row = logits + t * a.ld;
    const Row<E> r(row, a.V);
    const int v0 = r.part(rank, lg), v1 = r.part(rank + 1, lg);
    // the target's logit, needed at the end, and the next row's target
    const int y = ynext;
    const float xy = y >= 0 && y < a.V ? to_f32(row[y]) : 0.0f;
    if (a.logprob && k == 0 && rank == 0 && t + step < a.T) ynext = a.targets[t + step];
    Run<ENT> acc;
    int slot = 0, left = 1 << shift;
    float high = neg_inf();
    stream.row(v1 - v0, [](uint4*, int) {}, [&](const auto& v, int) {
      const float mx = acc.add(v, c, E());
      if (TOP) {
        high = fmaxf(high, mx);
        slots[slot * kLpThreads] = high;
        if (--left == 0) ++slot, left = 1 << shift, high = neg_inf();
      }
    });
    if (rank == 0) {
      if (k < r.head) {
        const float x[1] = {to_f32(row[k])};
        acc.add(x, c);
      }
      if (k < r.tail) {
        const float x[1] = {to_f32(row[r.tail_start() + k])};
        acc.add(x, c);
      }
    }
    const float mine = acc.m;
    uint32_t bound1 = 0;
    if (TOP && (TH > 32 || a.n_top <= 8)) bound1 = top_bound1<TH>(rank_value(mine), a.n_top, top);
    acc.template warp_merge<32>();
    if (NW > 1) {
      if (lane == 0) red[odd][threadIdx.x >> 5] = acc;
      group_sync<TH>();
      Run<ENT> b;
      if (lane < NW) b = red[odd][group * NW + lane];
      b.template warp_merge<NW>();
      // lanes of one result: NW is a power of two below 32, lanes 0 .. NW - 1 hold it
      acc.m = b.m, acc.M = b.M;
      acc.s = __shfl_sync(0xFFFFFFFFu, b.s, 0);
      if (ENT) acc.e = __shfl_sync(0xFFFFFFFFu, b.e, 0);
    }
    int found = 0;
    if (TOP) {
      if (NW == 1) __syncwarp();
      if (finite_max(acc.m)) found = group_top<TH>(r, v0, v1, rank == 0, mine, bound1, slots, shift, a.n_top, top);
    }
    if (nb > 1) {
      if (threadIdx.x == 0) cpart = acc;
      if (TOP) {
        if (threadIdx.x < 32) clist[threadIdx.x] = 0;
        __syncthreads();
        place_top<TH>(top.cand, found, a.n_top, [&](int at, uint64_t key) { clist[at] = key; });
      }
      cluster_arrive();
      cluster_wait();
      if (rank == 0) {
        Run<ENT> b;
        if (lane < nb) {
          b.m = cluster_load_f32(&cpart.m, lane);
          b.M = cluster_load_f32(&cpart.M, lane);
          b.s = cluster_load_f32(&cpart.s, lane);
          if (ENT) b.e = cluster_load_f32(&cpart.e, lane);
        }
        b.template warp_merge<8>();
        acc.m = b.m, acc.M = b.M;
        acc.s = __shfl_sync(0xFFFFFFFFu, b.s, 0);
        if (ENT) acc.e = __shfl_sync(0xFFFFFFFFu, b.e, 0);
        if (TOP) {  // the parts' lists, all threads done with this block's own candidates
          found = finite_max(acc.m) ? nb * 32 : 0;
          if ((int)threadIdx.x < found) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(&clist[lane]);
            const uint64_t lo = cluster_load(p, threadIdx.x >> 5), hi = cluster_load(p + 1, threadIdx.x >> 5);
            top.cand[threadIdx.x] = lo | (hi << 32);
          }
        }
      }
      cluster_arrive();  // the other blocks' shared memory is read no more
      cluster_wait();
      if (rank != 0) continue;
      if (TOP) __syncthreads();
    }
    // ln-sum about the maximum, and entropy, of the row
    const bool bad = !finite_max(acc.m);
    bool none = false;
    const float log2s = log2f(acc.s);
    float l = kLn2 * (log2s - fmaf(acc.m, c, -acc.M));
    float H = ENT ? kLn2 * (log2s - acc.e / acc.s) : 0.0f;
    if (!bad && !acc.shift_ok(c)) {  // beyond the shift's range, or nothing but masks: differences first
      Soft<ENT> all;
      for (int i = k; i < a.V; i += TH) {
        const float x[1] = {to_f32(row[i])};
        all.add(x, c);
      }
      all.warp_merge(c);
      if (NW > 1) {
        __shared__ Soft<ENT> sred[kLpThreads / 32];
        if (lane == 0) sred[threadIdx.x >> 5] = all;
        group_sync<TH>();
        all = Soft<ENT>();
        if (lane < NW) all = sred[group * NW + lane];
        all.warp_merge(c);
        group_sync<TH>();
      }
      none = all.s == 0.0f;
      l = logf(all.s);
      if (ENT) H = l - a.inv_t * (all.e / all.s);
    }
    const float nan = quiet_nan();
    auto logp = [&](float x) { return (x - acc.m) * a.inv_t - l; };
    if (k == 0) {
      if (bad) set_status(a.status, MOE_STATUS_NONFINITE_LOGITS);
      if (a.logprob) {
        if (y >= a.V) set_status(a.status, MOE_STATUS_BAD_TOKEN);
        a.logprob[t] = y < 0 || y >= a.V ? 0.0f : bad ? nan : none ? neg_inf() : logp(xy);
      }
      if (ENT) a.entropy[t] = bad ? nan : none ? 0.0f : H;
      if (a.stats) {
        a.stats[2 * t] = bad ? nan : none ? neg_inf() : acc.m;
        a.stats[2 * t + 1] = bad ? nan : none ? 0.0f : l;
      }
    }
    if (TOP) {
      int32_t* ids = a.top_ids + t * a.n_top;
      float* lps = a.top_logprob + t * a.n_top;
      if (found <= 32 || nb > 1) {  // places that may stay empty
        for (int q = k; q < a.n_top; q += TH) ids[q] = -1, lps[q] = bad ? nan : neg_inf();
        group_sync<TH>();
      }
      auto put = [&](int at, uint64_t key) {
        ids[at] = rank_id(key);
        lps[at] = logp(rank_logit(key));
      };
      if (nb > 1) place_lists(top.cand, found / 32, a.n_top, put);
      else place_top<TH>(top.cand, found, a.n_top, put);
      group_sync<TH>();  // the candidates are read no more
    }
  }
}

// d_v = inv_t (p_v (A - g_ent ln p_v) + g 1[v = target]), A = -g - g_ent H.
// TH threads per row; with whole blocks, blockIdx.x is a part of the row.
// 4096 x 131072 BF16: 307 us, 7.0 TB/s, 1.03 of the measured copy rate.
constexpr int kLbThreads = 256;
constexpr int kLbBatch = 4;
constexpr int kLbPart = kLbThreads * kLbBatch * 2;  // vectors of a block

template <typename E, int TH>
__global__ void __launch_bounds__(kLbThreads) token_logprobs_backward_kernel(LogprobBwdArgs a) {
  constexpr int N = Row<E>::kVec;
  const int tid = threadIdx.x % TH;
  const int64_t t = (blockIdx.y + (int64_t)blockIdx.z * gridDim.y) * (kLbThreads / TH) + threadIdx.x / TH;
  begin_kernel();
  if (t >= a.T) return;
  const E* row = static_cast<const E*>(a.logits) + t * a.ld;
  E* out = static_cast<E*>(a.dlogits) + t * a.ldd;
  const int y = a.targets ? a.targets[t] : -1;
  if (y >= a.V && tid == 0 && blockIdx.x == 0) set_status(a.status, MOE_STATUS_BAD_TOKEN);
  const bool has = y >= 0 && y < a.V;
  const float g = has && a.g_logprob ? a.g_logprob[t] * a.inv_t : 0.0f;
  const float ge = a.g_entropy ? a.g_entropy[t] * a.inv_t : 0.0f;
  const float m = a.stats[2 * t], l = a.stats[2 * t + 1];
  const bool zero = m == neg_inf() || (g == 0.0f && ge == 0.0f);
  const float A = -g - (a.g_entropy ? ge * a.entropy[t] : 0.0f);
  // a masked id gives p = 0 times a finite number: its ln p is held at a value
  // where p is 0 long since, small enough for any product with g_entropy
  // inv_temperature below 3e34; a NaN row's l makes all its values NaN
  auto grad = [&](float x) {
    const float lp = fmaxf((x - m) * a.inv_t, -1e4f) - l;
    return exp2_fast(lp * kLog2e) * fmaf(-ge, lp, A);
  };
  const Row<E> r(row, a.V);
  if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
    const int b = blockIdx.x, v0 = b * kLbPart, v1 = TH < kLbThreads ? r.nvec : min(v0 + kLbPart, r.nvec);
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
    int i = v0 + tid;
    if (zero) {
      for (; i < v1; i += TH) __stcs(ov + i, make_uint4(0u, 0u, 0u, 0u));
    } else {
      for (; i + (kLbBatch - 1) * TH < v1; i += kLbBatch * TH) {
        uint4 v[kLbBatch];
#pragma unroll
        for (int u = 0; u < kLbBatch; ++u) v[u] = __ldcs(r.vec() + i + u * TH);
#pragma unroll
        for (int u = 0; u < kLbBatch; ++u) store(v[u], i + u * TH);
      }
      for (; i < v1; i += TH) store(__ldcs(r.vec() + i), i);
    }
    if (b == 0) {
      const int k = tid < r.head ? tid : r.tail_start() + tid - r.head;
      if (tid < r.head + r.tail) {
        const float v = zero ? 0.0f : grad(to_f32(row[k])) + (k == y ? g : 0.0f);
        from_f32(v, out[k]);
      }
    }
  } else {  // rows of different alignment: element by element
    const int64_t per = (a.V + gridDim.x - 1) / gridDim.x, k0 = per * blockIdx.x;
    const int64_t k1 = k0 + per < a.V ? k0 + per : a.V;
    for (int64_t k = k0 + tid; k < k1; k += TH) {
      const float v = zero ? 0.0f : grad(to_f32(row[k])) + (k == y ? g : 0.0f);
      from_f32(v, out[k]);
    }
  }
}

// host launchers
template <typename E, int TH>
static void (*token_logprobs_of(bool ent, bool top))(LogprobArgs) {
  return ent ? (top ? token_logprobs_kernel<E, true, true, TH> : token_logprobs_kernel<E, true, false, TH>)
             : (top ? token_logprobs_kernel<E, false, true, TH> : token_logprobs_kernel<E, false, false, TH>);
}
template <typename E>
static void (*token_logprobs_of(int th, bool ent, bool top))(LogprobArgs) {
  return th == 32    ? token_logprobs_of<E, 32>(ent, top)
         : th == 128 ? token_logprobs_of<E, 128>(ent, top)
                     : token_logprobs_of<E, kLpThreads>(ent, top);
}
int launch_token_logprobs(const LogprobArgs& a, cudaStream_t s) {
  const bool bf = a.dtype == MOE_DTYPE_BF16, ent = a.entropy != nullptr, top = a.n_top > 0;
  const int64_t nvec = (int64_t)a.V * (bf ? 2 : 4) / 16;
  const int most = kLpBlocksPerSm * gemm_num_ctas();  // resident blocks
  // Threads per row.  256 where each row can have a block at once (400 x 16384
  // BF16 4.9 us, with 128 threads 5.9; with 20 alternatives 8.1 and 11).  With
  // more rows as few as hide a row's end (sums, alternatives) behind the others:
  // a warp for short rows, four for long ones (BF16, no alternatives: 4000 x 8192
  // 16, 19 and 29 us with 32, 128 and 256 threads; 2000 x 20000 17, 19 and 25;
  // 4000 x 50000 67, 62 and 70; 1500 x 16384 17, 14 and 15).  With alternatives
  // L2 should still hold a row at its end: 256 threads from 160 KB on (2000 x
  // 131072 with 20: 113 us with 128, 99 with 256; 4000 x 65536: 107 and 108).
  // Where blocks are left over, clusters of up to 8 of them, while each thread
  // keeps two vectors (2 x 131072 with 20: 18 us with one block per row, 14 with 8).
  const bool warp = nvec <= 128 || (nvec <= 256 && a.T >= 304) || (nvec <= 512 && a.T >= 1000) ||
                    (nvec <= 3072 && a.T >= 2000);
  const int th = warp ? 32 : a.T > most && !(top && nvec > 10240) ? 128 : kLpThreads;
  int nb = 1;
  if (th == kLpThreads)
    while (nb < 8 && (int64_t)a.T * nb * 2 <= most && nvec / (nb * 2) >= 2 * kLpThreads) nb *= 2;
  const int64_t per = kLpThreads / th, want = (a.T + per - 1) / per;
  const int64_t grid = nb > 1 ? most / nb : (int64_t)most * kLpTurns;
  const int smem = top ? kLpSmem<true> : kLpSmem<false>;
  auto f = bf ? token_logprobs_of<uint16_t>(th, ent, top) : token_logprobs_of<float>(th, ent, top);
  if (!allow_smem((const void*)f, smem, smem)) return -1;
  return launch_kernel(f, dim3(nb, (unsigned)(want < grid ? want : grid)), kLpThreads, smem, nb, s, a);
}
int launch_token_logprobs_backward(const LogprobBwdArgs& a, cudaStream_t s) {
  const int64_t nvec = (int64_t)a.V * (a.dtype == MOE_DTYPE_BF16 ? 2 : 4) / 16;
  // A warp per row where a row is too short for a block (40000 x 2000 BF16: 89
  // us with blocks, 53 with warps).
  const bool small = nvec <= 512 && a.T >= 1024;
  const unsigned rows = small ? ((unsigned)a.T + kLbThreads / 32 - 1) / (kLbThreads / 32) : (unsigned)a.T;
  const unsigned nb = (unsigned)(small || nvec <= kLbPart ? 1 : (nvec + kLbPart - 1) / kLbPart);
  const unsigned gy = rows < 65535 ? rows : 65535, gz = (rows + gy - 1) / gy;
  auto f = a.dtype == MOE_DTYPE_BF16 ? (small ? token_logprobs_backward_kernel<uint16_t, 32>
                                              : token_logprobs_backward_kernel<uint16_t, kLbThreads>)
                                     : (small ? token_logprobs_backward_kernel<float, 32>
                                              : token_logprobs_backward_kernel<float, kLbThreads>);
  return launch_kernel(f, dim3(nb, gy, gz), kLbThreads, 0, 1, s, a);
}

}  // namespace moe
