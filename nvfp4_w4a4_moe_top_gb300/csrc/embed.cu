// The embedding's rows and the gradient of its table.
//   out_t = scale table[ids_t];   dtable_v = scale sum_{t: ids_t = v} dy_t.
// Both are bound by HBM: the rows that tokens name in and one row per token
// out; one row per token in and every row of the table out.
//   65536 tokens, d = 2048, V = 131072: embedding 62.5 us, 0.86 of the measured
//   copy rate; gradient 232 us in five launches, 0.85 (counting 5, two passes of
//   the sort 16 and 10, sums and zeros 193, joining 14, each by itself).
//   512 tokens, d = 1024, V = 32768: gradient 23 us in one launch, 0.87.
// Added to a table (accumulate), where only the named rows are read and written: 144
// and 7 us.
#include "tokens.cuh"

namespace moe {

constexpr int kEmThreads = 256;

// Vectors of 8 values: TX threads along a row (a power of two), 256 / TX rows
// at a time, kEmRows rows per thread, their loads issued together, as each waits
// for its id first.
constexpr int kEmRows = 4;

__device__ __forceinline__ uint4 scaled8(const uint16_t* p, float scale) {
  float x[8];
  unpack(*reinterpret_cast<const uint4*>(p), x);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= scale;
  return pack(x);
}
__device__ __forceinline__ uint4 scaled8(const float* p, float scale) {
  float a[4], b[4], x[8];
  unpack(reinterpret_cast<const uint4*>(p)[0], a);
  unpack(reinterpret_cast<const uint4*>(p)[1], b);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = a[e] * scale, x[4 + e] = b[e] * scale;
  return pack(x);
}

template <typename E>
__global__ void __launch_bounds__(kEmThreads) embed_tokens_kernel(EmbedArgs a, int tx_log) {
  const int tx = 1 << tx_log, rows = kEmThreads >> tx_log;
  const int c = (blockIdx.y * tx + (threadIdx.x & (tx - 1))) * 8;
  const int64_t t0 = (int64_t)blockIdx.x * rows * kEmRows + (threadIdx.x >> tx_log);
  begin_kernel();
  if (c >= a.d) return;
  int id[kEmRows];
#pragma unroll
  for (int r = 0; r < kEmRows; ++r) id[r] = t0 + r * rows < a.T ? a.ids[t0 + r * rows] : -1;
  uint4 v[kEmRows];
#pragma unroll
  for (int r = 0; r < kEmRows; ++r) {
    v[r] = make_uint4(0u, 0u, 0u, 0u);
    if ((unsigned)id[r] < (unsigned)a.V) v[r] = scaled8(static_cast<const E*>(a.table) + (int64_t)id[r] * a.ldt + c, a.scale);
    else if (id[r] >= a.V && c == 0) set_status(a.status, MOE_STATUS_BAD_TOKEN);
  }
#pragma unroll
  for (int r = 0; r < kEmRows; ++r)
    if (t0 + r * rows < a.T) __stcs(reinterpret_cast<uint4*>(a.out + (t0 + r * rows) * a.ldo + c), v[r]);
}

// log2 of the threads along a row of `vecs` vectors.
static int threads_along(int vecs) {
  int l = 0;
  while (l < 8 && (1 << l) < vecs) ++l;
  return l;
}

int launch_embed_tokens(const EmbedArgs& a, cudaStream_t s) {
  const int l = threads_along(a.d / 8), rows = (kEmThreads >> l) * kEmRows;
  const dim3 grid((unsigned)((a.T + (int64_t)rows - 1) / rows), (unsigned)((a.d / 8 + (1 << l) - 1) >> l));
  auto f = a.dtype == MOE_DTYPE_BF16 ? embed_tokens_kernel<uint16_t> : embed_tokens_kernel<float>;
  return launch_kernel(f, grid, kEmThreads, 0, 1, s, a, l);
}

// ---- gradient ----
// Up to kFewTokens tokens: one launch, in which each token's first occurrence sums
// all of them.  More: the tokens are sorted by id (stable, so ascending t within an
// id) with a radix sort of up to 9 bits a pass; tiles of the sorted tokens are then
// summed run by run.  A run inside one tile goes to the table at once; the parts of
// a run that crosses tiles go to the workspace and are added in the order of the
// tiles by a last launch.  Ids out of range sort behind all others, as V.
//
// One launch looks through all ids in every block, the sort has five launches: with
// V = 131072 and d = 2048, 300 tokens 146 us and 155, 1000 tokens 159 and 158, 2000
// tokens 210 and 161; with V = 4096 and d = 512, 1000 tokens 8 and 19.
constexpr int kFewTokens = 1024;
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 9, kBins = 1 << kMaxBits;

struct SortPlan {
  int passes, bits;  // bits of a digit
  int items;         // tokens of a thread
  int blocks;
  int tile, tiles;   // sorted tokens summed by one group of threads
  size_t key[2], val[2], hist[3], bitmap, part, bytes;
};

static SortPlan sort_plan(int T, int V, int d) {
  SortPlan p = {};
  if (T <= kFewTokens) return p;
  int n = 1;
  while ((int64_t(1) << n) <= V) ++n;  // ids up to V
  p.passes = (n + kMaxBits - 1) / kMaxBits;
  p.bits = (n + p.passes - 1) / p.passes;
  // Up to 64 chunks, as every chunk reads the counts of all, while a thread then has
  // no more than 32 tokens, that is up to 2^20 tokens; beyond, a chunk per 16384
  // tokens, and the counts read grow with the square: at 2^24 tokens 1024 chunks of
  // 2 MB each in a pass (V = 131072, d = 8, two passes: 3.6 ms).  Tiles as long as leave
  // 1024 of them for the columns of a block, up to 64: a run's parts are then few
  // (32 tokens and 2048 tiles: 65536 x 2048 244 us, 236 so; 16003 x 1000 68 and 62).
  p.items = 1;
  while (p.items < 32 && (int64_t)p.items * kSortThreads * 64 < T) p.items *= 2;
  const int chunk = p.items * kSortThreads;
  p.blocks = (T + chunk - 1) / chunk;
  p.tile = 4;
  const int64_t cols = (d / 8 + 255) / 256;
  while (p.tile < 64 && T / p.tile * cols > 1024) p.tile *= 2;
  p.tiles = (T + p.tile - 1) / p.tile;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 255) / 256 * 256;
    return o;
  };
  for (int i = 0; i < 2; ++i) p.key[i] = take((size_t)T * 4), p.val[i] = take((size_t)T * 4);
  for (int i = 0; i < 3; ++i) p.hist[i] = i < p.passes ? take((size_t)p.blocks * kBins * 4) : 0;
  p.bitmap = take((size_t)(V + 31) / 32 * 4);
  p.part = take((size_t)p.tiles * 2 * d * 4);
  p.bytes = at;
  return p;
}
size_t embed_tokens_backward_ws(int T, int V, int d) {
  const size_t n = sort_plan(T, V, d).bytes;
  return n ? n : 8 * (size_t)kFewTokens;  // not used
}

__device__ __forceinline__ int sort_key(int id, int V) { return (unsigned)id < (unsigned)V ? id : V; }

// Digits of each chunk of the tokens, [chunk][bin]; clears the next passes'
// counts and the bit map.
__global__ void __launch_bounds__(kSortThreads)
    embed_sort_count_kernel(const int32_t* ids, int T, int V, int items, int bits, uint32_t* hist, uint32_t* clear,
                            int64_t clear_words, uint32_t* bitmap, int bitmap_words, int* status) {
  __shared__ uint32_t bins[kBins];
  const int k = threadIdx.x;
  bins[k] = 0;
  begin_kernel();
  __syncthreads();
  const int t0 = blockIdx.x * items * kSortThreads;
  bool bad = false;
  for (int i = 0; i < items; ++i) {
    const int t = t0 + i * kSortThreads + k;
    if (t < T) {
      const int id = ids[t];
      bad |= id >= V;
      atomicAdd(&bins[sort_key(id, V) & ((1 << bits) - 1)], 1u);
    }
  }
  if (bad) set_status(status, MOE_STATUS_BAD_TOKEN);
  __syncthreads();
  hist[(int64_t)blockIdx.x * kBins + k] = bins[k];
  const int64_t n = (int64_t)gridDim.x * kSortThreads, g = (int64_t)blockIdx.x * kSortThreads + k;
  for (int64_t i = g; i < clear_words; i += n) clear[i] = 0;
  for (int64_t i = g; i < bitmap_words; i += n) bitmap[i] = 0;
}

// One pass: each chunk's tokens to their places by the digit at `shift`, and
// the next digit's counts of the chunks where they land (next_hist, or NULL).
// key_in NULL: the first pass, of the ids themselves, which also marks them in
// the bit map.
__global__ void __launch_bounds__(kSortThreads)
    embed_sort_scatter_kernel(const int32_t* ids, const int32_t* key_in, const int32_t* val_in, int T, int V, int items,
                              int bits, int shift, const uint32_t* hist, uint32_t* next_hist, uint32_t* bitmap,
                              int32_t* key_out, int32_t* val_out) {
  __shared__ uint32_t place[kSortWarps][kBins];
  __shared__ uint32_t sums[kSortWarps];
  const int k = threadIdx.x, warp = k >> 5, lane = k & 31;
  const uint32_t mask = (1u << bits) - 1;
  for (int w = 0; w < kSortWarps; ++w) place[w][k] = 0;
  begin_kernel();
  // tokens of smaller digits, and of this digit in earlier chunks
  uint32_t before = 0, total = 0;
#pragma unroll 16
  for (int b = 0; b < (int)gridDim.x; ++b) {
    const uint32_t c = hist[(int64_t)b * kBins + k];
    before += b < (int)blockIdx.x ? c : 0;
    total += c;
  }
  uint32_t incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  uint32_t base = incl - total + before;
  for (int w = 0; w < warp; ++w) base += sums[w];
  // warp w takes items * 32 consecutive tokens
  const int64_t w0 = (int64_t)blockIdx.x * items * kSortThreads + (int64_t)warp * items * 32;
  auto load = [&](int i, int& key, int& val) {
    const int64_t t = w0 + i * 32 + lane;
    key = -1, val = (int)t;
    if (t < T) {
      if (key_in) key = key_in[t], val = val_in[t];
      else key = sort_key(ids[t], V);
    }
  };
  for (int i = 0; i < items; ++i) {
    int key, val;
    load(i, key, val);
    if (key >= 0) atomicAdd(&place[warp][(key >> shift) & mask], 1u);
  }
  __syncthreads();
  for (int w = 0; w < kSortWarps; ++w) {
    const uint32_t c = place[w][k];
    place[w][k] = base;
    base += c;
  }
  __syncthreads();
  const int chunk = items * kSortThreads;
  for (int i = 0; i < items; ++i) {
    int key, val;
    load(i, key, val);
    const uint32_t digit = key >= 0 ? (key >> shift) & mask : kBins;  // kBins: no token
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, digit);
    if (key >= 0) {
      const uint32_t at = place[warp][digit] + __popc(same & ((1u << lane) - 1));
      key_out[at] = key;
      val_out[at] = val;
      if (next_hist) atomicAdd(&next_hist[(int64_t)(at / chunk) * kBins + ((key >> (shift + bits)) & mask)], 1u);
    }
    if (!key_in) {  // one atomic per word of the bit map and warp: frequent ids are many
      const bool named = key >= 0 && key < V;
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, named ? key >> 5 : -1);
      const uint32_t bits = __reduce_or_sync(peers, named ? 1u << (key & 31) : 0u);
      if (named && lane == __ffs(peers) - 1) atomicOr(&bitmap[key >> 5], bits);
    }
    __syncwarp();
    if (key >= 0 && lane == __ffs(same) - 1) place[warp][digit] += __popc(same);
    __syncwarp();
  }
}

// Eight values, as one store where the address allows it: with two stores of half
// a sector each the 65536 x 2048 gradient took 296 us, 236 so.
__device__ __forceinline__ void store8(float* p, const float4& lo, const float4& hi) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(lo.x), "f"(lo.y), "f"(lo.z),
                 "f"(lo.w), "f"(hi.x), "f"(hi.y), "f"(hi.z), "f"(hi.w)
                 : "memory");
  } else {
    __stcs(reinterpret_cast<float4*>(p), lo);
    __stcs(reinterpret_cast<float4*>(p) + 1, hi);
  }
}
__device__ __forceinline__ void put8(float* p, const float (&x)[8], float scale, bool add) {
  float4 lo = make_float4(x[0] * scale, x[1] * scale, x[2] * scale, x[3] * scale);
  float4 hi = make_float4(x[4] * scale, x[5] * scale, x[6] * scale, x[7] * scale);
  if (add) {
    const float4 a = reinterpret_cast<float4*>(p)[0], b = reinterpret_cast<float4*>(p)[1];
    lo.x += a.x, lo.y += a.y, lo.z += a.z, lo.w += a.w;
    hi.x += b.x, hi.y += b.y, hi.z += b.z, hi.w += b.w;
  }
  store8(p, lo, hi);
}
__device__ __forceinline__ void zero8(float* p) {
  const float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  store8(p, z, z);
}

struct SumArgs {
  EmbedBwdArgs a;
  const int32_t* key;
  const int32_t* val;
  const uint32_t* bitmap;
  float* part;
  int tile, tiles, sum_blocks;
};

// Blocks 0 .. sum_blocks - 1: 256 / TX tiles of sorted tokens each.  The rest:
// zeros into the rows of the table that no token names.
__global__ void __launch_bounds__(kEmThreads) embed_sum_kernel(SumArgs s, int tx_log) {
  const EmbedBwdArgs& a = s.a;
  const int tx = 1 << tx_log, ty = threadIdx.x >> tx_log, rows = kEmThreads >> tx_log;
  const int c = (blockIdx.y * tx + (threadIdx.x & (tx - 1))) * 8;
  begin_kernel();
  if (c >= a.d) return;
  if ((int)blockIdx.x >= s.sum_blocks) {
    // 32 rows, a word of the bit map, per group of threads
    const int v0 = (((int)blockIdx.x - s.sum_blocks) * rows + ty) * 32, n = min(a.V - v0, 32);
    if (n <= 0) return;
    const uint32_t named = s.bitmap[v0 >> 5];
    for (int i = 0; i < n; ++i)
      if (!(named >> i & 1)) zero8(a.dtable + (int64_t)(v0 + i) * a.d + c);
    return;
  }
  const int64_t tile = (int64_t)blockIdx.x * rows + ty;
  if (tile >= s.tiles) return;
  const int64_t p0 = tile * s.tile, p1 = p0 + s.tile < a.T ? p0 + s.tile : a.T;
  int cur = s.key[p0];
  bool from = p0 > 0 && s.key[p0 - 1] == cur;  // the run began in an earlier tile
  const int next = p1 < a.T ? s.key[p1] : -1;
  float acc[8] = {};
  for (int64_t p = p0; p < p1; p += 4) {
    int id[4];
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      id[i] = p + i < p1 ? s.key[p + i] : -1;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (id[i] >= 0 && id[i] < a.V) v[i] = __ldcs(reinterpret_cast<const uint4*>(a.dy + (int64_t)s.val[p + i] * a.ldy + c));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (id[i] < 0) break;
      if (id[i] != cur) {
        if (cur < a.V) {
          if (from) put8(s.part + (tile * 2) * a.d + c, acc, 1.0f, false);
          else put8(a.dtable + (int64_t)cur * a.d + c, acc, a.scale, a.accumulate);
        }
        cur = id[i], from = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
      }
      float x[8];
      unpack(v[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += x[e];
    }
  }
  if (cur < a.V) {
    if (from) put8(s.part + (tile * 2) * a.d + c, acc, 1.0f, false);
    else if (next == cur) put8(s.part + (tile * 2 + 1) * a.d + c, acc, 1.0f, false);
    else put8(a.dtable + (int64_t)cur * a.d + c, acc, a.scale, a.accumulate);
  }
}

// The parts of each run that begins in a tile and ends in a later one, added in
// the order of the tiles, for 128 columns: a warp per tile; a frequent token's run,
// which crosses a hundred tiles, by the block's eight warps, a consecutive eighth
// each, and the eighths in turn.
constexpr int kJoinWarps = kEmThreads / 32;
__global__ void __launch_bounds__(kEmThreads) embed_join_kernel(SumArgs s) {
  __shared__ int64_t length[kJoinWarps];
  __shared__ float4 sums[kJoinWarps][32];
  const EmbedBwdArgs& a = s.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.y * 128 + lane * 4;
  const int64_t first = (int64_t)blockIdx.x * kJoinWarps, tile = first + warp;
  begin_kernel();
  const bool in = c < a.d;
  // the tiles after this one that the run goes on in, if it begins here
  int64_t n = 0;
  int id = -1;
  if (tile + 1 < s.tiles) {
    const int64_t p0 = tile * s.tile, p1 = p0 + s.tile;
    id = s.key[p1 - 1];
    if (id < a.V && s.key[p1] == id && !(s.key[p0] == id && p0 > 0 && s.key[p0 - 1] == id))
      for (;;) {
        const int64_t next = tile + 1 + n + lane;
        const uint32_t others = __ballot_sync(0xFFFFFFFFu, next >= s.tiles || s.key[next * s.tile] != id);
        n += others ? __ffs(others) - 1 : 32;
        if (others) break;
      }
  }
  // the sum of parts [j0, j1) of the run that begins in tile t
  auto sum = [&](int64_t t, int64_t j0, int64_t j1) {
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t j = j0; j < j1; j += 8) {
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t slot = j + i == 0 ? t * 2 + 1 : (t + j + i) * 2;
        v[i] = in && j + i < j1 ? *reinterpret_cast<const float4*>(s.part + slot * a.d + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i < j1) acc.x += v[i].x, acc.y += v[i].y, acc.z += v[i].z, acc.w += v[i].w;
    }
    return acc;
  };
  auto put = [&](float4 acc, int id) {
    if (!in) return;
    float4* out = reinterpret_cast<float4*>(a.dtable + (int64_t)id * a.d + c);
    acc.x *= a.scale, acc.y *= a.scale, acc.z *= a.scale, acc.w *= a.scale;
    if (a.accumulate) {
      const float4 o = *out;
      acc.x += o.x, acc.y += o.y, acc.z += o.z, acc.w += o.w;
    }
    __stcs(out, acc);
  };
  constexpr int kAlone = 16;
  if (n > 0 && n < kAlone) put(sum(tile, 0, n + 1), id);
  if (lane == 0) length[warp] = n;
  __syncthreads();
  for (int w = 0; w < kJoinWarps; ++w) {
    const int64_t m = length[w] + 1;
    if (m <= kAlone) continue;
    const int64_t t = first + w;
    sums[warp][lane] = sum(t, m * warp / kJoinWarps, m * (warp + 1) / kJoinWarps);
    __syncthreads();
    if (warp == 0) {
      float4 acc = sums[0][lane];
      for (int i = 1; i < kJoinWarps; ++i) {
        const float4 v = sums[i][lane];
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
      }
      put(acc, s.key[(t + 1) * s.tile]);
    }
    __syncthreads();
  }
}

// Few tokens: no sort, as each block can look through all ids (512 tokens, d =
// 1024, V = 32768: 23 us, sorted 37).  Blocks 0 .. T * parts - 1: a token and 256
// columns; the block of the id's first occurrence lists all of them in order, its
// eight warps sum a consecutive eighth each, and the eighths are added in turn.  The
// rest: zeros into the rows that no token names, `zero_rows` of them per block.
__global__ void __launch_bounds__(kEmThreads) embed_few_kernel(EmbedBwdArgs a, int parts, int zero_rows) {
  constexpr int kIds = kFewTokens / kEmThreads, kZeroWords = 8;
  __shared__ int list[kFewTokens];
  __shared__ int counts[kEmThreads / 32];
  __shared__ float sums[kEmThreads / 32][256];
  __shared__ uint32_t named[kZeroWords];
  const int k = threadIdx.x, lane = k & 31, warp = k >> 5;
  if (k < kZeroWords) named[k] = 0;
  begin_kernel();
  __syncthreads();
  const int64_t zero = (int64_t)blockIdx.x - (int64_t)a.T * parts;
  if (zero >= 0) {
    const int v0 = (int)zero * zero_rows, n = min(a.V - v0, zero_rows);  // at most 32 kZeroWords rows
    for (int t = k; t < a.T; t += kEmThreads) {
      const uint32_t at = (uint32_t)(a.ids[t] - v0);
      if (a.ids[t] >= v0 && at < (uint32_t)n) atomicOr(&named[at >> 5], 1u << (at & 31));
    }
    __syncthreads();
    const int vecs = a.d / 8;
    for (int i = k; i < n * vecs; i += kEmThreads) {
      const int v = i / vecs;
      if (!(named[v >> 5] >> (v & 31) & 1)) zero8(a.dtable + (int64_t)(v0 + v) * a.d + (i - v * vecs) * 8);
    }
    return;
  }
  const int t = (int)blockIdx.x / parts, c = ((int)blockIdx.x % parts) * 256 + lane * 8;
  // this thread's consecutive tokens
  int mine[kIds], n = 0;
  bool earlier = false;
  const int id = a.ids[t];
#pragma unroll
  for (int i = 0; i < kIds; ++i) {
    const int j = k * kIds + i;
    mine[i] = j < a.T && a.ids[j] == id;
    earlier |= mine[i] && j < t;
    n += mine[i];
  }
  if (id >= a.V && k == 0 && c == 0) set_status(a.status, MOE_STATUS_BAD_TOKEN);
  if (__syncthreads_or(earlier) || id < 0 || id >= a.V) return;
  int at = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, at, o);
    if (lane >= o) at += v;
  }
  if (lane == 31) counts[warp] = at;
  __syncthreads();
  at -= n;
  int total = 0;
#pragma unroll
  for (int w = 0; w < kEmThreads / 32; ++w) {
    if (w < warp) at += counts[w];
    total += counts[w];
  }
#pragma unroll
  for (int i = 0; i < kIds; ++i)
    if (mine[i]) list[at++] = k * kIds + i;
  __syncthreads();
  // one warp is enough for a few
  const int warps = total <= 8 ? 1 : kEmThreads / 32, p0 = total * warp / warps, p1 = warp < warps ? total * (warp + 1) / warps : p0;
  if (warp >= warps) return;
  float acc[8] = {};
  if (c < a.d)
    for (int p = p0; p < p1; p += 8) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = p + i < p1 ? __ldcs(reinterpret_cast<const uint4*>(a.dy + (int64_t)list[p + i] * a.ldy + c)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[8];
        unpack(v[i], x);
        if (p + i < p1) {
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += x[e];
        }
      }
    }
  if (warps > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[warp][lane * 8 + e] = acc[e];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < kEmThreads / 32; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += sums[w][lane * 8 + e];
  }
  if (c < a.d) put8(a.dtable + (int64_t)id * a.d + c, acc, a.scale, a.accumulate);
}

int launch_embed_tokens_backward(const EmbedBwdArgs& a, cudaStream_t s) {
  if (a.T <= kFewTokens) {
    const int parts = (a.d + 255) / 256;
    // zeros: some 32 KB per block, and 256 rows at most
    const int rows = a.d >= 8192 ? 1 : 8192 / a.d > 256 ? 256 : 8192 / a.d;
    const unsigned zero = a.accumulate ? 0u : ((unsigned)a.V + rows - 1) / rows;
    return launch_kernel(embed_few_kernel, (unsigned)(a.T * parts) + zero, kEmThreads, 0, 1, s, a, parts, rows);
  }
  const SortPlan p = sort_plan(a.T, a.V, a.d);
  auto ints = [&](size_t o) { return reinterpret_cast<int32_t*>(a.ws + o); };
  auto words = [&](size_t o) { return reinterpret_cast<uint32_t*>(a.ws + o); };
  int rc = launch_kernel(embed_sort_count_kernel, p.blocks, kSortThreads, 0, 1, s, a.ids, a.T, a.V, p.items, p.bits,
                         words(p.hist[0]), words(p.hist[1]),
                         p.passes > 1 ? (int64_t)(p.bitmap - p.hist[1]) / 4 : int64_t(0), words(p.bitmap), (a.V + 31) / 32,
                         a.status);
  for (int i = 0; i < p.passes && rc == 0; ++i)
    rc = launch_kernel(embed_sort_scatter_kernel, p.blocks, kSortThreads, 0, 1, s, a.ids,
                       i ? ints(p.key[(i - 1) & 1]) : nullptr, i ? ints(p.val[(i - 1) & 1]) : nullptr, a.T, a.V, p.items,
                       p.bits, i * p.bits, words(p.hist[i]), i + 1 < p.passes ? words(p.hist[i + 1]) : nullptr,
                       words(p.bitmap), ints(p.key[i & 1]), ints(p.val[i & 1]));
  if (rc != 0) return rc;
  const int last = (p.passes - 1) & 1, l = threads_along(a.d / 8), rows = kEmThreads >> l;
  SumArgs m = {a, ints(p.key[last]), ints(p.val[last]), words(p.bitmap), reinterpret_cast<float*>(a.ws + p.part),
               p.tile, p.tiles, (p.tiles + rows - 1) / rows};
  const unsigned cols = (unsigned)((a.d / 8 + (1 << l) - 1) >> l);
  const unsigned zero = a.accumulate ? 0u : (unsigned)((a.V + 32ll * rows - 1) / (32 * rows));
  rc = launch_kernel(embed_sum_kernel, dim3((unsigned)m.sum_blocks + zero, cols), kEmThreads, 0, 1, s, m, l);
  if (rc != 0) return rc;
  return launch_kernel(embed_join_kernel, dim3((unsigned)(p.tiles + kJoinWarps - 1) / kJoinWarps, (unsigned)(a.d + 127) / 128),
                       kEmThreads, 0, 1, s, m);
}

}  // namespace moe
