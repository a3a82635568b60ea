// Residual add + RMS norm with BF16 and block-scaled 8-bit outputs, and its
// gradient.  Both are bound by HBM: about ten operations per element against
// eight bytes.
//   forward   h = x + res, r = 1 / sqrt(mean h^2 + eps), y = h r w
//   backward  n = h r, a = dy w: dx = r (a - n mean(a n)) + dh, dw = sum dy n
// Sums are FP32; h is rounded to BF16 first, as the residual stream and the
// gradient read it, and every output is rounded once.
#include "learner.cuh"

namespace moe {


// Scale byte of a block from its largest magnitude: the smallest power of two
// S with amax / S <= 448 = 0.875 * 2^9, as its exponent + 127.
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  // amax = 2^(e - 127) (1 + f): S = 2^(e - 127 - 8), one more where 1 + f > 1.75
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 0);
}
// 1 / 2^(byte - 127)
__device__ __forceinline__ float mx_scale_inv(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 16 BF16 values of a row chunk in two 16-byte vectors.
struct Chunk {
  uint4 a, b;
  __device__ __forceinline__ void load(const uint16_t* p) {
    a = __ldcs(reinterpret_cast<const uint4*>(p));
    b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void load_kept(const uint16_t* p) {
    a = *reinterpret_cast<const uint4*>(p);
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    __stcs(reinterpret_cast<uint4*>(p), a);
    __stcs(reinterpret_cast<uint4*>(p) + 1, b);
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
    float lo[8], hi[8];
    unpack(a, lo);
    unpack(b, hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = lo[i], x[8 + i] = hi[i];
  }
  __device__ __forceinline__ void set(const float (&x)[16]) {
    const float lo[8] = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
    const float hi[8] = {x[8], x[9], x[10], x[11], x[12], x[13], x[14], x[15]};
    a = pack(lo);
    b = pack(hi);
  }
};

// TPR threads per row, each with up to NV chunks of 16 values, c = k, k + TPR,
// ..; h stays in registers (as BF16) between the sum of squares and the
// outputs, so x and res are read once.  A warp per row needs no barrier; more
// threads per row where rows are few or long.  Two lanes share a block of 32
// values of the 8-bit output, eight a word of four scale bytes, so codes leave
// in 16-byte and scales in 4-byte stores.
// 65536 x 2048: 156 us, 6.9 TB/s, 1.01 of the measured copy rate; 16384 x 2048
// 42 us, with the 8-bit output 47.5 us, 6.4 TB/s, 0.94.
template <int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) add_rmsnorm_kernel(NormArgs a) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR, NW = TPR / 32;
  __shared__ float red[NW];
  begin_kernel();
  const int k = threadIdx.x % TPR, n = a.d / 16;
  const int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  if (TPR == 32 && t >= a.T) return;  // whole warps
  const uint16_t* x = a.x + t * a.ldx;
  Chunk h[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = k + v * TPR;
    if (c < n) h[v].load(x + c * 16);
    else h[v].a = h[v].b = make_uint4(0u, 0u, 0u, 0u);
  }
  if (a.res) {
    const uint16_t* rs = a.res + t * a.ldr;
    Chunk r[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = k + v * TPR;
      if (c < n) r[v].load(rs + c * 16);
      else r[v].a = r[v].b = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float f[16], g[16];
      h[v].get(f);
      r[v].get(g);
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += g[i];
      h[v].set(f);
    }
  }
  float ss[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = k + v * TPR;
    if (a.h && c < n) h[v].store(a.h + t * a.d + c * 16);
    float f[16];
    h[v].get(f);
#pragma unroll
    for (int i = 0; i < 16; ++i) ss[i & 3] = fmaf(f[i], f[i], ss[i & 3]);
  }
  float sum = (ss[0] + ss[1]) + (ss[2] + ss[3]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (NW > 1) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += red[w];
  }
  if (!is_finite_f32(sum)) {  // a non-finite h, or an overflow of its square
    bool bad = false;
#pragma unroll
    for (int v = 0; v < NV; ++v) bad |= absmax_bits16(h[v].a, h[v].b) >= 0x7F80u;
    if (bad) set_status(a.status, MOE_STATUS_NONFINITE_X);
  }
  const float rstd = 1.0f / sqrtf(sum / (float)a.d + a.eps);
  if (k == 0 && a.rstd) a.rstd[t] = rstd;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = k + v * TPR;
    if (c - (int)(threadIdx.x & 31) >= n) break;  // warp-uniform
    const bool in = c < n;
    float y[16], w[16];
    h[v].get(y);
    Chunk wc;
    wc.load_kept(a.w + (in ? c : 0) * 16);
    wc.get(w);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = y[i] * rstd * w[i];
    if (a.y && in) {
      Chunk o;
      o.set(y);
      o.store(a.y + t * a.d + c * 16);
    }
    if (a.y8) {  // d is a multiple of 128: groups of eight lanes are all in or out
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(y[i]));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      const uint32_t sb = mx_scale_byte(m);
      const float inv = mx_scale_inv(sb);
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[i] = e4m3x2_hw(y[4 * i] * inv, y[4 * i + 1] * inv) |
               (e4m3x2_hw(y[4 * i + 2] * inv, y[4 * i + 3] * inv) << 16);
      uint32_t word = sb << (8 * (c >> 1 & 3));
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
      if (in) {
        __stcs(reinterpret_cast<uint4*>(a.y8 + t * a.d + c * 16), make_uint4(q[0], q[1], q[2], q[3]));
        if ((c & 7) == 0) *reinterpret_cast<uint32_t*>(a.sf + sf_tile_offset(t, c >> 1, a.d >> 7)) = word;
      }
    }
  }
}

// nt threads share a row, each with the same 8 * NV columns of every row, so
// that its part of dw stays in registers; a block holds blockDim.x / nt such
// groups.  A group takes R rows at a time (one barrier serves R row sums);
// each thread fetches its own columns of dy, h and dh D groups of
// rows ahead, by asynchronous copies into shared memory that only it reads.
// 65536 x 2048: 161 us, 6.7 TB/s, 0.98 of the measured copy rate (four rows of
// loads in registers and no ring: 194 us, the loads waited out at each barrier).
// GROUPS false: one group.
template <int NV, int R, int D, bool GROUPS>
__global__ void __launch_bounds__(512) add_rmsnorm_backward_kernel(NormBwdArgs a, int nt) {
  extern __shared__ uint4 ring[];  // [D][R][NV][3][blockDim.x]
  __shared__ float red[2][R][16];
  begin_kernel();
  const int n = a.d / 8, nb = blockDim.x, groups = GROUPS ? nb / nt : 1;
  const int group = GROUPS ? threadIdx.x / nt : 0, k = threadIdx.x - group * nt;
  const int lane = threadIdx.x & 31, nw = nt >> 5, warp0 = group * nw;  // the group's warps
  float dw[NV][8], w[NV][8];
  // largest magnitude of the thread's dx: any input that is no finite number
  // leaves one in its row (dh in its place)
  uint32_t big = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = k + v * nt;
    const uint4 wv = c < n ? reinterpret_cast<const uint4*>(a.w)[c] : make_uint4(0u, 0u, 0u, 0u);
    unpack(wv, w[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
  }
  const float inv_d = 1.0f / (float)a.d;
  const int64_t step = (int64_t)gridDim.x * groups * R;
  auto slot = [&](int g, int q, int v) { return ring + ((g * R + q) * NV + v) * 3 * nb + threadIdx.x; };
  float rnext[R];
  auto fetch = [&](int64_t t0, int g) {  // the R rows from t0 into group g of the ring
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const bool row = t0 + q < a.T;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = k + v * nt;
        const bool in = row && c < n;
        const int64_t at = in ? ((t0 + q) * n + c) * 8 : 0;
        uint4* s = slot(g, q, v);
        cp_async16(smem_u32(s), a.dy + at, in);
        cp_async16(smem_u32(s + nb), a.h + at, in);
        if (a.dh) cp_async16(smem_u32(s + 2 * nb), a.dh + at, in);
      }
    }
    cp_async_commit();
  };
  auto rstds = [&](int64_t t0) {
#pragma unroll
    for (int q = 0; q < R; ++q) rnext[q] = t0 + q < a.T ? a.rstd[t0 + q] : 0.0f;
  };
  const int64_t first = ((int64_t)blockIdx.x * groups + group) * R;
#pragma unroll
  for (int g = 0; g < D; ++g) fetch(first + g * step, g);
  rstds(first);
  int odd = 0, g = 0;
  for (int64_t t0 = first; t0 < a.T; t0 += step, odd ^= 1) {
    float r[R], sum[R];
#pragma unroll
    for (int q = 0; q < R; ++q) r[q] = rnext[q];
    rstds(t0 + step);
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    uint4 dy[R][NV], h[R][NV];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const uint4* p = slot(g, q, v);
        dy[q][v] = p[0];
        h[q][v] = p[nb];
        float y[8], x[8];
        unpack(dy[q][v], y);
        unpack(h[q][v], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float m = y[i] * (x[i] * r[q]);
          dw[v][i] += m;
          s[i & 1] = fmaf(m, w[v][i], s[i & 1]);
        }
      }
      sum[q] = s[0] + s[1];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int q = 0; q < R; ++q) sum[q] += __shfl_xor_sync(0xFFFFFFFFu, sum[q], o);
    if (nw > 1) {
      if (lane == 0)
#pragma unroll
        for (int q = 0; q < R; ++q) red[odd][q][threadIdx.x >> 5] = sum[q];
      if (GROUPS) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(nt) : "memory");
      else __syncthreads();
#pragma unroll
      for (int q = 0; q < R; ++q) {
        sum[q] = lane < nw ? red[odd][q][warp0 + lane] : 0.0f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum[q] += __shfl_xor_sync(0xFFFFFFFFu, sum[q], o);
      }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t t = t0 + q;
      const float c1 = __shfl_sync(0xFFFFFFFFu, sum[q], 0) * inv_d * r[q];
      if (t < a.T) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = k + v * nt;
          float y[8], x[8], o[8];
          unpack(dy[q][v], y);
          unpack(h[q][v], x);
          if (a.dh) unpack(slot(g, q, v)[2 * nb], o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float m = r[q] * (y[i] * w[v][i] - x[i] * c1);
            o[i] = a.dh ? o[i] + m : m;
          }
          if (c < n) {
            const uint4 p = pack(o);
            __stcs(reinterpret_cast<uint4*>(a.dx) + t * n + c, p);
            big = max_abs_nan_bf16x2(max_abs_nan_bf16x2(big, p.x), p.y);
            big = max_abs_nan_bf16x2(max_abs_nan_bf16x2(big, p.z), p.w);
          }
        }
      }
    }
    fetch(t0 + D * step, g);  // into the slots just read
    g = g + 1 == D ? 0 : g + 1;
  }
  if (!bf16x2_finite(big)) set_status(a.status, MOE_STATUS_NONFINITE_X);
  if (!a.dw) return;
  // the groups' parts of dw, added in order, make the block's
  if constexpr (GROUPS) {
    float* sum = reinterpret_cast<float*>(ring);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k < n) sum[(group * n + k) * 8 + i] = dw[0][i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += nb) {
      float s = sum[c];
      for (int g2 = 1; g2 < groups; ++g2) s += sum[g2 * a.d + c];
      a.part[(int64_t)blockIdx.x * a.d + c] = s;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = k + v * nt;
      if (c < n) {
        float4* p = reinterpret_cast<float4*>(a.part + (int64_t)blockIdx.x * a.d + c * 8);
        p[0] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
        p[1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
      }
    }
  }
}

// dw from the blocks' parts: 32 columns per block, the parts in 32 slices that
// meet in shared memory; always the same order.
__global__ void __launch_bounds__(1024) add_rmsnorm_dw_kernel(const float* part, int nb, int d, float* dw) {
  __shared__ float sh[32][33];
  begin_kernel();
  const int i = blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  if (i < d)
#pragma unroll 8
    for (int b = threadIdx.y; b < nb; b += 32) s += part[(int64_t)b * d + i];
  sh[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = sh[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < d) dw[blockIdx.x * 32 + threadIdx.y] = s;
}

// host launchers
template <int TPR, int NV>
static int launch_norm(const NormArgs& a, cudaStream_t s) {
  constexpr int rows = TPR < 128 ? 128 / TPR : 1;
  const unsigned blocks = ((unsigned)a.T + rows - 1) / rows;  // T may be the largest int
  return launch_kernel(add_rmsnorm_kernel<TPR, NV>, dim3(blocks), TPR < 128 ? 128 : TPR, 0, 1, s, a);
}
int launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  const int n = a.d / 16;  // chunks
  if (n <= 32) return launch_norm<32, 1>(a, s);
  if (n <= 64 && a.T >= 1024) return launch_norm<32, 2>(a, s);
  if (n <= 128 && a.T >= 1024) return launch_norm<32, 4>(a, s);
  if (n <= 128) return launch_norm<128, 1>(a, s);
  if (n <= 256) return launch_norm<128, 2>(a, s);
  if (n <= 512) return launch_norm<256, 2>(a, s);
  return launch_norm<512, 2>(a, s);
}

// The backward's launch for a size: threads per row, groups of threads per
// block, rows a group takes at a time, groups of rows in flight, blocks, shared
// memory of the launch and of the largest launch of the same kernel.
struct NormBwdPlan {
  int nv, depth, threads, groups, blocks, smem, smem_most;
};
static NormBwdPlan norm_bwd_plan(int T, int d) {
  NormBwdPlan p;
  const int n = d / 8;
  p.nv = d <= 4096 ? 1 : d <= 8192 ? 2 : 4;
  const int rows = p.nv == 1 ? 2 : 1;
  p.depth = d > 1024 && d <= 2048 ? 3 : 2;
  p.threads = ((n + p.nv - 1) / p.nv + 31) / 32 * 32;
  p.groups = p.threads <= 128 ? 256 / p.threads : 1;
  const int nb = p.threads * p.groups;
  p.smem = nb * p.nv * 3 * 16 * rows * p.depth;
  p.smem_most = (p.groups > 1 || p.depth == 3 ? 256 : 512) * p.nv * 3 * 16 * rows * p.depth;
  const int fit = 220 * 1024 / (p.smem + 2048), cap = 1536 / nb;
  const int per = fit < cap ? (fit < 1 ? 1 : fit) : cap;
  const int64_t all = ((int64_t)T + rows * p.groups - 1) / (rows * p.groups);
  p.blocks = 152 * per < all ? 152 * per : (int)all;
  return p;
}
size_t add_rmsnorm_backward_ws(int T, int d) { return (size_t)norm_bwd_plan(T, d).blocks * d * 4; }

int launch_add_rmsnorm_backward(const NormBwdArgs& a, cudaStream_t s) {
  const NormBwdPlan p = norm_bwd_plan(a.T, a.d);
  auto f = p.nv == 4      ? add_rmsnorm_backward_kernel<4, 1, 2, false>
           : p.nv == 2    ? add_rmsnorm_backward_kernel<2, 1, 2, false>
           : p.groups > 1 ? add_rmsnorm_backward_kernel<1, 2, 2, true>
           : p.depth == 3 ? add_rmsnorm_backward_kernel<1, 2, 3, false>
                          : add_rmsnorm_backward_kernel<1, 2, 2, false>;
  if (!allow_smem((const void*)f, p.smem, p.smem_most)) return -1;
  if (launch_kernel(f, dim3((unsigned)p.blocks), p.threads * p.groups, p.smem, 1, s, a, p.threads) != 0) return -1;
  if (!a.dw) return 0;
  return launch_kernel(add_rmsnorm_dw_kernel, dim3((unsigned)((a.d + 31) / 32)), dim3(32, 32), 0, 1, s, a.part, p.blocks,
                       a.d, a.dw);
}

}  // namespace moe
