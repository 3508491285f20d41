// Layer norm over the rows of [M, D], forward and backward.
//
//   mean = sum_j x_j / D,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / D + eps),
//   y_j = (x_j - mean) rstd gamma_j + beta_j.
// With xh = (x - mean) rstd and w = gamma dy:
//   dx = rstd (w - mean_j(w) - xh mean_j(w xh)),
//   dgamma_j = sum_rows dy xh,  dbeta_j = sum_rows dy.
//
// Both are bound by DRAM: the forward reads x and writes y once, the backward
// reads x and dy and writes dx once.  A row is held in registers between its
// statistics and its result, so nothing is read twice, and the variance is
// the mean of squared differences from the mean (no cancellation).  A row far
// from zero loses its offset's low bits in the first sum: the differences are
// summed along with their squares, and what their mean d differs from zero is
// taken off the result too (x - mean - d, variance sum d_j^2 / D - d^2).
// Sums are fp32 in a fixed order.
#include <stdio.h>

#include <algorithm>

#include "common.cuh"
#include "f32x2.cuh"
#include "ops.h"

namespace mlpk {

namespace {

constexpr int kSMs = 152;
constexpr int kMaxRow = 8192;          // the widest row held in registers
constexpr int64_t kMaxD = 65535 * 256; // the widest row taken (column blocks of the backward are a grid's y)

// VEC consecutive elements as fp32 (one 16-byte access, or one element).
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* src, float* v) {
  if constexpr (VEC == 1) {
    v[0] = to_f32(src[0]);
  } else if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(src);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(src);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      v[2 * h] = __uint_as_float(w[h] << 16);
      v[2 * h + 1] = __uint_as_float(w[h] & 0xFFFF0000u);
    }
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* dst, const float* v) {
  if constexpr (VEC == 1) {
    dst[0] = from_f32<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * h], v[2 * h + 1]);
      w[h] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

struct LnFwdParams {
  const void* x; int64_t ldx;
  const float* gamma; const float* beta;
  void* y; int64_t ldy;
  float* mean; float* rstd;
  int64_t M; int D;
  float eps;
  int tpr;              // threads per row (a multiple of 32 that divides the block)
};

// Sums of NS values over the WARPS warps that share a row, the same in every
// thread; each call of a kernel has its own sh.
template <int WARPS, int NS>
__device__ __forceinline__ void row_sums(float (&v)[NS], float (&sh)[NS][WARPS]) {
#pragma unroll
  for (int k = 0; k < NS; ++k) v[k] = warp_sum(v[k]);
  if constexpr (WARPS > 1) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < NS; ++k) sh[k][threadIdx.x >> 5] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v[k] += sh[k][w];
    }
  }
}
// What the sums of differences from a row's first mean say: the rest of the
// mean and 1 / sqrt(variance + eps).  The variance is kept from falling below
// zero by a comparison that NaN fails (fmaxf would turn it into 0): a row that
// holds NaN or an infinity has rstd NaN.
__device__ __forceinline__ void finish_stats(const float (&s)[2], float inv_d, float eps, float& rest, float& rstd) {
  rest = s[0] * inv_d;
  const float var = fmaf(-rest, rest, s[1] * inv_d);
  rstd = rsqrtf((var < 0.f ? 0.f : var) + eps);   // (2 ulp)
}

// How rows of at most kMaxRow elements are walked, forward and backward: tpr
// threads (whole warps) share a row, EPT elements each, and a block's groups of
// tpr threads take rows in turn, so that the gradients' columns stay with
// their threads.  Rows are prefetched into a ring in shared memory (cp.async, 16
// bytes at a time where they are aligned, else 4), each thread only its own
// elements, so a thread waits for no other; bf16 rows that start between two
// words are loaded when their turn comes.  (bf16 21746 x 3086, whose rows are
// 4-byte aligned: forward 136 us loaded so, 89 through the ring, backward 237
// and 116.)  The scale and the shift lie in shared memory.
//   EPT: with 8 elements a thread the kernels were bound by instruction issue
// (about 250 instructions a row and warp besides the elements: 94 us for the
// forward of 65536 x 1024 bf16); more elements share that.  The forward takes
// 32 of bf16 (47 us); the backward, whose 2 EPT column sums stay in registers,
// and fp32 and unaligned rows take 16 (backward of the same: 73 us; with 32
// the sums spill, 142 us); short rows 8.
template <bool FWD> struct RowCfg {   // one block to an SM
  static constexpr int THREADS = FWD ? 1024 : 512;   // at most (64 and 128 registers)
  static constexpr int RING = FWD ? 192 : 384;       // bytes of the ring per thread
};

template <typename T, int VEC, int EPT, int NT, bool FULL>   // NT tensors a row: x, or x and dy; FULL: no thread's elements end early
struct RowFetch {
  static constexpr int NV = EPT / VEC;
  static constexpr int CB = VEC * (int)sizeof(T);   // bytes of a unit
  static constexpr bool RING = CB >= 4;
  static constexpr int FIT = RowCfg<NT == 1>::RING / (EPT * (int)sizeof(T) * NT);
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static_assert(!RING || STAGES >= 2, "a row ahead at least");
  const T* src[NT];      // the tensors, at this thread's first element
  int64_t ld[NT];
  int64_t M, step;       // rows, rows from one to the next
  int cols;              // elements from this thread's first one to D
  int hop;               // elements from unit to unit
  uint32_t ring;         // this thread's place of unit 0 of stage 0
  uint32_t pitch;        // bytes from unit to unit
  uint32_t raw[NT][RING ? NV : 1][RING ? CB / 4 : 1];
  T one[NT][RING ? 1 : NV];

  __device__ __forceinline__ void setup(int t, int tpr, int D, uint32_t ring0) {
    cols = D - t * VEC;
    hop = tpr * VEC;
    ring = ring0 + threadIdx.x * CB;
    pitch = blockDim.x * CB;
#pragma unroll
    for (int k = 0; k < NT; ++k) src[k] += t * VEC;
  }
  // (tpr is the least multiple of 32 with tpr EPT >= D: with more than 8
  // elements a thread the first half of its units is always there)
  __device__ __forceinline__ bool in(int i) const { return FULL || (EPT > 8 && i < NV / 2) || i * hop < cols; }
  __device__ __forceinline__ void issue(int64_t row, int stage) {
    if constexpr (RING) {
      if (row < M) {
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          const T* r = src[k] + row * ld[k];
          const uint32_t to = ring + (uint32_t)(stage * NT + k) * NV * pitch;
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (in(i)) {
              if constexpr (CB == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + (uint32_t)i * pitch), "l"(r + i * hop)
                             : "memory");
              else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + (uint32_t)i * pitch), "l"(r + i * hop)
                             : "memory");
            }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  __device__ __forceinline__ static void clear(uint32_t at) {
    if constexpr (CB == 16)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0u) : "memory");
    else
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(0u) : "memory");
  }
  // The first rows' fetches.  Units that are not there are zeros in every
  // stage: the sums run over them without a branch (bf16 16384 x 1000,
  // forward: 16.7 us with branches, 15.5 without).
  template <int AHEAD>   // rows that are fetched before their turn
  __device__ __forceinline__ void start(int64_t row) {
    if constexpr (RING) {
      if constexpr (!FULL)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (!in(i))
            for (int s = 0; s < STAGES * NT; ++s) clear(ring + (uint32_t)(s * NV + i) * pitch);
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) issue(row + s * step, s);
    }
  }
  // A stage's elements into raw.
  __device__ __forceinline__ void read(int stage) {
    if constexpr (RING) {
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const uint32_t at = ring + (uint32_t)((stage * NT + k) * NV + i) * pitch;
          if constexpr (CB == 16)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(raw[k][i][0]), "=r"(raw[k][i][1]), "=r"(raw[k][i][2]), "=r"(raw[k][i][3])
                         : "r"(at)
                         : "memory");
          else
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(raw[k][i][0]) : "r"(at) : "memory");
        }
    }
  }
  // Row `row`'s elements into raw (stage by stage), the next fetch under way.
  template <int AHEAD>
  __device__ __forceinline__ void take(int64_t row, int& stage) {
    if constexpr (RING) {
      asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
      read(stage);
      // into a stage whose row has been read for the last time: the row before's
      // (AHEAD = STAGES - 1), or that of the one before it
      issue(row + AHEAD * step, stage + AHEAD >= STAGES ? stage + AHEAD - STAGES : stage + AHEAD);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) one[k][i] = in(i) ? src[k][row * ld[k] + i * hop] : from_f32<T>(0.f);
    }
  }
  // Elements 2 q and 2 q + 1 of this thread, zeros beyond D.
  __device__ __forceinline__ F2 get(int k, int q) const {
    if constexpr (!RING) {
      return pack2(to_f32(one[k][2 * q]), to_f32(one[k][2 * q + 1]));
    } else if constexpr (VEC == 1) {
      return pack2(__uint_as_float(raw[k][2 * q][0]), __uint_as_float(raw[k][2 * q + 1][0]));
    } else if constexpr (sizeof(T) == 4) {
      return pack2(__uint_as_float(raw[k][q / 2][2 * (q & 1)]), __uint_as_float(raw[k][q / 2][2 * (q & 1) + 1]));
    } else {
      const uint32_t w = raw[k][2 * q / VEC][VEC == 2 ? 0 : q & 3];
      return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
  }
  // v for pair q's elements, zeros beyond D.
  __device__ __forceinline__ F2 only(int q, float v) const {
    return pack2(has(q) ? v : 0.f, in((2 * q + 1) / VEC) ? v : 0.f);
  }
  // Whether pair q is there at all, and the row's elements it holds: offsets
  // from this thread's first one.
  __device__ __forceinline__ bool has(int q) const { return in(2 * q / VEC); }
  __device__ __forceinline__ int at(int q) const { return 2 * q / VEC * hop + (VEC == 1 ? 0 : 2 * q % VEC); }
  // A vector of D floats (and zeros up to tpr EPT) in shared memory, in the order the threads use it:
  // four consecutive elements of thread t at 16 t, so that a warp's 16-byte
  // loads run through it (in memory order, lanes 32 bytes apart conflicted
  // four ways: 52 us for the forward of 65536 x 1024).
  __device__ __forceinline__ static int place(int c, int tpr) {   // of element c
    if constexpr (VEC == 8) {
      const int unit = c >> 3, i = unit / tpr, t = unit - i * tpr;
      return ((2 * i + ((c >> 2) & 1)) * tpr + t) * 4 + (c & 3);
    } else {
      return c;
    }
  }
  // Pairs q and q + 1 (q even) of such a vector, v at this thread's first element.
  __device__ __forceinline__ void vec4(const float* v, int q, F2& a, F2& b) const {
    if constexpr (VEC >= 4) {
      const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(v + (2 * q / 4) * (hop / VEC) * 4);
      a.v = w.x;
      b.v = w.y;
    } else if constexpr (VEC == 2) {
      a.v = *reinterpret_cast<const uint64_t*>(v + at(q));
      b.v = *reinterpret_cast<const uint64_t*>(v + at(q + 1));
    } else {
      a = pack2(v[at(q)], v[at(q) + hop]);
      b = pack2(v[at(q + 1)], v[at(q + 1) + hop]);
    }
  }
};
// A thread's results to its elements of a row, a unit (of less than 16 bytes:
// two pairs) at a time: get(q, a, b) gives pairs q and q + 1.
template <typename T, int VEC, int EPT, class F, class Get>
__device__ __forceinline__ void put_row(const F& f, T* row, Get get) {
  constexpr int PAIRS = VEC <= 4 ? 2 : VEC / 2;
#pragma unroll
  for (int q = 0; q < EPT / 2; q += PAIRS) {
    if (!f.has(q)) continue;
    float v[2 * PAIRS];
#pragma unroll
    for (int h = 0; h < PAIRS; h += 2) {
      F2 a, b;
      get(q + h, a, b);
      unpack2(a, v[2 * h], v[2 * h + 1]);
      unpack2(b, v[2 * h + 2], v[2 * h + 3]);
    }
    if constexpr (VEC == 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (f.in(2 * q + j)) row[(2 * q + j) * f.hop] = from_f32<T>(v[j]);
    } else if constexpr (VEC == 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (f.has(q + j)) *reinterpret_cast<__nv_bfloat162*>(row + f.at(q + j)) = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    } else {
      store_vec<T, VEC>(row + f.at(q), v);
    }
  }
}

// Sums of NS values over the warps of a row's group, the same in every thread
// of it.  w: the block's [32 * NS] floats of one of two buffers used in turn
// (a group's next use of the same buffer lies two barriers later).
template <int NS>
__device__ __forceinline__ void post_sums(float (&v)[NS], float* w, int wpr) {
#pragma unroll
  for (int k = 0; k < NS; ++k) v[k] = warp_sum(v[k]);
  if (wpr > 1 && (threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < NS; ++k) w[NS * (threadIdx.x >> 5) + k] = v[k];
}
template <int NS>
__device__ __forceinline__ void read_sums(float (&v)[NS], const float* w, int group, int wpr) {   // (one warp: v as posted)
  if (wpr == 1) return;
#pragma unroll
  for (int k = 0; k < NS; ++k) v[k] = 0.f;
  for (int i = 0; i < wpr; ++i)
#pragma unroll
    for (int k = 0; k < NS; ++k) v[k] += w[NS * (group * wpr + i) + k];
}
template <int NS>
__device__ __forceinline__ void group_sums(float (&v)[NS], float* w, int group, int wpr) {
  post_sums<NS>(v, w, wpr);
  if (wpr > 1) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(wpr * 32) : "memory");
  read_sums<NS>(v, w, group, wpr);
}

constexpr int kSumBytes = 2 * 32 * 2 * 4;   // group_sums' two buffers

template <typename T, int VEC, int EPT, bool FULL>
__global__ void __launch_bounds__(RowCfg<true>::THREADS, 1) ln_fwd_kernel(const __grid_constant__ LnFwdParams p) {
  pdl_enter();
  using F = RowFetch<T, VEC, EPT, 1, FULL>;
  constexpr int NP = EPT / 2;
  extern __shared__ __align__(16) float ln_smem[];
  const int tpr = p.tpr, groups = (int)blockDim.x / tpr, wpr = tpr >> 5;
  float* scale = ln_smem + kSumBytes / 4;          // [tpr EPT]
  float* shift = scale + tpr * EPT;
  const int group = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
  F f;
  f.src[0] = reinterpret_cast<const T*>(p.x);
  f.ld[0] = p.ldx;
  f.M = p.M; f.step = (int64_t)gridDim.x * groups;
  f.setup(t, tpr, p.D, (uint32_t)__cvta_generic_to_shared(shift + tpr * EPT));
  int64_t row = blockIdx.x * (int64_t)groups + group;
  f.template start<F::STAGES - 1>(row);
  for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
    scale[F::place(c, tpr)] = p.gamma ? p.gamma[c] : 1.f;
    shift[F::place(c, tpr)] = p.beta ? p.beta[c] : 0.f;
  }
  if constexpr (!FULL)
    for (int c = p.D + threadIdx.x; c < tpr * EPT; c += blockDim.x) scale[F::place(c, tpr)] = shift[F::place(c, tpr)] = 0.f;
  __syncthreads();
  const float inv_d = 1.0f / (float)p.D;
  const int my = t * (VEC < 4 ? VEC : 4);   // this thread's first place in them
  int stage = 0;
  for (; row < p.M; row += f.step) {
    f.template take<F::STAGES - 1>(row, stage);
    F2 v[NP], a = pack2(0.f, 0.f), b = a;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      v[q] = f.get(0, q);
      a = add2(a, v[q]);
    }
    float s[1] = {sum2(a)}, sd[2];
    group_sums<1>(s, ln_smem, group, wpr);
    const float mean = s[0] * inv_d;
    a = b;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      v[q] = add2(v[q], f.only(q, -mean));
      a = add2(a, v[q]);
      b = fma2(v[q], v[q], b);
    }
    sd[0] = sum2(a);
    sd[1] = sum2(b);
    group_sums<2>(sd, ln_smem + 64, group, wpr);
    float rest, rstd;
    finish_stats(sd, inv_d, p.eps, rest, rstd);
    if (t == 0) {
      if (p.mean) p.mean[row] = mean + rest;
      if (p.rstd) p.rstd[row] = rstd;
    }
    const F2 less = pack2(-rest, -rest), times = pack2(rstd, rstd);
    put_row<T, VEC, EPT>(f, reinterpret_cast<T*>(p.y) + row * p.ldy + t * VEC, [&](int q, F2& y0, F2& y1) {
      F2 g0, g1, b0, b1;
      f.vec4(scale + my, q, g0, g1);
      f.vec4(shift + my, q, b0, b1);
      y0 = fma2(mul2(add2(v[q], less), times), g0, b0);
      y1 = fma2(mul2(add2(v[q + 1], less), times), g1, b1);
    });
  }
}

// Rows wider than kMaxRow: a block per row, three passes (the second and
// third from L2).
template <typename T>
__global__ void __launch_bounds__(1024) ln_fwd_wide_kernel(const __grid_constant__ LnFwdParams p) {
  pdl_enter();
  __shared__ float sh1[1][32], sh2[2][32];
  const int64_t row = blockIdx.x;
  const T* xr = reinterpret_cast<const T*>(p.x) + row * p.ldx;
  float s[1] = {0.f}, sd[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < p.D; c += 1024) s[0] += to_f32(xr[c]);
  const float inv_d = 1.0f / (float)p.D;
  row_sums<32, 1>(s, sh1);
  const float mean = s[0] * inv_d;
  for (int c = threadIdx.x; c < p.D; c += 1024) {
    const float d = to_f32(xr[c]) - mean;
    sd[0] += d;
    sd[1] = fmaf(d, d, sd[1]);
  }
  row_sums<32, 2>(sd, sh2);
  float rest, rstd;
  finish_stats(sd, inv_d, p.eps, rest, rstd);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean + rest;
    if (p.rstd) p.rstd[row] = rstd;
  }
  T* yr = reinterpret_cast<T*>(p.y) + row * p.ldy;
  for (int c = threadIdx.x; c < p.D; c += 1024) {
    const float g = p.gamma ? p.gamma[c] : 1.f, b = p.beta ? p.beta[c] : 0.f;
    yr[c] = from_f32<T>(fmaf((to_f32(xr[c]) - mean - rest) * rstd, g, b));
  }
}

struct LnBwdParams {
  const void* dy; int64_t lddy;
  const void* x; int64_t ldx;
  const float* gamma;
  const float* mean; const float* rstd;
  void* dx; int64_t lddx;
  float* part;          // [gridDim.x][2][D] partial dgamma, dbeta (null: not wanted)
  int64_t M; int D;
  int tpr;              // threads per row (a multiple of 32 that divides the block)
};

// The groups keep their columns' dgamma / dbeta sums in registers and add them
// over the block at the end: one partial row pair per block.  x and dy stay
// packed between the two uses of a row.
template <typename T, int VEC, int EPT, bool FULL>
__global__ void __launch_bounds__(RowCfg<false>::THREADS, 1) ln_bwd_kernel(const __grid_constant__ LnBwdParams p) {
  pdl_enter();
  using F = RowFetch<T, VEC, EPT, 2, FULL>;
  constexpr int NP = EPT / 2;
  constexpr bool DEFER = VEC == 8 && EPT == 16 && !FULL;
  constexpr int AHEAD = DEFER ? F::STAGES - 2 : F::STAGES - 1;
  extern __shared__ __align__(16) float ln_smem[];
  const int tpr = p.tpr, groups = (int)blockDim.x / tpr, wpr = tpr >> 5;
  float* scale = ln_smem + kSumBytes / 4;                 // [tpr EPT]
  float* colsum = scale + tpr * EPT;                      // the ring's place, once the rows are done
  const int group = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
  F f;
  f.src[0] = reinterpret_cast<const T*>(p.x);
  f.src[1] = reinterpret_cast<const T*>(p.dy);
  f.ld[0] = p.ldx; f.ld[1] = p.lddy;
  f.M = p.M; f.step = (int64_t)gridDim.x * groups;
  f.setup(t, tpr, p.D, (uint32_t)__cvta_generic_to_shared(colsum));
  int64_t row = blockIdx.x * (int64_t)groups + group;
  f.template start<AHEAD>(row);
  for (int c = threadIdx.x; c < p.D; c += blockDim.x) scale[F::place(c, tpr)] = p.gamma ? p.gamma[c] : 1.f;
  if constexpr (!FULL)
    for (int c = p.D + threadIdx.x; c < tpr * EPT; c += blockDim.x) scale[F::place(c, tpr)] = 0.f;
  const float inv_d = 1.0f / (float)p.D;
  const F2 zero = pack2(0.f, 0.f);
  F2 dg[NP], db[NP];
#pragma unroll
  for (int q = 0; q < NP; ++q) dg[q] = db[q] = zero;
  float mean = 0.f, rstd = 0.f;
  if (row < p.M) { mean = p.mean[row]; rstd = p.rstd[row]; }
  __syncthreads();
  const float* sc = scale + t * (VEC < 4 ? VEC : 4);
  // a row's two sums (this warp's share of them), the columns' sums on the way
  auto row_sums = [&](float (&s)[2]) {
    const F2 times = pack2(rstd, rstd);
    F2 a = zero, b = zero;
#pragma unroll
    for (int q0 = 0; q0 < NP; q0 += 2) {
      F2 g[2];
      f.vec4(sc, q0, g[0], g[1]);
#pragma unroll
      for (int q = q0; q < q0 + 2; ++q) {
        const F2 d = f.get(1, q), xh = mul2(add2(f.get(0, q), f.only(q, -mean)), times), w = mul2(d, g[q - q0]);
        dg[q] = fma2(d, xh, dg[q]);
        db[q] = add2(db[q], d);
        a = add2(a, w);
        b = fma2(w, xh, b);
      }
    }
    s[0] = sum2(a);
    s[1] = sum2(b);
  };
  auto put = [&](int64_t to, float mean, float rstd, const float (&s)[2]) {
    // rstd (w - c1 - xh c2), the last factor over all of it: rstd^2 would leave
    // fp32 where rstd does not (rows below 5e-20)
    const float c1 = -s[0] * inv_d, c2 = -s[1] * inv_d * rstd;
    const F2 times = pack2(rstd, rstd), minus = pack2(-mean, -mean), p1 = pack2(c1, c1), p2 = pack2(c2, c2);
    put_row<T, VEC, EPT>(f, reinterpret_cast<T*>(p.dx) + to * p.lddx + t * VEC, [&](int q, F2& o0, F2& o1) {
      F2 g0, g1;
      f.vec4(sc, q, g0, g1);
      o0 = mul2(fma2(add2(f.get(0, q), minus), p2, fma2(f.get(1, q), g0, p1)), times);
      o1 = mul2(fma2(add2(f.get(0, q + 1), minus), p2, fma2(f.get(1, q + 1), g1, p1)), times);
    });
  };
  int stage = 0, buf = 0;
  if constexpr (DEFER) {
    // a row's results a turn after its sums, so that no warp waits for the
    // others' with nothing to do; the row is read a second time from its stage,
    // which makes room for the column tests' registers (bf16 11503 x 5520: 146 us
    // at once, 106 so; 16384 x 1000: 31 and 27; full rows 16384 x 4096: 79 and 83,
    // rows in 4-byte units 21746 x 3086: 116 and 129)
    int64_t last = -1;
    float last_mean = 0.f, last_rstd = 0.f, s[2], last_s[2] = {0.f, 0.f};
    int last_stage = 0;
    for (; row < p.M; row += f.step) {
      float next_mean = 0.f, next_rstd = 0.f;
      if (row + f.step < p.M) { next_mean = p.mean[row + f.step]; next_rstd = p.rstd[row + f.step]; }
      const int at = stage;
      f.template take<AHEAD>(row, stage);
      row_sums(s);
      post_sums<2>(s, ln_smem + 64 * buf, wpr);
      if (last >= 0) {
        f.read(last_stage);
        read_sums<2>(last_s, ln_smem + 64 * (buf ^ 1), group, wpr);
        put(last, last_mean, last_rstd, last_s);
      }
      if (wpr > 1) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(wpr * 32) : "memory");
      last = row;
      last_mean = mean; last_rstd = rstd;
      last_s[0] = s[0]; last_s[1] = s[1];
      last_stage = at;
      buf ^= 1;
      mean = next_mean;
      rstd = next_rstd;
    }
    if (last >= 0) {
      f.read(last_stage);
      read_sums<2>(last_s, ln_smem + 64 * (buf ^ 1), group, wpr);
      put(last, last_mean, last_rstd, last_s);
    }
  } else {
    for (; row < p.M; row += f.step) {
      float next_mean = 0.f, next_rstd = 0.f;
      if (row + f.step < p.M) { next_mean = p.mean[row + f.step]; next_rstd = p.rstd[row + f.step]; }
      f.template take<AHEAD>(row, stage);
      float s[2];
      row_sums(s);
      group_sums<2>(s, ln_smem + 64 * buf, group, wpr);
      buf ^= 1;
      put(row, mean, rstd, s);
      mean = next_mean;
      rstd = next_rstd;
    }
  }
  if (!p.part) return;
  // every group's column sums, added in the groups' order
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float* mine = colsum + (int64_t)group * 2 * p.D + t * VEC;
#pragma unroll
  for (int q = 0; q < NP; ++q) {
    if (!f.has(q)) continue;
    const int c = f.at(q), second = VEC == 1 ? f.hop : 1;
    float x, y;
    unpack2(dg[q], x, y);
    mine[c] = x;
    if (VEC > 1 || f.in(2 * q + 1)) mine[c + second] = y;
    unpack2(db[q], x, y);
    mine[p.D + c] = x;
    if (VEC > 1 || f.in(2 * q + 1)) mine[p.D + c + second] = y;
  }
  __syncthreads();
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.D;
  for (int c = threadIdx.x; c < 2 * p.D; c += blockDim.x) {
    float sum = 0.f;
    for (int k = 0; k < groups; ++k) sum += colsum[(int64_t)k * 2 * p.D + c];
    out[c] = sum;
  }
}

// Rows wider than kMaxRow.  dx: a block per row, two passes.
template <typename T>
__global__ void __launch_bounds__(1024) ln_bwd_wide_kernel(const __grid_constant__ LnBwdParams p) {
  pdl_enter();
  __shared__ float sh[2][32];
  const int64_t row = blockIdx.x;
  const T* xr = reinterpret_cast<const T*>(p.x) + row * p.ldx;
  const T* dr = reinterpret_cast<const T*>(p.dy) + row * p.lddy;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float s[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < p.D; c += 1024) {
    const float w = to_f32(dr[c]) * (p.gamma ? p.gamma[c] : 1.f);
    s[0] += w;
    s[1] = fmaf(w, (to_f32(xr[c]) - mean) * rstd, s[1]);
  }
  const float inv_d = 1.0f / (float)p.D;
  row_sums<32, 2>(s, sh);
  const float c1 = s[0] * inv_d, c2 = s[1] * inv_d;
  T* or_ = reinterpret_cast<T*>(p.dx) + row * p.lddx;
  for (int c = threadIdx.x; c < p.D; c += 1024) {
    const float w = to_f32(dr[c]) * (p.gamma ? p.gamma[c] : 1.f);
    or_[c] = from_f32<T>(rstd * (w - c1 - (to_f32(xr[c]) - mean) * rstd * c2));
  }
}
// dgamma / dbeta of wide rows: a thread per column, the rows cut into
// gridDim.x chunks (run before the dx kernel, which may overwrite dy).
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_wide_cols_kernel(const __grid_constant__ LnBwdParams p) {
  pdl_enter();
  const int64_t c = blockIdx.y * (int64_t)256 + threadIdx.x;
  if (c >= p.D) return;
  float dg = 0.f, db = 0.f;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const float d = to_f32(reinterpret_cast<const T*>(p.dy)[row * p.lddy + c]);
    const float x = to_f32(reinterpret_cast<const T*>(p.x)[row * p.ldx + c]);
    dg = fmaf(d, (x - p.mean[row]) * p.rstd[row], dg);
    db += d;
  }
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.D;
  out[c] = dg;
  out[p.D + c] = db;
}

// dgamma and dbeta from the blocks' partial rows: 32 columns per block, 32
// warps that each add every 32nd partial, then the 32 sums in order.
struct LnReduceParams {
  const float* part; int parts; int D;
  float* dgamma; float* dbeta;
};
__global__ void __launch_bounds__(1024) ln_param_reduce_kernel(const __grid_constant__ LnReduceParams p) {
  pdl_enter();
  __shared__ float sh[32][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * (int64_t)32 + lane, n = 2 * (int64_t)p.D;
  float s = 0.f;
  if (c < n) {
#pragma unroll 4
    for (int k = w; k < p.parts; k += 32) s += p.part[k * n + c];
  }
  sh[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < n) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += sh[k][lane];
    if (c < p.D) {
      if (p.dgamma) p.dgamma[c] = s;
    } else if (p.dbeta) {
      p.dbeta[c - p.D] = s;
    }
  }
}

// The elements that move at once: 16 bytes of them, 4 bytes, or (bf16 between
// words) one.  bits: the row length, the pitches and the bases in bytes, or'ed.
int unit_of(bool f32, uint64_t bits) {
  const int es = f32 ? 4 : 2;
  return (bits & 15) == 0 ? 16 / es : (bits & 3) == 0 ? 4 / es : 1;
}

// How a block walks rows of D elements: elements per thread, threads per row,
// block and grid.
struct RowShape { int ept, tpr, threads; int64_t blocks; };
template <bool FWD>
RowShape row_shape(bool f32, int unit, int64_t M, int64_t D) {
  RowShape s;
  s.ept = D <= 256 ? 8 : D <= 512 || f32 || unit < 8 || !FWD ? 16 : 32;
  s.tpr = (int)(32 * ceil_div(D, 32 * s.ept));
  // (rows of two warps and more: 15 named barriers.  The forward's scale and
  // shift leave 768 threads' rings beside them from 4096 elements on.)
  int groups = (FWD && D > 4096 ? 768 : RowCfg<FWD>::THREADS) / s.tpr;
  if (s.tpr > 32) groups = std::min(groups, 15);
  s.threads = s.tpr * groups;
  s.blocks = std::min<int64_t>(ceil_div(M, groups), kSMs);
  return s;
}
template <bool FWD>
unsigned row_smem(const RowShape& s, bool ring, int64_t D) {
  const int64_t fixed = kSumBytes + (FWD ? 2 : 1) * (int64_t)s.tpr * s.ept * 4, cols = (int64_t)(s.threads / s.tpr) * 2 * D * 4;
  return (unsigned)(fixed + std::max<int64_t>(ring ? s.threads * RowCfg<FWD>::RING : 0, FWD ? 0 : cols));
}
// Blocks of the backward, each with its partial rows of dgamma and dbeta (the
// same for every type and alignment).
int64_t bwd_blocks(int64_t M, int64_t D) {
  return D > kMaxRow ? std::min<int64_t>(M, 32) : row_shape<false>(false, 1, M, D).blocks;
}

template <typename T, int VEC, int EPT, bool FULL, bool FWD>
const void* row_kernel() {
  if constexpr (FWD) return (const void*)ln_fwd_kernel<T, VEC, EPT, FULL>;
  else return (const void*)ln_bwd_kernel<T, VEC, EPT, FULL>;
}
// FULL where every thread's elements are all there (a row length that is a
// multiple of 32 EPT): no tests of the columns, half the instructions.
template <typename T, int VEC, int EPT, bool FWD>
const void* row_full(bool full) {
  return full ? row_kernel<T, VEC, EPT, true, FWD>() : row_kernel<T, VEC, EPT, false, FWD>();
}
template <bool FWD>
const void* row_pick(bool f32, int unit, const RowShape& s, int64_t D) {
  using B = __nv_bfloat16;
  const bool e8 = s.ept == 8, full = D == (int64_t)s.tpr * s.ept;
  if (f32) {
    if (unit == 1) return e8 ? row_kernel<float, 1, 8, false, FWD>() : row_kernel<float, 1, 16, false, FWD>();
    return e8 ? row_full<float, 4, 8, FWD>(full) : row_full<float, 4, 16, FWD>(full);
  }
  if (unit == 1) return e8 ? row_kernel<B, 1, 8, false, FWD>() : row_kernel<B, 1, 16, false, FWD>();
  if (unit == 2) return e8 ? row_kernel<B, 2, 8, false, FWD>() : row_kernel<B, 2, 16, false, FWD>();
  if constexpr (FWD)
    if (s.ept == 32) return row_full<B, 8, 32, FWD>(full);
  return e8 ? row_full<B, 8, 8, FWD>(full) : row_full<B, 8, 16, FWD>(full);
}

// The shapes taken, forward and backward.
bool shape_ok(int64_t M, int64_t D) { return M >= 1 && D >= 1 && M <= INT32_MAX && D <= kMaxD; }

}  // namespace

int layernorm_plan(const LayerNormOp& op, LaunchRec* rec, char* err, size_t errlen) {
  if (!shape_ok(op.M, op.D) || op.ldx < op.D || op.ldy < op.D) {
    snprintf(err, errlen, "bad layer-norm shape %lld x %lld", (long long)op.M, (long long)op.D);
    return -1;
  }
  const bool f32 = op.dtype == DT_F32;
  const int unit = unit_of(f32, (uintptr_t)op.x | (uintptr_t)op.y | (uint64_t)(op.D | op.ldx | op.ldy) * (f32 ? 4 : 2));
  LnFwdParams q{op.x, op.ldx, op.gamma, op.beta, op.y, op.ldy, op.mean, op.rstd, op.M, (int)op.D, op.eps, 0};
  if (op.D > kMaxRow) {
    rec->func = f32 ? (const void*)ln_fwd_wide_kernel<float> : (const void*)ln_fwd_wide_kernel<__nv_bfloat16>;
    rec->grid = dim3((unsigned)op.M);
    rec->block = dim3(1024);
    rec->smem = 0;
  } else {
    const RowShape s = row_shape<true>(f32, unit, op.M, op.D);
    q.tpr = s.tpr;
    rec->func = row_pick<true>(f32, unit, s, op.D);
    rec->grid = dim3((unsigned)s.blocks);
    rec->block = dim3((unsigned)s.threads);
    rec->smem = row_smem<true>(s, f32 || unit > 1, op.D);
  }
  rec->name = "layernorm_fwd";
  rec->set_args(q);
  return 1;
}

size_t layernorm_bwd_workspace_bytes(int64_t M, int64_t D) {
  return !shape_ok(M, D) ? 0 : (size_t)bwd_blocks(M, D) * 2 * (size_t)D * sizeof(float);
}

int layernorm_bwd_plan(const LayerNormBwdOp& op, LaunchRec* recs, char* err, size_t errlen) {
  if (!shape_ok(op.M, op.D) || op.ldx < op.D || op.lddy < op.D ||
      op.lddx < op.D) {
    snprintf(err, errlen, "bad layer-norm shape %lld x %lld", (long long)op.M, (long long)op.D);
    return -1;
  }
  const bool params = op.dgamma || op.dbeta;
  if (params && (!op.ws || op.ws_bytes < layernorm_bwd_workspace_bytes(op.M, op.D) || (uintptr_t)op.ws % 4)) {
    snprintf(err, errlen, "layer-norm backward workspace too small (%zu < %zu) or misaligned", op.ws_bytes,
             layernorm_bwd_workspace_bytes(op.M, op.D));
    return -1;
  }
  const bool f32 = op.dtype == DT_F32;
  const int unit = unit_of(f32, (uintptr_t)op.x | (uintptr_t)op.dy | (uintptr_t)op.dx |
                                    (uint64_t)(op.D | op.ldx | op.lddy | op.lddx) * (f32 ? 4 : 2));
  const int64_t blocks = bwd_blocks(op.M, op.D);
  LnBwdParams q{op.dy, op.lddy, op.x, op.ldx, op.gamma, op.mean, op.rstd, op.dx, op.lddx,
                params ? op.ws : nullptr, op.M, (int)op.D, 0};
  int n = 0;
  if (op.D > kMaxRow) {
    if (params) {
      recs[n].func = f32 ? (const void*)ln_bwd_wide_cols_kernel<float>
                         : (const void*)ln_bwd_wide_cols_kernel<__nv_bfloat16>;
      recs[n].grid = dim3((unsigned)blocks, (unsigned)ceil_div(op.D, 256));
      recs[n].block = dim3(256);
      recs[n].name = "layernorm_bwd_cols";
      recs[n++].set_args(q);
    }
    recs[n].func = f32 ? (const void*)ln_bwd_wide_kernel<float> : (const void*)ln_bwd_wide_kernel<__nv_bfloat16>;
    recs[n].grid = dim3((unsigned)op.M);
    recs[n].block = dim3(1024);
  } else {
    const RowShape s = row_shape<false>(f32, unit, op.M, op.D);
    q.tpr = s.tpr;
    recs[n].func = row_pick<false>(f32, unit, s, op.D);
    recs[n].grid = dim3((unsigned)s.blocks);
    recs[n].block = dim3((unsigned)s.threads);
    recs[n].smem = row_smem<false>(s, f32 || unit > 1, op.D);
  }
  recs[n].name = "layernorm_bwd";
  recs[n++].set_args(q);
  if (params) {
    const LnReduceParams r{op.ws, (int)blocks, (int)op.D, op.dgamma, op.dbeta};
    recs[n].func = (const void*)ln_param_reduce_kernel;
    recs[n].grid = dim3((unsigned)ceil_div(2 * op.D, 32));
    recs[n].block = dim3(1024);
    recs[n].name = "layernorm_param_reduce";
    recs[n++].set_args(r);
  }
  return n;
}

}  // namespace mlpk
