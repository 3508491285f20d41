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
// mean and 1 / sqrt(variance + eps).
__device__ __forceinline__ void finish_stats(const float (&s)[2], float inv_d, float eps, float& rest, float& rstd) {
  rest = s[0] * inv_d;
  rstd = 1.0f / sqrtf(fmaxf(fmaf(-rest, rest, s[1] * inv_d), 0.f) + eps);
}

// WARPS = 1: a warp per row, eight rows per block; else a block per row.
// Thread t of a row's threads holds vectors t, t + threads, ... (NV of them,
// VEC elements each).
template <typename T, int VEC, int NV, int WARPS>
__global__ void __launch_bounds__(256) ln_fwd_kernel(const __grid_constant__ LnFwdParams p) {
  pdl_enter();
  __shared__ float sh1[1][WARPS], sh2[2][WARPS];
  constexpr int TPR = 32 * WARPS;
  const int64_t row = WARPS == 1 ? blockIdx.x * (int64_t)8 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (row >= p.M) return;   // (a warp, or the whole block)
  const int t = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
  const T* xr = reinterpret_cast<const T*>(p.x) + row * p.ldx;
  float v[NV][VEC];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * TPR) * VEC;
    if (c < p.D) {
      load_vec<T, VEC>(xr + c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += v[i][j];
  const float inv_d = 1.0f / (float)p.D;
  row_sums<WARPS, 1>(s, sh1);
  const float mean = s[0] * inv_d;
  float sd[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = (t + i * TPR) * VEC < p.D;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      v[i][j] -= mean;
      if (in) {
        sd[0] += v[i][j];
        sd[1] = fmaf(v[i][j], v[i][j], sd[1]);
      }
    }
  }
  row_sums<WARPS, 2>(sd, sh2);
  float rest, rstd;
  finish_stats(sd, inv_d, p.eps, rest, rstd);
  if (t == 0) {
    if (p.mean) p.mean[row] = mean + rest;
    if (p.rstd) p.rstd[row] = rstd;
  }
  T* yr = reinterpret_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * TPR) * VEC;
    if (c >= p.D) continue;
    float g[VEC], b[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) { g[j] = 1.f; b[j] = 0.f; }
    if (p.gamma) {
#pragma unroll
      for (int j = 0; j < VEC; j += (VEC == 1 ? 1 : 4)) load_vec<float, VEC == 1 ? 1 : 4>(p.gamma + c + j, g + j);
    }
    if (p.beta) {
#pragma unroll
      for (int j = 0; j < VEC; j += (VEC == 1 ? 1 : 4)) load_vec<float, VEC == 1 ? 1 : 4>(p.beta + c + j, b + j);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[i][j] = fmaf((v[i][j] - rest) * rstd, g[j], b[j]);
    store_vec<T, VEC>(yr + c, v[i]);
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

constexpr int kBwdEpt = 8;   // elements of a row per thread

// `tpr` threads share a row, 8 elements each; the block's groups walk the
// rows and keep their columns' dgamma / dbeta sums in registers, adding them
// over the groups at the end: one partial row pair per block.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024) ln_bwd_kernel(const __grid_constant__ LnBwdParams p) {
  pdl_enter();
  constexpr int NV = kBwdEpt / VEC;
  extern __shared__ float ln_smem[];          // [2][32][2] warp sums, then the groups' column sums
  float* wsum = ln_smem;
  float* colsum = ln_smem + 128;
  const int tpr = p.tpr, groups = (int)blockDim.x / tpr;
  const int group = (int)threadIdx.x / tpr, t = (int)threadIdx.x % tpr;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int wpr = tpr >> 5, w0 = group * wpr;   // this row's warps
  const float inv_d = 1.0f / (float)p.D;
  float g[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * tpr) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      g[i][j] = c + j < p.D ? (p.gamma ? p.gamma[c + j] : 1.f) : 0.f;
      dg[i][j] = db[i][j] = 0.f;
    }
  }
  int buf = 0;
  for (int64_t row = blockIdx.x * (int64_t)groups + group; row < p.M; row += (int64_t)gridDim.x * groups) {
    const T* xr = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    const T* dr = reinterpret_cast<const T*>(p.dy) + row * p.lddy;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float x[NV][VEC], d[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * tpr) * VEC;
      if (c < p.D) {
        load_vec<T, VEC>(xr + c, x[i]);
        load_vec<T, VEC>(dr + c, d[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) { x[i][j] = mean; d[i][j] = 0.f; }
      }
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float xh = (x[i][j] - mean) * rstd;
        dg[i][j] = fmaf(d[i][j], xh, dg[i][j]);
        db[i][j] += d[i][j];
        x[i][j] = xh;
        d[i][j] *= g[i][j];
        s1 += d[i][j];
        s2 = fmaf(d[i][j], xh, s2);
      }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (wpr > 1) {
      float* w = wsum + buf * 64;
      if (lane == 0) { w[2 * warp] = s1; w[2 * warp + 1] = s2; }
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
      s1 = s2 = 0.f;
      for (int k = 0; k < wpr; ++k) {
        s1 += w[2 * (w0 + k)];
        s2 += w[2 * (w0 + k) + 1];
      }
      buf ^= 1;
    }
    const float c1 = s1 * inv_d, c2 = s2 * inv_d;
    T* or_ = reinterpret_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * tpr) * VEC;
      if (c >= p.D) continue;
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = rstd * (d[i][j] - c1 - x[i][j] * c2);
      store_vec<T, VEC>(or_ + c, o);
    }
  }
  if (!p.part) return;
  // the groups' column sums, group by group
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.D;
  for (int k = 0; k < groups; ++k) {
    if (group == k) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          if (c + j >= p.D) continue;
          if (k > 0) {
            dg[i][j] += colsum[c + j];
            db[i][j] += colsum[p.D + c + j];
          }
          if (k + 1 < groups) {
            colsum[c + j] = dg[i][j];
            colsum[p.D + c + j] = db[i][j];
          } else {
            out[c + j] = dg[i][j];
            out[p.D + c + j] = db[i][j];
          }
        }
      }
    }
    __syncthreads();
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

// dgamma and dbeta from the blocks' partial rows: 32 columns per block, eight
// warps that each add every eighth partial, then the eight sums in order.
struct LnReduceParams {
  const float* part; int parts; int D;
  float* dgamma; float* dbeta;
};
__global__ void __launch_bounds__(256) ln_param_reduce_kernel(const __grid_constant__ LnReduceParams p) {
  pdl_enter();
  __shared__ float sh[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * (int64_t)32 + lane, n = 2 * (int64_t)p.D;
  float s = 0.f;
  if (c < n) {
#pragma unroll 4
    for (int k = w; k < p.parts; k += 8) s += p.part[k * n + c];
  }
  sh[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < n) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sh[k][lane];
    if (c < p.D) {
      if (p.dgamma) p.dgamma[c] = s;
    } else if (p.dbeta) {
      p.dbeta[c - p.D] = s;
    }
  }
}

template <typename T, int VEC, int WARPS>
const void* fwd_pick(int64_t D) {
  constexpr int unit = 32 * WARPS;
  if (D <= unit * 8) return (const void*)ln_fwd_kernel<T, VEC, 8 / VEC, WARPS>;
  if (D <= unit * 16) return (const void*)ln_fwd_kernel<T, VEC, 16 / VEC, WARPS>;
  return (const void*)ln_fwd_kernel<T, VEC, 32 / VEC, WARPS>;
}

bool aligned16(const void* p, int64_t ld, size_t es) {
  return ((uintptr_t)p & 15) == 0 && (ld * (int64_t)es) % 16 == 0;
}

// Blocks (and partial rows) of the backward, and its threads per row.
struct BwdShape { int tpr, threads; int64_t blocks; };
BwdShape bwd_shape(int64_t M, int64_t D) {
  BwdShape s;
  if (D > kMaxRow) {
    s.tpr = s.threads = 0;
    s.blocks = std::min<int64_t>(M, 32);
    return s;
  }
  s.tpr = (int)(32 * ceil_div(D, 32 * kBwdEpt));
  const int groups = std::min(std::max(1, 512 / s.tpr), 15);   // (named barriers 1..15)
  s.threads = s.tpr * groups;
  s.blocks = std::min<int64_t>(ceil_div(M, groups), kSMs * std::max(1, 1024 / s.threads));
  return s;
}

}  // namespace

int layernorm_plan(const LayerNormOp& op, LaunchRec* rec, char* err, size_t errlen) {
  if (op.M < 1 || op.D < 1 || op.M > INT32_MAX || op.D > kMaxD || op.ldx < op.D || op.ldy < op.D) {
    snprintf(err, errlen, "bad layer-norm shape %lld x %lld", (long long)op.M, (long long)op.D);
    return -1;
  }
  const LnFwdParams q{op.x, op.ldx, op.gamma, op.beta, op.y, op.ldy, op.mean, op.rstd, op.M, (int)op.D, op.eps};
  const bool f32 = op.dtype == DT_F32;
  const size_t es = f32 ? 4 : 2;
  const int vec = f32 ? 4 : 8;
  const bool v = op.D % vec == 0 && aligned16(op.x, op.ldx, es) && aligned16(op.y, op.ldy, es) &&
                 aligned16(op.gamma, 0, 4) && aligned16(op.beta, 0, 4);
  rec->block = dim3(256);
  rec->grid = dim3((unsigned)op.M);
  if (op.D > kMaxRow) {
    rec->func = f32 ? (const void*)ln_fwd_wide_kernel<float> : (const void*)ln_fwd_wide_kernel<__nv_bfloat16>;
    rec->block = dim3(1024);
  } else if (op.D <= 1024) {
    rec->grid = dim3((unsigned)ceil_div(op.M, 8));
    rec->func = f32 ? (v ? fwd_pick<float, 4, 1>(op.D) : fwd_pick<float, 1, 1>(op.D))
                    : (v ? fwd_pick<__nv_bfloat16, 8, 1>(op.D) : fwd_pick<__nv_bfloat16, 1, 1>(op.D));
  } else {
    rec->func = f32 ? (v ? fwd_pick<float, 4, 8>(op.D) : fwd_pick<float, 1, 8>(op.D))
                    : (v ? fwd_pick<__nv_bfloat16, 8, 8>(op.D) : fwd_pick<__nv_bfloat16, 1, 8>(op.D));
  }
  rec->smem = 0;
  rec->name = "layernorm_fwd";
  rec->set_args(q);
  return 1;
}

size_t layernorm_bwd_workspace_bytes(int64_t M, int64_t D) {
  return (size_t)bwd_shape(M, D).blocks * 2 * (size_t)D * sizeof(float);
}

int layernorm_bwd_plan(const LayerNormBwdOp& op, LaunchRec* recs, char* err, size_t errlen) {
  if (op.M < 1 || op.D < 1 || op.M > INT32_MAX || op.D > kMaxD || op.ldx < op.D || op.lddy < op.D ||
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
  const BwdShape s = bwd_shape(op.M, op.D);
  const bool f32 = op.dtype == DT_F32;
  const size_t es = f32 ? 4 : 2;
  const int vec = f32 ? 4 : 8;
  const bool v = op.D % vec == 0 && aligned16(op.x, op.ldx, es) && aligned16(op.dy, op.lddy, es) &&
                 aligned16(op.dx, op.lddx, es);
  const LnBwdParams q{op.dy, op.lddy, op.x, op.ldx, op.gamma, op.mean, op.rstd, op.dx, op.lddx,
                      params ? op.ws : nullptr, op.M, (int)op.D, s.tpr};
  int n = 0;
  if (op.D > kMaxRow) {
    if (params) {
      recs[n].func = f32 ? (const void*)ln_bwd_wide_cols_kernel<float>
                         : (const void*)ln_bwd_wide_cols_kernel<__nv_bfloat16>;
      recs[n].grid = dim3((unsigned)s.blocks, (unsigned)ceil_div(op.D, 256));
      recs[n].block = dim3(256);
      recs[n].name = "layernorm_bwd_cols";
      recs[n++].set_args(q);
    }
    recs[n].func = f32 ? (const void*)ln_bwd_wide_kernel<float> : (const void*)ln_bwd_wide_kernel<__nv_bfloat16>;
    recs[n].grid = dim3((unsigned)op.M);
    recs[n].block = dim3(1024);
  } else {
    recs[n].func = f32 ? (v ? (const void*)ln_bwd_kernel<float, 4> : (const void*)ln_bwd_kernel<float, 1>)
                       : (v ? (const void*)ln_bwd_kernel<__nv_bfloat16, 8>
                            : (const void*)ln_bwd_kernel<__nv_bfloat16, 1>);
    recs[n].grid = dim3((unsigned)s.blocks);
    recs[n].block = dim3((unsigned)s.threads);
    // warp sums, and the column sums handed from group to group
    recs[n].smem = (unsigned)(128 * 4 + (s.threads > s.tpr ? 2 * op.D * 4 : 0));
  }
  recs[n].name = "layernorm_bwd";
  recs[n++].set_args(q);
  if (params) {
    const LnReduceParams r{op.ws, (int)s.blocks, (int)op.D, op.dgamma, op.dbeta};
    recs[n].func = (const void*)ln_param_reduce_kernel;
    recs[n].grid = dim3((unsigned)ceil_div(2 * op.D, 32));
    recs[n].block = dim3(256);
    recs[n].name = "layernorm_param_reduce";
    recs[n++].set_args(r);
  }
  return n;
}

}  // namespace mlpk
