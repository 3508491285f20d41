// Activation checkpoints in 8 bits (e4m3.cuh): quantise a matrix, read it
// back.  Both move each byte once and are bound by DRAM.
#include <stdio.h>

#include <algorithm>

#include "common.cuh"
#include "e4m3.cuh"
#include "ops.h"

namespace mlpk {

namespace {

constexpr int kSMs = 152;

struct Quant8Params {
  const void* x; int64_t ldx;
  uint8_t* q; int64_t ldq;
  uint8_t* e; int64_t lde;
  int64_t rows; int cols;
  int units;           // per row: 8-column groups (vectors), or 32-column blocks
};

// Eight elements as fp32 from 16-byte aligned memory.
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
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
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
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

// Aligned rows: eight columns per thread, so the four threads of a block of
// 32 columns are neighbours in a warp (units per row are padded to a multiple
// of four, and a warp's 32 units to whole blocks).
template <typename T>
__global__ void __launch_bounds__(256) quant8_vec_kernel(const __grid_constant__ Quant8Params p) {
  pdl_enter();
  const int64_t total = p.rows * p.units;
  const int64_t step = (int64_t)gridDim.x * 256;
  // every thread of a warp runs the same number of rounds (the shuffles)
  for (int64_t i0 = blockIdx.x * (int64_t)256 + (threadIdx.x & ~31); i0 < total; i0 += step) {
    const int64_t i = i0 + (threadIdx.x & 31);
    const int64_t row = i < total ? i / p.units : 0;
    const int c = i < total ? (int)(i - row * p.units) * 8 : p.cols;
    const T* xr = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    float v[8];
    if (c + 8 <= p.cols) {
      load8(xr + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < p.cols ? to_f32(xr[c + j]) : 0.f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m = max(m, q8_mag(v[j]));
      v[j] = q8_no_inf(v[j]);
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int k = q8_exponent(m);
    const float s = q8_pow2(-k);
    if (c >= p.cols) continue;
    uint8_t* qr = p.q + row * p.ldq + c;
    const uint2 w = make_uint2(q8_pack(v[0] * s, v[1] * s, v[2] * s, v[3] * s),
                               q8_pack(v[4] * s, v[5] * s, v[6] * s, v[7] * s));
    if (c + 8 <= p.cols) {
      *reinterpret_cast<uint2*>(qr) = w;
    } else {
      for (int j = 0; j < p.cols - c; ++j) qr[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    }
    if ((c & 31) == 0) p.e[row * p.lde + (c >> 5)] = (uint8_t)(k + 127);
  }
}

// Any alignment: a warp per block of 32 columns, a column per lane.
template <typename T>
__global__ void __launch_bounds__(256) quant8_kernel(const __grid_constant__ Quant8Params p) {
  pdl_enter();
  const int64_t total = p.rows * p.units;
  const int lane = threadIdx.x & 31;
  for (int64_t i = blockIdx.x * (int64_t)8 + (threadIdx.x >> 5); i < total; i += (int64_t)gridDim.x * 8) {
    const int64_t row = i / p.units;
    const int b = (int)(i - row * p.units), c = b * 32 + lane;
    const float v = c < p.cols ? to_f32(reinterpret_cast<const T*>(p.x)[row * p.ldx + c]) : 0.f;
    const int k = q8_exponent(__reduce_max_sync(0xffffffffu, q8_mag(v)));
    if (c < p.cols) p.q[row * p.ldq + c] = (uint8_t)q8_pack(q8_no_inf(v) * q8_pow2(-k), 0.f, 0.f, 0.f);
    if (lane == 0) p.e[row * p.lde + b] = (uint8_t)(k + 127);
  }
}

struct Dequant8Params {
  const uint8_t* q; int64_t ldq;
  const uint8_t* e; int64_t lde;
  void* y; int64_t ldy;
  int64_t rows; int cols;
  int units;
};

template <typename T>
__global__ void __launch_bounds__(256) dequant8_vec_kernel(const __grid_constant__ Dequant8Params p) {
  pdl_enter();
  const int64_t total = p.rows * p.units;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / p.units;
    const int c = (int)(i - row * p.units) * 8;
    const uint8_t* qr = p.q + row * p.ldq + c;
    T* yr = reinterpret_cast<T*>(p.y) + row * p.ldy + c;
    const float s = q8_scale(p.e[row * p.lde + (c >> 5)]);
    float v[8];
    if (c + 8 <= p.cols) {
      const uint2 w = *reinterpret_cast<const uint2*>(qr);
      q8_unpack(w.x, s, v);
      q8_unpack(w.y, s, v + 4);
      store8(yr, v);
    } else {
      for (int j = 0; j < p.cols - c; ++j) yr[j] = from_f32<T>(q8_value(qr[j], p.e[row * p.lde + (c >> 5)]));
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) dequant8_kernel(const __grid_constant__ Dequant8Params p) {
  pdl_enter();
  const int64_t total = p.rows * p.units;
  const int lane = threadIdx.x & 31;
  for (int64_t i = blockIdx.x * (int64_t)8 + (threadIdx.x >> 5); i < total; i += (int64_t)gridDim.x * 8) {
    const int64_t row = i / p.units;
    const int b = (int)(i - row * p.units), c = b * 32 + lane;
    if (c >= p.cols) continue;
    reinterpret_cast<T*>(p.y)[row * p.ldy + c] = from_f32<T>(q8_value(p.q[row * p.ldq + c], p.e[row * p.lde + b]));
  }
}

bool bad_shape(int64_t rows, int64_t cols, int64_t ld, int64_t ldq, int64_t lde, char* err, size_t errlen) {
  if (rows >= 1 && cols >= 1 && rows <= INT32_MAX && cols <= INT32_MAX - 64 && ld >= cols && ldq >= cols &&
      lde >= q8_blocks(cols))
    return false;
  snprintf(err, errlen, "bad 8-bit checkpoint shape %lld x %lld or leading dimension", (long long)rows,
           (long long)cols);
  return true;
}

void shape_launch(LaunchRec* rec, bool vec, int64_t rows, int64_t cols, int* units) {
  // vectors: 8 columns a thread, whole blocks of four threads; else a warp per block
  *units = (int)(q8_blocks(cols) * (vec ? 4 : 1));
  const int64_t blocks = ceil_div(rows * *units, vec ? 256 : 8);
  rec->grid = dim3((unsigned)std::min<int64_t>(blocks, kSMs * 64));
  rec->block = dim3(256);
  rec->smem = 0;
}

}  // namespace

int quant8_plan(int dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx, uint8_t* q, int64_t ldq,
                uint8_t* e, int64_t lde, LaunchRec* rec, char* err, size_t errlen) {
  if (bad_shape(rows, cols, ldx, ldq, lde, err, errlen)) return -1;
  const bool f32 = dtype == DT_F32;
  const bool vec = ((uintptr_t)x & 15) == 0 && (ldx * (f32 ? 4 : 2)) % 16 == 0 && ((uintptr_t)q & 7) == 0 &&
                   ldq % 8 == 0;
  Quant8Params p{x, ldx, q, ldq, e, lde, rows, (int)cols, 0};
  shape_launch(rec, vec, rows, cols, &p.units);
  rec->func = f32 ? (vec ? (const void*)quant8_vec_kernel<float> : (const void*)quant8_kernel<float>)
                  : (vec ? (const void*)quant8_vec_kernel<__nv_bfloat16> : (const void*)quant8_kernel<__nv_bfloat16>);
  rec->name = "quant8";
  rec->set_args(p);
  return 1;
}

int dequant8_plan(int dtype, int64_t rows, int64_t cols, const uint8_t* q, int64_t ldq, const uint8_t* e, int64_t lde,
                  void* y, int64_t ldy, LaunchRec* rec, char* err, size_t errlen) {
  if (bad_shape(rows, cols, ldy, ldq, lde, err, errlen)) return -1;
  const bool f32 = dtype == DT_F32;
  const bool vec = ((uintptr_t)y & 15) == 0 && (ldy * (f32 ? 4 : 2)) % 16 == 0 && ((uintptr_t)q & 7) == 0 &&
                   ldq % 8 == 0;
  Dequant8Params p{q, ldq, e, lde, y, ldy, rows, (int)cols, 0};
  shape_launch(rec, vec, rows, cols, &p.units);
  // (a row's padding groups of four hold no columns: units past cols are cut)
  if (vec) p.units = (int)ceil_div(cols, 8);
  rec->func = f32 ? (vec ? (const void*)dequant8_vec_kernel<float> : (const void*)dequant8_kernel<float>)
                  : (vec ? (const void*)dequant8_vec_kernel<__nv_bfloat16>
                         : (const void*)dequant8_kernel<__nv_bfloat16>);
  rec->name = "dequant8";
  rec->set_args(p);
  return 1;
}

}  // namespace mlpk
