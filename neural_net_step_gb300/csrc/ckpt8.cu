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

// A walk over units of all rows, `step` at a time: the units of a row, and how
// far a step goes in whole rows and units (so that no thread divides as it
// goes: 64-bit divisions took as long as the memory did).
struct Walk { int units, step_rows, step_units; int64_t step; };
struct Place { int64_t row; int unit; };
__device__ __forceinline__ Place walk_start(const Walk& w, int64_t i) {
  Place p;
  p.row = i / w.units;
  p.unit = (int)(i - p.row * w.units);
  return p;
}
__device__ __forceinline__ void walk_on(const Walk& w, Place& p) {
  p.row += w.step_rows;
  p.unit += w.step_units;
  if (p.unit >= w.units) { p.unit -= w.units; ++p.row; }
}
constexpr int kAhead = 4;   // units a thread has under way

struct Quant8Params {
  const void* x; int64_t ldx;
  uint8_t* q; int64_t ldq;
  uint8_t* e; int64_t lde;
  int64_t rows; int cols;
  Walk walk;           // units: 8-column groups (vectors), or 32-column blocks
};

// Eight elements from 16-byte aligned memory, as they come and as fp32.
template <typename T> struct Raw8 { uint4 w[sizeof(T) / 2]; };
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* src) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
  return r;
}
template <typename T>
__device__ __forceinline__ void open8(const Raw8<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
  } else {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
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
// of four, and a step is one too).  kAhead loads first, then their units.
template <typename T>
__global__ void __launch_bounds__(256) quant8_vec_kernel(const __grid_constant__ Quant8Params p) {
  pdl_enter();
  const int64_t first = blockIdx.x * (int64_t)256 + threadIdx.x;
  Place at = walk_start(p.walk, first);
  // (whole warps go round together, for the shuffles)
  for (int64_t i = first - (threadIdx.x & 31); i < p.rows * p.walk.units; i += kAhead * p.walk.step) {
    Raw8<T> raw[kAhead];
    Place pl[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      pl[k] = at;
      walk_on(p.walk, at);
      if (pl[k].row < p.rows && pl[k].unit * 8 + 8 <= p.cols)
        raw[k] = load8(reinterpret_cast<const T*>(p.x) + pl[k].row * p.ldx + pl[k].unit * 8);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t row = pl[k].row;
      const int c = pl[k].unit * 8;
      const bool whole = row < p.rows && c + 8 <= p.cols;
      float v[8];
      if (whole) {
        open8(raw[k], v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = row < p.rows && c + j < p.cols ? to_f32(reinterpret_cast<const T*>(p.x)[row * p.ldx + c + j]) : 0.f;
      }
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));   // (skips NaN)
      uint32_t m = __float_as_uint(a);
      if (m >= 0x7f800000u) {   // an infinity among them
        m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m = max(m, q8_mag(v[j]));
          v[j] = q8_no_inf(v[j]);
        }
      }
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = q8_exponent(m);
      const float s = q8_pow2(-e);
      if (row >= p.rows || c >= p.cols) continue;
      uint8_t* qr = p.q + row * p.ldq + c;
      const uint2 w = make_uint2(q8_pack(v[0] * s, v[1] * s, v[2] * s, v[3] * s),
                                 q8_pack(v[4] * s, v[5] * s, v[6] * s, v[7] * s));
      if (whole) {
        *reinterpret_cast<uint2*>(qr) = w;
      } else {
        for (int j = 0; j < p.cols - c; ++j) qr[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
      }
      if ((c & 31) == 0) p.e[row * p.lde + (c >> 5)] = (uint8_t)(e + 127);
    }
  }
}

// Any alignment: a warp per block of 32 columns, a column per lane.
template <typename T>
__global__ void __launch_bounds__(256) quant8_kernel(const __grid_constant__ Quant8Params p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  for (Place at = walk_start(p.walk, blockIdx.x * (int64_t)8 + (threadIdx.x >> 5)); at.row < p.rows; walk_on(p.walk, at)) {
    const int c = at.unit * 32 + lane;
    const float v = c < p.cols ? to_f32(reinterpret_cast<const T*>(p.x)[at.row * p.ldx + c]) : 0.f;
    const int k = q8_exponent(__reduce_max_sync(0xffffffffu, q8_mag(v)));
    if (c < p.cols) p.q[at.row * p.ldq + c] = (uint8_t)q8_pack(q8_no_inf(v) * q8_pow2(-k), 0.f, 0.f, 0.f);
    if (lane == 0) p.e[at.row * p.lde + at.unit] = (uint8_t)(k + 127);
  }
}

struct Dequant8Params {
  const uint8_t* q; int64_t ldq;
  const uint8_t* e; int64_t lde;
  void* y; int64_t ldy;
  int64_t rows; int cols;
  Walk walk;
};

template <typename T>
__global__ void __launch_bounds__(256) dequant8_vec_kernel(const __grid_constant__ Dequant8Params p) {
  pdl_enter();
  Place at = walk_start(p.walk, blockIdx.x * (int64_t)256 + threadIdx.x);
  while (at.row < p.rows) {
    uint2 w[kAhead];
    uint32_t e[kAhead];
    Place pl[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      pl[k] = at;
      walk_on(p.walk, at);
      const int c = pl[k].unit * 8;
      if (pl[k].row < p.rows) {
        if (c + 8 <= p.cols) w[k] = __ldg(reinterpret_cast<const uint2*>(p.q + pl[k].row * p.ldq + c));
        e[k] = __ldg(p.e + pl[k].row * p.lde + (c >> 5));
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (pl[k].row >= p.rows) break;
      const int c = pl[k].unit * 8;
      T* yr = reinterpret_cast<T*>(p.y) + pl[k].row * p.ldy + c;
      if (c + 8 <= p.cols) {
        const float s = q8_scale(e[k]);
        float v[8];
        q8_unpack(w[k].x, s, v);
        q8_unpack(w[k].y, s, v + 4);
        store8(yr, v);
      } else {
        const uint8_t* qr = p.q + pl[k].row * p.ldq + c;
        for (int j = 0; j < p.cols - c; ++j) yr[j] = from_f32<T>(q8_value(qr[j], e[k]));
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) dequant8_kernel(const __grid_constant__ Dequant8Params p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  for (Place at = walk_start(p.walk, blockIdx.x * (int64_t)8 + (threadIdx.x >> 5)); at.row < p.rows; walk_on(p.walk, at)) {
    const int c = at.unit * 32 + lane;
    if (c >= p.cols) continue;
    reinterpret_cast<T*>(p.y)[at.row * p.ldy + c] =
        from_f32<T>(q8_value(p.q[at.row * p.ldq + c], p.e[at.row * p.lde + at.unit]));
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

// The grid of a walk over `units` units a row, `per_block` at a time: blocks
// enough for every unit at `ahead` a thread, at most eight to an SM.
Walk shape_launch(LaunchRec* rec, int64_t rows, int64_t units, int per_block, int ahead) {
  const int64_t blocks = std::min<int64_t>(ceil_div(rows * units, per_block * ahead), kSMs * 8);
  rec->grid = dim3((unsigned)blocks);
  rec->block = dim3(256);
  rec->smem = 0;
  Walk w;
  w.units = (int)units;
  w.step = blocks * per_block;
  w.step_rows = (int)(w.step / units);
  w.step_units = (int)(w.step % units);
  return w;
}

}  // namespace

int quant8_plan(int dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx, uint8_t* q, int64_t ldq,
                uint8_t* e, int64_t lde, LaunchRec* rec, char* err, size_t errlen) {
  if (bad_shape(rows, cols, ldx, ldq, lde, err, errlen)) return -1;
  const bool f32 = dtype == DT_F32;
  const bool vec = ((uintptr_t)x & 15) == 0 && (ldx * (f32 ? 4 : 2)) % 16 == 0 && ((uintptr_t)q & 7) == 0 &&
                   ldq % 8 == 0;
  // (vectors: whole blocks of four threads)
  const Quant8Params p{x, ldx, q, ldq, e, lde, rows, (int)cols,
                       vec ? shape_launch(rec, rows, 4 * q8_blocks(cols), 256, kAhead)
                           : shape_launch(rec, rows, q8_blocks(cols), 8, 1)};
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
  const Dequant8Params p{q, ldq, e, lde, y, ldy, rows, (int)cols,
                         vec ? shape_launch(rec, rows, ceil_div(cols, 8), 256, kAhead)
                             : shape_launch(rec, rows, q8_blocks(cols), 8, 1)};
  rec->func = f32 ? (vec ? (const void*)dequant8_vec_kernel<float> : (const void*)dequant8_kernel<float>)
                  : (vec ? (const void*)dequant8_vec_kernel<__nv_bfloat16>
                         : (const void*)dequant8_kernel<__nv_bfloat16>);
  rec->name = "dequant8";
  rec->set_args(p);
  return 1;
}

}  // namespace mlpk
