// The gated feed-forward projection for a few rows (decoding), bf16.  Every
// weight is read once for at most 32 products a row of it, so W's 4 F K bytes
// bound it: 2.5 us from DRAM at F = 4096, K = 1024, where one row takes 5.6 us
// (13.6 us of 9.9 at F = 8192, K = 2048; launches back to back, 2.6 us for the
// smallest), the kernel of the large sizes 12 us with its 32 tiles.
//
// A block takes 16 gate rows of W and the 16 up rows that belong to them over
// all of K, cut into 32-wide chunks that its warps take in turn.  The products
// run on mma.sync.m16n8k16 with W as the 16-row operand and the tokens as the
// 8-column one.  The order of k inside a chunk is free as long as both operands
// share it, so lane (g = lane / 4, t = lane % 4) takes k = 8 t .. 8 t + 7 of
// the chunk: one 16-byte load per row of W (and per token of X) feeds two
// MMAs, straight from global memory, no staging.  The warps' partial sums are
// added in a fixed order through shared memory, where bias, gate and product
// finish.
#include <stdio.h>

#include <algorithm>

#include "common.cuh"
#include "gated.cuh"
#include "ops.h"

namespace mlpk {

namespace {

// The rows it takes.  Up to 16 it is ahead of the CTA pairs at every size
// measured (16 rows, F x K: 4096 x 1024 7.7 us against 12.6, 1024 x 4096 9.0
// against 25, 8192 x 2048 14.8 against 17.1); up to 32 its products and reads
// of X weigh in and it is ahead only where the pairs have few tiles (10.3
// against 12.6, 14.1 against 25, but 29 against 17).
bool rows_taken(int64_t M, int64_t F) { return M <= 16 || (M <= 32 && F <= 4096); }

struct GatedSmallParams {
  const __nv_bfloat16* x; int64_t ldx;
  const __nv_bfloat16* w; int64_t ldw;
  const float* bias;
  __nv_bfloat16* h; int64_t ldh;
  __nv_bfloat16* s; int64_t lds;
  int M, F, K, chunks;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p, bool in) {
  return in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

// NT tiles of 8 tokens.
template <int NT, int ACT>
__global__ void __launch_bounds__(512) gated_small_kernel(const __grid_constant__ GatedSmallParams p) {
  pdl_enter();
  extern __shared__ __align__(16) float part[];   // [warps][2 (gate, up)][16][8 NT + 1]
  constexpr int PITCH = 8 * NT + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int f0 = blockIdx.x * 16;
  // this lane's rows of W: gate f0 + g and + 8, up the same further down (F is
  // a multiple of 8: eight rows are there or not together)
  const __nv_bfloat16* w0 = p.w + (int64_t)(f0 + g) * p.ldw + 8 * t;
  const __nv_bfloat16* w1 = w0 + (int64_t)p.F * p.ldw;
  const bool two = f0 + 8 < p.F;
  const int64_t down8 = 8 * p.ldw;
  const __nv_bfloat16* xr = p.x + (int64_t)g * p.ldx + 8 * t;
  float dg[NT][4], du[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[n][i] = du[n][i] = 0.f;
#pragma unroll 4
  for (int c = warp; c < p.chunks; c += warps) {
    const int k = 32 * c;
    const bool in = k + 8 * t < p.K;   // (K is a multiple of 8)
    const uint4 a = load16(w0 + k, in), b = load16(w0 + down8 + k, in && two);
    const uint4 e = load16(w1 + k, in), f = load16(w1 + down8 + k, in && two);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 x = load16(xr + (int64_t)(8 * n) * p.ldx + k, in && 8 * n + g < p.M);
      mma16816(dg[n], a.x, b.x, a.y, b.y, x.x, x.y);
      mma16816(dg[n], a.z, b.z, a.w, b.w, x.z, x.w);
      mma16816(du[n], e.x, f.x, e.y, f.y, x.x, x.y);
      mma16816(du[n], e.z, f.z, e.w, f.w, x.z, x.w);
    }
  }
  // D: rows g and g + 8 (of W), columns 2 t and 2 t + 1 (tokens)
  float* mine = part + (int64_t)warp * 32 * PITCH;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = (g + (i >= 2 ? 8 : 0)) * PITCH + 8 * n + 2 * t + (i & 1);
      mine[at] = dg[n][i];
      mine[16 * PITCH + at] = du[n][i];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * p.M; i += blockDim.x) {
    const int m = i >> 4, r = i & 15, f = f0 + r;
    if (f >= p.F) continue;
    float a = 0.f, b = 0.f;
    for (int q = 0; q < warps; ++q) {
      a += part[(q * 32 + r) * PITCH + m];
      b += part[(q * 32 + 16 + r) * PITCH + m];
    }
    if (p.bias) {
      a += p.bias[f];
      b += p.bias[p.F + f];
    }
    if (p.s) {
      p.s[(int64_t)m * p.lds + f] = __float2bfloat16_rn(a);
      p.s[(int64_t)m * p.lds + p.F + f] = __float2bfloat16_rn(b);
    }
    p.h[(int64_t)m * p.ldh + f] = __float2bfloat16_rn(gate_act(a, ACT) * b);
  }
}

template <int NT, int ACT>
const void* small_kernel() {
  return (const void*)gated_small_kernel<NT, ACT>;
}
template <int NT>
const void* small_pick(int act) {
  switch (act) {
    case ACT_RELU: return small_kernel<NT, ACT_RELU>();
    case ACT_GELU_TANH: return small_kernel<NT, ACT_GELU_TANH>();
    case ACT_SILU: return small_kernel<NT, ACT_SILU>();
    default: return small_kernel<NT, ACT_NONE>();
  }
}

}  // namespace

bool gated_small_takes(const GatedOp& op) { return op.fwd && op.dtype == DT_BF16 && !op.se && rows_taken(op.M, op.F); }

int gated_small_plan(const GatedOp& op, LaunchRec* rec) {
  const GatedSmallParams p{(const __nv_bfloat16*)op.A, op.lda, (const __nv_bfloat16*)op.B, op.ldb, op.bias,
                           (__nv_bfloat16*)op.h, op.ldh, (__nv_bfloat16*)op.s, op.lds, (int)op.M, (int)op.F,
                           (int)op.K, (int)ceil_div(op.K, 32)};
  const int nt = op.M <= 8 ? 1 : op.M <= 16 ? 2 : 4;
  // four chunks a warp, so that all its loads are under way at once
  const int warps = (int)std::min<int64_t>(16, std::max<int64_t>(1, ceil_div(p.chunks, 4)));
  rec->func = nt == 1 ? small_pick<1>(op.act) : nt == 2 ? small_pick<2>(op.act) : small_pick<4>(op.act);
  rec->grid = dim3((unsigned)ceil_div(op.F, 16));
  rec->block = dim3((unsigned)(32 * warps));
  rec->smem = (unsigned)(warps * 32 * (8 * nt + 1) * 4);
  rec->name = "gated_small_fwd";
  rec->set_args(p);
  return 1;
}

}  // namespace mlpk
