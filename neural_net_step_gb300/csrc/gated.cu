// The gated feed-forward projection and its vector-Jacobian product:
//   forward   s = X W^T + b with W [2F, K] (F gate rows, then F up rows),
//             g = s[:, :F], u = s[:, F:], H = act(g) * u;
//   backward  dH = dY Wd (the down projection's dgrad),
//             dS = [dH * u * act'(g) | dH * act(g)], H = act(g) * u again.
// s is kept for the backward in the dtype or in 8 bits (e4m3.cuh).
//
// bf16 runs on the tensor cores (gated_tc.cu).  fp32 on the FFMA pipes: 128 x 128 tiles, 8 x 8 results per thread, 16-deep
// slices through shared memory.  The forward's tile is 64 gate and the 64 up
// columns that belong to them, so a thread holds both factors of its results.
#include <stdio.h>

#include <algorithm>

#include "common.cuh"
#include "e4m3.cuh"
#include "gated.cuh"
#include "ops.h"

namespace mlpk {

namespace {

struct GatedParams {
  const float* A; int64_t lda;      // X, or dY
  const float* B; int64_t ldb;      // W [2F, K], or Wd [K, F]
  const float* bias;               // [2F] or null
  float* h; int64_t ldh;           // (the backward's may be null)
  void* s; int64_t lds;            // kept pre-activations, or codes when se is set
  uint8_t* se; int64_t ldse;
  float* ds; int64_t ldds;         // the backward's result
  int M, F, K;
  int act;
};

constexpr int GT = 128, GK = 16;

template <bool FWD>
__global__ void __launch_bounds__(256) gated_simt_kernel(const __grid_constant__ GatedParams p) {
  pdl_enter();
  __shared__ __align__(16) float As[2][GK][GT + 4];
  __shared__ __align__(16) float Bs[2][GK][GT + 4];
  constexpr int PER = GT * GK / 256;
  constexpr int TF = FWD ? GT / 2 : GT;   // F columns per tile
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int m0 = blockIdx.y * GT, f0 = blockIdx.x * TF;
  const float* A = p.A;
  const float* B = p.B;
  float ra[PER], rb[PER];
  auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int idx = tid + i * 256, m = idx / GK, k = k0 + idx % GK;
      ra[i] = (m0 + m < p.M && k < p.K) ? A[(int64_t)(m0 + m) * p.lda + k] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int idx = tid + i * 256;
      if (FWD) {   // tile column n: gate row f0 + n, or up row F + f0 + n - 64
        const int n = idx / GK, k = k0 + idx % GK, f = f0 + (n & (TF - 1));
        rb[i] = (f < p.F && k < p.K) ? B[((int64_t)f + (n < TF ? 0 : p.F)) * p.ldb + k] : 0.f;
      } else {
        const int n = idx % GT, k = k0 + idx / GT;
        rb[i] = (f0 + n < p.F && k < p.K) ? B[(int64_t)k * p.ldb + f0 + n] : 0.f;
      }
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int idx = tid + i * 256;
      As[buf][idx % GK][idx / GK] = ra[i];
      if (FWD) Bs[buf][idx % GK][idx / GK] = rb[i];
      else Bs[buf][idx / GT][idx % GT] = rb[i];
    }
  };
  float acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  load(0);
  store(0);
  __syncthreads();
  const int nt = (p.K + GK - 1) / GK;
  for (int t = 0; t < nt; ++t) {
    const int cur = t & 1;
    if (t + 1 < nt) load((t + 1) * GK);
#pragma unroll
    for (int kk = 0; kk < GK; ++kk) {
      float a[8], b[8];
      *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(&As[cur][kk][ty * 4]);
      *reinterpret_cast<float4*>(a + 4) = *reinterpret_cast<const float4*>(&As[cur][kk][64 + ty * 4]);
      *reinterpret_cast<float4*>(b) = *reinterpret_cast<const float4*>(&Bs[cur][kk][tx * 4]);
      *reinterpret_cast<float4*>(b + 4) = *reinterpret_cast<const float4*>(&Bs[cur][kk][64 + tx * 4]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    if (t + 1 < nt) store(cur ^ 1);
    __syncthreads();
  }

  // thread (ty, tx): rows ty*4 + 0..3 and 64 + ty*4 + 0..3; tile columns
  // tx*4 + 0..3 and 64 + tx*4 + 0..3 (the forward's second four are the up
  // columns of its first four)
  float* h = p.h;
  const int64_t nb = q8_blocks(p.F);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + (i < 4 ? ty * 4 + i : 60 + ty * 4 + i);
    const bool row_ok = m < p.M;
    if (FWD) {
      const int f = f0 + tx * 4;
      float g[4], u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = f + j < p.F;
        g[j] = in ? acc[i][j] + (p.bias ? p.bias[f + j] : 0.f) : 0.f;
        u[j] = in ? acc[i][4 + j] + (p.bias ? p.bias[p.F + f + j] : 0.f) : 0.f;
      }
      if (p.se) {
        // the eight threads of a 32-column block are neighbours
        uint32_t mg = 0, mu = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mg = max(mg, q8_mag(g[j]));
          mu = max(mu, q8_mag(u[j]));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          mg = max(mg, __shfl_xor_sync(0xffffffffu, mg, o));
          mu = max(mu, __shfl_xor_sync(0xffffffffu, mu, o));
        }
        const int kg = q8_exponent(mg), ku = q8_exponent(mu);
        const float sg = q8_pow2(-kg), su = q8_pow2(-ku);
        const uint32_t cg = q8_pack(q8_no_inf(g[0]) * sg, q8_no_inf(g[1]) * sg, q8_no_inf(g[2]) * sg,
                                    q8_no_inf(g[3]) * sg);
        const uint32_t cu = q8_pack(q8_no_inf(u[0]) * su, q8_no_inf(u[1]) * su, q8_no_inf(u[2]) * su,
                                    q8_no_inf(u[3]) * su);
        uint8_t* q = reinterpret_cast<uint8_t*>(p.s) + (int64_t)m * p.lds;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (row_ok && f + j < p.F) {
            q[f + j] = (uint8_t)(cg >> (8 * j));
            q[p.F + f + j] = (uint8_t)(cu >> (8 * j));
          }
        if (row_ok && f < p.F && (f & 31) == 0) {
          p.se[(int64_t)m * p.ldse + (f >> 5)] = (uint8_t)(kg + 127);
          p.se[(int64_t)m * p.ldse + nb + (f >> 5)] = (uint8_t)(ku + 127);
        }
      } else if (p.s && row_ok) {
        float* s = reinterpret_cast<float*>(p.s) + (int64_t)m * p.lds;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (f + j < p.F) {
            s[f + j] = g[j];
            s[p.F + f + j] = u[j];
          }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (row_ok && f + j < p.F) h[(int64_t)m * p.ldh + f + j] = gate_act(g[j], p.act) * u[j];
    } else if (row_ok) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int f = f0 + (j < 4 ? tx * 4 + j : 60 + tx * 4 + j);
        if (f >= p.F) continue;
        float g, u;
        if (p.se) {
          const uint8_t* q = reinterpret_cast<const uint8_t*>(p.s) + (int64_t)m * p.lds;
          const uint8_t* e = p.se + (int64_t)m * p.ldse + (f >> 5);
          g = q8_value(q[f], e[0]);
          u = q8_value(q[p.F + f], e[nb]);
        } else {
          const float* s = reinterpret_cast<const float*>(p.s) + (int64_t)m * p.lds;
          g = s[f];
          u = s[p.F + f];
        }
        float a, da;
        gate_act_grad(g, p.act, a, da);
        const float d = acc[i][j];
        float* o = p.ds + (int64_t)m * p.ldds + f;
        o[0] = d * u * da;
        o[p.F] = d * a;
        if (h) h[(int64_t)m * p.ldh + f] = a * u;
      }
    }
  }
}

}  // namespace

int gated_plan(const GatedOp& op, LaunchRec* rec, char* err, size_t errlen) {
  if (op.M < 1 || op.F < 1 || op.K < 1 || op.M > INT32_MAX || op.F > INT32_MAX / 2 || op.K > INT32_MAX - GK) {
    snprintf(err, errlen, "bad gated shape M=%lld F=%lld K=%lld", (long long)op.M, (long long)op.F, (long long)op.K);
    return -1;
  }
  if (op.dtype == DT_BF16) return gated_tc_plan(op, rec, err, errlen);
  const GatedParams p{(const float*)op.A, op.lda, (const float*)op.B, op.ldb, op.bias, (float*)op.h, op.ldh,
                      op.s, op.lds, op.se, op.ldse, (float*)op.ds, op.ldds, (int)op.M, (int)op.F, (int)op.K, op.act};
  rec->func = op.fwd ? (const void*)gated_simt_kernel<true> : (const void*)gated_simt_kernel<false>;
  rec->grid = dim3((unsigned)ceil_div(op.F, op.fwd ? GT / 2 : GT), (unsigned)ceil_div(op.M, GT));
  if (rec->grid.y > 65535) {
    snprintf(err, errlen, "gated: %lld rows are too many", (long long)op.M);
    return -1;
  }
  rec->block = dim3(256);
  rec->smem = 0;
  rec->name = op.fwd ? "gated_fwd" : "gated_dgrad";
  rec->set_args(p);
  return 1;
}

}  // namespace mlpk
