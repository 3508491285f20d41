// The gated feed-forward projection and its vector-Jacobian product:
//   forward   s = X W^T + b with W [2F, K] (F gate rows, then F up rows),
//             g = s[:, :F], u = s[:, F:], H = act(g) * u;
//   backward  dH = dY Wd (the down projection's dgrad),
//             dS = [dH * u * act'(g) | dH * act(g)], H = act(g) * u again.
// s is kept for the backward in the dtype or in 8 bits (e4m3.cuh).
//
// bf16 runs on the tensor cores (gated_tc.cu; a few rows: gated_small.cu).  fp32
// on the FFMA pipes: tiles of 16 RM rows by 128 columns, RM x 8 results per
// thread.  The forward's tile is 64 gate and the 64 up columns that belong to
// them, so a thread holds both factors of its results.  Where there are few
// tiles, the blocks of a cluster share a tile's reduction and add their sums
// through one another's shared memory.
#include <stdio.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "f32x2.cuh"
#include "gated.cuh"
#include "ops.h"
#include "tc.cuh"

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

// Tile of 16 RM rows by GT columns, GK deep, in a ring of GSTAGES slices that
// cp.async fills an element at a time (any alignment; elements outside the
// matrices as zeros) and transposes on the way.
// Every kChunk slices (512 k) the accumulators are added to sums in shared
// memory, which keeps the error of a long reduction near that of a short one
// (K = 4000: 1.1e-6 of the result in one sequence of FMAs, 4.0e-7 so).  Ring
// and sums of two blocks fit an SM (10000 x 784 x 500, forward: 359 us, 410 with
// one block); a fourth slice, which they would not leave room for, gains
// nothing, and chunks of 256 cost 1 to 3%.
constexpr int GT = 128, GK = 16, GSTAGES = 3, kChunk = 32;

// A row of a slice: a k's elements of A, then of B, then four of padding (so
// that the transposing copies of neighbouring k meet in two lanes at most).
__host__ __device__ constexpr int simt_rows(int rm) { return rm > 4 ? 128 : 16 * rm; }
__host__ __device__ constexpr int simt_pitch(int rm) { return simt_rows(rm) + GT + 4; }

__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// RM (2, 4 .. 8) rows and 8 columns per thread: rows ty R1 .. of the tile's first
// 16 R1, and ty R2 .. of the 16 R2 after them.  In a slice the second rows of
// a thread stand four apart, so that it reads them at once whatever R2 is.
template <bool FWD, int RM, bool SPLIT>
__global__ void __launch_bounds__(256, 2) gated_simt_kernel(const __grid_constant__ GatedParams p) {
  pdl_enter();
  constexpr int BM = 16 * RM, R1 = RM < 4 ? RM : 4, R2 = RM - R1;
  constexpr int P = simt_pitch(RM), SLICE = GK * P;
  extern __shared__ __align__(16) float gated_smem[];     // [GSTAGES][GK][P], [8 RM][256]
  constexpr int TF = FWD ? GT / 2 : GT;   // F columns per tile
  const int tid = threadIdx.x;
  // a warp takes 4 x 8 threads' results: as many elements of A as of B to read
  // for them (shared memory serves half a warp at a time)
  const int tx = (tid >> 5) % 2 * 8 + tid % 8, ty = (tid >> 5) / 2 * 4 + (tid >> 3) % 4;
  const int m0 = blockIdx.y * BM, f0 = blockIdx.x * TF;
  const float* A = p.A;
  const float* B = p.B;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(gated_smem);
  // this block's slices of the reduction
  const int all = (p.K + GK - 1) / GK, parts = SPLIT ? (int)gridDim.z : 1, per = SPLIT ? (all + parts - 1) / parts : all;
  const int first = SPLIT ? (int)blockIdx.z * per : 0, nt = SPLIT ? max(0, min(all - first, per)) : all;
  auto load = [&](int t) {
    const int k0 = (first + t) * GK;
    const uint32_t as = base + (uint32_t)((t % GSTAGES) * SLICE) * 4u, bs = as + simt_rows(RM) * 4u;
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int idx = tid + i * 256, m = idx / GK, kk = idx % GK, k = k0 + kk;
      const bool in = m0 + m < p.M && k < p.K;
      const int at = R2 == 0 || m < 16 * R1 ? m : 64 + (m - 64) / (R2 ? R2 : 1) * 4 + (m - 64) % (R2 ? R2 : 1);
      copy4(as + (uint32_t)(kk * P + at) * 4u, in ? A + (int64_t)(m0 + m) * p.lda + k : A, in);
    }
#pragma unroll
    for (int i = 0; i < GT * GK / 256; ++i) {
      const int idx = tid + i * 256;
      if (FWD) {   // tile column n: gate row f0 + n, or up row F + f0 + n - 64
        const int n = idx / GK, kk = idx % GK, k = k0 + kk, f = f0 + (n & (TF - 1));
        const bool in = f < p.F && k < p.K;
        copy4(bs + (uint32_t)(kk * P + n) * 4u, in ? B + ((int64_t)f + (n < TF ? 0 : p.F)) * p.ldb + k : B, in);
      } else {
        const int n = idx % GT, kk = idx / GT, k = k0 + kk;
        const bool in = f0 + n < p.F && k < p.K;
        copy4(bs + (uint32_t)(kk * P + n) * 4u, in ? B + (int64_t)k * p.ldb + f0 + n : B, in);
      }
    }
  };
  // two columns to an accumulator: one instruction forms both products
  F2 acc2[RM][4];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc2[i][j] = pack2(0.f, 0.f);
  float* sums = gated_smem + GSTAGES * SLICE + tid;
#pragma unroll
  for (int s = 0; s < GSTAGES - 1; ++s) {
    if (s < nt) load(s);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (int t = 0; t < nt; ++t) {
    asm volatile("cp.async.wait_group %0;" ::"n"(GSTAGES - 2) : "memory");
    __syncthreads();   // slice t has landed for every thread, and slice t - 1 is read
    if (t + GSTAGES - 1 < nt) load(t + GSTAGES - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const float* As = gated_smem + (t % GSTAGES) * SLICE;
    const float* Bs = As + simt_rows(RM);
#pragma unroll
    for (int kk = 0; kk < GK; ++kk) {
      float a[8];
      if constexpr (RM == 2) {
        *reinterpret_cast<float2*>(a) = *reinterpret_cast<const float2*>(As + kk * P + ty * 2);
      } else {
        *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(As + kk * P + ty * 4);
        if constexpr (R2 > 0) *reinterpret_cast<float4*>(a + 4) = *reinterpret_cast<const float4*>(As + kk * P + 64 + ty * 4);
      }
      ulonglong2 b[2];
      b[0] = *reinterpret_cast<const ulonglong2*>(Bs + kk * P + tx * 4);
      b[1] = *reinterpret_cast<const ulonglong2*>(Bs + kk * P + 64 + tx * 4);
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        const F2 aa = pack2(a[i], a[i]);
        acc2[i][0] = fma2(aa, F2{b[0].x}, acc2[i][0]);
        acc2[i][1] = fma2(aa, F2{b[0].y}, acc2[i][1]);
        acc2[i][2] = fma2(aa, F2{b[1].x}, acc2[i][2]);
        acc2[i][3] = fma2(aa, F2{b[1].y}, acc2[i][3]);
      }
    }
    if ((t + 1) % kChunk == 0 && t + 1 < nt) {
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float* sum = sums + (i * 8 + 2 * j) * 256;
          const F2 old = t + 1 == kChunk ? pack2(0.f, 0.f) : pack2(sum[0], sum[256]);
          unpack2(add2(acc2[i][j], old), sum[0], sum[256]);
          acc2[i][j] = pack2(0.f, 0.f);
        }
    }
  }

  float acc[RM][8];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* sum = sums + (i * 8 + 2 * j) * 256;
      unpack2(nt > kChunk ? add2(acc2[i][j], pack2(sum[0], sum[256])) : acc2[i][j], acc[i][2 * j], acc[i][2 * j + 1]);
    }
  if constexpr (SPLIT) {
    // the other blocks of the cluster read them from here
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[(i * 8 + j) * 256] = acc[i][j];
    tc::cluster_sync_all();
  }
  // thread (ty, tx): its rows; tile columns tx*4 + 0..3 and 64 + tx*4 + 0..3 (the forward's second four are the up
  // columns of its first four)
  float* h = p.h;
  const int64_t nb = q8_blocks(p.F);
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int m = m0 + (i < R1 ? ty * R1 + i : 16 * R1 + ty * R2 + i - R1);
    const bool row_ok = m < p.M;
    if constexpr (SPLIT) {   // a thread's rows go round the blocks, the parts' sums are added in their order
      if (i % parts != (int)blockIdx.z) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
      for (int r = 0; r < parts; ++r) {
        const uint32_t from = tc::mapa_cluster((uint32_t)__cvta_generic_to_shared(sums + i * 8 * 256), (uint32_t)r);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] += ld_cluster(from + (uint32_t)j * 1024u);
      }
    }
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
  if constexpr (SPLIT) tc::cluster_sync_all();   // no block leaves while another reads its sums
}

// the ring, and the sums of several chunks or parts
unsigned simt_smem(int rm, bool sums) { return (unsigned)((GSTAGES * GK * simt_pitch(rm) + (sums ? 8 * rm * 256 : 0)) * 4); }
template <bool FWD, int RM, bool SPLIT>
const void* simt_kernel() {
  return (const void*)gated_simt_kernel<FWD, RM, SPLIT>;
}
template <bool FWD, bool SPLIT>
const void* simt_pick(int rm) {
  switch (rm) {
    case 8: return simt_kernel<FWD, 8, SPLIT>();
    case 7: return simt_kernel<FWD, 7, SPLIT>();
    case 6: return simt_kernel<FWD, 6, SPLIT>();
    case 5: return simt_kernel<FWD, 5, SPLIT>();
    case 4: return simt_kernel<FWD, 4, SPLIT>();
    default: return simt_kernel<FWD, 2, SPLIT>();
  }
}

// Rows per thread and parts of the reduction (a block each, in clusters along
// z) of least estimated time.  A slice of a tile takes about rm + 4 (forward of
// one tile, K = 784, rm = 2, 4 .. 8: 48, 58, 62, 66, 78, 82 us), two blocks beside
// one another on an SM 1.8 times as long, joining the parts about a slice;
// clusters of 4 and 8 blocks find room on 136 and 120 SMs; several parts have to
// promise 5%.  Of all heights and parts timed it takes the fastest or one within
// 2% at 28 of 30 sizes, and one within 13% at two.  The tallest tile (few rows: the
// lowest) in one part, and as chosen, in us:
//   forward 1 x 553 x 1379    89 (rm = 2) -> 18     backward 401 x 1592 x 1125  91 -> 58
//   forward 16 x 256 x 4000  240 (rm = 2) -> 37     backward 2500 x 900 x 600  139 -> 91
//   forward 300 x 2000 x 1000 113 -> 85             backward 1000 x 1000 x 784  97 -> 56
//   forward 2500 x 900 x 600  134, kept             forward 1000 x 1000 x 784   88 -> 85 (one part)
struct Simt { int rm, parts; };
Simt simt_choice(int64_t cols, int64_t M, int64_t K) {
  constexpr int64_t room[4] = {152, 152, 136, 120};
  const int64_t slices = ceil_div(K, GK);
  Simt best{8, 1};
  int64_t least = INT64_MAX;
  for (int i = 0; i < 4; ++i) {
    const int64_t per = ceil_div(slices, (int64_t)1 << i) + (i > 0);
    for (int r : {8, 7, 6, 5, 4, 2}) {
      const int64_t q = ceil_div((cols * ceil_div(M, 16 * r)) << i, room[i]);
      const int64_t cost = (q / 2 * 9 + q % 2 * 5) * (r + 4) * per * (i > 0 ? 20 : 19);
      if (cost < least) { least = cost; best = Simt{r, 1 << i}; }
    }
    if (cols * ceil_div(M, 128) > 8 * room[0]) break;   // (many tiles: in one part)
  }
  return best;
}

}  // namespace

int gated_plan(const GatedOp& op, LaunchRec* rec, char* err, size_t errlen) {
  if (gated_small_takes(op)) return gated_small_plan(op, rec);
  if (op.dtype == DT_BF16) return gated_tc_plan(op, rec, err, errlen);
  const GatedParams p{(const float*)op.A, op.lda, (const float*)op.B, op.ldb, op.bias, (float*)op.h, op.ldh,
                      op.s, op.lds, op.se, op.ldse, (float*)op.ds, op.ldds, (int)op.M, (int)op.F, (int)op.K, op.act};
  const int64_t cols = ceil_div(op.F, op.fwd ? GT / 2 : GT);
  const Simt t = simt_choice(cols, op.M, op.K);
  const int rm = t.rm, parts = t.parts;
  rec->func = parts > 1 ? (op.fwd ? simt_pick<true, true>(rm) : simt_pick<false, true>(rm))
                        : (op.fwd ? simt_pick<true, false>(rm) : simt_pick<false, false>(rm));
  rec->grid = dim3((unsigned)cols, (unsigned)ceil_div(op.M, 16 * rm), (unsigned)parts);
  rec->cluster = (unsigned)parts;
  if (rec->grid.y > 65535) {
    snprintf(err, errlen, "gated: %lld rows are too many", (long long)op.M);
    return -1;
  }
  rec->block = dim3(256);
  rec->smem = simt_smem(rm, parts > 1 || op.K > GK * kChunk);
  rec->name = op.fwd ? "gated_fwd" : "gated_dgrad";
  rec->set_args(p);
  return 1;
}

}  // namespace mlpk
