// The gated feed-forward projection and its vector-Jacobian product (gated.cu
// has the formulas) for bf16 on the tensor cores: CTA pairs with 2-SM MMAs.
//
// Forward: a pair's 256-column accumulator holds 128 gate columns and the 128
// up columns that belong to them.  The two CTAs of a pair each keep half of
// the B columns in shared memory, so CTA 0 loads 128 gate rows of W and CTA 1
// the 128 up rows F further down, and the accumulator of every row has both
// factors of its results side by side in TMEM: the epilogue multiplies them
// without leaving the thread.  Backward: 256 x 256 tiles of dH = dY Wd, whose
// epilogue reads the kept g and u of its tile and writes dg, du and h.
//
// What bounds them: the forward is 4 M F K flops against 2 M F (+ 4 M F kept)
// bytes, so at K = 1024 the tensor cores (0.143 ms at 16384 x 4096 x 1024)
// before DRAM (0.067 ms); the backward at N = 1024 moves 5 tensors of M F
// elements for 2 M N F flops and DRAM comes first (0.104 ms against 0.071).
// Producer, MMA and epilogue warps, barriers and waits are those of the 2-SM
// GEMM (tc_gemm.cu): the epilogue of tile i runs beside the main loop of tile
// i + 1 (double-buffered accumulator).
#include <cuda.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "e4m3.cuh"
#include "gated.cuh"
#include "ops.h"
#include "tc.cuh"

namespace mlpk {
namespace tc {

constexpr int GT_EPI_WARPS = 8;
constexpr int GT_THREADS = 64 + 32 * GT_EPI_WARPS;   // producer warp, MMA warp, 8 epilogue warps

// Stages of 32 KB and the epilogue's staging per warp.  Forward: two 32 x 64
// boxes (4 KB) that the stores of g, u and h take in turn.  Backward: two
// sets of three 32 x 32 boxes (2 KB) for dg, du and h.
template <bool FWD> struct GtCfg {
  static constexpr int TBM = 2 * BM;
  static constexpr int TF = FWD ? 128 : 256;             // F columns per tile
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_BYTES = 128 * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = FWD ? 5 : 4;
  static constexpr int EPI_WARP_BYTES = FWD ? 2 * 4096 : 6 * 2048;
  static constexpr int EPI_BYTES = GT_EPI_WARPS * EPI_WARP_BYTES;
  static constexpr int ACC_COLS = 256;
  static constexpr int TMEM_COLS = 2 * ACC_COLS;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + 1024 + 256;
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};

struct GtParams {
  CUtensorMap tmA;       // X or dY, box {64, 128}
  CUtensorMap tmB;       // W, box {64, 128}; Wd (MN-major), box {64, 64}
  CUtensorMap tmG, tmU;  // forward: the halves of S (bf16); backward: of dS
  CUtensorMap tmH;
  int M, F, K;
  int num_kb, tiles_m, tiles_f, num_tiles, m_fast;
  int act;
  int keep;              // forward: S in bf16 is wanted
  int want_h;            // backward: H is wanted
  uint32_t idesc;
  const float* bias;
  const __nv_bfloat16* s; int64_t lds;   // backward: kept in bf16
  uint8_t* q; int64_t ldq;               // codes (forward writes, backward reads)
  uint8_t* e; int64_t lde;
  int nb;                                // scale bytes of half a row
  uint32_t* err;
};

// 32 values (one row's block) as an 8-bit checkpoint: 8 words of codes; the scale byte is returned.
__device__ __forceinline__ uint32_t q8_block(const float* v, uint32_t (&w)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) m = max(m, q8_mag(v[j]));
  const int k = q8_exponent(m);
  const float s = q8_pow2(-k);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = q8_pack(v[4 * j] * s, v[4 * j + 1] * s, v[4 * j + 2] * s, v[4 * j + 3] * s);
  return (uint32_t)(k + 127);
}

template <bool FWD, bool Q8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GT_THREADS, 1)
gated_cg2_kernel(const __grid_constant__ GtParams p) {
  using C = GtCfg<FWD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw_addr);
  const uint32_t a_base = base;
  const uint32_t b_base = base + C::STAGES * C::A_BYTES;
  const uint32_t epi_base = b_base + C::STAGES * C::B_BYTES;
  const uint32_t bar_base = epi_base + C::EPI_BYTES;
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (C::STAGES + s); };
  auto tfull_bar = [&](int b) { return bar_base + 8u * (2 * C::STAGES + b); };
  auto tempty_bar = [&](int b) { return bar_base + 8u * (2 * C::STAGES + 2 + b); };
  const uint32_t tmem_slot = bar_base + 8u * (2 * C::STAGES + 4);
  volatile uint32_t* tmem_slot_ptr = reinterpret_cast<volatile uint32_t*>(base_ptr + (tmem_slot - base));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();   // 0: the CTA whose thread issues the MMAs
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 2 * GT_EPI_WARPS);   // the epilogue warps of both CTAs
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc_cg2(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  cluster_sync_all();   // both CTAs' barriers exist before either signals the other's
  tc_fence_after();
  const uint32_t tmem = *tmem_slot_ptr;
  pdl_enter();
  const uint32_t lead_full0 = mapa_cluster(full_bar(0), 0);
  const uint32_t lead_tempty0 = mapa_cluster(tempty_bar(0), 0);
  const int t0 = (int)(blockIdx.x >> 1), tstep = (int)(gridDim.x >> 1);
  auto origin = [&](int t, int& m0, int& f0) {
    if (p.m_fast) {
      m0 = (t % p.tiles_m) * C::TBM;
      f0 = (t / p.tiles_m) * C::TF;
    } else {
      m0 = (t / p.tiles_f) * C::TBM;
      f0 = (t % p.tiles_f) * C::TF;
    }
    m0 += (int)rank * BM;   // this CTA's rows
  };

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    if (lane == 0) {
      prefetch_tmap(&p.tmA);
      prefetch_tmap(&p.tmB);
      if (FWD || p.want_h) prefetch_tmap(&p.tmH);
      int it = 0;
      bool ok = true;
      for (int t = t0; t < p.num_tiles && ok; t += tstep) {
        int m0, f0;
        origin(t, m0, f0);
        // this CTA's half of the B columns: gate rows of W in CTA 0, their up rows in CTA 1; or columns of Wd
        const int nb = FWD ? f0 + (int)rank * p.F : f0 + (int)rank * 128;
        for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
          const int s = it % C::STAGES;
          const uint32_t ph = (uint32_t)(it / C::STAGES) & 1u;
          if (!mbar_wait(empty_bar(s), ph ^ 1u, p.err)) { ok = false; break; }
          if (rank == 0) mbar_expect_tx(full_bar(s), 2u * C::STAGE_BYTES);   // both CTAs' bytes
          const uint32_t fb = lead_full0 + 8u * (uint32_t)s;
          const int k0 = kb * BK;
          const uint32_t sa = a_base + s * C::A_BYTES;
          const uint32_t sb = b_base + s * C::B_BYTES;
          tma_load_2d_cg2(sa, &p.tmA, k0, m0, fb);
          if (FWD) {
            tma_load_2d_cg2(sb, &p.tmB, k0, nb, fb);
          } else {
            tma_load_2d_cg2(sb, &p.tmB, nb, k0, fb);
            tma_load_2d_cg2(sb + 8192u, &p.tmB, nb + 64, k0, fb);
          }
        }
      }
      // every stage this CTA filled has been read by the MMAs (its empty
      // barrier completed), so no copy into this CTA's memory is in flight
      for (int i = max(0, it - C::STAGES); i < it; ++i)
        mbar_wait(empty_bar(i % C::STAGES), (uint32_t)(i / C::STAGES) & 1u, p.err);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (CTA 0) ----------------
    if (rank == 0 && lane == 0) {
      constexpr uint32_t b_kstep = FWD ? 32u : 2048u;
      constexpr uint32_t b_lbo = FWD ? 16u : 8192u;
      int it = 0, tc = 0;
      bool ok = true;
      for (int t = t0; t < p.num_tiles && ok; t += tstep, ++tc) {
        const int buf = tc & 1;
        if (!mbar_wait_cluster(tempty_bar(buf), (((uint32_t)tc >> 1) & 1u) ^ 1u, p.err)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * C::ACC_COLS);
        for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (!mbar_wait(full_bar(s), (uint32_t)(it / C::STAGES) & 1u, p.err)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = a_base + s * C::A_BYTES;
          const uint32_t sb = b_base + s * C::B_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_bf16_cg2(d, sdesc(sa + kk * 32u, 16u, 1024u), sdesc(sb + kk * b_kstep, b_lbo, 1024u), p.idesc,
                         (kb > 0 || kk > 0) ? 1u : 0u);
          mma_commit_cg2(empty_bar(s));
        }
        mma_commit_cg2(tfull_bar(buf));
      }
    }
  } else {
    // ---------------- epilogue warps 2..9: this CTA's 128 rows ----------------
    // warp w reads TMEM lanes 32 (w % 4) .. +31: lane l owns tile row
    // 32 (w % 4) + l, in the columns of its half of the tile
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t stage0 = epi_base + (uint32_t)((warp - 2) * C::EPI_WARP_BYTES);
    uint8_t* stage_ptr = base_ptr + (stage0 - base);
    int tc = 0;
    bool ok = true;
    if (FWD) {
      for (int t = t0; t < p.num_tiles && ok; t += tstep, ++tc) {
        int m0, f0;
        origin(t, m0, f0);
        const int buf = tc & 1;
        const int f = f0 + half * 64, gm = m0 + q * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * C::ACC_COLS + half * 64);
        // the chunk's bias (lane j: columns j and 32 + j), before the accumulator wait
        float bg0 = 0.f, bg1 = 0.f, bu0 = 0.f, bu1 = 0.f;
        if (p.bias) {
          if (f + lane < p.F) { bg0 = __ldg(p.bias + f + lane); bu0 = __ldg(p.bias + p.F + f + lane); }
          if (f + 32 + lane < p.F) { bg1 = __ldg(p.bias + f + 32 + lane); bu1 = __ldg(p.bias + p.F + f + 32 + lane); }
        }
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(tfull_bar(buf), ((uint32_t)tc >> 1) & 1u, p.err));
        if (!ok) break;
        tc_fence_after();
        float g[64], u[64];
        tmem_ld64(trow, g);
        tmem_ld64(trow + 128u, u);
        // this warp's part of the accumulator is in registers: hand it back to CTA 0
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead_tempty0 + 8u * (uint32_t)buf);
        if (f >= p.F) continue;   // wholly beyond F
        if (p.bias) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            g[j] += __shfl_sync(0xffffffffu, bg0, j);
            g[32 + j] += __shfl_sync(0xffffffffu, bg1, j);
            u[j] += __shfl_sync(0xffffffffu, bu0, j);
            u[32 + j] += __shfl_sync(0xffffffffu, bu1, j);
          }
        }
        uint8_t* srow = stage_ptr + lane * 128;
        if (Q8) {
          // a lane's 64 columns are two whole blocks (columns beyond F hold
          // the next rows of W: they count as 0)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int fb = f + 32 * b;
            if (fb + 32 > p.F) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (fb + j >= p.F) g[32 * b + j] = u[32 * b + j] = 0.f;
            }
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t w[8];
              const uint32_t byte = q8_block((part ? u : g) + 32 * b, w);
              if (gm < p.M && fb < p.F) {
                uint8_t* qr = p.q + (int64_t)gm * p.ldq + (int64_t)part * p.F + fb;
#pragma unroll
                for (int j = 0; j < 4; ++j)   // (F is a multiple of 8)
                  if (fb + 8 * j < p.F) *reinterpret_cast<uint2*>(qr + 8 * j) = make_uint2(w[2 * j], w[2 * j + 1]);
                p.e[(int64_t)gm * p.lde + part * p.nb + (fb >> 5)] = (uint8_t)byte;
              }
            }
          }
        } else if (p.keep) {
          // g and u through the two staging boxes and TMA stores (which clip the ragged edges)
          if (lane == 0) bulk_wait_read0();
          __syncwarp();
          stage_plane(srow, lane, g, false);
          stage_plane(srow + 4096, lane, u, false);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.tmG, stage0, f, m0 + q * 32);
            bulk_commit();
            tma_store_2d(&p.tmU, stage0 + 4096u, f, m0 + q * 32);
            bulk_commit();
          }
        }
        if (p.act == ACT_SILU) {
#pragma unroll
          for (int j = 0; j < 64; ++j) g[j] = gate_act(g[j], ACT_SILU) * u[j];
        } else if (p.act == ACT_GELU_TANH) {
#pragma unroll
          for (int j = 0; j < 64; ++j) g[j] = gelu_tanh(g[j]) * u[j];
        } else if (p.act == ACT_RELU) {
#pragma unroll
          for (int j = 0; j < 64; ++j) g[j] = fmaxf(g[j], 0.f) * u[j];
        } else {
#pragma unroll
          for (int j = 0; j < 64; ++j) g[j] *= u[j];
        }
        // h through the first box, free once g's store (or the last tile's) has read it
        if (lane == 0) {
          if (!Q8 && p.keep) bulk_wait_read1();
          else bulk_wait_read0();
        }
        __syncwarp();
        stage_plane(srow, lane, g, false);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&p.tmH, stage0, f, m0 + q * 32);
          bulk_commit();
        }
      }
    } else {
      int set = 0;
      for (int t = t0; t < p.num_tiles && ok; t += tstep, ++tc) {
        int m0, f0;
        origin(t, m0, f0);
        const int buf = tc & 1;
        const int gm = m0 + q * 32 + lane;
        const bool row_ok = gm < p.M;
        const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * C::ACC_COLS + half * 128);
        // the kept g and u of 32 columns: bf16 pairs (16 words each) or codes (8 words each) and scales
        constexpr int NW = Q8 ? 8 : 16;
        uint32_t ng[NW], nu[NW];
        uint32_t ne = 0;
        auto fetch = [&](int c) {
          const int f = f0 + half * 128 + c;
          ne = 0x7f7fu;
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // eight columns at a time (F is a multiple of 8)
            const bool in = row_ok && f + 8 * j < p.F;
            if (Q8) {
              const uint8_t* qr = p.q + (int64_t)gm * p.ldq + f + 8 * j;
              const uint2 a = in ? __ldg(reinterpret_cast<const uint2*>(qr)) : make_uint2(0u, 0u);
              const uint2 b = in ? __ldg(reinterpret_cast<const uint2*>(qr + p.F)) : make_uint2(0u, 0u);
              ng[2 * j] = a.x; ng[2 * j + 1] = a.y;
              nu[2 * j] = b.x; nu[2 * j + 1] = b.y;
            } else {
              const __nv_bfloat16* sr = p.s + (int64_t)gm * p.lds + f + 8 * j;
              const uint4 a = in ? __ldg(reinterpret_cast<const uint4*>(sr)) : make_uint4(0u, 0u, 0u, 0u);
              const uint4 b = in ? __ldg(reinterpret_cast<const uint4*>(sr + p.F)) : make_uint4(0u, 0u, 0u, 0u);
              ng[(4 * j) % NW] = a.x; ng[(4 * j + 1) % NW] = a.y; ng[(4 * j + 2) % NW] = a.z; ng[(4 * j + 3) % NW] = a.w;
              nu[(4 * j) % NW] = b.x; nu[(4 * j + 1) % NW] = b.y; nu[(4 * j + 2) % NW] = b.z; nu[(4 * j + 3) % NW] = b.w;
            }
          }
          if (Q8 && row_ok && f < p.F) {
            const uint8_t* er = p.e + (int64_t)gm * p.lde + (f >> 5);
            ne = (uint32_t)__ldg(er) | ((uint32_t)__ldg(er + p.nb) << 8);
          }
        };
        fetch(0);
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(tfull_bar(buf), ((uint32_t)tc >> 1) & 1u, p.err));
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          const int f = f0 + half * 128 + c;
          float d[32];
          tmem_ld32(trow, d, c);
          if (c == 96) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead_tempty0 + 8u * (uint32_t)buf);
          }
          if (f >= p.F) continue;   // wholly beyond F
          uint32_t cg[NW], cu[NW];
#pragma unroll
          for (int j = 0; j < NW; ++j) { cg[j] = ng[j]; cu[j] = nu[j]; }
          const float eg = q8_scale(ne & 0xffu), eu = q8_scale(ne >> 8);
          if (c < 96) fetch(c + 32);
          // the staging set of two chunks ago is free
          if (lane == 0) bulk_wait_read1();
          __syncwarp();
          uint8_t* srow = stage_ptr + set * 6144 + lane * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // eight columns: one 16-byte unit of each box
            float g[8], u[8];
            if (Q8) {
              q8_unpack(cg[2 * j], eg, g);
              q8_unpack(cg[2 * j + 1], eg, g + 4);
              q8_unpack(cu[2 * j], eu, u);
              q8_unpack(cu[2 * j + 1], eu, u + 4);
            } else {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                g[2 * h] = __uint_as_float(cg[(4 * j + h) % NW] << 16);
                g[2 * h + 1] = __uint_as_float(cg[(4 * j + h) % NW] & 0xFFFF0000u);
                u[2 * h] = __uint_as_float(cu[(4 * j + h) % NW] << 16);
                u[2 * h + 1] = __uint_as_float(cu[(4 * j + h) % NW] & 0xFFFF0000u);
              }
            }
            uint32_t wg[4], wu[4], wh[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              float a0, a1, d0, d1;
              gate_act_grad(g[2 * h], p.act, a0, d0);
              gate_act_grad(g[2 * h + 1], p.act, a1, d1);
              const float e0 = d[8 * j + 2 * h], e1 = d[8 * j + 2 * h + 1];
              const __nv_bfloat162 x = __floats2bfloat162_rn(e0 * u[2 * h] * d0, e1 * u[2 * h + 1] * d1);
              const __nv_bfloat162 y = __floats2bfloat162_rn(e0 * a0, e1 * a1);
              const __nv_bfloat162 z = __floats2bfloat162_rn(a0 * u[2 * h], a1 * u[2 * h + 1]);
              wg[h] = *reinterpret_cast<const uint32_t*>(&x);
              wu[h] = *reinterpret_cast<const uint32_t*>(&y);
              wh[h] = *reinterpret_cast<const uint32_t*>(&z);
            }
            // 64-byte rows, 64B swizzle: unit j of row r at j ^ ((r >> 1) & 3)
            const int at = (j ^ ((lane >> 1) & 3)) << 4;
            *reinterpret_cast<uint4*>(srow + at) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
            *reinterpret_cast<uint4*>(srow + 2048 + at) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
            if (p.want_h) *reinterpret_cast<uint4*>(srow + 4096 + at) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            const uint32_t st = stage0 + (uint32_t)(set * 6144);
            tma_store_2d(&p.tmG, st, f, m0 + q * 32);
            tma_store_2d(&p.tmU, st + 2048u, f, m0 + q * 32);
            if (p.want_h) tma_store_2d(&p.tmH, st + 4096u, f, m0 + q * 32);
            bulk_commit();
          }
          set ^= 1;
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other may still signal its barriers, or the
  // MMAs may still read this CTA's shared memory or write its TMEM
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg2(tmem, C::TMEM_COLS);
  }
}

}  // namespace tc

namespace {
template <bool FWD, bool Q8>
const void* gated_kernel_ptr() {
  static std::once_flag once;
  std::call_once(once, [] {
    cudaFuncSetAttribute((const void*)tc::gated_cg2_kernel<FWD, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         tc::GtCfg<FWD>::SMEM_BYTES);
  });
  return (const void*)tc::gated_cg2_kernel<FWD, Q8>;
}
}  // namespace

int gated_tc_plan(const GatedOp& op, LaunchRec* rec, char* err, size_t errlen) {
  tc::GtParams p;
  memset(&p, 0, sizeof(p));
  const int tf = op.fwd ? tc::GtCfg<true>::TF : tc::GtCfg<false>::TF;
  if (!make_tmap(&p.tmA, op.A, op.K, op.M, op.lda, 64, tc::BM, err, errlen)) return -1;
  if (op.fwd ? !make_tmap(&p.tmB, op.B, op.K, 2 * op.F, op.ldb, 64, 128, err, errlen)
             : !make_tmap(&p.tmB, op.B, op.F, op.K, op.ldb, 64, 64, err, errlen))
    return -1;
  // the halves of S / dS as matrices of F columns each, so that stores clip at F
  __nv_bfloat16* two = (__nv_bfloat16*)(op.fwd ? (op.se ? nullptr : op.s) : op.ds);
  const int64_t ld2 = op.fwd ? op.lds : op.ldds;
  auto out_map = [&](CUtensorMap* tm, const void* ptr, int64_t ld) {
    return op.fwd ? make_tmap(tm, ptr, op.F, op.M, ld, 64, 32, err, errlen)
                  : make_tmap_sw64(tm, ptr, op.F, op.M, ld, 32, 32, err, errlen);
  };
  if (two && (!out_map(&p.tmG, two, ld2) || !out_map(&p.tmU, two + op.F, ld2))) return -1;
  if (op.h && !out_map(&p.tmH, op.h, op.ldh)) return -1;
  p.M = (int)op.M; p.F = (int)op.F; p.K = (int)op.K;
  p.num_kb = (int)ceil_div(op.K, tc::BK);
  p.tiles_m = (int)ceil_div(op.M, tc::GtCfg<true>::TBM);
  p.tiles_f = (int)ceil_div(op.F, tf);
  if ((int64_t)p.tiles_m * p.tiles_f > INT32_MAX) {
    snprintf(err, errlen, "gated: too many tiles");
    return -1;
  }
  p.num_tiles = p.tiles_m * p.tiles_f;
  // rows first where A is the smaller operand, so that B is read from DRAM about once
  p.m_fast = op.M < (op.fwd ? 2 * op.F : op.F) ? 1 : 0;
  p.act = op.act;
  p.keep = two != nullptr;
  p.want_h = op.h != nullptr;
  p.idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((op.fwd ? 0u : 1u) << 16) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
  p.bias = op.bias;
  if (op.se) {
    p.q = (uint8_t*)op.s; p.ldq = op.lds; p.e = op.se; p.lde = op.ldse;
  } else if (!op.fwd) {
    p.s = (const __nv_bfloat16*)op.s; p.lds = op.lds;
  }
  p.nb = (int)q8_blocks(op.F);
  p.err = op.err;
  rec->func = op.fwd ? (op.se ? gated_kernel_ptr<true, true>() : gated_kernel_ptr<true, false>())
                     : (op.se ? gated_kernel_ptr<false, true>() : gated_kernel_ptr<false, false>());
  rec->smem = op.fwd ? tc::GtCfg<true>::SMEM_BYTES : tc::GtCfg<false>::SMEM_BYTES;
  rec->grid = dim3((unsigned)(2 * std::min(p.num_tiles, cg2_max_clusters())));
  rec->block = dim3(tc::GT_THREADS);
  rec->name = op.fwd ? "tc2_gated_fwd" : "tc2_gated_dgrad";
  rec->set_args(p);
  return 1;
}

}  // namespace mlpk
