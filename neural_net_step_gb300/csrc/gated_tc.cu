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

// Producer warp, MMA warp, 16 epilogue warps.  The epilogues do 20 to 30
// instructions per element with little to overlap inside a warp: with 8 warps
// (2 per scheduler) the backward issued in a third of the cycles.
constexpr int GT_EPI_WARPS = 16;
constexpr int GT_THREADS = 64 + 32 * GT_EPI_WARPS;

// Stages of 32 KB, and per epilogue warp three boxes of 32 rows x 32 bf16
// (2 KB).  A lane computes along its own row (that is how TMEM is read), but
// a warp's global accesses go row by row, four lanes to the 64 bytes of a row:
// the boxes turn one into the other.  (Lanes reading or writing their own rows
// cost 32 cache lines per instruction; bulk-tensor stores of 64-byte rows,
// tried before, kept the TMA unit busy that the main loop needs: 218 us for
// the GELU backward at 16384 x 4096 x 1024.)
template <bool FWD> struct GtCfg {
  static constexpr int TBM = 2 * BM;
  static constexpr int TF = FWD ? 128 : 256;             // F columns per tile
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_BYTES = 128 * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = 4;
  static constexpr int EPI_WARP_BYTES = 3 * 2048;
  static constexpr int EPI_BYTES = GT_EPI_WARPS * EPI_WARP_BYTES;
  static constexpr int ACC_COLS = 256;
  static constexpr int TMEM_COLS = 2 * ACC_COLS;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + 1024 + 256;
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};

struct GtParams {
  CUtensorMap tmA;       // X or dY, box {64, 128}
  CUtensorMap tmB;       // W, box {64, 128}; Wd (MN-major), box {64, 64}
  int M, F, K;
  int num_kb, tiles_m, tiles_f, num_tiles, m_fast;
  uint32_t idesc;
  const float* bias;
  __nv_bfloat16* h; int64_t ldh;         // (the backward's may be null)
  __nv_bfloat16* s; int64_t lds;         // kept in bf16 (null: in 8 bits, or not at all)
  __nv_bfloat16* ds; int64_t ldds;       // backward
  uint8_t* q; int64_t ldq;               // codes (forward writes, backward reads)
  uint8_t* e; int64_t lde;
  int nb;                                // scale bytes of half a row
  uint32_t* err;
};

// 32 values (one row's block) as an 8-bit checkpoint: 8 words of codes; the
// scale byte is returned.  The maximum of the magnitudes skips NaN by itself;
// a block that holds an infinity takes the long way.
__device__ __forceinline__ uint32_t q8_block(const float* v, uint32_t (&w)[8]) {
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 32; ++j) a[j & 3] = fmaxf(a[j & 3], fabsf(v[j]));
  uint32_t m = __float_as_uint(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])));
  if (m >= 0x7f800000u) {
    m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) m = max(m, q8_mag(v[j]));
    const int k = q8_exponent(m);
    const float s = q8_pow2(-k);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = q8_pack(q8_no_inf(v[4 * j]) * s, q8_no_inf(v[4 * j + 1]) * s, q8_no_inf(v[4 * j + 2]) * s,
                     q8_no_inf(v[4 * j + 3]) * s);
    return (uint32_t)(k + 127);
  }
  const int k = q8_exponent(m);
  const float s = q8_pow2(-k);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = q8_pack(v[4 * j] * s, v[4 * j + 1] * s, v[4 * j + 2] * s, v[4 * j + 3] * s);
  return (uint32_t)(k + 127);
}

// Byte offset of 16-byte unit j of row r in a box (64-byte rows; units
// exchanged so that neither 8 rows' units j nor 2 whole rows share banks), and
// of 8-byte unit j of row r in a box of codes (32-byte rows).
__device__ __forceinline__ int box_at(int r, int j) { return r * 64 + ((j ^ ((r >> 1) & 3)) << 4); }
__device__ __forceinline__ int code_at(int r, int j) { return r * 32 + ((j ^ ((r >> 2) & 3)) << 3); }

// A lane's 32 values in bf16 into its row of a box.
__device__ __forceinline__ void stage_row32(uint8_t* box, int lane, const float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[8 * j + 2 * h], v[8 * j + 2 * h + 1]);
      w[h] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    *reinterpret_cast<uint4*>(box + box_at(lane, j)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// A box to rows m, m + 1, .. of a matrix at column f, clipped at M and F (F a
// multiple of 8): lane l moves units l % 4 of rows l / 4, l / 4 + 8, ..
__device__ __forceinline__ void store_box(const uint8_t* box, int lane, __nv_bfloat16* out, int64_t ld, int m, int M,
                                          int f, int F) {
  const int j = lane & 3;
  if (f + 8 * j >= F) return;
  __nv_bfloat16* o = out + f + 8 * j;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    if (m + r < M) *reinterpret_cast<uint4*>(o + (int64_t)(m + r) * ld) = *reinterpret_cast<const uint4*>(box + box_at(r, j));
  }
}

template <bool FWD, bool Q8, int ACT>
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
    // ---------------- epilogue warps 2..17: this CTA's 128 rows ----------------
    // warp w reads TMEM lanes 32 (w % 4) .. +31: lane l owns tile row
    // 32 (w % 4) + l, in the columns of its quarter of the tile
    const int q = warp & 3;
    const int quarter = (warp - 2) >> 2;
    const uint32_t stage0 = epi_base + (uint32_t)((warp - 2) * C::EPI_WARP_BYTES);
    uint8_t* box0 = base_ptr + (stage0 - base);
    uint8_t* box1 = box0 + 2048;
    uint8_t* box2 = box0 + 4096;
    const int lr = lane >> 2, lj = lane & 3;   // a lane's row and unit in row-by-row accesses
    int tc = 0;
    bool ok = true;
    // backward: the kept g and u of a 32-column chunk, fetched a chunk ahead
    // row by row: lane l holds units l % 4 (8 columns) of rows l / 4 + 8 i, and
    // the scale bytes of its own row
    constexpr int NW = FWD ? 1 : Q8 ? 8 : 16;
    uint32_t ng[NW], nu[NW];
    uint32_t ne = 0x7f7fu;
    auto fetch = [&](int m, int f) {   // rows m .., columns f ..
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = m + 8 * i + lr, c = f + 8 * lj;
        const bool in = r < p.M && c < p.F;   // (F is a multiple of 8)
        if constexpr (Q8 && !FWD) {
          const uint8_t* qr = p.q + (int64_t)r * p.ldq + c;
          const uint2 a = in ? __ldg(reinterpret_cast<const uint2*>(qr)) : make_uint2(0u, 0u);
          const uint2 b = in ? __ldg(reinterpret_cast<const uint2*>(qr + p.F)) : make_uint2(0u, 0u);
          ng[2 * i] = a.x; ng[2 * i + 1] = a.y;
          nu[2 * i] = b.x; nu[2 * i + 1] = b.y;
        } else if constexpr (!FWD) {
          const __nv_bfloat16* sr = p.s + (int64_t)r * p.lds + c;
          const uint4 a = in ? __ldg(reinterpret_cast<const uint4*>(sr)) : make_uint4(0u, 0u, 0u, 0u);
          const uint4 b = in ? __ldg(reinterpret_cast<const uint4*>(sr + p.F)) : make_uint4(0u, 0u, 0u, 0u);
          ng[4 * i] = a.x; ng[4 * i + 1] = a.y; ng[4 * i + 2] = a.z; ng[4 * i + 3] = a.w;
          nu[4 * i] = b.x; nu[4 * i + 1] = b.y; nu[4 * i + 2] = b.z; nu[4 * i + 3] = b.w;
        }
      }
      if (Q8 && m + lane < p.M && f < p.F) {
        const uint8_t* er = p.e + (int64_t)(m + lane) * p.lde + (f >> 5);
        ne = (uint32_t)__ldg(er) | ((uint32_t)__ldg(er + p.nb) << 8);
      }
    };
    for (int t = t0; t < p.num_tiles && ok; t += tstep, ++tc) {
      int m0, f0;
      origin(t, m0, f0);
      m0 += q * 32;   // this warp's rows
      const int buf = tc & 1;
      const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * C::ACC_COLS);
      if constexpr (FWD) {
        // 32 columns: gate and up
        const int f = f0 + quarter * 32;
        float bg = 0.f, bu = 0.f;   // lane j: the bias of column j, before the accumulator wait
        if (p.bias && f + lane < p.F) { bg = __ldg(p.bias + f + lane); bu = __ldg(p.bias + p.F + f + lane); }
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(tfull_bar(buf), ((uint32_t)tc >> 1) & 1u, p.err));
        if (!ok) break;
        tc_fence_after();
        float g[32], u[32];
        tmem_ld32(trow, g, quarter * 32);
        tmem_ld32(trow, u, 128 + quarter * 32);
        // this warp's part of the accumulator is in registers: hand it back to CTA 0
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead_tempty0 + 8u * (uint32_t)buf);
        if (f >= p.F) continue;   // wholly beyond F
        if (p.bias) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            g[j] += __shfl_sync(0xffffffffu, bg, j);
            u[j] += __shfl_sync(0xffffffffu, bu, j);
          }
        }
        if constexpr (Q8) {
          // a lane's 32 columns are one block (columns beyond F hold the
          // next rows of W: they count as 0)
          if (f + 32 > p.F) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (f + j >= p.F) g[j] = u[j] = 0.f;
          }
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t w[8];
            const uint32_t byte = q8_block(part ? u : g, w);
            uint8_t* box = part ? box2 : box1;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint2*>(box + code_at(lane, j)) = make_uint2(w[2 * j], w[2 * j + 1]);
            if (m0 + lane < p.M) p.e[(int64_t)(m0 + lane) * p.lde + part * p.nb + (f >> 5)] = (uint8_t)byte;
          }
        } else if (p.s) {
          stage_row32(box1, lane, g);
          stage_row32(box2, lane, u);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) g[j] = gate_act(g[j], ACT) * u[j];
        stage_row32(box0, lane, g);
        __syncwarp();
        store_box(box0, lane, p.h, p.ldh, m0, p.M, f, p.F);
        if constexpr (Q8) {
          if (f + 8 * lj < p.F) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + lr;
              if (m0 + r >= p.M) continue;
              uint8_t* o = p.q + (int64_t)(m0 + r) * p.ldq + f + 8 * lj;
              *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(box1 + code_at(r, lj));
              *reinterpret_cast<uint2*>(o + p.F) = *reinterpret_cast<const uint2*>(box2 + code_at(r, lj));
            }
          }
        } else if (p.s) {
          store_box(box1, lane, p.s, p.lds, m0, p.M, f, p.F);
          store_box(box2, lane, p.s + p.F, p.lds, m0, p.M, f, p.F);
        }
        __syncwarp();   // the boxes are read before the next tile fills them
      } else {
        if (tc == 0) fetch(m0, f0 + quarter * 64);
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(tfull_bar(buf), ((uint32_t)tc >> 1) & 1u, p.err));
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {   // 64 columns, 32 at a time
          const int f = f0 + quarter * 64 + c;
          // the fetched units into the boxes, their own rows out of them below
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (Q8) {
              *reinterpret_cast<uint2*>(box0 + code_at(8 * i + lr, lj)) = make_uint2(ng[2 * i], ng[2 * i + 1]);
              *reinterpret_cast<uint2*>(box1 + code_at(8 * i + lr, lj)) = make_uint2(nu[2 * i], nu[2 * i + 1]);
            } else {
              *reinterpret_cast<uint4*>(box0 + box_at(8 * i + lr, lj)) =
                  make_uint4(ng[4 * i], ng[4 * i + 1], ng[4 * i + 2], ng[4 * i + 3]);
              *reinterpret_cast<uint4*>(box1 + box_at(8 * i + lr, lj)) =
                  make_uint4(nu[4 * i], nu[4 * i + 1], nu[4 * i + 2], nu[4 * i + 3]);
            }
          }
          const float eg = q8_scale(ne & 0xffu), eu = q8_scale(ne >> 8);
          __syncwarp();
          float d[32];
          tmem_ld32(trow, d, quarter * 64 + c);
          if (c == 0) {
            fetch(m0, f + 32);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead_tempty0 + 8u * (uint32_t)buf);
            if (t + tstep < p.num_tiles) {
              int m1, f1;
              origin(t + tstep, m1, f1);
              fetch(m1 + q * 32, f1 + quarter * 64);
            }
          }
          uint32_t cg[Q8 ? 8 : 1], cu[Q8 ? 8 : 1];
          if constexpr (Q8) {   // all of the row's codes, before results take their place
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint2 a = *reinterpret_cast<const uint2*>(box0 + code_at(lane, j));
              const uint2 b = *reinterpret_cast<const uint2*>(box1 + code_at(lane, j));
              cg[2 * j] = a.x; cg[2 * j + 1] = a.y;
              cu[2 * j] = b.x; cu[2 * j + 1] = b.y;
            }
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // eight columns: one 16-byte unit of each box
            float g[8], u[8];
            if constexpr (Q8) {
              q8_unpack(cg[2 * j], eg, g);
              q8_unpack(cg[2 * j + 1], eg, g + 4);
              q8_unpack(cu[2 * j], eu, u);
              q8_unpack(cu[2 * j + 1], eu, u + 4);
            } else {
              const uint4 a = *reinterpret_cast<const uint4*>(box0 + box_at(lane, j));
              const uint4 b = *reinterpret_cast<const uint4*>(box1 + box_at(lane, j));
              const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                g[2 * h] = __uint_as_float(wa[h] << 16);
                g[2 * h + 1] = __uint_as_float(wa[h] & 0xFFFF0000u);
                u[2 * h] = __uint_as_float(wb[h] << 16);
                u[2 * h + 1] = __uint_as_float(wb[h] & 0xFFFF0000u);
              }
            }
            uint32_t wg[4], wu[4], wh[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              float a0, a1, d0, d1;
              gate_act_grad(g[2 * h], ACT, a0, d0);
              gate_act_grad(g[2 * h + 1], ACT, a1, d1);
              const float e0 = d[8 * j + 2 * h], e1 = d[8 * j + 2 * h + 1];
              const __nv_bfloat162 x = __floats2bfloat162_rn(e0 * u[2 * h] * d0, e1 * u[2 * h + 1] * d1);
              const __nv_bfloat162 y = __floats2bfloat162_rn(e0 * a0, e1 * a1);
              const __nv_bfloat162 z = __floats2bfloat162_rn(a0 * u[2 * h], a1 * u[2 * h + 1]);
              wg[h] = *reinterpret_cast<const uint32_t*>(&x);
              wu[h] = *reinterpret_cast<const uint32_t*>(&y);
              wh[h] = *reinterpret_cast<const uint32_t*>(&z);
            }
            *reinterpret_cast<uint4*>(box0 + box_at(lane, j)) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
            *reinterpret_cast<uint4*>(box1 + box_at(lane, j)) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
            *reinterpret_cast<uint4*>(box2 + box_at(lane, j)) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
          }
          __syncwarp();
          store_box(box0, lane, p.ds, p.ldds, m0, p.M, f, p.F);
          store_box(box1, lane, p.ds + p.F, p.ldds, m0, p.M, f, p.F);
          if (p.h) store_box(box2, lane, p.h, p.ldh, m0, p.M, f, p.F);
          __syncwarp();   // the boxes are read before the next chunk fills them
        }
      }
    }
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
template <bool FWD, bool Q8, int ACT>
const void* gated_kernel_ptr() {
  static std::once_flag once;
  std::call_once(once, [] {
    cudaFuncSetAttribute((const void*)tc::gated_cg2_kernel<FWD, Q8, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         tc::GtCfg<FWD>::SMEM_BYTES);
  });
  return (const void*)tc::gated_cg2_kernel<FWD, Q8, ACT>;
}
template <bool FWD, bool Q8>
const void* gated_pick(int act) {
  switch (act) {
    case ACT_RELU: return gated_kernel_ptr<FWD, Q8, ACT_RELU>();
    case ACT_GELU_TANH: return gated_kernel_ptr<FWD, Q8, ACT_GELU_TANH>();
    case ACT_SILU: return gated_kernel_ptr<FWD, Q8, ACT_SILU>();
    default: return gated_kernel_ptr<FWD, Q8, ACT_NONE>();
  }
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
  p.idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((op.fwd ? 0u : 1u) << 16) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
  p.bias = op.bias;
  p.h = (__nv_bfloat16*)op.h; p.ldh = op.ldh;
  p.ds = (__nv_bfloat16*)op.ds; p.ldds = op.ldds;
  if (op.se) {
    p.q = (uint8_t*)op.s; p.ldq = op.lds; p.e = op.se; p.lde = op.ldse;
  } else {
    p.s = (__nv_bfloat16*)op.s; p.lds = op.lds;
  }
  p.nb = (int)q8_blocks(op.F);
  p.err = op.err;
  rec->func = op.fwd ? (op.se ? gated_pick<true, true>(op.act) : gated_pick<true, false>(op.act))
                     : (op.se ? gated_pick<false, true>(op.act) : gated_pick<false, false>(op.act));
  rec->smem = op.fwd ? tc::GtCfg<true>::SMEM_BYTES : tc::GtCfg<false>::SMEM_BYTES;
  rec->grid = dim3((unsigned)(2 * std::min(p.num_tiles, cg2_max_clusters())));
  rec->block = dim3(tc::GT_THREADS);
  rec->name = op.fwd ? "tc2_gated_fwd" : "tc2_gated_dgrad";
  rec->set_args(p);
  return 1;
}

}  // namespace mlpk
