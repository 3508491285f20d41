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

#include "common.cuh"
#include "e4m3.cuh"
#include "f32x2.cuh"
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

// TMEM is read a row per lane, but global memory wants whole rows: 64-byte
// pieces of rows (a warp's 32 columns) ran the backward's reads and writes at
// 3.9 TB/s together, 128-byte pieces at 5.0, 512-byte ones at 5.3.  So the
// four warps that read the same 32 TMEM lanes hand their columns to one
// another through shared memory, as one box of 32 whole tile rows, and each
// then moves 8 of the rows:
//   forward: g and u in bf16, two boxes of 32 x 256 bytes, then h in the first
//   of them (or h and the codes together);
//   backward: dH in fp32, 32 x 512 bytes, the tile's columns in two halves; the
//   gate's arithmetic is then done row by row, eight columns per lane, on g and
//   u straight from global memory (fetched four steps ahead) and its results
//   go straight back.
// Small boxes leave the main loop five stages (backward of 16384 x 4096 x 1024
// with three to five, ReLU: 163, 150, 143 us; forward with s in bf16 and two to
// five: 263, 201, 181, 173 us).
template <bool FWD> struct GtCfg {
  static constexpr int TBM = 2 * BM;
  static constexpr int TF = FWD ? 128 : 256;             // F columns per tile
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_BYTES = 128 * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;  // 32 KB
  static constexpr int STAGES = 5;
  static constexpr int EPI_GROUP_BYTES = 16384 + 256;     // box(es), and the scale bytes of 32 rows
  static constexpr int EPI_BYTES = 4 * EPI_GROUP_BYTES;
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
  int e_words;                           // scale bytes may be written four at a time
  uint32_t* err;
};

// 32 values (one row's block) as an 8-bit checkpoint: 8 words of codes; the
// scale byte is returned.  The maximum of the magnitudes skips NaN by itself;
// a block that holds an infinity takes the long way (and v loses it).
__device__ __forceinline__ uint32_t q8_block(float (&v)[32], uint32_t (&w)[8]) {
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 32; ++j) a[j & 3] = fmaxf(a[j & 3], fabsf(v[j]));
  uint32_t m = __float_as_uint(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])));
  if (m >= 0x7f800000u) {
    m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      m = max(m, q8_mag(v[j]));
      v[j] = q8_no_inf(v[j]);
    }
  }
  const int k = q8_exponent(m);
  const float s = q8_pow2(-k);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = q8_pack(v[4 * j] * s, v[4 * j + 1] * s, v[4 * j + 2] * s, v[4 * j + 3] * s);
  return (uint32_t)(k + 127);
}

// Barrier `id` over the 128 threads of four warps; true where every one of
// them arrives with `ok` (so that they give up together).
__device__ __forceinline__ bool group_sync(uint32_t id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(id)
      : "memory");
  return r != 0;
}

// Hand a drained accumulator back.  Relaxed: the MMAs that follow overwrite
// only what this thread's TMEM loads have already returned; a release would
// wait for the epilogue's outstanding global stores (3% of the backward).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(F2 x) {
  float a, b;
  unpack2(x, a, b);
  const __nv_bfloat162 b2 = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&b2);
}

// Byte offsets in the boxes: 16-byte unit j (0..15) of row r with 256-byte
// rows, 8-byte unit j (0..15) of a row of codes (128 bytes), 16-byte unit j
// (0..31) of a row of fp32 (512 bytes).  Units are exchanged so that neither
// the same unit of a quarter-warp's rows nor a quarter-warp's units of one row
// share banks (fp32: units 2 l and 2 l + 1 of lane l).
__device__ __forceinline__ int box_at(int r, int j) { return r * 256 + ((j ^ (r & 7)) << 4); }
__device__ __forceinline__ int code_at(int r, int j) { return r * 128 + ((j ^ (r & 15)) << 3); }
__device__ __forceinline__ int fbox_at(int r, int j) { return r * 512 + ((j ^ ((j >> 3) & 1) ^ (r & 7)) << 4); }

// A lane's 32 values in bf16 into its row of a box, from unit j0 on.
__device__ __forceinline__ void stage_row32(uint8_t* box, int lane, int j0, const float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[8 * j + 2 * h], v[8 * j + 2 * h + 1]);
      w[h] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    *reinterpret_cast<uint4*>(box + box_at(lane, j0 + j)) = make_uint4(w[0], w[1], w[2], w[3]);
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
    // 32 (w % 4) + l, in the columns of its quarter of the tile; afterwards
    // it moves rows 8 quarter .. +7 of the same 32
    const int q = warp & 3;
    const int quarter = (warp - 2) >> 2;
    uint8_t* box = base_ptr + (epi_base - base) + q * C::EPI_GROUP_BYTES;
    int tc = 0;
    bool ok = true;
    // backward: the kept g and u of eight columns (8 (lane % 16) ..) of the rows
    // to come (lanes 16 .. 31 one further), as bf16 pairs or codes, four steps
    // ahead; step i of a half tile in slot i
    constexpr int AHEAD = 4, NW = FWD ? 1 : Q8 ? 2 : 4;
    uint32_t ng[AHEAD][NW], nu[AHEAD][NW];
    // scale bytes a half tile ahead: lane l holds those of row l / 4 and block
    // l % 4 of the 8 rows' gate and up parts (a load of its own for every lane
    // and step cost 20 us of 141)
    uint32_t eg = 0, eu = 0;
    auto fetch = [&](int slot, int r, int f) {   // row r, columns f ..
      const int c = f + 8 * (lane & 15);
      const bool in = r < p.M && c < p.F;   // (F is a multiple of 8)
      if constexpr (Q8 && !FWD) {
        const uint8_t* qr = p.q + (int64_t)r * p.ldq + c;
        const uint2 a = in ? __ldg(reinterpret_cast<const uint2*>(qr)) : make_uint2(0u, 0u);
        const uint2 b = in ? __ldg(reinterpret_cast<const uint2*>(qr + p.F)) : make_uint2(0u, 0u);
        ng[slot][0] = a.x; ng[slot][1] = a.y;
        nu[slot][0] = b.x; nu[slot][1] = b.y;
      } else if constexpr (!FWD) {
        const __nv_bfloat16* sr = p.s + (int64_t)r * p.lds + c;
        const uint4 a = in ? __ldg(reinterpret_cast<const uint4*>(sr)) : make_uint4(0u, 0u, 0u, 0u);
        const uint4 b = in ? __ldg(reinterpret_cast<const uint4*>(sr + p.F)) : make_uint4(0u, 0u, 0u, 0u);
        ng[slot][0] = a.x; ng[slot][1] = a.y; ng[slot][2] = a.z; ng[slot][3] = a.w;
        nu[slot][0] = b.x; nu[slot][1] = b.y; nu[slot][2] = b.z; nu[slot][3] = b.w;
      }
    };
    auto fetch_scales = [&](int m, int f) {   // rows m .. m + 7, columns f .. f + 127
      const int r = m + (lane >> 2), c = f + 32 * (lane & 3);
      if (Q8 && !FWD && r < p.M && c < p.F) {
        const uint8_t* er = p.e + (int64_t)r * p.lde + (c >> 5);
        eg = __ldg(er);
        eu = __ldg(er + p.nb);
      }
    };
    for (int t = t0; t < p.num_tiles && ok; t += tstep, ++tc) {
      int m0, f0;
      origin(t, m0, f0);
      m0 += q * 32;   // these four warps' rows
      const int buf = tc & 1;
      const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * C::ACC_COLS);
      const int mr = m0 + 8 * quarter;   // the rows this warp moves
      if constexpr (FWD) {
        // 32 columns: gate and up
        const int f = f0 + quarter * 32;
        float bg = 0.f, bu = 0.f;   // lane j: the bias of column j, before the accumulator wait
        if (p.bias && f + lane < p.F) { bg = __ldg(p.bias + f + lane); bu = __ldg(p.bias + p.F + f + lane); }
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(tfull_bar(buf), ((uint32_t)tc >> 1) & 1u, p.err));
        tc_fence_after();
        float g[32], u[32];
        tmem_ld32(trow, g, quarter * 32);
        tmem_ld32(trow, u, 128 + quarter * 32);
        // this warp's part of the accumulator is in registers: hand it back to CTA 0
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(lead_tempty0 + 8u * (uint32_t)buf);
        if (p.bias) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            g[j] += __shfl_sync(0xffffffffu, bg, j);
            u[j] += __shfl_sync(0xffffffffu, bu, j);
          }
        }
        // 16 lanes to a row: 16 bytes of bf16 or 8 codes each
        const int j = lane & 15, c = f0 + 8 * j;
        if (!Q8 && p.s) {
          stage_row32(box, lane, 4 * quarter, g);
          stage_row32(box + 8192, lane, 4 * quarter, u);
          ok = group_sync(1 + q, ok);
          if (!ok) break;
          if (c < p.F) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 2 * i + (lane >> 4), br = 8 * quarter + r, m = mr + r;
              if (m >= p.M) continue;
              __nv_bfloat16* o = p.s + (int64_t)m * p.lds + c;
              *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(box + box_at(br, j));
              *reinterpret_cast<uint4*>(o + p.F) = *reinterpret_cast<const uint4*>(box + 8192 + box_at(br, j));
            }
          }
          named_bar_sync(1 + q, 128);
        }
        {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            F2 a, da;
            gate2<ACT>(pack2(g[2 * i], g[2 * i + 1]), a, da);
            w[i] = bf16_pair(mul2(a, pack2(u[2 * i], u[2 * i + 1])));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(box + box_at(lane, 4 * quarter + i)) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        if constexpr (Q8) {
          // a lane's 32 columns are one block (columns beyond F hold the
          // next rows of W: they count as 0)
          if (f + 32 > p.F) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (f + i >= p.F) g[i] = u[i] = 0.f;
          }
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t w[8];
            const uint32_t byte = q8_block(part ? u : g, w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint2*>(box + 8192 + 4096 * part + code_at(lane, 4 * quarter + i)) =
                  make_uint2(w[2 * i], w[2 * i + 1]);
            box[16384 + 128 * part + 4 * lane + quarter] = (uint8_t)byte;
          }
        }
        ok = group_sync(1 + q, ok);
        if (!ok) break;
        if (c < p.F) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 2 * i + (lane >> 4), br = 8 * quarter + r, m = mr + r;
            if (m >= p.M) continue;
            *reinterpret_cast<uint4*>(p.h + (int64_t)m * p.ldh + c) =
                *reinterpret_cast<const uint4*>(box + box_at(br, j));
            if constexpr (Q8) {
              uint8_t* o = p.q + (int64_t)m * p.ldq + c;
              *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(box + 8192 + code_at(br, j));
              *reinterpret_cast<uint2*>(o + p.F) = *reinterpret_cast<const uint2*>(box + 12288 + code_at(br, j));
            }
          }
        }
        if constexpr (Q8) {
          // the four scale bytes of a row's gate or up blocks, a lane to each
          // (a byte at a time from every lane cost 12 us of 185)
          const int part = lane >> 3, br = 8 * quarter + (lane & 7), m = mr + (lane & 7);
          if (part < 2 && m < p.M) {
            uint8_t* o = p.e + (int64_t)m * p.lde + part * p.nb + (f0 >> 5);
            const uint32_t four = *reinterpret_cast<const uint32_t*>(box + 16384 + 128 * part + 4 * br);
            if (p.e_words && f0 + 128 <= p.F) {
              *reinterpret_cast<uint32_t*>(o) = four;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (f0 + 32 * i < p.F) o[i] = (uint8_t)(four >> (8 * i));
            }
          }
        }
        named_bar_sync(1 + q, 128);   // the boxes are read before the next tile fills them
      } else {
        const int up = lane >> 4;   // which of a step's two rows
        if (tc == 0) {
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) fetch(i, mr + 2 * i + up, f0);
          fetch_scales(mr, f0);
        }
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(tfull_bar(buf), ((uint32_t)tc >> 1) & 1u, p.err));
        tc_fence_after();
        // the rows to fetch while the second half's are worked on: the next tile's
        int next_m = p.M, next_f = 0;   // (none: nothing is read)
        if (t + tstep < p.num_tiles) {
          origin(t + tstep, next_m, next_f);
          next_m += q * 32 + 8 * quarter;
        }
#pragma unroll 1
        for (int hc = 0; hc < 256; hc += 128) {   // half a tile's columns
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float d[16];
            tmem_ld16(trow + (uint32_t)(hc + quarter * 32 + 16 * c), d);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<float4*>(box + fbox_at(lane, 8 * quarter + 4 * c + j)) =
                  make_float4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]);
          }
          if (hc > 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(lead_tempty0 + 8u * (uint32_t)buf);
          }
          ok = group_sync(1 + q, ok);
          if (!ok) break;
          const int c = f0 + hc + 8 * (lane & 15);
          const int fm = (hc == 0 ? mr : next_m) + up, ff = hc == 0 ? f0 + 128 : next_f;
          const uint32_t cg = eg, cu = eu;
          fetch_scales(fm - up, ff);
#pragma unroll
          for (int slot = 0; slot < AHEAD; ++slot) {   // two rows a step
            const int m = mr + 2 * slot + up;
            F2 g[4], u[4];
            if constexpr (Q8) {
              float v[8];
              const int from = 4 * (2 * slot + up) + ((lane & 15) >> 2);
              const float xg = q8_scale(__shfl_sync(0xffffffffu, cg, from));
              const float xu = q8_scale(__shfl_sync(0xffffffffu, cu, from));
              const F2 sg = pack2(xg, xg), su = pack2(xu, xu);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                q8_unpack(ng[slot][h], 1.0f, v);
                q8_unpack(nu[slot][h], 1.0f, v + 4);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  g[2 * h + i] = mul2(pack2(v[2 * i], v[2 * i + 1]), sg);
                  u[2 * h + i] = mul2(pack2(v[4 + 2 * i], v[5 + 2 * i]), su);
                }
              }
            } else {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                g[h] = pack2(__uint_as_float(ng[slot][h % NW] << 16), __uint_as_float(ng[slot][h % NW] & 0xFFFF0000u));
                u[h] = pack2(__uint_as_float(nu[slot][h % NW] << 16), __uint_as_float(nu[slot][h % NW] & 0xFFFF0000u));
              }
            }
            fetch(slot, fm + 2 * slot, ff);
            const int br = 8 * quarter + 2 * slot + up;
            const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(box + fbox_at(br, 2 * (lane & 15)));
            const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(box + fbox_at(br, 2 * (lane & 15) + 1));
            const F2 d[4] = {F2{lo.x}, F2{lo.y}, F2{hi.x}, F2{hi.y}};
            uint32_t wg[4], wu[4], wh[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              F2 a, da;
              gate2<ACT>(g[h], a, da);
              wg[h] = bf16_pair(mul2(mul2(d[h], u[h]), da));
              wu[h] = bf16_pair(mul2(d[h], a));
              wh[h] = bf16_pair(mul2(a, u[h]));
            }
            if (m < p.M && c < p.F) {
              __nv_bfloat16* o = p.ds + (int64_t)m * p.ldds + c;
              *reinterpret_cast<uint4*>(o) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
              *reinterpret_cast<uint4*>(o + p.F) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
              if (p.h) *reinterpret_cast<uint4*>(p.h + (int64_t)m * p.ldh + c) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
            }
          }
          named_bar_sync(1 + q, 128);   // the box is read before the next half fills it
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
  p.e_words = (uintptr_t)op.se % 4 == 0 && op.ldse % 4 == 0 && p.nb % 4 == 0;
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
