// Distillation from a teacher's top logits: the loss of every row and its
// gradient, hard labels besides where they are given.
//
// The teacher keeps k logits t_j of a row with their columns i_j, and the log of
// what its other columns add up to, r = log sum_{others} exp(t / T).  With
//   L = log(sum_j exp(t_j / T) + exp(r)),  p_j = exp(t_j / T - L),  p_r = exp(r - L),
//   q = softmax(z / T),  R = sum of q over the columns that are no i_j:
//   KD = sum_j p_j log(p_j / q_{i_j}) + p_r log(p_r / R),  CE = logsumexp(z) - z_y,
//   loss = w (a CE + b KD),
//   dz_i = w g (a (softmax(z)_i - [i = y]) + (b / T) (q_i - p_j             at i = i_j,
//                                                      q_i (1 - p_r / R)    elsewhere)).
//
// Bound by DRAM: the row is read once into shared memory, becomes its gradient
// there, and leaves by one bulk copy.  The k columns are taken out first (what
// stays in their place is -infinity), so the others' sum needs no subtraction,
// the pass over the row needs no test, and 1 - p_r / R is exact to fp32 however
// small R is; the k gradients are written over the row's before it leaves.
//
// Near the teacher KD is a small difference of large terms.  It is summed as
//   KD = sum over the k columns and the rest of  p log(p / q) - p + q,
// which is the same (both distributions add up to 1), and of which every term is
// positive and as exact as its p / q.
//   16384 x 32000 bf16, k = 64, T = 2: 339 us, 0.93 of the copy rate (each row read twice
// from DRAM, once to be summed and once for its gradient, it could not be below 470).  The loss
// alone 241 of 158, the row staged all the same; a gradient whose rows lie at another address
// modulo 16 516, element by element.
#pragma once
#include "distill.h"

namespace mlpk {
namespace ds {

using namespace lg;

// What a block knows of its slice's columns besides the k.
struct DistillPart {
  float most, sum, sum1;            // largest, sums of exp((z - most) / T) and exp(z - most)
  uint32_t bad;
};
struct DistillShared {
  Red red[9];
  DistillPart part[8];
  float zy;
};

template <typename T> struct BitsOf { typedef uint32_t type; };
template <> struct BitsOf<__nv_bfloat16> { typedef uint16_t type; };

// Zeros over a block's slice of the gradient: 16 bytes at a time but at its ends.
template <typename T>
__device__ __forceinline__ void clear(T* dz, int n) {
  constexpr int E = kPer16<T>;
  const int head = min(n, (int)((16 - ((uintptr_t)dz & 15)) & 15) / (int)sizeof(T)), units = (n - head) / E;
  for (int v = threadIdx.x; v < units; v += blockDim.x) reinterpret_cast<uint4*>(dz + head)[v] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < head; i += blockDim.x) dz[i] = from_f32<T>(0.f);
  for (int i = head + units * E + threadIdx.x; i < n; i += blockDim.x) dz[i] = from_f32<T>(0.f);
}

// p log(p / q) - p + q for log(p / q) = r = d / T + l: p (r - 1 + e^-r), for small r by
// its series (the terms left out are below 2^-24 of it at 1/2).  A logit masked by
// the type's lowest value can leave fp32 as d / T, but not as p d / T where p is as small.
__device__ __forceinline__ float divergence(float p, float q, float d, float T, float l) {
  if (p == 0.f) return q;
  const float r = d / T + l;
  if (!(fabsf(r) < INFINITY) && fabsf(d) < INFINITY) return fmaf(p / T, d, fmaf(p, l - 1.f, q));
  if (!(fabsf(r) < 0.5f)) return fmaf(p, r - 1.f, q);
  float h = fmaf(r, 1.f / 40320.f, -1.f / 5040.f);
  h = fmaf(r, h, 1.f / 720.f);
  h = fmaf(r, h, -1.f / 120.f);
  h = fmaf(r, h, 1.f / 24.f);
  h = fmaf(r, h, -1.f / 6.f);
  h = fmaf(r, h, 0.5f);
  return p * (r * r) * h;
}

template <typename T, bool CLUSTER, int HARD, int NT>
__global__ void __launch_bounds__(NT, NT == 32 ? 16 : NT == 64 ? 10 : NT == 128 ? 5 : NT == 256 ? 3 : 1) distill_kernel(const __grid_constant__ DistillParams p) {
  pdl_enter();
  constexpr int E = kPer16<T>;
  constexpr bool TWO = HARD != SAME;
  typedef typename BitsOf<T>::type Bits;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ DistillShared sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int rank = CLUSTER ? (int)blockIdx.z : 0, blocks = CLUSTER ? (int)gridDim.z : 1;
  const int lo = rank * p.per, n = max(0, min(p.per, p.C - lo));
  T* dz = p.dz ? reinterpret_cast<T*>(p.dz) + row * p.lddz + lo : nullptr;
  // the small reads first: behind the row's they would wait for it
  const bool mine = tid < p.k;                  // (at least k threads)
  const float w = p.w ? p.w[row] : 1.f;
  int col = mine ? p.ti[row * p.ldti + tid] : -1;
  float t = mine ? p.tv[row * p.ldtv + tid] : -INFINITY;
  const int y = p.labels ? p.labels[row] : -1;
  const float tail = p.tail ? p.tail[row] : -INFINITY;
  if (w == 0.f) {   // a row that does not count, whatever it holds
    if (dz) clear(dz, n);
    if (rank == 0 && tid == 0) p.loss[row] = 0.f;
    return;
  }

  float* zt = reinterpret_cast<float*>(smem);   // [k] the student's logits at the teacher's columns
  unsigned char* buf = smem + (p.k * 4 + 15) / 16 * 16;
  if (mine) zt[tid] = -INFINITY;
  if (CLUSTER) cluster_arrive();
  Slice<T, NT> s;
  s.load(buf, reinterpret_cast<const T*>(p.z) + row * p.ldz, lo, n);
  if (tid == 0) {
    const int64_t next = row + kAhead / blocks;
    if (next < gridDim.x && n > 0 && !(p.w && p.w[next] == 0.f))
      prefetch_row(reinterpret_cast<const T*>(p.z) + next * p.ldz, lo, n);
  }

  // ---- the teacher, while the row is on its way
  bool bad = mine && (col < -1 || col >= p.C);
  if (p.labels) bad |= y < 0 || y >= p.C;
  if (col < 0) t = -INFINITY;                   // (unused entries' values are not looked at)
  const float tm = block_max<NT>(t, sh.red[0]);
  const float tm0 = tm > -INFINITY ? tm : 0.f;
  float tref = fmaxf(tm / p.T, tail), dl = tm0 / p.T;   // a reference, and what the largest is below it
  if (!(fabsf(tref) < INFINITY)) {   // T takes the largest out of fp32 (and no tail counts beside it), or nothing is there
    dl = 0.f;
    tref = fmaxf(tref, 0.f);
  } else {
    dl -= tref;
  }
  const float pe = mine ? expf((t - tm0) / p.T + dl) : 0.f;
  const float U = expf(tail - tref);
  const float St = block_sum<NT>(pe, sh.red[1]) + U;
  const bool has = !(St == 0.f);

  // ---- the k columns out of the row
  copies_wait();
  const int own = col - lo;
  const bool here = mine && col >= 0 && own >= 0 && own < n;
  const bool label_here = p.labels && y >= lo && y < lo + n;
  const bool label_in_top = __syncthreads_or(mine && col >= 0 && col == y) != 0;   // (and the row is there)
  float ztj = -INFINITY;
  if (here) ztj = to_f32(s.at(own));
  if (label_here && tid == 0) sh.zy = to_f32(s.at(y - lo));
  __syncthreads();
  if (here) reinterpret_cast<Bits*>(s.elems())[s.ph + own] = (Bits)tid;
  __syncthreads();
  bad |= here && reinterpret_cast<Bits*>(s.elems())[s.ph + own] != (Bits)tid;   // a column given twice
  bad = __syncthreads_or(bad) != 0;
  if (here) s.at(own) = minus_inf<T>();
  __syncthreads();

  // ---- the sums over the others
  float most = block_max<NT>(max_of(s), sh.red[2]);
  const float ref = most > -INFINITY ? most : 0.f;
  float none, sum1 = 0.f, sum = sum_exp<HARD == SQUARE>(s, Exponent(ref, p.c), sum1);
  if constexpr (HARD == OTHER) sum1 = sum_exp<false>(s, Exponent(ref, kLog2e), none);
  if constexpr (TWO) block_sums<NT>(sum, sum1, sh.red[3], sh.red[4]);
  else sum = block_sum<NT>(sum, sh.red[3]);

  // ---- all slices together
  float zy = 0.f;
  if (CLUSTER) {
    cluster_wait();   // (every block of the cluster runs and has cleared its zt)
    for (int b = 0; b < blocks; ++b) {
      if (here) put32(in_block(smem_addr(zt + tid), b), __float_as_uint(ztj));
      if (tid == 0) {
        const uint32_t to = in_block(smem_addr(&sh.part[rank]), b);
        put32(to, __float_as_uint(most));
        put32(to + 4, __float_as_uint(sum));
        put32(to + 8, __float_as_uint(sum1));
        put32(to + 12, bad);
        if (label_here) put32(in_block(smem_addr(&sh.zy), b), __float_as_uint(sh.zy));
      }
    }
    cluster_arrive();
    cluster_wait();
    most = -INFINITY;   // (of all slices from here on)
    for (int b = 0; b < blocks; ++b) {
      most = fmaxf(most, sh.part[b].most);
      bad |= sh.part[b].bad != 0;
    }
    const float all = most > -INFINITY ? most : 0.f;
    sum = sum1 = 0.f;
    for (int b = 0; b < blocks; ++b) {
      const DistillPart q = sh.part[b];
      const float d = (q.most > -INFINITY ? q.most : 0.f) - all;
      if (q.sum != 0.f) sum += q.sum * ex2(d * p.c);
      if (TWO && q.sum1 != 0.f) sum1 += q.sum1 * ex2(d * kLog2e);
    }
    if (mine) ztj = zt[tid];
  }
  if (p.labels) zy = sh.zy;
  if (bad) {
    if (dz) clear(dz, n);
    if (rank == 0 && tid == 0) {
      p.loss[row] = 0.f;
      if (p.err) atomicOr(p.err, ERRBIT_LABEL_RANGE);
    }
    return;
  }
  const float rest = most > -INFINITY ? most : 0.f;   // the others' exponents are relative to this
  const float m = fmaxf(most, block_max<NT>(mine ? ztj : -INFINITY, sh.red[5]));
  const float m0 = m > -INFINITY ? m : 0.f;
  // (t - z) - (tm - m): two rows near one another leave t - z few roundings.  One far from the other (32: the usual
  // distance of an entry from its row's largest) leaves them in tm - m, and what counts is (t - tm) - (z - m).
  const bool apart = !(fabsf(tm0 - m0) < 32.f);
  const float from = apart ? tm0 : ztj, to = apart ? ztj : tm0, d = (t - from) - (to - m0);
  const float q = mine ? expf((ztj - m0) / p.T) : 0.f;
  const float f = sum != 0.f ? ex2((rest - m0) * p.c) : 0.f;
  const float S = fmaf(sum, f, block_sum<NT>(q, sh.red[6]));
  float q1 = q, f1 = f, S1 = S;
  if constexpr (TWO) {
    q1 = mine ? expf(ztj - m0) : 0.f;
    f1 = sum1 != 0.f ? ex2((rest - m0) * kLog2e) : 0.f;
    S1 = fmaf(sum1, f1, block_sum<NT>(q1, sh.red[7]));
  }
  const float pj = has ? pe / St : 0.f, pr = has ? U / St : 0.f;

  // ---- the gradient, in the row's place
  if (dz) {
    const float wg = w * p.g, kb = has ? wg * p.b * p.inv_T : 0.f, ka = p.labels ? wg * p.a : 0.f;
    float A = sum == 0.f ? 0.f : kb * (f / S - pr / sum);
    const float A1 = sum1 == 0.f && TWO ? 0.f : ka * (f1 / S1);
    if constexpr (!TWO) A += p.labels ? A1 : 0.f;
    const Exponent eg(rest, p.c), eg1(rest, kLog2e);
    A *= eg.scale;
    const float B1 = A1 * (HARD == SQUARE ? eg.scale * eg.scale : eg1.scale);
    const auto grad = [&](float x) {
      const float e = eg.one(x);
      return HARD == SAME ? e * A : HARD == SQUARE ? e * fmaf(e, B1, A) : fmaf(eg1.one(x), B1, e * A);
    };
    if (eg.far || (HARD == OTHER && eg1.far)) {
      for (int i = tid; i < s.nvec * E; i += NT) s.elems()[i] = from_f32<T>(grad(to_f32(s.elems()[i])));
    } else {
      const F2 c2 = pack2(p.c, p.c), r2 = pack2(-eg.rc, -eg.rc), A2 = pack2(A, A);
      const F2 c12 = pack2(kLog2e, kLog2e), r12 = pack2(-eg1.rc, -eg1.rc), B2 = pack2(B1, B1);
      const auto step = [&](const uint4& in) {
        uint32_t o[4];
#pragma unroll
        for (int h = 0; h < E / 2; ++h) {
          const F2 x2 = pair_of<T>(in, h);
          float x, y;
          unpack2(fma2(x2, c2, r2), x, y);
          const F2 e2 = pack2(ex2(x), ex2(y));
          F2 d;
          if constexpr (HARD == SQUARE) {
            d = mul2(e2, fma2(e2, B2, A2));
          } else {
            d = mul2(e2, A2);
            if constexpr (HARD == OTHER) {
              unpack2(fma2(x2, c12, r12), x, y);
              d = fma2(pack2(ex2(x), ex2(y)), B2, d);
            }
          }
          unpack2(d, x, y);
          if constexpr (sizeof(T) == 4) {
            o[2 * h] = __float_as_uint(x);
            o[2 * h + 1] = __float_as_uint(y);
          } else {
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(x, y);
            o[h] = *reinterpret_cast<const uint32_t*>(&b2);
          }
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
      };
      int u = 0;
      for (; u + 4 <= s.nu; u += 4) {   // (four loads in flight)
        const uint4 u0 = s.mine(u), u1 = s.mine(u + 1), u2 = s.mine(u + 2), u3 = s.mine(u + 3);
        s.mine(u) = step(u0);
        s.mine(u + 1) = step(u1);
        s.mine(u + 2) = step(u2);
        s.mine(u + 3) = step(u3);
      }
      for (; u < s.nu; ++u) s.mine(u) = step(s.mine(u));
    }
    __syncthreads();
    if (here) {
      float r = kb * (q / S - pj);
      if (p.labels) r += ka * (q1 / S1 - (col == y ? 1.f : 0.f));
      s.at(own) = from_f32<T>(r);
    }
    if (label_here && !label_in_top && tid == 0) s.at(y - lo) = from_f32<T>(grad(zy) - ka);

    // ---- and out
    if ((((uintptr_t)dz) & 15) / sizeof(T) == (unsigned)s.ph) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      const int v0 = s.ph > 0 ? 1 : 0, v1 = (s.ph + n) / E;   // the whole units
      if (tid == 0 && v1 > v0) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dz - s.ph + v0 * E),
                     "r"(smem_addr(s.units() + v0)), "r"((v1 - v0) * 16)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      if (tid < 2 * E) {   // the units that the slice only partly covers
        const int i = tid < E ? tid - s.ph : max(v1, v0) * E + (tid - E) - s.ph;
        if (i >= 0 && i < n && (tid < E ? v0 == 1 : true) && !(tid >= E && v1 < v0)) dz[i] = s.at(i);
      }
    } else {
      __syncthreads();
      for (int i = tid; i < n; i += NT) dz[i] = s.at(i);
    }
  }

  // ---- the loss, while the gradient leaves
  if (rank == 0) {
    const bool soft = has && p.b != 0.f;
    const float ln = soft ? logf(St / S) : 0.f;
    float kd = soft && mine && col >= 0 ? divergence(pj, q / S, d, p.T, dl - ln) : 0.f;
    if (p.k > 32) kd = block_sum<NT>(kd, sh.red[8]);
    else if (tid < 32) kd = warp_sum(kd);
    if (tid == 0) {
      if (soft) {
        const float R = sum * f / S;
        kd += R > 1e-30f ? divergence(pr, R, 0.f, p.T, logf(pr / R))
                         : divergence(pr, R, m0 - rest, p.T, logf(pr) - logf(sum) + logf(S));
      }
      p.loss[row] = w * (p.b * kd + (p.labels ? p.a * (logf(S1) + (m0 - zy)) : 0.f));
    }
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

template <typename T, bool CLUSTER, int HARD>
const void* distill_func(int threads) {
  if constexpr (!CLUSTER)
    if (threads == 32) return (const void*)distill_kernel<T, CLUSTER, HARD, 32>;
  return threads == 64    ? (const void*)distill_kernel<T, CLUSTER, HARD, 64>
         : threads == 128 ? (const void*)distill_kernel<T, CLUSTER, HARD, 128>
         : threads == 256 ? (const void*)distill_kernel<T, CLUSTER, HARD, 256>
                          : (const void*)distill_kernel<T, CLUSTER, HARD, 512>;
}
template <typename T, bool CLUSTER>
const void* distill_func(int hard, int threads) {
  return hard == SAME    ? distill_func<T, CLUSTER, SAME>(threads)
         : hard == OTHER ? distill_func<T, CLUSTER, OTHER>(threads)
                         : distill_func<T, CLUSTER, SQUARE>(threads);
}
template <typename T>
const void* distill_func(bool cluster, int hard, int threads) {
  return cluster ? distill_func<T, true>(hard, threads) : distill_func<T, false>(hard, threads);
}

}  // namespace ds
}  // namespace mlpk
