// Beam search's selection once every beam's best entries are known: used by the
// kernel that finds them, where the beams of a batch entry are the blocks of a
// cluster (topk.cu), and by a kernel of its own (beam.cu).
//
// total(w, c) = score_w + z_wc - logsumexp(z_w); a finished beam offers its end token
// at its score.  Totals are formed and compared in 64 bits: scores of -50 leave an
// fp32 sum a step of 4e-6, which would make equals of tokens of different beams.
#pragma once
#include "logits.cuh"

namespace mlpk {
namespace lg {

constexpr int kMaxBeams = 32;
constexpr int kMaxOut = 64;

struct BeamOut {
  int beams, m, per, eos;           // per = min(m, C) entries of a beam
  float* scores; int32_t* parents; int32_t* tokens; uint8_t* done;   // [batch, m]; done nullable
};
// What a beam's logits are added to, and what it offers: 0 base + logit; 1 every
// token at base; 2 the end token at base, every other at -infinity.
struct __align__(16) BeamBase {
  double base;
  int kind, done;
};

// Order of totals as unsigned integers; NaN is 1, below -infinity (0: no pair).
__device__ __forceinline__ uint64_t total_key(double t) {
  const uint64_t u = (uint64_t)__double_as_longlong(t + 0.0);
  const uint64_t k = (u >> 63) ? ~u : (u | 0x8000000000000000ull);
  return t == t ? k : 1ull;
}
__device__ __forceinline__ double total_of(uint64_t k) {
  const uint64_t u = (k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k;
  return __longlong_as_double(k > 1 ? (long long)u : 0x7FF8000000000000ll);
}
// log s for a normal s > 0 to 3e-8 (fp64 is slow here: the exponent's part alone is).
__device__ __forceinline__ double log_of(float s) {
  const int u = __float_as_int(s);
  int e = (u >> 23) - 127;
  float m = __int_as_float((u & 0x007FFFFF) | 0x3F800000);
  if (m > 1.4142135f) {
    m *= 0.5f;
    ++e;
  }
  return fma((double)e, 0.693147180559945309, (double)log1pf(m - 1.f));
}

__device__ __forceinline__ bool beam_reads_row(float score, bool done) { return !done && fabsf(score) < INFINITY; }
// largest, sum: of the beam's row, sum of exp(z - largest) (not looked at where it reads none).
__device__ __forceinline__ BeamBase beam_base(float score, bool done, float largest, float sum) {
  BeamBase b{(double)score, 0, done};
  const double nan = __longlong_as_double(0x7FF8000000000000ll);
  if (!(fabsf(score) < INFINITY)) {   // (finished or not: a list has to descend)
    b.kind = 1;
    if (!(score < 0.f)) b.base = nan;
  } else if (done) {
    b.kind = 2;
  } else if (largest == -INFINITY && !(sum != 0.f)) {   // nothing but -infinity
    b.kind = 1;
    b.base = -(double)INFINITY;
  } else if (!(largest < INFINITY) || !(sum >= 0.5f)) {  // +infinity or NaN (the largest counts 1)
    b.kind = 1;
    b.base = nan;
  } else {
    b.base -= (double)largest + log_of(sum);
  }
  return b;
}

// Lists are searched eight at a time and without bounds: the merge holds them in
// places for a power of two of entries, and as many beams as eights go.
__host__ __device__ inline int merge_stride(int per) {
  int s = 1;
  while (s < per) s *= 2;
  return s;
}
__host__ __device__ inline int merge_bytes(int beams, int per) { return (beams + 7) / 8 * 8 * merge_stride(per) * 12; }

// The m best of batch entry b from every beam's `per` best entries, descending; room:
// merge_bytes in shared memory.  Pairs of equal totals go by beam, then by their place
// in the beam's list.
__device__ __forceinline__ void merge_beams(const BeamOut& p, int64_t b, const uint64_t* entries, const BeamBase* base,
                                            uint64_t* room) {
  const int S = merge_stride(p.per), shift = 31 - __clz(S), lists = (p.beams + 7) / 8 * 8;
  uint64_t* keys = room;                                     // [lists][S]
  int* toks = reinterpret_cast<int*>(room + lists * S);
  for (int a = threadIdx.x; a < lists * S; a += blockDim.x) {
    const int w = a >> shift, j = a & (S - 1);
    uint64_t key = 0;
    int tok = 0;
    if (w < p.beams && j < p.per) {
      const BeamBase o = base[w];
      if (o.kind == 0) {
        const uint64_t e = entries[w * p.per + j];
        tok = entry_col(e);
        key = total_key(o.base + (double)value_of(entry_key(e)));
      } else if (o.kind == 1) {
        tok = j;
        key = total_key(o.base);
      } else {   // the end token, then the others in order, at -infinity
        tok = j == 0 ? p.eos : j - 1 + (j - 1 >= p.eos);
        key = total_key(j == 0 ? o.base : -(double)INFINITY);
      }
    }
    keys[a] = key;
    toks[a] = tok;
  }
  __syncthreads();
  for (int a = threadIdx.x; a < p.beams * S; a += blockDim.x) {
    const int w = a >> shift;
    const uint64_t key = keys[a];
    if (key == 0) continue;
    int place = a & (S - 1);
    for (int o0 = 0; o0 < lists; o0 += 8) {   // those before this pair: larger, or equal of a lower beam
      const uint64_t* l = keys + o0 * S;
      int at[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int step = S / 2; step > 0; step >>= 1) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (l[q * S + at[q] + step - 1] > key - (o0 + q < w)) at[q] += step;
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        at[q] += l[q * S + at[q]] > key - (o0 + q < w);
        place += o0 + q != w ? at[q] : 0;
      }
    }
    if (place < p.m) {
      const int64_t at = b * p.m + place;
      p.scores[at] = (float)total_of(key);
      p.parents[at] = w;
      p.tokens[at] = toks[a];
      if (p.done) p.done[at] = (base[w].done || toks[a] == p.eos) ? 1 : 0;
    }
  }
}

}  // namespace lg
}  // namespace mlpk
