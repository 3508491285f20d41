// The k largest entries of every row of logits [B, C] with the log-sums of
// the whole row and of what is left of it:
//   v_j, i_j  in descending order, lowest column first among equals,
//   lse = log sum_i exp(z_i / T),  tail = log sum_{i not taken} exp(z_i / T).
//
// Bound by DRAM: the row is read once into shared memory and everything else
// happens there.
//   1. Every thread finds the largest of its elements; a warp sorts its 32.  The
//      smallest, over the warps, of each warp's ceil(k / warps)-th largest is a
//      threshold that at least k elements reach, and few more do where the row
//      is in no particular order.
//   2. Elements that reach it are candidates; each counts the candidates before it,
//      which is its place.  Where they are too many (equal values, sorted rows) or
//      too few (padding, NaN), the k-th largest is found by halving the range of
//      keys, then of columns among equals, counting each time.
//   3. The elements taken become -infinity in shared memory, and the sum of the
//      others is relative to the smallest taken: the tail needs no subtraction
//      and cannot underflow before its largest term does.
// The blocks of a cluster do this for their slices; the first of them merges
// their lists (each place by binary search in the others) and adds what was
// taken from a slice but not from the row to the tail.
#include <stdio.h>

#include <algorithm>

#include "logits.cuh"
#include "ops.h"

namespace mlpk {
namespace lg {

Cut cut_rows(int64_t rows, int64_t C, int es, int k) {
  int cs = 1;
  while (cs < 8 && ceil_div(C, cs) * es > kSliceBytes) cs *= 2;
  while (cs < 8 && rows * cs * 2 <= kSMs * 2 && C / (cs * 2) >= 2048) cs *= 2;
  Cut c;
  c.cluster = cs;
  c.per = (int)round_up(ceil_div(C, cs), 16 / es);
  const int64_t units = c.per * es / 16;
  c.threads = units <= 256 ? 128 : units <= 1024 ? 256 : 512;
  if (c.threads < k) c.threads = (int)round_up(k, 128);
  return c;
}

}  // namespace lg

namespace {

using namespace lg;

struct TopkParams {
  const void* z; int64_t ldz;
  int C, k, per;
  float T, c;                       // temperature, log2(e) / T
  float* values; int64_t ldv;
  int32_t* indices; int64_t ldi;
  float* lse; float* tail;          // nullable
  // beam selection instead of the outputs above: entries [B, k] and
  // {largest logit, sum of exp(z - largest)} of each row
  uint64_t* entries; float2* stats;
  const float* scores; const uint8_t* done;
};

struct TopkShared {
  float red[4][16];
  uint32_t tau[16];
  int count;
  int total[16];
  float2 part[8];                   // of each block of the cluster: smallest taken, sum of the rest
};

// Number of set flags over the block, the same in every thread.
__device__ __forceinline__ int block_count(int v, TopkShared& sh) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.total[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) s += sh.total[w];
  return s;
}

// Lane l gets the l-th largest of the warp's values.
__device__ __forceinline__ uint32_t warp_sort_down(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
    for (int stride = size / 2; stride > 0; stride /= 2) {
      const uint32_t y = __shfl_xor_sync(0xffffffffu, x, stride);
      x = ((lane & size) == 0) == ((lane & stride) == 0) ? max(x, y) : min(x, y);
    }
  }
  return x;
}

// Candidates where the threshold did not leave a fit number of them: exactly
// those not below the kk-th largest, or the kk largest themselves.  tau: a key
// that at least kk elements reach, or 0.
template <typename T>
__device__ __noinline__ void search(const Slice<T>& s, int kk, uint32_t tau, uint64_t* cand, TopkShared& sh) {
  const auto reach = [&](uint32_t key) {
    int c = 0;
    s.each([&](int, float x) { c += key_of(x) >= key; });
    return block_count(c, sh);
  };
  uint32_t v = tau;
  if (tau == 0 || tau == 0xFFFFFFFFu || reach(tau + 1) >= kk) {
    v = 0;
    for (int b = 31; b >= 0; --b)
      if (reach(v | (1u << b)) >= kk) v |= 1u << b;
  }
  int last = s.n;   // among those equal to v: columns up to here
  if (reach(v) > kCand) {
    const int above = v == 0xFFFFFFFFu ? 0 : reach(v + 1);
    int lo = 0, hi = s.n - 1;   // the smallest column with enough of them up to it
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      int c = 0;
      s.each([&](int i, float x) { c += i <= mid && key_of(x) == v; });
      if (above + block_count(c, sh) >= kk) hi = mid;
      else lo = mid + 1;
    }
    last = lo;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  s.each([&](int i, float x) {
    const uint32_t key = key_of(x);
    if (key > v || (key == v && i <= last)) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kCand) cand[at] = entry_of(key, s.lo + i);
    }
  });
  __syncthreads();
}

// Entries of the descending list a[0..n) that are larger than e.
__device__ __forceinline__ int larger_in(const uint64_t* a, int n, uint64_t e) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] > e) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(512) topk_kernel(const __grid_constant__ TopkParams p) {
  pdl_enter();
  constexpr int E = kPer16<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ TopkShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, NT = blockDim.x, warps = NT >> 5;
  const int64_t row = blockIdx.x;
  const int rank = CLUSTER ? (int)blockIdx.z : 0, blocks = CLUSTER ? (int)gridDim.z : 1;
  // beams that offer nothing of their row: the merge knows without it
  if (p.stats && ((p.done && p.done[row]) || !(fabsf(p.scores[row]) < INFINITY))) return;
  if (CLUSTER) cluster_arrive();

  uint64_t* lists = reinterpret_cast<uint64_t*>(smem);                 // [blocks][k], in the first block: all of them
  uint64_t* out = lists + (CLUSTER ? (int64_t)blocks * p.k : 0);       // [k]
  uint64_t* cand = out + p.k;                                          // [kCand]
  unsigned char* buf = reinterpret_cast<unsigned char*>(
      ((uintptr_t)(cand + kCand) + 15) & ~(uintptr_t)15);

  Slice<T> s;
  s.load(buf, reinterpret_cast<const T*>(p.z) + row * p.ldz, rank * p.per, min(p.per, p.C - rank * p.per));
  const int kk = min(p.k, s.n);
  if (tid == 0) sh.count = 0;
  copies_wait();

  // 1. a threshold that at least kk elements reach
  float top = -INFINITY;
  for (int v = tid; v < s.nvec; v += NT) top = fmaxf(top, unit_max<T>(s.units()[v]));
  const int need = (kk + warps - 1) / warps;
  const uint32_t sorted = warp_sort_down(key_of(top));
  if (lane == (need > 0 ? need - 1 : 0)) sh.tau[warp] = sorted;
  __syncthreads();
  uint32_t tau = sh.tau[0];
  for (int w = 1; w < warps; ++w) tau = min(tau, sh.tau[w]);

  // 2. candidates and their places
  const float least = value_of(tau);
  if (key_of(top) >= tau) {
    for (int v = tid; v < s.nvec; v += NT) {
      const uint4 a = s.units()[v];
      if (!(unit_max<T>(a) >= least)) continue;
      float x[E];
      unit_floats<T>(a, x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = v * E + e - s.ph;
        if (x[e] >= least && i >= 0 && i < s.n) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kCand) cand[at] = entry_of(key_of(x[e]), s.lo + i);
        }
      }
    }
  }
  __syncthreads();
  int count = sh.count;
  if (count > kCand || count < kk) {
    search<T>(s, kk, count > kCand ? tau : 0u, cand, sh);
    count = sh.count;
  }
  for (int a = tid; a < count; a += NT) {
    const uint64_t e = cand[a];
    int place = 0;
    for (int b = 0; b < count; ++b) place += cand[b] > e;
    if (place < kk) out[place] = e;
  }
  __syncthreads();

  // 3. the sum of what is not taken, relative to the smallest that is
  const bool sums = p.lse || p.tail || p.stats;
  float ref = kk > 0 ? value_of(entry_key(out[kk - 1])) : -INFINITY, rest = 0.f;
  if (!(ref > -INFINITY)) ref = 0.f;   // (then the rest is -infinity or NaN too)
  if (sums) {
    for (int j = tid; j < kk; j += NT) s.at(entry_col(out[j]) - s.lo) = minus_inf<T>();
    __syncthreads();
    for (int v = tid; v < s.nvec; v += NT) {
      float x[E];
      unit_floats<T>(s.units()[v], x);
#pragma unroll
      for (int e = 0; e < E; ++e) rest += ex2((x[e] - ref) * p.c);   // (the difference first: ref c can overflow)
    }
    rest = block_sum(rest, sh.red[0]);
  }

  uint64_t* best = out;
  int kept = kk;
  if (CLUSTER) {
    cluster_wait();   // (every block of the cluster runs)
    const uint32_t to = in_block(smem_addr(lists + (int64_t)rank * p.k), 0);
    for (int j = tid; j < p.k; j += NT) put64(to + 8u * j, j < kk ? out[j] : 0ull);
    if (tid == 0) {
      const uint32_t t2 = in_block(smem_addr(&sh.part[rank]), 0);
      put32(t2, __float_as_uint(ref));
      put32(t2 + 4, __float_as_uint(rest));
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    // every entry's place in the row (entries of 0 are none)
    kept = min(p.k, p.C);
    for (int a = tid; a < blocks * p.k; a += NT) {
      const uint64_t e = lists[a];
      if (e == 0) continue;
      const int from = a / p.k;
      int place = a - from * p.k;
      for (int b = 0; b < blocks; ++b)
        if (b != from) place += larger_in(lists + b * p.k, p.k, e);
      if (place < kept) out[place] = e;
    }
    __syncthreads();
    if (sums) {
      // what slices took and the row does not, and the slices' rests
      const uint64_t least_e = out[kept - 1];
      ref = value_of(entry_key(least_e));
      if (!(ref > -INFINITY)) ref = 0.f;
      float more = 0.f;
      for (int a = tid; a < blocks * p.k; a += NT) {
        const uint64_t e = lists[a];
        if (e != 0 && e < least_e) more += ex2((value_of(entry_key(e)) - ref) * p.c);
      }
      if (tid < blocks && sh.part[tid].y != 0.f) more += sh.part[tid].y * ex2((sh.part[tid].x - ref) * p.c);
      rest = block_sum(more, sh.red[1]);
    }
  }

  if (p.stats) {
    float most = value_of(entry_key(best[0]));
    const float m0 = most > -INFINITY ? most : 0.f;
    float sum = 0.f;
    for (int j = tid; j < kept; j += NT) {
      p.entries[row * p.k + j] = best[j];
      sum += ex2((value_of(entry_key(best[j])) - m0) * p.c);
    }
    sum = block_sum(sum, sh.red[2]);
    if (tid == 0) p.stats[row] = make_float2(most, sum + (rest != 0.f ? rest * ex2((ref - m0) * p.c) : 0.f));
    return;
  }
  const float m0 = value_of(entry_key(best[0])) > -INFINITY ? value_of(entry_key(best[0])) : 0.f;
  float sum = 0.f;
  for (int j = tid; j < kept; j += NT) {
    const float v = value_of(entry_key(best[j]));
    p.values[row * p.ldv + j] = v;
    p.indices[row * p.ldi + j] = entry_col(best[j]);
    sum += ex2((v - m0) * p.c);
  }
  if (p.lse) {
    sum = block_sum(sum, sh.red[2]);
    if (tid == 0) p.lse[row] = m0 / p.T + logf(sum + (rest != 0.f ? rest * ex2((ref - m0) * p.c) : 0.f));
  }
  if (p.tail && tid == 0) p.tail[row] = ref / p.T + logf(rest);
}

// Places for the row in shared memory behind the lists.
unsigned topk_smem(const Cut& cut, int k, int es) {
  const int64_t lists = (cut.cluster > 1 ? (int64_t)cut.cluster * k : 0) + k + kCand;
  return (unsigned)(lists * 8 + 16 + slice_buffer(cut.per, es));
}

void topk_launch(int dtype, int64_t rows, const TopkParams& q, LaunchRec* rec) {
  const int es = dtype == DT_F32 ? 4 : 2;
  const Cut cut = cut_rows(rows, q.C, es, q.k);
  TopkParams p = q;
  p.per = cut.per;
  rec->grid = dim3((unsigned)rows, 1, (unsigned)cut.cluster);
  rec->block = dim3((unsigned)cut.threads);
  rec->cluster = (unsigned)cut.cluster;
  rec->smem = topk_smem(cut, p.k, es);
  if (dtype == DT_F32)
    rec->func = cut.cluster > 1 ? (const void*)topk_kernel<float, true> : (const void*)topk_kernel<float, false>;
  else
    rec->func = cut.cluster > 1 ? (const void*)topk_kernel<__nv_bfloat16, true>
                                : (const void*)topk_kernel<__nv_bfloat16, false>;
  rec->name = "topk";
  rec->set_args(p);
}

}  // namespace

int topk_plan(const TopkOp& op, LaunchRec* rec, char* err, size_t errlen) {
  if (op.B < 1 || op.B > INT32_MAX || op.C < 1 || op.C > kMaxC || op.k < 1 || op.k > kMaxK || op.k > op.C ||
      op.ldz < op.C || op.ldv < op.k || op.ldi < op.k) {
    snprintf(err, errlen, "topk: bad shape B=%lld C=%lld k=%lld or leading dimension", (long long)op.B,
             (long long)op.C, (long long)op.k);
    return -1;
  }
  TopkParams p{};
  p.z = op.z; p.ldz = op.ldz; p.C = (int)op.C; p.k = (int)op.k;
  p.T = op.temperature; p.c = kLog2e / op.temperature;
  p.values = op.values; p.ldv = op.ldv; p.indices = op.indices; p.ldi = op.ldi; p.lse = op.lse; p.tail = op.tail;
  topk_launch(op.dtype, op.B, p, rec);
  return 1;
}

int beam_rows_plan(const BeamSelectOp& op, int entries, uint64_t* lists, float* stats, LaunchRec* rec) {
  TopkParams p{};
  p.z = op.z; p.ldz = op.ldz; p.C = (int)op.C; p.k = entries;
  p.T = 1.f; p.c = kLog2e;
  p.entries = lists; p.stats = reinterpret_cast<float2*>(stats);
  p.scores = op.scores; p.done = op.done;
  topk_launch(op.dtype, op.batch * op.beams, p, rec);
  rec->name = "beam_rows";
  return 1;
}

}  // namespace mlpk
