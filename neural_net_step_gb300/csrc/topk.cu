// The k largest entries of every row of logits [B, C] with the log-sums of
// the whole row and of what is left of it:
//   v_j, i_j  in descending order, lowest column first among equals,
//   lse = log sum_i exp(z_i / T),  tail = log sum_{i not taken} exp(z_i / T).
//
// Bound by DRAM: the row is read once into shared memory and everything else
// happens there.
//   1. Every thread keeps the largest of each of its units.  The smallest, over the
//      warps, of each warp's ceil(k / warps)-th largest lane is a threshold that at
//      least k elements reach, and not many more do where the row is in no
//      particular order.
//   2. The elements that reach it are the candidates; each counts those before it,
//      which is its place (where they are many, warps sort them 32 at a time and
//      each searches the other runs).  Where they are too many (equal values,
//      sorted rows) or too few (padding, NaN), the k-th largest is found by halving
//      the range of keys, then of columns among equals, counting each time.
//   3. The elements taken become -infinity in shared memory, and the sum of the
//      others is relative to the smallest taken: the tail needs no subtraction
//      and cannot underflow before its largest term does.
// The blocks of a cluster do this for their slices and send lists and sums to the
// first, which finds the entries' places in the row and adds what a slice took
// and the row does not to the rest.
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
  c.threads = units <= 256 ? 128 : units < 4096 ? 256 : 512;   // (a row's phase adds a unit)
  while (c.threads < 2 * k && c.threads < 512) c.threads *= 2;
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
  Red red[3];
  uint32_t tau[16];
  int count;
  int total[16];
  float2 part[8];                   // of each block of the cluster: reference and sum of the rest
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
template <typename U>
__device__ __forceinline__ U warp_sort_down(U x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
    for (int stride = size / 2; stride > 0; stride /= 2) {
      const U y = __shfl_xor_sync(0xffffffffu, x, stride);
      x = ((lane & size) == 0) == ((lane & stride) == 0) ? max(x, y) : min(x, y);
    }
  }
  return x;
}
// The n-th largest of the warp's values, n from 1.
__device__ __forceinline__ uint32_t warp_nth(uint32_t x, int n) {
  if (n > 8) return __shfl_sync(0xffffffffu, warp_sort_down(x), n - 1);
  uint32_t m = 0;
  while (true) {
    m = __reduce_max_sync(0xffffffffu, x);
    if (--n <= 0) return m;
    const unsigned who = __ballot_sync(0xffffffffu, x == m);
    if ((threadIdx.x & 31) == __ffs(who) - 1) x = 0;
  }
}

// Candidates where the threshold did not leave a fit number of them: exactly
// those not below the kk-th largest, or the kk largest themselves.  tau: a first
// guess of the kk-th largest's key, or 0.
template <typename T>
__device__ __noinline__ void search(const Slice<T>& s, int kk, uint32_t tau, uint64_t* cand, TopkShared& sh) {
  const auto reach = [&](uint32_t key) {
    int c = 0;
    s.each([&](int, float x) { c += key_of(x) >= key; });
    return block_count(c, sh);
  };
  uint32_t v = tau;
  if (tau == 0 || tau == 0xFFFFFFFFu || reach(tau) < kk || reach(tau + 1) >= kk) {
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

// Adds to `place` how many entries of the descending lists 0 .. n - 1 but `not_in`
// are larger than e.  Lists are `len` entries long and lie one behind the other;
// eight of them are searched side by side.
__device__ __forceinline__ void add_larger(int& place, const uint64_t* lists, int n, int not_in, int len, uint64_t e) {
  const int top = 1 << (31 - __clz(len));
  for (int b0 = 0; b0 < n; b0 += 8) {
    int at[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int step = top; step > 0; step >>= 1) {
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const int to = at[b] + step;
        if (b0 + b < n && to <= len && lists[(b0 + b) * len + to - 1] > e) at[b] = to;
      }
    }
#pragma unroll
    for (int b = 0; b < 8; ++b) place += b0 + b == not_in ? 0 : at[b];
  }
}

// U: units a thread has at most.
template <typename T, bool CLUSTER, int U>
__global__ void __launch_bounds__(U <= 16 ? 256 : 512, U <= 16 ? 3 : 1) topk_kernel(const __grid_constant__ TopkParams p) {
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

  uint64_t* cand = reinterpret_cast<uint64_t*>(smem);    // [kCand]
  uint64_t* lists = cand + kCand;                        // [blocks][k], descending (0: none); the first block has all
  uint64_t* own = lists + (int64_t)rank * p.k;
  unsigned char* buf = reinterpret_cast<unsigned char*>(((uintptr_t)(lists + (int64_t)blocks * p.k) + 15) & ~(uintptr_t)15);

  Slice<T> s;
  s.load(buf, reinterpret_cast<const T*>(p.z) + row * p.ldz, rank * p.per, min(p.per, p.C - rank * p.per));
  const int kk = min(p.k, s.n);
  if (tid == 0) sh.count = 0;
  copies_wait();

  // 1. a threshold that at least kk elements reach
  float um[U], most = -INFINITY;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int v = tid + u * NT;
    um[u] = v < s.nvec ? unit_max<T>(s.units()[v]) : -INFINITY;
    most = fmaxf(most, um[u]);
  }
  const uint32_t nth = warp_nth(key_of(most), (kk + warps - 1) / warps);
  if (lane == 0) sh.tau[warp] = nth;
  __syncthreads();
  uint32_t tau = sh.tau[0];
  for (int w = 1; w < warps; ++w) tau = min(tau, sh.tau[w]);
  const float least = value_of(tau);

  // 2. candidates and their places
  uint32_t reach = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) reach |= (uint32_t)(um[u] >= least && tid + u * NT < s.nvec) << u;
  for (; reach; reach &= reach - 1) {
    const int v = tid + (__ffs(reach) - 1) * NT, i0 = v * E - s.ph;
    float x[E];
    unit_floats<T>(s.units()[v], x);
    uint32_t in = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) in |= (uint32_t)(x[e] >= least && i0 + e >= 0 && i0 + e < s.n) << e;
    int at = atomicAdd(&sh.count, __popc(in));
    for (; in && at < kCand; in &= in - 1, ++at) {
      const int i = i0 + __ffs(in) - 1;
      cand[at] = entry_of(key_of(to_f32(s.at(i))), s.lo + i);
    }
  }
  __syncthreads();
  int count = sh.count;
  if (count > kCand || count < kk) {
    search<T>(s, kk, count > kCand ? tau : 0u, cand, sh);
    count = sh.count;
  }
  if (count <= 256) {
    for (int a = tid; a < count; a += NT) {
      const uint64_t e = cand[a];
      const ulonglong2* c2 = reinterpret_cast<const ulonglong2*>(cand);
      int place = 0;
#pragma unroll 4
      for (int b = 0; b < count >> 1; ++b) {
        const ulonglong2 o = c2[b];
        place += (o.x > e) + (o.y > e);
      }
      if (count & 1) place += cand[count - 1] > e;
      if (place < kk) own[place] = e;
    }
  } else {
    const int runs = (count + 31) / 32;
    for (int r = warp; r < runs; r += warps)
      cand[r * 32 + lane] = warp_sort_down(r * 32 + lane < count ? cand[r * 32 + lane] : 0ull);
    __syncthreads();
    for (int a = tid; a < count; a += NT) {
      int place = a & 31;
      add_larger(place, cand, runs, a >> 5, 32, cand[a]);
      if (place < kk) own[place] = cand[a];
    }
  }
  __syncthreads();

  // 3. the sum of what is not taken, relative to the smallest that is
  const bool sums = p.lse || p.tail || p.stats;
  const uint64_t e = tid < kk ? own[tid] : 0;            // (at least k threads)
  float ref = 0.f, rest = 0.f;                           // (with nothing but -infinity and NaN left any reference will do)
  if (sums && kk > 0) {
    if (tid < kk) s.at(entry_col(e) - s.lo) = minus_inf<T>();
    __syncthreads();
    ref = value_of(entry_key(own[kk - 1]));
    if (ref == INFINITY) ref = block_max(max_of(s), sh.red[2]);
    if (!(ref > -INFINITY)) ref = 0.f;
    rest = block_sum(sum_exp(s, Exponent(ref, p.c)), sh.red[0]);
  }

  uint64_t* best = own;
  if (CLUSTER) {
    cluster_wait();   // (every block of the cluster runs)
    if (rank != 0) {
      if (tid < p.k) put64(in_block(smem_addr(own + tid), 0), e);
      if (tid == 0) {
        const uint32_t to = in_block(smem_addr(&sh.part[rank]), 0);
        put32(to, __float_as_uint(ref));
        put32(to + 4, __float_as_uint(rest));
      }
    } else {
      if (tid >= kk && tid < p.k) own[tid] = 0;
      if (tid == 0) sh.part[0] = make_float2(ref, rest);
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    best = cand;
    for (int a = tid; a < blocks * p.k; a += NT) {
      const uint64_t c = lists[a];
      const int from = a / p.k;
      int place = a - from * p.k;
      if (c == 0) continue;
      add_larger(place, lists, blocks, from, p.k, c);
      if (place < p.k) best[place] = c;
    }
    __syncthreads();
  }

  const uint64_t mine = tid < p.k ? best[tid] : 0;
  const float x = value_of(entry_key(mine)), first = value_of(entry_key(best[0]));
  if (tid < p.k) {
    if (p.stats) {
      p.entries[row * p.k + tid] = mine;
    } else {
      p.values[row * p.ldv + tid] = x;
      p.indices[row * p.ldi + tid] = entry_col(mine);
    }
  }
  if (!sums) return;
  const float first0 = first > -INFINITY ? first : 0.f;
  const float taken = block_sum(tid < p.k ? ex2((x - first0) * p.c) : 0.f, sh.red[1]);
  if (CLUSTER) {
    // the rests of the slices and what they took and the row does not, relative to the largest of those
    const uint64_t last = best[p.k - 1];
    ref = -INFINITY;
    for (int b = 0; b < blocks; ++b)
      if (sh.part[b].y != 0.f) ref = fmaxf(ref, sh.part[b].x);
    const float l = value_of(entry_key(last));
    if (l < INFINITY) ref = fmaxf(ref, l);
    if (!(ref > -INFINITY)) ref = 0.f;
    rest = 0.f;
    for (int a = tid; a < blocks * p.k; a += NT)
      if (lists[a] != 0 && lists[a] < last) rest += ex2((value_of(entry_key(lists[a])) - ref) * p.c);
    if (tid < blocks && sh.part[tid].y != 0.f) rest += sh.part[tid].y * ex2((sh.part[tid].x - ref) * p.c);
    rest = block_sum(rest, sh.red[0]);
  }
  if (tid == 0) {
    const float all = taken + (rest != 0.f ? rest * ex2((ref - first0) * p.c) : 0.f);
    if (p.stats) p.stats[row] = make_float2(first, all);
    if (p.lse) p.lse[row] = first0 / p.T + logf(all);
    if (p.tail) p.tail[row] = ref / p.T + logf(rest);
  }
}

// Places for the row in shared memory behind the lists.
unsigned topk_smem(const Cut& cut, int k, int es) {
  return (unsigned)(((int64_t)cut.cluster * k + kCand) * 8 + 16 + slice_buffer(cut.per, es));
}

template <typename T>
const void* topk_func(const Cut& cut) {
  if (cut.threads <= 256)   // (slices below 64 KB)
    return cut.cluster > 1 ? (const void*)topk_kernel<T, true, 16> : (const void*)topk_kernel<T, false, 16>;
  return cut.cluster > 1 ? (const void*)topk_kernel<T, true, 25> : (const void*)topk_kernel<T, false, 25>;
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
  rec->func = dtype == DT_F32 ? topk_func<float>(cut) : topk_func<__nv_bfloat16>(cut);
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
