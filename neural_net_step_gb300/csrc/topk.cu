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
//   2. Every warp lists its units that reach it, then their elements that do: the
//      candidates.  Each counts those before it, which is its place; where they are
//      64 bits wide, warps sort them 32 at a time instead and each searches the
//      other runs.  Where they are too many
//      (equal values, sorted rows) or too few (padding, NaN), the k-th largest is
//      found by halving the range of keys, then of columns among equals.
//   3. The elements taken become -infinity in shared memory, and the sum of the
//      others is relative to the smallest taken, or to their own largest where that
//      leaves next to nothing: the tail needs no subtraction and does not underflow.
// The blocks of a cluster do this for their slices and send lists and sums to the
// first, which finds the entries' places in the row and adds what a slice took
// and the row does not to the rest.
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "logits.cuh"
#include "ops.h"

namespace mlpk {
namespace lg {

// A slice of at most 64 KB leaves room for three blocks on an SM.  Rows are not
// cut further where they are few: what the blocks of a cluster then have to tell
// one another takes longer than a block for the whole row (one row of 32000 bf16,
// k = 50: 6.6 us, eight blocks 8.1).
Cut cut_rows(int64_t C, int es, int threads) {
  int cs = 1;
  while (cs < 8 && ceil_div(C, cs) * es > kSliceBytes) cs *= 2;
  Cut c;
  c.cluster = cs;
  c.per = (int)round_up(ceil_div(C, cs), 16 / es);
  const int64_t units = c.per * es / 16 + 1;   // (a row's phase adds one)
  c.threads = units <= 3 * 128 && threads <= 128 ? 128 : units <= 16 * 256 && threads <= 256 ? 256 : 512;
  c.units = c.threads == 128 ? 3 : c.threads == 256 ? 16 : units <= 9 * 512 ? 9 : 24;
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
  Red red[7];
  uint32_t tau[16];                 // (16-byte aligned)
  int count;
  int total[16];
  float2 part[8];                   // of each block of the cluster: reference and sum of the rest
};

// Number of set flags over the block, the same in every thread.
template <int NT>
__device__ __forceinline__ int block_count(int v, TopkShared& sh) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.total[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int w = 0; w < NT / 32; ++w) s += sh.total[w];
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
  if (n > 4) return __shfl_sync(0xffffffffu, warp_sort_down(x), n - 1);
  while (true) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, x);
    if (--n <= 0) return m;
    if ((threadIdx.x & 31) == __ffs(__ballot_sync(0xffffffffu, x == m)) - 1) x = 0;
  }
}

// A candidate of a slice: larger is better, lower element first among equals; 0
// is none.  bf16 slices of at most 65535 elements need 32 bits.
template <typename K> struct Cand;
template <> struct Cand<uint64_t> {
  static __device__ __forceinline__ uint64_t of(float x, int i) { return entry_of(key_of(x), i); }
  static __device__ __forceinline__ int at(uint64_t c) { return entry_col(c); }
  static __device__ __forceinline__ uint32_t key(uint64_t c) { return entry_key(c); }
};
template <> struct Cand<uint32_t> {
  static __device__ __forceinline__ uint32_t of(float x, int i) {
    return (key_of(x) & 0xFFFF0000u) | (uint32_t)(0xFFFF - i);
  }
  static __device__ __forceinline__ int at(uint32_t c) { return 0xFFFF - (int)(c & 0xFFFFu); }
  // (the low half of a bf16's key: zeros, or ones below zero)
  static __device__ __forceinline__ uint32_t key(uint32_t c) {
    const uint32_t h = c & 0xFFFF0000u;
    return h == 0 ? 0u : (c & 0x80000000u) ? h : h | 0xFFFFu;
  }
};

// Candidates where the threshold did not leave a fit number of them: exactly
// those not below the kk-th largest, or the kk largest themselves.  tau: a first
// guess of the kk-th largest's key, or 0.
template <typename T, typename K, int NT>
__device__ __noinline__ void search(const Slice<T, NT>& s, int kk, uint32_t tau, K* cand, TopkShared& sh) {
  const auto reach = [&](uint32_t key) {
    int c = 0;
    s.each([&](int, float x) { c += key_of(x) >= key; });
    return block_count<NT>(c, sh);
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
      if (above + block_count<NT>(c, sh) >= kk) hi = mid;
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
      if (at < kCand) cand[at] = Cand<K>::of(x, i);
    }
  });
  __syncthreads();
}

// Entries larger than e in N lists side by side, `stride` apart, each `len` long and
// descending.  Every load has a place to go: none waits for a branch.
template <int N, typename K>
__device__ __forceinline__ void larger_in(int (&at)[N], const K* lists, int stride, int len, K e) {
#pragma unroll
  for (int b = 0; b < N; ++b) at[b] = 0;
  for (int step = 1 << (31 - __clz(len)); step > 0; step >>= 1) {
#pragma unroll
    for (int b = 0; b < N; ++b) {
      const int to = at[b] + step;
      const K v = lists[b * stride + min(to, len) - 1];
      at[b] = to <= len && v > e ? to : at[b];
    }
  }
}
// The same for runs of 32 one behind the other.
template <int N, typename K>
__device__ __forceinline__ int larger_in_runs(const K* runs, int not_in, K e) {
  int at[N], sum = 0;
#pragma unroll
  for (int b = 0; b < N; ++b) at[b] = 0;
#pragma unroll
  for (int step = 16; step > 0; step >>= 1)
#pragma unroll
    for (int b = 0; b < N; ++b)
      if (runs[b * 32 + at[b] + step - 1] > e) at[b] += step;
#pragma unroll
  for (int b = 0; b < N; ++b) {
    at[b] += runs[b * 32 + at[b]] > e;
    if (b != not_in) sum += at[b];
  }
  return sum;
}

// Sum of n over the lanes before this one and over all, n < 2^BITS.
template <int BITS>
__device__ __forceinline__ int before_lane(int n, int& all) {
  const uint32_t below = (1u << (threadIdx.x & 31)) - 1;
  int before = 0;
  all = 0;
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const uint32_t who = __ballot_sync(0xffffffffu, n >> b & 1);
    before += __popc(who & below) << b;
    all += __popc(who) << b;
  }
  return before;
}

// U: units a thread has at most.
template <typename T, bool CLUSTER, int NT, int U>
__global__ void __launch_bounds__(NT, U <= 16 ? (NT <= 256 ? 3 : 2) : 1) topk_kernel(const __grid_constant__ TopkParams p) {
  pdl_enter();
  constexpr int E = kPer16<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ TopkShared sh;
  constexpr int warps = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const int rank = CLUSTER ? (int)blockIdx.z : 0, blocks = CLUSTER ? (int)gridDim.z : 1;
  // beams that offer nothing of their row: the merge knows without it
  if (p.stats && ((p.done && p.done[row]) || !(fabsf(p.scores[row]) < INFINITY))) return;
  if (CLUSTER) cluster_arrive();

  typedef typename std::conditional<sizeof(T) == 2 && NT * U * 8 <= 65536, uint32_t, uint64_t>::type K;
  uint64_t* best = reinterpret_cast<uint64_t*>(smem);    // [k, even]: the row's, descending
  uint64_t* lists = best + ((p.k + 1) & ~1);             // [blocks][k], descending (0: none); the first block has all
  uint64_t* own = CLUSTER ? lists + (int64_t)rank * p.k : best;
  K* cand = reinterpret_cast<K*>(lists + (CLUSTER ? 8 * p.k : 0));   // [kCand]
  uint16_t* hits = reinterpret_cast<uint16_t*>(cand + kCand);                      // [kHits]
  unsigned char* buf = reinterpret_cast<unsigned char*>(((uintptr_t)(hits + kHits) + 15) & ~(uintptr_t)15);

  Slice<T, NT> s;
  s.load(buf, reinterpret_cast<const T*>(p.z) + row * p.ldz, rank * p.per, min(p.per, p.C - rank * p.per));
  const int kk = min(p.k, s.n);
  if (tid == 0) {
    sh.count = 0;
    const int64_t next = row + kAhead / blocks;
    if (next < gridDim.x && s.n > 0) prefetch_row(reinterpret_cast<const T*>(p.z) + next * p.ldz, s.lo, s.n);
  }
  copies_wait();

  // 1. a threshold that at least kk elements reach
  Most<T> um[U], most;
#pragma unroll
  for (int u0 = 0; u0 < U; u0 += 4) {   // (four loads in flight)
    if (u0 + 4 <= U && u0 + 4 <= s.nu) {
      uint4 a[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) a[q] = s.mine(u0 + q);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (u0 + q < U) um[u0 + q] = Most<T>(a[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (u0 + q < U && u0 + q < s.nu) um[u0 + q] = Most<T>(s.mine(u0 + q));
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (u0 + q < U) most.take(um[u0 + q]);
  }
  const uint32_t nth = warp_nth(key_of(most.value()), (kk + warps - 1) / warps);
  if (lane == 0) sh.tau[warp] = nth;
  __syncthreads();
  uint32_t tau = 0xFFFFFFFFu;
#pragma unroll
  for (int w = 0; w < warps; w += 4) {
    const uint4 q = *reinterpret_cast<const uint4*>(sh.tau + w);
    tau = min(tau, min(min(q.x, q.y), min(q.z, q.w)));
  }
  const float least = value_of(tau);

  // 2. candidates and their places
  uint32_t reach = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) reach |= (uint32_t)um[u].reaches(least) << u;
  constexpr int room = kHits / warps;
  uint16_t* hit = hits + warp * room;
  int n_hits;
  for (int at = before_lane<5>(__popc(reach), n_hits); reach && at < room; reach &= reach - 1, ++at)
    hit[at] = (uint16_t)(tid + (__ffs(reach) - 1) * NT);
  __syncwarp();
  if (n_hits > room && lane == 0) atomicAdd(&sh.count, kCand + 1);
  for (int a = lane; a - lane < min(n_hits, room); a += 32) {
    uint32_t in = 0;
    int v = 0;
    if (a < min(n_hits, room) && hit[a] < s.nvec) {
      v = hit[a];
      float x[E];
      unit_floats<T>(s.units()[v], x);
#pragma unroll
      for (int e = 0; e < E; ++e) in |= (uint32_t)(x[e] >= least) << e;
      if (least == -INFINITY)   // (what fills the units at a slice's ends does not count)
        for (int e = 0; e < E; ++e)
          if (v * E + e < s.ph || v * E + e >= s.ph + s.n) in &= ~(1u << e);
    }
    int n_in, at = 0;
    const int before = before_lane<4>(__popc(in), n_in);
    if (lane == 0) at = atomicAdd(&sh.count, n_in);
    at = __shfl_sync(0xffffffffu, at, 0) + before;
    for (; in && at < kCand; in &= in - 1, ++at) {
      const int i = v * E + __ffs(in) - 1 - s.ph;
      cand[at] = Cand<K>::of(to_f32(s.at(i)), i);
    }
  }
  __syncthreads();
  int count = sh.count;
  if (count > kCand || count < kk) {
    search<T>(s, kk, count > kCand ? tau : 0u, cand, sh);
    count = sh.count;
  }
  const bool sums = p.lse || p.tail || p.stats;
  const auto place_at = [&](int place, K c) {   // (an element taken leaves the row)
    const int i = Cand<K>::at(c);
    own[place] = entry_of(Cand<K>::key(c), s.lo + i);
    if (sums) s.at(i) = minus_inf<T>();
  };
  const int runs = (count + 31) / 32, width = runs <= 4 ? 4 : 8;
  for (int r = warp; r < (runs + width - 1) / width * width; r += warps)
    cand[r * 32 + lane] = warp_sort_down(r * 32 + lane < count ? cand[r * 32 + lane] : (K)0);
  __syncthreads();
  for (int a = tid; a < count; a += NT) {
    const K c = cand[a];
    int place = a & 31;
    if (width == 4) place += larger_in_runs<4>(cand, a >> 5, c);
    else
      for (int r = 0; r < runs; r += 8) place += larger_in_runs<8>(cand + r * 32, (a >> 5) - r, c);
    if (place < kk) place_at(place, c);
  }
  __syncthreads();

  // 3. the sum of what is not taken, relative to the smallest that is
  const uint64_t e = tid < kk ? own[tid] : 0;            // (at least k threads)
  const auto write = [&](uint64_t c) {
    if (p.stats) {
      p.entries[row * p.k + tid] = c;
    } else {
      p.values[row * p.ldv + tid] = value_of(entry_key(c));
      p.indices[row * p.ldi + tid] = entry_col(c);
    }
  };
  if (!CLUSTER && tid < p.k) write(e);
  float ref = 0.f, rest = 0.f;                           // (with nothing but -infinity and NaN left any reference will do)
  if (sums && kk > 0) {
    ref = value_of(entry_key(own[kk - 1]));
    if (ref == INFINITY) ref = block_max<NT>(max_of(s), sh.red[6]);
    if (!(ref > -INFINITY)) ref = 0.f;
    rest = sum_exp(s, Exponent(ref, p.c));
  }

  // where the others are so far below that nothing is left of them
  const auto look_closer = [&]() {
    if (!sums || !(rest < 0x1p-60f)) return;
    const float m = block_max<NT>(max_of(s), sh.red[3]);
    if (!(m > -INFINITY)) return;
    ref = m;
    rest = block_sum<NT>(sum_exp(s, Exponent(ref, p.c)), sh.red[4]);
  };
  if (CLUSTER) {
    rest = block_sum<NT>(rest, sh.red[0]);
    look_closer();
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
    // the k-th is no smaller than the smallest of the slices' ceil(k / blocks)-th
    // (a slice with fewer entries bounds nothing)
    const int each = (p.k + blocks - 1) / blocks;
    uint64_t bound = ~0ull;
    for (int b = 0; b < blocks; ++b) bound = min(bound, lists[b * p.k + each - 1]);
    const int groups = min(warps, blocks);   // (powers of two both)
    for (int from = warp % groups; from < blocks; from += groups) {
      for (int j = warp / groups * 32 + lane; j < p.k; j += warps / groups * 32) {
        const uint64_t c = lists[from * p.k + j];
        if (c == 0 || c < bound) break;
        int place = 0, at[8];
        larger_in(at, lists, p.k, p.k, c);   // (its own list too: its place there)
        for (int b = 0; b < 8; ++b) place += b < blocks ? at[b] : 0;
        if (place < p.k) best[place] = c;
      }
    }
    __syncthreads();
  }

  if (CLUSTER && tid < p.k) write(best[tid]);
  if (!sums) return;
  const float first = value_of(entry_key(best[0])), first0 = first > -INFINITY ? first : 0.f;
  float taken = tid < p.k ? ex2((value_of(entry_key(best[tid])) - first0) * p.c) : 0.f;
  if (CLUSTER) {
    // the rests of the slices and what they took and the row does not, relative to the largest of those
    const uint64_t last = best[p.k - 1];
    ref = -INFINITY;
    for (int b = 0; b < blocks; ++b)
      if (sh.part[b].y != 0.f) ref = fmaxf(ref, sh.part[b].x);
    float left = -INFINITY;
    for (int a = tid; a < blocks * p.k; a += NT)
      if (lists[a] != 0 && lists[a] < last) left = fmaxf(left, value_of(entry_key(lists[a])));
    ref = fmaxf(ref, block_max<NT>(left, sh.red[5]));
    if (!(ref > -INFINITY)) ref = 0.f;
    rest = 0.f;
    for (int a = tid; a < blocks * p.k; a += NT)
      if (lists[a] != 0 && lists[a] < last) rest += ex2((value_of(entry_key(lists[a])) - ref) * p.c);
    if (tid < blocks && sh.part[tid].y != 0.f) rest += sh.part[tid].y * ex2((sh.part[tid].x - ref) * p.c);
  }
  block_sums<NT>(taken, rest, sh.red[1], sh.red[2]);
  if (!CLUSTER) look_closer();
  const float all = taken + (rest != 0.f ? rest * ex2((ref - first0) * p.c) : 0.f);
  if (tid == 0) {
    if (p.stats) p.stats[row] = make_float2(first, all);
    if (p.lse) p.lse[row] = first0 / p.T + logf(all);
  }
  if (tid == 32 && p.tail) p.tail[row] = ref / p.T + logf(rest);
}

// Places for the row in shared memory behind the lists.
unsigned topk_smem(const Cut& cut, int k, int es) {
  const int64_t entries = (k + 1) / 2 * 2 + (cut.cluster > 1 ? 8 * k : 0);   // (eight lists are looked through)
  const int64_t word = es == 2 && cut.threads * cut.units * 8 <= 65536 ? 4 : 8;
  return (unsigned)(entries * 8 + kCand * word + kHits * 2 + 16 + slice_buffer(cut.per, es, cut.threads));
}

template <typename T, bool CLUSTER>
const void* topk_func(const Cut& cut) {
  if (cut.threads == 128) return (const void*)topk_kernel<T, CLUSTER, 128, 3>;
  if (cut.threads == 256) return (const void*)topk_kernel<T, CLUSTER, 256, 16>;
  return cut.units == 9 ? (const void*)topk_kernel<T, CLUSTER, 512, 9> : (const void*)topk_kernel<T, CLUSTER, 512, 24>;
}

void topk_launch(int dtype, int64_t rows, const TopkParams& q, LaunchRec* rec) {
  const int es = dtype == DT_F32 ? 4 : 2;
  // twice as many threads as entries: their largest elements set the threshold
  const Cut cut = cut_rows(q.C, es, 2 * q.k);
  TopkParams p = q;
  p.per = cut.per;
  rec->grid = dim3((unsigned)rows, 1, (unsigned)cut.cluster);
  rec->block = dim3((unsigned)cut.threads);
  rec->cluster = (unsigned)cut.cluster;
  rec->smem = topk_smem(cut, p.k, es);
  if (cut.cluster > 1) rec->func = dtype == DT_F32 ? topk_func<float, true>(cut) : topk_func<__nv_bfloat16, true>(cut);
  else rec->func = dtype == DT_F32 ? topk_func<float, false>(cut) : topk_func<__nv_bfloat16, false>(cut);
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
