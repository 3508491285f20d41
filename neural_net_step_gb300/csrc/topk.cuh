// The k largest entries of every row of logits [B, C] with the log-sums of
// the whole row and of what is left of it:
//   v_j, i_j  in descending order, lowest column first among equals,
//   lse = log sum_i exp(z_i / T),  tail = log sum_{i not taken} exp(z_i / T).
//
// Bound by DRAM, and by instruction issue close behind it.  A row is read twice, the
// second time from L2 and backwards (what was read last is nearest), so that
// nothing of it is held on the SM and many rows are under way there.
//   1. Every thread finds the largest of its elements.  The k-th largest of those is a
//      threshold that at least k elements reach, and not many more do where the
//      row is in no particular order.
//   2. The second time, 16-byte units that reach it are marked and the
//      others' exponentials summed; then the marked units' elements are
//      candidates or join the sum.  Where candidates are too many (equal values, sorted
//      rows) or too few (NaN), the k-th largest is found by halving the range of
//      keys, counting each time (up to 34 counts of the row), and the columns of equals
//      in their order.  A row with fewer units than entries (bf16 C < 8 k, fp32 C < 4 k) has no
//      threshold: all its elements are candidates, and where they are too many it goes the
//      same way (bf16 16384 x 1500, k = 256: 1625 us; x 4000: 545).
//   3. Warps sort the candidates 32 at a time; each one's place is its own in its run
//      and what binary searches in the other runs say.  Those that are not taken
//      join the sum: the tail needs no subtraction, and where next to nothing is left of it
//      relative to the smallest taken it is formed again relative to its own largest.
// The blocks of a cluster do this for their slices of a row and send lists and sums to
// the first, which finds the entries' places in the row and adds what a slice took
// and the row does not to the rest.
//   16384 x 32000 bf16, k = 64: 202 us, 5.2 TB/s of rows (0.78 of the copy rate); staged in
// shared memory instead, once from DRAM, three rows fit an SM and it took 260 us.
#pragma once
#include <type_traits>

#include "beam.cuh"
#include "logits.cuh"
#include "topk.h"

namespace mlpk {
namespace tk {

using namespace lg;

struct __align__(16) TopkShared {
  Red red[7];
  uint32_t top[16], nth[16];        // of each warp (read 16 bytes at a time)
  uint32_t tau;
  int count, over;                  // candidates; units found no place in a warp's list
  int total[16];
  int found;
  uint32_t last_key;                // the smallest taken
  int last_at;
  float2 part[8];                   // of each block of the cluster: reference and sum of the rest
  BeamBase base[8];                 // of each beam of a batch entry
};

// The slice of a row that a block walks: elements [lo, lo + n) from g on, whole
// 16-byte units from element `head` on.
template <typename T, int NT>
struct Walk {
  const T* g;
  int lo, n, head, units;

  __device__ __forceinline__ Walk(const T* row, int lo_, int n_) : g(row + lo_), lo(lo_), n(n_ > 0 ? n_ : 0) {
    head = min(n, (int)((16 - ((uintptr_t)g & 15)) & 15) / (int)sizeof(T));
    units = (n - head) / kPer16<T>;
  }
  __device__ __forceinline__ const uint4* unit(int v) const { return reinterpret_cast<const uint4*>(g + head) + v; }
  __device__ __forceinline__ int at(int v) const { return head + v * kPer16<T>; }   // a unit's first element
  // The elements at the ends: this thread's at most one of each (-1: none).
  __device__ __forceinline__ int first_edge() const { return (int)threadIdx.x < head ? (int)threadIdx.x : -1; }
  __device__ __forceinline__ int last_edge() const {
    const int i = at(units) + (int)threadIdx.x;
    return i < n ? i : -1;
  }
  // f(i, value), every element once over the block.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int v = threadIdx.x; v < units; v += NT) {
      float x[kPer16<T>];
      unit_floats<T>(*unit(v), x);
#pragma unroll
      for (int e = 0; e < kPer16<T>; ++e) f(at(v) + e, x[e]);
    }
    if (first_edge() >= 0) f(first_edge(), to_f32(g[first_edge()]));
    if (last_edge() >= 0) f(last_edge(), to_f32(g[last_edge()]));
  }
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

// What makes an element a candidate: a key above `key`, or `key` up to element `last`.
struct Limit {
  uint32_t key;
  int last;
  __device__ __forceinline__ bool takes(uint32_t k, int i) const { return k > key || (k == key && i <= last); }
};

// Candidates where the threshold did not leave a fit number of them: exactly
// those not below the kk-th largest, or the kk largest themselves.  tau: a first
// guess of the kk-th largest's key, or 0.
template <typename T, typename K, int NT>
__device__ __noinline__ Limit search(const Walk<T, NT> s, int kk, uint32_t tau, K* cand, TopkShared& sh) {
  const auto reach = [&](uint32_t key) {
    int c = 0;
    s.each([&](int, float x) { c += key_of(x) >= key; });
    return block_count<NT>(c, sh);
  };
  Limit l;
  l.key = tau;
  l.last = s.n;
  if (tau == 0 || tau == 0xFFFFFFFFu || reach(tau) < kk || reach(tau + 1) >= kk) {
    l.key = 0;
    for (int b = 31; b >= 0; --b)
      if (reach(l.key | (1u << b)) >= kk) l.key |= 1u << b;
  }
  if (reach(l.key) > kRoom<NT>) {
    // of those equal to it the first that are needed, NT elements at a time
    int need = kk - (l.key == 0xFFFFFFFFu ? 0 : reach(l.key + 1));
    for (int i0 = 0; i0 < s.n; i0 += NT) {
      const int i = i0 + (int)threadIdx.x;
      const bool equal = i < s.n && key_of(to_f32(s.g[i])) == l.key;
      const uint32_t who = __ballot_sync(0xffffffffu, equal);
      __syncthreads();
      if ((threadIdx.x & 31) == 0) sh.total[threadIdx.x >> 5] = __popc(who);
      __syncthreads();
      int before = 0, all = 0;
      for (int w = 0; w < NT / 32; ++w) {
        before += w < (int)threadIdx.x >> 5 ? sh.total[w] : 0;
        all += sh.total[w];
      }
      if (all >= need) {
        if (equal && before + __popc(who & ((1u << (threadIdx.x & 31)) - 1)) == need - 1) sh.found = i;
        __syncthreads();
        l.last = sh.found;
        break;
      }
      need -= all;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  s.each([&](int i, float x) {
    if (l.takes(key_of(x), i)) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kRoom<NT>) cand[at] = Cand<K>::of(x, i);
    }
  });
  __syncthreads();
  return l;
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

template <typename T, int MODE, int NT, typename K>
__global__ void __launch_bounds__(NT, NT == 32 ? 28 : 1024 / NT) topk_kernel(const __grid_constant__ TopkParams p) {
  pdl_enter();
  constexpr int E = kPer16<T>, warps = NT / 32, room = kRoom<NT> / warps;
  constexpr int kCounted = NT > 128 ? NT / 4 : 0;   // candidates whose places are counted: sooner known, more instructions
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ TopkShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr bool CLUSTER = MODE == SLICES;
  const int rank = MODE != ALONE ? (int)blockIdx.z : 0, blocks = MODE != ALONE ? (int)gridDim.z : 1;
  const int64_t row = MODE == BEAMS ? (int64_t)blockIdx.x * p.out.beams + rank : (int64_t)blockIdx.x;
  if (MODE != ALONE) cluster_arrive();
  // beams that offer nothing of their row
  const bool beam = MODE == BEAMS ? rank < p.out.beams : p.stats != nullptr;
  const float score = beam ? p.scores[row] : 0.f;
  const bool done = beam && p.done && p.done[row];
  const bool reads = MODE == BEAMS ? beam && beam_reads_row(score, done) : !beam || beam_reads_row(score, done);
  if (MODE != BEAMS && !reads) {   // (the merge knows without it)
    if (MODE == SLICES) cluster_wait();
    return;
  }

  K* cand = reinterpret_cast<K*>(smem);                            // [kRoom]
  int* hits = reinterpret_cast<int*>(cand + kRoom<NT>);            // [kRoom]: units, warp by warp; then
  float* sorted = reinterpret_cast<float*>(hits);                  //   the candidates' values by place
  uint64_t* best = reinterpret_cast<uint64_t*>(hits + kRoom<NT>);  // of a cluster's first block: [k] the row's, descending,
  uint64_t* lists = best + p.k;                                    //   [blocks][k] every block's (0: none)
  uint64_t* own = lists + (int64_t)rank * p.k;
  // the beams' lists and what their logits are added to go to the first block, which merges them
  const auto finish_beams = [&](const BeamBase& b) {
    cluster_wait();   // (every block of the cluster runs)
    if (beam) {
      if (rank != 0 && reads && tid < p.k) put64(in_block(smem_addr(own + tid), 0), own[tid]);
      if (tid == 0) {
        const uint32_t to = in_block(smem_addr(&sh.base[rank]), 0);
        put64(to, (uint64_t)__double_as_longlong(b.base));
        put32(to + 8, (uint32_t)b.kind);
        put32(to + 12, (uint32_t)b.done);
      }
    }
    cluster_arrive();
    cluster_wait();
    if (rank == 0) merge_beams(p.out, blockIdx.x, lists, sh.base, lists + 8 * p.k);
  };
  if (MODE == BEAMS && !reads) {
    finish_beams(beam_base(score, done, 0.f, 0.f));
    return;
  }

  const int lo = CLUSTER ? rank * p.per : 0;
  const Walk<T, NT> s(reinterpret_cast<const T*>(p.z) + row * p.ldz, lo, reads ? min(p.per, p.C - lo) : 0);
  const int kk = min(p.k, s.n), e0 = s.first_edge(), e1 = s.last_edge();
  const float x0 = e0 >= 0 ? to_f32(s.g[e0]) : -INFINITY, x1 = e1 >= 0 ? to_f32(s.g[e1]) : -INFINITY;
  if (tid == 0) sh.count = sh.over = 0;

  // 1. a threshold that at least kk elements reach.  Rounds of NT units; the last eight
  // stay in registers for the second time.
  const uint32_t none = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;   // (-infinity)
  const int rounds = (s.units + NT - 1) / NT, kept = max(rounds - 8, 0);
  Most<T> most;
  uint4 held[8];
  {
    int r = 0;
    for (; r + 8 <= kept; r += 8) {
      const uint4* u = s.unit(tid + r * NT);
#pragma unroll
      for (int q = 0; q < 8; ++q) held[q] = u[q * NT];
#pragma unroll
      for (int q = 0; q < 8; ++q) most.take(Most<T>(held[q]));
    }
#pragma unroll 4
    for (; r < kept; ++r) most.take(Most<T>(*s.unit(tid + r * NT)));
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int v = tid + (kept + q) * NT;
      held[q] = v < s.units ? *s.unit(v) : make_uint4(none, none, none, none);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) most.take(Most<T>(held[q]));
  }
  const uint32_t most_key = key_of(fmaxf(most.value(), fmaxf(x0, x1)));
  uint32_t* keys = reinterpret_cast<uint32_t*>(hits);   // [NT]
  const bool few = NT > 128 && kk * 4 <= NT;
  uint32_t mine;
  if (few) {   // the smallest of the warps' ceil(kk / warps)-th largest: a little lower, and sooner known
    mine = warp_nth(most_key, (kk + warps - 1) / warps);
    if (lane == 0) sh.nth[warp] = mine;
  } else {     // distinct by the threads' numbers, sorted by warps and searched like the candidates below
    mine = warp_sort_down((most_key & 0xFFFFFE00u) | (uint32_t)tid);
    keys[tid] = mine;
  }
  const uint32_t top_key = __reduce_max_sync(0xffffffffu, most_key);
  if (lane == 0) sh.top[warp] = top_key;
  if (tid < kCounted) cand[tid] = 0;
  __syncthreads();
  uint32_t tau = 0xFFFFFFFFu, row_key = 0;
  if constexpr (warps <= 2) {
    row_key = max(sh.top[0], sh.top[warps - 1]);
  } else {
#pragma unroll
    for (int w = 0; w < warps; w += 4) {
      const uint4 r = *reinterpret_cast<const uint4*>(sh.top + w), q = *reinterpret_cast<const uint4*>(sh.nth + w);
      row_key = max(row_key, max(max(r.x, r.y), max(r.z, r.w)));
      tau = min(tau, min(min(q.x, q.y), min(q.z, q.w)));
    }
  }
  if (!few) {
    constexpr int N = warps < 8 ? warps : 8;
    int place = lane;
#pragma unroll
    for (int w = 0; w < warps; w += N) place += larger_in_runs<N>(keys + w * 32, warp - w, mine);
    if (place == max(kk, 1) - 1) sh.tau = mine & 0xFFFFFE00u;
    __syncthreads();
    tau = sh.tau;
    if (sizeof(T) == 2) tau = (tau & 0x80000000u) ? tau & 0xFFFF0000u : tau | 0xFFFFu;   // (a bf16's key again)
  }
  tau = max(tau, key_of(-INFINITY));

  // 2. candidates, and the sum of the others relative to the threshold that they are below
  const bool sums = MODE == BEAMS || p.lse || p.tail || p.stats;
  const float least = value_of(tau);
  float ref = least > -INFINITY ? least : 0.f, rest = 0.f;
  const Exponent ex(ref, p.c);
  {
    int* hit = hits + warp * room;
    const auto limit = Most<T>::limit(least);
    F2 acc0 = pack2(0.f, 0.f), acc1 = acc0;
    const F2 c2 = pack2(p.c, p.c), r2 = pack2(-ex.rc, -ex.rc);
    uint32_t marks = 0;   // this thread's units that reach it, the latest in bit 0
    const auto take = [&](const uint4& u, F2& acc) {
      const bool in = Most<T>(u).reaches(limit);
      marks = marks * 2 + in;
      if (!sums) return;
      F2 e[E / 2];
#pragma unroll
      for (int h = 0; h < E / 2; ++h) {
        float x, y;
        unpack2(fma2(pair_of<T>(u, h), c2, r2), x, y);
        e[h] = pack2(ex2(x), ex2(y));
      }
#pragma unroll
      for (int h = E / 4; h > 0; h /= 2)
#pragma unroll
        for (int q = 0; q < h; ++q) e[q] = add2(e[q], e[q + h]);
      if (!in) acc = add2(acc, e[0]);
    };
    int n_hits = 0;
    const uint32_t below = (1u << lane) - 1;
    const auto list = [&](int round) {   // the marked units; bit 0: of this round
      while (const uint32_t who = __ballot_sync(0xffffffffu, marks != 0)) {
        const int at = n_hits + __popc(who & below);
        if (marks && at < room) hit[at] = tid + (round + __ffs(marks) - 1) * NT;
        marks &= marks - 1;
        n_hits += __popc(who);
      }
    };
#pragma unroll
    for (int q = 7; q >= 0; --q)
      if (kept + q < rounds) take(held[q], q & 1 ? acc1 : acc0);
    int marked = min(rounds, 8), r = kept - 1;
    for (; r >= 7; r -= 8) {
      if (marked > 24) {
        list(r + 1);
        marked = 0;
      }
      marked += 8;
      const uint4* u = s.unit(tid + r * NT);
#pragma unroll
      for (int q = 0; q < 8; ++q) held[q] = u[-q * NT];
#pragma unroll
      for (int q = 0; q < 8; ++q) take(held[q], q & 1 ? acc1 : acc0);
    }
    if (marked > 25) list(r + 1);   // (at most seven more)
    for (; r >= 0; --r) take(*s.unit(tid + r * NT), acc0);
    list(0);
    rest = sum2(add2(acc0, acc1));

    __syncwarp();
    if (n_hits > room) sh.over = 1;   // (count stays the number of candidates that have a place)
    n_hits = min(n_hits, room);
    const auto keep = [&](float x, int i, int at) {
      if (at < kRoom<NT>) cand[at] = Cand<K>::of(x, i);
    };
    for (int a = lane; a - lane < n_hits; a += 32) {
      const int v = a < n_hits ? hit[a] : s.units;
      uint32_t in = 0;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (v < s.units) {
        u = *s.unit(v);
        float x[E];
        unit_floats<T>(u, x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          in |= (uint32_t)(x[e] >= least) << e;
          if (sums && !(x[e] >= least)) rest += ex2(fmaf(x[e], p.c, -ex.rc));
        }
      }
      const int n_in = __reduce_add_sync(0xffffffffu, __popc(in));
      int base = 0;
      if (lane == 0) base = atomicAdd(&sh.count, n_in);
      base = __shfl_sync(0xffffffffu, base, 0);
      while (const uint32_t who = __ballot_sync(0xffffffffu, in != 0)) {
        if (in) {
          const int e = __ffs(in) - 1, w = sizeof(T) == 4 ? e : e >> 1;
          const uint32_t word = w < 2 ? (w == 0 ? u.x : u.y) : (w == 2 ? u.z : u.w);
          keep(__uint_as_float(sizeof(T) == 4 ? word : (e & 1) ? word & 0xFFFF0000u : word << 16), s.at(v) + e,
               base + __popc(who & below));
          in &= in - 1;
        }
        base += __popc(who);
      }
    }
    if (e0 >= 0) {
      if (x0 >= least) keep(x0, e0, atomicAdd(&sh.count, 1));
      else rest += ex2(fmaf(x0, p.c, -ex.rc));
    }
    if (e1 >= 0) {
      if (x1 >= least) keep(x1, e1, atomicAdd(&sh.count, 1));
      else rest += ex2(fmaf(x1, p.c, -ex.rc));
    }
    rest *= ex.scale;
  }
  __syncthreads();
  int count = sh.count;
  const bool many = count > kRoom<NT> || sh.over;
  if (many || count < kk || (sums && ex.far)) {
    Limit limit{tau, s.n};
    if (many || count < kk) {
      __syncthreads();
      limit = search<T>(s, kk, many ? tau : 0u, cand, sh);
      count = sh.count;
      if (count <= kCounted) {   // (zeros behind the last again)
        if (tid >= count && tid < kCounted) cand[tid] = 0;
        __syncthreads();
      }
    }
    if (sums) {
      float m = -INFINITY;
      s.each([&](int i, float x) {
        if (!limit.takes(key_of(x), i)) m = fmaxf(m, x);
      });
      m = block_max<NT>(m, sh.red[6]);
      ref = m > -INFINITY ? m : 0.f;
      rest = 0.f;
      s.each([&](int i, float x) {
        if (!limit.takes(key_of(x), i)) rest += ex2((x - ref) * p.c);
      });
    }
  }

  // 3. the candidates' places
  const auto write = [&](int place, float x, int col) {
    if (p.stats) {
      p.entries[row * p.k + place] = entry_of(key_of(x), col);
    } else {
      p.values[row * p.ldv + place] = x;
      p.indices[row * p.ldi + place] = col;
    }
  };
  const auto put = [&](int place, K c) {
    const float x = value_of(Cand<K>::key(c));
    const int i = Cand<K>::at(c);
    sorted[place] = x;
    if (place < kk) {
      if (MODE != ALONE) own[place] = entry_of(Cand<K>::key(c), s.lo + i);
      else write(place, x, s.lo + i);
      if (place == kk - 1) {
        sh.last_key = Cand<K>::key(c);
        sh.last_at = i;
      }
    }
  };
  if (count <= kCounted) {   // four neighbouring threads count for one candidate (zeros behind the last)
    const K c = tid < count * 4 ? cand[tid >> 2] : (K)0;
    const uint4* all = reinterpret_cast<const uint4*>(cand);
    constexpr int per16 = 16 / (int)sizeof(K);
    int n[2] = {0, 0};
    for (int b = tid & 3; b * 2 * per16 < count; b += 4) {
      const uint4 o = all[2 * b], q = all[2 * b + 1];
      if constexpr (sizeof(K) == 4) {
        n[0] += (o.x > c) + (o.y > c) + (o.z > c) + (o.w > c);
        n[1] += (q.x > c) + (q.y > c) + (q.z > c) + (q.w > c);
      } else {
        const auto two = [](uint32_t l, uint32_t h) { return (uint64_t)h << 32 | l; };
        n[0] += (two(o.x, o.y) > c) + (two(o.z, o.w) > c);
        n[1] += (two(q.x, q.y) > c) + (two(q.z, q.w) > c);
      }
    }
    int place = n[0] + n[1];
    place += __shfl_xor_sync(0xffffffffu, place, 1);
    place += __shfl_xor_sync(0xffffffffu, place, 2);
    if (tid < count * 4 && (tid & 3) == 0) put(place, c);
  } else {
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
      put(place, c);
    }
  }
  if (!CLUSTER && !sums) return;
  __syncthreads();

  // what is not taken of them, relative to the smallest that is (by place: the order
  // in which candidates were found changes no sum)
  float first = value_of(row_key), first0 = first > -INFINITY ? first : 0.f;
  float taken = !CLUSTER && tid < kk ? ex2((sorted[tid] - first0) * p.c) : 0.f;   // (at least k threads)
  if (sums && kk > 0) {
    const float l = sorted[kk - 1], to = l > -INFINITY ? l : 0.f;
    if (rest != 0.f && ref != to) rest *= ex2((ref - to) * p.c);
    ref = to;
    for (int j = kk + tid; j < count; j += NT) rest += ex2((sorted[j] - ref) * p.c);
  }
  // where next to nothing is left: relative to the largest that is not taken
  const auto look_closer = [&]() {
    if (!p.tail || !(rest < 0x1p-60f)) return;
    const Limit limit{sh.last_key, sh.last_at};
    float m = -INFINITY;
    s.each([&](int i, float x) {
      if (!limit.takes(key_of(x), i)) m = fmaxf(m, x);
    });
    m = block_max<NT>(m, sh.red[3]);
    if (!(m > -INFINITY)) return;
    ref = m;
    rest = 0.f;
    s.each([&](int i, float x) {
      if (!limit.takes(key_of(x), i)) rest += ex2((x - ref) * p.c);
    });
    rest = block_sum<NT>(rest, sh.red[4]);
  };
  if (CLUSTER) {
    rest = block_sum<NT>(rest, sh.red[0]);
    look_closer();
    cluster_wait();   // (every block of the cluster runs)
    if (rank != 0) {
      if (tid < p.k) put64(in_block(smem_addr(own + tid), 0), tid < kk ? own[tid] : 0ull);   // (at least k threads)
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

  if (CLUSTER) {
    if (tid < p.k) write(tid, value_of(entry_key(best[tid])), entry_col(best[tid]));
    if (!sums) return;
    first = value_of(entry_key(best[0]));
    first0 = first > -INFINITY ? first : 0.f;
    taken = tid < p.k ? ex2((value_of(entry_key(best[tid])) - first0) * p.c) : 0.f;
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
  if (MODE == BEAMS) {
    finish_beams(beam_base(score, done, first, all));
    return;
  }
  if (tid == 0) {
    if (p.stats) p.stats[row] = make_float2(first, all);
    if (p.lse) p.lse[row] = first0 / p.T + logf(all);
  }
  if (tid == (NT > 32 ? 32 : 1) && p.tail) p.tail[row] = ref / p.T + logf(rest);
}

// Of blocks that share a row there are only the largest (topk_cut), and slices of
// more than 65535 bf16 elements are never walked by fewer than 128 threads.
template <typename T, typename K>
const void* topk_func(int mode, int threads) {
  constexpr bool wide = sizeof(T) == 2 && sizeof(K) == 8;
  if (mode == SLICES) return (const void*)topk_kernel<T, SLICES, 512, K>;
  if (threads == 512)
    return mode == ALONE ? (const void*)topk_kernel<T, ALONE, 512, K> : (const void*)topk_kernel<T, BEAMS, 512, K>;
  if (threads == 256)
    return mode == ALONE ? (const void*)topk_kernel<T, ALONE, 256, K> : (const void*)topk_kernel<T, BEAMS, 256, K>;
  if (threads == 128 || wide)
    return mode == ALONE ? (const void*)topk_kernel<T, ALONE, 128, K> : (const void*)topk_kernel<T, BEAMS, 128, K>;
  if constexpr (!wide) {
    if (threads == 64)
      return mode == ALONE ? (const void*)topk_kernel<T, ALONE, 64, K> : (const void*)topk_kernel<T, BEAMS, 64, K>;
    return mode == ALONE ? (const void*)topk_kernel<T, ALONE, 32, K> : (const void*)topk_kernel<T, BEAMS, 32, K>;
  }
  return nullptr;
}

}  // namespace tk
}  // namespace mlpk
