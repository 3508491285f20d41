// What the top-k, distillation and beam kernels share: the order of logits, units
// of 16 bytes, exponentials relative to a reference, sums over a block, the blocks of a
// cluster; and, for distillation, a row or a slice of it in shared memory (top-k
// reads its rows from global memory, twice).
//
// A row of C elements is cut into slices of `per` elements, one for each block
// of a cluster.  A Slice is copied in 16-byte units whatever the row's
// alignment: shared memory keeps the row's phase (its address modulo 16), the
// units that the row only partly covers are copied element by element, and
// what they and the units behind them hold besides is -infinity, so that
// every pass runs over whole units, as many for each thread, without tests.  A
// thread copies the units that it later reads first (tid, tid + NT, ...) and need
// not wait for other threads to read them.
//
// These kernels are bound by instruction issue before they are by DRAM (a row of
// 32000 bf16 leaves an SM about 11000 issue slots), so block sizes are constants
// and loops have uniform counts.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"

namespace mlpk {
namespace lg {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSMs = 152;
constexpr int kMaxK = 256;                 // entries kept of a row
constexpr int64_t kMaxC = 384000;          // columns: eight slices of 192000 bytes of fp32
constexpr int kAhead = kSMs;                // rows are asked for so many blocks ahead
constexpr int64_t kSliceBytes = 64 * 1024; // a slice of at most this leaves room for three blocks on an SM

// 2^t; subnormal results are flushed to zero (PTX ex2.approx).
__device__ __forceinline__ float ex2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The blocks of a cluster.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t in_block(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void put64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void put32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Order of logits as unsigned integers: NaN is 0, below -infinity; -0 is +0.
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return f == f ? k : 0u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  const uint32_t u = (k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k;
  return k ? __uint_as_float(u) : __uint_as_float(0x7FC00000u);
}
// A candidate: larger is better, lower column first among equals; 0 is none.
__device__ __forceinline__ uint64_t entry_of(uint32_t key, int col) {
  return ((uint64_t)key << 32) | (uint32_t)~col;
}
__device__ __forceinline__ int entry_col(uint64_t e) { return (int)~(uint32_t)e; }
__device__ __forceinline__ uint32_t entry_key(uint64_t e) { return (uint32_t)(e >> 32); }

template <typename T> constexpr int kPer16 = 16 / (int)sizeof(T);

// The E elements of a unit as fp32.
template <typename T>
__device__ __forceinline__ void unit_floats(uint4 a, float (&v)[kPer16<T>]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if constexpr (sizeof(T) == 4) {
      v[h] = __uint_as_float(w[h]);
    } else {
      v[2 * h] = __uint_as_float(w[h] << 16);
      v[2 * h + 1] = __uint_as_float(w[h] & 0xFFFF0000u);
    }
  }
}
// The largest element of a unit, or of several, NaN passed over; bf16: of the
// even elements and of the odd ones, side by side.
template <typename T> struct Most;
template <> struct Most<float> {
  float m = -INFINITY;
  __device__ __forceinline__ Most() {}
  __device__ __forceinline__ explicit Most(const uint4& a) {
    m = fmaxf(fmaxf(__uint_as_float(a.x), __uint_as_float(a.y)), fmaxf(__uint_as_float(a.z), __uint_as_float(a.w)));
  }
  __device__ __forceinline__ void take(const Most& o) { m = fmaxf(m, o.m); }
  // Whether it reaches a limit.
  static __device__ __forceinline__ float limit(float x) { return x; }
  __device__ __forceinline__ bool reaches(float x) const { return m >= x; }
  __device__ __forceinline__ float value() const { return fmaxf(m, -INFINITY); }
};
template <> struct Most<__nv_bfloat16> {
  __nv_bfloat162 m;
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
  __device__ __forceinline__ Most() { m = two(0xFF80FF80u); }
  __device__ __forceinline__ explicit Most(const uint4& a) {
    m = __hmax2(__hmax2(two(a.x), two(a.y)), __hmax2(two(a.z), two(a.w)));
  }
  __device__ __forceinline__ void take(const Most& o) { m = __hmax2(m, o.m); }
  static __device__ __forceinline__ uint32_t limit(float x) {   // (a bf16's value)
    const uint32_t h = __float_as_uint(x) >> 16;
    return h | h << 16;
  }
  __device__ __forceinline__ bool reaches(uint32_t limit) const {
    uint32_t r;
    asm("{\n\t.reg .pred p, q;\n\tsetp.ge.bf16x2 p|q, %1, %2;\n\tor.pred p, p, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(*reinterpret_cast<const uint32_t*>(&m)), "r"(limit));
    return r != 0;
  }
  __device__ __forceinline__ float value() const { return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY); }
};
template <typename T> __device__ __forceinline__ T minus_inf();
template <> __device__ __forceinline__ float minus_inf<float>() { return -INFINITY; }
template <> __device__ __forceinline__ __nv_bfloat16 minus_inf<__nv_bfloat16>() { return __ushort_as_bfloat16(0xFF80); }

// The slice [lo, lo + n) of a row as shared memory holds it: element i is at
// elems()[ph + i], units() unit v holds the elements v E - ph .. + E.  Thread tid
// has the units tid + u NT, u < nu; unit nvec is the first behind the slice.
template <typename T, int NT_>
struct Slice {
  static constexpr int NT = NT_;
  unsigned char* buf;
  int lo, n, ph, nvec, nu;

  __device__ __forceinline__ T* elems() const { return reinterpret_cast<T*>(buf); }
  __device__ __forceinline__ uint4* units() const { return reinterpret_cast<uint4*>(buf); }
  __device__ __forceinline__ uint4& mine(int u) const { return units()[threadIdx.x + u * NT]; }
  __device__ __forceinline__ T& at(int i) const { return elems()[ph + i]; }

  // Starts the copies of this thread's units.
  __device__ __forceinline__ void load(unsigned char* buf_, const T* row, int lo_, int n_) {
    constexpr int E = kPer16<T>;
    buf = buf_;
    lo = lo_;
    n = n_ > 0 ? n_ : 0;
    const T* g = row + lo;
    ph = (int)(((uintptr_t)g & 15) / sizeof(T));
    nvec = n > 0 ? (ph + n + E - 1) / E : 0;
    nu = (nvec + NT - 1) / NT;
    const int whole = (ph + n) / E;   // the units from ph > 0 on to here are the row's alone
    const int full = whole / NT;
    const unsigned char* g0 = reinterpret_cast<const unsigned char*>(g - ph) + 16 * threadIdx.x;
    const uint32_t s0 = smem_addr(buf) + 16u * threadIdx.x;
    const auto edge = [&](int u) {
      const int v = threadIdx.x + u * NT;
      if (v >= (ph > 0) && v < whole) {
        copy16_async(s0 + 16u * NT * u, g0 + 16ll * NT * u);
      } else {
        for (int e = 0; e < E; ++e) {
          const int i = v * E + e - ph;
          elems()[v * E + e] = i >= 0 && i < n ? g[i] : minus_inf<T>();
        }
      }
    };
    int u = 0;
    if (ph > 0 && nu > 0) edge(u++);
#pragma unroll 4
    for (; u < full; ++u) copy16_async(s0 + 16u * NT * u, g0 + 16ll * NT * u);
    for (; u < nu; ++u) edge(u);
  }
  // f(unit) for this thread's units, four loads in flight.
  template <typename F>
  __device__ __forceinline__ void each_unit(F f) const {
    int u = 0;
    for (; u + 4 <= nu; u += 4) {
      const uint4 a = mine(u), b = mine(u + 1), c = mine(u + 2), d = mine(u + 3);
      f(a);
      f(b);
      f(c);
      f(d);
    }
    for (; u < nu; ++u) f(mine(u));
  }
  // f(i, value) for the elements of this thread's units.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    constexpr int E = kPer16<T>;
    for (int u = 0; u < nu; ++u) {
      float x[E];
      unit_floats<T>(mine(u), x);
      const int i0 = ((int)threadIdx.x + u * NT) * E - ph;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (i0 + e >= 0 && i0 + e < n) f(i0 + e, x[e]);
    }
  }
};
// Asks for elements [lo, lo + n) of a row to be in L2 (the whole 16-byte units).
template <typename T>
__device__ __forceinline__ void prefetch_row(const T* row, int lo, int n) {
  const uintptr_t a = ((uintptr_t)(row + lo) + 15) & ~(uintptr_t)15, b = (uintptr_t)(row + lo + n) & ~(uintptr_t)15;
  if (b > a)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"((uint32_t)(b - a)) : "memory");
}
// Bytes of a slice's buffer: whole rounds of units (the phase can add one).
inline int64_t slice_buffer(int64_t per, int es, int threads) { return round_up(per * es / 16 + 1, threads) * 16; }

// Sums and maxima over the block of NT threads, the same in every thread;
// red: a place of its own for each call.
struct __align__(16) Red { float v[16]; };
template <int NT>
__device__ __forceinline__ float red_sum(const Red& red) {
  if constexpr (NT == 32) return red.v[0];
  if constexpr (NT == 64) return red.v[0] + red.v[1];
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 32; w += 4) {
    const float4 a = *reinterpret_cast<const float4*>(red.v + w);
    s += (a.x + a.y) + (a.z + a.w);
  }
  return s;
}
template <int NT>
__device__ __forceinline__ float block_sum(float v, Red& red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red.v[threadIdx.x >> 5] = v;
  __syncthreads();
  return red_sum<NT>(red);
}
template <int NT>
__device__ __forceinline__ void block_sums(float& u, float& v, Red& ru, Red& rv) {
  u = warp_sum(u);
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) {
    ru.v[threadIdx.x >> 5] = u;
    rv.v[threadIdx.x >> 5] = v;
  }
  __syncthreads();
  u = red_sum<NT>(ru);
  v = red_sum<NT>(rv);
}
template <int NT>
__device__ __forceinline__ float block_max(float v, Red& red) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) red.v[threadIdx.x >> 5] = v;
  __syncthreads();
  if constexpr (NT == 32) return red.v[0];
  if constexpr (NT == 64) return fmaxf(red.v[0], red.v[1]);
  float s = -INFINITY;
#pragma unroll
  for (int w = 0; w < NT / 32; w += 4) {
    const float4 a = *reinterpret_cast<const float4*>(red.v + w);
    s = fmaxf(s, fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)));
  }
  return s;
}

// Two neighbouring elements (bf16: of one word) as fp32.
template <typename T>
__device__ __forceinline__ F2 pair_of(const uint4& a, int h) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  if constexpr (sizeof(T) == 4) return pack2(__uint_as_float(w[2 * h]), __uint_as_float(w[2 * h + 1]));
  else return pack2(__uint_as_float(w[h] << 16), __uint_as_float(w[h] & 0xFFFF0000u));
}

// exp((x - ref) / T) for many x as 2^(x c - ref c), one FMA and one ex2 each.
// ref c is rounded once for all of them, which scales every term alike by
// 2^(its rounding): `scale` takes that out of their sum.  Where ref c is so large that
// its rounding passes 1 (masks of the lowest value, small T) the difference is
// formed first.
struct Exponent {
  float c, ref, rc, scale;
  bool far;
  __device__ __forceinline__ Exponent(float ref_, float c_) : c(c_), ref(ref_), rc(ref_ * c_) {
    far = !(fabsf(rc) < 0x1p24f);
    const float off = fmaf(ref, c, -rc);
    scale = far ? 1.f : fabsf(off) < 0x1p-12f ? fmaf(-kLn2, off, 1.f) : ex2(-off);
  }
  // of one x, without the scale
  __device__ __forceinline__ float one(float x) const { return ex2(far ? (x - ref) * c : fmaf(x, c, -rc)); }
};
// The sum over this thread's units of exp((x - ref) / T), and with SQUARES the sum
// of their squares.
template <bool SQUARES, typename T, int NT>
__device__ __forceinline__ float sum_exp(const Slice<T, NT>& s, const Exponent& q, float& squares) {
  float sum;
  if (q.far) {
    sum = squares = 0.f;
    s.each([&](int, float x) {
      const float e = ex2((x - q.ref) * q.c);
      sum += e;
      if (SQUARES) squares = fmaf(e, e, squares);
    });
  } else {
    const F2 c2 = pack2(q.c, q.c), r2 = pack2(-q.rc, -q.rc);
    F2 a0 = pack2(0.f, 0.f), a1 = a0, b0 = a0, b1 = a0;
    s.each_unit([&](const uint4& u) {
#pragma unroll
      for (int h = 0; h < kPer16<T> / 2; ++h) {
        float x, y;
        unpack2(fma2(pair_of<T>(u, h), c2, r2), x, y);
        const F2 e = pack2(ex2(x), ex2(y));
        if (h & 1) {
          a1 = add2(a1, e);
          if (SQUARES) b1 = fma2(e, e, b1);
        } else {
          a0 = add2(a0, e);
          if (SQUARES) b0 = fma2(e, e, b0);
        }
      }
    });
    sum = sum2(add2(a0, a1));
    squares = SQUARES ? sum2(add2(b0, b1)) * (q.scale * q.scale) : 0.f;
  }
  return sum * q.scale;
}
template <typename T, int NT>
__device__ __forceinline__ float max_of(const Slice<T, NT>& s) {
  Most<T> m;
  s.each_unit([&](const uint4& u) { m.take(Most<T>(u)); });
  return m.value();
}

}  // namespace lg
}  // namespace mlpk
