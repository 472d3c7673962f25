// rowstream.hpp — device helpers of the kernels that stream one logits row at
// a time (top.hip, beam.hip, distill.hip): 16-byte granules of a row at any
// alignment, log-sum-exp masses, order keys and workgroup counting.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace dspark {

// ---- granules ------------------------------------------------------------------
// A row of V elements is read in 16-byte granules of the address space:
// granule q holds the row's elements q EPL - head + [0, EPL), where head is
// the number of elements between the 16-byte boundary at or below the row's
// start and the start itself.  Interior granules are one 16-byte load; the
// first and last ones, which may hold other rows' elements, are read element
// by element, so nothing outside the row is touched at any alignment.
template <typename T>
struct Row {
  static constexpr int EPL = 16 / static_cast<int>(sizeof(T));
  const T* p;  // element 0
  int head;    // elements before it in its granule
  int V;
  int Q;       // granules
};

template <typename T>
__device__ __forceinline__ Row<T> make_row(const T* p, int V) {
  Row<T> r;
  r.p = p;
  r.head = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  r.V = V;
  r.Q = (r.head + V + Row<T>::EPL - 1) / Row<T>::EPL;
  return r;
}

// Element j of a granule.
__device__ __forceinline__ float gran_elem(const uint4& u, int j, uint16_t) {
  const uint32_t w = (j >> 1) == 0 ? u.x : (j >> 1) == 1 ? u.y : (j >> 1) == 2 ? u.z : u.w;
  return (j & 1) ? bf_hi(w) : bf_lo(w);
}
__device__ __forceinline__ float gran_elem(const uint4& u, int j, float) {
  return __uint_as_float(j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w);
}

// A granule with elements of the row and others: element by element, the others
// as -inf.  A row has two of them at most.
template <typename T>
__device__ __forceinline__ uint4 gran_partial(const Row<T>& r, int e0) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      const int e = e0 + 2 * i;
      const uint32_t a = (e >= 0 && e < r.V) ? r.p[e] : 0xFF80u;
      const uint32_t b = (e + 1 >= 0 && e + 1 < r.V) ? r.p[e + 1] : 0xFF80u;
      w[i] = a | (b << 16);
    } else {
      const int e = e0 + i;
      w[i] = (e >= 0 && e < r.V) ? __float_as_uint(r.p[e]) : 0xFF800000u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Granule q, elements outside the row as -inf.
template <typename T>
__device__ __forceinline__ uint4 gran_load(const Row<T>& r, int q) {
  constexpr int EPL = Row<T>::EPL;
  const int e0 = q * EPL - r.head;
  if (e0 >= 0 && e0 + EPL <= r.V) return *reinterpret_cast<const uint4*>(r.p + e0);
  return gran_partial(r, e0);
}

// Keeps the compiler from holding a granule's unpacked elements in registers
// from one pass over them to the next (they are one instruction away).
__device__ __forceinline__ void repack(uint4& u) { asm volatile("" : "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w)); }

// L granules per thread, q0 + i NT + tid: one branch on the whole group (uniform)
// keeps the interior loads free of per-lane checks.  ONCE: non-temporal loads.
template <typename T, int NT, int L, bool ONCE = false>
__device__ __forceinline__ void group_load(const Row<T>& r, int q0, int tid, uint4 (&u)[L]) {
  constexpr int EPL = Row<T>::EPL;
  if ((q0 > 0 || r.head == 0) && (q0 + NT * L) * EPL - r.head <= r.V) {
    const T* p = r.p + (static_cast<ptrdiff_t>(q0 + tid) * EPL - r.head);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const u32x4* a = reinterpret_cast<const u32x4*>(p + i * NT * EPL);
      const u32x4 v = ONCE ? __builtin_nontemporal_load(a) : *a;
      u[i] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  } else {
    // the whole granules first, all in flight together; others read the row's
    // first whole granule in their place
    constexpr uint32_t kNeg = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    const int whole = r.head ? EPL - r.head : 0;
    if (whole + EPL <= r.V) {
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int e0 = (q0 + i * NT + tid) * EPL - r.head;
        u[i] = *reinterpret_cast<const uint4*>(r.p + (e0 >= 0 && e0 + EPL <= r.V ? e0 : whole));
      }
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int e0 = (q0 + i * NT + tid) * EPL - r.head;
      if (e0 < 0 || e0 + EPL > r.V) {
        u[i] = make_uint4(kNeg, kNeg, kNeg, kNeg);
        if (e0 + EPL > 0 && e0 < r.V) u[i] = gran_partial(r, e0);
      }
    }
  }
}

// ---- masses ----------------------------------------------------------------------
// A mass is sum exp(x / T) held as (m, s): s = sum 2^(x c - fl(m c)), with m
// the largest x, c = fl(log2(e) / T) and fl the rounding to fp32 (one fused
// multiply-add and one exponential per element).  Values beyond kHugeLogit,
// where m c could overflow, take s = sum 2^((x - m) c) instead.  s = 0: empty;
// a NaN or +inf among the x makes s a NaN.
constexpr float kHugeLogit = 1e30f;

struct Mass {
  float m;
  float s;
};

__device__ __forceinline__ Mass mass_none() { return Mass{neg_inf(), 0.0f}; }

// Exponent by which a mass relative to m becomes one relative to n >= m.
// The products are rounded by themselves, as in the sums (where m c overflows
// and n c does not, it is -inf, as it should be).
__device__ __forceinline__ float mass_gap(float m, float n, float c) {
#pragma clang fp contract(off)
  return fabsf(n) > kHugeLogit ? (m - n) * c : m * c - n * c;
}

__device__ __forceinline__ Mass mass_add(Mass a, Mass b, float c) {
#pragma clang fp contract(off)
  const float n = fmaxf(a.m, b.m);
  if (n == neg_inf()) return Mass{n, a.s + b.s};  // 0, or the NaN of either
  float ga = a.m * c - n * c, gb = b.m * c - n * c;
  if (fabsf(n) > kHugeLogit) {
    ga = (a.m - n) * c;
    gb = (b.m - n) * c;
  }
  return Mass{n, a.s * __builtin_amdgcn_exp2f(ga) + b.s * __builtin_amdgcn_exp2f(gb)};
}

// The N masses m[i] for which take[i], as one (s = 0 where there is none).
template <int N>
__device__ __forceinline__ Mass mass_sum(const Mass (&m)[N], uint32_t take, float c) {
#pragma clang fp contract(off)
  float n = neg_inf(), s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) n = fmaxf(n, (take >> i) & 1u ? m[i].m : neg_inf());
  if (__any(fabsf(n) > kHugeLogit && n > neg_inf())) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      s += ((take >> i) & 1u) && m[i].m > neg_inf() ? m[i].s * __builtin_amdgcn_exp2f(mass_gap(m[i].m, n, c)) : 0.0f;
  } else {
    const float r = n > neg_inf() ? n * c : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      s += (take >> i) & 1u ? m[i].s * __builtin_amdgcn_exp2f(m[i].m * c - r) : 0.0f;
  }
  return Mass{n, s};
}

// Mass of L granules held by one thread.
template <typename T, int L>
__device__ __forceinline__ Mass group_mass(const uint4 (&u)[L], float c) {
  constexpr int EPL = Row<T>::EPL;
  float m = neg_inf();
#pragma unroll
  for (int i = 0; i < L; ++i)
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, gran_elem(u[i], j, T{}));
  float s = 0.0f;
  if (__any(fabsf(m) > kHugeLogit && m > neg_inf())) {
    const float ref = m > neg_inf() ? m : 0.0f;
#pragma unroll
    for (int i = 0; i < L; ++i)
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const float x = gran_elem(u[i], j, T{});
        s += __builtin_amdgcn_exp2f(fabsf(ref) > kHugeLogit ? (x - ref) * c : fmaf(x, c, -(ref * c)));
      }
  } else {
    const float r = m > neg_inf() ? m * c : 0.0f;
#pragma unroll
    for (int i = 0; i < L; ++i)
#pragma unroll
      for (int j = 0; j < EPL; ++j) s += __builtin_amdgcn_exp2f(fmaf(gran_elem(u[i], j, T{}), c, -r));
  }
  return Mass{m, s};
}

// 2^d in 64 bits for d <= 1 or so: Taylor's series of e^(f ln 2) on |f| <= 1/2,
// whose first term left out, (ln 2 / 2)^12 / 12!, is under 2^-46.
__device__ __forceinline__ double exp2_64(double d) {
  d = fmax(d, -2000.0);
  const double n = rint(d), x = (d - n) * 0.69314718055994530942;
  double p = 1.0 / 39916800;
  p = fma(p, x, 1.0 / 3628800);
  p = fma(p, x, 1.0 / 362880);
  p = fma(p, x, 1.0 / 40320);
  p = fma(p, x, 1.0 / 5040);
  p = fma(p, x, 1.0 / 720);
  p = fma(p, x, 1.0 / 120);
  p = fma(p, x, 1.0 / 24);
  p = fma(p, x, 1.0 / 6);
  p = fma(p, x, 0.5);
  p = fma(p, x, 1.0);
  p = fma(p, x, 1.0);
  return __builtin_amdgcn_ldexp(p, static_cast<int>(n));
}

// log2 of a normal x > 0 in 64 bits: x = 2^e m with m in [1/sqrt 2, sqrt 2], and
// ln m = 2 artanh t, t = (m - 1) / (m + 1), |t| < 0.172: the series' first term
// left out is under 2^-45 of it, so a logarithm near 0 keeps its relative accuracy.
__device__ __forceinline__ double log2_64(double x) {
  double m = __builtin_amdgcn_frexp_mant(x), e = static_cast<double>(__builtin_amdgcn_frexp_exp(x));
  if (m < 0.70710678118654752440) {
    m += m;
    e -= 1.0;
  }
  const double t = (m - 1.0) / (m + 1.0), q = t * t;
  double p = 1.0 / 15;
  p = fma(p, q, 1.0 / 13);
  p = fma(p, q, 1.0 / 11);
  p = fma(p, q, 1.0 / 9);
  p = fma(p, q, 1.0 / 7);
  p = fma(p, q, 1.0 / 5);
  p = fma(p, q, 1.0 / 3);
  p = fma(p, q, 1.0);
  return fma(p * t, 2.8853900817779268147, e);
}

// log2 of a mass, with c64 = log2(e) / T: the rounding of m c that s carries is
// taken out again.  The terms are added in 64 bits; the logarithm of s is one
// of 32 bits on its mantissa, off by less than 2^-23 (the sum itself is no better).
__device__ __forceinline__ double mass_log2(Mass a, float c, double c64) {
#pragma clang fp contract(off)
  if (!(a.s > 0.0f) || a.m == neg_inf()) return a.s == 0.0f ? -__builtin_inf() : __builtin_nan("");
  const double m = static_cast<double>(a.m);
  const double fix = fabsf(a.m) > kHugeLogit ? 0.0 : static_cast<double>(a.m * c) - m * static_cast<double>(c);
  const float lg = __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(a.s));  // log2
  return m * c64 + fix + (static_cast<double>(lg) + static_cast<double>(__builtin_amdgcn_frexp_expf(a.s)));
}

// log2(2^a + 2^b), the sum's logarithm in 32 bits (it lies in [0, 1]).
__device__ __forceinline__ double log2_add(double a, double b) {
  const double n = fmax(a, b), d = fmin(a, b);
  if (n == -__builtin_inf()) return a + b;  // -inf, or a NaN
  return n + static_cast<double>(__builtin_amdgcn_logf(1.0f + __builtin_amdgcn_exp2f(static_cast<float>(d - n))));
}

__device__ __forceinline__ Mass wave_mass(Mass a, float c) {
  const float n = wave_max(a.m);
  const float k = n == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(mass_gap(a.m, n, c));
  return Mass{n, wave_sum(a.s * k)};
}

// Sum over the wave in 64 bits, the same on every lane: DPP within each row of
// 16 lanes, then the four row sums.
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = static_cast<uint32_t>(dpp_i<CTRL>(static_cast<int>(b)));
  const uint32_t hi = static_cast<uint32_t>(dpp_i<CTRL>(static_cast<int>(b >> 32)));
  return __longlong_as_double(static_cast<long long>((static_cast<uint64_t>(hi) << 32) | lo));
}
__device__ __forceinline__ double lane_d(double v, int l) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = static_cast<uint32_t>(lane_i(static_cast<int>(b), l));
  const uint32_t hi = static_cast<uint32_t>(lane_i(static_cast<int>(b >> 32), l));
  return __longlong_as_double(static_cast<long long>((static_cast<uint64_t>(hi) << 32) | lo));
}
__device__ __forceinline__ double wave_sum64(double v) {
  v += dpp_d<kDppXor1>(v);
  v += dpp_d<kDppXor2>(v);
  v += dpp_d<kDppHalfMirror>(v);
  v += dpp_d<kDppMirror>(v);
  return (lane_d(v, 0) + lane_d(v, 16)) + (lane_d(v, 32) + lane_d(v, 48));
}

// ---- order keys --------------------------------------------------------------------
// Unsigned keys in the order of the values (-0 as +0).  A candidate's 64-bit
// key also orders equal values by the lower index; keys of one row are unique.
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t cand_key(uint32_t okey, int32_t index) {
  return (static_cast<uint64_t>(okey) << 32) | static_cast<uint32_t>(~index);
}
__device__ __forceinline__ int32_t key_index(uint64_t k) { return static_cast<int32_t>(~static_cast<uint32_t>(k)); }
__device__ __forceinline__ float key_value(uint64_t k) { return key_value(static_cast<uint32_t>(k >> 32)); }

// The same order for 64-bit values.
constexpr uint64_t kKey64NegInf = 0x000FFFFFFFFFFFFFull;
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_double(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k ^ 0x8000000000000000ull : ~k));
}

// Exclusive prefix sum over the workgroup's threads, and the total.  slots: NW
// ints, free again after the next barrier.
template <int NW>
__device__ __forceinline__ int block_scan(int v, int* slots, int& total) {
  const int lane = threadIdx.x & 63;
  // within rows of 16 lanes by DPP row shifts (lanes shifted in from outside give
  // 0), then the last lanes of the rows before
  int inc = v;
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x111, 0xF, 0xF, true);
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x112, 0xF, 0xF, true);
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x114, 0xF, 0xF, true);
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x118, 0xF, 0xF, true);
  const int r0 = lane_i(inc, 15), r1 = r0 + lane_i(inc, 31), r2 = r1 + lane_i(inc, 47);
  const int all = r2 + lane_i(inc, 63);
  inc += lane < 16 ? 0 : lane < 32 ? r0 : lane < 48 ? r1 : r2;
  if constexpr (NW == 1) {
    total = all;
    return inc - v;
  } else {
    const int wave = threadIdx.x >> 6;
    if (lane == 0) slots[wave] = all;
    __syncthreads();
    int base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      base += w < wave ? slots[w] : 0;
      total += slots[w];
    }
    return base + inc - v;
  }
}

// Three per-wave counts (under 2^21 in total) summed over the workgroup, on every
// thread.  slots: 2 NW words, used in turn by `step`, so that one barrier a call
// is enough.
struct Count3 {
  int a, b, c;
};
template <int NW>
__device__ __forceinline__ Count3 block_count(Count3 n, uint64_t* slots, int& step) {
  if constexpr (NW == 1) {
    return n;
  } else {
    uint64_t* s = slots + (step++ & 1) * NW;
    if ((threadIdx.x & 63) == 0)
      s[threadIdx.x >> 6] = static_cast<uint64_t>(n.a) | static_cast<uint64_t>(n.b) << 21 |
                            static_cast<uint64_t>(n.c) << 42;
    __syncthreads();
    uint64_t t = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) t += s[w];
    constexpr uint64_t m = (1u << 21) - 1;
    return Count3{static_cast<int>(t & m), static_cast<int>(t >> 21 & m), static_cast<int>(t >> 42)};
  }
}

// Largest-first threshold by a search in quarters: a key t with want <=
// count(>= t) <= most, or the largest t with count(>= t) >= want where no such t
// exists.  lo: a key with count(>= lo) = n_lo >= want; hi: one with count(>= hi)
// < want.  count(t1, t2, t3), t1 <= t2 <= t3, gives the counts of keys at or above
// each, the same on every thread.  On return n_lo is count(>= t).
template <typename Key, class Count>
__device__ __forceinline__ Key search_key(Key lo, Key hi, int& n_lo, int want, int most, Count&& count) {
  while (n_lo > most && hi - lo > 1) {
    const Key d = hi - lo;
    const Key t1 = lo + max(d / 4, static_cast<Key>(1)), t2 = lo + max(d / 2, static_cast<Key>(1));
    const Key t3 = lo + max(d / 4 + d / 2, static_cast<Key>(1));
    const Count3 n = count(t1, t2, t3);
    if (n.c >= want) {
      lo = t3;
      n_lo = n.c;
    } else if (n.b >= want) {
      lo = t2;
      n_lo = n.b;
      hi = t3;
    } else if (n.a >= want) {
      lo = t1;
      n_lo = n.a;
      hi = t2;
    } else {
      hi = t1;
    }
  }
  return lo;
}

}  // namespace dspark
