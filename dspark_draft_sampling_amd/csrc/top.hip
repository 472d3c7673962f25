// top.hip — the K highest logits of each row with the mass of the others.
//
// Semantics (include/dspark.h, dspark_top_logits): per row the K largest
// logits in descending order, the lower index first among equal ones, the
// natural logarithm of sum exp(x / T) over the other tokens and over all.
//
// One pass over the row.  A workgroup takes a segment of a row, every thread
// up to 16 groups of 4 granules (32 bf16 or 16 fp32 logits), and keeps of each
// group its maximum and its mass (rowstream.hpp) in LDS: one exponential and
// about 7.5 VALU slots per element, no running maximum and no candidate test in
// the stream.  K or a few more of the threads' maxima (of the groups' where K
// is large beside the threads), found by a search over their order keys, bound
// the K-th largest logit from below: only the granules of the groups that reach
// the bound are read again, from the caches, and their elements at or above it
// become candidates in LDS.  The candidates' unique 64-bit keys (value, then
// index) give each its rank by counting.  The mass of the rest is summed from
// the other groups and, element by element, from those few: nothing is
// subtracted, so it keeps its relative accuracy however small it is beside the
// top.
//
// The bound can let too many elements through (rows of equal values, a few
// finite values in few groups): then the K-th key is found by a search over
// the segment itself, read once per step.
//
// Rows cut into several segments (few rows, or long ones) leave each
// segment's candidates and mass in the workspace; top_merge_kernel takes the K
// best of those.  Every choice is by unique keys and every sum in an order set
// by positions, so results do not depend on timing.
#include <algorithm>

#include "common.hpp"
#include "internal.hpp"
#include "rowstream.hpp"

namespace dspark {
namespace {

constexpr int kMergeThreads = 256;
constexpr int kMaxGrid = 1 << 20;  // workgroups of a launch; each then takes several items
constexpr int kL = 4;              // granules of a group
constexpr int kG = 16;             // groups of a thread at most

// Candidates a list may hold beyond K: the searches stop at the first bound
// within it.
__host__ __device__ constexpr int list_len(int K) { return K + K / 4 + 8; }
constexpr int kMaxList = list_len(DSPARK_MAX_TOP);

struct TopOut {
  float* values;   // [R, K]
  int32_t* ids;    // [R, K]
  float* rest;     // [R]
  float* lse;      // [R]
  uint8_t* flags;  // [R]
  uint64_t* keys;  // [R, P, list_len(K)]: a segment's candidates, 0: none
  Mass* parts;     // [R, P]: the mass of its other elements
};

// skip: rows (beams) that are not read at all.
struct TopSkip {
  const float* scores;      // NULL: none is skipped
  const uint8_t* finished;  // or NULL
};
__device__ __forceinline__ bool skipped(const TopSkip& s, size_t row) {
  if (!s.scores) return false;
  const float sc = s.scores[row];
  return !(sc > neg_inf() && sc < pos_inf()) || (s.finished && s.finished[row]);
}

// A key with K <= count(>= it) <= list_len(K) among n distinct keys in LDS (0:
// none), all of them below hi and the others at or above lo; lo itself where
// there are no more.  found: the number of keys that are not 0.
template <int NT>
__device__ __forceinline__ uint64_t list_bound(const uint64_t* cand, int n, int found, int K, uint64_t lo, uint64_t hi,
                                               int* slots, int& step) {
  constexpr int NW = NT / 64;
  if (found <= list_len(K)) return lo;
  const int n64 = (n + 63) / 64 * 64;
  return search_key<uint64_t>(lo, hi, found, K, list_len(K), [&](uint64_t t1, uint64_t t2, uint64_t t3) {
    Count3 c{0, 0, 0};
    for (int i = threadIdx.x; i < n64; i += NT) {
      const uint64_t k = i < n ? cand[i] : 0;
      c.a += __popcll(__ballot(k >= t1));
      c.b += __popcll(__ballot(k >= t2));
      c.c += __popcll(__ballot(k >= t3));
    }
    return block_count<NW>(c, slots, step);
  });
}

// The K best of n <= kMaxList distinct keys in LDS in descending order into
// sorted[0, K) (0 where there are fewer).  list is padded to a multiple of 4
// with 0.  Complete on return.
template <int NT>
__device__ __forceinline__ void rank_list(uint64_t* list, int n, int K, uint64_t* sorted) {
  const int tid = threadIdx.x;
  for (int j = tid; j < K; j += NT) sorted[j] = 0;
  if (tid < 4) list[n + tid] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    const uint64_t k = list[i];
    int rank = 0;
    for (int j = 0; j < n; j += 4) {
      const uint64_t k0 = list[j], k1 = list[j + 1], k2 = list[j + 2], k3 = list[j + 3];
      rank += (k0 > k) + (k1 > k) + (k2 > k) + (k3 > k);
    }
    if (rank < K) sorted[rank] = k;
  }
  __syncthreads();
}

// A row's outputs from its sorted keys and the mass of the others (by the
// first wave; `others` valid on its lanes, bad: a NaN or +inf was seen).
__device__ __forceinline__ void write_row(const TopOut& o, size_t row, const uint64_t* sorted, int K, Mass others,
                                          bool bad, float c, double c64) {
  const int lane = threadIdx.x;
  Mass top = mass_none();
  for (int j = lane; j < K; j += 64) {
    const uint64_t k = bad ? 0 : sorted[j];
    const float x = k ? key_value(k) : neg_inf();
    o.values[row * K + j] = x;
    o.ids[row * K + j] = k ? key_index(k) : -1;
    if (k) top = mass_add(top, Mass{x, 1.0f}, c);
  }
  top = wave_mass(top, c);
  if (lane == 0) {
    const double r = mass_log2(others, c, c64);
    const double l = log2_add(r, mass_log2(top, c, c64));
    const float nan = __builtin_nanf("");
    o.rest[row] = bad ? nan : static_cast<float>(r * 0.69314718055994530942);
    o.lse[row] = bad ? nan : static_cast<float>(l * 0.69314718055994530942);
    o.flags[row] = bad ? DSPARK_FLAG_NONFINITE : l == -__builtin_inf() ? DSPARK_FLAG_EMPTY_ROW : 0;
  }
}

// Mass of a granule's elements for which keep(value, index) holds.
template <typename T, class F>
__device__ __forceinline__ Mass gran_mass(const uint4& u, int e0, float c, F&& keep) {
  constexpr int EPL = Row<T>::EPL;
  float x[EPL], m = neg_inf();
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    x[j] = gran_elem(u, j, T{});
    if (!keep(x[j], e0 + j)) x[j] = neg_inf();
    m = fmaxf(m, x[j]);
  }
  if (m == neg_inf()) return mass_none();
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) s += __builtin_amdgcn_exp2f(mass_gap(x[j], m, c));
  return Mass{m, s};
}

template <int NT>
struct TopLds {
  union {
    Mass grp[kG * NT];       // the groups
    uint64_t cand[kG * NT];  // then the candidates
  };
  uint64_t list[kMaxList + 4];
  uint64_t sorted[DSPARK_MAX_TOP];
  uint16_t qual[NT == 64 ? 256 : 512];  // groups read again
  int slots[6 * (NT / 64)];
  int scan[2][NT / 64];
  float red[3][NT / 64];
  Mass mass[NT / 64];
};

// Candidates of a segment by a search over its elements (rows where the bound
// lets too many through): exactly K keys into s.cand, returned, and the mass of
// all other elements as each thread's share.
template <typename T, int NT>
__device__ __forceinline__ int exact_candidates(const Row<T>& r, int q0, int q1, int K, uint32_t kmax, float c,
                                                TopLds<NT>& s, int& step, Mass& others) {
  constexpr int NW = NT / 64;
  constexpr int EPL = Row<T>::EPL;
  const int tid = threadIdx.x;
  auto wave_total = [](int v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
    return v;
  };
  int n_lo = INT32_MAX;
  const uint32_t t = search_key<uint32_t>(kKeyNegInf + 1, kmax + 1, n_lo, K, K, [&](uint32_t t1, uint32_t t2, uint32_t t3) {
    Count3 n{0, 0, 0};
    for (int q = q0 + tid; q < q1; q += NT) {
      const uint4 u = gran_load(r, q);
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const uint32_t k = order_key(gran_elem(u, j, T{}));
        n.a += k >= t1;
        n.b += k >= t2;
        n.c += k >= t3;
      }
    }
    return block_count<NW>(Count3{wave_total(n.a), wave_total(n.b), wave_total(n.c)}, s.slots, step);
  });
  // of the elements at t the lowest indices: the least `last` with K keys above t or at t up to it
  int32_t last = r.V - 1;
  if (n_lo > K) {
    int32_t lo = -1;
    while (last - lo > 1) {
      const int32_t mid = lo + (last - lo) / 2;
      Count3 n{0, 0, 0};
      for (int q = q0 + tid; q < q1; q += NT) {
        const uint4 u = gran_load(r, q);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const uint32_t k = order_key(gran_elem(u, j, T{}));
          n.a += k > t || (k == t && q * EPL - r.head + j <= mid);
        }
      }
      n.a = wave_total(n.a);
      if (block_count<NW>(n, s.slots, step).a >= K) {
        last = mid;
      } else {
        lo = mid;
      }
    }
  }
  const uint64_t kth = cand_key(t, last);  // every key at or above it is in
  others = mass_none();
  int mine = 0;
  for (int q = q0 + tid; q < q1; q += NT) {
    const uint4 u = gran_load(r, q);
    others = mass_add(others, gran_mass<T>(u, q * EPL - r.head, c, [&](float x, int e) {
      const bool in = cand_key(order_key(x), e) >= kth && x > neg_inf();
      mine += in;
      return !in;
    }), c);
  }
  int total;
  int pos = block_scan<NW>(mine, s.scan[0], total);
  __syncthreads();
  for (int q = q0 + tid; q < q1; q += NT) {
    const uint4 u = gran_load(r, q);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float x = gran_elem(u, j, T{});
      const uint64_t k = cand_key(order_key(x), q * EPL - r.head + j);
      if (k >= kth && x > neg_inf()) s.cand[pos++] = k;
    }
  }
  __syncthreads();
  return total;
}

template <typename T, int NT, bool FINAL>
__global__ __launch_bounds__(NT, 4) void top_segment_kernel(const T* __restrict__ logits, int64_t items, int32_t V,
                                                            int32_t K, int32_t P, int32_t groups, float c, double c64,
                                                            TopSkip skip, TopOut o) {
  constexpr int NW = NT / 64;
  constexpr int EPL = Row<T>::EPL;
  constexpr int TILE = NT * kL;  // granules of a group over the workgroup
  __shared__ TopLds<NT> s;
  constexpr int QUAL = sizeof(s.qual) / sizeof(uint16_t), CAND = kG * NT;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  int step = 0;

  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const size_t row = static_cast<size_t>(item / P);
    const int seg = static_cast<int>(item - static_cast<int64_t>(row) * P);
    if (skipped(skip, row)) continue;
    const Row<T> r = make_row(logits + row * V, V);
    const int first = seg * groups * TILE;
    const int n = min(groups, (r.Q - first + TILE - 1) / TILE);  // <= 0: nothing left of this row

    // ---- stream: every group's maximum and mass ----
    float lmax = neg_inf();
    bool bad = false;
    {
      uint4 a[kL], b[kL];
      auto take = [&](const uint4(&u)[kL], int g) {
        const Mass m = group_mass<T, kL>(u, c);
        s.grp[g * NT + tid] = m;
        lmax = fmaxf(lmax, m.m);
        bad |= !(m.s >= 0.0f);
      };
      if (n > 0) group_load<T, NT, kL>(r, first, tid, a);
      for (int g = 0; g < n; g += 2) {
        if (g + 1 < n) group_load<T, NT, kL>(r, first + (g + 1) * TILE, tid, b);
        take(a, g);
        if (g + 1 >= n) break;
        if (g + 2 < n) group_load<T, NT, kL>(r, first + (g + 2) * TILE, tid, a);
        take(b, g + 1);
      }
    }

    // ---- range of the maxima, bad values ----
    float wmax = wave_max(lmax), wmin = -wave_max(-lmax);
    bad = __any(bad);
    if constexpr (NW > 1) {
      if (lane == 0) {
        s.red[0][wave] = wmax;
        s.red[1][wave] = wmin;
        s.red[2][wave] = bad ? 1.0f : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        wmax = fmaxf(wmax, s.red[0][w]);
        wmin = fminf(wmin, s.red[1][w]);
        bad |= s.red[2][w] != 0.0f;
      }
    }

    Mass others = mass_none();
    int nl = 0;  // candidates in s.list
    if (!bad && wmax > neg_inf()) {
      // ---- bound: at least K threads' (or groups') maxima reach it, or all finite ones ----
      const uint32_t kmax = order_key(wmax);
      uint32_t bound = kKeyNegInf + 1;
      if (K <= NT / 2) {
        const uint32_t k = order_key(lmax);
        int nb = wmin > neg_inf() ? NT : INT32_MAX;
        if (wmin > neg_inf()) {
          bound = order_key(wmin);
        } else {
          const int w = __popcll(__ballot(k >= bound));
          nb = block_count<NW>(Count3{w, 0, 0}, s.slots, step).a;
        }
        if (nb > K)
          bound = search_key<uint32_t>(bound, kmax + 1, nb, K, list_len(K), [&](uint32_t t1, uint32_t t2, uint32_t t3) {
            return block_count<NW>(Count3{static_cast<int>(__popcll(__ballot(k >= t1))), static_cast<int>(__popcll(__ballot(k >= t2))),
                                          static_cast<int>(__popcll(__ballot(k >= t3)))}, s.slots, step);
          });
      } else {
        auto groups_at = [&](uint32_t t1, uint32_t t2, uint32_t t3) {
          Count3 w{0, 0, 0};
          for (int g = 0; g < n; ++g) {
            const uint32_t k = order_key(s.grp[g * NT + tid].m);
            w.a += __popcll(__ballot(k >= t1));
            w.b += __popcll(__ballot(k >= t2));
            w.c += __popcll(__ballot(k >= t3));
          }
          return block_count<NW>(w, s.slots, step);
        };
        int nb = groups_at(bound, bound, bound).a;
        if (nb > K) bound = search_key<uint32_t>(bound, kmax + 1, nb, K, list_len(K), groups_at);
      }
      const float at = key_value(bound);

      // ---- the groups at the bound, in thread order; the mass of the others ----
      int mine = 0;
      float om = neg_inf(), os = 0.0f;
      for (int g = 0; g < n; ++g) {
        const float m = s.grp[g * NT + tid].m;
        if (m >= at) {
          ++mine;
        } else {
          om = fmaxf(om, m);
        }
      }
      int nq;
      int pos = block_scan<NW>(mine, s.scan[0], nq);
      const bool fits = nq <= QUAL;
      for (int g = 0; g < n; ++g) {
        const Mass m = s.grp[g * NT + tid];
        if (m.m >= at) {
          if (fits) s.qual[pos++] = static_cast<uint16_t>(g * NT + tid);
        } else if (m.m > neg_inf()) {
          os += m.s * __builtin_amdgcn_exp2f(mass_gap(m.m, om, c));
        }
      }
      others = Mass{om, os};
      __syncthreads();

      // ---- candidates: their elements at or above the bound, in thread order ----
      const int q1 = min(r.Q, first + n * TILE);
      int nc = CAND + 1;
      if (fits) {
        auto granule = [&](int i) {  // i-th granule read again
          const int g = s.qual[i / kL];
          return first + (g / NT * kL + i % kL) * NT + g % NT;
        };
        mine = 0;
        for (int i = tid; i < nq * kL; i += NT) {
          const int q = granule(i);
          if (q >= q1) continue;
          others = mass_add(others, gran_mass<T>(gran_load(r, q), 0, c, [&](float x, int) {
            mine += x >= at;
            return !(x >= at);
          }), c);
        }
        pos = block_scan<NW>(mine, s.scan[1], nc);
        if (nc <= CAND) {
          for (int i = tid; i < nq * kL; i += NT) {
            const int q = granule(i);
            if (q >= q1) continue;
            const uint4 u = gran_load(r, q);
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
              const float x = gran_elem(u, j, T{});
              if (x >= at) s.cand[pos++] = cand_key(order_key(x), q * EPL - r.head + j);
            }
          }
          __syncthreads();
        }
      }
      if (nc > CAND) nc = exact_candidates<T, NT>(r, first, q1, K, kmax, c, s, step, others);

      // ---- the K best of them or a few more; the others' mass ----
      const uint64_t lo = static_cast<uint64_t>(bound) << 32;
      const uint64_t t = list_bound<NT>(s.cand, nc, nc, K, lo, static_cast<uint64_t>(kmax + 1) << 32, s.slots, step);
      mine = 0;
      for (int i = tid; i < nc; i += NT) mine += s.cand[i] >= t;
      pos = block_scan<NW>(mine, s.scan[0], nl);
      for (int i = tid; i < nc; i += NT) {
        const uint64_t k = s.cand[i];
        if (k >= t) {
          s.list[pos++] = k;
        } else {
          others = mass_add(others, Mass{key_value(k), 1.0f}, c);
        }
      }
      __syncthreads();
      if constexpr (FINAL) {
        rank_list<NT>(s.list, nl, K, s.sorted);
        const uint64_t kth = s.sorted[K - 1];  // 0: fewer than K, all of them are in
        for (int i = tid; i < nl; i += NT)
          if (s.list[i] < kth) others = mass_add(others, Mass{key_value(s.list[i]), 1.0f}, c);
      }
    } else if constexpr (FINAL) {
      for (int j = tid; j < K; j += NT) s.sorted[j] = 0;
    }

    // ---- the segment's mass, outputs ----
    others = wave_mass(others, c);
    if constexpr (NW > 1) {
      if (lane == 0) s.mass[wave] = others;
      __syncthreads();
      if (wave == 0) others = wave_mass(lane < NW ? s.mass[lane] : mass_none(), c);
    } else {
      __syncthreads();
    }
    if constexpr (FINAL) {
      if (wave == 0) write_row(o, row, s.sorted, K, others, bad, c, c64);
    } else {
      const size_t part = row * P + seg;
      const int len = list_len(K);
      for (int j = tid; j < len; j += NT) o.keys[part * len + j] = j < nl ? s.list[j] : 0;
      if (tid == 0) o.parts[part] = bad ? Mass{neg_inf(), __builtin_nanf("")} : others;
    }
    __syncthreads();  // LDS is reused by the next item
  }
}

// The K best of the candidates of a row's P segments, one workgroup a row.
// FINAL: the row's outputs; otherwise its keys and mass at o.keys / o.parts as
// one segment's.
template <bool FINAL>
__global__ __launch_bounds__(kMergeThreads) void top_merge_kernel(const uint64_t* __restrict__ keys,
                                                                  const Mass* __restrict__ parts, int32_t R, int32_t K,
                                                                  int32_t P, float c, double c64, TopSkip skip,
                                                                  TopOut o) {
  constexpr int NT = kMergeThreads, NW = NT / 64;
  extern __shared__ uint64_t all[];  // P list_len(K) keys
  __shared__ uint64_t list[kMaxList + 4];
  __shared__ uint64_t sorted[DSPARK_MAX_TOP];
  __shared__ int slots[6 * NW];
  __shared__ int scan[2][NW];
  __shared__ uint64_t red[NW];
  __shared__ Mass shm[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int len = list_len(K), n = P * len;
  int step = 0;
  for (int row = blockIdx.x; row < R; row += gridDim.x) {
    const size_t at = static_cast<size_t>(row);
    if (skipped(skip, at)) continue;
    uint64_t top = 0;
    int found = 0;
    for (int i = tid; i < n; i += NT) {
      const uint64_t k = keys[at * n + i];
      all[i] = k;
      top = max(top, k);
      found += k != 0;
    }
    Mass others = mass_none();
    for (int p = tid; p < P; p += NT) others = mass_add(others, parts[at * P + p], c);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = max(top, static_cast<uint64_t>(__shfl_xor(static_cast<long long>(top), d, 64)));
    if (lane == 0) red[wave] = top;
    block_scan<NW>(found, scan[0], found);  // its barrier completes all and red
#pragma unroll
    for (int w = 0; w < NW; ++w) top = max(top, red[w]);
    const uint64_t t = list_bound<NT>(all, n, found, K, 1, top + 1, slots, step);
    int mine = 0, nl;
    for (int i = tid; i < n; i += NT) mine += all[i] >= t;
    int pos = block_scan<NW>(mine, scan[1], nl);
    for (int i = tid; i < n; i += NT) {
      const uint64_t k = all[i];
      if (k >= t) {
        list[pos++] = k;
      } else if (k) {
        others = mass_add(others, Mass{key_value(k), 1.0f}, c);
      }
    }
    __syncthreads();
    if constexpr (FINAL) {
      rank_list<NT>(list, nl, K, sorted);
      const uint64_t kth = sorted[K - 1];
      for (int i = tid; i < nl; i += NT)
        if (list[i] < kth) others = mass_add(others, Mass{key_value(list[i]), 1.0f}, c);
    }
    others = wave_mass(others, c);
    if (lane == 0) shm[wave] = others;
    __syncthreads();
    if (wave == 0) {
      others = wave_mass(lane < NW ? shm[lane] : mass_none(), c);
      const bool bad = !(others.s >= 0.0f);
      if constexpr (FINAL) {
        write_row(o, at, sorted, K, others, bad, c, c64);
      } else {
        for (int j = lane; j < len; j += 64) o.keys[at * len + j] = j < nl ? list[j] : 0;
        if (lane == 0) o.parts[at] = others;
      }
    }
    __syncthreads();
  }
}

// Rows are cut into segments of `groups` groups a thread.  Many short rows are
// taken by a wave each; others by workgroups of 256 threads, in shorter segments
// where that is needed to fill the GPU.
TopSplit top_split(int epl, int64_t R, int32_t V, int32_t K, bool any) {
  // granules of a row, at the least favourable alignment
  const int q = any ? (V + 2 * epl - 2) / epl : V / epl;
  TopSplit s{};
  const int wave = 64 * kL, block = 256 * kL;
  if (q <= 2 * wave || (q <= kG * wave && R >= 4096)) {
    s.NT = 64;
    s.groups = (q + wave - 1) / wave;
    s.P = 1;
    return s;
  }
  s.NT = 256;
  int g = std::min(kG, (q + block - 1) / block);
  // every segment's list goes through the merge's LDS
  const int most = 56 * 1024 / (list_len(K) * static_cast<int>(sizeof(uint64_t)));
  while (g > 1 && R * ((q + block * g - 1) / (block * g)) < 512) {
    const int h = g / 2;
    if ((q + block * h - 1) / (block * h) > most) break;
    g = h;
  }
  s.groups = g;
  s.P = (q + block * g - 1) / (block * g);
  return s;
}

template <typename T, bool FINAL>
hipError_t launch_segments(const T* logits, int32_t R, int32_t V, int32_t K, const TopSplit& sp, float c, double c64,
                           TopSkip skip, TopOut o, hipStream_t st) {
  const int64_t items = static_cast<int64_t>(R) * sp.P;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(items, kMaxGrid)));
  if (sp.NT == 64)
    DSPARK_LAUNCH("top_segment", (top_segment_kernel<T, 64, FINAL>), grid, dim3(64), 0, st, logits, items, V, K, sp.P,
                  sp.groups, c, c64, skip, o);
  else
    DSPARK_LAUNCH("top_segment", (top_segment_kernel<T, 256, FINAL>), grid, dim3(256), 0, st, logits, items, V, K, sp.P,
                  sp.groups, c, c64, skip, o);
  return hipGetLastError();
}

template <bool FINAL>
hipError_t launch_merge(const uint64_t* keys, const Mass* parts, int32_t R, int32_t K, int32_t P, float c, double c64,
                        TopSkip skip, TopOut o, hipStream_t st) {
  DSPARK_LAUNCH("top_merge", (top_merge_kernel<FINAL>), dim3(static_cast<unsigned>(std::min(R, kMaxGrid))),
                dim3(kMergeThreads), static_cast<size_t>(P) * list_len(K) * sizeof(uint64_t), st, keys, parts, R, K, P,
                c, c64, skip, o);
  return hipGetLastError();
}

bool any_alignment(const void* p, int32_t V, int epl) {
  return V % epl != 0 || (reinterpret_cast<uintptr_t>(p) & 15u) != 0;
}

}  // namespace

float mass_scale(float temperature) { return static_cast<float>(1.4426950408889634074 / static_cast<double>(temperature)); }
double mass_scale64(float temperature) { return 1.4426950408889634074 / static_cast<double>(temperature); }
int top_list_len(int K) { return list_len(K); }

// Sized for either type and any alignment of the rows.
TopPlan plan_top(int32_t R, int32_t V, int32_t K) {
  TopPlan p{};
  int P = 1;
  for (const int epl : {4, 8})
    for (const bool any : {false, true})
      if (any || V % epl == 0) P = std::max(P, top_split(epl, R, V, K, any).P);
  p.P = P;
  const size_t rp = static_cast<size_t>(R) * P;
  size_t off = 0;
  if (P > 1) {
    off = align_up(off + rp * list_len(K) * sizeof(uint64_t), 256);
    p.off_parts = off;
    off = align_up(off + rp * sizeof(Mass), 256);
  }
  p.bytes = off;
  return p;
}

hipError_t launch_top(const void* logits, int dtype, int32_t R, int32_t V, int32_t K, float temperature, float* values,
                      int32_t* ids, float* rest, float* lse, uint8_t* flags, void* ws, const TopPlan& pl,
                      hipStream_t st) {
  const int epl = dtype == DSPARK_BF16 ? 8 : 4;
  const TopSplit sp = top_split(epl, R, V, K, any_alignment(logits, V, epl));
  const float c = mass_scale(temperature);
  const double c64 = mass_scale64(temperature);
  char* w = static_cast<char*>(ws);
  TopOut o{values, ids, rest, lse, flags, nullptr, nullptr};
  const TopSkip none{nullptr, nullptr};
  if (sp.P == 1) {
    if (dtype == DSPARK_BF16)
      return launch_segments<uint16_t, true>(static_cast<const uint16_t*>(logits), R, V, K, sp, c, c64, none, o, st);
    return launch_segments<float, true>(static_cast<const float*>(logits), R, V, K, sp, c, c64, none, o, st);
  }
  o.keys = reinterpret_cast<uint64_t*>(w);
  o.parts = reinterpret_cast<Mass*>(w + pl.off_parts);
  hipError_t e;
  if (dtype == DSPARK_BF16)
    e = launch_segments<uint16_t, false>(static_cast<const uint16_t*>(logits), R, V, K, sp, c, c64, none, o, st);
  else
    e = launch_segments<float, false>(static_cast<const float*>(logits), R, V, K, sp, c, c64, none, o, st);
  if (e != hipSuccess) return e;
  return launch_merge<true>(o.keys, o.parts, R, K, sp.P, c, c64, none, o, st);
}

// Beams: rows of live beams, their lists left in the workspace.
int top_lists_segments(int dtype, int32_t R, int32_t V, int32_t K, const void* logits) {
  const int epl = dtype == DSPARK_BF16 ? 8 : 4;
  return top_split(epl, R, V, K, any_alignment(logits, V, epl)).P;
}

hipError_t launch_top_lists(const void* logits, int dtype, int32_t R, int32_t V, int32_t K, const float* scores,
                            const uint8_t* finished, uint64_t* keys, Mass* parts, hipStream_t st) {
  const int epl = dtype == DSPARK_BF16 ? 8 : 4;
  const TopSplit sp = top_split(epl, R, V, K, any_alignment(logits, V, epl));
  const TopSkip skip{scores, finished};
  const TopOut o{nullptr, nullptr, nullptr, nullptr, nullptr, keys, parts};
  const float c = mass_scale(1.0f);
  const double c64 = mass_scale64(1.0f);
  if (dtype == DSPARK_BF16)
    return launch_segments<uint16_t, false>(static_cast<const uint16_t*>(logits), R, V, K, sp, c, c64, skip, o, st);
  return launch_segments<float, false>(static_cast<const float*>(logits), R, V, K, sp, c, c64, skip, o, st);
}

hipError_t launch_top_lists_merge(const uint64_t* keys, const Mass* parts, int32_t R, int32_t K, int32_t P,
                                  const float* scores, const uint8_t* finished, uint64_t* out_keys, Mass* out_parts,
                                  hipStream_t st) {
  const TopOut o{nullptr, nullptr, nullptr, nullptr, nullptr, out_keys, out_parts};
  return launch_merge<false>(keys, parts, R, K, P, mass_scale(1.0f), mass_scale64(1.0f), TopSkip{scores, finished}, o,
                             st);
}

}  // namespace dspark
