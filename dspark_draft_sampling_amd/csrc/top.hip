// top.hip — the K highest logits of each row with the mass of the others.
//
// Semantics (include/dspark.h, dspark_top_logits): per row the K largest
// logits in descending order, the lower index first among equal ones, the
// natural logarithm of sum exp(x / T) over the other tokens and over all.
//
// One pass over the row.  A workgroup takes a row (or, of rows longer than it can
// hold, a segment), every thread up to 16 groups of 4 granules, and keeps of each
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
// Rows cut into several segments leave each segment's candidates and mass in the
// workspace; top_merge_kernel takes the K best of those.  Every choice is by unique keys and every sum in an order set
// by positions, so results do not depend on timing.
//
// Many rows are bound by HBM: 14336 rows of 129280 bf16, K = 64: 633 us, 5.9 TB/s,
// 15% more fetched than the rows hold (the groups read again; the first version,
// with a running maximum and a candidate test an element, 1255).  One row a compute
// unit is bound by its VALU and then by the tail's barriers: one row of 129280, K =
// 8: 13 us, 5 of them the stream; 256 rows 18.5.
#include <algorithm>

#include "common.hpp"
#include "rowstream.hpp"
#include "vocab.hpp"

namespace dspark {
namespace {

constexpr int kMergeThreads = 256;
constexpr int kMaxGrid = 1 << 22;  // workgroups of a launch; more are further launches

// Groups of a thread at most (they are kept in LDS) and keys that are ranked at
// once: more are first cut by a search.
template <int NT>
struct TopCaps {
  static constexpr int kG = NT == 512 ? 8 : 16;
  static constexpr int kRank = NT == 64 ? 448 : 512;
};

// Candidates a list may hold beyond K: the searches stop at the first bound
// within it.
__host__ __device__ constexpr int list_len(int K) { return K + K / 4 + 8; }
constexpr int kMaxList = list_len(DSPARK_MAX_TOP);

// What a launch leaves: a segment's candidates and mass for the merge, a row's
// outputs, or a beam's candidates with their scores for beam_final.
enum TopMode { kLists, kRows, kBeams };

struct TopOut {
  float* values;   // [R, K]
  int32_t* ids;    // [R, K]
  float* rest;     // [R]
  float* lse;      // [R]
  uint8_t* flags;  // [R]
  uint64_t* keys;  // a segment's candidates [R, P, list_len(K)], or a beam's K best in order [R, K]; 0: none
  Mass* parts;     // [R, P]: the mass of its other elements
};

// Beams (scores NULL: plain rows).  An ended beam is one candidate, a beam
// whose score is not finite is none; their rows are not read.
struct TopBeams {
  const float* scores;      // [R]
  const uint8_t* finished;  // [R] or NULL
  int32_t eos;
  uint64_t* sums;  // [R, K]: order keys of the candidates' 64-bit scores
  uint8_t* flags;  // [R]
};

// Whether the row is a beam that is not read; in mode kBeams its candidates
// are written here.
template <int NT, TopMode MODE>
__device__ __forceinline__ bool unread_beam(const TopBeams& bm, const TopOut& o, size_t row, int K) {
  if (MODE == kRows || !bm.scores) return false;
  const float sc = bm.scores[row];
  const bool ended = bm.finished && bm.finished[row];
  if (sc > neg_inf() && sc < pos_inf() && !ended) return false;
  if constexpr (MODE == kBeams) {
    const bool fine = sc > neg_inf() && sc < pos_inf();
    for (int j = threadIdx.x; j < K; j += NT) {
      const bool one = fine && j == 0;
      bm.sums[row * K + j] = one ? order_key(static_cast<double>(sc)) : kKey64NegInf;
      o.keys[row * K + j] = one ? cand_key(0, bm.eos) : 0;
    }
    if (threadIdx.x == 0) bm.flags[row] = isnan(sc) || sc == pos_inf() ? DSPARK_FLAG_NONFINITE : 0;
  }
  return true;
}

// A key with K <= count(>= it) <= list_len(K) among n distinct keys in LDS (0:
// none), all of them below hi and the others at or above lo; lo itself where
// there are no more.  found: the number of keys that are not 0.
template <int NT>
__device__ __forceinline__ uint64_t list_bound(const uint64_t* cand, int n, int found, int K, uint64_t lo, uint64_t hi,
                                               uint64_t* slots, int& step) {
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

template <int NT>
struct RankLds {
  uint16_t rank[TopCaps<NT>::kRank];
  Mass others[NT / 64];
  float top[NT / 64];
  double sum[NT / 64];
};

// Outputs of a row or beam from its n candidates in LDS (distinct keys, 0s
// among them are none; nv of them are not 0) and the threads'
// shares of the mass of all other elements.  A candidate's rank is the number of
// greater keys; those below K are the outputs, the others' mass joins the rest.
// list is complete, with 4 zeros after it.
// wmax: the row's largest value.  bad, or a NaN mass: a NaN or +inf was seen.
// A beam's normaliser is formed in 64 bits, its K best tokens one by one.
template <int NT, TopMode MODE>
__device__ __forceinline__ void write_best(uint64_t* list, int n, int nv, int K, Mass others, bool bad, float wmax,
                                           size_t row, float c, double c64, const TopBeams& bm, const TopOut& o,
                                           RankLds<NT>& s) {
  constexpr int NW = NT / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  float top = 0.0f;  // mass of the outputs relative to wmax
  double sum = 0.0;
  for (int i = tid; i < n; i += NT) {
    const uint64_t k = list[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 4) {
      const uint64_t k0 = list[j], k1 = list[j + 1], k2 = list[j + 2], k3 = list[j + 3];
      rank += (k0 > k) + (k1 > k) + (k2 > k) + (k3 > k);
    }
    if (MODE == kBeams) s.rank[i] = static_cast<uint16_t>(rank);
    if (k == 0) continue;
    const float x = key_value(k);
    if (rank >= K) {
      others = mass_add(others, Mass{x, 1.0f}, c);
    } else if constexpr (MODE == kRows) {
      o.values[row * K + rank] = x;
      o.ids[row * K + rank] = key_index(k);
      top += __builtin_amdgcn_exp2f(mass_gap(x, wmax, c));
    } else {
      sum += exp2_64((static_cast<double>(x) - static_cast<double>(wmax)) * c64);
    }
  }
  others = wave_mass(others, c);
  if constexpr (MODE == kRows)
    top = wave_sum(top);
  else
    sum = wave_sum64(sum);
  if constexpr (NW > 1) {
    if (lane == 0) {
      s.others[wave] = others;
      if constexpr (MODE == kRows)
        s.top[wave] = top;
      else
        s.sum[wave] = sum;
    }
    __syncthreads();
    others = wave_mass(lane < NW ? s.others[lane] : mass_none(), c);
    if constexpr (MODE == kRows) {
      top = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) top += s.top[w];
    } else {
      sum = 0.0;
#pragma unroll
      for (int w = 0; w < NW; ++w) sum += s.sum[w];
    }
  }
  bad |= !(others.s >= 0.0f);
  if (bad) nv = 0;
  if constexpr (MODE == kRows) {
    if (bad) __syncthreads();  // its candidates have been written: now none are there
    for (int j = nv + tid; j < K; j += NT) {
      o.values[row * K + j] = neg_inf();
      o.ids[row * K + j] = -1;
    }
    if (tid == 0) {
      const double r = mass_log2(others, c, c64);
      const double l = log2_add(r, mass_log2(Mass{wmax, top}, c, c64));
      const float nan = __builtin_nanf("");
      o.rest[row] = bad ? nan : static_cast<float>(r * 0.69314718055994530942);
      o.lse[row] = bad ? nan : static_cast<float>(l * 0.69314718055994530942);
      o.flags[row] = bad ? DSPARK_FLAG_NONFINITE : l == -__builtin_inf() ? DSPARK_FLAG_EMPTY_ROW : 0;
    }
  } else {
    const double ref = static_cast<double>(wmax);
    const double lse = ref + log2_64(sum + exp2_64(mass_log2(others, c, c64) - ref * c64)) / c64;
    const double sc = static_cast<double>(bm.scores[row]);
    if (!bad)
      for (int i = tid; i < n; i += NT) {
        const int rank = s.rank[i];
        const uint64_t k = list[i];
        if (k == 0 || rank >= K) continue;
        bm.sums[row * K + rank] = order_key(sc + (static_cast<double>(key_value(k)) - lse));
        o.keys[row * K + rank] = k;
      }
    for (int j = nv + tid; j < K; j += NT) {
      bm.sums[row * K + j] = kKey64NegInf;
      o.keys[row * K + j] = 0;
    }
    if (tid == 0) bm.flags[row] = bad ? DSPARK_FLAG_NONFINITE : nv == 0 ? DSPARK_FLAG_EMPTY_ROW : 0;
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
  float s = 0.0f;  // a NaN, too, ends up here
  if (__any(fabsf(m) > kHugeLogit && m > neg_inf())) {
    const float ref = m > neg_inf() ? m : 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      s += __builtin_amdgcn_exp2f(fabsf(ref) > kHugeLogit ? (x[j] - ref) * c : fmaf(x[j], c, -(ref * c)));
  } else {
    const float r = m > neg_inf() ? m * c : 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) s += __builtin_amdgcn_exp2f(fmaf(x[j], c, -r));
  }
  return Mass{m, s};
}

template <int NT>
struct TopLds {
  static constexpr int kCand = TopCaps<NT>::kG * NT;
  union {
    Mass grp[kCand];           // the groups
    uint64_t cand[kCand + 4];  // then the candidates
  };
  uint64_t list[kMaxList + 4];
  uint16_t qual[NT == 64 ? 256 : 512];  // groups read again
  uint64_t slots[2 * (NT / 64)];
  int scan[2][NT / 64];
  float red[3][NT / 64];
  Mass mass[NT / 64];
  RankLds<NT> out;
};

// Candidates of a segment by a search over its elements (rows where the bound
// lets too many through): exactly K keys into cand, their number returned, and
// the mass of all other elements as each thread's share.  scan: NW ints.
template <typename T, int NT>
__device__ __forceinline__ int exact_candidates(const Row<T>& r, int q0, int q1, int K, uint32_t kmax, float c,
                                                uint64_t* cand, uint64_t* slots, int* scan, int& step, Mass& others) {
  constexpr int NW = NT / 64;
  constexpr int EPL = Row<T>::EPL;
  const int tid = threadIdx.x;
  auto wave_total = [](int v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
    return v;
  };
  int n_lo = INT32_MAX;
  const uint32_t t = search_key<uint32_t>(kKeyNegInf + 1, kmax + 1, n_lo, K, K, [&](uint32_t t1, uint32_t t2,
                                                                                    uint32_t t3) {
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
    return block_count<NW>(Count3{wave_total(n.a), wave_total(n.b), wave_total(n.c)}, slots, step);
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
      if (block_count<NW>(n, slots, step).a >= K) {
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
  int pos = block_scan<NW>(mine, scan, total);
  __syncthreads();
  for (int q = q0 + tid; q < q1; q += NT) {
    const uint4 u = gran_load(r, q);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float x = gran_elem(u, j, T{});
      const uint64_t k = cand_key(order_key(x), q * EPL - r.head + j);
      if (k >= kth && x > neg_inf()) cand[pos++] = k;
    }
  }
  if (tid < 4) cand[total + tid] = 0;
  __syncthreads();
  return total;
}

template <typename T, int NT, int kL, TopMode MODE>
__global__ __launch_bounds__(NT, 4) void top_segment_kernel(const T* __restrict__ logits, int64_t base, int32_t V,
                                                            int32_t K, int32_t P, int32_t groups, float c, double c64,
                                                            TopBeams bm, TopOut o) {
  constexpr int NW = NT / 64;
  constexpr int EPL = Row<T>::EPL, G = TopCaps<NT>::kG;
  constexpr int TILE = NT * kL;  // granules of a group over the workgroup
  __shared__ TopLds<NT> s;
  constexpr int QUAL = sizeof(s.qual) / sizeof(uint16_t), CAND = TopLds<NT>::kCand;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  int step = 0;

  const int64_t item = base + blockIdx.x;
  const size_t row = static_cast<size_t>(item / P);
  const int seg = static_cast<int>(item - static_cast<int64_t>(row) * P);
  if (unread_beam<NT, MODE>(bm, o, row, K)) return;
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
  int nl = 0;  // candidates listed
  uint64_t* list = s.cand;
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
          Count3 w{0, 0, 0};
          w.a = __popcll(__ballot(k >= t1));
          w.b = __popcll(__ballot(k >= t2));
          w.c = __popcll(__ballot(k >= t3));
          return block_count<NW>(w, s.slots, step);
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
    uint32_t in = 0;  // bit g: group g is at the bound
    int mine = 0;
    Mass share[G / 4];
#pragma unroll
    for (int g0 = 0; g0 < G; g0 += 4) {
      share[g0 / 4] = mass_none();
      if (g0 < n) {
        Mass m[4];  // the reads overlap
        uint32_t out = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          m[k] = s.grp[min(g0 + k, n - 1) * NT + tid];
          const bool ok = g0 + k < n, at_bound = ok && m[k].m >= at;
          in |= at_bound ? 1u << (g0 + k) : 0u;
          out |= ok && !at_bound ? 1u << k : 0u;
        }
        share[g0 / 4] = mass_sum<4>(m, out, c);
      }
    }
    mine = __popc(in);
    int nq;
    int pos = block_scan<NW>(mine, s.scan[0], nq);
    const bool fits = nq <= QUAL;
    if (fits)
      for (; in != 0; in &= in - 1) s.qual[pos++] = static_cast<uint16_t>((__ffs(in) - 1) * NT + tid);
    others = mass_sum<G / 4>(share, (1u << (G / 4)) - 1, c);
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
      uint4 mineu = make_uint4(0, 0, 0, 0);  // the thread's first granule
      for (int i = tid; i < nq * kL; i += NT) {
        const int q = granule(i);
        if (q >= q1) continue;
        const uint4 u = gran_load(r, q);
        if (i == tid) mineu = u;
        others = mass_add(others, gran_mass<T>(u, 0, c, [&](float x, int) {
          mine += x >= at;
          return !(x >= at);
        }), c);
      }
      pos = block_scan<NW>(mine, s.scan[1], nc);
      if (nc <= CAND && mine > 0) {
        for (int i = tid; i < nq * kL; i += NT) {
          const int q = granule(i);
          if (q >= q1) continue;
          const uint4 u = i == tid ? mineu : gran_load(r, q);
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            const float x = gran_elem(u, j, T{});
            if (x >= at) s.cand[pos++] = cand_key(order_key(x), q * EPL - r.head + j);
          }
        }
      }
      if (nc <= CAND && tid < 4) s.cand[nc + tid] = 0;
      __syncthreads();
    }
    if (nc > CAND) nc = exact_candidates<T, NT>(r, first, q1, K, kmax, c, s.cand, s.slots, s.scan[0], step, others);

    // ---- the K best of them or a few more; the others' mass ----
    nl = nc;
    if (nc > (MODE == kLists ? list_len(K) : NT == 64 ? 2 * list_len(K) : TopCaps<NT>::kRank)) {
      const uint64_t t = list_bound<NT>(s.cand, nc, nc, K, static_cast<uint64_t>(bound) << 32,
                                        static_cast<uint64_t>(kmax + 1) << 32, s.slots, step);
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
      if (tid < 4) s.list[nl + tid] = 0;
      __syncthreads();
      list = s.list;
    }
  }
  if constexpr (MODE != kLists) {
    write_best<NT, MODE>(list, nl, nl, K, others, bad, wmax, row, c, c64, bm, o, s.out);
  } else {
    const size_t part = row * P + seg;
    const int len = list_len(K);
    for (int j = tid; j < len; j += NT) o.keys[part * len + j] = j < nl ? list[j] : 0;
    others = wave_mass(others, c);
    if constexpr (NW > 1) {
      if (lane == 0) s.mass[wave] = others;
      __syncthreads();
      others = wave_mass(lane < NW ? s.mass[lane] : mass_none(), c);
    }
    if (tid == 0) o.parts[part] = bad ? Mass{neg_inf(), __builtin_nanf("")} : others;
  }
}

// Short rows: one wave a row, the row in registers (L granules a lane); 400000 rows
// of 1500 bf16, K = 20: 532 us, 2.3 TB/s, bound by VALU (the exponentials, and a
// search and ranking for every 1500 elements).  The
// bound comes from the granules' maxima; candidates leave the registers, and one
// pass of exponentials over what stays gives the others' mass.  Nothing is read
// twice.
constexpr int kSmallCand = TopCaps<64>::kRank;

template <typename T, int L, TopMode MODE>
__global__ __launch_bounds__(64, 4) void top_small_kernel(const T* __restrict__ logits, int32_t base, int32_t V,
                                                          int32_t K, float c, double c64, TopBeams bm, TopOut o) {
  constexpr int EPL = Row<T>::EPL;
  __shared__ uint64_t cand[kSmallCand + 4];
  __shared__ RankLds<64> out;
  const int lane = threadIdx.x;
  int step = 0;
  const size_t at_row = static_cast<size_t>(base) + blockIdx.x;
  if (unread_beam<64, MODE>(bm, o, at_row, K)) return;
  const Row<T> r = make_row(logits + at_row * V, V);
  uint4 u[L];
  group_load<T, 64, L>(r, 0, lane, u);
  float gm[L], lmax = neg_inf();
#pragma unroll
  for (int i = 0; i < L; ++i) {
    gm[i] = neg_inf();
#pragma unroll
    for (int j = 0; j < EPL; ++j) gm[i] = fmaxf(gm[i], gran_elem(u[i], j, T{}));
    lmax = fmaxf(lmax, gm[i]);
  }
  const float wmax = wave_max(lmax);
  bool bad = wmax == pos_inf(), slow = false;
  Mass others = mass_none();
  int nl = 0;  // candidates listed
  if (!bad && wmax > neg_inf()) {
    // ---- bound: at least K granules (or all finite ones) reach it ----
    const uint32_t kmax = order_key(wmax);
    const float wmin = -wave_max(-lmax);
    auto granules_at = [&](uint32_t t1, uint32_t t2, uint32_t t3) {
      Count3 n{0, 0, 0};
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const uint32_t k = order_key(gm[i]);
        n.a += __popcll(__ballot(k >= t1));
        n.b += __popcll(__ballot(k >= t2));
        n.c += __popcll(__ballot(k >= t3));
      }
      return n;
    };
    uint32_t bound = K <= 64 && wmin > neg_inf() ? order_key(wmin) : kKeyNegInf + 1;
    int nb = granules_at(bound, bound, bound).a;
    if (nb > K) bound = search_key<uint32_t>(bound, kmax + 1, nb, K, list_len(K), granules_at);
    // ---- the elements that reach it leave the registers ----
    const float at = key_value(bound);
    int mine = 0;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      repack(u[i]);
      if (__any(gm[i] >= at)) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) mine += gran_elem(u[i], j, T{}) >= at;
      }
    }
    int pos = block_scan<1>(mine, nullptr, nl);
    slow = nl > kSmallCand;
    if (slow) {
      nl = exact_candidates<T, 64>(r, 0, r.Q, K, kmax, c, cand, nullptr, nullptr, step, others);
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i) {
        repack(u[i]);
        if (__any(gm[i] >= at)) {
          uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            const float x = gran_elem(u[i], j, T{});
            if (x >= at) {
              cand[pos++] = cand_key(order_key(x), (i * 64 + lane) * EPL - r.head + j);
              if constexpr (sizeof(T) == 2)
                w[j / 2] = (j & 1) ? (w[j / 2] & 0x0000ffffu) | 0xFF800000u : (w[j / 2] & 0xffff0000u) | 0xFF80u;
              else
                w[j] = 0xFF800000u;
            }
          }
          u[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (lane < 4) cand[nl + lane] = 0;
      __syncthreads();
    }
  }
  if (!slow) {
#pragma unroll
    for (int i = 0; i < L; i += 4) {
      uint4 v[4] = {u[i], u[i + 1], u[i + 2], u[i + 3]};
#pragma unroll
      for (int k = 0; k < 4; ++k) repack(v[k]);
      others = mass_add(others, group_mass<T, 4>(v, c), c);
    }
  }
  write_best<64, MODE>(cand, nl, nl, K, others, bad, wmax, at_row, c, c64, bm, o, out);
}

// The K best of the candidates of a row's P segments (in: their lists), one
// workgroup a row; kRows or kBeams.  P (5 K / 4 + 8) keys: a launch's latency.
template <TopMode MODE>
__global__ __launch_bounds__(kMergeThreads) void top_merge_kernel(const uint64_t* __restrict__ in,
                                                                  const Mass* __restrict__ parts, int32_t base,
                                                                  int32_t K, int32_t P, float c, double c64,
                                                                  TopBeams bm, TopOut o) {
  constexpr int NT = kMergeThreads, NW = NT / 64;
  extern __shared__ uint64_t all[];  // P list_len(K) keys and 4 more
  __shared__ uint64_t list[kMaxList + 4];
  __shared__ RankLds<NT> out;
  __shared__ uint64_t slots[2 * NW];
  __shared__ int scan[2][NW];
  __shared__ uint64_t red[2][NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int len = list_len(K), n = P * len;
  int step = 0;
  const size_t at = static_cast<size_t>(base) + blockIdx.x;
  if (unread_beam<NT, MODE>(bm, o, at, K)) return;
  uint64_t top = 0, low = ~0ull;
  int found = 0;
  for (int i = tid; i < n; i += NT) {
    const uint64_t k = in[at * n + i];
    all[i] = k;
    top = max(top, k);
    if (k) low = min(low, k);
    found += k != 0;
  }
  Mass others = mass_none();
  for (int p = tid; p < P; p += NT) others = mass_add(others, parts[at * P + p], c);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    top = max(top, static_cast<uint64_t>(__shfl_xor(static_cast<long long>(top), d, 64)));
    low = min(low, static_cast<uint64_t>(__shfl_xor(static_cast<long long>(low), d, 64)));
  }
  if (tid < 4) all[n + tid] = 0;
  if (lane == 0) {
    red[0][wave] = top;
    red[1][wave] = low;
  }
  block_scan<NW>(found, scan[0], found);  // its barrier completes all and red
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    top = max(top, red[0][w]);
    low = min(low, red[1][w]);
  }
  uint64_t* best = all;
  int nl = n;
  if (n > 2 * list_len(K)) {
    const uint64_t t = list_bound<NT>(all, n, found, K, found ? low : 1, top + 1, slots, step);
    int mine = 0;
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
    if (tid < 4) list[nl + tid] = 0;
    __syncthreads();
    best = list;
  }
  const int nv = best == all ? found : nl;
  write_best<NT, MODE>(best, nl, nv, K, others, false, found ? key_value(top) : neg_inf(), at, c, c64, bm, o, out);
}

// Rows are cut into segments of `groups` groups a thread; groups = 0: short rows,
// NT granules a lane of one wave.  Measured, one side against the other:
//  * a row in one wave's registers, up to 512 granules: 400000 rows of 1500 bf16, K =
//    20, 532 us against 974 of the segment kernel with one wave a row (K = 100 and
//    100000 rows of 3500: 415 against 1150 with 256 threads);
//  * one wave a row where rows are many, of up to 16 groups for K <= 32, whose bound
//    comes from 64 threads' maxima (3000 rows of 20000 bf16, K = 20: 31 us against 42
//    of 256 threads), of up to 4 for larger K, whose bound comes from the groups'
//    (20000 rows of 8000, K = 100: 193 against 226; 5000 of 20000, K = 64: 87
//    against 75);
//  * 512 threads for long rows that have a compute unit each: 256 rows of 129280 bf16
//    17.7 us against 21.3 of 256 threads, 128 rows of 50257 11.8 against 13.7; 300 rows
//    of 90000 20.2 against 18.5, 700 of 129280 49 against 43 (several workgroups of
//    256 share a compute unit, and one's tail runs beside the others' streams);
//  * several segments a row only where one cannot hold it: the merge is a launch
//    more (64 rows of 129280: 17 us against 16 with one; one row: 13 against 15, less
//    than the second launch costs the host).
TopSplit top_split(int epl, int64_t R, int32_t V, int32_t K, bool any) {
  // granules of a row, at the least favourable alignment
  const int q = any ? (V + 2 * epl - 2) / epl : V / epl;
  TopSplit s{};
  s.P = 1;
  if (q <= 8 * 64) {
    s.NT = q <= 4 * 64 ? 4 : 8;
    return s;
  }
  int most, kL = 4;
  if (R >= 2048 && q <= (K <= 32 ? TopCaps<64>::kG : 4) * 64 * kL) {
    s.NT = 64;
    most = TopCaps<64>::kG;
  } else if (q > 4 * 256 * kL && R <= 256) {
    s.NT = 512;
    most = TopCaps<512>::kG;
  } else {
    s.NT = 256;
    most = TopCaps<256>::kG;
  }
  // float32 rows too long for one segment of 4 granules a group take 8: the
  // groups then hold 32 logits, as those of bf16 do
  if (epl == 4 && q > most * s.NT * kL) kL = 8;
  s.L = kL;
  const int need = (q + s.NT * kL - 1) / (s.NT * kL);  // groups of a thread over the row
  s.P = (need + most - 1) / most;
  s.groups = (need + s.P - 1) / s.P;
  return s;
}

template <typename T, TopMode MODE>
hipError_t launch_segments(const T* logits, int32_t R, int32_t V, int32_t K, const TopSplit& sp, float c, double c64,
                           const TopBeams& bm, const TopOut& o, hipStream_t st) {
  const int64_t items = static_cast<int64_t>(R) * sp.P;
#define DSPARK_TOP(NT, L) \
  DSPARK_LAUNCH("top_segment", (top_segment_kernel<T, NT, L, MODE>), grid, dim3(NT), 0, st, logits, base, V, K, sp.P, \
                sp.groups, c, c64, bm, o)
  for (int64_t base = 0; base < items; base += kMaxGrid) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(items - base, kMaxGrid)));
    if (sp.NT == 64)
      DSPARK_TOP(64, 4);
    else if (sp.L == 4 && sp.NT == 256)
      DSPARK_TOP(256, 4);
    else if (sp.L == 4)
      DSPARK_TOP(512, 4);
    else if constexpr (sizeof(T) == 4) {
      if (sp.NT == 256)
        DSPARK_TOP(256, 8);
      else
        DSPARK_TOP(512, 8);
    }
  }
#undef DSPARK_TOP
  return hipGetLastError();
}

template <typename T, TopMode MODE>
hipError_t launch_small(const T* logits, int32_t R, int32_t V, int32_t K, const TopSplit& sp, float c, double c64,
                        const TopBeams& bm, const TopOut& o, hipStream_t st) {
#define DSPARK_SMALL(L)                                                                                             \
  DSPARK_LAUNCH("top_small", (top_small_kernel<T, L, MODE>), grid, dim3(64), 0, st, logits, base, V, K, c, c64, bm, o)
  for (int32_t base = 0, n; base < R; base += n) {
    n = std::min(R - base, kMaxGrid);
    const dim3 grid(static_cast<unsigned>(n));
    if (sp.NT == 4)
      DSPARK_SMALL(4);
    else
      DSPARK_SMALL(8);
  }
#undef DSPARK_SMALL
  return hipGetLastError();
}

// The segments' candidates, then (rows of several segments) the merge.
template <TopMode MODE>
hipError_t launch_rows(const void* logits, int dtype, int32_t R, int32_t V, int32_t K, const TopSplit& sp,
                       float temperature, const TopBeams& bm, TopOut o, uint64_t* lists, Mass* parts, hipStream_t st) {
  const float c = mass_scale(temperature);
  const double c64 = mass_scale64(temperature);
  const uint16_t* h = static_cast<const uint16_t*>(logits);
  const float* f = static_cast<const float*>(logits);
  if (sp.groups == 0)
    return dtype == DSPARK_BF16 ? launch_small<uint16_t, MODE>(h, R, V, K, sp, c, c64, bm, o, st)
                                : launch_small<float, MODE>(f, R, V, K, sp, c, c64, bm, o, st);
  if (sp.P == 1)
    return dtype == DSPARK_BF16 ? launch_segments<uint16_t, MODE>(h, R, V, K, sp, c, c64, bm, o, st)
                                : launch_segments<float, MODE>(f, R, V, K, sp, c, c64, bm, o, st);
  TopOut part = o;
  part.keys = lists;
  part.parts = parts;
  const hipError_t e = dtype == DSPARK_BF16 ? launch_segments<uint16_t, kLists>(h, R, V, K, sp, c, c64, bm, part, st)
                                            : launch_segments<float, kLists>(f, R, V, K, sp, c, c64, bm, part, st);
  if (e != hipSuccess) return e;
  for (int32_t base = 0, n; base < R; base += n) {
    n = std::min(R - base, kMaxGrid);
    DSPARK_LAUNCH("top_merge", (top_merge_kernel<MODE>), dim3(static_cast<unsigned>(n)), dim3(kMergeThreads),
                  (static_cast<size_t>(sp.P) * list_len(K) + 4) * sizeof(uint64_t), st, lists, parts, base, K, sp.P, c,
                  c64, bm, o);
  }
  return hipGetLastError();
}

bool any_alignment(const void* p, int32_t V, int epl) {
  return V % epl != 0 || (reinterpret_cast<uintptr_t>(p) & 15u) != 0;
}

}  // namespace

double mass_scale64(float temperature) { return 1.4426950408889634074 / static_cast<double>(temperature); }
float mass_scale(float temperature) { return static_cast<float>(mass_scale64(temperature)); }

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
  char* w = static_cast<char*>(ws);
  return launch_rows<kRows>(logits, dtype, R, V, K, top_split(epl, R, V, K, any_alignment(logits, V, epl)), temperature,
                            TopBeams{}, TopOut{values, ids, rest, lse, flags, nullptr, nullptr},
                            reinterpret_cast<uint64_t*>(w), reinterpret_cast<Mass*>(w + pl.off_parts), st);
}

hipError_t launch_beam_rows(const void* logits, int dtype, int32_t R, int32_t V, int32_t M, const float* scores,
                            const uint8_t* finished, int32_t eos, uint64_t* sums, uint64_t* keys, uint8_t* flags,
                            void* ws, const TopPlan& pl, hipStream_t st) {
  const int epl = dtype == DSPARK_BF16 ? 8 : 4;
  char* w = static_cast<char*>(ws);
  return launch_rows<kBeams>(logits, dtype, R, V, M, top_split(epl, R, V, M, any_alignment(logits, V, epl)), 1.0f,
                             TopBeams{scores, finished, eos, sums, flags},
                             TopOut{nullptr, nullptr, nullptr, nullptr, nullptr, keys, nullptr},
                             reinterpret_cast<uint64_t*>(w), reinterpret_cast<Mass*>(w + pl.off_parts), st);
}

}  // namespace dspark
