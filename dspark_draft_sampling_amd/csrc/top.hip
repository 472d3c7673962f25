// top.hip — the K highest logits of each row with the mass of the others.
//
// Semantics (include/dspark.h, dspark_top_logits): per row the K largest
// logits in descending order, the lower index first among equal ones, the
// natural logarithm of sum exp(x / T) over the other tokens and over all.
//
// One pass over the row.  A workgroup takes a segment of a row, every thread
// G groups of L 16-byte granules, and keeps of each group only its maximum
// and its mass (rowstream.hpp): one exponential and about 7.5 VALU slots per
// element, no running maximum and no candidate test in the stream.  K or a
// few more of the group maxima, found by a bisection over their order keys,
// bound the K-th largest logit from below: only the granules of those groups
// (about K L of them) are read again, from the caches, and the elements at or
// above the bound become candidates in LDS.  The candidates' unique 64-bit
// keys (value, then index) give each its rank by counting.  The mass of the
// rest is summed from the groups below the bound and, element by element,
// from the few others: nothing is subtracted, so it keeps its relative
// accuracy however small it is beside the top.
//
// The bound can let too many elements through (rows of equal values, a few
// finite values in few groups): then the K-th key is found by bisection over
// the segment itself, read once per step.
//
// Rows cut into several segments (few rows, or long ones) leave each
// segment's K best keys and mass in the workspace; top_merge_kernel takes the
// K best of those.  Every choice is by unique keys and every sum in an order
// set by positions, so results do not depend on timing.
#include <algorithm>

#include "common.hpp"
#include "internal.hpp"
#include "rowstream.hpp"

namespace dspark {
namespace {

constexpr int kMergeThreads = 256;
constexpr int kMaxGrid = 1 << 20;  // workgroups of a launch; each then takes several items

template <int NT>
struct TopCaps {
  static constexpr int kCand = NT == 64 ? 1024 : 2048;  // candidates in LDS
  static constexpr int kQual = NT == 64 ? 512 : 1024;   // groups read again
};

// The K best keys of n candidates in LDS (unique, 0: none) in descending
// order into sorted[0, K) (0 where there are fewer).  Every thread calls it;
// sorted is complete on return.
template <int NT>
__device__ __forceinline__ void rank_top(const uint64_t* cand, int n, int K, uint64_t* sorted, int* slots, int& step) {
  constexpr int NW = NT / 64;
  const int tid = threadIdx.x;
  uint64_t t = 1;
  const int most = K + K / 4 + 8;
  if (n > most) {
    int n_lo = 0;
    {
      int c = 0;
      for (int i = tid; i < (n + 63) / 64 * 64; i += NT) c += __popcll(__ballot(i < n && cand[min(i, n - 1)] != 0));
      n_lo = block_count<NW>(c, slots, step++);
    }
    if (n_lo > most)
      t = bisect<uint64_t>(1, ~0ull, n_lo, K, most, [&](uint64_t mid) {
        int c = 0;
        for (int i = tid; i < (n + 63) / 64 * 64; i += NT) c += __popcll(__ballot(i < n && cand[min(i, n - 1)] >= mid));
        return block_count<NW>(c, slots, step++);
      });
  }
  for (int j = tid; j < K; j += NT) sorted[j] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    const uint64_t k = cand[i];
    if (k < t) continue;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += cand[j] > k;
    if (rank < K) sorted[rank] = k;
  }
  __syncthreads();
}

struct TopOut {
  float* values;   // [R, K]
  int32_t* ids;    // [R, K]
  float* rest;     // [R]
  float* lse;      // [R]
  uint8_t* flags;  // [R]
  uint64_t* keys;  // [R, P, K]: a segment's best keys, 0: none
  Mass* parts;     // [R, P]: the mass of its other elements
};

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

// skip: rows (beams) that are not read at all.
struct TopSkip {
  const float* scores;     // NULL: none is skipped
  const uint8_t* finished; // or NULL
};

template <typename T, int NT, int L, int G, bool FINAL>
__global__ __launch_bounds__(NT) void top_segment_kernel(const T* __restrict__ logits, int64_t items, int32_t V,
                                                         int32_t K, int32_t P, float c, double c64, TopSkip skip,
                                                         TopOut o) {
  constexpr int NW = NT / 64;
  constexpr int EPL = Row<T>::EPL;
  constexpr int CAND = TopCaps<NT>::kCand, QUAL = TopCaps<NT>::kQual;
  __shared__ uint64_t cand[CAND];
  __shared__ uint64_t sorted[DSPARK_MAX_TOP];
  __shared__ uint32_t qual[QUAL];
  __shared__ int slots[2 * NW];
  __shared__ uint32_t shu[3][NW];
  __shared__ Mass shm[NW];
  __shared__ int ncand;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  int step = 0;

  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const size_t row = static_cast<size_t>(item / P);
    const int seg = static_cast<int>(item - static_cast<int64_t>(row) * P);
    if (skip.scores) {
      const float sc = skip.scores[row];
      if (!(sc > neg_inf() && sc < pos_inf()) || (skip.finished && skip.finished[row])) continue;
    }
    const Row<T> r = make_row(logits + row * V, V);
    const int first = seg * (NT * L * G);

    // ---- stream: every group's maximum and mass ----
    float gm[G], gs[G];
    {
      uint4 a[L], b[L];
      group_load<T, NT, L>(r, first, tid, a);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int q0 = first + g * NT * L;
        uint4(&cur)[L] = (g & 1) ? b : a;
        uint4(&nxt)[L] = (g & 1) ? a : b;
        if (g + 1 < G && q0 + NT * L < r.Q) group_load<T, NT, L>(r, q0 + NT * L, tid, nxt);
        if (q0 < r.Q) {
          const Mass m = group_mass<T, L>(cur, c);
          gm[g] = m.m;
          gs[g] = m.s;
        } else {
          gm[g] = neg_inf();
          gs[g] = 0.0f;
        }
      }
    }

    // ---- range of the group maxima, bad values ----
    uint32_t kmax = kKeyNegInf, bad = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      kmax = max(kmax, order_key(gm[g]));
      bad |= !(gs[g] >= 0.0f) ? 1u : 0u;
    }
    uint32_t wmax = kmax, wmin = kmax;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      wmax = max(wmax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(wmax), d, 64)));
      wmin = min(wmin, static_cast<uint32_t>(__shfl_xor(static_cast<int>(wmin), d, 64)));
    }
    bad = __any(bad) ? 1u : 0u;
    if constexpr (NW > 1) {
      if (lane == 0) {
        shu[0][wave] = wmax;
        shu[1][wave] = wmin;
        shu[2][wave] = bad;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        wmax = max(wmax, shu[0][w]);
        wmin = min(wmin, shu[1][w]);
        bad |= shu[2][w];
      }
    }
    if (tid == 0) ncand = 0;

    Mass others = mass_none();
    if (!bad && wmax > kKeyNegInf) {
      // ---- bound: at least K groups (or all finite ones) reach it ----
      auto groups_at = [&](uint32_t t) {
        int n = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) n += __popcll(__ballot(order_key(gm[g]) >= t));
        return block_count<NW>(n, slots, step++);
      };
      uint32_t bound = kKeyNegInf + 1;
      if (NT >= K && wmin > bound) bound = wmin;  // every thread's maximum reaches it
      int ngroups = groups_at(bound);
      if (ngroups > K) bound = bisect<uint32_t>(bound, wmax + 1, ngroups, K, K + K / 4 + 8, groups_at);

      // ---- the groups at the bound, in an order set by thread and group ----
      bool slow = ngroups > QUAL;
      if (!slow) {
        int nw = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) nw += __popcll(__ballot(order_key(gm[g]) >= bound));
        int base = 0;
        if constexpr (NW > 1) {
          if (lane == 0) shu[0][wave] = nw;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < NW; ++w) base += w < wave ? static_cast<int>(shu[0][w]) : 0;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const bool in = order_key(gm[g]) >= bound;
          const uint64_t mask = __ballot(in);
          if (in) {
            qual[base + __popcll(mask & ((1ull << lane) - 1))] = static_cast<uint32_t>(g * NT * L + tid);
          } else {
            others = mass_add(others, Mass{gm[g], gs[g]}, c);
          }
          base += __popcll(mask);
        }
        __syncthreads();
        // ---- candidates: the elements at or above the bound of those groups ----
        const float at = key_value(bound);
        for (int i = tid; i < ngroups * L; i += NT) {
          const int q = first + static_cast<int>(qual[i / L]) + (i % L) * NT;
          if (q >= r.Q) continue;
          const uint4 u = gran_load(r, q);
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            const float x = gran_elem(u, j, T{});
            if (x >= at) {
              const int pos = atomicAdd(&ncand, 1);
              if (pos < CAND) cand[pos] = cand_key(order_key(x), q * EPL - r.head + j);
            }
          }
        }
        __syncthreads();
        slow = ncand > CAND;
      }
      const int q1 = min(r.Q, first + NT * L * G);
      if (slow) {
        // ---- too many: the K-th key by bisection over the segment ----
        auto elems_at = [&](uint32_t t, int32_t last) {  // keys above t, and at t up to index `last`
          int n = 0;
          for (int q = first + tid; q < q1; q += NT) {
            const uint4 u = gran_load(r, q);
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
              const uint32_t k = order_key(gran_elem(u, j, T{}));
              n += k > t || (k == t && q * EPL - r.head + j <= last);
            }
          }
#pragma unroll
          for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d, 64);
          return block_count<NW>(n, slots, step++);
        };
        int n_lo = INT32_MAX;
        const uint32_t t = bisect<uint32_t>(kKeyNegInf + 1, wmax + 1, n_lo, K, K,
                                            [&](uint32_t mid) { return elems_at(mid, INT32_MAX); });
        // the lowest indices among the elements at t: the least `last` with K keys
        int32_t lo = -1, hi = V - 1;
        if (n_lo == K) lo = hi - 1;
        while (hi - lo > 1) {
          const int32_t mid = lo + (hi - lo) / 2;
          if (elems_at(t, mid) >= K) {
            hi = mid;
          } else {
            lo = mid;
          }
        }
        __syncthreads();
        if (tid == 0) ncand = 0;
        __syncthreads();
        for (int q = first + tid; q < q1; q += NT) {
          const uint4 u = gran_load(r, q);
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            const uint32_t k = order_key(gran_elem(u, j, T{}));
            const int32_t e = q * EPL - r.head + j;
            if (k > t || (k == t && e <= hi)) {
              const int pos = atomicAdd(&ncand, 1);
              if (pos < CAND) cand[pos] = cand_key(k, e);
            }
          }
        }
        __syncthreads();
        others = mass_none();
      }
      rank_top<NT>(cand, min(ncand, CAND), K, sorted, slots, step);

      // ---- mass of the elements read again that are not among the K ----
      const uint64_t kth = sorted[K - 1];  // 0: fewer than K, all of them are in
      auto add_others = [&](int q) {
        const uint4 u = gran_load(r, q);
        float x[EPL], m = neg_inf();
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          x[j] = gran_elem(u, j, T{});
          if (cand_key(order_key(x[j]), q * EPL - r.head + j) >= kth) x[j] = neg_inf();
          m = fmaxf(m, x[j]);
        }
        if (m == neg_inf()) return;
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) s += __builtin_amdgcn_exp2f(mass_gap(x[j], m, c));
        others = mass_add(others, Mass{m, s}, c);
      };
      if (slow) {
        for (int q = first + tid; q < q1; q += NT) add_others(q);
      } else {
        for (int i = tid; i < ngroups * L; i += NT) {
          const int q = first + static_cast<int>(qual[i / L]) + (i % L) * NT;
          if (q < r.Q) add_others(q);
        }
      }
    } else {
      for (int j = tid; j < K; j += NT) sorted[j] = 0;
    }

    // ---- the segment's mass, outputs ----
    others = wave_mass(others, c);
    if constexpr (NW > 1) {
      if (lane == 0) shm[wave] = others;
      __syncthreads();
      if (wave == 0) others = wave_mass(lane < NW ? shm[lane] : mass_none(), c);
    } else {
      __syncthreads();
    }
    if constexpr (FINAL) {
      if (wave == 0) write_row(o, row, sorted, K, others, bad != 0, c, c64);
    } else {
      const size_t part = row * P + seg;
      for (int j = tid; j < K; j += NT) o.keys[part * K + j] = sorted[j];
      if (tid == 0) o.parts[part] = bad ? Mass{neg_inf(), __builtin_nanf("")} : others;
    }
    __syncthreads();  // LDS is reused by the next item
  }
}

// The K best of the P segments' keys of a row, one workgroup a row.  FINAL:
// the row's outputs; otherwise the row's keys and mass at o.keys / o.parts
// with P = 1.
template <bool FINAL>
__global__ __launch_bounds__(kMergeThreads) void top_merge_kernel(const uint64_t* __restrict__ keys,
                                                                  const Mass* __restrict__ parts, int32_t R, int32_t K,
                                                                  int32_t P, float c, double c64, TopSkip skip,
                                                                  TopOut o) {
  constexpr int NT = kMergeThreads, NW = NT / 64;
  extern __shared__ uint64_t all[];  // P K keys
  __shared__ uint64_t sorted[DSPARK_MAX_TOP];
  __shared__ int slots[2 * NW];
  __shared__ Mass shm[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int n = P * K;
  int step = 0;
  for (int row = blockIdx.x; row < R; row += gridDim.x) {
    if (skip.scores) {
      const float sc = skip.scores[row];
      if (!(sc > neg_inf() && sc < pos_inf()) || (skip.finished && skip.finished[row])) continue;
    }
    const size_t at = static_cast<size_t>(row);
    for (int i = tid; i < n; i += NT) all[i] = keys[at * n + i];
    Mass others = mass_none();
    for (int p = tid; p < P; p += NT) others = mass_add(others, parts[at * P + p], c);
    __syncthreads();
    rank_top<NT>(all, n, K, sorted, slots, step);
    const uint64_t kth = sorted[K - 1];
    for (int i = tid; i < n; i += NT)
      if (all[i] != 0 && all[i] < kth) others = mass_add(others, Mass{key_value(all[i]), 1.0f}, c);
    others = wave_mass(others, c);
    if (lane == 0) shm[wave] = others;
    __syncthreads();
    if (wave == 0) {
      others = wave_mass(lane < NW ? shm[lane] : mass_none(), c);
      const bool bad = !(others.s >= 0.0f);
      if constexpr (FINAL) {
        write_row(o, at, sorted, K, others, bad, c, c64);
      } else {
        for (int j = lane; j < K; j += 64) o.keys[at * K + j] = sorted[j];
        if (lane == 0) o.parts[at] = others;
      }
    }
    __syncthreads();
  }
}

// Granules of a row at the least favourable alignment (any: the row may start
// inside a granule).
int row_granules(int epl, int32_t V, bool any) { return any ? (V + 2 * epl - 2) / epl : V / epl; }

// Rows of at most kWaveGran granules are taken by a wave each; others by
// workgroups of 512 threads, G groups of 4 granules a thread.
constexpr int kWaveL = 2, kWaveG = 8, kWaveGran = 64 * kWaveL * kWaveG;
constexpr int kBlockNT = 512, kBlockL = 4;
constexpr int kMaxSegments = 40;  // of a row: their K best keys fit top_merge's LDS

TopSplit top_split(int epl, int64_t R, int32_t V, bool any) {
  TopSplit s{};
  const int q = row_granules(epl, V, any);
  if (q <= kWaveGran) {
    s.G = 0;
    s.P = 1;
    return s;
  }
  const int tile = kBlockNT * kBlockL;
  int g = 8;
  while (g > 1 && (tile * (g / 2) >= q || R * ((q + tile * g - 1) / (tile * g)) < 512) &&
         (q + tile * (g / 2) - 1) / (tile * (g / 2)) <= kMaxSegments)
    g /= 2;
  s.G = g;
  s.P = (q + tile * g - 1) / (tile * g);
  return s;
}

template <typename T, bool FINAL>
hipError_t launch_segments(const T* logits, int32_t R, int32_t V, int32_t K, const TopSplit& sp, float c, double c64,
                           TopSkip skip, TopOut o, hipStream_t st) {
  const int64_t items = static_cast<int64_t>(R) * sp.P;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(items, kMaxGrid)));
#define DSPARK_TOP(NT, L, G)                                                                                     \
  DSPARK_LAUNCH("top_segment", (top_segment_kernel<T, NT, L, G, FINAL>), grid, dim3(NT), 0, st, logits, items, V, \
                K, sp.P, c, c64, skip, o)
  switch (sp.G) {
    case 0:
      DSPARK_TOP(64, kWaveL, kWaveG);
      break;
    case 1:
      DSPARK_TOP(kBlockNT, kBlockL, 1);
      break;
    case 2:
      DSPARK_TOP(kBlockNT, kBlockL, 2);
      break;
    case 4:
      DSPARK_TOP(kBlockNT, kBlockL, 4);
      break;
    default:
      DSPARK_TOP(kBlockNT, kBlockL, 8);
      break;
  }
#undef DSPARK_TOP
  return hipGetLastError();
}

template <bool FINAL>
hipError_t launch_merge(const uint64_t* keys, const Mass* parts, int32_t R, int32_t K, int32_t P, float c, double c64,
                        TopSkip skip, TopOut o, hipStream_t st) {
  DSPARK_LAUNCH("top_merge", (top_merge_kernel<FINAL>), dim3(static_cast<unsigned>(std::min(R, kMaxGrid))),
                dim3(kMergeThreads), static_cast<size_t>(P) * K * sizeof(uint64_t), st, keys, parts, R, K, P, c, c64,
                skip, o);
  return hipGetLastError();
}

bool any_alignment(const void* p, int32_t V, int epl) {
  return V % epl != 0 || (reinterpret_cast<uintptr_t>(p) & 15u) != 0;
}

}  // namespace

float mass_scale(float temperature) { return static_cast<float>(1.4426950408889634074 / static_cast<double>(temperature)); }
double mass_scale64(float temperature) { return 1.4426950408889634074 / static_cast<double>(temperature); }

// Sized for either type and any alignment of the rows.
TopPlan plan_top(int32_t R, int32_t V, int32_t K) {
  TopPlan p{};
  int P = 1;
  for (const int epl : {4, 8})
    for (const bool any : {false, true})
      if (any || V % epl == 0) P = std::max(P, top_split(epl, R, V, any).P);
  p.P = P;
  const size_t rp = static_cast<size_t>(R) * P;
  size_t off = 0;
  if (P > 1) {
    off = align_up(off + rp * K * sizeof(uint64_t), 256);
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
  const TopSplit sp = top_split(epl, R, V, any_alignment(logits, V, epl));
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
int top_lists_segments(int dtype, int32_t R, int32_t V, const void* logits) {
  const int epl = dtype == DSPARK_BF16 ? 8 : 4;
  return top_split(epl, R, V, any_alignment(logits, V, epl)).P;
}

hipError_t launch_top_lists(const void* logits, int dtype, int32_t R, int32_t V, int32_t K, const float* scores,
                            const uint8_t* finished, uint64_t* keys, Mass* parts, hipStream_t st) {
  const int epl = dtype == DSPARK_BF16 ? 8 : 4;
  const TopSplit sp = top_split(epl, R, V, any_alignment(logits, V, epl));
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
