// beam.hip — one step of a beam search: the selection over a request's beams
// and vocabulary, and the reordering of the beams' states.
//
// Semantics (include/dspark.h, dspark_beam_select, dspark_beam_reorder): the M
// best of score_w + x_v - lse_w over a request's live beams w and tokens v.
//
// Selection: a beam's M best tokens hold all that the request can take from
// it, so the rows go through the pass of top.hip (each live beam's M highest
// logits and the mass of the others, one read of the row); ended and dead
// beams are not read.  beam_final, one workgroup a request, forms each beam's
// normaliser in 64 bits (the listed tokens one by one, the others as their
// 32-bit mass) and every candidate's score in 64 bits: candidates of two beams
// can stand closer than 32 bits tell apart.  Few candidates are ranked by
// counting at once; of many, a bisection over the scores' order keys keeps M
// or a few more first.  Equal scores go by beam, logit and token, so the
// order is total and does not depend on timing.
//
// Reordering: a copy.  A thread moves the same 16 bytes of every beam of a
// request, all loads before all stores, so a parent with several children is
// read once and the copy may be done in place.
#include <algorithm>

#include "common.hpp"
#include "internal.hpp"
#include "rowstream.hpp"

namespace dspark {
namespace {

constexpr int kFinalThreads = 256;
constexpr int kFinalWaves = kFinalThreads / 64;
constexpr int kMaxCand = 5632;  // candidates of a request: DSPARK_MAX_BEAMS lists of the longest length fit
constexpr int kMaxGrid = 1 << 20;
constexpr double kLn2d = 0.69314718055994530942;
constexpr double kLog2ed = 1.4426950408889634074;

__device__ __forceinline__ uint64_t order_key64(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
}
constexpr uint64_t kKey64NegInf = 0x000FFFFFFFFFFFFFull;

struct BeamArgs {
  const float* scores;
  const uint8_t* finished;  // or NULL
  int32_t eos, B, W, M, E;  // E: list entries per beam
  int32_t P;                // masses per beam
  int32_t* tokens;
  int32_t* parents;
  float* out_scores;
  uint8_t* flags;
};

__global__ __launch_bounds__(kFinalThreads) void beam_final_kernel(const uint64_t* __restrict__ keys,
                                                                   const Mass* __restrict__ parts, float c, double c64,
                                                                   BeamArgs a) {
  constexpr int NT = kFinalThreads, NW = kFinalWaves;
  __shared__ double sh_score[kMaxCand];
  __shared__ uint16_t sh_list[kMaxCand];
  __shared__ double sh_lse[DSPARK_MAX_BEAMS];
  __shared__ uint8_t sh_state[DSPARK_MAX_BEAMS];  // 0: none, 1: live, 2: ended
  __shared__ int slots[6 * NW];
  __shared__ int nlist;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int n = a.W * a.E;
  int step = 0;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    // ---- the beams' normalisers ----
    for (int w = wave; w < a.W; w += NW) {
      const size_t row = static_cast<size_t>(b) * a.W + w;
      const float sc = a.scores[row];
      const bool ended = a.finished && a.finished[row] != 0;
      uint8_t state = 0, flag = 0;
      double lse = 0.0;
      if (isnan(sc) || sc == pos_inf()) {
        flag = DSPARK_FLAG_NONFINITE;
      } else if (sc > neg_inf()) {
        if (ended) {
          state = 2;
        } else {
          Mass m = mass_none();
          for (int p = lane; p < a.P; p += 64) m = mass_add(m, parts[row * a.P + p], c);
          m = wave_mass(m, c);
          if (!(m.s >= 0.0f)) {
            flag = DSPARK_FLAG_NONFINITE;
          } else {
            const double others = mass_log2(m, c, c64);
            float top = neg_inf();
            for (int i = lane; i < a.E; i += 64) {
              const uint64_t k = keys[row * a.E + i];
              if (k) top = fmaxf(top, key_value(k));
            }
            top = wave_max(top);
            if (top == neg_inf()) {
              flag = DSPARK_FLAG_EMPTY_ROW;
            } else {
              const double ref = static_cast<double>(top);
              double s = 0.0;
              for (int i = lane; i < a.E; i += 64) {
                const uint64_t k = keys[row * a.E + i];
                if (k) s += exp2((static_cast<double>(key_value(k)) - ref) * kLog2ed);
              }
              s = wave_sum64(s) + exp2(others - ref * kLog2ed);
              lse = ref + log2(s) * kLn2d;
              state = 1;
            }
          }
        }
      }
      if (lane == 0) {
        sh_lse[w] = lse;
        sh_state[w] = state;
        a.flags[row] = flag;
      }
    }
    if (tid == 0) nlist = 0;
    __syncthreads();
    // ---- the candidates' scores ----
    int found = 0;
    for (int i = tid; i < (n + 63) / 64 * 64; i += NT) {
      double d = -__builtin_inf();
      if (i < n) {
        const int w = i / a.E, e = i - w * a.E;
        const size_t row = static_cast<size_t>(b) * a.W + w;
        const uint8_t state = sh_state[w];
        if (state == 1) {
          const uint64_t k = keys[row * a.E + e];
          if (k) d = static_cast<double>(a.scores[row]) + (static_cast<double>(key_value(k)) - sh_lse[w]);
        } else if (state == 2 && e == 0) {
          d = static_cast<double>(a.scores[row]);
        }
        sh_score[i] = d;
      }
      found += __popcll(__ballot(d > -__builtin_inf()));
    }
    found = block_count<NW>(Count3{found, 0, 0}, slots, step).a;  // its barrier completes sh_score
    // ---- those that can be among the M ----
    uint64_t bound = kKey64NegInf + 1;
    const int most = a.M + a.M / 4 + 8;
    if (found > std::max(most, 64)) {
      int n_lo = found;
      bound = search_key<uint64_t>(bound, order_key64(__builtin_inf()) + 1, n_lo, a.M, most,
                                   [&](uint64_t t1, uint64_t t2, uint64_t t3) {
        Count3 k{0, 0, 0};
        for (int i = tid; i < (n + 63) / 64 * 64; i += NT) {
          const uint64_t d = i < n ? order_key64(sh_score[i]) : 0;
          k.a += __popcll(__ballot(d >= t1));
          k.b += __popcll(__ballot(d >= t2));
          k.c += __popcll(__ballot(d >= t3));
        }
        return block_count<NW>(k, slots, step);
      });
    }
    for (int i = tid; i < n; i += NT)
      if (order_key64(sh_score[i]) >= bound) sh_list[atomicAdd(&nlist, 1)] = static_cast<uint16_t>(i);
    __syncthreads();
    // ---- rank: score, then beam, logit, token ----
    const int nl = nlist;
    const size_t base = static_cast<size_t>(b) * a.W;
    for (int i = tid; i < nl; i += NT) {
      const int ci = sh_list[i], w = ci / a.E;
      const double d = sh_score[ci];
      const uint64_t k = sh_state[w] == 1 ? keys[base * a.E + ci] : 0;
      int rank = 0;
      for (int j = 0; j < nl; ++j) {
        const int cj = sh_list[j];
        const double dj = sh_score[cj];
        if (dj > d) {
          ++rank;
        } else if (dj == d && cj != ci) {
          const int wj = cj / a.E;
          if (wj < w || (wj == w && keys[base * a.E + cj] > k)) ++rank;
        }
      }
      if (rank < a.M) {
        const size_t o = static_cast<size_t>(b) * a.M + rank;
        a.tokens[o] = k ? key_index(k) : a.eos;
        a.parents[o] = w;
        a.out_scores[o] = static_cast<float>(d);
      }
    }
    for (int j = found + tid; j < a.M; j += NT) {  // fewer candidates than picks
      const size_t o = static_cast<size_t>(b) * a.M + j;
      a.tokens[o] = -1;
      a.parents[o] = -1;
      a.out_scores[o] = neg_inf();
    }
    __syncthreads();  // LDS is reused by the next request
  }
}

// ---- reordering -------------------------------------------------------------------
// Unit: the widest of 16, 4, 2 and 1 bytes that divides every extent and
// address.  A row of a beam is S runs of T tokens of U units; only the tokens
// before the request's length move.  One workgroup moves a stretch of units of
// one run of every beam of a request: MB children at a time, all of them
// loaded before any is stored (in place: MB >= M).
constexpr int kMoveThreads = 256;

template <typename U, int MB>
__global__ __launch_bounds__(kMoveThreads) void beam_reorder_kernel(const U* src, U* dst,
                                                                    const int32_t* __restrict__ parents,
                                                                    const int32_t* __restrict__ lengths, int64_t items,
                                                                    int64_t chunks, int32_t B, int32_t W, int32_t M,
                                                                    int32_t S, int32_t T, int64_t unit, bool in_place) {
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t run = item / chunks;
    const int64_t chunk = item - run * chunks;
    const int s = static_cast<int>(run % S);
    const int64_t lb = run / S;
    const int b = static_cast<int>(lb % B);
    int64_t t = T;
    if (lengths) t = min(max(lengths[b], 0), T);
    const int64_t used = t * unit;
    const int64_t at = chunk * kMoveThreads + threadIdx.x;
    const int64_t seg = static_cast<int64_t>(T) * unit, row = seg * S;
    if (at >= used) continue;
    const U* from = src + lb * W * row + s * seg + at;
    U* to = dst + lb * M * row + s * seg + at;
    for (int j0 = 0; j0 < M; j0 += MB) {
      U v[MB];
      int p[MB];
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        p[j] = -1;
        if (j0 + j < M) p[j] = parents[static_cast<int64_t>(b) * M + j0 + j];
        if (p[j] >= W || (in_place && p[j] == j0 + j)) p[j] = -1;
        if (p[j] >= 0) v[j] = from[p[j] * row];
      }
#pragma unroll
      for (int j = 0; j < MB; ++j)
        if (p[j] >= 0) to[(j0 + j) * row] = v[j];
    }
  }
}

template <typename U>
hipError_t move(const void* src, void* dst, const int32_t* parents, const int32_t* lengths, int64_t L, int32_t B,
                int32_t W, int32_t M, int32_t S, int32_t T, int64_t bytes, hipStream_t st) {
  const int64_t unit = bytes / static_cast<int64_t>(sizeof(U));
  const int64_t chunks = (T * unit + kMoveThreads - 1) / kMoveThreads;
  const int64_t items = L * B * S * chunks;
  const bool in_place = src == dst;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(items, kMaxGrid)));
  const U* s = static_cast<const U*>(src);
  U* d = static_cast<U*>(dst);
#define DSPARK_MOVE(MB)                                                                                            \
  DSPARK_LAUNCH("beam_reorder", (beam_reorder_kernel<U, MB>), grid, dim3(kMoveThreads), 0, st, s, d, parents, \
                lengths, items, chunks, B, W, M, S, T, unit, in_place)
  if (M <= 4)
    DSPARK_MOVE(4);
  else if (M <= 8 || !in_place)
    DSPARK_MOVE(8);
  else if (M <= 16)
    DSPARK_MOVE(16);
  else
    DSPARK_MOVE(32);
#undef DSPARK_MOVE
  return hipGetLastError();
}

}  // namespace

// Keys and masses of the beams' segments; where a request's lists would not
// fit beam_final, the beams' merged ones too.
BeamPlan plan_beam(int32_t B, int32_t W, int32_t V, int32_t M) {
  BeamPlan p{};
  const int32_t R = B * W;
  const TopPlan t = plan_top(R, V, M);
  p.P = t.P;
  const size_t rp = static_cast<size_t>(R) * t.P;
  size_t off = 0;
  p.off_keys = off;
  off = align_up(off + rp * top_list_len(M) * sizeof(uint64_t), 256);
  p.off_parts = off;
  off = align_up(off + rp * sizeof(Mass), 256);
  if (static_cast<int64_t>(W) * top_list_len(M) * t.P > kMaxCand) {
    p.off_mkeys = off;
    off = align_up(off + static_cast<size_t>(R) * top_list_len(M) * sizeof(uint64_t), 256);
    p.off_mparts = off;
    off = align_up(off + static_cast<size_t>(R) * sizeof(Mass), 256);
  }
  p.bytes = off;
  return p;
}

hipError_t launch_beam_select(const void* logits, int dtype, const float* scores, const uint8_t* finished, int32_t eos,
                              int32_t B, int32_t W, int32_t V, int32_t M, int32_t* tokens, int32_t* parents,
                              float* out_scores, uint8_t* flags, void* ws, const BeamPlan& pl, hipStream_t st) {
  const int32_t R = B * W;
  char* w = static_cast<char*>(ws);
  uint64_t* keys = reinterpret_cast<uint64_t*>(w + pl.off_keys);
  Mass* parts = reinterpret_cast<Mass*>(w + pl.off_parts);
  int P = top_lists_segments(dtype, R, V, M, logits);
  hipError_t e = launch_top_lists(logits, dtype, R, V, M, scores, finished, keys, parts, st);
  if (e != hipSuccess) return e;
  if (static_cast<int64_t>(W) * top_list_len(M) * P > kMaxCand) {
    uint64_t* mkeys = reinterpret_cast<uint64_t*>(w + pl.off_mkeys);
    Mass* mparts = reinterpret_cast<Mass*>(w + pl.off_mparts);
    e = launch_top_lists_merge(keys, parts, R, M, P, scores, finished, mkeys, mparts, st);
    if (e != hipSuccess) return e;
    keys = mkeys;
    parts = mparts;
    P = 1;
  }
  const BeamArgs a{scores, finished, eos, B, W, M, P * top_list_len(M), P, tokens, parents, out_scores, flags};
  DSPARK_LAUNCH("beam_final", beam_final_kernel, dim3(static_cast<unsigned>(std::min(B, kMaxGrid))),
                dim3(kFinalThreads), 0, st, keys, parts, mass_scale(1.0f), mass_scale64(1.0f), a);
  return hipGetLastError();
}

hipError_t launch_beam_reorder(const void* src, void* dst, const int32_t* parents, const int32_t* lengths, int64_t L,
                               int32_t B, int32_t W, int32_t M, int32_t S, int32_t T, int64_t bytes, hipStream_t st) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) | static_cast<uintptr_t>(bytes);
  if (all % 16 == 0) return move<u32x4>(src, dst, parents, lengths, L, B, W, M, S, T, bytes, st);
  if (all % 4 == 0) return move<uint32_t>(src, dst, parents, lengths, L, B, W, M, S, T, bytes, st);
  if (all % 2 == 0) return move<uint16_t>(src, dst, parents, lengths, L, B, W, M, S, T, bytes, st);
  return move<uint8_t>(src, dst, parents, lengths, L, B, W, M, S, T, bytes, st);
}

}  // namespace dspark
