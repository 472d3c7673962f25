// beam.hip — one step of a beam search: the selection over a request's beams
// and vocabulary, and the reordering of the beams' states.
//
// Semantics (include/dspark.h, dspark_beam_select, dspark_beam_reorder): the M
// best of score_w + x_v - lse_w over a request's live beams w and tokens v.
//
// Selection: a beam's M best tokens hold all that the request can take from
// it, so the rows go through the pass of top.hip (one read of each live beam's
// row; ended and dead beams are not read), which leaves per beam its M best
// candidates in order with their scores in 64 bits: candidates of two beams can
// stand closer than 32 bits tell apart.  beam_final, one workgroup a request,
// ranks them: a candidate's rank is the number of better ones; of many, a search
// over the scores' order keys keeps M or a few more first.  Equal scores go by
// beam, logit and token, so the order is total and does not depend on timing.
//
// Reordering: a copy.  A thread moves the same 16 bytes of every beam of a
// request, all loads before all stores, so a parent with several children is
// read once and the copy may be done in place.
#include <algorithm>

#include "common.hpp"
#include "rowstream.hpp"
#include "vocab.hpp"

namespace dspark {
namespace {

constexpr int kFinalThreads = 256;
constexpr int kFinalWaves = kFinalThreads / 64;
constexpr int kMaxCand = DSPARK_MAX_BEAMS * DSPARK_MAX_TOP;
constexpr int kRankAll = 64;  // candidates ranked at once; more are first cut by a search (128: 7 us against 4.6)
constexpr int kMaxGrid = 1 << 22;  // workgroups of a launch; more are further launches

// W M candidates a request: a chain of a few barriers, 3.4 us for 32 candidates, 4.6
// for 256, of which 3 are any launch's.
__global__ __launch_bounds__(kFinalThreads) void beam_final_kernel(const uint64_t* __restrict__ sums,
                                                                   const uint64_t* __restrict__ keys, int32_t base,
                                                                   int32_t W, int32_t M,
                                                                   int32_t* __restrict__ tokens,
                                                                   int32_t* __restrict__ parents,
                                                                   float* __restrict__ scores) {
  constexpr int NT = kFinalThreads, NW = kFinalWaves;
  __shared__ uint64_t sh_sum[kMaxCand + 4];
  __shared__ uint64_t sh_best[kMaxCand + 4];
  __shared__ uint16_t sh_from[kMaxCand];
  __shared__ uint64_t slots[2 * NW];
  __shared__ int scan[2][NW];
  __shared__ uint64_t red[2][NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int n = W * M;
  const int each = (n + NT - 1) / NT;  // a thread's stretch, so that positions keep their order
  int step = 0;
  const int b = base + static_cast<int>(blockIdx.x);
  const uint64_t* key = keys + static_cast<size_t>(b) * n;
  // ---- the candidates that there are, in order ----
  uint64_t top = 0, low = ~0ull;
  int mine = 0, found;
  for (int i = tid; i < n; i += NT) {
    const uint64_t d = sums[static_cast<size_t>(b) * n + i];
    sh_sum[i] = d;
    if (d > kKey64NegInf) {
      ++mine;
      top = max(top, d);
      low = min(low, d);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    top = max(top, static_cast<uint64_t>(__shfl_xor(static_cast<long long>(top), d, 64)));
    low = min(low, static_cast<uint64_t>(__shfl_xor(static_cast<long long>(low), d, 64)));
  }
  if (lane == 0) {
    red[0][wave] = top;
    red[1][wave] = low;
  }
  block_scan<NW>(mine, scan[0], found);  // its barrier completes sh_sum and red
  uint64_t bound = kKey64NegInf + 1;
  if (found > kRankAll) {
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      top = max(top, red[0][w]);
      low = min(low, red[1][w]);
    }
    int n_lo = found;
    bound = search_key<uint64_t>(low, top + 1, n_lo, M, M + M / 4 + 8, [&](uint64_t t1, uint64_t t2, uint64_t t3) {
      Count3 k{0, 0, 0};
      for (int i = tid; i < (n + 63) / 64 * 64; i += NT) {
        const uint64_t d = i < n ? sh_sum[i] : 0;
        k.a += __popcll(__ballot(d >= t1));
        k.b += __popcll(__ballot(d >= t2));
        k.c += __popcll(__ballot(d >= t3));
      }
      return block_count<NW>(k, slots, step);
    });
  }
  // ---- those that can be among the M ----
  int nb;
  mine = 0;
  const int i0 = tid * each, i1 = min(n, i0 + each);
  for (int i = i0; i < i1; ++i) mine += sh_sum[i] >= bound;
  int pos = block_scan<NW>(mine, scan[1], nb);
  for (int i = i0; i < i1; ++i)
    if (sh_sum[i] >= bound) {
      sh_best[pos] = sh_sum[i];
      sh_from[pos++] = static_cast<uint16_t>(i);
    }
  if (tid < 4) sh_best[nb + tid] = 0;
  __syncthreads();
  // ---- rank: score, then position, which is beam, logit, token ----
  for (int i = tid; i < nb; i += NT) {
    const uint64_t d = sh_best[i];
    int rank = 0;
    for (int j = 0; j < nb; j += 4) {
      const uint64_t d0 = sh_best[j], d1 = sh_best[j + 1], d2 = sh_best[j + 2], d3 = sh_best[j + 3];
      rank += d0 > d - (j < i) ? 1 : 0;
      rank += d1 > d - (j + 1 < i) ? 1 : 0;
      rank += d2 > d - (j + 2 < i) ? 1 : 0;
      rank += d3 > d - (j + 3 < i) ? 1 : 0;
    }
    if (rank < M) {
      const int from = sh_from[i];
      const uint64_t k = key[from];
      const size_t o = static_cast<size_t>(b) * M + rank;
      tokens[o] = key_index(k);
      parents[o] = from / M;
      scores[o] = static_cast<float>(key_double(d));
    }
  }
  for (int j = found + tid; j < M; j += NT) {  // fewer candidates than picks
    const size_t o = static_cast<size_t>(b) * M + j;
    tokens[o] = -1;
    parents[o] = -1;
    scores[o] = neg_inf();
  }
}

// ---- reordering -------------------------------------------------------------------
// A row of a beam is S runs of T tokens; only the tokens before the request's
// length move, in units of 16 bytes at any address.  A run's last unit ends with
// it; in place, and in runs of less than a unit, its last bytes move as 8, 4, 2 and
// 1.  One workgroup moves a stretch of units of one run of every beam of a request:
// MB children at a time, all of them loaded before any is stored (in place: MB >=
// M).  Bound by HBM: 1.6 GB of caches 505 us, 5.7 TB/s, a parent with several
// children read once.  Units that fit token and address took 58 us for 50 MB of
// 1023 tokens of 6 bytes a run where these take 18, and 147 for 201 MB of tokens of
// 12 against 53; aligned runs are no slower.  The stores of 16 bytes are
// non-temporal (563 us without; non-temporal loads, 606: a parent's children read
// it again).
constexpr int kMoveThreads = 256;
constexpr int64_t kUnit = 16;
constexpr int32_t kNotInPlace = 1 << 30;  // above every parent

// Units at any address: vector memory instructions take unaligned ones.
struct Unit16 {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(1)));
};
struct Unit8 {
  typedef uint64_t type __attribute__((aligned(1)));
};
struct Unit4 {
  typedef uint32_t type __attribute__((aligned(1)));
};
struct Unit2 {
  typedef uint16_t type __attribute__((aligned(1)));
};
struct Unit1 {
  typedef uint8_t type;
};

// One unit of the children j0 + [0, MB) of the parents p (-1: none; beam 0 is read
// in its place, so that no branch parts the loads).
template <typename U, int MB>
__device__ __forceinline__ void move_unit(const char* from, char* to, int64_t row, int j0, const int (&p)[MB]) {
  typename U::type v[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) v[j] = *reinterpret_cast<const typename U::type*>(from + max(p[j], 0) * row);
#pragma unroll
  for (int j = 0; j < MB; ++j)
    if (p[j] >= 0) {
      typename U::type* a = reinterpret_cast<typename U::type*>(to + (j0 + j) * row);
      if constexpr (sizeof(*a) == 16)
        __builtin_nontemporal_store(v[j], a);
      else
        *a = v[j];
    }
}

template <int MB>
__global__ __launch_bounds__(kMoveThreads) void beam_reorder_kernel(const char* src, char* dst,
                                                                    const int32_t* __restrict__ parents,
                                                                    const int32_t* __restrict__ lengths, int64_t base,
                                                                    int64_t chunks, int32_t B, int32_t W, int32_t M,
                                                                    int32_t S, int32_t T, int64_t token,
                                                                    int32_t own) {
  const int64_t item = base + blockIdx.x;
  const int64_t run = item / chunks, chunk = item - run * chunks;
  const int64_t lb = run / S;
  const int s = static_cast<int>(run - lb * S);
  const int b = static_cast<int>(lb % B);
  int64_t t = T;
  if (lengths) t = min(max(lengths[b], 0), T);
  int64_t at = (chunk * blockDim.x + threadIdx.x) * kUnit, left = t * token - at;
  if (left <= 0) return;
  if (left < kUnit && at > 0 && own == kNotInPlace) {
    at -= kUnit - left;  // part of it is moved twice, from a source that does not change
    left = kUnit;
  }
  const int64_t seg = static_cast<int64_t>(T) * token, row = seg * S;
  const char* from = src + lb * W * row + s * seg + at;
  char* to = dst + lb * M * row + s * seg + at;
#pragma unroll 1
  for (int j0 = 0; j0 < M; j0 += MB) {
    int p[MB], some = -1;
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      p[j] = -1;
      if (j0 + j < M) p[j] = parents[static_cast<int64_t>(b) * M + j0 + j];
      p[j] = __builtin_amdgcn_readfirstlane(p[j]);  // the same for the workgroup: scalar addresses and branches
      if (p[j] >= W || p[j] == own + j0 + j) p[j] = -1;
      some = max(some, p[j]);
    }
    if (some < 0) continue;
    if (left >= kUnit) {
      move_unit<Unit16, MB>(from, to, row, j0, p);
    } else {
      const int l4 = static_cast<int>(left) & 8, l2 = static_cast<int>(left) & 12, l1 = static_cast<int>(left) & 14;
      if (left & 8) move_unit<Unit8, MB>(from, to, row, j0, p);
      if (left & 4) move_unit<Unit4, MB>(from + l4, to + l4, row, j0, p);
      if (left & 2) move_unit<Unit2, MB>(from + l2, to + l2, row, j0, p);
      if (left & 1) move_unit<Unit1, MB>(from + l1, to + l1, row, j0, p);
    }
  }
}

}  // namespace

BeamPlan plan_beam(int32_t B, int32_t W, int32_t V, int32_t M) {
  BeamPlan p{};
  const int32_t R = B * W;
  p.rows = plan_top(R, V, M);
  const size_t list = static_cast<size_t>(R) * M * sizeof(uint64_t);
  size_t off = 0;
  p.off_sums = off;
  off = align_up(off + list, 256);
  p.off_keys = off;
  off = align_up(off + list, 256);
  p.off_rows = off;
  p.bytes = align_up(off + p.rows.bytes, 256);
  return p;
}

hipError_t launch_beam_select(const void* logits, int dtype, const float* scores, const uint8_t* finished, int32_t eos,
                              int32_t B, int32_t W, int32_t V, int32_t M, int32_t* tokens, int32_t* parents,
                              float* out_scores, uint8_t* flags, void* ws, const BeamPlan& pl, hipStream_t st) {
  char* w = static_cast<char*>(ws);
  uint64_t* sums = reinterpret_cast<uint64_t*>(w + pl.off_sums);
  uint64_t* keys = reinterpret_cast<uint64_t*>(w + pl.off_keys);
  const hipError_t e = launch_beam_rows(logits, dtype, B * W, V, M, scores, finished, eos, sums, keys, flags,
                                        w + pl.off_rows, pl.rows, st);
  if (e != hipSuccess) return e;
  for (int32_t base = 0, n; base < B; base += n) {
    n = std::min(B - base, kMaxGrid);
    DSPARK_LAUNCH("beam_final", beam_final_kernel, dim3(static_cast<unsigned>(n)), dim3(kFinalThreads), 0, st, sums,
                  keys, base, W, M, tokens, parents, out_scores);
  }
  return hipGetLastError();
}

hipError_t launch_beam_reorder(const void* src, void* dst, const int32_t* parents, const int32_t* lengths, int64_t L,
                               int32_t B, int32_t W, int32_t M, int32_t S, int32_t T, int64_t token, hipStream_t st) {
  const int64_t units = (T * token + kUnit - 1) / kUnit;
  const int threads = units <= 64 ? 64 : kMoveThreads;  // of a run
  const int64_t chunks = (units + threads - 1) / threads;
  const int64_t items = L * B * S * chunks;
  const bool in_place = src == dst;
  const char* s = static_cast<const char*>(src);
  char* d = static_cast<char*>(dst);
#define DSPARK_MOVE(MB)                                                                                        \
  DSPARK_LAUNCH("beam_reorder", (beam_reorder_kernel<MB>), grid, dim3(threads), 0, st, s, d, parents, \
                lengths, base, chunks, B, W, M, S, T, token, in_place ? 0 : kNotInPlace)
  for (int64_t base = 0; base < items; base += kMaxGrid) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(items - base, kMaxGrid)));
    if (M <= 4)
      DSPARK_MOVE(4);
    else if (M <= 8 || !in_place)
      DSPARK_MOVE(8);
    else if (M <= 16)
      DSPARK_MOVE(16);
    else
      DSPARK_MOVE(32);
  }
#undef DSPARK_MOVE
  return hipGetLastError();
}

}  // namespace dspark
