// distill.hip — distillation from a teacher's highest logits: loss and gradient.
//
// Semantics (include/dspark.h, dspark_distill): the outcomes are the K tokens
// that the teacher lists and, where its remaining mass is given, everything
// else as one more; kl = sum_j t_j (log t_j - log s_j) over them, with t the
// teacher's and s the draft's probabilities at temperature T.
//
// Loss: a workgroup streams a draft row once and sums the mass of the tokens
// outside the teacher's list, and of nothing else: the list becomes a bit mask in
// LDS, one word per thread and group of 4 granules, so a group without a listed
// token (nearly all) costs one LDS read and a branch.  Its first wave then forms
// the K + 1 outcomes in 64 bits from that mass, the teacher's values and the
// draft's logits at its tokens: where one probability is nearly 1, its logarithm
// and its difference from the other side keep their accuracy, as no 32-bit
// normaliser of the whole row enters.  That costs one wave a few hundred 64-bit
// operations while the compute unit's other workgroups stream.  A second, small
// launch adds up the sums; a batch of a few short rows is one launch of one
// workgroup, a wave a row.
//
// Gradient, one launch: with d_v the derivative of kl by x_v / T,
//   v in the list:  d_v = s_v - sum_{j: id_j = v} t_j
//   otherwise:      d_v = (s_r - t_r) exp(x_v / T) / sum_{u outside} exp(x_u / T)
// so a row is one factor and one exponential per element, and K values that
// are written over it at the end.
#include <algorithm>

#include "common.hpp"
#include "rowstream.hpp"
#include "vocab.hpp"

namespace dspark {
namespace {

constexpr int kMaxGrid = 1 << 22;  // workgroups of a launch; more are further launches
constexpr int kL = 4;              // granules of a group
constexpr int kMaxTiles = 16;      // groups of a thread whose mask words are held at a time
constexpr int kTinyThreads = 1024; // one-launch form: a wave a row
constexpr int kTinyWaves = kTinyThreads / 64;
constexpr int kTinyTiles = 2;
constexpr int kSumThreads = 1024;
constexpr int kMaxSumBlocks = 64;
constexpr double kLn2d = 0.69314718055994530942;
constexpr double kLog2ed = 1.4426950408889634074;

struct DistillArgs {
  const float* values;
  const int32_t* ids;
  const float* teacher_rest;  // or NULL
  const uint8_t* block_mask;  // or NULL
  int32_t N, gamma, V, K;
  float c;
  double c64;
  float weight;
};

// Barrier of the NT threads that share a row (one wave needs its LDS traffic
// ordered, no barrier).
template <int NT>
__device__ __forceinline__ void row_sync() {
  if constexpr (NT == 64) {
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }
}

// L granules with -inf at the elements whose bit is set.
template <typename T, int L>
__device__ __forceinline__ void mask_out(uint4 (&u)[L], uint32_t word) {
  constexpr int EPL = Row<T>::EPL;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if ((word >> (i * EPL + j)) & 1u) {
        if constexpr (sizeof(T) == 2)
          w[j / 2] = (j & 1) ? (w[j / 2] & 0x0000ffffu) | 0xFF800000u : (w[j / 2] & 0xffff0000u) | 0xFF80u;
        else
          w[j] = 0xFF800000u;
      }
    }
    u[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---- the K + 1 outcomes of a row, by one wave --------------------------------------
// Lane l holds entries l, l + 64, ..  ENT: entries of a lane (K <= 64 ENT).
template <int ENT>
struct Entries {
  int32_t id[ENT];  // its token, -1: none
  float v[ENT];     // the teacher's logit
  float x[ENT];     // the draft's
  float trest;      // the teacher's other mass
};

template <typename T, int ENT>
__device__ __forceinline__ Entries<ENT> load_entries(const Row<T>& r, const DistillArgs& a, size_t row) {
  const int lane = threadIdx.x & 63;
  Entries<ENT> e;
  e.trest = a.teacher_rest ? a.teacher_rest[row] : neg_inf();
#pragma unroll
  for (int i = 0; i < ENT; ++i) {
    const int j = i * 64 + lane;
    e.id[i] = -1;
    e.v[i] = e.x[i] = neg_inf();
    if (j < a.K) {
      const int32_t id = a.ids[row * a.K + j];
      const float v = a.values[row * a.K + j];
      if (id >= 0 && id < r.V) {
        e.id[i] = id;
        e.v[i] = v;
        e.x[i] = load_logit(r.p, static_cast<size_t>(id));
      }
    }
  }
  return e;
}

// In 64 bits, logarithms to base 2.  The teacher's weights are et / st, relative to
// 2^rt, the draft's es / ss, relative to 2^rs.
template <int ENT>
struct Outcomes {
  double zt[ENT], zs[ENT];  // logits (-inf: no such entry)
  double et[ENT], es[ENT];
  double zr;                // the teacher's logit of everything else
  double et_r, es_r;
  double rt, rs, st, ss;
  uint32_t first;  // bit i: no earlier entry of the row has entry i's token
  bool twice;      // some token is listed more than once
  bool bad;        // a NaN or +inf
  bool empty;      // no mass on one side
};

template <int ENT>
__device__ __forceinline__ Outcomes<ENT> outcomes(const Entries<ENT>& e, int K, double rest2, double c64,
                                                  int32_t* sh_ids) {
#pragma clang fp contract(off)  // a value less itself as the reference is 0
  const int lane = threadIdx.x & 63;
  Outcomes<ENT> o;
  bool bad = isnan(rest2) || rest2 == __builtin_inf() || !(e.trest < pos_inf());
  // the largest values, as references (in 32 bits: they only set the scale)
  o.zr = static_cast<double>(e.trest) * kLog2ed;
  float mt = neg_inf(), ms = neg_inf();
#pragma unroll
  for (int i = 0; i < ENT; ++i) {
    sh_ids[i * 64 + lane] = e.id[i];
    bad |= e.id[i] >= 0 && (!(e.v[i] < pos_inf()) || !(e.x[i] < pos_inf()));
    mt = fmaxf(mt, e.v[i]);
    ms = fmaxf(ms, e.x[i]);
  }
  row_sync<64>();
  // entries of the same token
  int same[ENT] = {};
#pragma unroll 4
  for (int j = 0; j < K; j += 4) {
    const int4 d = *reinterpret_cast<const int4*>(sh_ids + j);
#pragma unroll
    for (int i = 0; i < ENT; ++i)
      same[i] += (d.x == e.id[i]) + (d.y == e.id[i]) + (d.z == e.id[i]) + (d.w == e.id[i]);
  }
  o.first = 0;
  bool twice = false;
#pragma unroll
  for (int i = 0; i < ENT; ++i) {
    o.first |= e.id[i] >= 0 ? 1u << i : 0u;
    twice |= e.id[i] >= 0 && same[i] > 1;
  }
  o.twice = __any(twice);
  if (o.twice)
    for (int j = 0; j < K; ++j) {
      const int32_t id = sh_ids[j];
#pragma unroll
      for (int i = 0; i < ENT; ++i)
        if (id == e.id[i] && j < i * 64 + lane) o.first &= ~(1u << i);
    }
  const double nt = fmax(static_cast<double>(wave_max(mt)) * c64, o.zr);
  const double ns = fmax(static_cast<double>(wave_max(ms)) * c64, rest2);
  o.rt = nt == -__builtin_inf() ? 0.0 : nt;
  o.rs = ns == -__builtin_inf() ? 0.0 : ns;
  double st = 0.0, ss = 0.0;
#pragma unroll
  for (int i = 0; i < ENT; ++i) {
    o.zt[i] = static_cast<double>(e.v[i]) * c64;
    o.zs[i] = static_cast<double>(e.x[i]) * c64;
    o.et[i] = e.v[i] > neg_inf() ? exp2_64(o.zt[i] - o.rt) : 0.0;
    o.es[i] = e.x[i] > neg_inf() ? exp2_64(o.zs[i] - o.rs) : 0.0;
    st += o.et[i];
    if ((o.first >> i) & 1u) ss += o.es[i];
  }
  // everything else: the teacher's side on lane 0, the draft's on lane 1
  const double zl = lane == 0 ? o.zr : rest2;
  const double el = zl > -__builtin_inf() ? exp2_64(zl - (lane == 0 ? o.rt : o.rs)) : 0.0;
  o.et_r = lane_d(el, 0);
  o.es_r = lane_d(el, 1);
  o.st = wave_sum64(st) + o.et_r;
  o.ss = wave_sum64(ss) + o.es_r;
  o.bad = __any(bad);
  o.empty = !(o.st > 0.0) || !(o.ss > 0.0);
  return o;
}

// ---- loss ---------------------------------------------------------------------------

// Log2 of the draft's mass outside the list, by the NT threads of a row; valid
// on the first wave.  member: TILES NT words; shm: one Mass a wave.  The row is
// read once, by non-temporal loads (14336 rows of 129280 bf16: 590 us, 6.3 TB/s,
// against 613 with plain ones).
template <typename T, int NT, int TILES>
__device__ __forceinline__ double outside_mass(const Row<T>& r, const DistillArgs& a, size_t row, int tid,
                                               uint32_t* member, Mass* shm) {
  constexpr int EPL = Row<T>::EPL, L = kL, TILE = NT * L;
  const int groups = (r.Q + TILE - 1) / TILE;
  Mass acc = mass_none();
  uint4 u[L], w[L];
  group_load<T, NT, L, true>(r, 0, tid, u);
  for (int g0 = 0; g0 < groups; g0 += TILES) {
    const int n = min(TILES, groups - g0);
    for (int g = 0; g < n; ++g) member[g * NT + tid] = 0u;
    row_sync<NT>();
    for (int j = tid; j < a.K; j += NT) {
      const int32_t id = a.ids[row * a.K + j];
      if (id >= 0 && id < r.V) {
        const int e = id + r.head, q = e / EPL - g0 * TILE;
        if (q >= 0 && q < n * TILE)
          atomicOr(&member[q / TILE * NT + q % NT], 1u << (q / NT % L * EPL + e % EPL));
      }
    }
    row_sync<NT>();
    auto take = [&](uint4(&v)[L], int g) {
      const uint32_t word = member[g * NT + tid];
      if (__any(word != 0)) mask_out<T, L>(v, word);
      acc = mass_add(acc, group_mass<T, L>(v, a.c), a.c);
    };
    for (int g = 0; g < n; g += 2) {
      if (g0 + g + 1 < groups) group_load<T, NT, L, true>(r, (g0 + g + 1) * TILE, tid, w);
      take(u, g);
      if (g + 1 >= n) break;  // n is even where more groups follow
      if (g0 + g + 2 < groups) group_load<T, NT, L, true>(r, (g0 + g + 2) * TILE, tid, u);
      take(w, g + 1);
    }
    row_sync<NT>();
  }
  acc = wave_mass(acc, a.c);
  if constexpr (NT > 64) {
    const int lane = tid & 63, wave = wave_id();
    if (lane == 0) shm[wave] = acc;
    __syncthreads();
    if (wave == 0) acc = wave_mass(lane < NT / 64 ? shm[lane] : mass_none(), a.c);
  }
  return mass_log2(acc, a.c, a.c64);
}

struct LossOut {
  float* kl;
  float* lse;
  float* rest;
  uint8_t* flags;
};

// A row's outputs, by one wave; returns its loss as written.
template <int ENT>
__device__ __forceinline__ float finish_row(const Entries<ENT>& e, const DistillArgs& a, size_t row, double rest2,
                                            int32_t* sh_ids, const LossOut& out) {
  const Outcomes<ENT> o = outcomes<ENT>(e, a.K, rest2, a.c64, sh_ids);
  // sum t (log t - log s) with log t = z - rt - log st, log s = z - rs - log ss
  double k = 0.0;
#pragma unroll
  for (int i = 0; i < ENT; ++i)
    if (o.et[i] > 0.0) k += o.et[i] * (o.zt[i] - o.zs[i]);
  k = wave_sum64(k);
  if (o.et_r > 0.0) k += o.et_r * (o.zr - rest2);
  k = k / o.st - (o.rt - o.rs) + log2_64(o.ss / o.st);
  // the normaliser is an output of 32 bits: its logarithm, too, is one
  const double lse = o.rs + static_cast<double>(__builtin_amdgcn_logf(static_cast<float>(o.ss)));
  const float nan = __builtin_nanf("");
  const float loss = o.bad ? nan : o.empty ? 0.0f : static_cast<float>(k * kLn2d);
  if ((threadIdx.x & 63) == 0) {
    out.kl[row] = loss;
    out.lse[row] = o.bad ? nan : static_cast<float>(lse * kLn2d);
    out.rest[row] = o.bad ? nan : static_cast<float>(rest2 * kLn2d);
    out.flags[row] = o.bad ? DSPARK_FLAG_NONFINITE : o.empty ? DSPARK_FLAG_EMPTY_ROW : 0;
  }
  return loss;
}

// One workgroup a row.  Bound by HBM where rows are many (the figure above).
template <typename T, int NT, int ENT>
__global__ __launch_bounds__(NT, 4) void distill_loss_kernel(const T* __restrict__ draft, DistillArgs a, int32_t base,
                                                             LossOut out) {
  __shared__ uint32_t member[kMaxTiles * NT];
  __shared__ __align__(16) int32_t sh_ids[64 * ENT];
  __shared__ Mass shm[NT / 64];
  const size_t row = static_cast<size_t>(base) + blockIdx.x;
  const Row<T> r = make_row(draft + row * a.V, a.V);
  Entries<ENT> e;
  if (wave_id() == 0) e = load_entries<T, ENT>(r, a, row);  // on their way while the row streams
  const double rest2 = outside_mass<T, NT, kMaxTiles>(r, a, row, threadIdx.x, member, shm);
  if (wave_id() == 0) finish_row<ENT>(e, a, row, rest2, sh_ids, out);
}

// Sums over the rows that count.
struct Sums {
  double num, sum, cnt;
};
// Weights exp(-k / gamma) of the positions into LDS, by 16 threads; the caller
// synchronises.
__device__ __forceinline__ void position_weights(double* w, int32_t gamma) {
  if (threadIdx.x < DSPARK_MAX_GAMMA) w[threadIdx.x] = exp(-static_cast<double>(threadIdx.x + 1) / gamma);
}
__device__ __forceinline__ void add_row(Sums& s, double weight, float loss) {
  s.num += weight * loss;
  s.sum += loss;
  s.cnt += 1.0;
}
__device__ __forceinline__ void write_sums(float* sums, const Sums& s, float weight) {
  sums[0] = static_cast<float>(weight * s.num);
  sums[1] = static_cast<float>(s.cnt);
  sums[2] = static_cast<float>(s.sum);
  sums[3] = static_cast<float>(s.cnt);
}

// A few short rows: one workgroup, a wave a row, the sums included.  Bound by a
// wave's chain of loads and 64-bit arithmetic: 20 rows of 1024 fp32, 8 us.
template <typename T, int ENT>
__global__ __launch_bounds__(kTinyThreads) void distill_tiny_kernel(const T* __restrict__ draft, DistillArgs a,
                                                                    int32_t R, LossOut out, float* __restrict__ sums) {
  __shared__ uint32_t member[kTinyWaves][kTinyTiles * 64];
  __shared__ __align__(16) int32_t sh_ids[kTinyWaves][64 * ENT];
  __shared__ Sums shs[kTinyWaves];
  __shared__ double shw[DSPARK_MAX_GAMMA];
  const int lane = threadIdx.x & 63, wave = wave_id();
  position_weights(shw, a.gamma);
  __syncthreads();
  Sums s{0.0, 0.0, 0.0};
  for (int rr = wave; rr < R; rr += kTinyWaves) {
    const size_t row = static_cast<size_t>(rr);
    const Row<T> r = make_row(draft + row * a.V, a.V);
    const Entries<ENT> e = load_entries<T, ENT>(r, a, row);
    const double rest2 = outside_mass<T, 64, kTinyTiles>(r, a, row, lane, member[wave], nullptr);
    const float loss = finish_row<ENT>(e, a, row, rest2, sh_ids[wave], out);
    const int b = rr / a.gamma;
    if (!a.block_mask || a.block_mask[b]) add_row(s, shw[rr - b * a.gamma], loss);
  }
  if (lane == 0) shs[wave] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    Sums t{0.0, 0.0, 0.0};
    for (int w = 0; w < kTinyWaves; ++w) {
      t.num += shs[w].num;
      t.sum += shs[w].sum;
      t.cnt += shs[w].cnt;
    }
    write_sums(sums, t, a.weight);
  }
}

// Sums of the rows' losses: a workgroup's stretch of rows, added in a fixed
// order; several workgroups leave partial sums for distill_sums_final.  inverse: 1 /
// gamma, rounded; (row + 1/2) / gamma is at least 1/32 away from every integer, the
// product's rounding under 2^-20 for rows below 2^31, so its integer part is row /
// gamma.  14336 masked rows: 5.8 us, of which 3 are any launch's; with the integer
// division and the mask's loads behind branches 12.9.
__global__ __launch_bounds__(kSumThreads) void distill_sums_kernel(const float* __restrict__ kl, DistillArgs a,
                                                                   int32_t R, int64_t stretch, double inverse,
                                                                   Sums* __restrict__ partial,
                                                                   float* __restrict__ sums) {
  __shared__ Sums shs[kSumThreads / 64];
  __shared__ double shw[DSPARK_MAX_GAMMA];
  position_weights(shw, a.gamma);
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t r0 = blockIdx.x * stretch;
  const int64_t r1 = min(r0 + stretch, static_cast<int64_t>(R));
  Sums s{0.0, 0.0, 0.0};
  // without a mask a byte of kl is read in its place, so that no branch parts the loads
  const uint8_t* mask = a.block_mask ? a.block_mask : reinterpret_cast<const uint8_t*>(kl);
  constexpr int U = 8;  // rows whose loads are in flight together
  for (int64_t row = r0 + threadIdx.x; row < r1; row += U * kSumThreads) {
    float v[U];
    uint32_t k[U];
    bool on[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t q = min(row + i * kSumThreads, r1 - 1);
      const uint32_t b = static_cast<uint32_t>((static_cast<double>(q) + 0.5) * inverse);
      k[i] = static_cast<uint32_t>(q) - b * static_cast<uint32_t>(a.gamma);
      v[i] = kl[q];
      on[i] = mask[a.block_mask ? b : 0u] != 0 || !a.block_mask;
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (on[i] && row + i * kSumThreads < r1) add_row(s, shw[k[i]], v[i]);
  }
  s = Sums{wave_sum64(s.num), wave_sum64(s.sum), wave_sum64(s.cnt)};
  if (lane == 0) shs[wave] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    Sums t{0.0, 0.0, 0.0};
    for (int w = 0; w < kSumThreads / 64; ++w) {
      t.num += shs[w].num;
      t.sum += shs[w].sum;
      t.cnt += shs[w].cnt;
    }
    if (gridDim.x == 1)
      write_sums(sums, t, a.weight);
    else
      partial[blockIdx.x] = t;
  }
}
__global__ __launch_bounds__(64) void distill_sums_final_kernel(const Sums* __restrict__ partial, int32_t n,
                                                                float weight, float* __restrict__ sums) {
  static_assert(kMaxSumBlocks <= 64, "a lane each");
  const int lane = threadIdx.x;
  const Sums p = lane < n ? partial[lane] : Sums{0.0, 0.0, 0.0};
  const Sums s{wave_sum64(p.num), wave_sum64(p.sum), wave_sum64(p.cnt)};
  if (lane == 0) write_sums(sums, s, weight);
}

// ---- gradient -------------------------------------------------------------------------

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two values as bf16, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

template <typename T>
__device__ __forceinline__ void store_elem(T* p, float v) {
  if constexpr (sizeof(T) == 2)
    *p = static_cast<uint16_t>(pack_bf16(v, v));
  else
    *p = v;
}

// Granule q of a gradient row; vec: the row starts as the draft row does, so
// that interior granules are 16-byte stores.  The stores are non-temporal: the
// gradient is written once and is as large as the logits (14336 rows of 129280
// bf16: 1342 us against 1444 with plain stores, 305 rows of 32003: 11.1 against
// 12.3; non-temporal loads of the logits beside them: 1401).
template <typename T>
__device__ __forceinline__ void gran_store(T* g, const Row<T>& r, int q, bool vec, const float (&v)[Row<T>::EPL]) {
  constexpr int EPL = Row<T>::EPL;
  const int e0 = q * EPL - r.head;
  if (vec && e0 >= 0 && e0 + EPL <= r.V) {
    u32x4 u;
    if constexpr (sizeof(T) == 2)
      u = u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    else
      u = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(g + e0));
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j >= 0 && e0 + j < r.V) store_elem(g + e0 + j, v[j]);
  }
}

// One segment of a row a workgroup: `groups` groups a thread.  Bound by HBM, the row
// read and written once: 14336 rows of 129280 bf16, an eighth of the blocks masked:
// 1372 us, 5.1 TB/s, where a plain copy reaches 4.9.
// At most 5 waves per SIMD where workgroups share a row's size of work: more rows
// in flight at once cost bandwidth (14336 rows of 129280 bf16: 1342 us against
// 1370 with 7); short rows want all.
template <typename T, int NT, int ENT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(4, NT == 64 ? 8 : 5))) void distill_grad_kernel(
    const T* __restrict__ draft, DistillArgs a, const float* __restrict__ rest, const float* __restrict__ grad_scale,
    int64_t base, int32_t P, int32_t groups, T* __restrict__ grad) {
  constexpr int EPL = Row<T>::EPL, L = kL, TILE = NT * L;
  __shared__ __align__(16) int32_t sh_ids[64 * ENT];  // tokens to write over
  __shared__ float sh_d[64 * ENT];
  __shared__ double sh_t[64 * ENT];
  __shared__ float shc[2];  // factor, reference
  __shared__ int shf[2];    // a row of zeros; the reference is a logit
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int64_t item = base + blockIdx.x;
  const size_t row = static_cast<size_t>(item / P);
  const int seg = static_cast<int>(item - static_cast<int64_t>(row) * P);
  const size_t b = row / a.gamma;
  const Row<T> r = make_row(draft + row * a.V, a.V);
  T* g = grad + row * a.V;
  const bool vec = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(r.p)) & 15u) == 0;
  const int first = seg * groups * TILE;
  const int n = min(groups, (r.Q - first + TILE - 1) / TILE);
  const bool live = !a.block_mask || a.block_mask[b] != 0;
  uint4 ua[L], ub[L];
  if (live && n > 0) group_load<T, NT, L>(r, first, tid, ua);
  if (wave == 0) {
    bool zero = true;
    if (live) {
      const float rst = rest[row];
      const float scale = grad_scale ? grad_scale[0] : 1.0f;
      const double rest2 = static_cast<double>(rst) * kLog2ed;
      const Entries<ENT> e = load_entries<T, ENT>(r, a, row);
      const Outcomes<ENT> o = outcomes<ENT>(e, a.K, rest2, a.c64, sh_ids);
      const double w = static_cast<double>(scale) * a.weight * (a.c64 / kLog2ed) *
                       exp(-static_cast<double>(row - b * a.gamma + 1) / a.gamma);
      zero = o.empty && !o.bad;
      const double it = 1.0 / o.st, is = 1.0 / o.ss;
      double t[ENT];
#pragma unroll
      for (int i = 0; i < ENT; ++i) t[i] = o.et[i] * it;
      if (o.twice) {
#pragma unroll
        for (int i = 0; i < ENT; ++i) sh_t[i * 64 + lane] = t[i];
        row_sync<64>();
#pragma unroll
        for (int i = 0; i < ENT; ++i) {
          t[i] = 0.0;
          for (int j = 0; j < a.K; ++j) t[i] += sh_ids[j] == e.id[i] ? sh_t[j] : 0.0;
        }
        row_sync<64>();
      }
      const int32_t e0 = first * EPL - r.head, e1 = (first + groups * TILE) * EPL - r.head;  // of this segment
#pragma unroll
      for (int i = 0; i < ENT; ++i) {
        sh_d[i * 64 + lane] = o.bad ? __builtin_nanf("") : static_cast<float>(w * (o.es[i] * is - t[i]));
        sh_ids[i * 64 + lane] = ((o.first >> i) & 1u) && e.id[i] >= e0 && e.id[i] < e1 ? e.id[i] : -1;
      }
      if (lane == 0) {
        // the reference is rounded to fp32; what that loses (2^-lost, with |lost|
        // under 2^-15 where a probability is not 0) goes into the factor
        float ref = static_cast<float>(rest2);
        double lost = rest2 - static_cast<double>(ref);
        const bool huge = fabsf(rst) >= kHugeLogit && rst != neg_inf();
        if (huge) {  // x / T - rest is formed as (x - rest T) / T
          ref = static_cast<float>(rest2 / a.c64);
          lost = 0.0;
        } else if (rst == neg_inf()) {  // no other token has mass
          ref = 0.0f;
          lost = 0.0;
        }
        const double f = w * (o.es_r * is - o.et_r * it) * (1.0 - lost * kLn2d);
        shc[0] = o.bad ? __builtin_nanf("") : static_cast<float>(f);
        shc[1] = ref;
        shf[1] = huge ? 1 : 0;
      }
    }
    if (lane == 0) shf[0] = zero ? 1 : 0;
  }
  __syncthreads();
  const float A = shc[0], ref = shc[1];
  if (shf[0]) {
    const float z[EPL] = {};
    for (int t = 0; t < n; ++t)
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int q = first + (t * L + i) * NT + tid;
        if (q < r.Q) gran_store(g, r, q, vec, z);
      }
  } else {
    const bool huge = shf[1] != 0;
    auto put = [&](const uint4(&u)[L], int t) {
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int q = first + (t * L + i) * NT + tid;
        float v[EPL];
        if (huge) {
#pragma unroll
          for (int j = 0; j < EPL; ++j) v[j] = A * __builtin_amdgcn_exp2f((gran_elem(u[i], j, T{}) - ref) * a.c);
        } else {
#pragma unroll
          for (int j = 0; j < EPL; ++j) v[j] = A * __builtin_amdgcn_exp2f(fmaf(gran_elem(u[i], j, T{}), a.c, -ref));
        }
        if (q < r.Q) gran_store(g, r, q, vec, v);
      }
    };
    for (int t = 0; t < n; t += 2) {
      if (t + 1 < n) group_load<T, NT, L>(r, first + (t + 1) * TILE, tid, ub);
      put(ua, t);
      if (t + 1 >= n) break;
      if (t + 2 < n) group_load<T, NT, L>(r, first + (t + 2) * TILE, tid, ua);
      put(ub, t + 1);
    }
    __syncthreads();  // the listed tokens are written after the granules that hold them
    for (int j = tid; j < a.K; j += NT)
      if (sh_ids[j] >= 0) store_elem(g + sh_ids[j], sh_d[j]);
  }
}

// Granules of a row at the least favourable alignment.
int row_granules(int epl, int32_t V) { return static_cast<int>((static_cast<int64_t>(V) + 2 * epl - 2) / epl); }

template <typename T, int ENT>
hipError_t launch_loss(const T* draft, const DistillArgs& a, int32_t R, const LossOut& out, float* sums, Sums* partial,
                       hipStream_t st) {
  constexpr int L = kL;
  const int q = row_granules(Row<T>::EPL, a.V);
  // One launch where the rows are hardly more than a workgroup's waves (V = 1024
  // fp32: 16 rows 7.2 us against 8.9 of two launches, 24 rows 9.3 against 9.1 but a
  // launch less, 32 rows 13.5 against 8.8).
  if (R <= kTinyWaves + kTinyWaves / 2 && q <= kTinyTiles * 64 * L) {
    DSPARK_LAUNCH("distill_tiny", (distill_tiny_kernel<T, ENT>), dim3(1), dim3(kTinyThreads), 0, st, draft, a, R, out,
                  sums);
    return hipGetLastError();
  }
  // A wave a row where rows are short, or many and not long (16000 rows of 16000
  // bf16: 108 us against 121 of 256 threads; 8000 of 1500: 23 against 46); 512
  // threads where rows are few and long (256 rows of 129280: 23 us against 29 of 256
  // threads; 1024 rows: 55 against 53).
  const bool wave = q <= 2 * 64 * L || (R >= 4096 && q <= kMaxTiles * 64 * L);
  const int nt = wave ? 64 : R > 512 || q <= 2 * 256 * L ? 256 : 512;
  for (int32_t base = 0, n; base < R; base += n) {
    n = std::min(R - base, kMaxGrid);
    const dim3 grid(static_cast<unsigned>(n));
    if (nt == 64)
      DSPARK_LAUNCH("distill_loss", (distill_loss_kernel<T, 64, ENT>), grid, dim3(64), 0, st, draft, a, base, out);
    else if (nt == 256)
      DSPARK_LAUNCH("distill_loss", (distill_loss_kernel<T, 256, ENT>), grid, dim3(256), 0, st, draft, a, base, out);
    else
      DSPARK_LAUNCH("distill_loss", (distill_loss_kernel<T, 512, ENT>), grid, dim3(512), 0, st, draft, a, base, out);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t rows = R;
  const int blocks = static_cast<int>(std::min<int64_t>(kMaxSumBlocks, (rows + 16383) / 16384));
  DSPARK_LAUNCH("distill_sums", distill_sums_kernel, dim3(blocks), dim3(kSumThreads), 0, st, out.kl, a, R,
                (rows + blocks - 1) / blocks, 1.0 / a.gamma, partial, sums);
  if (blocks > 1)
    DSPARK_LAUNCH("distill_sums_final", distill_sums_final_kernel, dim3(1), dim3(64), 0, st, partial, blocks, a.weight,
                  sums);
  return hipGetLastError();
}

template <typename T, int ENT>
hipError_t launch_grad(const T* draft, const DistillArgs& a, int32_t R, const float* rest, const float* grad_scale,
                       T* grad, hipStream_t st) {
  constexpr int L = kL;
  const int q = row_granules(Row<T>::EPL, a.V);
  // a wave a row where rows are short (8000 rows of 4000 bf16: 28 us against 37 of
  // 256 threads; of 8000: 59 against 55)
  const int nt = q <= 2 * 64 * L ? 64 : 256;
  const int need = (q + nt * L - 1) / (nt * L);  // groups of a thread over the row
  // shorter segments where that fills the GPU (128 rows of 129280 bf16: 14 us with 8
  // segments a row, 24 with one)
  int groups = need;
  while (groups > 1 && static_cast<int64_t>(R) * ((need + groups - 1) / groups) < 512) groups = (groups + 1) / 2;
  const int P = (need + groups - 1) / groups;
  const int64_t items = static_cast<int64_t>(R) * P;
  for (int64_t base = 0; base < items; base += kMaxGrid) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(items - base, kMaxGrid)));
    if (nt == 64)
      DSPARK_LAUNCH("distill_grad", (distill_grad_kernel<T, 64, ENT>), grid, dim3(64), 0, st, draft, a, rest,
                    grad_scale, base, P, groups, grad);
    else
      DSPARK_LAUNCH("distill_grad", (distill_grad_kernel<T, 256, ENT>), grid, dim3(256), 0, st, draft, a, rest,
                    grad_scale, base, P, groups, grad);
  }
  return hipGetLastError();
}

// Sums of an empty batch.
__global__ void distill_zero_kernel(float* sums) {
  if (threadIdx.x < 4) sums[threadIdx.x] = 0.0f;
}

DistillArgs distill_args(const float* values, const int32_t* ids, const float* teacher_rest, const uint8_t* block_mask,
                         int32_t N, int32_t gamma, int32_t V, int32_t K, float temperature, float weight) {
  return DistillArgs{values, ids, teacher_rest, block_mask, N, gamma, V, K, mass_scale(temperature),
                     mass_scale64(temperature), weight};
}

}  // namespace

size_t distill_bytes() { return align_up(kMaxSumBlocks * sizeof(Sums), 256); }

hipError_t launch_distill(const void* draft, int dtype, const float* values, const int32_t* ids,
                          const float* teacher_rest, const uint8_t* block_mask, int32_t N, int32_t gamma, int32_t V,
                          int32_t K, float temperature, float weight, float* kl, float* lse, float* rest,
                          uint8_t* flags, float* sums, void* ws, hipStream_t st) {
  const int32_t R = N * gamma;
  if (R == 0) {
    DSPARK_LAUNCH("distill_zero", distill_zero_kernel, dim3(1), dim3(64), 0, st, sums);
    return hipGetLastError();
  }
  Sums* partial = static_cast<Sums*>(ws);
  const LossOut out{kl, lse, rest, flags};
  const DistillArgs a = distill_args(values, ids, teacher_rest, block_mask, N, gamma, V, K, temperature, weight);
  const uint16_t* h = static_cast<const uint16_t*>(draft);
  const float* f = static_cast<const float*>(draft);
  if (dtype == DSPARK_BF16)
    return K <= 64 ? launch_loss<uint16_t, 1>(h, a, R, out, sums, partial, st)
                   : launch_loss<uint16_t, 2>(h, a, R, out, sums, partial, st);
  return K <= 64 ? launch_loss<float, 1>(f, a, R, out, sums, partial, st)
                 : launch_loss<float, 2>(f, a, R, out, sums, partial, st);
}

hipError_t launch_distill_backward(const void* draft, int dtype, const float* values, const int32_t* ids,
                                   const float* rest, const float* teacher_rest, const uint8_t* block_mask, int32_t N,
                                   int32_t gamma, int32_t V, int32_t K, float temperature, float weight,
                                   const float* grad_scale, void* grad_draft, hipStream_t st) {
  const int32_t R = N * gamma;
  const DistillArgs a = distill_args(values, ids, teacher_rest, block_mask, N, gamma, V, K, temperature, weight);
  const uint16_t* h = static_cast<const uint16_t*>(draft);
  const float* f = static_cast<const float*>(draft);
  uint16_t* gh = static_cast<uint16_t*>(grad_draft);
  float* gf = static_cast<float*>(grad_draft);
  if (dtype == DSPARK_BF16)
    return K <= 64 ? launch_grad<uint16_t, 1>(h, a, R, rest, grad_scale, gh, st)
                   : launch_grad<uint16_t, 2>(h, a, R, rest, grad_scale, gh, st);
  return K <= 64 ? launch_grad<float, 1>(f, a, R, rest, grad_scale, gf, st)
                 : launch_grad<float, 2>(f, a, R, rest, grad_scale, gf, st);
}

}  // namespace dspark
