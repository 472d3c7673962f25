// distill.hip — distillation from a teacher's highest logits: loss and gradient.
//
// Semantics (include/dspark.h, dspark_distill): the outcomes are the K tokens
// that the teacher lists and, where its remaining mass is given, everything
// else as one more; kl = sum_j t_j (log t_j - log s_j) over them, with t the
// teacher's and s the draft's probabilities at temperature T.
//
// Loss, two launches.  distill_mass streams the draft rows once and sums the
// mass of the tokens outside the teacher's list, and of nothing else: the
// list becomes a bit mask in LDS, one word per thread and group of 4
// granules, so a group without a listed token (nearly all) costs one LDS read
// and a branch.  distill_rows, one wave a row, forms the K + 1 outcomes in 64
// bits from that mass, the teacher's values and the draft's logits at its
// tokens: where one probability is nearly 1, its logarithm and its difference
// from the other side keep their accuracy, as no 32-bit normaliser of the
// whole row enters.
//
// Gradient, one launch: with d_v the derivative of kl by x_v / T,
//   v in the list:  d_v = s_v - sum_{j: id_j = v} t_j
//   otherwise:      d_v = (s_r - t_r) exp(x_v / T) / sum_{u outside} exp(x_u / T)
// so a row is one factor and one exponential per element, and K values that
// are written over it at the end.
#include <algorithm>

#include "common.hpp"
#include "internal.hpp"
#include "rowstream.hpp"

namespace dspark {
namespace {

constexpr int kMaxGrid = 1 << 20;  // workgroups of a launch; each then takes several items
constexpr int kL = 4;              // granules per thread and group
constexpr int kMaxTiles = 16;      // groups per segment
constexpr int kRowsThreads = 1024; // distill_rows: one wave a row
constexpr int kRowsWaves = kRowsThreads / 64;
constexpr int kRowsGrid = 256;
constexpr double kLn2d = 0.69314718055994530942;
constexpr double kLog2ed = 1.4426950408889634074;

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

template <typename T, int NT>
__global__ __launch_bounds__(NT) void distill_mass_kernel(const T* __restrict__ draft, const int32_t* __restrict__ ids,
                                                          int64_t items, int32_t V, int32_t K, int32_t P, int32_t tiles,
                                                          float c, Mass* __restrict__ parts,
                                                          uint32_t* __restrict__ ticket) {
  constexpr int NW = NT / 64;
  constexpr int EPL = Row<T>::EPL;
  __shared__ uint32_t member[kMaxTiles * NT];
  __shared__ Mass shm[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  if (blockIdx.x == 0 && tid == 0) *ticket = 0u;  // of distill_rows
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const size_t row = static_cast<size_t>(item / P);
    const int seg = static_cast<int>(item - static_cast<int64_t>(row) * P);
    const Row<T> r = make_row(draft + row * V, V);
    const int first = seg * tiles * (NT * kL);
    const int n = min(tiles, (r.Q - first + NT * kL - 1) / (NT * kL));  // groups; <= 0: none
    uint4 a[kL], b[kL];
    if (n > 0) group_load<T, NT, kL>(r, first, tid, a);
    for (int g = 0; g < n; ++g) member[g * NT + tid] = 0u;
    __syncthreads();
    for (int j = tid; j < K; j += NT) {
      const int32_t id = ids[row * K + j];
      if (id >= 0 && id < V) {
        const int e = id + r.head, q = e / EPL - first;
        if (q >= 0 && q < n * NT * kL) {
          const int g = q / (NT * kL), i = (q / NT) % kL;
          atomicOr(&member[g * NT + q % NT], 1u << (i * EPL + e % EPL));
        }
      }
    }
    __syncthreads();
    Mass acc = mass_none();
    auto take = [&](uint4(&u)[kL], int g) {
      const uint32_t word = member[g * NT + tid];
      if (__any(word != 0)) mask_out<T, kL>(u, word);
      acc = mass_add(acc, group_mass<T, kL>(u, c), c);
    };
    for (int g = 0; g < n; g += 2) {
      if (g + 1 < n) group_load<T, NT, kL>(r, first + (g + 1) * NT * kL, tid, b);
      take(a, g);
      if (g + 1 >= n) break;
      if (g + 2 < n) group_load<T, NT, kL>(r, first + (g + 2) * NT * kL, tid, a);
      take(b, g + 1);
    }
    acc = wave_mass(acc, c);
    if constexpr (NW > 1) {
      if (lane == 0) shm[wave] = acc;
      __syncthreads();
      if (wave == 0) acc = wave_mass(lane < NW ? shm[lane] : mass_none(), c);
    }
    if (tid == 0) parts[item] = acc;
    __syncthreads();  // LDS is reused by the next item
  }
}

// ---- the K + 1 outcomes of a row, by one wave --------------------------------------
// Lane l holds entries l and l + 64.  Everything in base-2 logarithms and 64 bits.
constexpr int kEnt = DSPARK_MAX_TOP / 64;

struct Outcomes {
  double lt[kEnt];     // log2 t_j (-inf: no such entry)
  double ls[kEnt];     // log2 s at its token
  int32_t id[kEnt];    // its token, -1: none
  bool first[kEnt];    // no earlier entry of the row has the same token
  double lt_r, ls_r;   // everything else
  double lse;          // log2 of the draft's whole mass
  bool bad;            // a NaN or +inf
  bool empty;          // no mass on one side
};

template <typename T>
__device__ __forceinline__ Outcomes outcomes(const Row<T>& r, const float* __restrict__ values,
                                             const int32_t* __restrict__ ids, const float* __restrict__ teacher_rest,
                                             size_t row, int K, double rest2, double c64, int32_t* sh_ids) {
  const int lane = threadIdx.x & 63;
  Outcomes o;
  double zt[kEnt], zs[kEnt];
  bool bad = isnan(rest2) || rest2 == __builtin_inf();
  double zr = -__builtin_inf();
  if (teacher_rest) {
    const float t = teacher_rest[row];
    bad |= !(t < pos_inf());
    zr = static_cast<double>(t) * kLog2ed;
  }
  double mt = zr, ms = rest2;
#pragma unroll
  for (int i = 0; i < kEnt; ++i) {
    const int j = i * 64 + lane;
    o.id[i] = -1;
    zt[i] = zs[i] = -__builtin_inf();
    if (j < K) {
      const int32_t id = ids[row * K + j];
      if (id >= 0 && id < r.V) {
        o.id[i] = id;
        const float v = values[row * K + j], x = load_logit(r.p, static_cast<size_t>(id));
        bad |= !(v < pos_inf()) || !(x < pos_inf());
        zt[i] = static_cast<double>(v) * c64;
        zs[i] = static_cast<double>(x) * c64;
      }
    }
    sh_ids[j] = o.id[i];
    mt = fmax(mt, zt[i]);
    ms = fmax(ms, zs[i]);
  }
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
  // an earlier entry with the same token
#pragma unroll
  for (int i = 0; i < kEnt; ++i) o.first[i] = o.id[i] >= 0;
  for (int j = 0; j < K; ++j) {
    const int32_t id = sh_ids[j];
#pragma unroll
    for (int i = 0; i < kEnt; ++i) o.first[i] = o.first[i] && !(id == o.id[i] && j < i * 64 + lane);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    mt = fmax(mt, __shfl_xor(mt, d, 64));
    ms = fmax(ms, __shfl_xor(ms, d, 64));
  }
  double st = 0.0, ss = 0.0;
  const double nt = mt == -__builtin_inf() ? 0.0 : mt, ns = ms == -__builtin_inf() ? 0.0 : ms;
#pragma unroll
  for (int i = 0; i < kEnt; ++i) {
    if (i * 64 >= K) break;
    st += exp2(zt[i] - nt);
    if (o.first[i]) ss += exp2(zs[i] - ns);
  }
  st = wave_sum64(st) + exp2(zr - nt);
  ss = wave_sum64(ss) + exp2(rest2 - ns);
  o.bad = __any(bad);
  o.empty = !(st > 0.0) || !(ss > 0.0);
  const double lt = nt + log2(st);
  o.lse = ns + log2(ss);
#pragma unroll
  for (int i = 0; i < kEnt; ++i) {
    o.lt[i] = zt[i] - lt;
    o.ls[i] = zs[i] - o.lse;
  }
  o.lt_r = zr - lt;
  o.ls_r = rest2 - o.lse;
  return o;
}

struct DistillArgs {
  const float* values;
  const int32_t* ids;
  const float* teacher_rest;  // or NULL
  const uint8_t* block_mask;  // or NULL
  int32_t N, gamma, V, K, P;
  float c;
  double c64;
  float weight;
};

// The rows' losses, then (the workgroup that is done last) the sums, of
// per-workgroup sums in a fixed order.
template <typename T>
__global__ __launch_bounds__(kRowsThreads) void distill_rows_kernel(const T* __restrict__ draft, DistillArgs a,
                                                                    const Mass* __restrict__ parts, int32_t R,
                                                                    float* __restrict__ kl, float* __restrict__ lse,
                                                                    float* __restrict__ rest, uint8_t* __restrict__ flags,
                                                                    float* __restrict__ sums, double* partial,
                                                                    uint32_t* ticket) {
  __shared__ int32_t sh_ids[kRowsWaves][DSPARK_MAX_TOP];
  __shared__ double shs[3][kRowsWaves];
  __shared__ uint32_t shl;
  const int lane = threadIdx.x & 63, wave = wave_id();
  double num = 0.0, sum = 0.0, cnt = 0.0;
  for (int64_t rr = static_cast<int64_t>(blockIdx.x) * kRowsWaves + wave; rr < R;
       rr += static_cast<int64_t>(gridDim.x) * kRowsWaves) {
    const size_t row = static_cast<size_t>(rr);
    const Row<T> r = make_row(draft + row * a.V, a.V);
    Mass m = mass_none();
    for (int p = lane; p < a.P; p += 64) m = mass_add(m, parts[row * a.P + p], a.c);
    m = wave_mass(m, a.c);
    const double rest2 = mass_log2(m, a.c, a.c64);
    const Outcomes o = outcomes(r, a.values, a.ids, a.teacher_rest, row, a.K, rest2, a.c64, sh_ids[wave]);
    double k = 0.0;
#pragma unroll
    for (int i = 0; i < kEnt; ++i) {
      if (i * 64 >= a.K) break;
      const double t = exp2(o.lt[i]);
      if (t > 0.0) k += t * (o.lt[i] - o.ls[i]);
    }
    k = wave_sum64(k);
    const double tr = exp2(o.lt_r);
    if (tr > 0.0) k += tr * (o.lt_r - o.ls_r);
    const double loss = o.bad ? __builtin_nan("") : o.empty ? 0.0 : k * kLn2d;
    if (lane == 0) {
      kl[row] = static_cast<float>(loss);
      lse[row] = o.bad ? __builtin_nanf("") : static_cast<float>(o.lse * kLn2d);
      rest[row] = o.bad ? __builtin_nanf("") : static_cast<float>(rest2 * kLn2d);
      flags[row] = o.bad ? DSPARK_FLAG_NONFINITE : o.empty ? DSPARK_FLAG_EMPTY_ROW : 0;
    }
    const int b = static_cast<int>(row / a.gamma), pos = static_cast<int>(row - static_cast<size_t>(b) * a.gamma);
    if (!a.block_mask || a.block_mask[b]) {
      num += exp(-static_cast<double>(pos + 1) / a.gamma) * loss;
      sum += loss;
      cnt += 1.0;
    }
  }
  if (lane == 0) {
    shs[0][wave] = num;
    shs[1][wave] = sum;
    shs[2][wave] = cnt;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double t[3] = {0.0, 0.0, 0.0};
    for (int q = 0; q < 3; ++q)
      for (int w = 0; w < kRowsWaves; ++w) t[q] += shs[q][w];
    for (int q = 0; q < 3; ++q) {
      const uint64_t v = static_cast<uint64_t>(__double_as_longlong(t[q]));
      uint32_t* p = reinterpret_cast<uint32_t*>(partial + static_cast<size_t>(blockIdx.x) * 3 + q);
      store_coherent(p, static_cast<uint32_t>(v));
      store_coherent(p + 1, static_cast<uint32_t>(v >> 32));
    }
    shl = publish(ticket) == gridDim.x - 1 ? 1u : 0u;
  }
  __syncthreads();
  if (shl && wave == 0) {
    double t[3] = {0.0, 0.0, 0.0};
    for (int i = lane; i < static_cast<int>(gridDim.x); i += 64)
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(partial + static_cast<size_t>(i) * 3 + q);
        const uint64_t lo = load_coherent(p), hi = load_coherent(p + 1);
        t[q] += __longlong_as_double(static_cast<long long>(lo | (hi << 32)));
      }
#pragma unroll
    for (int q = 0; q < 3; ++q) t[q] = wave_sum64(t[q]);
    if (lane == 0) {
      sums[0] = static_cast<float>(a.weight * t[0]);
      sums[1] = static_cast<float>(t[2]);
      sums[2] = static_cast<float>(t[1]);
      sums[3] = static_cast<float>(t[2]);
    }
  }
}

// Sums of an empty batch.
__global__ void distill_zero_kernel(float* sums) {
  if (threadIdx.x < 4) sums[threadIdx.x] = 0.0f;
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
// that interior granules are 16-byte stores.
template <typename T>
__device__ __forceinline__ void gran_store(T* g, const Row<T>& r, int q, bool vec, const float (&v)[Row<T>::EPL]) {
  constexpr int EPL = Row<T>::EPL;
  const int e0 = q * EPL - r.head;
  if (vec && e0 >= 0 && e0 + EPL <= r.V) {
    uint4 u;
    if constexpr (sizeof(T) == 2)
      u = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    else
      u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    *reinterpret_cast<uint4*>(g + e0) = u;
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j >= 0 && e0 + j < r.V) store_elem(g + e0 + j, v[j]);
  }
}

template <typename T, int NT>
__global__ __launch_bounds__(NT) void distill_grad_kernel(const T* __restrict__ draft, DistillArgs a,
                                                          const float* __restrict__ rest,
                                                          const float* __restrict__ grad_scale, int64_t items,
                                                          int32_t tiles, T* __restrict__ grad) {
  constexpr int EPL = Row<T>::EPL;
  __shared__ int32_t sh_ids[DSPARK_MAX_TOP];  // tokens to write over
  __shared__ float sh_d[DSPARK_MAX_TOP];
  __shared__ double sh_t[DSPARK_MAX_TOP];
  __shared__ float shc[2];  // factor, reference
  __shared__ int shf[2];    // a row of zeros; the reference is a logit
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const size_t row = static_cast<size_t>(item / a.P);
    const int seg = static_cast<int>(item - static_cast<int64_t>(row) * a.P);
    const size_t b = row / a.gamma;
    const Row<T> r = make_row(draft + row * a.V, a.V);
    T* g = grad + row * a.V;
    const bool vec = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(r.p)) & 15u) == 0;
    const int first = seg * tiles * (NT * kL);
    const int n = min(tiles, (r.Q - first + NT * kL - 1) / (NT * kL));
    const bool live = !a.block_mask || a.block_mask[b] != 0;
    uint4 ua[kL], ub[kL];
    if (live && n > 0) group_load<T, NT, kL>(r, first, tid, ua);
    if (wave == 0) {
      bool zero = true;
      if (live) {
        const float rst = rest[row];
        const double rest2 = static_cast<double>(rst) * kLog2ed;
        const Outcomes o = outcomes(r, a.values, a.ids, a.teacher_rest, row, a.K, rest2, a.c64, sh_ids);
        const double w = (grad_scale ? static_cast<double>(grad_scale[0]) : 1.0) * a.weight * a.c64 / kLog2ed *
                         exp(-static_cast<double>(row - b * a.gamma + 1) / a.gamma);
        zero = o.empty && !o.bad;
#pragma unroll
        for (int i = 0; i < kEnt; ++i) sh_t[i * 64 + lane] = o.id[i] >= 0 ? exp2(o.lt[i]) : 0.0;
        __builtin_amdgcn_wave_barrier();
        __threadfence_block();
#pragma unroll
        for (int i = 0; i < kEnt; ++i) {
          double t = 0.0;
          for (int j = 0; j < a.K; ++j) t += sh_ids[j] == o.id[i] ? sh_t[j] : 0.0;
          sh_d[i * 64 + lane] = o.bad ? __builtin_nanf("") : static_cast<float>(w * (exp2(o.ls[i]) - t));
        }
        __builtin_amdgcn_wave_barrier();
        __threadfence_block();
        const int32_t e0 = first * EPL - r.head, e1 = (first + tiles * NT * kL) * EPL - r.head;  // of this segment
#pragma unroll
        for (int i = 0; i < kEnt; ++i)
          sh_ids[i * 64 + lane] = o.first[i] && o.id[i] >= e0 && o.id[i] < e1 ? o.id[i] : -1;
        if (lane == 0) {
          // the reference is rounded to fp32; what that loses goes into the factor
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
          shc[0] = o.bad ? __builtin_nanf("") : static_cast<float>(w * (exp2(o.ls_r) - exp2(o.lt_r)) * exp2(-lost));
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
        for (int i = 0; i < kL; ++i) {
          const int q = first + (t * kL + i) * NT + tid;
          if (q < r.Q) gran_store(g, r, q, vec, z);
        }
    } else {
      const bool huge = shf[1] != 0;
      auto put = [&](const uint4(&u)[kL], int t) {
#pragma unroll
        for (int i = 0; i < kL; ++i) {
          const int q = first + (t * kL + i) * NT + tid;
          float v[EPL];
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            const float x = gran_elem(u[i], j, T{});
            v[j] = A * __builtin_amdgcn_exp2f(huge ? (x - ref) * a.c : fmaf(x, a.c, -ref));
          }
          if (q < r.Q) gran_store(g, r, q, vec, v);
        }
      };
      for (int t = 0; t < n; t += 2) {
        if (t + 1 < n) group_load<T, NT, kL>(r, first + (t + 1) * NT * kL, tid, ub);
        put(ua, t);
        if (t + 1 >= n) break;
        if (t + 2 < n) group_load<T, NT, kL>(r, first + (t + 2) * NT * kL, tid, ua);
        put(ub, t + 1);
      }
      __syncthreads();  // the listed tokens are written after the granules that hold them
      for (int j = tid; j < a.K; j += NT)
        if (sh_ids[j] >= 0) store_elem(g + sh_ids[j], sh_d[j]);
    }
    __syncthreads();  // LDS is reused by the next item
  }
}

struct Split {
  int NT, tiles, P;
};

// Rows of at most kMaxTiles groups of a wave are taken by waves; others by
// workgroups of 256, in segments of at most kMaxTiles groups, shorter ones
// where that fills the GPU.
Split split(int epl, int64_t R, int32_t V) {
  const int64_t q = (static_cast<int64_t>(V) + 2 * epl - 2) / epl;
  Split s{};
  s.NT = q <= 2 * 64 * kL ? 64 : 256;
  const int64_t need = (q + s.NT * kL - 1) / (s.NT * kL);  // groups of a row
  int t = static_cast<int>(std::min<int64_t>(kMaxTiles, need));
  while (t > 1 && R * ((need + t - 1) / t) < 1024) t = (t + 1) / 2;
  s.tiles = t;
  s.P = static_cast<int>((need + t - 1) / t);
  return s;
}

dim3 item_grid(int64_t items) { return dim3(static_cast<unsigned>(std::min<int64_t>(items, kMaxGrid))); }

template <typename T>
hipError_t launch_loss(const T* draft, const DistillArgs& a, const Split& s, int32_t R, float* kl, float* lse,
                       float* rest, uint8_t* flags, float* sums, Mass* parts, double* partial, uint32_t* ticket,
                       hipStream_t st) {
  const int64_t items = static_cast<int64_t>(R) * s.P;
  if (s.NT == 64)
    DSPARK_LAUNCH("distill_mass", (distill_mass_kernel<T, 64>), item_grid(items), dim3(64), 0, st, draft, a.ids, items,
                  a.V, a.K, s.P, s.tiles, a.c, parts, ticket);
  else
    DSPARK_LAUNCH("distill_mass", (distill_mass_kernel<T, 256>), item_grid(items), dim3(256), 0, st, draft, a.ids,
                  items, a.V, a.K, s.P, s.tiles, a.c, parts, ticket);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int wgs = std::min(kRowsGrid, (R + kRowsWaves - 1) / kRowsWaves);
  DSPARK_LAUNCH("distill_rows", (distill_rows_kernel<T>), dim3(wgs), dim3(kRowsThreads), 0, st, draft, a, parts, R, kl,
                lse, rest, flags, sums, partial, ticket);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_grad(const T* draft, const DistillArgs& a, const Split& s, int32_t R, const float* rest,
                       const float* grad_scale, T* grad, hipStream_t st) {
  const int64_t items = static_cast<int64_t>(R) * s.P;
  if (s.NT == 64)
    DSPARK_LAUNCH("distill_grad", (distill_grad_kernel<T, 64>), item_grid(items), dim3(64), 0, st, draft, a, rest,
                  grad_scale, items, s.tiles, grad);
  else
    DSPARK_LAUNCH("distill_grad", (distill_grad_kernel<T, 256>), item_grid(items), dim3(256), 0, st, draft, a, rest,
                  grad_scale, items, s.tiles, grad);
  return hipGetLastError();
}

DistillArgs distill_args(const float* values, const int32_t* ids, const float* teacher_rest, const uint8_t* block_mask,
                         int32_t N, int32_t gamma, int32_t V, int32_t K, int32_t P, float temperature, float weight) {
  return DistillArgs{values, ids, teacher_rest, block_mask, N, gamma, V, K, P, mass_scale(temperature),
                     mass_scale64(temperature), weight};
}

}  // namespace

DistillPlan plan_distill(int32_t N, int32_t gamma, int32_t V) {
  DistillPlan p{};
  const int64_t R = static_cast<int64_t>(N) * gamma;
  const int P = std::max(split(4, R, V).P, split(8, R, V).P);
  size_t off = 0;
  p.off_ticket = off;
  off = align_up(off + sizeof(uint32_t), 256);
  p.off_partial = off;
  off = align_up(off + static_cast<size_t>(kRowsGrid) * 3 * sizeof(double), 256);
  p.off_parts = off;
  off = align_up(off + static_cast<size_t>(R) * P * sizeof(Mass), 256);
  p.bytes = off;
  return p;
}

hipError_t launch_distill(const void* draft, int dtype, const float* values, const int32_t* ids,
                          const float* teacher_rest, const uint8_t* block_mask, int32_t N, int32_t gamma, int32_t V,
                          int32_t K, float temperature, float weight, float* kl, float* lse, float* rest,
                          uint8_t* flags, float* sums, void* ws, const DistillPlan& pl, hipStream_t st) {
  const int32_t R = N * gamma;
  if (R == 0) {
    DSPARK_LAUNCH("distill_zero", distill_zero_kernel, dim3(1), dim3(64), 0, st, sums);
    return hipGetLastError();
  }
  char* w = static_cast<char*>(ws);
  Mass* parts = reinterpret_cast<Mass*>(w + pl.off_parts);
  double* partial = reinterpret_cast<double*>(w + pl.off_partial);
  uint32_t* ticket = reinterpret_cast<uint32_t*>(w + pl.off_ticket);
  const Split s = split(dtype == DSPARK_BF16 ? 8 : 4, R, V);
  const DistillArgs a = distill_args(values, ids, teacher_rest, block_mask, N, gamma, V, K, s.P, temperature, weight);
  if (dtype == DSPARK_BF16)
    return launch_loss(static_cast<const uint16_t*>(draft), a, s, R, kl, lse, rest, flags, sums, parts, partial,
                       ticket, st);
  return launch_loss(static_cast<const float*>(draft), a, s, R, kl, lse, rest, flags, sums, parts, partial, ticket, st);
}

hipError_t launch_distill_backward(const void* draft, int dtype, const float* values, const int32_t* ids,
                                   const float* rest, const float* teacher_rest, const uint8_t* block_mask, int32_t N,
                                   int32_t gamma, int32_t V, int32_t K, float temperature, float weight,
                                   const float* grad_scale, void* grad_draft, hipStream_t st) {
  const int32_t R = N * gamma;
  const Split s = split(dtype == DSPARK_BF16 ? 8 : 4, R, V);
  const DistillArgs a = distill_args(values, ids, teacher_rest, block_mask, N, gamma, V, K, s.P, temperature, weight);
  if (dtype == DSPARK_BF16)
    return launch_grad(static_cast<const uint16_t*>(draft), a, s, R, rest, grad_scale,
                       static_cast<uint16_t*>(grad_draft), st);
  return launch_grad(static_cast<const float*>(draft), a, s, R, rest, grad_scale, static_cast<float*>(grad_draft), st);
}

}  // namespace dspark
