// vocab.hpp — host-side plumbing of the vocabulary operators (top.hip,
// distill.hip, beam.hip): plans and launchers behind the C ABI.
#pragma once

#include "internal.hpp"

namespace dspark {

// ---- highest logits of rows (top.hip) ----
struct Mass;  // rowstream.hpp

// fp32 and 64-bit log2(e) / T.
float mass_scale(float temperature);
double mass_scale64(float temperature);

// How a row is cut: P segments of `groups` groups of L granules a thread,
// workgroups of NT threads; groups = 0: short rows, NT granules a lane of one wave.
struct TopSplit {
  int NT, L, groups, P;
};
struct TopPlan {
  int P;  // most segments of a row
  size_t off_parts, bytes;
};
TopPlan plan_top(int32_t R, int32_t V, int32_t K);
hipError_t launch_top(const void* logits, int dtype, int32_t R, int32_t V, int32_t K, float temperature, float* values,
                      int32_t* ids, float* rest, float* lse, uint8_t* flags, void* ws, const TopPlan& pl,
                      hipStream_t st);
// Per beam its M best candidates in order: the order keys of their 64-bit scores
// and their keys (0: none); and the beams' flags.
hipError_t launch_beam_rows(const void* logits, int dtype, int32_t R, int32_t V, int32_t M, const float* scores,
                            const uint8_t* finished, int32_t eos, uint64_t* sums, uint64_t* keys, uint8_t* flags,
                            void* ws, const TopPlan& pl, hipStream_t st);

// ---- distillation from a teacher's highest logits (distill.hip) ----
size_t distill_bytes();  // workspace of the loss
hipError_t launch_distill(const void* draft, int dtype, const float* values, const int32_t* ids,
                          const float* teacher_rest, const uint8_t* block_mask, int32_t N, int32_t gamma, int32_t V,
                          int32_t K, float temperature, float weight, float* kl, float* lse, float* rest,
                          uint8_t* flags, float* sums, void* ws, hipStream_t st);
hipError_t launch_distill_backward(const void* draft, int dtype, const float* values, const int32_t* ids,
                                   const float* rest, const float* teacher_rest, const uint8_t* block_mask, int32_t N,
                                   int32_t gamma, int32_t V, int32_t K, float temperature, float weight,
                                   const float* grad_scale, void* grad_draft, hipStream_t st);

// ---- beam search (beam.hip) ----
struct BeamPlan {
  TopPlan rows;
  size_t off_sums, off_keys, off_rows, bytes;
};
BeamPlan plan_beam(int32_t B, int32_t W, int32_t V, int32_t M);
hipError_t launch_beam_select(const void* logits, int dtype, const float* scores, const uint8_t* finished, int32_t eos,
                              int32_t B, int32_t W, int32_t V, int32_t M, int32_t* tokens, int32_t* parents,
                              float* out_scores, uint8_t* flags, void* ws, const BeamPlan& pl, hipStream_t st);
hipError_t launch_beam_reorder(const void* src, void* dst, const int32_t* parents, const int32_t* lengths, int64_t L,
                               int32_t B, int32_t W, int32_t M, int32_t S, int32_t T, int64_t token, hipStream_t st);

}  // namespace dspark
