// Pieces shared by the entry points of the training operators: argument checks, and the two passes over
// rows that token_logprobs.cu offers to preference_loss.cu.
#pragma once

#include <cuda_runtime.h>
#include <initializer_list>
#include <math.h>
#include <stdint.h>

#include "abi_common.h"

namespace tail {

constexpr int TRAIN_MAX_V = 1 << 20;
constexpr int TRAIN_MAX_ROWS = 1 << 24;

// A row's score for a later pass: statistics as in row_softmax.cuh; token -1: not counted.
struct RowScore {
  float m, s, logprob;
  int32_t token;
};

// Log-probabilities of the rows' tokens.  `score` (with `cu`: rows outside [cu[0], cu[nseq]) are not
// counted, and `coef` is cleared), or the four arrays.
struct ScoreArgs {
  const void* logits;
  int64_t ld;
  const int32_t* tokens;
  int V;
  float k, inv_t;  // log2(e) / T, 1 / T
  float inv_t_low;  // what inv_t leaves of 1 / T, where lse is asked for
  float *logprob, *lse, *entropy, *stats;
  RowScore* score;
  float* coef;
  const int32_t* cu;
  int nseq;
  uint64_t wait_ns;  // (launch_scores')
};
cudaError_t launch_scores(const ScoreArgs& a, int dtype, int rows, cudaStream_t stream);

// The gradient of sum a logprob + b entropy from the rows' statistics or log-sum-exps, or of sum coef logprob from their
// scores.
struct SpreadArgs {
  const void* logits;
  int64_t ld;
  void* grad;
  int64_t gld;
  const int32_t* tokens;
  int V;
  float k, inv_t;
  double t64, inv_t64;  // T (1 with statistics), 1 / T
  const float *lse, *stats, *a, *b, *entropy;
  const RowScore* score;
  const float* coef;
  int size;  // CTAs a row (launch_spread's)
};
cudaError_t launch_spread(const SpreadArgs& a, int dtype, int rows, cudaStream_t stream);

// How long the CTAs of a row wait for one another's sums, in ns (tail_training_set_wait_limit's).
uint64_t row_wait_limit();

// ---------------------------------------------------------------- argument checks

struct Range {
  const void* p;
  int64_t bytes;
};

// Whether an output meets an input or another output (absent arrays meet nothing).
inline bool outputs_meet(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  const Range* o = outs.begin();
  for (size_t i = 0; i < outs.size(); ++i) {
    if (!o[i].p) continue;
    for (const Range& in : ins)
      if (in.p && overlap(o[i].p, o[i].bytes, in.p, in.bytes)) return true;
    for (size_t j = 0; j < i; ++j)
      if (o[j].p && overlap(o[i].p, o[i].bytes, o[j].p, o[j].bytes)) return true;
  }
  return false;
}

inline bool words_ok(std::initializer_list<const void*> ps) {  // each null or 4-byte aligned
  for (const void* p : ps)
    if (p && !aligned(p, 4)) return false;
  return true;
}

// A matrix [rows][ld] of dtype with V columns.
inline bool matrix_ok(const void* p, int dtype, int64_t ld, int V) {
  return p && dtype >= TAIL_F32 && dtype <= TAIL_BF16 && ld >= V && aligned(p, elem_bytes(dtype));
}

// Temperatures whose inverse and log2(e) / T are ordinary fp32 numbers.
inline bool temperature_ok(double t) { return t >= 0x1p-64 && t <= 0x1p64; }

inline int sizes_ok(int rows, int V, const char* what) {
  if (rows < 0 || V < 1) return TAIL_ERR_INVALID_ARG;
  if (rows > TRAIN_MAX_ROWS || V > TRAIN_MAX_V) {
    set_last_error(what);
    return TAIL_ERR_UNSUPPORTED;
  }
  return TAIL_OK;
}

constexpr double LOG2E = 1.4426950408889634074;

}  // namespace tail
