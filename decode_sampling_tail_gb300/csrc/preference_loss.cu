// The paired preference loss over whole sequences and its gradient.
//
// Three launches: the log-probabilities of all counted rows (token_logprobs.cu); a CTA a pair, which adds up
// its two sequences' log-probabilities in row order (64-bit sums: a margin is the difference of two sums of hundreds),
// forms the loss and leaves each row its factor; the gradient from the rows' statistics.  The factor of a row needs
// every row of both sequences, so the logits pass twice; the second pass begins with the rows that the first has read last,
// which are still in L2.
//
// Measured (GB300, by graph replay): one pair, 26 rows of 32000 in fp16, 9.9 us (floor 0.4: three launches in a chain);
// 8 pairs, 1300 rows of 201088 in bf16, 216 (134 for one pass of reads; 217 for two from HBM).
#include "../../include/tail.h"
#include "row_softmax.cuh"
#include "training.h"

namespace tail {

namespace {

constexpr int PAIR_THREADS = 256;

struct PairArgs {
  const int32_t* cu;
  int rows;
  const RowScore* score;
  float* coef;
  const float *ref, *weight;
  float *loss, *seq;
  float beta, eps, margin;
  int average, grad;
};

__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < PAIR_THREADS / 32; ++i) v += sh[i];
  return v;
}

__global__ void __launch_bounds__(PAIR_THREADS) pair_kernel(const __grid_constant__ PairArgs a) {
  __shared__ double sh[PAIR_THREADS / 32];
  const int pair = blockIdx.x, tid = threadIdx.x;
  pdl_wait();
  double L[2];
  int lo[2], hi[2];
  float each[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    lo[q] = min(max(a.cu[2 * pair + q], 0), a.rows);
    hi[q] = min(max(a.cu[2 * pair + q + 1], lo[q]), a.rows);
    double v = 0;
    int n = 0;
    for (int r = lo[q] + tid; r < hi[q]; r += PAIR_THREADS) {
      const RowScore s = a.score[r];
      v += s.logprob;
      n += s.token >= 0;
    }
    L[q] = block_sum(v, sh);
    each[q] = 1.f;
    if (a.average) {
      const double number = block_sum(n, sh);
      each[q] = number > 1 ? static_cast<float>(1.0 / number) : 1.f;
      L[q] *= number > 1 ? 1.0 / number : 1.0;
    }
  }
  const double r0 = a.ref ? a.ref[2 * pair] : 0.f, r1 = a.ref ? a.ref[2 * pair + 1] : 0.f;
  const float w = a.weight ? a.weight[pair] : 1.f;
  const float h = static_cast<float>(a.beta * ((L[0] - r0) - (L[1] - r1)) - a.margin);
  if (tid == 0) {
    if (a.seq) {
      a.seq[2 * pair] = static_cast<float>(L[0]);
      a.seq[2 * pair + 1] = static_cast<float>(L[1]);
    }
    // log(1 + exp(-h)) and, h above it, log(1 + exp(h)); a factor of 0 takes nothing of an infinite term
    const float up = fmaxf(-h, 0.f) + log1pf(expf(-fabsf(h))), down = fmaxf(h, 0.f) + log1pf(expf(-fabsf(h)));
    const float one = a.eps < 1.f ? (1.f - a.eps) * up : 0.f, two = a.eps > 0.f ? a.eps * down : 0.f;
    a.loss[pair] = w == 0.f ? 0.f : h != h ? h : w * (one + two);
  }
  if (!a.grad) return;
  // dloss / dh = eps - sigmoid(-h) = eps sigmoid(h) - (1 - eps) sigmoid(-h)
  const float e = expf(-fabsf(h)), small = e / (1.f + e), large = 1.f / (1.f + e);
  const float neg = h >= 0.f ? small : large, pos = h >= 0.f ? large : small;
  const float d = w == 0.f ? 0.f : w * a.beta * (a.eps * pos - (1.f - a.eps) * neg) + (h != h ? h : 0.f);
#pragma unroll
  for (int q = 0; q < 2; ++q)
    for (int r = lo[q] + tid; r < hi[q]; r += PAIR_THREADS) a.coef[r] = (q ? -d : d) * each[q];
}

int64_t round256(int64_t v) { return (v + 255) & ~int64_t(255); }

int64_t workspace_bytes_for(int64_t rows) { return round256(rows * sizeof(RowScore)) + round256(rows * sizeof(float)); }

}  // namespace

}  // namespace tail

using namespace tail;

static const char* PREF_LIMITS = "more than 1048576 columns, 16777216 rows or 16777216 sequences";

extern "C" int tail_preference_loss_workspace(int32_t rows, int64_t* bytes) {
  if (!bytes || rows < 0) return TAIL_ERR_INVALID_ARG;
  if (rows > TRAIN_MAX_ROWS) {
    set_last_error(PREF_LIMITS);
    return TAIL_ERR_UNSUPPORTED;
  }
  *bytes = workspace_bytes_for(rows);
  return TAIL_OK;
}

extern "C" int tail_preference_loss(int32_t rows, int32_t V, int32_t nseq, const void* logits, int32_t logits_dtype,
                                    int64_t logits_ld, const int32_t* tokens, const int32_t* cu_rows,
                                    double temperature, const float* ref_logprob_opt, float beta, float label_smoothing,
                                    float margin, int32_t average, const float* weight_opt, void* workspace,
                                    int64_t workspace_bytes, float* out_loss, float* out_seq_logprob_opt,
                                    void* out_grad_opt, int64_t grad_ld, void* stream) {
  const int rc = sizes_ok(rows, V, PREF_LIMITS);
  if (rc) return rc;
  if (nseq < 0 || nseq % 2 || !temperature_ok(temperature) || !isfinite(beta) || !isfinite(margin) ||
      !(label_smoothing >= 0.f && label_smoothing <= 1.f) || average < 0 || average > 1)
    return TAIL_ERR_INVALID_ARG;
  if (nseq > TRAIN_MAX_ROWS) {
    set_last_error(PREF_LIMITS);
    return TAIL_ERR_UNSUPPORTED;
  }
  if (!cu_rows || (nseq > 0 && !out_loss)) return TAIL_ERR_INVALID_ARG;
  const int64_t need = workspace_bytes_for(rows);
  if (rows > 0) {
    if (!matrix_ok(logits, logits_dtype, logits_ld, V) || !tokens) return TAIL_ERR_INVALID_ARG;
    if (out_grad_opt && !matrix_ok(out_grad_opt, logits_dtype, grad_ld, V)) return TAIL_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) return TAIL_ERR_INVALID_ARG;
  }
  if (!words_ok({tokens, cu_rows, ref_logprob_opt, weight_opt, out_loss, out_seq_logprob_opt}))
    return TAIL_ERR_INVALID_ARG;
  const int64_t n = 4LL * rows, pairs = nseq / 2;
  const int es = rows > 0 ? elem_bytes(logits_dtype) : 4;
  const Range lg = {rows > 0 ? logits : nullptr, extent(rows, logits_ld, V, es)};
  const Range gr = {rows > 0 ? out_grad_opt : nullptr, extent(rows, grad_ld, V, es)};
  const Range ws = {rows > 0 ? workspace : nullptr, need};
  const Range in1 = {tokens, n}, in2 = {cu_rows, 4LL * (nseq + 1)}, in3 = {ref_logprob_opt, 4LL * nseq},
              in4 = {weight_opt, 4LL * pairs};
  const Range o1 = {out_loss, 4LL * pairs}, o2 = {out_seq_logprob_opt, 4LL * nseq};
  if (outputs_meet({o1, o2, ws, gr}, {in1, in2, in3, in4}) || outputs_meet({o1, o2, ws}, {lg}) ||
      (gr.p && !grad_apart(logits, logits_ld, out_grad_opt, grad_ld, rows, V, es)))
    return TAIL_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  RowScore* score = static_cast<RowScore*>(workspace);
  float* coef = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + round256(rows * sizeof(RowScore)));
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    ScoreArgs a = {};
    a.logits = logits;
    a.ld = logits_ld;
    a.tokens = tokens;
    a.V = V;
    a.k = static_cast<float>(LOG2E / temperature);
    a.inv_t = static_cast<float>(1.0 / temperature);
    a.score = score;
    a.coef = coef;
    a.cu = cu_rows;
    a.nseq = nseq;
    e = launch_scores(a, logits_dtype, rows, s);
  }
  if (e == cudaSuccess && pairs > 0) {
    PairArgs a = {};
    a.cu = cu_rows;
    a.rows = rows;
    a.score = score;
    a.coef = coef;
    a.ref = ref_logprob_opt;
    a.weight = weight_opt;
    a.loss = out_loss;
    a.seq = out_seq_logprob_opt;
    a.beta = beta;
    a.eps = label_smoothing;
    a.margin = margin;
    a.average = average;
    a.grad = rows > 0 && out_grad_opt;
    e = launch_rows<pair_kernel>(RowPlan{1, PAIR_THREADS, 0}, 0, pairs, s, a);
  }
  if (e == cudaSuccess && rows > 0 && out_grad_opt) {
    SpreadArgs a = {};
    a.logits = logits;
    a.ld = logits_ld;
    a.grad = out_grad_opt;
    a.gld = grad_ld;
    a.V = V;
    a.k = static_cast<float>(LOG2E / temperature);
    a.inv_t = static_cast<float>(1.0 / temperature);
    a.score = score;
    a.coef = coef;
    e = launch_spread(a, logits_dtype, rows, s);
  }
  return e == cudaSuccess ? TAIL_OK : cuda_fail(e, "tail_preference_loss: kernel launch");
}
