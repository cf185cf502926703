// Log-probabilities of given tokens under softmax(z / T), and the gradient of a sum of them and of the
// rows' entropies.
//
// Forward: one pass over the logits, a cluster a row where rows are few (row_softmax.cuh).
// Gradient: from the rows' statistics (maximum m, log(1 + s)) with p_v = 2^((z_v - m) k) / (1 + s), as exact as the losses'
//   own; or from their log-sum-exps alone, with p_v = 2^((z_v - R) k + r), R = fp32(lse T) and r the rest of lse that
//   R leaves (formed in 64 bits, once a row): differences from R keep their bits near the
//   maximum, where z k - lse log2(e) would lose up to 2^-19 of p; what lse's own rounding takes, 2^-24 |lse| of every p, is
//   lost.  Every column is read and written once; the parts of a row need nothing of one another.  At the token 1 - p is
//   -expm1(log p).
//
// Both are bound by memory.  Measured (GB300, by graph replay): 4 rows of 201088 in fp32, scored with their entropies,
// 3.4 us (floor 0.5: one CTA's chain of launch, first load, six batches, exchange); 1536 rows of 201088 in bf16, a tenth
// ignored, 87 (83; 91 with each batch loaded behind the one before it); the gradient of 777 rows of 50021 in bf16
// 25.1 (22.7; 30 without the prefetch of a part, 28 with a cluster barrier before it).
#include "../../include/tail.h"
#include "row_softmax.cuh"
#include "training.h"

namespace tail {

namespace {

template <typename T, bool ENT, int NT>
__global__ void __launch_bounds__(NT, ROW_SM_THREADS / NT) score_kernel(const __grid_constant__ ScoreArgs a) {
  __shared__ Board<1> board;
  const int size = cluster_size(), rank = cluster_rank();
  const int64_t r = blockIdx.x / size;
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  const RowPart p = row_part(row, a.V, rank, size);
  if (size > 1) board.init();
  pdl_wait();
  const int t = a.tokens[r];
  // the first of the row's logits come with its token, whether they will count or not
  Batch v = Batch::from<NT>(part_vectors(row, p), 0, p.count);
  bool live = static_cast<uint32_t>(t) < static_cast<uint32_t>(a.V);
  if (a.cu) live = live && r >= a.cu[0] && r < a.cu[a.nseq];
  const bool first = rank == 0 && threadIdx.x == 0;
  if (first && a.coef) a.coef[r] = 0.f;
  if (!live) {
    if (first) {
      if (a.score) a.score[r] = RowScore{0.f, 0.f, 0.f, -1};
      if (a.logprob) a.logprob[r] = 0.f;
      if (a.lse) a.lse[r] = 0.f;
      if (a.stats) a.stats[2 * r] = a.stats[2 * r + 1] = 0.f;
      if (ENT) a.entropy[r] = 0.f;
    }
    return;
  }
  if (size > 1) cluster_started();
  const float z = first ? Vec<T>::widen1(row[t]) : 0.f;
  if (size > 1) cluster_wait();
  const RowStat mine = merge(stat_pass<T, ENT, NT>(row, p, nullptr, v, a.k, NoMask{}), stat_of(edge_of(row, p)), a.k);
  const RowStat all = cluster_stat<ENT, false>(board, mine, 0.f, a.k, rank, size, a.wait_ns);
  if (!first) return;
  const float ln = log1pf(all.s);
  const bool empty = all.m == -INFINITY;
  const float lp = empty ? -INFINITY : (z - all.m) * a.inv_t - ln;
  if (a.score) a.score[r] = RowScore{all.m, all.s, empty ? 0.f : lp, empty ? -1 : t};
  if (a.logprob) a.logprob[r] = lp;
  // m / T enters exactly: a gradient may take every p from lse
  if (a.lse) a.lse[r] = empty ? -INFINITY : fmaf(all.m, a.inv_t, fmaf(all.m, a.inv_t_low, ln));
  if (a.stats) a.stats[2 * r] = all.m, a.stats[2 * r + 1] = empty ? 0.f : ln;
  if (ENT) a.entropy[r] = empty ? 0.f : ln - 0.693147181f * all.u / (1.f + all.s);
}

// The factors of a row's gradient; false: there is none.  (By one thread: the 64-bit pipe is narrow.)
template <typename T, bool ENT, bool SCORED>
__device__ __forceinline__ bool spread_factors(const SpreadArgs& a, int64_t r, const T* row, const RowPart& p, int rank,
                                               int size, int from, RowGrad& g) {
  g.k = a.k;
  g.B = 0.f;
  if (SCORED) {
    const RowScore sc = a.score[r];
    const float c = a.coef[r] * a.inv_t;
    g.token = sc.token;
    if (sc.token < 0 || c == 0.f) return false;
    prefetch_part(row, p, from);
    g.ref = sc.m;
    g.A = -c / (1.f + sc.s);
    if (!has_column<T>(p, rank, size, sc.token)) return true;  // in place, its part's CTA may have written it
    const float z = Vec<T>::widen1(row[sc.token]);
    g.at_token = c * (z == sc.m ? sc.s : 1.f + sc.s - ex2((z - sc.m) * a.k)) / (1.f + sc.s);
    return true;
  }
  g.token = a.tokens[r];
  const float da = a.a[r] * a.inv_t, db = ENT ? a.b[r] * a.inv_t : 0.f, H = ENT ? a.entropy[r] : 0.f;
  const float* st = a.stats ? a.stats + 2 * r : a.lse + r;
  const float top = st[0], ln = st[a.stats ? 1 : 0];  // the maximum and log(1 + s), or lse twice
  if (static_cast<uint32_t>(g.token) >= static_cast<uint32_t>(a.V) || (da == 0.f && db == 0.f) || top == -INFINITY)
    return false;
  prefetch_part(row, p, from);
  const double off = a.stats ? top : 0.f;  // log p = (z - off) / T - ln
  g.ref = static_cast<float>(top * a.t64);
  const float at = static_cast<float>((g.ref - off) * a.inv_t64 - ln), f = expf(at);  // log p, p at z = ref
  g.A = f * (-da - (ENT ? db * (at + H) : 0.f));
  g.B = -f * db * 0.693147181f;
  if (!has_column<T>(p, rank, size, g.token)) return true;
  const float l = static_cast<float>((Vec<T>::widen1(row[g.token]) - off) * a.inv_t64 - ln);
  g.at_token = -da * expm1f(l);
  if (ENT && l > -INFINITY) g.at_token -= db * expf(l) * (l + H);
  return true;
}

template <typename T, bool ENT, bool SCORED, int NT>
__global__ void __launch_bounds__(NT, ROW_SM_THREADS / NT) spread_kernel(const __grid_constant__ SpreadArgs a) {
  __shared__ RowGrad s_grad;
  __shared__ bool s_live;
  const int size = a.size, rank = blockIdx.x % a.size;
  // after a pass over all rows the last of them are still in L2
  const int64_t r = (SCORED ? gridDim.x - 1 - blockIdx.x : blockIdx.x) / size;
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  T* grad = static_cast<T*>(a.grad) + r * a.gld;
  const RowPart p = row_part(row, a.V, rank, size);
  pdl_wait();
  // the first of the row's logits come with its factors, whether they will count or not
  Batch v = Batch::from<NT, SCORED>(part_vectors(row, p), 0, p.count);
  const float edge = edge_of(row, p);
  if (threadIdx.x == 0) {
    RowGrad g;
    s_live = spread_factors<T, ENT, SCORED>(a, r, row, p, rank, size, ROW_BATCH * NT, g);
    s_grad = g;
  }
  __syncthreads();
  if (!s_live) {
    zero_part(grad, a.V, rank, size);
    return;
  }
  // the loss of pairs begins with the rows that the pass before it has read last, and lets go of what it has read: 217 us
  // instead of 225 at 1,300 rows of 201,088 in bf16
  grad_pass<T, ENT, NT, SCORED, true>(s_grad, GradRow<T>{row, grad, p, nullptr, edge}, v);
}

template <typename T, bool ENT>
cudaError_t scores(const ScoreArgs& a, int rows, cudaStream_t stream) {
  const RowPlan p = plan_stream(rows, a.V, sizeof(T));
  return p.threads == 512   ? launch_rows<score_kernel<T, ENT, 512>>(p, 0, rows, stream, a)
         : p.threads == 256 ? launch_rows<score_kernel<T, ENT, 256>>(p, 0, rows, stream, a)
                            : launch_rows<score_kernel<T, ENT, 128>>(p, 0, rows, stream, a);
}
template <typename T>
cudaError_t scores(const ScoreArgs& a, int rows, cudaStream_t stream) {
  return a.entropy ? scores<T, true>(a, rows, stream) : scores<T, false>(a, rows, stream);
}

template <typename T, bool ENT, bool SCORED>
cudaError_t spread(const SpreadArgs& args, int rows, cudaStream_t stream) {
  RowPlan p = plan_rows(rows, args.V, sizeof(T), 8, -1);
  SpreadArgs a = args;
  a.size = p.size;  // the parts of a row need nothing of one another: no cluster
  const int64_t parts = static_cast<int64_t>(rows) * p.size;
  p.size = 1;
  return p.threads == 256 ? launch_rows<spread_kernel<T, ENT, SCORED, 256>>(p, 0, parts, stream, a)
                          : launch_rows<spread_kernel<T, ENT, SCORED, 128>>(p, 0, parts, stream, a);
}
template <typename T>
cudaError_t spread(const SpreadArgs& a, int rows, cudaStream_t stream) {
  if (a.score) return spread<T, false, true>(a, rows, stream);
  return a.b ? spread<T, true, false>(a, rows, stream) : spread<T, false, false>(a, rows, stream);
}

const char* LIMITS = "more than 1048576 columns or 16777216 rows";

}  // namespace

std::atomic<uint64_t> wait_limit{ROW_WAIT_NS};

uint64_t row_wait_limit() { return wait_limit.load(std::memory_order_relaxed); }

cudaError_t launch_scores(const ScoreArgs& args, int dtype, int rows, cudaStream_t stream) {
  ScoreArgs a = args;
  a.wait_ns = row_wait_limit();
  return dtype == TAIL_F32   ? scores<float>(a, rows, stream)
         : dtype == TAIL_F16 ? scores<__half>(a, rows, stream)
                             : scores<__nv_bfloat16>(a, rows, stream);
}

cudaError_t launch_spread(const SpreadArgs& a, int dtype, int rows, cudaStream_t stream) {
  return dtype == TAIL_F32   ? spread<float>(a, rows, stream)
         : dtype == TAIL_F16 ? spread<__half>(a, rows, stream)
                             : spread<__nv_bfloat16>(a, rows, stream);
}

}  // namespace tail

using namespace tail;

extern "C" int tail_training_set_wait_limit(uint64_t ns) {
  wait_limit.store(ns, std::memory_order_relaxed);
  return TAIL_OK;
}

extern "C" int tail_token_logprobs_ex(int32_t rows, int32_t V, const void* logits, int32_t logits_dtype,
                                      int64_t logits_ld, const int32_t* tokens, double temperature,
                                      float* out_logprob_opt, float* out_lse_opt, float* out_entropy_opt,
                                      float* out_stats_opt, void* stream) {
  const int rc = sizes_ok(rows, V, LIMITS);
  if (rc) return rc;
  if (!temperature_ok(temperature)) return TAIL_ERR_INVALID_ARG;
  if (rows == 0) return TAIL_OK;
  if (!out_logprob_opt && !out_lse_opt && !out_entropy_opt && !out_stats_opt) return TAIL_ERR_INVALID_ARG;
  if (!matrix_ok(logits, logits_dtype, logits_ld, V) || !tokens) return TAIL_ERR_INVALID_ARG;
  if (!words_ok({tokens, out_logprob_opt, out_lse_opt, out_entropy_opt, out_stats_opt})) return TAIL_ERR_INVALID_ARG;
  const int64_t n = 4LL * rows;
  if (outputs_meet({{out_logprob_opt, n}, {out_lse_opt, n}, {out_entropy_opt, n}, {out_stats_opt, 2 * n}},
                   {{tokens, n}, {logits, extent(rows, logits_ld, V, elem_bytes(logits_dtype))}}))
    return TAIL_ERR_INVALID_ARG;
  ScoreArgs a = {};
  a.logits = logits;
  a.ld = logits_ld;
  a.tokens = tokens;
  a.V = V;
  a.k = static_cast<float>(LOG2E / temperature);
  a.inv_t = static_cast<float>(1.0 / temperature);
  a.inv_t_low = static_cast<float>(1.0 / temperature - a.inv_t);
  a.logprob = out_logprob_opt;
  a.lse = out_lse_opt;
  a.entropy = out_entropy_opt;
  a.stats = out_stats_opt;
  const cudaError_t e = launch_scores(a, logits_dtype, rows, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TAIL_OK : cuda_fail(e, "tail_token_logprobs: kernel launch");
}

extern "C" int tail_token_logprobs(int32_t rows, int32_t V, const void* logits, int32_t logits_dtype,
                                   int64_t logits_ld, const int32_t* tokens, double temperature,
                                   float* out_logprob_opt, float* out_lse_opt, float* out_entropy_opt, void* stream) {
  return tail_token_logprobs_ex(rows, V, logits, logits_dtype, logits_ld, tokens, temperature, out_logprob_opt,
                                out_lse_opt, out_entropy_opt, nullptr, stream);
}

extern "C" int tail_token_logprobs_grad_ex(int32_t rows, int32_t V, const void* logits, int32_t logits_dtype,
                                           int64_t logits_ld, const int32_t* tokens, double temperature,
                                           const float* lse_opt, const float* stats_opt, const float* d_logprob,
                                           const float* d_entropy_opt, const float* entropy_opt, void* out_grad,
                                           int64_t grad_ld, void* stream) {
  const int rc = sizes_ok(rows, V, LIMITS);
  if (rc) return rc;
  if (!temperature_ok(temperature) || (d_entropy_opt != nullptr) != (entropy_opt != nullptr)) return TAIL_ERR_INVALID_ARG;
  if (rows == 0) return TAIL_OK;
  if (!matrix_ok(logits, logits_dtype, logits_ld, V) || !matrix_ok(out_grad, logits_dtype, grad_ld, V) || !tokens ||
      (!lse_opt && !stats_opt) || !d_logprob)
    return TAIL_ERR_INVALID_ARG;
  if (!words_ok({tokens, lse_opt, stats_opt, d_logprob, d_entropy_opt, entropy_opt})) return TAIL_ERR_INVALID_ARG;
  const int64_t n = 4LL * rows;
  const int es = elem_bytes(logits_dtype);
  if (!grad_apart(logits, logits_ld, out_grad, grad_ld, rows, V, es) ||
      outputs_meet({{out_grad, extent(rows, grad_ld, V, es)}},
                   {{tokens, n}, {lse_opt, n}, {stats_opt, 2 * n}, {d_logprob, n}, {d_entropy_opt, n}, {entropy_opt, n}}))
    return TAIL_ERR_INVALID_ARG;
  SpreadArgs a = {};
  a.logits = logits;
  a.ld = logits_ld;
  a.grad = out_grad;
  a.gld = grad_ld;
  a.tokens = tokens;
  a.V = V;
  a.t64 = stats_opt ? 1.0 : temperature;
  a.inv_t64 = 1.0 / temperature;
  a.k = static_cast<float>(LOG2E / temperature);
  a.inv_t = static_cast<float>(a.inv_t64);
  a.lse = lse_opt;
  a.stats = stats_opt;
  a.a = d_logprob;
  a.b = d_entropy_opt;
  a.entropy = entropy_opt;
  const cudaError_t e = launch_spread(a, logits_dtype, rows, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TAIL_OK : cuda_fail(e, "tail_token_logprobs_grad: kernel launch");
}

extern "C" int tail_token_logprobs_grad(int32_t rows, int32_t V, const void* logits, int32_t logits_dtype,
                                        int64_t logits_ld, const int32_t* tokens, double temperature, const float* lse,
                                        const float* d_logprob, const float* d_entropy_opt, const float* entropy_opt,
                                        void* out_grad, int64_t grad_ld, void* stream) {
  return tail_token_logprobs_grad_ex(rows, V, logits, logits_dtype, logits_ld, tokens, temperature, lse, nullptr,
                                     d_logprob, d_entropy_opt, entropy_opt, out_grad, grad_ld, stream);
}
