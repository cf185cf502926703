// The clipped policy loss with its KL and entropy terms, and its gradient, in one launch that reads the logits once.
//
// A row's loss depends on that row alone: its statistics, its token's log-probability l and its entropy H give the loss,
// the slope c of the loss by l and the entropy's factor f, and these dz_v = (c (1[v = t] - p_v) + f p_v (log p_v + H)) / T
// in a second pass over the row, from L2 or shared memory (row_softmax.cuh).  At the token 1 - p is s / (1 + s) where it is
// the likeliest.  One warp forms the factors; formed by every thread they cost 1.5 instructions a column.
//
// Measured (GB300, by graph replay): 12 rows of 201088 in fp32 7.5 us (floor 2.9: the chain of one CTA: first loads 1.6,
// statistics 1.5, exchange and factors 1.5, gradient 1.9); 333 rows of 50021 in fp16 with the entropy term, a fifth ignored,
// 16.6 (9.0: 533 counted parts in 608 places, so that reads, chain and writes follow one another in each, and half of the
// time goes to issuing 14,300 instructions a scheduler); 2048 rows of 201088 in bf16 254 (234).  The loss alone: 5.4 (1.4),
// 8.9 (4.0) and 118 (111).
#include "../../include/tail.h"
#include "row_softmax.cuh"
#include "training.h"

namespace tail {

namespace {

struct PolicyArgs {
  const void* logits;
  int64_t ld;
  void* grad;
  int64_t gld;
  const int32_t* tokens;
  const float *old, *adv, *ref, *weight;
  float *loss, *logprob, *entropy;
  int V;
  float k, inv_t;
  float lo, hi, kl, ent;  // 1 - clip_low, 1 + clip_high, the terms' factors
  int kept;  // vectors of a part that shared memory holds
  uint64_t wait_ns;
};

// A row's loss and the factors of its gradient.
struct PolicyRow {
  int64_t r;
  int t;
  float w, z, old, adv, ref;
};
template <bool ENT>
__device__ __forceinline__ RowGrad policy_row(const PolicyArgs& a, const PolicyRow& x, const RowStat& all, bool first) {
  const float ln = log1pf(all.s), sum = 1.f + all.s, inv = 1.f / sum;
  const bool empty = all.m == -INFINITY;  // no distribution
  const float lp = empty ? -INFINITY : (x.z - all.m) * a.inv_t - ln;
  const float excess = ENT ? -0.693147181f * all.u * inv : 0.f;  // H - log of the sum
  const float R = expf(lp - x.old);
  // an advantage of 0 gives 0 of any ratio, one behind fp32's range too; NaN of the row, or of what it is given, stays
  const bool none = x.adv == 0.f && R == R;
  const float open = none ? 0.f : -x.adv * R, clipped = none ? 0.f : -x.adv * min_nan(max_nan(R, a.lo), a.hi);
  float loss = max_nan(open, clipped), c = open < clipped ? 0.f : open;
  if (a.kl != 0.f) {
    const float d = x.ref - lp, k = expm1f(d);
    loss += a.kl * (k > 1e30f ? k : k - d);  // (k and d may both be infinite)
    c -= a.kl * k;
  }
  if (ENT) loss -= a.ent * (ln + excess);
  if (first) {
    a.loss[x.r] = empty ? 0.f : x.w * loss;
    if (a.logprob) a.logprob[x.r] = lp;
    if (ENT && a.entropy) a.entropy[x.r] = empty ? 0.f : ln + excess;
  }
  RowGrad g;
  g.ref = finite_ref(all.m);
  g.k = a.k;
  g.token = x.t;
  const float cw = x.w * c * a.inv_t, fw = ENT ? x.w * a.ent * a.inv_t : 0.f;
  const float et = ex2((x.z - g.ref) * a.k);
  g.A = (fw * excess - cw) * inv;
  g.B = fw * 0.693147181f * inv;
  g.at_token = cw * (x.z == all.m ? all.s : sum - et) * inv;
  if (ENT && et > 0.f) g.at_token += fw * (et * inv) * (lp + ln + excess);
  if (empty) g.A = g.B = g.at_token = 0.f;
  return g;
}

template <typename T, bool ENT, bool GRAD, int NT>
__global__ void __launch_bounds__(NT, ROW_SM_THREADS / NT) policy_kernel(const __grid_constant__ PolicyArgs a) {
  extern __shared__ uint4 cache[];
  __shared__ Board<1> board;
  __shared__ RowGrad s_grad;
  const int size = cluster_size(), rank = cluster_rank();
  PolicyRow x;
  x.r = blockIdx.x / size;
  const T* row = static_cast<const T*>(a.logits) + x.r * a.ld;
  T* grad = static_cast<T*>(a.grad) + x.r * a.gld;
  const bool first = rank == 0 && threadIdx.x == 0;
  const RowPart p = row_part(row, a.V, rank, size);
  const bool kept = GRAD && a.kept > 0;
  if (size > 1) board.init();
  pdl_wait();
  x.t = a.tokens[x.r];
  x.w = a.weight ? a.weight[x.r] : 1.f;
  // the first of the row's logits come with its token, whether they will count or not
  Batch v;
  if (kept)
    fetch_part<T, NT>(row, p, cache);
  else
    v = Batch::from<NT>(part_vectors(row, p), 0, p.count);
  if (static_cast<uint32_t>(x.t) >= static_cast<uint32_t>(a.V) || x.w == 0.f) {
    if (kept) copy_wait(0);
    if (first) {
      a.loss[x.r] = 0.f;
      if (a.logprob) a.logprob[x.r] = 0.f;
      if (a.entropy) a.entropy[x.r] = 0.f;
    }
    if (GRAD) zero_part(grad, a.V, rank, size);
    return;
  }
  if (GRAD && !kept) prefetch_part(row, p, ROW_BATCH * NT);
  if (size > 1) cluster_started();
  const float edge = edge_of(row, p);
  x.z = 0.f;
  if (threadIdx.x < 32) {
    x.z = Vec<T>::widen1(row[x.t]);
    x.old = a.old[x.r];
    x.adv = a.adv[x.r];
    x.ref = a.kl != 0.f ? a.ref[x.r] : 0.f;
  }
  if (size > 1) cluster_wait();
  RowStat st = stat_pass<T, ENT, NT>(row, p, kept ? cache : nullptr, v, a.k, NoMask{});
  if (p.edge_n) st = merge(st, stat_of(edge), a.k);
  // the second pass's first vectors come while the factors are formed
  if (GRAD && !kept) v = Batch::from<NT>(part_vectors(row, p), 0, p.count);
  st = cluster_stat<ENT, GRAD>(board, st, x.z, a.k, rank, size, a.wait_ns);
  if (threadIdx.x < 32 && (GRAD || rank == 0)) {  // one warp forms the row's factors for all
    const RowGrad g = policy_row<ENT>(a, x, st, first);
    if (GRAD && threadIdx.x == 0) s_grad = g;
  }
  if (!GRAD) return;
  __syncthreads();
  grad_pass<T, ENT, NT>(s_grad, GradRow<T>{row, grad, p, kept ? cache : nullptr, edge}, v);
  if (threadIdx.x < 32 && s_grad.ref != s_grad.ref) board.leave();  // its wait may have run out
}

template <typename T, bool ENT>
cudaError_t launch(PolicyArgs& a, int rows, cudaStream_t stream) {
  if (!a.grad) {
    const RowPlan p = plan_stream(rows, a.V, sizeof(T));
    return p.threads == 512   ? launch_rows<policy_kernel<T, ENT, false, 512>>(p, 0, rows, stream, a)
           : p.threads == 256 ? launch_rows<policy_kernel<T, ENT, false, 256>>(p, 0, rows, stream, a)
                              : launch_rows<policy_kernel<T, ENT, false, 128>>(p, 0, rows, stream, a);
  }
  const RowPlan p = plan_rows(rows, a.V, sizeof(T), 8, 0);
  a.kept = p.kept;
  return p.threads == 256 ? launch_rows<policy_kernel<T, ENT, true, 256>>(p, 16 * p.kept, rows, stream, a)
                          : launch_rows<policy_kernel<T, ENT, true, 128>>(p, 16 * p.kept, rows, stream, a);
}

template <typename T>
cudaError_t launch(PolicyArgs& a, int rows, bool ent, cudaStream_t s) {
  return ent ? launch<T, true>(a, rows, s) : launch<T, false>(a, rows, s);
}

}  // namespace

}  // namespace tail

using namespace tail;

extern "C" int tail_policy_loss(int32_t rows, int32_t V, const void* logits, int32_t logits_dtype, int64_t logits_ld,
                                const int32_t* tokens, double temperature, const float* old_logprob,
                                const float* advantage, const float* ref_logprob_opt, float clip_low, float clip_high,
                                float kl_coef, float entropy_coef, const float* weight_opt, float* out_loss,
                                float* out_logprob_opt, float* out_entropy_opt, void* out_grad_opt, int64_t grad_ld,
                                void* stream) {
  const int rc = sizes_ok(rows, V, "more than 1048576 columns or 16777216 rows");
  if (rc) return rc;
  if (!temperature_ok(temperature) || !(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) ||
      !isfinite(kl_coef) || !isfinite(entropy_coef) || (kl_coef != 0.f && rows > 0 && !ref_logprob_opt))
    return TAIL_ERR_INVALID_ARG;
  if (rows == 0) return TAIL_OK;
  if (!matrix_ok(logits, logits_dtype, logits_ld, V) || !tokens || !old_logprob || !advantage || !out_loss)
    return TAIL_ERR_INVALID_ARG;
  if (out_grad_opt && !matrix_ok(out_grad_opt, logits_dtype, grad_ld, V)) return TAIL_ERR_INVALID_ARG;
  if (!words_ok({tokens, old_logprob, advantage, ref_logprob_opt, weight_opt, out_loss, out_logprob_opt,
                 out_entropy_opt}))
    return TAIL_ERR_INVALID_ARG;
  const int64_t n = 4LL * rows;
  const int es = elem_bytes(logits_dtype);
  const Range lg = {logits, extent(rows, logits_ld, V, es)}, gr = {out_grad_opt, extent(rows, grad_ld, V, es)};
  if (outputs_meet({{out_loss, n}, {out_logprob_opt, n}, {out_entropy_opt, n}, gr},
                   {{tokens, n}, {old_logprob, n}, {advantage, n}, {ref_logprob_opt, n}, {weight_opt, n}}) ||
      outputs_meet({{out_loss, n}, {out_logprob_opt, n}, {out_entropy_opt, n}}, {lg}) ||
      (out_grad_opt && !grad_apart(logits, logits_ld, out_grad_opt, grad_ld, rows, V, es)))
    return TAIL_ERR_INVALID_ARG;
  PolicyArgs a = {};
  a.logits = logits;
  a.ld = logits_ld;
  a.grad = out_grad_opt;
  a.gld = grad_ld;
  a.tokens = tokens;
  a.old = old_logprob;
  a.adv = advantage;
  a.ref = ref_logprob_opt;
  a.weight = weight_opt;
  a.loss = out_loss;
  a.logprob = out_logprob_opt;
  a.entropy = out_entropy_opt;
  a.V = V;
  a.k = static_cast<float>(LOG2E / temperature);
  a.inv_t = static_cast<float>(1.0 / temperature);
  a.lo = static_cast<float>(1.0 - clip_low);
  a.hi = static_cast<float>(1.0 + clip_high);
  a.kl = kl_coef;
  a.ent = entropy_coef;
  a.wait_ns = row_wait_limit();
  const bool ent = entropy_coef != 0.f || out_entropy_opt;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == TAIL_F32   ? launch<float>(a, rows, ent, s)
                        : logits_dtype == TAIL_F16 ? launch<__half>(a, rows, ent, s)
                                                   : launch<__nv_bfloat16>(a, rows, ent, s);
  return e == cudaSuccess ? TAIL_OK : cuda_fail(e, "tail_policy_loss: kernel launch");
}
