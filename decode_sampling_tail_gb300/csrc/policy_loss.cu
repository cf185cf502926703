// The clipped policy loss with its KL and entropy terms, and its gradient, in one pass over the logits.
//
// A row's loss depends on that row alone, so a cluster that holds the row on chip reads it once: its CTAs take
// their parts into shared memory while they form the statistics, exchange those through the cluster, and write the
// gradient from what they hold.  The slope of the loss by the token's log-probability, c, and
// the entropy's factor give dz_v = (c (1[v = t] - p_v) + f p_v (log p_v + H)) / T.
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
  int cached;
};

template <typename T, bool ENT>
__global__ void __launch_bounds__(512, 2) policy_kernel(const __grid_constant__ PolicyArgs a) {
  extern __shared__ uint4 cache[];
  __shared__ StatShared sh;
  const int size = cluster_size(), rank = cluster_rank();
  const int64_t r = blockIdx.x / size;
  pdl_wait();
  const int t = a.tokens[r];
  const float w = a.weight ? a.weight[r] : 1.f;
  T* grad = static_cast<T*>(a.grad) + r * a.gld;
  const bool first = rank == 0 && threadIdx.x == 0;
  if (static_cast<uint32_t>(t) >= static_cast<uint32_t>(a.V) || w == 0.f) {
    if (first) {
      a.loss[r] = 0.f;
      if (a.logprob) a.logprob[r] = 0.f;
      if (a.entropy) a.entropy[r] = 0.f;
    }
    if (a.grad) zero_part(grad, a.V, rank, size);
    return;
  }
  if (size > 1) cluster_arrive();
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  const RowPart p = row_part(row, a.V, rank, size);
  const int cached = min(a.cached, p.count);
  fetch_part(row, p, cache, cached);
  const float z = Vec<T>::widen1(row[t]);
  RowStat st = stat_cached<T, ENT>(row, p, cache, cached, a.k, [](int) { return 0u; });
  if (p.edge_n) st = merge(st, stat_of(Vec<T>::widen1(row[p.edge_lo])), a.k);
  st = cluster_merge(st, a.k, sh, rank, size);
  const float ln = log1pf(st.s), sum = 1.f + st.s;
  if (st.m == -INFINITY) {  // no distribution
    if (first) {
      a.loss[r] = 0.f;
      if (a.logprob) a.logprob[r] = -INFINITY;
      if (a.entropy) a.entropy[r] = 0.f;
    }
    if (a.grad) zero_part(grad, a.V, rank, size);
    return;
  }
  const float lp = (z - st.m) * a.inv_t - ln;
  const float excess = ENT ? -0.693147181f * st.u / sum : 0.f;  // H - log of the sum
  const float R = expf(lp - a.old[r]), A = a.adv[r];
  const float open = -A * R, clipped = -A * fminf(fmaxf(R, a.lo), a.hi);
  float loss = fmaxf(open, clipped), c = open >= clipped ? open : 0.f;
  if (a.kl != 0.f) {
    const float d = a.ref[r] - lp, k = expm1f(d);
    loss += a.kl * (k > 1e30f ? k : k - d);  // (k and d may both be infinite)
    c -= a.kl * k;
  }
  if (ENT) loss -= a.ent * (ln + excess);
  if (first) {
    a.loss[r] = w * loss;
    if (a.logprob) a.logprob[r] = lp;
    if (ENT && a.entropy) a.entropy[r] = ln + excess;
  }
  if (!a.grad) return;
  RowGrad g;
  g.ref = st.m;
  g.k = a.k;
  g.token = t;
  const float cw = w * c * a.inv_t, fw = ENT ? w * a.ent * a.inv_t : 0.f;
  const float et = ex2((z - st.m) * a.k);
  g.A = (fw * excess - cw) / sum;
  g.B = fw * 0.693147181f / sum;
  g.at_token = cw * (z == st.m ? st.s : sum - et) / sum;
  if (ENT && et > 0.f) g.at_token += fw * (et / sum) * (lp + ln + excess);
  grad_part<T, ENT>(g, row, grad, p, cache, cached);
}

template <typename T>
cudaError_t launch(PolicyArgs& a, int rows, bool ent, cudaStream_t stream) {
  const RowPlan p = plan_rows(rows, a.V, sizeof(T), a.grad ? ROW_SM_SMEM / 2 : 0);
  a.cached = p.cached;
  return ent ? launch_rows(policy_kernel<T, true>, p, rows, p.cached * 16, stream, a)
             : launch_rows(policy_kernel<T, false>, p, rows, p.cached * 16, stream, a);
}

}  // namespace

}  // namespace tail

using namespace tail;

extern "C" int tail_policy_loss(int32_t rows, int32_t V, const void* logits, int32_t logits_dtype, int64_t logits_ld,
                                const int32_t* tokens, float temperature, const float* old_logprob,
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
  const bool ent = entropy_coef != 0.f || out_entropy_opt;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == TAIL_F32   ? launch<float>(a, rows, ent, s)
                        : logits_dtype == TAIL_F16 ? launch<__half>(a, rows, ent, s)
                                                   : launch<__nv_bfloat16>(a, rows, ent, s);
  return e == cudaSuccess ? TAIL_OK : cuda_fail(e, "tail_policy_loss: kernel launch");
}
