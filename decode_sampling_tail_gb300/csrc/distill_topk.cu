// Distillation from a teacher's top logits and its gradient, in one pass over the student's logits.
//
// The teacher's list (and the weight of what lies outside it) gives q; the student's p is over the whole
// vocabulary.  Listed columns are marked in a bit map and left out of the pass, so that
// the weight of the others is a sum of its own: 1 - sum of the listed p would lose it where the list holds nearly
// everything.  The listed columns' statistics come from the entries.  Outside the list dz_v is a multiple of the
// softmax over the others, p_rest - q_rest times it; the entries' values p_i - q_i are written
// over it afterwards.  Where both p and q are above one half their difference is taken of 1 - q and 1 - p.
#include "../../include/tail.h"
#include "row_softmax.cuh"
#include "training.h"

namespace tail {

namespace {

constexpr int DISTILL_MAX_K = 1024;

struct DistillArgs {
  const void* logits;
  int64_t ld;
  void* grad;
  int64_t gld;
  const void* vals;
  int64_t vld;
  const int32_t* idx;
  int64_t ild;
  const float *rest, *weight;
  float* loss;
  int V, k_list;
  float k, inv_t;
  double k64;
  int vals_dtype;
  int cached, map_words;
};

__device__ __forceinline__ float list_value(const DistillArgs& a, int64_t r, int i) {
  const int64_t at = r * a.vld + i;
  if (a.vals_dtype == TAIL_F32) return static_cast<const float*>(a.vals)[at];
  if (a.vals_dtype == TAIL_F16) return __half2float(static_cast<const __half*>(a.vals)[at]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(a.vals)[at]);
}

// The teacher's distribution: q_i = 2^((t_i - m) k - D) / (1 + others), and so the rest's.
struct Teacher {
  float m, D, others, ln;  // ln = log(1 + others)
  float q_rest, lq_rest;   // and its logarithm
  float q_list;            // 1 - q_rest
  bool rest_is_max;
};

__device__ __forceinline__ Teacher teacher_of(const RowStat& st, const float* rest, int64_t r, float k, double k64) {
  Teacher t;
  t.m = finite_ref(st.m);
  const bool listed = st.m != -INFINITY;
  const float in = listed ? 1.f + st.s : 0.f;  // relative to m
  t.D = 0.f;
  t.others = st.s;
  t.q_rest = 0.f;
  t.lq_rest = -INFINITY;
  t.q_list = 1.f;
  t.rest_is_max = false;
  t.ln = log1pf(st.s);
  if (!rest || rest[r] == -INFINITY) return t;
  if (!listed) {  // the list's values are all -inf: everything is outside it
    t.others = 0.f, t.ln = 0.f, t.q_rest = 1.f, t.lq_rest = 0.f, t.q_list = 0.f, t.rest_is_max = true;
    return t;
  }
  const float d = static_cast<float>(rest[r] * LOG2E - t.m * k64);  // the rest's weight is 2^d
  if (d <= 0.f) {
    const float w = ex2(fmaxf(d, -200.f));
    t.others = st.s + w;
    t.ln = log1pf(t.others);
    t.q_rest = w / (1.f + t.others);
    t.lq_rest = d * 0.693147181f - t.ln;
    t.q_list = in / (1.f + t.others);
  } else {
    t.rest_is_max = true;
    t.D = d;
    t.others = in * ex2(fmaxf(-d, -200.f));
    if (d != d) t.others = d;
    t.ln = log1pf(t.others);
    t.q_rest = 1.f / (1.f + t.others);
    t.lq_rest = -t.ln;
    t.q_list = t.others / (1.f + t.others);
  }
  return t;
}

template <typename T, bool GRAD>
__global__ void __launch_bounds__(512, 2) distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ uint4 smem[];
  __shared__ StatShared sh;
  uint4* cache = smem;
  uint32_t* map = reinterpret_cast<uint32_t*>(cache + a.cached);
  int32_t* ids = reinterpret_cast<int32_t*>(map + a.map_words);
  float* tv = reinterpret_cast<float*>(ids + a.k_list);  // the teacher's values
  float* zv = tv + a.k_list;                             // the student's logits at the entries
  const int size = cluster_size(), rank = cluster_rank(), tid = threadIdx.x, nt = blockDim.x;
  const int64_t r = blockIdx.x / size;
  pdl_wait();
  const float w = a.weight ? a.weight[r] : 1.f;
  T* grad = static_cast<T*>(a.grad) + r * a.gld;
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  const RowPart p = row_part(row, a.V, rank, size);
  const int cached = GRAD ? min(a.cached, p.count) : 0;
  // The part's columns: [lo, hi), its bits from one vector in front of its first whole one.
  const int body = p.head + p.first * N;
  const int lo = rank == 0 ? 0 : body, hi = rank == size - 1 ? a.V : body + p.count * N;
  const int origin = body - N;

  for (int i = tid; i < a.map_words; i += nt) map[i] = 0;
  bool any = false;
  RowStat ts = no_stat();
  for (int i = tid; i < a.k_list; i += nt) {
    const int id = a.idx[r * a.ild + i];
    const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.V);
    const float v = list_value(a, r, i);
    ids[i] = ok ? id : -1;
    tv[i] = v;
    any = any || ok;
    if (ok) ts = merge(ts, stat_of(v), a.k);
  }
  if (!__syncthreads_or(any && w != 0.f)) {
    if (rank == 0 && tid == 0) a.loss[r] = 0.f;
    if (GRAD) zero_part(grad, a.V, rank, size);
    return;
  }
  if (size > 1) cluster_arrive();
  fetch_part(row, p, cache, cached);
  // The entries of this part (the loss, on rank 0, wants all of them), their bits, and whether an id comes twice.
  bool twice = false;
  for (int i = tid; i < a.k_list; i += nt) {
    const int id = ids[i];
    if (id < 0) continue;
    const bool mine = id >= lo && id < hi;
    if (mine || rank == 0) zv[i] = Vec<T>::widen1(row[id]);
    if (mine) {
      const uint32_t bit = 1u << ((id - origin) & 31);
      twice = (atomicOr(map + ((id - origin) >> 5), bit) & bit) || twice;
    }
  }
  twice = __syncthreads_or(twice);
  // The first of an id's entries stands for its column.
  const auto owner = [&](int i) {
    if (ids[i] < lo || ids[i] >= hi) return false;
    if (twice)
      for (int j = 0; j < i; ++j)
        if (ids[j] == ids[i]) return false;
    return true;
  };
  RowStat in = no_stat();
  for (int i = tid; i < a.k_list; i += nt)
    if (owner(i)) in = merge(in, stat_of(zv[i]), a.k);
  const auto bits = [&](int i) {
    const int at = (i + 1) * N;
    return (map[at >> 5] >> (at & 31)) & ((1u << N) - 1);
  };
  RowStat out = stat_cached<T, false>(row, p, cache, cached, a.k, bits);
  const bool edge = p.edge_n && !(map[(p.edge_lo - origin) >> 5] >> ((p.edge_lo - origin) & 31) & 1);
  if (edge) out = merge(out, stat_of(Vec<T>::widen1(row[p.edge_lo])), a.k);

  ts = warp_merge(ts, a.k);
  __syncthreads();
  if ((tid & 31) == 0) sh.warp[tid >> 5] = ts;
  __syncthreads();
  ts = no_stat();
  for (int i = 0; i < nt / 32; ++i) ts = merge(ts, sh.warp[i], a.k);
  __syncthreads();
  out.u = 0.f;
  out = cluster_merge(out, a.k, sh, rank, size);
  if (size > 1) cluster_arrive();
  __syncthreads();
  in = cluster_merge(in, a.k, sh, rank, size);

  const Teacher t = teacher_of(ts, a.rest, r, a.k, a.k64);
  const RowStat all = merge(out, in, a.k);
  const bool target = ts.m != -INFINITY || t.q_rest > 0.f;
  if (all.m == -INFINITY || !target) {  // no distribution, or nothing to aim at
    if (rank == 0 && tid == 0) a.loss[r] = 0.f;
    if (GRAD) zero_part(grad, a.V, rank, size);
    return;
  }
  const float ln = log1pf(all.s), sum = 1.f + all.s;
  const float out_w = out.m == -INFINITY ? 0.f : (1.f + out.s) * ex2(dist(out.m, all.m, a.k));
  const float in_w = in.m == -INFINITY ? 0.f : (1.f + in.s) * ex2(dist(in.m, all.m, a.k));
  const float p_rest = out_w / sum;
  const float tln = t.ln;

  if (rank == 0) {
    float loss = 0.f;
    for (int i = tid; i < a.k_list; i += nt) {
      if (ids[i] < 0) continue;
      const float y = (tv[i] - t.m) * a.k - t.D, q = ex2(y) / (1.f + t.others);
      if (!(q == 0.f)) loss += q * ((y * 0.693147181f - tln) - ((zv[i] - all.m) * a.inv_t - ln));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
    if ((tid & 31) == 0) sh.warp[tid >> 5].m = loss;
  }
  __syncthreads();
  if (rank == 0 && tid == 0) {
    float loss = 0.f;
    for (int i = 0; i < nt / 32; ++i) loss += sh.warp[i].m;
    if (!(t.q_rest == 0.f)) {
      const float lp = out_w >= in_w ? -log1pf(in_w / out_w)
                                     : (out.m - all.m) * a.inv_t + log1pf(out.s) - ln;
      loss += t.q_rest * (t.lq_rest - (out.m == -INFINITY ? -INFINITY : lp));
    }
    a.loss[r] = w * loss;
  }
  if (!GRAD) return;
  const float wt = w * a.inv_t;
  RowGrad g;
  g.ref = finite_ref(out.m);
  g.k = a.k;
  g.token = -1;
  g.B = 0.f;
  g.at_token = 0.f;
  const float off = p_rest > 0.5f && t.q_rest > 0.5f ? t.q_list - in_w / sum : p_rest - t.q_rest;
  g.A = wt * off / (1.f + out.s);
  grad_part<T, false>(g, row, grad, p, cache, cached);
  __syncthreads();  // the entries' values go over what the pass has written
  for (int i = tid; i < a.k_list; i += nt) {
    if (!owner(i)) continue;
    const float y = (tv[i] - t.m) * a.k - t.D;
    float q = ex2(y) / (1.f + t.others);
    float q_left = !t.rest_is_max && tv[i] == t.m ? t.others / (1.f + t.others) : 1.f - q;
    if (twice) {
      for (int j = i + 1; j < a.k_list; ++j)
        if (ids[j] == ids[i]) q += ex2((tv[j] - t.m) * a.k - t.D) / (1.f + t.others);
      q_left = 1.f - q;
    }
    const float e = ex2((zv[i] - all.m) * a.k), pv = e / sum;
    const float p_left = (zv[i] == all.m ? all.s : sum - e) / sum;
    grad[ids[i]] = Vec<T>::narrow1(wt * (pv > 0.5f && q > 0.5f ? q_left - p_left : pv - q));
  }
}

template <typename T>
cudaError_t launch(DistillArgs& a, int rows, cudaStream_t stream) {
  // the map takes a bit a column and the lists 12 bytes an entry of what a CTA has
  const int lists = 12 * a.k_list;
  const int fit = ROW_SM_SMEM / 2 - lists;
  const RowPlan p = plan_rows(rows, a.V, sizeof(T), a.grad ? fit - fit / 16 : 0);
  const int64_t vecs = (static_cast<int64_t>(a.V) * sizeof(T) + 15) / 16;
  const int64_t part = (vecs + p.size - 1) / p.size;
  a.map_words = static_cast<int>(((part + 2) * Vec<T>::N + 31) / 32 + 1);
  a.cached = p.cached;
  if (a.grad) {
    const int64_t room = (ROW_SM_SMEM / 2 - lists - 4LL * a.map_words) / 16;
    if (a.cached > room) a.cached = static_cast<int>(room < 0 ? 0 : room);
  }
  const int smem = a.cached * 16 + a.map_words * 4 + lists;
  return a.grad ? launch_rows(distill_kernel<T, true>, p, rows, smem, stream, a)
                : launch_rows(distill_kernel<T, false>, p, rows, smem, stream, a);
}

}  // namespace

}  // namespace tail

using namespace tail;

extern "C" int tail_distill_topk(int32_t rows, int32_t V, int32_t k, const void* logits, int32_t logits_dtype,
                                 int64_t logits_ld, const void* topk_vals, int32_t vals_dtype, int64_t vals_ld,
                                 const int32_t* topk_idx, int64_t idx_ld, float temperature,
                                 const float* teacher_rest_opt, const float* weight_opt, float* out_loss,
                                 void* out_grad_opt, int64_t grad_ld, void* stream) {
  const int rc = sizes_ok(rows, V, "more than 1048576 columns or 16777216 rows");
  if (rc) return rc;
  if (k < 1 || k > DISTILL_MAX_K || !temperature_ok(temperature)) return TAIL_ERR_INVALID_ARG;
  if (rows == 0) return TAIL_OK;
  if (!matrix_ok(logits, logits_dtype, logits_ld, V) || !matrix_ok(topk_vals, vals_dtype, vals_ld, k) || !topk_idx ||
      idx_ld < k || !out_loss)
    return TAIL_ERR_INVALID_ARG;
  if (out_grad_opt && !matrix_ok(out_grad_opt, logits_dtype, grad_ld, V)) return TAIL_ERR_INVALID_ARG;
  if (!words_ok({topk_idx, teacher_rest_opt, weight_opt, out_loss})) return TAIL_ERR_INVALID_ARG;
  const int64_t n = 4LL * rows;
  const int es = elem_bytes(logits_dtype);
  const Range lg = {logits, extent(rows, logits_ld, V, es)}, gr = {out_grad_opt, extent(rows, grad_ld, V, es)};
  if (outputs_meet({{out_loss, n}, gr}, {{topk_vals, extent(rows, vals_ld, k, elem_bytes(vals_dtype))},
                                         {topk_idx, extent(rows, idx_ld, k, 4)}, {teacher_rest_opt, n},
                                         {weight_opt, n}}) ||
      outputs_meet({{out_loss, n}}, {lg}) ||
      (out_grad_opt && !grad_apart(logits, logits_ld, out_grad_opt, grad_ld, rows, V, es)))
    return TAIL_ERR_INVALID_ARG;
  DistillArgs a = {};
  a.logits = logits;
  a.ld = logits_ld;
  a.grad = out_grad_opt;
  a.gld = grad_ld;
  a.vals = topk_vals;
  a.vals_dtype = vals_dtype;
  a.vld = vals_ld;
  a.idx = topk_idx;
  a.ild = idx_ld;
  a.rest = teacher_rest_opt;
  a.weight = weight_opt;
  a.loss = out_loss;
  a.V = V;
  a.k_list = k;
  a.k64 = LOG2E / temperature;
  a.k = static_cast<float>(a.k64);
  a.inv_t = static_cast<float>(1.0 / temperature);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == TAIL_F32   ? launch<float>(a, rows, s)
                        : logits_dtype == TAIL_F16 ? launch<__half>(a, rows, s)
                                                   : launch<__nv_bfloat16>(a, rows, s);
  return e == cudaSuccess ? TAIL_OK : cuda_fail(e, "tail_distill_topk: kernel launch");
}
