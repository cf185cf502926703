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
  int map_words, flag_words, cache_at, kept;  // cache_at, kept: in vectors
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
  bool any;  // whether there is anything to aim at
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
  t.any = listed;
  if (!rest || rest[r] == -INFINITY) return t;
  t.any = true;
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
    t.lq_rest = d > -100.f ? logf(t.q_rest) : d * 0.693147181f - t.ln;
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

// A CTA's shared memory behind the board: the list (ids and the teacher's values), the student's logits at its
// entries, the bit map of the part's listed columns, and a byte a thread and batch that says which of its
// vectors have one.  What is kept of the part follows.
struct List {
  int32_t* ids;
  float* t;
  float* z;
  uint32_t* map;
  uint32_t* flags;
};

// Bits from one vector in front of a part's first whole one to the columns behind its last.
inline int map_words(int64_t part, int n) { return static_cast<int>(((part + 2) * n + 31) / 32 + 1); }
inline int flag_words(int64_t part, int nt) { return batches(static_cast<int>(part), nt) * nt / 4; }

template <int N, int NT>
struct ListMask {
  const uint32_t* map;
  const uint8_t* flag;
  __device__ __forceinline__ uint32_t flags(int b) const { return flag[b * NT + static_cast<int>(threadIdx.x)]; }
  __device__ __forceinline__ uint32_t bits(int i) const {
    const int at = (i + 1) * N;
    return (map[at >> 5] >> (at & 31)) & ((1u << N) - 1);
  }
};

// What a row's gradient needs at the entries: the student's statistics over all columns, weight / T (0: no gradient).
struct EntryGrad {
  float m, s, wt;
};

// A row's loss and the factors of its gradient from the board, by one warp.
__device__ __forceinline__ void distill_row(const DistillArgs& a, int64_t r, float w, const Teacher& t,
                                            const Board<2>& board, RowGrad* g, EntryGrad* e) {
  const int lane = threadIdx.x;
  const RowStat o = board.stat<false>(0, a.k), n = board.stat<false>(1, a.k);
  const RowStat all = merge(o, n, a.k);
  const bool live = all.m != -INFINITY && t.any;  // a distribution, and something to aim at
  const float ln = log1pf(all.s), sum = 1.f + all.s;
  const float out_w = o.m == -INFINITY ? 0.f : (1.f + o.s) * ex2(dist(o.m, finite_ref(all.m), a.k));
  const float in_w = n.m == -INFINITY ? 0.f : (1.f + n.s) * ex2(dist(n.m, finite_ref(all.m), a.k));
  const float p_rest = out_w / sum;
  if (board.rank == 0) {
    float loss = 0.f, q = 0.f;
    for (int i = lane; i < board.sets; i += 32) {
      const float4 x = board.get(0, i);
      if (!(x.w == 0.f)) loss += x.z - x.w * ((finite_ref(board.get(1, i).x) - all.m) * a.inv_t);
      q += x.w;
    }
    // log q_i - l_i is a difference of two logits and of two log-sums: the logarithm of the sums' quotient does not
    // leave each one's rounding behind
    const float scale = 1.f + t.others;
    const float x = t.D == 0.f ? all.s - t.others : sum * ex2(-t.D) - scale;
    const float lead = t.D < 100.f ? log1pf(x / scale) : ln - t.ln - t.D * 0.693147181f;
    loss = warp_sum(loss) + lead * warp_sum(q);
    if (!(t.q_rest == 0.f)) {
      const float lp = out_w >= in_w    ? -log1pf(in_w / out_w)
                       : out_w > 1e-30f ? logf(p_rest)
                                        : (o.m - all.m) * a.inv_t + log1pf(o.s) - ln;
      loss += t.q_rest * (t.lq_rest - (o.m == -INFINITY ? -INFINITY : lp));
    }
    if (lane == 0) a.loss[r] = live ? w * loss : 0.f;
  }
  if (lane == 0) {
    const float wt = live ? w * a.inv_t : 0.f;
    const float off = p_rest > 0.5f && t.q_rest > 0.5f ? t.q_list - in_w / sum : p_rest - t.q_rest;
    *g = RowGrad{finite_ref(o.m), a.k, live ? wt * off / (1.f + o.s) : 0.f, 0.f, 0.f, -1};
    *e = EntryGrad{finite_ref(all.m), all.s, wt};
  }
}

template <typename T, bool GRAD, int NT>
__global__ void __launch_bounds__(NT, ROW_SM_THREADS / NT) distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ uint4 smem[];
  __shared__ RowStat s_warp[NT / 32];
  __shared__ Teacher s_teacher;
  __shared__ RowGrad s_grad;
  __shared__ EntryGrad s_entry;
  const int size = cluster_size(), rank = cluster_rank(), tid = threadIdx.x;
  const Board<2> board = board_at<2>(smem, rank, size);
  List l;
  l.ids = reinterpret_cast<int32_t*>(smem + Board<2>::bytes(board.sets) / 16);
  l.t = reinterpret_cast<float*>(l.ids + a.k_list);
  l.z = l.t + a.k_list;
  l.map = reinterpret_cast<uint32_t*>(l.z + a.k_list);
  l.flags = l.map + a.map_words;
  uint4* cache = smem + a.cache_at;
  const int64_t r = blockIdx.x / size;
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  T* grad = static_cast<T*>(a.grad) + r * a.gld;
  const RowPart p = row_part(row, a.V, rank, size);
  const int cached = GRAD ? min(a.kept, p.count) : 0;
  // The part's columns [lo, hi); bit 0 of the map is one vector in front of its first whole one.
  const int body = p.head + p.first * N, origin = body - N;
  const int lo = rank == 0 ? 0 : body, hi = rank == size - 1 ? a.V : body + p.count * N;
  const auto entries = [&](auto f) {  // f(entry, its column) for this thread's entries in the part
    for (int i = tid; i < a.k_list; i += NT) {
      const int id = l.ids[i];
      if (id >= lo && id < hi) f(i, id);
    }
  };
  for (int i = tid; i < a.map_words + a.flag_words; i += NT) l.map[i] = 0;  // (the flags lie behind the map)
  pdl_wait();

  // The list.  A row is fetched at once when its first entry is one.
  const float w = a.weight ? a.weight[r] : 1.f;
  const bool early = w != 0.f && static_cast<uint32_t>(a.idx[r * a.ild]) < static_cast<uint32_t>(a.V);
  const auto fetch = [&] {
    if (cached > 0)
      fetch_part<T, NT>(row, p, cache, cached);
    else
      prefetch_part(row, p);
  };
  if (early) fetch();
  bool any = false;
  RowStat st[1] = {no_stat()};
  if (w != 0.f)
    for (int i = tid; i < a.k_list; i += NT) {
      const int id = a.idx[r * a.ild + i];
      const float v = list_value(a, r, i);
      const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.V);
      l.ids[i] = ok ? id : -1;
      l.t[i] = v;
      any = any || ok;
      if (ok) st[0] = merge(st[0], stat_of(v), a.k);
    }
  st[0] = warp_merge<1, false>(st, a.k);
  if ((tid & 31) == 0) s_warp[tid >> 5] = st[0];
  if (!__syncthreads_or(any)) {
    if (rank == 0 && tid == 0) a.loss[r] = 0.f;
    if (GRAD) zero_part(grad, a.V, rank, size);
    return;
  }
  if (size > 1) cluster_arrive();
  if (!early) fetch();
  // The entries of this part: their bits, and whether an id comes twice.
  bool twice = false;
  entries([&](int i, int id) {
    const int at = id - origin, v = at / N - 1;
    const uint32_t bit = 1u << (at & 31);
    twice = (atomicOr(l.map + (at >> 5), bit) & bit) || twice;
    if (v >= 0 && v < p.count) {
      const int f = v / (ROW_BATCH * NT) * NT + v % NT;  // its thread's byte of its batch
      atomicOr(l.flags + (f >> 2), 1u << (v / NT % ROW_BATCH + 8 * (f & 3)));
    }
    l.z[i] = Vec<T>::widen1(row[id]);
  });
  if (tid < 32) {
    st[0] = tid < NT / 32 ? s_warp[tid] : no_stat();
    st[0] = warp_merge<1, false>(st, a.k);
    if (tid == 0) s_teacher = teacher_of(st[0], a.rest, r, a.k, a.k64);
  }
  twice = __syncthreads_or(twice);
  const Teacher& t = s_teacher;
  const auto weight = [&](int i) { return ex2((l.t[i] - t.m) * a.k - t.D) / (1.f + t.others); };
  const auto owner = [&](int i, int id) {  // the first of an id's entries stands for its column
    if (twice)
      for (int j = 0; j < i; ++j)
        if (l.ids[j] == id) return false;
    return true;
  };

  // Statistics of the columns outside the list and of the listed ones, and, relative to the latter's maximum in
  // the warp, sum q_i (t_i - z_i) / T and sum q_i.
  const float edge = edge_of(row, p);
  RowStat out[1] = {stat_pass<T, false, NT>(row, p, cache, cached, a.k,
                                            ListMask<N, NT>{l.map, reinterpret_cast<const uint8_t*>(l.flags)})};
  if (p.edge_n && !(l.map[(p.edge_lo - origin) >> 5] >> ((p.edge_lo - origin) & 31) & 1))
    out[0] = merge(out[0], stat_of(edge), a.k);
  RowStat in[1] = {no_stat()};
  entries([&](int i, int id) {
    if (owner(i, id)) in[0] = merge(in[0], stat_of(l.z[i]), a.k);
  });
  out[0] = warp_merge<1, false>(out, a.k);
  in[0] = warp_merge<1, false>(in, a.k);
  float C = 0.f, Q = 0.f;
  entries([&](int i, int) {
    const float q = weight(i);
    if (q == 0.f) return;
    C += q * (((l.t[i] - t.m) - (l.z[i] - finite_ref(in[0].m))) * a.inv_t);
    Q += q;
  });
  const float4 post[2] = {make_float4(out[0].m, out[0].s, warp_sum(C), warp_sum(Q)),
                          make_float4(in[0].m, in[0].s, 0.f, 0.f)};
  if (size > 1) cluster_wait();
  board.post(post);
  board.wait();
  if (tid < 32) distill_row(a, r, w, t, board, &s_grad, &s_entry);
  if (!GRAD) return;
  __syncthreads();
  grad_pass<T, false, NT>(s_grad, GradRow<T>{row, grad, p, cache, cached, edge});
  __syncthreads();  // the entries' values go over what the pass has written
  const EntryGrad e = s_entry;
  entries([&](int i, int id) {
    if (!owner(i, id)) return;
    float q = weight(i), q_left = 1.f - q;
    if (twice) {
      for (int j = i + 1; j < a.k_list; ++j)
        if (l.ids[j] == id) q += weight(j);
      q_left = 1.f - q;
    } else if (q > 0.5f && !t.rest_is_max) {
      q_left = t.others / (1.f + t.others);  // above one half: the largest
    }
    const float x = ex2((l.z[i] - e.m) * a.k), sum = 1.f + e.s, pv = x / sum;
    const float p_left = (l.z[i] == e.m ? e.s : sum - x) / sum;
    grad[id] = Vec<T>::narrow1(e.wt == 0.f ? 0.f : e.wt * (pv > 0.5f && q > 0.5f ? q_left - p_left : pv - q));
  });
}

template <typename T, bool GRAD>
cudaError_t launch(DistillArgs& a, int rows, cudaStream_t stream) {
  const RowPlan p = plan_rows(rows, a.V, sizeof(T), 16, GRAD ? 24 * 1024 : -1);
  const int64_t part = part_of(row_vectors(a.V, sizeof(T)), p.size);
  a.map_words = map_words(part, Vec<T>::N);
  a.flag_words = flag_words(part, p.threads);
  const int beside = Board<2>::bytes(p.size * p.threads / 32) + 4 * (3 * a.k_list + a.map_words + a.flag_words);
  a.cache_at = (beside + 15) / 16;
  a.kept = p.kept;
  const int smem = 16 * (a.cache_at + a.kept);
  return p.threads == 512   ? launch_rows<distill_kernel<T, GRAD, 512>>(p, smem, rows, stream, a)
         : p.threads == 256 ? launch_rows<distill_kernel<T, GRAD, 256>>(p, smem, rows, stream, a)
                            : launch_rows<distill_kernel<T, GRAD, 128>>(p, smem, rows, stream, a);
}

template <typename T>
cudaError_t launch(DistillArgs& a, int rows, cudaStream_t stream) {
  return a.grad ? launch<T, true>(a, rows, stream) : launch<T, false>(a, rows, stream);
}

}  // namespace

}  // namespace tail

using namespace tail;

extern "C" int tail_distill_topk(int32_t rows, int32_t V, int32_t k, const void* logits, int32_t logits_dtype,
                                 int64_t logits_ld, const void* topk_vals, int32_t vals_dtype, int64_t vals_ld,
                                 const int32_t* topk_idx, int64_t idx_ld, double temperature,
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
