// Distillation from a teacher's top logits and its gradient, in one launch that reads the student's logits once.
//
// The teacher's list (and the weight of what lies outside it) gives q; the student's p is over the whole
// vocabulary.  Listed columns are marked in a bit map and left out of the statistics' pass, so that
// the weight of the others is a sum of its own: 1 - sum of the listed p would lose it where the list holds nearly
// everything.  The listed columns' statistics come from the entries.  Outside the list dz_v is a multiple of the
// softmax over the others, p_rest - q_rest times it; the entries' values p_i - q_i are written
// over it afterwards.  Where both p and q are above one half their difference is taken of 1 - q and 1 - p.
//
// Measured (GB300, by graph replay): 8 rows of 201088 in fp32 with 256 entries 10.3 us (floor 1.9: one CTA's chain, in
// it two dependent loads for the list and its logits); 500 rows of 50021 in bf16 with 77 entries and the rest 27.7 (14.3: one
// wave of CTAs, reads, chain and writes one after another, 18 instructions a column); 1024 rows of 201088 in fp32 with 256
// entries 262 (241; 299 with cluster barriers in the exchange and the list's loads one after another, 264 with every warp
// going through the whole list).  The loss alone: 6.3 (1.0), 17.7 (6.8) and 129 (117).
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
  double k64, t64;  // log2(e) / T, T
  int vals_dtype;
  int map_words, flag_words, cache_at, kept;  // cache_at, kept: in vectors
  uint64_t wait_ns;
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
  float inv;               // 1 / (1 + others)
  bool rest_is_max;
  bool any;  // whether there is anything to aim at
};

__device__ __forceinline__ Teacher teacher_of(const RowStat& st, float rest, double k64, double t64) {
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
  if (st.s != st.s) t.q_rest = st.s;  // NaN in the list: no column's share of q is known
  if (rest == -INFINITY) return t;
  t.any = true;
  if (!listed) {  // the list's values are all -inf: everything is outside it
    t.others = 0.f, t.ln = 0.f, t.q_rest = 1.f, t.lq_rest = 0.f, t.q_list = 0.f, t.rest_is_max = true;
    if (rest != rest) t.D = t.q_rest = rest;
    return t;
  }
  // the rest's weight is 2^d: rest - m / T by one rounding, since at a small T both are far larger than their difference
  const float d = static_cast<float>(fma(static_cast<double>(rest), t64, -static_cast<double>(t.m)) * k64);
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

// A CTA's dynamic shared memory: the list's entries in its part, in their order (ids, the teacher's values, the student's
// logits), the bit map of the part's listed columns, and a byte a thread and batch that says which of its
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

// What a List takes at most beside a part that is kept: 12 bytes an entry, and of the at most 12416 vectors that then find
// room a byte each for the map (8 columns of 16 bits) and a quarter for the flags, each rounded up: 28040 bytes.
constexpr int DISTILL_BESIDE = 28 * 1024;
static_assert((ROW_SMEM - DISTILL_BESIDE - 2048) / 16 == 12416 && 12 * DISTILL_MAX_K + 12416 + 12 + 13 * 256 <= DISTILL_BESIDE);

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

// What a set of columns says of a row: statistics of those outside the list and of the listed ones, and, relative to the
// latter's maximum, C = sum q_i (t_i - z_i) / T and Q = sum q_i.
struct Sums {
  RowStat out, in;
  float C, Q;
};
__device__ __forceinline__ void pack(const Sums& s, float4 (&v)[2]) {
  v[0] = make_float4(s.out.m, s.out.s, s.C, s.Q);
  v[1] = make_float4(s.in.m, s.in.s, 0.f, 0.f);
}
__device__ __forceinline__ Sums unpack(const float4& a, const float4& b) {
  return Sums{RowStat{a.x, a.y, 0.f}, RowStat{b.x, b.y, 0.f}, a.z, a.w};
}
// A warp's lanes' together: of the listed columns, and of all.
__device__ __forceinline__ void merge_listed(Sums& s, float k, float inv_t) {
  const RowStat in = warp_merge<false>(s.in, k);
  if (!(s.Q == 0.f)) s.C += s.Q * ((finite_ref(in.m) - finite_ref(s.in.m)) * inv_t);
  s.in = in;
  s.C = warp_sum(s.C);
  s.Q = warp_sum(s.Q);
}
__device__ __forceinline__ Sums merge_sums(Sums s, float k, float inv_t) {
  s.out = warp_merge<false>(s.out, k);
  merge_listed(s, k, inv_t);
  return s;
}

// A row's loss and the factors of its gradient, by one warp.
__device__ __forceinline__ void distill_row(const DistillArgs& a, int64_t r, float w, const Teacher& t, const Sums& x,
                                            int rank, RowGrad* g, EntryGrad* e) {
  const RowStat &o = x.out, &n = x.in;
  const RowStat all = merge(o, n, a.k);
  const bool live = all.m != -INFINITY;  // a distribution
  const float ln = log1pf(all.s), sum = 1.f + all.s, inv = 1.f / sum;
  const float out_w = o.m == -INFINITY ? 0.f : (1.f + o.s) * ex2(dist(o.m, finite_ref(all.m), a.k));
  const float in_w = n.m == -INFINITY ? 0.f : (1.f + n.s) * ex2(dist(n.m, finite_ref(all.m), a.k));
  const float p_rest = out_w * inv;
  if (threadIdx.x != 0) return;
  if (rank == 0) {
    // log q_i - l_i is a difference of two logits and of two log-sums: near one another these give the logarithm of
    // their quotient, which does not leave each one's rounding behind; far below, the quotient less 1 would cancel (to -1,
    // and a loss of -inf, once the rest outweighs the list by 2^25), while the difference is large beside its roundings
    const float scale = 1.f + t.others;
    const float y = (t.D == 0.f ? all.s - t.others : sum * ex2(-t.D) - scale) / scale;
    const float lead = y > -0.5f ? log1pf(y) : ln - t.ln - t.D * 0.693147181f;
    float loss = x.Q == 0.f ? 0.f : lead * x.Q + x.C + x.Q * ((all.m - finite_ref(n.m)) * a.inv_t);
    if (!(t.q_rest == 0.f)) {
      const float lp = out_w >= in_w    ? -log1pf(in_w / out_w)
                       : out_w > 1e-30f ? logf(p_rest)
                                        : (o.m - all.m) * a.inv_t + log1pf(o.s) - ln;
      loss += t.q_rest * (t.lq_rest - (o.m == -INFINITY ? -INFINITY : lp));
    }
    a.loss[r] = live ? w * loss : 0.f;
  }
  const float wt = live ? w * a.inv_t : 0.f;
  const float off = p_rest > 0.5f && t.q_rest > 0.5f ? t.q_list - in_w * inv : p_rest - t.q_rest;
  *g = RowGrad{finite_ref(o.m), a.k, live ? wt * off / (1.f + o.s) : 0.f, 0.f, 0.f, -1};
  *e = EntryGrad{finite_ref(all.m), all.s, wt};
}

template <typename T, bool GRAD, int NT>
__global__ void __launch_bounds__(NT, ROW_SM_THREADS / NT) distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ uint4 smem[];
  __shared__ Board<2> board;
  constexpr int WARPS = NT / 32;
  static_assert(DISTILL_MAX_K / NT * WARPS <= 32, "a lane a round and warp");
  __shared__ RowStat s_warp[WARPS];
  __shared__ int s_count[32];  // entries in the part by round of NT and warp
  __shared__ Teacher s_teacher;
  __shared__ RowGrad s_grad;
  __shared__ EntryGrad s_entry;
  const int size = cluster_size(), rank = cluster_rank(), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  List l;
  l.ids = reinterpret_cast<int32_t*>(smem);
  l.t = reinterpret_cast<float*>(l.ids + a.k_list);
  l.z = l.t + a.k_list;
  l.map = reinterpret_cast<uint32_t*>(l.z + a.k_list);
  l.flags = l.map + a.map_words;
  uint4* cache = smem + a.cache_at;
  const int64_t r = blockIdx.x / size;
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  T* grad = static_cast<T*>(a.grad) + r * a.gld;
  const RowPart p = row_part(row, a.V, rank, size);
  const bool kept = GRAD && a.kept > 0;
  // The part's columns [lo, hi); bit 0 of the map is one vector in front of its first whole one.
  const int body = p.head + p.first * N, origin = body - N;
  const int lo = rank == 0 ? 0 : body, hi = rank == size - 1 ? a.V : body + p.count * N;
  const auto in_part = [&](int id) { return id >= lo && id < hi; };
  if (size > 1) board.init();
  for (int i = tid; i < a.map_words + a.flag_words; i += NT) l.map[i] = 0;  // (the flags lie behind the map)
  pdl_wait();

  // The list: a thread's first entry and the logit at it are under way while the part is requested, which waits for
  // the row's first id at most.
  const float w = a.weight ? a.weight[r] : 1.f;
  const int head_id = a.idx[r * a.ild];
  const float rest = a.rest && tid == 0 ? a.rest[r] : -INFINITY;  // the first thread's
  const bool listed = tid < a.k_list;
  int id0 = listed ? a.idx[r * a.ild + tid] : -1;
  const float v0 = listed ? list_value(a, r, tid) : 0.f;
  const bool early = w != 0.f && static_cast<uint32_t>(head_id) < static_cast<uint32_t>(a.V);
  if (kept)
    fetch_part<T, NT>(row, p, cache);
  else if (early)
    prefetch_part(row, p, 0);
  if (static_cast<uint32_t>(id0) >= static_cast<uint32_t>(a.V)) id0 = -1;
  const bool mine0 = in_part(id0);
  const float z0 = mine0 ? Vec<T>::widen1(row[id0]) : 0.f;
  bool any = id0 >= 0;
  RowStat st = stat_of(any ? v0 : -INFINITY);
  const int rounds = (a.k_list + NT - 1) / NT;
  const auto count = [&](int j, bool mine) {
    const uint32_t at = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) s_count[j * WARPS + warp] = __popc(at);
  };
  count(0, mine0);
  for (int j = 1; j < rounds; ++j) {
    const int i = j * NT + tid;
    const int id = i < a.k_list ? a.idx[r * a.ild + i] : -1;
    const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.V);
    any = any || ok;
    if (ok) st = merge(st, stat_of(list_value(a, r, i)), a.k);
    count(j, ok && in_part(id));
  }
  if (warp * 32 < a.k_list) st = warp_merge<false>(st, a.k);
  if (lane == 0) s_warp[warp] = st;
  if (!__syncthreads_or(any && w != 0.f)) {
    if (kept) copy_wait(0);
    if (rank == 0 && tid == 0) a.loss[r] = 0.f;
    if (GRAD) zero_part(grad, a.V, rank, size);
    return;
  }
  if (size > 1) cluster_started();
  if (!kept && !early) prefetch_part(row, p, 0);
  // The entries of this part, in the list's order: their bits, and whether an id comes twice.
  const int counted = lane < rounds * WARPS ? s_count[lane] : 0, n = __reduce_add_sync(0xffffffffu, counted);
  bool twice = false;
  const auto enter = [&](int j, bool mine, int id, float v, float z) {
    const uint32_t others = __ballot_sync(0xffffffffu, mine);
    const int before = __reduce_add_sync(0xffffffffu, lane < j * WARPS + warp ? counted : 0);
    if (!mine) return;
    const int e = before + __popc(others & lanemask_lt()), at = id - origin, c = at / N - 1;
    l.ids[e] = id;
    l.t[e] = v;
    l.z[e] = z;
    const uint32_t bit = 1u << (at & 31);
    twice = (atomicOr(l.map + (at >> 5), bit) & bit) || twice;
    if (c >= 0 && c < p.count) {
      const int f = c / (ROW_BATCH * NT) * NT + c % NT;  // its thread's byte of its batch
      atomicOr(l.flags + (f >> 2), 1u << (c / NT % ROW_BATCH + 8 * (f & 3)));
    }
  };
  if (warp * 32 < a.k_list) enter(0, mine0, id0, v0, z0);
  for (int j = 1; j < rounds; ++j) {
    const int i = j * NT + tid;
    const int id = i < a.k_list ? a.idx[r * a.ild + i] : -1;
    const bool mine = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.V) && in_part(id);
    enter(j, mine, id, mine ? list_value(a, r, i) : 0.f, mine ? Vec<T>::widen1(row[id]) : 0.f);
  }
  Batch v;
  if (!kept) v = Batch::from<NT>(part_vectors(row, p), 0, p.count);
  const float edge = edge_of(row, p);
  if (size > 1) cluster_wait();
  if (tid < 32) {
    st = tid < WARPS ? s_warp[tid] : no_stat();
    st = warp_merge<false>(st, a.k);
    if (tid == 0) {
      Teacher t = teacher_of(st, rest, a.k64, a.t64);
      t.inv = 1.f / (1.f + t.others);
      s_teacher = t;
    }
  }
  twice = __syncthreads_or(twice);
  const Teacher& t = s_teacher;
  if (!t.any) {  // the values and the rest are all -inf: whatever the logits hold
    if (kept) copy_wait(0);
    if (rank == 0 && tid == 0) a.loss[r] = 0.f;
    if (GRAD) zero_part(grad, a.V, rank, size);
    return;
  }
  const auto weight = [&](int e) { return ex2((l.t[e] - t.m) * a.k - t.D) * t.inv; };
  const auto owner = [&](int e) {  // the first of an id's entries stands for its column
    if (twice)
      for (int f = 0; f < e; ++f)
        if (l.ids[f] == l.ids[e]) return false;
    return true;
  };

  Sums x;
  x.out = stat_pass<T, false, NT>(row, p, kept ? cache : nullptr, v, a.k,
                                  ListMask<N, NT>{l.map, reinterpret_cast<const uint8_t*>(l.flags)});
  if (p.edge_n && !(l.map[(p.edge_lo - origin) >> 5] >> ((p.edge_lo - origin) & 31) & 1))
    x.out = merge(x.out, stat_of(edge), a.k);
  if (GRAD && !kept) v = Batch::from<NT>(part_vectors(row, p), 0, p.count);  // for the second pass, while the factors are formed
  x.out = warp_merge<false>(x.out, a.k);
  x.in = no_stat();
  x.C = x.Q = 0.f;
  if (warp * 32 < n) {
    for (int e = tid; e < n; e += NT)
      if (owner(e)) x.in = merge(x.in, stat_of(l.z[e]), a.k);
    for (int e = tid; e < n; e += NT) {
      const float q = weight(e);
      if (q == 0.f) continue;
      x.C += q * (((l.t[e] - t.m) - (l.z[e] - finite_ref(x.in.m))) * a.inv_t);
      x.Q += q;
    }
    merge_listed(x, a.k, a.inv_t);
  }
  float4 mine[2], all[2];
  pack(x, mine);
  if (lane == 0) board.warp[0][warp] = mine[0], board.warp[1][warp] = mine[1];
  __syncthreads();
  if (tid < 32) {  // one warp forms the row's loss and factors for all
    x = tid < WARPS ? unpack(board.warp[0][tid], board.warp[1][tid]) : Sums{no_stat(), no_stat(), 0.f, 0.f};
    x = merge_sums(x, a.k, a.inv_t);
    if (size > 1) {
      pack(x, mine);
      const bool ok = board.template exchange<true>(rank, size, mine, all, a.wait_ns);
      x = merge_sums(unpack(all[0], tid < size ? all[1] : make_float4(-INFINITY, 0.f, 0.f, 0.f)), a.k, a.inv_t);
      if (!ok) {
        x.out.m = NAN;
        if (!GRAD) board.leave();  // (the other warps are done)
      }
    }
    distill_row(a, r, w, t, x, rank, &s_grad, &s_entry);
  }
  if (!GRAD) return;
  __syncthreads();
  grad_pass<T, false, NT>(s_grad, GradRow<T>{row, grad, p, kept ? cache : nullptr, edge}, v);
  __syncthreads();  // the entries' values go over what the pass has written
  const EntryGrad e = s_entry;
  for (int i = tid; i < n; i += NT) {
    if (!owner(i)) continue;
    float q = weight(i), q_left = q > 0.5f && !t.rest_is_max ? t.others * t.inv : 1.f - q;  // above one half: the largest
    if (twice)
      for (int j = i + 1; j < n; ++j)
        if (l.ids[j] == l.ids[i]) q += weight(j), q_left = 1.f - q;
    const float x = ex2((l.z[i] - e.m) * a.k), sum = 1.f + e.s, pv = x / sum;
    const float p_left = (l.z[i] == e.m ? e.s : sum - x) / sum;
    grad[l.ids[i]] = Vec<T>::narrow1(e.wt == 0.f ? 0.f : e.wt * (pv > 0.5f && q > 0.5f ? q_left - p_left : pv - q));
  }
  if (tid < 32 && s_grad.ref != s_grad.ref) board.leave();  // its wait may have run out
}

template <typename T, bool GRAD>
cudaError_t launch(DistillArgs& a, int rows, cudaStream_t stream) {
  const RowPlan p = plan_rows(rows, a.V, sizeof(T), 16, GRAD ? DISTILL_BESIDE : -1);
  const int64_t part = part_of(row_vectors(a.V, sizeof(T)), p.size);
  a.map_words = map_words(part, Vec<T>::N);
  a.flag_words = flag_words(part, p.threads);
  const int beside = 4 * (3 * a.k_list + a.map_words + a.flag_words);
  a.cache_at = (beside + 15) / 16;
  a.kept = p.kept;
  const int smem = 16 * (a.cache_at + a.kept);
  return p.threads == 256 ? launch_rows<distill_kernel<T, GRAD, 256>>(p, smem, rows, stream, a)
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
  a.t64 = temperature;
  a.k64 = LOG2E / temperature;
  a.k = static_cast<float>(a.k64);
  a.inv_t = static_cast<float>(1.0 / temperature);
  a.wait_ns = row_wait_limit();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == TAIL_F32   ? launch<float>(a, rows, s)
                        : logits_dtype == TAIL_F16 ? launch<__half>(a, rows, s)
                                                   : launch<__nv_bfloat16>(a, rows, s);
  return e == cudaSuccess ? TAIL_OK : cuda_fail(e, "tail_distill_topk: kernel launch");
}
