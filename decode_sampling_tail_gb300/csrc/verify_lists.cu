// Verification of drafted tokens against the tail's own distribution: the
// sampler's (top_k, top_p, temperature; sampler.cuh) over the row's sorted
// top-k.  A sequence's rows are the positions of its d drafts and one more; row
// j's target P_j is compared with the draft distribution q_j (speculative
// sampling):
//   draft x_j is accepted iff a_j q_j(x_j) < P_j(x_j) and every earlier one was;
//   at the first refused row the token is drawn from max(P_j - q_j, 0) (from P_j
//   when that is zero everywhere), after d accepted drafts from P_d, each by
//   inverse transform with the row's u over the candidates in list order.
// The tokens so emitted are distributed as the tail's own draws.
//
// P is zero outside the list, so q is read at the draft and, at the refused row
// alone, at the list's ids; no pass over the vocabulary is needed.  Weights are
// the integers of fixed_exp.cuh in units of 2^-52 (at most 1024 of at most 1:
// below 2^63), so decisions match 64-bit arithmetic.
//
// One CTA a sequence, one warp a row; every warp settles its row whole, drawing
// before it knows whether earlier drafts held: what bounds the kernel is one
// row's chain of loads, exponentials, scans and gathers, and rows in parallel
// cost no more than one.  Measured by graph replay: one sequence of 4 rows, k = 256:
// 6.2 us; 64 sequences of 6 rows 8.4 us (called from Python one by one, 10.7 and
// 12.3 to 15.7: the host's part); 200 of 1 to 10 rows, k = 1000: 24.4 us either way
// (a chain four times as long: a lane owns 32 candidates instead of 8; 9 MB of lists,
// DRAM 7 MB, issue slots 7 % busy).
#include "../../include/tail.h"
#include "abi_common.h"
#include "internal.h"
#include "sampler.cuh"
#include "verify.cuh"

namespace tail {

namespace {

struct VerifyArgs {
  const float* vals;    // [rows][k] descending
  const int32_t* idx;   // [rows][k]
  const float* params;  // [rows][ncols]
  const int32_t* cu;    // [nseq + 1]
  const int32_t* drafts;
  const float* accept;
  DraftProbs q;
  int32_t* tokens;
  int32_t* count;
  int rows, k, ncols;
};

// A warp's weights w[0, n) in shared memory with their chunk sums: lane l owns [l * E, (l + 1) * E).
struct Chunks {
  const int64_t* w;
  int n, E;
  int64_t incl;  // sum through this lane's chunk
  int64_t total;
};

__device__ __forceinline__ Chunks sum_chunks(const int64_t* w, int n) {
  Chunks c;
  const int lane = threadIdx.x & 31;
  c.w = w;
  c.n = n;
  c.E = (n + 31) >> 5;
  int64_t s = 0;
  int r = lane % c.E;  // lanes start apart: chunks lie E * 8 bytes apart and would share banks
  for (int t = 0; t < c.E; ++t) {
    const int i = lane * c.E + r;
    if (i < n) s += w[i];
    if (++r == c.E) r = 0;
  }
  c.incl = warp_scan(s);
  c.total = __shfl_sync(0xffffffffu, c.incl, 31);
  return c;
}

// The smallest i whose running sum S_i exceeds t; n when there is none.  *sum receives S_i.
__device__ __forceinline__ int first_above(const Chunks& c, int64_t t, int64_t* sum) {
  const int lane = threadIdx.x & 31;
  const uint32_t who = __ballot_sync(0xffffffffu, c.incl > t);
  if (who == 0u) return c.n;
  const int src = __ffs(who) - 1;
  const int64_t upto = __shfl_sync(0xffffffffu, c.incl, src > 0 ? src - 1 : 0);
  const int i = src * c.E + lane;
  const bool mine = lane < c.E && i < c.n;
  const int64_t S = (src > 0 ? upto : 0) + warp_scan(mine ? c.w[i] : 0);
  const uint32_t in = __ballot_sync(0xffffffffu, mine && S > t);
  if (in == 0u) return c.n;  // not reached: the chunk's last sum is the one that was found
  *sum = __shfl_sync(0xffffffffu, S, __ffs(in) - 1);
  return src * c.E + __ffs(in) - 1;
}

// The draw: the smallest i with weight and u * total < S_i; past the end (u >= 1) the last with weight.
__device__ __forceinline__ int draw(const Chunks& c, float u) {
  int64_t s;
  const int i = first_above(c, draw_threshold(u, c.total), &s);
  if (i < c.n && c.w[i] > 0) return i;
  const bool past = i >= c.n;  // else u < 0, before the first weight
  int v = past ? -1 : 0x7fffffff;
  for (int j = threadIdx.x & 31; j < c.n; j += 32)
    if (c.w[j] > 0) v = past ? max(v, j) : min(v, j);
  v = past ? __reduce_max_sync(0xffffffffu, v) : __reduce_min_sync(0xffffffffu, v);
  return v >= 0 && v < c.n ? v : -1;
}

constexpr int BATCH = 8;  // candidates whose loads a lane has under way together

__global__ void __launch_bounds__(VERIFY_THREADS) verify_lists_kernel(const VerifyArgs a) {
  extern __shared__ __align__(16) int64_t s_w[];  // [VERIFY_WARPS][k]
  __shared__ float2 s_table[EXP_TABLE];
  __shared__ int s_ok[VERIFY_WARPS];
  __shared__ int32_t s_token[VERIFY_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < EXP_TABLE) s_table[tid] = EXP2_TABLE[tid];
  pdl_wait();
  int lo, hi;
  sequence_rows(a.cu, blockIdx.x, a.rows, lo, hi);
  int64_t* w = s_w + static_cast<int64_t>(warp) * a.k;
  int sel = hi;
  for (int j0 = lo; j0 < hi; j0 += VERIFY_WARPS) {
    __syncthreads();
    const int row = j0 + warp;
    if (row < hi) {
      const float* vals = a.vals + static_cast<int64_t>(row) * a.k;
      const int32_t* idx = a.idx + static_cast<int64_t>(row) * a.k;
      const SampleParams p = load_sample_params(a.params + static_cast<int64_t>(row) * a.ncols, a.ncols);
      const bool bonus = row == hi - 1;
      const int x = bonus ? -1 : a.drafts[row];
      const float u_a = bonus ? 0.f : a.accept[row];
      const float qx = bonus ? 0.f : a.q.p ? draft_prob(a.q, row, x) : 1.f;
      const float l0 = vals[0];
      const int k = a.k;
      const int kk = (p.top_k >= 1.0f && p.top_k < static_cast<float>(k) + 1.0f) ? static_cast<int>(p.top_k) : k;
      bool ok = false;
      int pick = -1;
      if (l0 == -INFINITY) {
        // nothing is left to draw from
      } else if (!(p.temp > 0.0f) || kk == 1) {  // greedy: P is 1 at the first candidate
        pick = 0;
        ok = !bonus && x == idx[0] && static_cast<double>(u_a) * qx < 1.0;
      } else {
        const ExpScale c = exp_scale(p.temp);
        int64_t ex = 0;
        int at = k;
        auto weigh = [&] {
          for (int i0 = lane; i0 < kk; i0 += 32 * BATCH) {
            float v[BATCH];
            int32_t id[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
              const int i = i0 + 32 * b;
              v[b] = i < kk ? __ldg(vals + i) : 0.f;
              id[b] = i < kk ? __ldg(idx + i) : 0;
            }
#pragma unroll 2
            for (int b = 0; b < BATCH; ++b) {
              const int i = i0 + 32 * b;
              if (i < kk) {
                const int64_t e = exp_fixed(v[b], l0, c, s_table, 52);
                w[i] = e;
                if (id[b] == x && !bonus) {
                  at = i;
                  ex = e;
                }
              }
            }
          }
          __syncwarp();
        };
        weigh();
        Chunks ch = sum_chunks(w, kk);
        int m = kk;
        if (p.top_p < 1.0f) {  // the first candidate whose sum reaches top_p of all
          int64_t cm;
          const double cut = static_cast<double>(p.top_p) * static_cast<double>(ch.total);
          const int i = first_above(ch, __double2ll_ru(cut) - 1, &cm);
          if (i < kk) m = i + 1;
          if (m < kk) ch = sum_chunks(w, m);  // the kept prefix alone
        }
        if (!bonus && ch.total > 0) {
          const double t = static_cast<double>(u_a) * qx * static_cast<double>(ch.total);
          ok = __any_sync(0xffffffffu, at < m && t < static_cast<double>(ex));
        }
        if (!ok && !bonus && ch.total > 0) {  // the residual max(P - q, 0), in the same units
          const int64_t total = ch.total;
          __syncwarp();  // the list's weights have been read
          for (int i0 = lane; i0 < m; i0 += 32 * BATCH) {
            float q[BATCH];
            int32_t id[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) id[b] = i0 + 32 * b < m ? __ldg(idx + i0 + 32 * b) : -1;
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
              q[b] = a.q.p ? draft_prob(a.q, row, id[b]) : (id[b] == x ? 1.f : 0.f);
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
              const int i = i0 + 32 * b;
              if (i < m) {
                const int64_t r = w[i] - prod_fixed(q[b], total);
                w[i] = r > 0 ? r : 0;
              }
            }
          }
          __syncwarp();
          ch = sum_chunks(w, m);
          if (ch.total == 0) {  // q covers P: the draw is from P itself
            weigh();
            ch = sum_chunks(w, m);
          }
        }
        if (!ok && ch.total > 0) pick = draw(ch, p.u);
      }
      if (lane == 0) {
        s_ok[warp] = ok;
        s_token[warp] = pick >= 0 ? idx[pick] : -1;
      }
    }
    __syncthreads();
    const int n = min(VERIFY_WARPS, hi - j0);
    int f = 0;
    while (f < n && s_ok[f]) ++f;
    if (f < n) {
      sel = j0 + f;
      if (tid == 0) a.tokens[sel] = s_token[f];
      break;
    }
  }
  write_sequence(lo, hi, sel, a.drafts, a.tokens, a.count + blockIdx.x);
}

}  // namespace

}  // namespace tail

using namespace tail;

extern "C" int tail_verify(int32_t rows, int32_t nseq, int32_t k, const float* topk_vals, const int32_t* topk_idx,
                           const float* params, int32_t n_param_cols, const int32_t* cu_rows, const int32_t* drafts,
                           const float* u_accept, const void* draft_probs_opt, int32_t draft_dtype,
                           int64_t draft_ld, int32_t V, int32_t* out_tokens, int32_t* out_count, void* stream) {
  if (rows < 0 || nseq < 0 || k < 1 || k > MAX_K) return TAIL_ERR_INVALID_ARG;
  if (n_param_cols != 3 && n_param_cols != 4) return TAIL_ERR_INVALID_ARG;
  if (nseq == 0) return TAIL_OK;
  if (!cu_rows || !out_count || !aligned(cu_rows, 4) || !aligned(out_count, 4)) return TAIL_ERR_INVALID_ARG;
  if (rows > 0) {
    if (!topk_vals || !topk_idx || !params || !drafts || !u_accept || !out_tokens) return TAIL_ERR_INVALID_ARG;
    if (!aligned(topk_vals, 4) || !aligned(topk_idx, 4) || !aligned(params, 4) || !aligned(drafts, 4) ||
        !aligned(u_accept, 4) || !aligned(out_tokens, 4))
      return TAIL_ERR_INVALID_ARG;
    const int64_t n = rows;
    const struct {
      const void* p;
      int64_t words;
    } in[] = {{cu_rows, nseq + 1LL}, {drafts, n}, {u_accept, n}, {topk_vals, n * k}, {topk_idx, n * k},
              {params, n * n_param_cols}};
    for (const auto& i : in)
      if (meets(out_tokens, n, i.p, i.words) || meets(out_count, nseq, i.p, i.words)) return TAIL_ERR_INVALID_ARG;
    if (meets(out_tokens, n, out_count, nseq)) return TAIL_ERR_INVALID_ARG;
  }
  if (draft_probs_opt) {
    if (draft_dtype < TAIL_F32 || draft_dtype > TAIL_BF16 || V < 1 || draft_ld < V) return TAIL_ERR_INVALID_ARG;
    if (!aligned(draft_probs_opt, elem_bytes(draft_dtype))) return TAIL_ERR_INVALID_ARG;
  }
  VerifyArgs a;
  a.vals = topk_vals;
  a.idx = topk_idx;
  a.params = params;
  a.cu = cu_rows;
  a.drafts = drafts;
  a.accept = u_accept;
  a.q = DraftProbs{draft_probs_opt, draft_dtype, draft_ld, V};
  a.tokens = out_tokens;
  a.count = out_count;
  a.rows = rows;
  a.k = k;
  a.ncols = n_param_cols;
  const int smem = VERIFY_WARPS * k * static_cast<int>(sizeof(int64_t));
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024)  // above the default limit with the static part; idempotent, per device
    e = cudaFuncSetAttribute(verify_lists_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             VERIFY_WARPS * MAX_K * static_cast<int>(sizeof(int64_t)));
  if (e != cudaSuccess) return cuda_fail(e, "tail_verify: shared memory opt-in");
  e = launch_overlapped(verify_lists_kernel, dim3(nseq), smem, static_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return cuda_fail(e, "tail_verify: kernel launch");
  return TAIL_OK;
}
