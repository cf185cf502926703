// Verification of drafted tokens against whole-vocabulary distributions: the
// rule of verify_lists.cu with P_j = softmax(l_j / T_j) over all V logits (the
// lowest index of the maximum when T <= 0).
//
// Three kernels, over chunks of 8192 columns, which a CTA holds in registers, or parts of them:
//   verify_stats (chunk, row): the chunk's maximum m_c, its lowest column and sum exp((l - m_c) / T)
//     in fp32.  Every row has to be read, since which one is settled is not known yet; this pass is
//     bound by memory and only has to decide acceptances.  Z is off by at most a relative 2^-17: 2^-23 for
//     every binary order that a term lies below the maximum, in the terms' mean (their share times their orders sums
//     to log2 V at most: 2^-18.6), and up to 46 additions of 2^-24; 2^-21 is usual.
//   verify_settle (part, sequence): each CTA judges the sequence's rows from those statistics (all
//     of them compute the same bits, none waits) and finds the settled row; then the sums of that row's
//     segments (1024 columns) as integers (fixed_exp.cuh, units of 2^-49 relative to m_c).
//   verify_draw (part, sequence): after d accepted drafts, or with one-hot drafts (P without x_j), the
//     segments' sums already say which one holds the token; one CTA reads its columns again.  The
//     residual max(P - q, 0) needs one pass over that row's l and q: every CTA sums its segments,
//     the last of the sequence to finish (a counter that verify_settle cleared) picks one and the token.
// Sums over segments are integers of 2^-shift relative to the row's maximum, with V 2^shift below 2^62;
// the residual is max(e - q Z, 0) in the same units.  The draft's row is read only for sequences that
// refuse a draft.
//
// Measured at V = 201088: 96 sequences (384 fp32 rows, and fp32 draft rows where one is refused) 164-167 us back to back, of
// them stats 53-59 us (309 MB: 5.3-5.8 TB/s, 0.8-0.87 of the copy rate), settle 46 and draw 65: both form
// 19 million exponentials to 2^-36, 55 to 75 instructions each, on 66 % of the issue slots; 16 sequences 42 us;
// one sequence of 5 rows 10.7 us by graph replay, the latency of three launches (17-20 called from Python one by
// one: the host's part).
#include "../../include/tail.h"
#include "abi_common.h"
#include "verify.cuh"

namespace tail {

namespace {

constexpr int VL_GROUPS = 8;                                  // groups of 4 columns a thread holds
constexpr int VL_WARP_COLS = 128 * VL_GROUPS;                 // a warp's columns, contiguous
constexpr int VL_CHUNK = VL_WARP_COLS * VERIFY_WARPS;         // 8192
constexpr int VL_SHIFT = 49;
constexpr int VL_MAX_V = 1 << 20;
constexpr int VL_MAX_CHUNKS = (VL_MAX_V + 3) / VL_CHUNK + 1;
constexpr int VL_MAX_SEGS = VL_MAX_CHUNKS * VERIFY_WARPS;
constexpr int VL_MAX_ROWS = 65535;                            // a grid dimension

struct ChunkStat {
  float max;
  float sum;    // of exp((l - max) / T); 0 for greedy rows
  int32_t arg;  // lowest column of the maximum
  int32_t pad;
};

// What a sequence's settled row is, from verify_settle to verify_draw.
struct Settled {
  int32_t row;
  float max;
  int32_t token;    // >= -1: known without a draw (greedy, or nothing to draw from); -2: to be drawn
  int32_t refused;
};

struct LogitsArgs {
  const void* logits;
  int64_t ld;
  const float* temp;
  const int32_t* cu;
  const int32_t* drafts;
  const float* accept;
  const float* u;
  DraftProbs q;
  ChunkStat* stats;    // [rows][nchunk]
  int64_t* sums;       // [nseq][nseg] the settled row's segment sums, units of 2^-49 relative to m_c
  int64_t* rsum;       // [nseq][nseg] its residual sums
  Settled* settled;    // [nseq]
  uint32_t* done;      // [nseq] CTAs whose residual sum is written
  int32_t* tokens;
  int32_t* count;
  int rows, nseq, V, nchunk;
  int shift;
};

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ void unpack4(const float* p, float (&v)[4]) {
  const float4 t = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
}
__device__ __forceinline__ void unpack4(const __half* p, float (&v)[4]) {
  const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
  const float2 a = __half22float2(reinterpret_cast<const __half2&>(t.x));
  const float2 b = __half22float2(reinterpret_cast<const __half2&>(t.y));
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
__device__ __forceinline__ void unpack4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
  v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xffff0000u);
  v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xffff0000u);
}

// A thread's groups of 4 columns of a row, at col0 + 128 i; `fill` outside [0, V).  All vector loads are
// under way together; a group across a row's end takes single loads, and so do rows that do not lie on
// whole vectors (draft probabilities whose rows start elsewhere than the logits').
template <typename T, int N>
__device__ __forceinline__ void load_groups(const T* row, int col0, int V, float fill, float (&v)[N][4]) {
  const bool whole = (reinterpret_cast<uintptr_t>(row + col0) & (4 * sizeof(T) - 1)) == 0;
  bool rest = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int col = col0 + i * 128;
    const bool inside = col >= 0 && col + 4 <= V;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] = fill;
    if (whole && inside) unpack4(row + col, v[i]);
    rest = rest || (inside ? !whole : col + 4 > 0 && col < V);
  }
  if (!rest) return;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = col0 + i * 128;
      const bool done = whole && col >= 0 && col + 4 <= V;
      if (!done && col + e >= 0 && col + e < V) v[i][e] = widen<T>(row[col + e]);
    }
}

// First column of chunk c: chunks start `off` columns early so that groups of 4 lie on whole
// vectors when a row starts inside one (an odd leading dimension).
template <typename T>
__device__ __forceinline__ int chunk_col(const T* row, int c) {
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 3);
  return c * VL_CHUNK - off;
}

// The first of a thread's columns of part p of 1 / P of a chunk, p counted over the row; it has VL_GROUPS / P
// groups of them.  A part is 8 / P segments, with P warps on each.
template <int P, typename T>
__device__ __forceinline__ int first_col(const T* row, int p) {
  const int warp = threadIdx.x >> 5;
  return chunk_col(row, p / P) + (p % P * (VERIFY_WARPS / P) + warp / P) * VL_WARP_COLS +
         warp % P * (VL_WARP_COLS / P) + (threadIdx.x & 31) * 4;
}

// The sums of part p's segments, from its warps'; the whole CTA.
template <int P>
__device__ __forceinline__ void store_segments(int64_t sum, int64_t* out, int p, int64_t* s_sum) {
  const int tid = threadIdx.x;
  if ((tid & 31) == 0) s_sum[tid >> 5] = sum;
  __syncthreads();
  if (tid < VERIFY_WARPS / P) {
    int64_t s = 0;
#pragma unroll
    for (int k = 0; k < P; ++k) s += s_sum[tid * P + k];
    __stcg(reinterpret_cast<long long*>(out) + p * (VERIFY_WARPS / P) + tid, static_cast<long long>(s));
  }
}

// A part's values in shared memory, each read back by the thread that wrote it: the weights' loops stay
// rolled (code that runs once is bound by fetching it).
template <int P>
struct PartVals {
  float4 l[VL_GROUPS / P][VERIFY_THREADS];
};

template <int P, typename T>
__device__ __forceinline__ void stage_part(const T* row, int p, int V, PartVals<P>& s) {
  float v[VL_GROUPS / P][4];
  load_groups(row, first_col<P>(row, p), V, -INFINITY, v);
#pragma unroll
  for (int i = 0; i < VL_GROUPS / P; ++i) s.l[i][threadIdx.x] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
}

template <typename T>
__global__ void __launch_bounds__(VERIFY_THREADS) verify_stats_kernel(const LogitsArgs a) {
  __shared__ float s_max[VERIFY_WARPS];
  __shared__ float s_sum[VERIFY_WARPS];
  __shared__ int s_arg[VERIFY_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x, row = blockIdx.y;
  pdl_wait();
  if (row >= __ldg(a.cu + a.nseq)) return;  // behind the last sequence
  const T* lrow = static_cast<const T*>(a.logits) + row * a.ld;
  const float temp = __ldg(a.temp + row);
  const int col0 = first_col<1>(lrow, c);
  float v[VL_GROUPS][4];
  load_groups(lrow, col0, a.V, -INFINITY, v);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VL_GROUPS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, v[i][e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // each warp relative to its own maximum: no barrier between the loads and the exponentials
  const bool greedy = !(temp > 0.0f);
  const float scale = greedy ? 0.f : exp_scale(temp).h;
  float sum = 0.f;
  int arg = a.V;
  if (greedy) {
#pragma unroll
    for (int i = VL_GROUPS - 1; i >= 0; --i)
#pragma unroll
      for (int e = 3; e >= 0; --e)
        if (v[i][e] == m && col0 + i * 128 + e >= 0) arg = col0 + i * 128 + e;
    arg = __reduce_min_sync(0xffffffffu, arg);
  } else if (m != -INFINITY) {
#pragma unroll
    for (int i = 0; i < VL_GROUPS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += exp_fast(v[i][e], m, scale);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  if (lane == 0) {
    s_max[warp] = m;
    s_sum[warp] = sum;
    s_arg[warp] = arg;
  }
  __syncthreads();
  if (warp == 0) {
    const float mw = lane < VERIFY_WARPS ? s_max[lane] : -INFINITY;
    float top = mw;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float z = mw > -INFINITY && !greedy ? s_sum[lane] * exp_fast(mw, top, scale) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const int at = __reduce_min_sync(0xffffffffu, lane < VERIFY_WARPS && mw == top ? s_arg[lane] : a.V);
    if (lane == 0) a.stats[static_cast<int64_t>(row) * a.nchunk + c] = ChunkStat{top, z, at, 0};
  }
}

// One warp: whether the row's draft is accepted, and what its token is if it is settled here.  The draft's own
// weight is formed by exp_single: exp_fast would be off by 2^-23 for every binary order it lies below the maximum.
template <typename T>
__device__ __forceinline__ bool judge_row(const LogitsArgs& a, int row, bool bonus, Settled& s) {
  const int lane = threadIdx.x & 31;
  const ChunkStat* st = a.stats + static_cast<int64_t>(row) * a.nchunk;
  const float temp = __ldg(a.temp + row);
  const bool greedy = !(temp > 0.0f);
  const int x = bonus ? -1 : __ldg(a.drafts + row);
  const bool known = x >= 0 && x < a.V;
  const float u_a = bonus ? 0.f : __ldg(a.accept + row);
  const float qx = !known ? 0.f : a.q.p ? draft_prob(a.q, row, x) : 1.f;
  const float lx = known ? widen<T>(static_cast<const T*>(a.logits)[row * a.ld + x]) : -INFINITY;
  constexpr int PER = (VL_MAX_CHUNKS + 31) / 32;
  float cm[PER], cz[PER];
  int ca[PER];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = lane + 32 * i;
    cm[i] = -INFINITY, cz[i] = 0.f, ca[i] = a.V;
    if (c < a.nchunk) {
      const ChunkStat t = st[c];
      cm[i] = t.max, cz[i] = t.sum, ca[i] = t.arg;
    }
    m = fmaxf(m, cm[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  s.row = row;
  s.max = m;
  s.token = -2;
  float ex = 0.f, z = 1.f;
  if (m == -INFINITY) {
    s.token = -1;
  } else if (greedy) {
    int arg = a.V;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (cm[i] == m) arg = min(arg, ca[i]);
    arg = __reduce_min_sync(0xffffffffu, arg);
    s.token = arg < a.V ? arg : -1;
    ex = known && x == arg ? 1.f : 0.f;
  } else {
    const ExpScale sc = exp_scale(temp);
    z = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) z = fmaf(cz[i], exp_fast(cm[i], m, sc.h), z);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (known) ex = exp_single(lx, m, sc);
    if (!(z > 0.f)) s.token = -1;
  }
  const bool ok = !bonus && u_a * qx * z < ex;
  s.refused = !bonus && !ok;
  return ok;
}

template <typename T, int P>
__global__ void __launch_bounds__(VERIFY_THREADS) verify_settle_kernel(const LogitsArgs a) {
  __shared__ float2 s_table[EXP_TABLE];
  __shared__ Settled s_row[VERIFY_WARPS];
  __shared__ PartVals<P> s_vals;
  __shared__ int64_t s_sum[VERIFY_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seq = blockIdx.y, part = blockIdx.x;
  if (tid < EXP_TABLE) s_table[tid] = EXP2_TABLE[tid];
  __syncthreads();
  pdl_wait();
  int lo, hi;
  sequence_rows(a.cu, seq, a.rows, lo, hi);
  Settled st = {hi, 0.f, -1, 0};
  for (int j0 = lo; j0 < hi; j0 += VERIFY_WARPS) {
    if (j0 + warp < hi) {
      Settled s;
      const bool ok = judge_row<T>(a, j0 + warp, j0 + warp == hi - 1, s);
      if (lane == 0) {
        if (ok) s.row = hi;  // goes on
        s_row[warp] = s;
      }
    }
    __syncthreads();
    const int n = min(VERIFY_WARPS, hi - j0);
    int f = 0;
    while (f < n && s_row[f].row == hi) ++f;
    if (f < n) {
      st = s_row[f];
      break;
    }
    __syncthreads();
  }
  if (part == 0) {
    write_sequence(lo, hi, st.row, a.drafts, a.tokens, a.count + seq);
    if (tid == 0) {
      a.settled[seq] = st;
      a.done[seq] = 0u;
      if (hi > lo && st.token > -2) a.tokens[st.row] = st.token;
    }
  }
  if (st.token > -2) return;
  const float m = a.stats[static_cast<int64_t>(st.row) * a.nchunk + part / P].max;
  int64_t sum = 0;
  if (m != -INFINITY) {
    stage_part<P>(static_cast<const T*>(a.logits) + st.row * a.ld, part, a.V, s_vals);
    const ExpScale sc = exp_scale(__ldg(a.temp + st.row));
#pragma unroll 1
    for (int i = 0; i < VL_GROUPS / P; ++i) {
      const float4 v = s_vals.l[i][tid];
      int64_t r[4];
      exp_fixed4(v, m, sc, s_table, VL_SHIFT, r);
      sum += (r[0] + r[1]) + (r[2] + r[3]);
    }
    sum = warp_sum(sum);
  }
  store_segments<P>(sum, a.sums + static_cast<int64_t>(seq) * a.nchunk * VERIFY_WARPS, part, s_sum);
}

enum DrawMode : int {
  DRAW_P = 0,         // from P
  DRAW_OTHERS = 1,    // from P without the draft (the residual of a one-hot draft)
  DRAW_RESIDUAL = 2,  // from max(P - q, 0)
};

// The weight of one column as an integer: exp in units of 2^-49 relative to the chunk's maximum
// (DRAW_P, DRAW_OTHERS), or the residual in units of 2^-shift relative to the row's.
struct Weigh {
  int mode, x, shift;
  float max;
  int64_t z;  // the row's Z in units of 2^-shift
  ExpScale sc;
};

// Weights of columns col .. col + 3.
__device__ __forceinline__ void weigh4(float4 l, float4 q, int col, const Weigh& g, const float2* table,
                                       int64_t (&w)[4]) {
  exp_fixed4(l, g.max, g.sc, table, g.shift, w);
  if (g.mode == DRAW_RESIDUAL) {
    const float qf[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = max(w[e] - prod_fixed(as_prob(qf[e]), g.z), static_cast<int64_t>(0));
  } else if (g.mode == DRAW_OTHERS) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e == g.x) w[e] = 0;
  }
}

// The draw kernel's columns, each value read back by the thread that wrote it, and the residual's segments.
template <int P>
struct DrawVals {
  float4 l[VL_GROUPS / P][VERIFY_THREADS];
  float4 q[VL_GROUPS / P][VERIFY_THREADS];
  int64_t r[VL_MAX_SEGS];
};

// Draft probabilities of the groups at col0 + 128 i.
template <int N>
__device__ __forceinline__ void load_draft(const LogitsArgs& a, int row, int col0, float (&v)[N][4]) {
  const int64_t o = row * a.q.ld;
  if (a.q.dtype == 0)
    load_groups(static_cast<const float*>(a.q.p) + o, col0, a.V, 0.f, v);
  else if (a.q.dtype == 1)
    load_groups(static_cast<const __half*>(a.q.p) + o, col0, a.V, 0.f, v);
  else
    load_groups(static_cast<const __nv_bfloat16*>(a.q.p) + o, col0, a.V, 0.f, v);
}

// One warp: the first of n weights whose running sum exceeds u * total, the last with weight when none
// does (-1 when none has any); `left` receives u * total less the sum before it.
__device__ __forceinline__ int find_segment(const int64_t* w, int n, float u, double& left) {
  const int lane = threadIdx.x & 31;
  int64_t total = 0;
  for (int k = lane; k < n; k += 32) total += w[k];
  total = warp_sum(total);
  const int64_t t = draw_threshold(u, total);
  int64_t upto = 0, before = 0;
  int at = -1, some = -1;
  for (int c0 = 0; c0 < n && at < 0; c0 += 32) {
    const int64_t v = c0 + lane < n ? w[c0 + lane] : 0;
    const int64_t incl = warp_scan(v) + upto;
    const uint32_t has = __ballot_sync(0xffffffffu, v > 0);
    const uint32_t hit = __ballot_sync(0xffffffffu, v > 0 && incl > t);
    const int src = hit ? __ffs(hit) - 1 : has ? 31 - __clz(has) : -1;
    if (src >= 0) {
      before = __shfl_sync(0xffffffffu, incl - v, src);
      some = c0 + src;
      if (hit) at = some;
    }
    upto = __shfl_sync(0xffffffffu, incl, 31);
  }
  left = static_cast<double>(u) * static_cast<double>(total) - static_cast<double>(before);
  return at >= 0 ? at : some;
}

// The whole CTA: the first column of segment `seg` whose running weight exceeds t, the last with any
// weight when none does, to tokens[row]; -1 when it has none.
template <typename T>
__device__ __forceinline__ void draw_in_segment(const LogitsArgs& a, int row, int seg, const Weigh& g, int64_t t,
                                                const float2* table, int64_t* s_sum) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const T* lrow = static_cast<const T*>(a.logits) + row * a.ld;
  const int col = chunk_col(lrow, seg / VERIFY_WARPS) + seg % VERIFY_WARPS * VL_WARP_COLS + tid * 4;
  static_assert(VL_WARP_COLS == 4 * VERIFY_THREADS, "a group a thread");
  float l[1][4], q[1][4] = {};
  load_groups(lrow, col, a.V, -INFINITY, l);
  if (g.mode == DRAW_RESIDUAL) load_draft(a, row, col, q);
  int64_t w[4];
  weigh4(make_float4(l[0][0], l[0][1], l[0][2], l[0][3]), make_float4(q[0][0], q[0][1], q[0][2], q[0][3]), col, g,
         table, w);
  const int64_t sum = w[0] + w[1] + w[2] + w[3];
  int64_t incl = warp_scan(sum);
  __syncthreads();  // s_sum may still be read
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int k = 0; k < VERIFY_WARPS; ++k) {
    if (k < warp) incl += s_sum[k];
    total += s_sum[k];
  }
  // the group that takes the sum past t; past the end (t at or above the total) the last with weight
  const int64_t cut = t < total ? t : total - 1;
  int64_t S = incl - sum;
  if (sum > 0 && S <= max(cut, static_cast<int64_t>(0)) && incl > cut) {
    int token = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      S += w[e];
      if (w[e] > 0 && S > cut && token < 0) token = col + e;
    }
    a.tokens[row] = token;
  } else if (tid == 0 && total <= 0) {
    a.tokens[row] = -1;
  }
}

template <typename T, int P>
__global__ void __launch_bounds__(VERIFY_THREADS) verify_draw_kernel(const LogitsArgs a) {
  __shared__ float2 s_table[EXP_TABLE];
  extern __shared__ __align__(16) uint8_t smem[];
  DrawVals<P>& s_vals = *reinterpret_cast<DrawVals<P>*>(smem);
  __shared__ int64_t s_w[VL_MAX_SEGS];
  __shared__ int64_t s_sum[VERIFY_WARPS];
  __shared__ int s_seg, s_flag;
  __shared__ int64_t s_t;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seq = blockIdx.y, part = blockIdx.x;
  if (tid < EXP_TABLE) s_table[tid] = EXP2_TABLE[tid];
  __syncthreads();
  pdl_wait();
  const Settled st = a.settled[seq];
  if (st.token > -2) return;  // empty, greedy, or nothing to draw from
  const bool residual = st.refused && a.q.p;
  if (!residual && part != 0) return;
  const int row = st.row, nseg = a.nchunk * VERIFY_WARPS;
  const T* lrow = static_cast<const T*>(a.logits) + row * a.ld;
  const ChunkStat* cs = a.stats + static_cast<int64_t>(row) * a.nchunk;
  const int64_t* sums = a.sums + static_cast<int64_t>(seq) * nseg;
  const float u = __ldg(a.u + row);
  Weigh g;
  g.mode = !st.refused ? DRAW_P : residual ? DRAW_RESIDUAL : DRAW_OTHERS;
  g.x = st.refused ? __ldg(a.drafts + row) : -1;
  g.sc = exp_scale(__ldg(a.temp + row));
  float v[VL_GROUPS / P][4];  // this CTA's columns, under way while the sums are scaled
  const int col0 = first_col<P>(lrow, part);
  if (residual) load_groups(lrow, col0, a.V, -INFINITY, v);

  // the segments' sums relative to the row's maximum, a one-hot draft's own weight taken out unless that
  // leaves nothing (the draft holds all of P: a refusal by an a of 1 or more)
  auto scale_sums = [&](bool others) {
    const int k0 = others ? g.x - chunk_col(lrow, 0) : -1;  // the draft's place in the chunks
    int64_t any = 0;
#pragma unroll 1
    for (int k = tid; k < nseg; k += VERIFY_THREADS) {
      const float m = cs[k / VERIFY_WARPS].max;
      int64_t s = sums[k];
      if (others && k0 / VL_WARP_COLS == k && g.x >= 0 && g.x < a.V) {
        const float l = widen<T>(lrow[g.x]);
        int64_t own[4];  // by the arithmetic of the segment's sum
        exp_fixed4(make_float4(l, l, l, l), m, g.sc, s_table, VL_SHIFT, own);
        s -= own[0];
      }
      const int64_t w = scale_fixed(s, VL_SHIFT, m, st.max, g.sc, s_table, a.shift);
      s_w[k] = w;
      any |= w;
    }
    return __syncthreads_or(any != 0);
  };
  if (!scale_sums(g.mode == DRAW_OTHERS) && g.mode == DRAW_OTHERS) {
    g.mode = DRAW_P;
    scale_sums(false);
  }

  if (residual) {
    int64_t total = 0;
    for (int k = lane; k < nseg; k += 32) total += s_w[k];
    total = warp_sum(total);
    g.shift = a.shift;
    g.max = st.max;
    g.z = total;
#pragma unroll
    for (int i = 0; i < VL_GROUPS / P; ++i) s_vals.l[i][tid] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
    load_draft(a, row, col0, v);
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < VL_GROUPS / P; ++i) s_vals.q[i][tid] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
#pragma unroll 1
    for (int i = 0; i < VL_GROUPS / P; ++i) {
      const float4 l = s_vals.l[i][tid], q = s_vals.q[i][tid];
      int64_t w[4];
      weigh4(l, q, 0, g, s_table, w);
      sum += (w[0] + w[1]) + (w[2] + w[3]);
    }
    sum = warp_sum(sum);
    int64_t* rsum = a.rsum + static_cast<int64_t>(seq) * nseg;
    store_segments<P>(sum, rsum, part, s_sum);
    __threadfence();
    __syncthreads();
    if (tid == 0) s_flag = atomicAdd(a.done + seq, 1u) == static_cast<uint32_t>(a.nchunk * P - 1);
    __syncthreads();
    if (!s_flag) return;
    __threadfence();
    int64_t any = 0;
    for (int k = tid; k < nseg; k += VERIFY_THREADS) {
      s_vals.r[k] = __ldcg(reinterpret_cast<const long long*>(rsum) + k);
      any |= s_vals.r[k];
    }
    if (!__syncthreads_or(any != 0)) g.mode = DRAW_P;  // q covers P: the draw is from P itself
  }

  if (warp == 0) {
    double left;
    const int seg = find_segment(g.mode == DRAW_RESIDUAL ? s_vals.r : s_w, nseg, u, left);
    if (lane == 0) {
      s_seg = seg;
      if (g.mode != DRAW_RESIDUAL && seg >= 0)  // in units of the chunk's own weights
        left *= pow2_double(VL_SHIFT - a.shift) / exp_double(cs[seg / VERIFY_WARPS].max, st.max, g.sc, s_table);
      s_t = __double2ll_rd(left);
    }
  }
  __syncthreads();
  const int seg = s_seg;
  if (seg < 0) {
    if (tid == 0) a.tokens[row] = -1;
    return;
  }
  if (g.mode != DRAW_RESIDUAL) {
    g.shift = VL_SHIFT;
    g.max = cs[seg / VERIFY_WARPS].max;
  }
  draw_in_segment<T>(a, row, seg, g, s_t, s_table, s_sum);
}

int64_t round256(int64_t v) { return (v + 255) & ~int64_t(255); }

int chunks(int V) { return (V + 3 + VL_CHUNK - 1) / VL_CHUNK; }

// Bytes of the workspace's parts, each on a 256-byte boundary.
struct Parts {
  int64_t stats, sums, settled, done;
};
Parts parts(int rows, int nseq, int V) {
  const int64_t nc = chunks(V);
  return Parts{round256(rows * nc * static_cast<int64_t>(sizeof(ChunkStat))), round256(nseq * nc * VERIFY_WARPS * 8),
               round256(nseq * static_cast<int64_t>(sizeof(Settled))), round256(nseq * 4LL)};
}

template <typename T, int P>
cudaError_t launch_parts(const LogitsArgs& a, cudaStream_t stream) {
  const dim3 grid(a.nchunk * P, a.nseq);
  cudaError_t e = launch_overlapped(verify_settle_kernel<T, P>, grid, 0, stream, a);
  constexpr int smem = static_cast<int>(sizeof(DrawVals<P>));
  if (e == cudaSuccess)  // idempotent, per device
    e = cudaFuncSetAttribute(verify_draw_kernel<T, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = launch_overlapped(verify_draw_kernel<T, P>, grid, smem, stream, a);
  return e;
}

// CTAs a chunk of the settled rows.  A few sequences leave SMs idle and take quarters, which end sooner; more
// take halves, since every CTA judges the rows and scales the segments' sums again.  (us with quarters, halves and
// whole chunks: 25 chunks 17.2, 17.9, 18.6; 259 32.3, 35.4, 37.9; 400 43.7, 41.5, 45.8; 2400 194, 167, 176.)
constexpr int QUARTERS_UP_TO = 2 * 152;

template <typename T>
cudaError_t launch(const LogitsArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) e = launch_overlapped(verify_stats_kernel<T>, dim3(a.nchunk, a.rows), 0, stream, a);
  if (e != cudaSuccess) return e;
  return a.nchunk * a.nseq <= QUARTERS_UP_TO ? launch_parts<T, 4>(a, stream) : launch_parts<T, 2>(a, stream);
}

}  // namespace

}  // namespace tail

using namespace tail;

extern "C" int tail_verify_logits_workspace(int32_t rows, int32_t nseq, int32_t V, int64_t* bytes) {
  if (!bytes || rows < 0 || nseq < 0 || V < 1) return TAIL_ERR_INVALID_ARG;
  if (V > VL_MAX_V || rows > VL_MAX_ROWS || nseq > VL_MAX_ROWS) {
    set_last_error("tail_verify_logits: more than 1048576 columns, 65535 rows or 65535 sequences");
    return TAIL_ERR_UNSUPPORTED;
  }
  const Parts p = parts(rows, nseq, V);
  *bytes = p.stats + 2 * p.sums + p.settled + p.done;
  return TAIL_OK;
}

extern "C" int tail_verify_logits(int32_t rows, int32_t nseq, int32_t V, const void* logits, int32_t logits_dtype,
                                  int64_t logits_ld, const float* temperature, const int32_t* cu_rows,
                                  const int32_t* drafts, const float* u_accept, const float* u_draw,
                                  const void* draft_probs_opt, int32_t draft_dtype, int64_t draft_ld, void* workspace,
                                  int64_t workspace_bytes, int32_t* out_tokens, int32_t* out_count, void* stream) {
  int64_t need = 0;
  const int rc = tail_verify_logits_workspace(rows, nseq, V, &need);
  if (rc) return rc;
  if (nseq == 0) return TAIL_OK;
  if (!cu_rows || !out_count || !aligned(cu_rows, 4) || !aligned(out_count, 4)) return TAIL_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) return TAIL_ERR_INVALID_ARG;
  if (logits_dtype < TAIL_F32 || logits_dtype > TAIL_BF16) return TAIL_ERR_INVALID_ARG;
  if (rows > 0) {
    if (!logits || !temperature || !drafts || !u_accept || !u_draw || !out_tokens || logits_ld < V)
      return TAIL_ERR_INVALID_ARG;
    if (!aligned(logits, elem_bytes(logits_dtype)) || !aligned(temperature, 4) || !aligned(drafts, 4) ||
        !aligned(u_accept, 4) || !aligned(u_draw, 4) || !aligned(out_tokens, 4))
      return TAIL_ERR_INVALID_ARG;
    const int64_t n = rows;
    const struct {
      const void* p;
      int64_t words;
    } in[] = {{cu_rows, nseq + 1LL}, {drafts, n}, {u_accept, n}, {u_draw, n}, {temperature, n}, {workspace, need / 4}};
    for (const auto& i : in)
      if (meets(out_tokens, n, i.p, i.words) || meets(out_count, nseq, i.p, i.words)) return TAIL_ERR_INVALID_ARG;
    if (meets(out_tokens, n, out_count, nseq)) return TAIL_ERR_INVALID_ARG;
  }
  if (draft_probs_opt) {
    if (draft_dtype < TAIL_F32 || draft_dtype > TAIL_BF16 || draft_ld < V) return TAIL_ERR_INVALID_ARG;
    if (!aligned(draft_probs_opt, elem_bytes(draft_dtype))) return TAIL_ERR_INVALID_ARG;
  }
  LogitsArgs a;
  a.logits = logits;
  a.ld = logits_ld;
  a.temp = temperature;
  a.cu = cu_rows;
  a.drafts = drafts;
  a.accept = u_accept;
  a.u = u_draw;
  a.q = DraftProbs{draft_probs_opt, draft_dtype, draft_ld, V};
  a.rows = rows;
  a.nseq = nseq;
  a.V = V;
  a.nchunk = chunks(V);
  const Parts n = parts(rows, nseq, V);
  uint8_t* p = static_cast<uint8_t*>(workspace);
  a.stats = reinterpret_cast<ChunkStat*>(p);
  a.sums = reinterpret_cast<int64_t*>(p += n.stats);
  a.rsum = reinterpret_cast<int64_t*>(p += n.sums);
  a.settled = reinterpret_cast<Settled*>(p += n.sums);
  a.done = reinterpret_cast<uint32_t*>(p += n.settled);
  a.tokens = out_tokens;
  a.count = out_count;
  int bits = 0;
  while ((int64_t(1) << bits) < V) ++bits;
  a.shift = 62 - bits < 44 ? 62 - bits : 44;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == TAIL_F32   ? launch<float>(a, s)
                        : logits_dtype == TAIL_F16 ? launch<__half>(a, s)
                                                   : launch<__nv_bfloat16>(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "tail_verify_logits: kernel launch");
  return TAIL_OK;
}
