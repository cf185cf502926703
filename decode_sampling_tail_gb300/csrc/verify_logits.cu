// Verification of drafted tokens against whole-vocabulary distributions: the
// rule of verify_lists.cu with P_j = softmax(l_j / T_j) over all V logits (the
// lowest index of the maximum when T <= 0).
//
// Three kernels, over chunks of 8192 columns that a CTA holds in registers:
//   verify_stats (chunk, row): the chunk's maximum m_c, its lowest column and sum exp((l - m_c) / T)
//     in fp32.  Every row has to be read, since which one is settled is not known yet; this pass is
//     bound by memory and only has to decide acceptances (a relative 2^-21 of Z).
//   verify_settle (chunk, sequence): each CTA judges the sequence's rows from those statistics (all
//     of them compute the same bits, none waits) and finds the settled row; then the chunk's sum of that
//     row alone as an integer (fixed_exp.cuh, units of 2^-49: 8192 of at most 1 stay below 2^63).
//   verify_draw (chunk, sequence): after d accepted drafts, or with one-hot drafts (P without x_j), the
//     chunk sums already say which chunk holds the token, and that chunk's CTA alone reads its columns
//     again.  The residual max(P - q, 0) needs one pass over that row's l and q: every CTA sums its
//     chunk, the last of the sequence to finish (a counter that verify_settle cleared) picks the chunk
//     and the token.
// Sums over chunks are integers of 2^-shift relative to the row's maximum, with V 2^shift below 2^62;
// the residual is max(e - q Z, 0) in the same units.  The draft's row is read only for sequences that
// refuse a draft.
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
constexpr int VL_MAX_CHUNKS = (VL_MAX_V + 3) / VL_CHUNK + 1;  // a thread each in the draw kernel
static_assert(VL_MAX_CHUNKS <= VERIFY_THREADS, "one thread a chunk");
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
  int64_t* sums;       // [nseq][nchunk] the settled row's chunk sums, units of 2^-49 relative to m_c
  int64_t* rsum;       // [nseq][nchunk] its residual sums
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
template <typename T>
__device__ __forceinline__ void load_groups(const T* row, int col0, int V, float fill, float (&v)[VL_GROUPS][4]) {
  const bool whole = (reinterpret_cast<uintptr_t>(row + col0) & (4 * sizeof(T) - 1)) == 0;
  bool rest = false;
#pragma unroll
  for (int i = 0; i < VL_GROUPS; ++i) {
    const int col = col0 + i * 128;
    const bool inside = col >= 0 && col + 4 <= V;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] = fill;
    if (whole && inside) unpack4(row + col, v[i]);
    rest = rest || (inside ? !whole : col + 4 > 0 && col < V);
  }
  if (!rest) return;
#pragma unroll
  for (int i = 0; i < VL_GROUPS; ++i)
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

// The first of a thread's columns of chunk c.
template <typename T>
__device__ __forceinline__ int first_col(const T* row, int c) {
  return chunk_col(row, c) + (threadIdx.x >> 5) * VL_WARP_COLS + (threadIdx.x & 31) * 4;
}

// A chunk's values in shared memory, each read back by the thread that wrote it: the weights' loops stay
// rolled (code that runs once is bound by fetching it).
struct ChunkVals {
  float4 l[VL_GROUPS][VERIFY_THREADS];
};

template <typename T>
__device__ __forceinline__ int stage_chunk(const T* row, int c, int V, ChunkVals& s) {
  const int col0 = first_col(row, c);
  float v[VL_GROUPS][4];
  load_groups(row, col0, V, -INFINITY, v);
#pragma unroll
  for (int i = 0; i < VL_GROUPS; ++i) s.l[i][threadIdx.x] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
  return col0;
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
  const int col0 = first_col(lrow, c);
  float v[VL_GROUPS][4];
  load_groups(lrow, col0, a.V, -INFINITY, v);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VL_GROUPS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, v[i][e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
  m = s_max[0];
#pragma unroll
  for (int w = 1; w < VERIFY_WARPS; ++w) m = fmaxf(m, s_max[w]);
  float sum = 0.f;
  int arg = a.V;
  if (!(temp > 0.0f)) {
#pragma unroll
    for (int i = VL_GROUPS - 1; i >= 0; --i)
#pragma unroll
      for (int e = 3; e >= 0; --e)
        if (v[i][e] == m && col0 + i * 128 + e >= 0) arg = col0 + i * 128 + e;
    arg = __reduce_min_sync(0xffffffffu, arg);
  } else if (m != -INFINITY) {
    const float scale = exp_scale(temp).h;
#pragma unroll
    for (int i = 0; i < VL_GROUPS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += exp_fast(v[i][e], m, scale);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  if (lane == 0) {
    s_sum[warp] = sum;
    s_arg[warp] = arg;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    ChunkStat st = {m, 0.f, a.V, 0};
    for (int w = 0; w < VERIFY_WARPS; ++w) {
      st.sum += s_sum[w];
      st.arg = min(st.arg, s_arg[w]);
    }
    a.stats[static_cast<int64_t>(row) * a.nchunk + c] = st;
  }
}

// One warp: whether the row's draft is accepted, and what its token is if it is settled here.
template <typename T>
__device__ __forceinline__ bool judge_row(const LogitsArgs& a, int row, bool bonus, const float2* table, Settled& s) {
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
  double ex = 0.0, Z = 1.0;
  if (m == -INFINITY) {
    s.token = -1;
  } else if (greedy) {
    int arg = a.V;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (cm[i] == m) arg = min(arg, ca[i]);
    arg = __reduce_min_sync(0xffffffffu, arg);
    s.token = arg < a.V ? arg : -1;
    ex = known && x == arg ? 1.0 : 0.0;
  } else {
    const ExpScale sc = exp_scale(temp);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) z = fmaf(cz[i], exp_fast(cm[i], m, sc.h), z);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    Z = static_cast<double>(z);
    if (known) ex = exp_double(lx, m, sc, table);
    if (!(z > 0.f)) s.token = -1;
  }
  const bool ok = !bonus && static_cast<double>(u_a) * qx * Z < ex;
  s.refused = !bonus && !ok;
  return ok;
}

template <typename T>
__global__ void __launch_bounds__(VERIFY_THREADS) verify_settle_kernel(const LogitsArgs a) {
  __shared__ float2 s_table[EXP_TABLE];
  __shared__ Settled s_row[VERIFY_WARPS];
  __shared__ int64_t s_sum[VERIFY_WARPS];
  __shared__ ChunkVals s_vals;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seq = blockIdx.y, c = blockIdx.x;
  if (tid < EXP_TABLE) s_table[tid] = EXP2_TABLE[tid];
  __syncthreads();
  pdl_wait();
  int lo, hi;
  sequence_rows(a.cu, seq, a.rows, lo, hi);
  Settled st = {hi, 0.f, -1, 0};
  for (int j0 = lo; j0 < hi; j0 += VERIFY_WARPS) {
    if (j0 + warp < hi) {
      Settled s;
      const bool ok = judge_row<T>(a, j0 + warp, j0 + warp == hi - 1, s_table, s);
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
  if (c == 0) {
    write_sequence(lo, hi, st.row, a.drafts, a.tokens, a.count + seq);
    if (tid == 0) {
      a.settled[seq] = st;
      a.done[seq] = 0u;
      if (hi > lo && st.token > -2) a.tokens[st.row] = st.token;
    }
  }
  if (st.token > -2) return;
  const float m = a.stats[static_cast<int64_t>(st.row) * a.nchunk + c].max;
  int64_t sum = 0;
  if (m != -INFINITY) {
    stage_chunk(static_cast<const T*>(a.logits) + st.row * a.ld, c, a.V, s_vals);
    const ExpScale sc = exp_scale(__ldg(a.temp + st.row));
#pragma unroll 1
    for (int i = 0; i < VL_GROUPS; ++i) {
      const float4 v = s_vals.l[i][tid];
      sum += exp_fixed(v.x, m, sc, s_table, VL_SHIFT) + exp_fixed(v.y, m, sc, s_table, VL_SHIFT) +
             exp_fixed(v.z, m, sc, s_table, VL_SHIFT) + exp_fixed(v.w, m, sc, s_table, VL_SHIFT);
    }
    sum = warp_sum(sum);
  }
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < VERIFY_WARPS; ++w) sum += s_sum[w];
    a.sums[static_cast<int64_t>(seq) * a.nchunk + c] = sum;
  }
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
  float max, zh, zl, scale;
  ExpScale sc;
};

// Shared memory of the draw kernel.
struct DrawVals {
  ChunkVals v;
  float4 q[VL_GROUPS][VERIFY_THREADS];
  int64_t g[VL_GROUPS][VERIFY_THREADS];  // the groups' sums
};

__device__ __forceinline__ int64_t weight_of(float l, float q, int col, const Weigh& g, const float2* table) {
  int64_t r = exp_fixed(l, g.max, g.sc, table, g.shift);
  if (g.mode == DRAW_RESIDUAL) r = max(r - prod_fixed(as_prob(q), g.zh, g.zl, g.scale), static_cast<int64_t>(0));
  return l == -INFINITY || (g.mode == DRAW_OTHERS && col == g.x) ? 0 : r;
}

// The whole CTA: chunk c's values, the groups' sums, and their sum over the warp.
template <typename T>
__device__ __noinline__ int64_t weigh_chunk(const LogitsArgs& a, int row, int c, const Weigh& g, const float2* table,
                                            DrawVals& s) {
  const int tid = threadIdx.x;
  const int col0 = stage_chunk(static_cast<const T*>(a.logits) + row * a.ld, c, a.V, s.v);
  if (g.mode == DRAW_RESIDUAL) {
    float v[VL_GROUPS][4];
    const int64_t o = row * a.q.ld;
    if (a.q.dtype == 0)
      load_groups(static_cast<const float*>(a.q.p) + o, col0, a.V, 0.f, v);
    else if (a.q.dtype == 1)
      load_groups(static_cast<const __half*>(a.q.p) + o, col0, a.V, 0.f, v);
    else
      load_groups(static_cast<const __nv_bfloat16*>(a.q.p) + o, col0, a.V, 0.f, v);
#pragma unroll
    for (int i = 0; i < VL_GROUPS; ++i) s.q[i][tid] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
  }
  int64_t sum = 0;
#pragma unroll 1
  for (int i = 0; i < VL_GROUPS; ++i) {
    const float4 l = s.v.l[i][tid];
    const float4 q = g.mode == DRAW_RESIDUAL ? s.q[i][tid] : make_float4(0.f, 0.f, 0.f, 0.f);
    const int col = col0 + i * 128;
    const int64_t w = weight_of(l.x, q.x, col, g, table) + weight_of(l.y, q.y, col + 1, g, table) +
                      weight_of(l.z, q.z, col + 2, g, table) + weight_of(l.w, q.w, col + 3, g, table);
    s.g[i][tid] = w;
    sum += w;
  }
  return warp_sum(sum);
}

// The whole CTA, after weigh_chunk of chunk c (`sum` its result): the first column whose running weight
// exceeds t, the last with any weight when none does; -1 when the chunk has no weight.
template <typename T>
__device__ __noinline__ int find_column(const LogitsArgs& a, int row, int c, const Weigh& g, const float2* table,
                                        const DrawVals& s, int64_t sum, int64_t t, int64_t* s_sum, int* s_col) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __syncthreads();  // s_sum may still be read
  if (lane == 0) s_sum[warp] = sum;
  if (tid == 0) *s_col = -1;
  __syncthreads();
  int at = -1, some = -1;
  int64_t before = 0, upto = 0;
#pragma unroll
  for (int k = 0; k < VERIFY_WARPS; ++k) {
    if (s_sum[k] > 0) some = k;
    if (at < 0 && s_sum[k] > 0 && upto + s_sum[k] > t) {
      at = k;
      before = upto;
    }
    upto += s_sum[k];
  }
  const bool past = at < 0;
  if (past) at = some;
  if (warp == at) {
    int gi = -1, src = -1;  // the group: index and lane
    int64_t S = 0;          // the sum before it
#pragma unroll 1
    for (int i = 0; i < VL_GROUPS; ++i) {
      const int64_t w = s.g[i][tid];
      const int64_t incl = before + warp_scan(w);
      const uint32_t any = __ballot_sync(0xffffffffu, w > 0);
      const uint32_t hit = past ? 0u : __ballot_sync(0xffffffffu, w > 0 && incl > t);
      if (any) {
        gi = i;
        src = hit ? __ffs(hit) - 1 : 31 - __clz(any);
        S = __shfl_sync(0xffffffffu, incl - w, src);
      }
      if (hit) break;
      before = __shfl_sync(0xffffffffu, incl, 31);
    }
    if (gi >= 0 && lane == src) {
      const float l[4] = {s.v.l[gi][tid].x, s.v.l[gi][tid].y, s.v.l[gi][tid].z, s.v.l[gi][tid].w};
      const float q[4] = {s.q[gi][tid].x, s.q[gi][tid].y, s.q[gi][tid].z, s.q[gi][tid].w};
      const int col0 = first_col(static_cast<const T*>(a.logits) + row * a.ld, c) + gi * 128;
      int found = -1, last = -1;
      for (int e = 0; e < 4; ++e) {
        const int64_t w = weight_of(l[e], q[e], col0 + e, g, table);
        S += w;
        if (w > 0) {
          last = col0 + e;
          if (found < 0 && !past && S > t) found = last;
        }
      }
      *s_col = found >= 0 ? found : last;
    }
  }
  __syncthreads();
  return *s_col;
}

// One warp: the first of n weights whose running sum exceeds u * total, the last with weight when none
// does (-1 when none has any); `left` receives u * total less the sum before it.
__device__ __forceinline__ int find_chunk(const int64_t* w, int n, float u, int64_t total, double& left) {
  const int lane = threadIdx.x & 31;
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

template <typename T>
__global__ void __launch_bounds__(VERIFY_THREADS) verify_draw_kernel(const LogitsArgs a) {
  __shared__ float2 s_table[EXP_TABLE];
  __shared__ int64_t s_w[VL_MAX_CHUNKS], s_all[VL_MAX_CHUNKS];
  __shared__ int64_t s_sum[VERIFY_WARPS];
  __shared__ int s_col, s_chunk, s_flag;
  __shared__ int64_t s_t;
  extern __shared__ __align__(16) uint8_t smem[];
  DrawVals& vals = *reinterpret_cast<DrawVals*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seq = blockIdx.y, c = blockIdx.x;
  if (tid < EXP_TABLE) s_table[tid] = EXP2_TABLE[tid];
  __syncthreads();
  pdl_wait();
  const Settled st = a.settled[seq];
  if (st.token > -2) return;  // empty, greedy, or nothing to draw from
  const int row = st.row;
  const ChunkStat* cs = a.stats + static_cast<int64_t>(row) * a.nchunk;
  const int64_t* sums = a.sums + static_cast<int64_t>(seq) * a.nchunk;
  const float u = __ldg(a.u + row);
  Weigh g;
  g.mode = !st.refused ? DRAW_P : a.q.p ? DRAW_RESIDUAL : DRAW_OTHERS;
  g.x = st.refused ? __ldg(a.drafts + row) : -1;
  g.sc = exp_scale(__ldg(a.temp + row));
  // the chunks' sums relative to the row's maximum: all of P (s_all), and without a one-hot draft (s_w)
  if (tid < a.nchunk) {
    const float m = cs[tid].max;
    const int64_t all = sums[tid];
    int64_t own = 0;
    if (g.mode == DRAW_OTHERS && g.x >= 0 && g.x < a.V) {
      const T* lrow = static_cast<const T*>(a.logits) + row * a.ld;
      const int k0 = chunk_col(lrow, tid);
      if (g.x >= k0 && g.x < k0 + VL_CHUNK) {
        const float l = widen<T>(lrow[g.x]);
        if (l > -INFINITY) own = exp_fixed(l, m, g.sc, s_table, VL_SHIFT);
      }
    }
    s_all[tid] = scale_fixed(all, VL_SHIFT, m, st.max, g.sc, s_table, a.shift);
    s_w[tid] = scale_fixed(all - own, VL_SHIFT, m, st.max, g.sc, s_table, a.shift);
  }
  __syncthreads();
  auto total_of = [&](const int64_t* w) {
    int64_t t = 0;
    for (int k = lane; k < a.nchunk; k += 32) t += w[k];
    return warp_sum(t);
  };

  if (g.mode == DRAW_RESIDUAL) {
    const double Z = static_cast<double>(total_of(s_all)) * pow2_double(-a.shift);
    g.shift = a.shift;
    g.scale = ldexpf(1.f, a.shift);
    g.max = st.max;
    g.zh = static_cast<float>(Z);
    g.zl = static_cast<float>(Z - static_cast<double>(g.zh));
    const int64_t mine = weigh_chunk<T>(a, row, c, g, s_table, vals);
    if (lane == 0) s_sum[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      int64_t sum = mine;
      for (int k = 1; k < VERIFY_WARPS; ++k) sum += s_sum[k];
      __stcg(reinterpret_cast<long long*>(a.rsum) + static_cast<int64_t>(seq) * a.nchunk + c, sum);
      __threadfence();
      s_flag = atomicAdd(a.done + seq, 1u) == static_cast<uint32_t>(a.nchunk - 1);
    }
    __syncthreads();
    if (!s_flag) return;
    __threadfence();
    if (tid < a.nchunk)
      s_w[tid] = __ldcg(reinterpret_cast<const long long*>(a.rsum) + static_cast<int64_t>(seq) * a.nchunk + tid);
    __syncthreads();
    if (warp == 0) {
      double left;
      const int at = find_chunk(s_w, a.nchunk, u, total_of(s_w), left);
      if (lane == 0) {
        s_chunk = at;
        s_t = __double2ll_rd(left);
      }
    }
    __syncthreads();
    const int at = s_chunk;
    if (at >= 0) {
      const int64_t sum = at == c ? mine : weigh_chunk<T>(a, row, at, g, s_table, vals);
      const int col = find_column<T>(a, row, at, g, s_table, vals, sum, s_t, s_sum, &s_col);
      if (tid == 0) a.tokens[row] = col;
      return;
    }
    g.mode = DRAW_P;  // q covers P: the draw is from P itself, by this CTA
  }

  const bool alone = st.refused && a.q.p;  // the last CTA of a residual without weight does any chunk
  g.shift = VL_SHIFT;
  if (warp == 0) {
    int64_t total = total_of(alone ? s_all : s_w);
    const bool others = !alone && total > 0;
    if (!others) total = total_of(s_all);  // the draft holds all of P (a refusal by an a of 1 or more): from P
    double left;
    const int at = find_chunk(others ? s_w : s_all, a.nchunk, u, total, left);
    if (lane == 0) {
      s_chunk = at;
      s_flag = others ? g.mode : DRAW_P;
      if (at >= 0)  // in units of the chunk's own weights
        s_t = __double2ll_rd(left * pow2_double(VL_SHIFT - a.shift) / exp_double(cs[at].max, st.max, g.sc, s_table));
    }
  }
  __syncthreads();
  g.mode = s_flag;
  const int at = s_chunk;
  if (at < 0) {
    if ((c == 0 || alone) && tid == 0) a.tokens[row] = -1;
    return;
  }
  if (!alone && at != c) return;
  g.max = cs[at].max;
  const int64_t sum = weigh_chunk<T>(a, row, at, g, s_table, vals);
  const int col = find_column<T>(a, row, at, g, s_table, vals, sum, s_t, s_sum, &s_col);
  if (tid == 0) a.tokens[row] = col;
}

int64_t round256(int64_t v) { return (v + 255) & ~int64_t(255); }

int chunks(int V) { return (V + 3 + VL_CHUNK - 1) / VL_CHUNK; }

// Bytes of the workspace's parts, each on a 256-byte boundary.
struct Parts {
  int64_t stats, sums, settled, done;
};
Parts parts(int rows, int nseq, int V) {
  const int64_t nc = chunks(V);
  return Parts{round256(rows * nc * static_cast<int64_t>(sizeof(ChunkStat))), round256(nseq * nc * 8),
               round256(nseq * static_cast<int64_t>(sizeof(Settled))), round256(nseq * 4LL)};
}

template <typename T>
cudaError_t launch(const LogitsArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) e = launch_overlapped(verify_stats_kernel<T>, dim3(a.nchunk, a.rows), 0, stream, a);
  if (e == cudaSuccess) e = launch_overlapped(verify_settle_kernel<T>, dim3(a.nchunk, a.nseq), 0, stream, a);
  constexpr int smem = static_cast<int>(sizeof(DrawVals));
  if (e == cudaSuccess)  // idempotent, per device
    e = cudaFuncSetAttribute(verify_draw_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = launch_overlapped(verify_draw_kernel<T>, dim3(a.nchunk, a.nseq), smem, stream, a);
  return e;
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
