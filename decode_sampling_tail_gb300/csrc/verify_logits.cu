// Verification of drafted tokens against whole-vocabulary distributions: the
// rule of verify_lists.cu with P_j = softmax(l_j / T_j) over all V logits (the
// lowest index of the maximum when T <= 0).
//
// Two kernels.
//   verify_stats: CTA (chunk, row) reads 8192 columns once into registers and
//     writes their maximum m_c, its lowest column and S_c = sum exp((l - m_c)/T)
//     as an integer (fixed_exp.cuh, units of 2^-49: 8192 of at most 1 stay below
//     2^63).  Every row has to be read: which one is settled is not known yet.
//   verify_draw: CTA (chunk, sequence).  Each forms the rows' maxima and sums Z
//     from the chunk statistics and finds the settled row; all CTAs of a sequence
//     compute the same bits, so none waits for another.  After d accepted drafts,
//     or with one-hot drafts (P without x_j), the chunk sums already say which
//     chunk holds the token, and that chunk's CTA alone reads its columns again.
//     The residual max(P - q, 0) needs one pass over that row's l and q: every CTA
//     sums its chunk, the last of the sequence to finish (a counter that
//     verify_stats zeroed) picks the chunk and the token.
// The residual is formed as max(e - q Z, 0) in integers of 2^-shift relative to
// the row's maximum, with V 2^shift below 2^62.
//
// The draft's row is read only for sequences that refuse a draft.
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
  int64_t sum;  // of exp((l - max) / T) in units of 2^-49; 0 for greedy rows
  float max;
  int32_t arg;  // lowest column of the maximum
};

struct LogitsArgs {
  const void* logits;
  int dtype;
  int64_t ld;
  const float* temp;
  const int32_t* cu;
  const int32_t* drafts;
  const float* accept;
  const float* u;
  DraftProbs q;
  ChunkStat* stats;    // [rows][nchunk]
  int64_t* rsum;       // [nseq][nchunk] residual sums of the chunks
  uint32_t* done;      // [nseq] CTAs whose residual sum is written
  int32_t* tokens;
  int32_t* count;
  int rows, nseq, V, nchunk;
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

// Columns [col, col + 4) of a row; `fill` outside [0, V).  One vector load where all four are inside
// and aligned.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int col, int V, float fill, float (&v)[4]) {
  const T* p = row + col;
  if (col >= 0 && col + 4 <= V && (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(T) - 1)) == 0) {
    unpack4(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (col + e >= 0 && col + e < V) ? widen<T>(p[e]) : fill;
  }
}

__device__ __forceinline__ void load4_draft(const DraftProbs& q, int64_t row, int col, float (&v)[4]) {
  const int64_t o = row * q.ld;
  if (q.dtype == 0)
    load4(static_cast<const float*>(q.p) + o, col, q.V, 0.f, v);
  else if (q.dtype == 1)
    load4(static_cast<const __half*>(q.p) + o, col, q.V, 0.f, v);
  else
    load4(static_cast<const __nv_bfloat16*>(q.p) + o, col, q.V, 0.f, v);
}

// First column of chunk c: chunks start `off` columns early so that groups of 4 lie on whole
// vectors when a row starts inside one (an odd leading dimension).
template <typename T>
__device__ __forceinline__ int chunk_col(const T* row, int c) {
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 3);
  return c * VL_CHUNK - off;
}

template <typename T>
__global__ void __launch_bounds__(VERIFY_THREADS) verify_stats_kernel(const LogitsArgs a) {
  __shared__ float2 s_table[EXP_TABLE];
  __shared__ float s_max[VERIFY_WARPS];
  __shared__ int s_arg[VERIFY_WARPS];
  __shared__ int64_t s_sum[VERIFY_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, row = blockIdx.y;
  // the draw kernel's counters
  const int cta = row * a.nchunk + c;
  for (int64_t s = static_cast<int64_t>(cta) * VERIFY_THREADS + tid; s < a.nseq;
       s += static_cast<int64_t>(a.rows) * a.nchunk * VERIFY_THREADS)
    a.done[s] = 0u;
  if (row >= __ldg(a.cu + a.nseq)) return;  // behind the last sequence
  if (tid < EXP_TABLE) s_table[tid] = EXP2_TABLE[tid];
  const T* lrow = static_cast<const T*>(a.logits) + row * a.ld;
  const int col0 = chunk_col(lrow, c) + warp * VL_WARP_COLS + lane * 4;
  const float temp = __ldg(a.temp + row);
  float v[VL_GROUPS][4];
#pragma unroll
  for (int i = 0; i < VL_GROUPS; ++i) load4(lrow, col0 + i * 128, a.V, -INFINITY, v[i]);
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
  const bool greedy = !(temp > 0.0f);
  int64_t sum = 0;
  int arg = a.V;
  if (greedy) {
#pragma unroll
    for (int i = VL_GROUPS - 1; i >= 0; --i)
#pragma unroll
      for (int e = 3; e >= 0; --e)
        if (v[i][e] == m && col0 + i * 128 + e >= 0) arg = col0 + i * 128 + e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) arg = min(arg, __shfl_xor_sync(0xffffffffu, arg, o));
  } else if (m != -INFINITY) {
    const ExpScale sc = exp_scale(temp);
#pragma unroll
    for (int i = 0; i < VL_GROUPS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += exp_fixed(v[i][e], m, sc, s_table, VL_SHIFT);
    sum = warp_sum(sum);
  }
  if (lane == 0) {
    s_sum[warp] = sum;
    s_arg[warp] = arg;
  }
  __syncthreads();
  if (tid == 0) {
    ChunkStat st;
    st.sum = 0;
    st.arg = a.V;
    st.max = m;
    for (int w = 0; w < VERIFY_WARPS; ++w) {
      st.sum += s_sum[w];
      st.arg = min(st.arg, s_arg[w]);
    }
    a.stats[static_cast<int64_t>(row) * a.nchunk + c] = st;
  }
}

enum DrawMode : int {
  DRAW_P = 0,         // from P
  DRAW_OTHERS = 1,    // from P without the draft (the residual of a one-hot draft)
  DRAW_RESIDUAL = 2,  // from max(P - q, 0)
};

struct Settled {
  int row;
  float max;
  double Z;      // sum of exp((l - max) / T) over the row
  int token;     // >= -1: known without a draw (greedy, or nothing to draw from); -2: to be drawn
  int refused;
};

// One warp: the row's statistics and whether its draft is accepted.
template <typename T>
__device__ __forceinline__ bool judge_row(const LogitsArgs& a, int row, bool bonus, const float2* table, Settled& s) {
  const int lane = threadIdx.x & 31;
  const ChunkStat* st = a.stats + static_cast<int64_t>(row) * a.nchunk;
  const float temp = __ldg(a.temp + row);
  const bool greedy = !(temp > 0.0f);
  const int x = bonus ? -1 : a.drafts[row];
  const bool known = x >= 0 && x < a.V;
  const float u_a = bonus ? 0.f : a.accept[row];
  const float qx = !known ? 0.f : a.q.p ? draft_prob(a.q, row, x) : 1.f;
  const float lx = known ? widen<T>(static_cast<const T*>(a.logits)[row * a.ld + x]) : -INFINITY;
  float m = -INFINITY;
  for (int c = lane; c < a.nchunk; c += 32) m = fmaxf(m, st[c].max);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  s.row = row;
  s.max = m;
  s.Z = 1.0;
  s.token = -2;
  double ex = 0.0;
  if (m == -INFINITY) {
    s.token = -1;
  } else if (greedy) {
    int arg = a.V;
    for (int c = lane; c < a.nchunk; c += 32)
      if (st[c].max == m) arg = min(arg, st[c].arg);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) arg = min(arg, __shfl_xor_sync(0xffffffffu, arg, o));
    s.token = arg < a.V ? arg : -1;
    ex = known && x == arg ? 1.0 : 0.0;
  } else {
    const ExpScale sc = exp_scale(temp);
    double z = 0.0;
    for (int c = lane; c < a.nchunk; c += 32)
      z += ldexp(static_cast<double>(st[c].sum), -VL_SHIFT) * exp_double(st[c].max, m, sc, table);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    s.Z = z;
    if (known) ex = exp_double(lx, m, sc, table);
    if (!(z > 0.0)) s.token = -1;
  }
  const bool ok = !bonus && static_cast<double>(u_a) * qx * s.Z < ex;
  s.refused = !bonus && !ok;
  return ok;
}

// The weight of one column as an integer: exp in units of 2^-49 relative to the chunk's maximum
// (DRAW_P, DRAW_OTHERS), or the residual in units of 2^-shift relative to the row's.
struct Weigh {
  int mode, x, shift;
  float max, zh, zl, scale;
  ExpScale sc;
};

// A thread's VL_GROUPS x 4 weights of chunk c.
template <typename T>
__device__ __forceinline__ void chunk_weights(const LogitsArgs& a, int row, int c, const Weigh& g, const float2* table,
                                              int64_t (&w)[VL_GROUPS][4], int& col0) {
  const T* lrow = static_cast<const T*>(a.logits) + row * a.ld;
  col0 = chunk_col(lrow, c) + (threadIdx.x >> 5) * VL_WARP_COLS + (threadIdx.x & 31) * 4;
#pragma unroll
  for (int i = 0; i < VL_GROUPS; ++i) {
    float v[4];
    const int col = col0 + i * 128;
    load4(lrow, col, a.V, -INFINITY, v);
    if (g.mode == DRAW_RESIDUAL) {
      float q[4];
      load4_draft(a.q, row, col, q);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t r =
            exp_fixed(v[e], g.max, g.sc, table, g.shift) - prod_fixed(as_prob(q[e]), g.zh, g.zl, g.scale);
        w[i][e] = v[e] > -INFINITY && r > 0 ? r : 0;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t r = v[e] > -INFINITY ? exp_fixed(v[e], g.max, g.sc, table, g.shift) : 0;
        w[i][e] = g.mode == DRAW_OTHERS && col + e == g.x ? 0 : r;
      }
    }
  }
}

// The whole CTA: the first column of the chunk whose running weight exceeds t, the last with any
// weight when none does; -1 when the chunk has no weight.
__device__ __forceinline__ int find_column(const int64_t (&w)[VL_GROUPS][4], int col0, double t, int64_t* s_sum,
                                           int* s_col) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t sum = 0;
#pragma unroll
  for (int i = 0; i < VL_GROUPS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += w[i][e];
  sum = warp_sum(sum);
  __syncthreads();  // s_sum may still be read
  if (lane == 0) s_sum[warp] = sum;
  if (threadIdx.x == 0) *s_col = -1;
  __syncthreads();
  int at = -1, some = -1;
  int64_t before = 0, upto = 0;
  for (int k = 0; k < VERIFY_WARPS; ++k) {
    if (s_sum[k] > 0) some = k;
    if (at < 0 && s_sum[k] > 0 && static_cast<double>(upto + s_sum[k]) > t) {
      at = k;
      before = upto;
    }
    upto += s_sum[k];
  }
  const bool past = at < 0;
  if (past) at = some;
  if (warp == at) {
    int found = -1, last = -1;
    for (int i = 0; i < VL_GROUPS && found < 0; ++i) {
      const int64_t g = w[i][0] + w[i][1] + w[i][2] + w[i][3];
      const int64_t incl = warp_scan(g);
      const uint32_t any = __ballot_sync(0xffffffffu, g > 0);
      const uint32_t hit = past ? 0u : __ballot_sync(0xffffffffu, g > 0 && static_cast<double>(before + incl) > t);
      const int src = hit ? __ffs(hit) - 1 : any ? 31 - __clz(any) : -1;
      if (src >= 0) {
        int64_t S = before + incl - g;
        int c = -1, z = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S += w[i][e];
          if (w[i][e] > 0) {
            z = e;
            if (c < 0 && static_cast<double>(S) > t) c = e;
          }
        }
        const int e = hit ? (c >= 0 ? c : z) : z;
        const int col = __shfl_sync(0xffffffffu, col0 + i * 128 + e, src);
        if (hit)
          found = col;
        else
          last = col;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) *s_col = found >= 0 ? found : last;
  }
  __syncthreads();
  return *s_col;
}

template <typename T>
__global__ void __launch_bounds__(VERIFY_THREADS) verify_draw_kernel(const LogitsArgs a, int shift) {
  __shared__ float2 s_table[EXP_TABLE];
  __shared__ Settled s_row[VERIFY_WARPS];
  __shared__ int64_t s_sum[VERIFY_WARPS];
  __shared__ int s_col, s_chunk, s_last;
  __shared__ double s_t;
  __shared__ double s_w[VL_MAX_CHUNKS], s_all[VL_MAX_CHUNKS], s_f[VL_MAX_CHUNKS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seq = blockIdx.y, c = blockIdx.x;
  if (tid < EXP_TABLE) s_table[tid] = EXP2_TABLE[tid];
  int lo, hi;
  sequence_rows(a.cu, seq, a.rows, lo, hi);
  Settled st;
  st.row = hi;
  __syncthreads();
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
  if (c == 0) write_sequence(lo, hi, st.row, a.drafts, a.tokens, a.count + seq);
  if (hi == lo) return;
  if (st.token > -2) {
    if (c == 0 && tid == 0) a.tokens[st.row] = st.token;
    return;
  }
  const int row = st.row;
  const ChunkStat* cs = a.stats + static_cast<int64_t>(row) * a.nchunk;
  Weigh g;
  g.mode = !st.refused ? DRAW_P : a.q.p ? DRAW_RESIDUAL : DRAW_OTHERS;
  g.x = st.refused ? a.drafts[row] : -1;
  g.sc = exp_scale(__ldg(a.temp + row));
  const float u = __ldg(a.u + row);
  int64_t w[VL_GROUPS][4];
  int col0;

  if (g.mode == DRAW_RESIDUAL) {
    g.shift = shift;
    g.scale = ldexpf(1.f, shift);
    g.max = st.max;
    g.zh = static_cast<float>(st.Z);
    g.zl = static_cast<float>(st.Z - static_cast<double>(g.zh));
    chunk_weights<T>(a, row, c, g, s_table, w, col0);
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < VL_GROUPS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += w[i][e];
    sum = warp_sum(sum);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      int64_t t = 0;
      for (int k = 0; k < VERIFY_WARPS; ++k) t += s_sum[k];
      __stcg(reinterpret_cast<long long*>(a.rsum) + static_cast<int64_t>(seq) * a.nchunk + c, t);
      __threadfence();
      s_last = atomicAdd(a.done + seq, 1u) == static_cast<uint32_t>(a.nchunk - 1);
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const long long* rs = reinterpret_cast<const long long*>(a.rsum) + static_cast<int64_t>(seq) * a.nchunk;
    if (tid < a.nchunk) s_w[tid] = __longlong_as_double(__ldcg(rs + tid));
    __syncthreads();
    if (tid == 0) {
      int64_t total = 0;
      for (int k = 0; k < a.nchunk; ++k) total += __double_as_longlong(s_w[k]);
      const double t = static_cast<double>(u) * static_cast<double>(total);
      int64_t upto = 0;
      int at = -1;
      double left = 0.0;
      for (int k = 0; k < a.nchunk && total > 0; ++k) {
        const int64_t s = __double_as_longlong(s_w[k]);
        if (s > 0) {
          at = k;
          left = t - static_cast<double>(upto);
          if (static_cast<double>(upto + s) > t) break;
        }
        upto += s;
      }
      s_chunk = at;
      s_t = left;
    }
    __syncthreads();
    if (s_chunk >= 0) {
      if (s_chunk != c) chunk_weights<T>(a, row, s_chunk, g, s_table, w, col0);
      const int col = find_column(w, col0, s_t, s_sum, &s_col);
      if (tid == 0) a.tokens[row] = col;
      return;
    }
    g.mode = DRAW_P;  // q covers P: the draw is from P itself, by this CTA
  }

  const bool alone = st.refused && a.q.p;  // the last CTA of a residual without weight does any chunk
  g.shift = VL_SHIFT;
  __syncthreads();
  // chunk sums relative to the row's maximum, a one-hot draft's own weight taken out of its chunk's
  if (tid < a.nchunk) {
    const ChunkStat k = cs[tid];
    int64_t own = 0;
    if (g.mode == DRAW_OTHERS && g.x >= 0 && g.x < a.V) {
      const T* lrow = static_cast<const T*>(a.logits) + row * a.ld;
      const int k0 = chunk_col(lrow, tid);
      if (g.x >= k0 && g.x < k0 + VL_CHUNK) {
        const float l = widen<T>(lrow[g.x]);
        if (l > -INFINITY) own = exp_fixed(l, k.max, g.sc, s_table, VL_SHIFT);
      }
    }
    const double f = ldexp(exp_double(k.max, st.max, g.sc, s_table), -VL_SHIFT);
    s_f[tid] = f;
    s_w[tid] = static_cast<double>(k.sum - own) * f;
    s_all[tid] = static_cast<double>(k.sum) * f;
  }
  __syncthreads();
  if (tid == 0) {
    const double* ws = s_w;
    double total = 0.0;
    for (int k = 0; k < a.nchunk; ++k) total += ws[k];
    if (!(total > 0.0)) {  // the draft holds all of P (a refusal by an a of 1 or more): from P
      g.mode = DRAW_P;
      ws = s_all;
      total = 0.0;
      for (int k = 0; k < a.nchunk; ++k) total += ws[k];
    }
    const double t = static_cast<double>(u) * total;
    double upto = 0.0;
    int at = -1;
    double left = 0.0, f = 1.0;
    for (int k = 0; k < a.nchunk; ++k) {
      if (ws[k] > 0.0) {
        at = k;
        left = t - upto;
        f = s_f[k];
        if (upto + ws[k] > t) break;
      }
      upto += ws[k];
    }
    s_chunk = at;
    s_t = left / f;
    s_last = g.mode;
  }
  __syncthreads();
  g.mode = s_last;
  const int at = s_chunk;
  if (at < 0) {
    if ((c == 0 || alone) && tid == 0) a.tokens[row] = -1;
    return;
  }
  if (!alone && at != c) return;
  g.max = cs[at].max;
  chunk_weights<T>(a, row, at, g, s_table, w, col0);
  const int col = find_column(w, col0, s_t, s_sum, &s_col);
  if (tid == 0) a.tokens[row] = col;
}

int64_t round256(int64_t v) { return (v + 255) & ~int64_t(255); }

int chunks(int V) { return (V + 3 + VL_CHUNK - 1) / VL_CHUNK; }

template <typename T>
cudaError_t launch(const LogitsArgs& a, int shift, cudaStream_t stream) {
  if (a.rows > 0) {
    verify_stats_kernel<T><<<dim3(a.nchunk, a.rows), VERIFY_THREADS, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  verify_draw_kernel<T><<<dim3(a.nchunk, a.nseq), VERIFY_THREADS, 0, stream>>>(a, shift);
  return cudaGetLastError();
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
  const int64_t nc = chunks(V);
  *bytes = round256(rows * nc * static_cast<int64_t>(sizeof(ChunkStat))) + round256(nseq * nc * 8) +
           round256(nseq * 4LL);
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
  a.dtype = logits_dtype;
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
  uint8_t* p = static_cast<uint8_t*>(workspace);
  a.stats = reinterpret_cast<ChunkStat*>(p);
  p += round256(rows * static_cast<int64_t>(a.nchunk) * static_cast<int64_t>(sizeof(ChunkStat)));
  a.rsum = reinterpret_cast<int64_t*>(p);
  p += round256(nseq * static_cast<int64_t>(a.nchunk) * 8);
  a.done = reinterpret_cast<uint32_t*>(p);
  a.tokens = out_tokens;
  a.count = out_count;
  int bits = 0;
  while ((int64_t(1) << bits) < V) ++bits;
  const int shift = 62 - bits < 44 ? 62 - bits : 44;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == TAIL_F32   ? launch<float>(a, shift, s)
                        : logits_dtype == TAIL_F16 ? launch<__half>(a, shift, s)
                                                   : launch<__nv_bfloat16>(a, shift, s);
  if (e != cudaSuccess) return cuda_fail(e, "tail_verify_logits: kernel launch");
  return TAIL_OK;
}
