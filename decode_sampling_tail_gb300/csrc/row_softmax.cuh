// Row passes of the training operators on vocabulary logits (token_logprobs.cu, policy_loss.cu,
// preference_loss.cu, distill_topk.cu): a row's softmax statistics and its gradient, the row split over
// the CTAs of a cluster.
//
// What bounds them is memory: 10 to 12 instructions a column leave HBM the limit of large calls, and the latency of a
// CTA's chain (token, statistics, exchange, factors, gradient) that of small ones.  A loss that depends on its row
// alone reads the row from HBM once: the statistics' pass is followed at once by the gradient's, which finds the
// row in L2, as long as no more than ROW_FLIGHT bytes of rows are under way, or in shared memory when all of a call's rows fit
// there.  Measured at 2048 rows of 201088 columns (1.57 GB of bf16 read and written): 253 us, 0.93 of the copy rate.  Before:
// parts in shared memory by 2 CTAs an SM 341 us; 4 CTAs of 256 threads an SM that read twice 295; each part brought to
// L2 by one bulk prefetch 266; the exchange without cluster barriers, first loads ahead of their need 256; loads a batch
// ahead in the statistics 253.  Persistent CTAs that fetch their next row into shared memory while they write the present
// one's gradient took 337 to 438: one or two CTAs an SM do not cover the chain.
//
// Statistics.  With m the row's maximum and a_v = (z_v - m) log2(e) / T <= 0:
//   s = sum of 2^a_v over every column but one at the maximum,  u = sum of a_v 2^a_v  (fp32).
// One instance of the maximum stays out of s, since its weight 1 would swallow what the others add up to: with
// it apart, -log1p(s) is a likely token's log-probability and s / (1 + s) its distance from 1 to a few
// units of 2^-24 of themselves.  It costs a minimum a column: a running pair of maxima keeps the
// larger of each two values, and the smaller one goes into the sum, so that every value but the
// maxima enters exactly once.  The sums are taken 16 or 32 columns at a time against the maximum so far, and a batch's own
// sum enters the running one by one fused operation, which also takes a change of the maximum.  So a term passes at most 8 or
// 16 additions in its batch, one a batch behind it (25 of fp32, 13 of 16 bits at 201088 columns and 512 threads), and 19
// merges of pairs, lanes, warps and CTAs, each 2^-24 of the sum; with its exponential (2^-22) and its argument's three
// roundings (20 ln 2 of 3 2^-24 in the mean) s is within 2^-17 of itself up to 2^18 columns, 2^-16 up to 2^20.  Measured, from
// 32000 to 2^20 columns of all spreads: 2^-20.7 at most.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <math.h>
#include <stdint.h>

#include "abi_common.h"
#include "common.cuh"

namespace tail {

constexpr int ROW_BATCH = 4;            // vectors a thread takes at a time
constexpr int ROW_MAX_CLUSTER = 8;      // CTAs a row, the portable size
constexpr int ROW_SMEM = 224 * 1024;    // dynamic shared memory of a CTA at most
constexpr uint64_t ROW_WAIT_NS = 1000000000ull;  // how long a row's CTAs wait for one another, if not set otherwise

// ---------------------------------------------------------------- arithmetic

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{\n.reg .b64 p, q;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %5};\nadd.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{\n.reg .b64 p, q;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %5};\nmul.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{\n.reg .b64 p, q, r;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %5};\nmov.b64 r, {%6, %7};\n"
      "fma.rn.f32x2 p, p, q, r;\nmov.b64 {%0, %1}, p;\n}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}

// ---------------------------------------------------------------- 16-byte vectors as pairs of columns

template <typename T>
struct Vec;

template <>
struct Vec<float> {
  static constexpr int N = 4, PAIRS = 2;
  using Pair = float2;
  static __device__ __forceinline__ Pair pair(const uint4& v, int i) {
    return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                  : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ Pair lowest() { return make_float2(-INFINITY, -INFINITY); }
  static __device__ __forceinline__ Pair hi(Pair a, Pair b) { return make_float2(max_nan(a.x, b.x), max_nan(a.y, b.y)); }
  static __device__ __forceinline__ Pair lo(Pair a, Pair b) { return make_float2(min_nan(a.x, b.x), min_nan(a.y, b.y)); }
  static __device__ __forceinline__ float2 widen(Pair p) { return p; }
  static __device__ __forceinline__ void set(uint4& v, int i, float2 f) {
    if (i == 0)
      v.x = __float_as_uint(f.x), v.y = __float_as_uint(f.y);
    else
      v.z = __float_as_uint(f.x), v.w = __float_as_uint(f.y);
  }
  static __device__ __forceinline__ float widen1(float v) { return v; }
  static __device__ __forceinline__ float narrow1(float v) { return v; }
  // columns whose bit is set become -inf
  static __device__ __forceinline__ void mask(uint4& v, uint32_t bits) {
    if (bits & 1) v.x = 0xff800000u;
    if (bits & 2) v.y = 0xff800000u;
    if (bits & 4) v.z = 0xff800000u;
    if (bits & 8) v.w = 0xff800000u;
  }
};

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ void set_word(uint4& v, int i, uint32_t w) {
  if (i == 0) v.x = w;
  if (i == 1) v.y = w;
  if (i == 2) v.z = w;
  if (i == 3) v.w = w;
}
template <uint32_t LOWEST>
__device__ __forceinline__ void mask16(uint4& v, uint32_t bits) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w = word(v, i);
    if (bits & (1u << 2 * i)) w = (w & 0xffff0000u) | LOWEST;
    if (bits & (2u << 2 * i)) w = (w & 0xffffu) | (LOWEST << 16);
    set_word(v, i, w);
  }
}

template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8, PAIRS = 4;
  using Pair = __nv_bfloat162;
  static __device__ __forceinline__ Pair pair(const uint4& v, int i) {
    const uint32_t w = word(v, i);
    return reinterpret_cast<const Pair&>(w);
  }
  static __device__ __forceinline__ Pair lowest() {
    const uint32_t w = 0xff80ff80u;
    return reinterpret_cast<const Pair&>(w);
  }
  static __device__ __forceinline__ Pair hi(Pair a, Pair b) { return __hmax2_nan(a, b); }
  static __device__ __forceinline__ Pair lo(Pair a, Pair b) { return __hmin2_nan(a, b); }
  static __device__ __forceinline__ float2 widen(Pair p) {
    const uint32_t w = reinterpret_cast<const uint32_t&>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ void set(uint4& v, int i, float2 f) {
    const Pair p = __float22bfloat162_rn(f);
    set_word(v, i, reinterpret_cast<const uint32_t&>(p));
  }
  static __device__ __forceinline__ float widen1(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 narrow1(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void mask(uint4& v, uint32_t bits) { mask16<0xff80u>(v, bits); }
};

template <>
struct Vec<__half> {
  static constexpr int N = 8, PAIRS = 4;
  using Pair = __half2;
  static __device__ __forceinline__ Pair pair(const uint4& v, int i) {
    const uint32_t w = word(v, i);
    return reinterpret_cast<const Pair&>(w);
  }
  static __device__ __forceinline__ Pair lowest() {
    const uint32_t w = 0xfc00fc00u;
    return reinterpret_cast<const Pair&>(w);
  }
  static __device__ __forceinline__ Pair hi(Pair a, Pair b) { return __hmax2_nan(a, b); }
  static __device__ __forceinline__ Pair lo(Pair a, Pair b) { return __hmin2_nan(a, b); }
  static __device__ __forceinline__ float2 widen(Pair p) { return __half22float2(p); }
  static __device__ __forceinline__ void set(uint4& v, int i, float2 f) {
    const Pair p = __float22half2_rn(f);
    set_word(v, i, reinterpret_cast<const uint32_t&>(p));
  }
  static __device__ __forceinline__ float widen1(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half narrow1(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ void mask(uint4& v, uint32_t bits) { mask16<0xfc00u>(v, bits); }
};

// ---------------------------------------------------------------- statistics

// The statistics of a set of columns: maximum (-inf for none, NaN when a column is), and the sums
// without one instance of it.
struct RowStat {
  float m, s, u;
};

// Log2-domain distance of a maximum (or logit) from a larger one, cut at -200, where 2^d is 0 in
// fp32: keeps 0 * -inf out of u.  (NaN stays.)
__device__ __forceinline__ float dist(float z, float ref, float k) { return max_nan((z - ref) * k, -200.f); }

__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ RowStat merge(const RowStat& a, const RowStat& b, float k) {
  RowStat r;
  r.m = max_nan(a.m, b.m);
  const bool first = a.m >= b.m;
  const float low = first ? b.m : a.m;
  const float d = dist(low, finite_ref(r.m), k);
  const float c = ex2(d);
  const float sl = first ? b.s : a.s, ul = first ? b.u : a.u;
  r.s = (first ? a.s : b.s) + c * (1.f + sl);
  r.u = (first ? a.u : b.u) + c * (ul + d * (1.f + sl));
  return r;
}

__device__ __forceinline__ RowStat stat_of(float z) { return RowStat{z, 0.f, 0.f}; }
__device__ __forceinline__ RowStat no_stat() { return RowStat{-INFINITY, 0.f, 0.f}; }

// A thread's running statistics.
template <typename T, bool ENT>
struct RowAcc {
  using V = Vec<T>;
  typename V::Pair top = V::lowest();  // the two maxima so far, in neither sum
  float m = -INFINITY;                 // what the sums refer to
  float2 s = {0.f, 0.f}, u = {0.f, 0.f};

  template <int U>
  __device__ __forceinline__ void batch(const uint4 (&v)[U], float k) {
    typename V::Pair w[U * V::PAIRS];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < V::PAIRS; ++j) {
        const typename V::Pair p = V::pair(v[i], j);
        w[i * V::PAIRS + j] = V::lo(p, top);
        top = V::hi(p, top);
      }
    const float2 t = V::widen(top);
    const float mx = max_nan(t.x, t.y), ref = finite_ref(mx);
    const float d = dist(m, ref, k), c = ex2(d);
    m = mx;
    if (ENT) u = fma2(s, make_float2(d, d), u);
    const float2 off = {-ref, -ref}, kk = {k, k};
    float2 sb, ub;  // the batch's own sums: one addition a batch to the running ones, however many columns it has
#pragma unroll
    for (int i = 0; i < U * V::PAIRS; ++i) {
      float2 a = mul2(add2(V::widen(w[i]), off), kk);
      if (ENT) a.x = max_nan(a.x, -200.f), a.y = max_nan(a.y, -200.f);
      const float2 e = {ex2(a.x), ex2(a.y)};
      sb = i ? add2(sb, e) : e;
      if (ENT) ub = i ? fma2(e, a, ub) : mul2(e, a);
    }
    s = fma2(s, make_float2(c, c), sb);
    if (ENT) u = fma2(u, make_float2(c, c), ub);
  }

  __device__ __forceinline__ RowStat done(float k) const {
    const float2 t = V::widen(top);
    RowStat r{m, s.x + s.y, u.x + u.y};
    const float d = dist(fminf(t.x, t.y), finite_ref(m), k), c = ex2(d);
    r.s += c;
    r.u += c * d;
    return r;
  }
};

__device__ __forceinline__ float warp_max(float v) {  // NaN when any is
  float y;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(v));
  return y;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The statistics of a warp's lanes, the same bits in every lane: they are brought to the common maximum once, and
// the first lane that holds it gives the instance that stays out of the sum.
template <bool ENT>
__device__ __forceinline__ RowStat warp_merge(const RowStat& v, float k) {
  RowStat r{warp_max(v.m), 0.f, 0.f};
  const uint32_t at = __ballot_sync(0xffffffffu, v.m == r.m);
  const bool out = static_cast<int>(threadIdx.x & 31) == __ffs(at) - 1;
  const float d = dist(v.m, finite_ref(r.m), k), c = ex2(d);
  r.s = warp_sum(c * (v.s + (out ? 0.f : 1.f)));
  if (ENT) r.u = warp_sum(c * (v.u + d * (1.f + v.s)));
  return r;
}

// ---------------------------------------------------------------- a row's part of a CTA

// The columns of a row as a CTA sees them: whole vectors [first, first + count), and single columns
// in front of the row's first vector (rank 0) or behind its last (last rank).
struct RowPart {
  int head;   // columns in front of the first vector
  int nvec;   // whole vectors of the row
  int first;  // this CTA's first vector
  int count;
  int edge_lo, edge_n;  // this thread's single column, if edge_n: its index
};

template <typename T>
__device__ __forceinline__ RowPart row_part(const T* row, int V, int rank, int size) {
  constexpr int N = Vec<T>::N;
  RowPart p;
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / static_cast<int>(sizeof(T));
  p.head = min(mis ? N - mis : 0, V);
  p.nvec = (V - p.head) / N;
  const int per = (p.nvec + size - 1) / size;
  p.first = min(per * rank, p.nvec);
  p.count = min(per, p.nvec - p.first);
  const int tid = threadIdx.x, tail = V - p.head - p.nvec * N;
  p.edge_n = 0;
  p.edge_lo = 0;
  if (rank == 0 && tid < p.head) {
    p.edge_n = 1;
    p.edge_lo = tid;
  }
  if (rank == size - 1 && tid >= N && tid - N < tail) {
    p.edge_n = 1;
    p.edge_lo = p.head + p.nvec * N + tid - N;
  }
  return p;
}

// Whether a column of the row is this CTA's.
template <typename T>
__device__ __forceinline__ bool has_column(const RowPart& p, int rank, int size, int col) {
  const int lo = p.head + p.first * Vec<T>::N;
  return (col >= lo || rank == 0) && (col < lo + p.count * Vec<T>::N || rank == size - 1);
}

// ---------------------------------------------------------------- asynchronous copies of a thread's own vectors

__device__ __forceinline__ void copy_async16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `left` of the thread's groups are under way (7 stands for 7 and more).
__device__ __forceinline__ void copy_wait(int left) {
  switch (left < 7 ? left : 7) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}

// ---------------------------------------------------------------- cluster

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Says that this CTA has started (and what thread 0 has initialised); the others' shared memory may be written behind the
// wait.  Both stand at a kernel's start, beside its first loads: a wait has every warp invalidate L1, one after another,
// about 1 us for 8 warps where the row's statistics would wait for it.
__device__ __forceinline__ void cluster_started() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Writes four words to the same shared variable of CTA `rank` of the cluster, and counts their bytes on its barrier.
__device__ __forceinline__ void store_remote(float4* mine, uint64_t* bar, int rank, float4 v) {
  uint32_t at, to;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(to)
               : "memory");
}

// Where a cluster's CTAs leave W words of four each for one another, by their first warps alone.
template <int W>
struct Board {
  float4 warp[W][16];              // this CTA's warps'
  float4 cta[W][ROW_MAX_CLUSTER];  // the CTAs'
  uint64_t bar;

  // All threads, at the start; then cluster_started().
  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      mbar_init(smem_u32(&bar), 1);
      fence_mbar_init();
    }
  }
  __device__ __forceinline__ bool arrived() {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(&bar))
        : "memory");
    return ok != 0;
  }
  // (0: one look, since arrived() may itself wait for as long as the device sees fit)
  __device__ __forceinline__ bool wait(uint64_t ns) {
    if (ns == 0) {
      uint32_t ok;
      asm volatile(
          "{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\nselp.u32 %0, 1, 0, p;\n}"
          : "=r"(ok)
          : "r"(smem_u32(&bar))
          : "memory");
      return ok != 0;
    }
    if (arrived()) return true;
    const uint64_t since = global_timer_ns();
    while (!arrived())
      if (global_timer_ns() - since > ns) return false;
    return true;
  }
  // The first warp: its CTA's words to every CTA (ALL) or to the first, and in return all the CTAs', lane i CTA i's.
  // False when they have not come in wait_ns; then leave() has to end the kernel for this warp.
  template <bool ALL>
  __device__ __forceinline__ bool exchange(int rank, int size, const float4 (&mine)[W], float4 (&all)[W],
                                           uint64_t wait_ns) {
    const int lane = threadIdx.x & 31;
    if (lane == 0 && (ALL || rank == 0)) mbar_arrive_expect_tx(smem_u32(&bar), size * W * sizeof(float4));
    if (ALL ? lane < size : lane == 0)
#pragma unroll
      for (int w = 0; w < W; ++w) store_remote(&cta[w][rank], &bar, lane, mine[w]);
    __syncwarp();
    if (!ALL && rank != 0) return true;
    const bool ok = __all_sync(0xffffffffu, wait(wait_ns));
#pragma unroll
    for (int w = 0; w < W; ++w) all[w] = lane < size ? cta[w][lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    return ok;
  }
  // The first warp's last step where its wait has run out, behind every barrier of its CTA: the others may still write to
  // this CTA's shared memory, which goes when the CTA ends.  It stays until every thread of the cluster has ended or waits
  // here too, so that all of them have sent what they send, and then until that has come.  (The barrier counts ended threads
  // as arrived; nobody else waits for it, and every other wait is bounded.)
  __device__ __forceinline__ void leave() {
    if (cluster_size() == 1) return;
    cluster_started();
    cluster_wait();
    wait(ROW_WAIT_NS);
  }
};

// The cluster's statistics in the first warp of every CTA (ALL) or of the first, from each thread's; the same bits in all
// lanes.  NaN when another CTA's have not come in wait_ns (ALL: the first warp ends by board.leave()).  Ends without a
// barrier.  `seen`: what the first warp has read of the
// row's other parts; it goes with its statistics, so that a CTA that has all of them may write its part in place.
template <bool ENT, bool ALL>
__device__ __forceinline__ RowStat cluster_stat(Board<1>& board, RowStat st, float seen, float k, int rank, int size,
                                                uint64_t wait_ns) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  st = warp_merge<ENT>(st, k);
  if (lane == 0) board.warp[0][warp] = make_float4(st.m, st.s, st.u, 0.f);
  __syncthreads();
  if (warp != 0) return st;
  st = no_stat();
  if (lane < static_cast<int>(blockDim.x >> 5)) {
    const float4 x = board.warp[0][lane];
    st = RowStat{x.x, x.y, x.z};
  }
  st = warp_merge<ENT>(st, k);
  if (size == 1) return st;
  const float4 mine[1] = {make_float4(st.m, st.s, st.u, seen)};
  float4 all[1];
  const bool ok = board.template exchange<ALL>(rank, size, mine, all, wait_ns);
  if (!ALL && rank != 0) return st;
  st = warp_merge<ENT>(RowStat{all[0].x, all[0].y, all[0].z}, k);
  if (!ok) {
    st.m = st.s = st.u = NAN;
    if (!ALL) board.leave();  // (the other warps are done)
  }
  return st;
}

// ---------------------------------------------------------------- gradient

// dz_v = e (A + B a) at the columns, e = 2^a, a = (z_v - ref) k; `at_token` replaces it at column `token`.
struct RowGrad {
  float ref, k, A, B, at_token;
  int token;
};

template <typename T, bool ENT>
__device__ __forceinline__ float grad1(const RowGrad& g, T z) {
  float a = (Vec<T>::widen1(z) - g.ref) * g.k;
  if (ENT) a = max_nan(a, -200.f);
  return ENT ? ex2(a) * fmaf(g.B, a, g.A) : ex2(a) * g.A;
}

template <typename T, bool ENT>
__device__ __forceinline__ uint4 grad_vec(const RowGrad& g, const uint4& z) {
  using V = Vec<T>;
  uint4 out;
  const float2 off = {-g.ref, -g.ref}, kk = {g.k, g.k}, A = {g.A, g.A}, B = {g.B, g.B};
#pragma unroll
  for (int j = 0; j < V::PAIRS; ++j) {
    float2 a = mul2(add2(V::widen(V::pair(z, j)), off), kk);
    if (ENT) a.x = max_nan(a.x, -200.f), a.y = max_nan(a.y, -200.f);
    const float2 e = {ex2(a.x), ex2(a.y)};
    V::set(out, j, ENT ? mul2(e, fma2(B, a, A)) : mul2(e, A));
  }
  return out;
}

// Whether a row's gradient lies on the same whole vectors as its logits.
__device__ __forceinline__ bool same_phase(const void* a, const void* b) {
  return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

// Zeros over this CTA's part of a row of the gradient.
template <typename T>
__device__ __forceinline__ void zero_part(T* grad, int V, int rank, int size) {
  const RowPart p = row_part(grad, V, rank, size);
  uint4* at = reinterpret_cast<uint4*>(grad + p.head) + p.first;
  for (int i = threadIdx.x; i < p.count; i += blockDim.x) __stcs(at + i, make_uint4(0, 0, 0, 0));
  if (p.edge_n) grad[p.edge_lo] = Vec<T>::narrow1(0.f);
}

// This thread's single column of a part, if it has one.
template <typename T>
__device__ __forceinline__ float edge_of(const T* row, const RowPart& p) {
  return p.edge_n ? Vec<T>::widen1(row[p.edge_lo]) : -INFINITY;
}

template <typename T>
__device__ __forceinline__ const uint4* part_vectors(const T* row, const RowPart& p) {
  return reinterpret_cast<const uint4*>(row + p.head) + p.first;
}

// ---------------------------------------------------------------- passes over a part
// A thread takes vectors tid, tid + NT, .. of the part, ROW_BATCH of them at a time; in all passes the same ones, so
// that its copies into shared memory need no barrier.  Whole batches run without a bound in sight: with one, and a
// token to look for, a vector cost more instructions than its columns' arithmetic.  A part is kept in shared memory
// whole or not at all; what is not kept is read from L2 in each pass, into which one instruction has brought it.  A pass over
// memory gets its first batch from the caller, who loads it before whatever else the pass has to wait for.

__host__ __device__ constexpr int batches(int n, int nt) { return (n + ROW_BATCH * nt - 1) / (ROW_BATCH * nt); }

// Requests the whole part into shared memory, each vector by the thread that takes it, one group a batch.
template <typename T, int NT>
__device__ __forceinline__ void fetch_part(const T* row, const RowPart& p, uint4* cache) {
  const uint4* in = part_vectors(row, p);
  for (int b = 0; b < batches(p.count, NT); ++b) {
    const int end = min((b + 1) * ROW_BATCH * NT, p.count);
    for (int i = b * ROW_BATCH * NT + static_cast<int>(threadIdx.x); i < end; i += NT) copy_async16(cache + i, in + i);
    copy_commit();
  }
}

// Has the part, from vector `from` on, brought into L2, by one instruction of one thread: the loads behind it then wait for
// L2 alone.
template <typename T>
__device__ __forceinline__ void prefetch_part(const T* row, const RowPart& p, int from) {
  if (threadIdx.x == 0 && p.count > from)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(part_vectors(row, p) + from),
                 "r"((p.count - from) * 16)
                 : "memory");
}

// A load of what is not needed again: its place in L2 goes first.
__device__ __forceinline__ uint4 load_last(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy_evict_first())
               : "memory");
  return v;
}

// A thread's vectors of a batch.
struct Batch {
  uint4 v[ROW_BATCH];

  // Batch b of n vectors in memory; zeros, unread, behind the end.
  template <int NT, bool LAST = false>
  static __device__ __forceinline__ Batch from(const uint4* in, int b, int n) {
    Batch x;
    const int i0 = b * ROW_BATCH * NT + static_cast<int>(threadIdx.x);
    const uint4* at = in + i0;
    if ((b + 1) * ROW_BATCH * NT <= n) {
#pragma unroll
      for (int j = 0; j < ROW_BATCH; ++j) x.v[j] = LAST ? load_last(at + j * NT) : __ldcg(at + j * NT);
    } else {
#pragma unroll
      for (int j = 0; j < ROW_BATCH; ++j)
        x.v[j] = i0 + j * NT >= n ? make_uint4(0, 0, 0, 0) : LAST ? load_last(at + j * NT) : __ldcg(at + j * NT);
    }
    return x;
  }
};

// Columns that count as -inf: flags(b) of this thread's batch b has a bit a vector with any, bits(i) the columns of
// vector i.
struct NoMask {
  __device__ __forceinline__ uint32_t flags(int) const { return 0; }
  __device__ __forceinline__ uint32_t bits(int) const { return 0; }
};

template <typename T, bool ENT, int NT, typename Mask>
__device__ __forceinline__ void stat_batch(RowAcc<T, ENT>& acc, uint4 (&v)[ROW_BATCH], int b, float k,
                                           const Mask& mask) {
  const uint32_t f = mask.flags(b);
  if (f)
#pragma unroll
    for (int j = 0; j < ROW_BATCH; ++j)
      if (f & (1u << j))
        Vec<T>::mask(v[j], mask.bits((b * ROW_BATCH + j) * NT + static_cast<int>(threadIdx.x)));
  acc.batch(v, k);
}

template <typename T, bool ENT, int NT, typename Mask>
__device__ __forceinline__ void stat_single(RowAcc<T, ENT>& acc, const uint4& z, int i, float k, const Mask& mask) {
  uint4 v[1] = {z};
  const uint32_t m = mask.bits(i);
  if (m) Vec<T>::mask(v[0], m);
  acc.batch(v, k);
}

// Statistics over this CTA's part, without the thread's single column: from shared memory as its copies arrive (the
// thread has no other copies under way), or from memory with the first batch in x.
template <typename T, bool ENT, int NT, typename Mask>
__device__ __forceinline__ RowStat stat_pass(const T* row, const RowPart& p, const uint4* cache, Batch& x, float k,
                                             const Mask& mask) {
  constexpr int U = ROW_BATCH;
  const int tid = threadIdx.x, whole = p.count / (U * NT), all = batches(p.count, NT);
  RowAcc<T, ENT> acc;
  if (cache) {
    const uint4* c = cache + tid;
    for (int b = 0; b < whole; ++b, c += U * NT) {
      copy_wait(all - 1 - b);
      uint4 v[U];
#pragma unroll
      for (int j = 0; j < U; ++j) v[j] = c[j * NT];
      stat_batch<T, ENT, NT>(acc, v, b, k, mask);
    }
    copy_wait(0);
    for (int i = whole * U * NT + tid; i < p.count; i += NT) stat_single<T, ENT, NT>(acc, cache[i], i, k, mask);
  } else {
    const uint4* in = part_vectors(row, p);
    for (int b = 0; b + 1 < all; ++b) {  // a batch is under way while the one before it is taken
      const Batch n = Batch::from<NT>(in, b + 1, p.count);
      stat_batch<T, ENT, NT>(acc, x.v, b, k, mask);
      x = n;
    }
    if (whole == all) {
      if (all > 0) stat_batch<T, ENT, NT>(acc, x.v, all - 1, k, mask);
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = (whole * U + j) * NT + tid;
        if (i < p.count) stat_single<T, ENT, NT>(acc, x.v[j], i, k, mask);
      }
    }
  }
  return acc.done(k);
}

// A row whose gradient is written, and where its part is kept (or null).
template <typename T>
struct GradRow {
  const T* row;
  T* grad;
  RowPart p;
  const uint4* cache;
  float edge;
};

// The gradient over this CTA's part of a row, from shared memory or from memory with the first batch in x.  Rows whose
// gradient lies elsewhere in its 16-byte vectors are written column by column; then what is kept must be visible
// to all threads.  DEEP: a batch is under way while the one before it is written.
template <typename T, bool ENT, int NT, bool LAST = false, bool DEEP = false>
__device__ __forceinline__ void grad_pass(const RowGrad& g, const GradRow<T>& r, Batch& x) {
  constexpr int N = Vec<T>::N, U = ROW_BATCH;
  const int tid = threadIdx.x;
  const RowPart& p = r.p;
  const int body = p.head + p.first * N;  // the part's first column in a vector
  if (same_phase(r.row, r.grad)) {
    const int whole = p.count / (U * NT), all = batches(p.count, NT);
    uint4* out = reinterpret_cast<uint4*>(r.grad + p.head) + p.first + tid;
    const uint4* in = part_vectors(r.row, p);
    const uint4* c = r.cache + tid;
    int b = 0;
    if (r.cache) {
      for (; b < whole; ++b, c += U * NT, out += U * NT) {
#pragma unroll
        for (int j = 0; j < U; ++j) x.v[j] = c[j * NT];
#pragma unroll
        for (int j = 0; j < U; ++j) __stcs(out + j * NT, grad_vec<T, ENT>(g, x.v[j]));
      }
#pragma unroll
      for (int j = 0; j < U; ++j)
        if ((whole * U + j) * NT + tid < p.count) x.v[j] = c[j * NT];
    } else {
      for (; b + 1 < all; ++b, out += U * NT) {
        if constexpr (DEEP) {
          const Batch n = Batch::from<NT, LAST>(in, b + 1, p.count);
#pragma unroll
          for (int j = 0; j < U; ++j) __stcs(out + j * NT, grad_vec<T, ENT>(g, x.v[j]));
          x = n;
        } else {
#pragma unroll
          for (int j = 0; j < U; ++j) __stcs(out + j * NT, grad_vec<T, ENT>(g, x.v[j]));
          x = Batch::from<NT, LAST>(in, b + 1, p.count);
        }
      }
      if (whole == all && all > 0) {
#pragma unroll
        for (int j = 0; j < U; ++j) __stcs(out + j * NT, grad_vec<T, ENT>(g, x.v[j]));
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
      if ((whole * U + j) * NT + tid < p.count) __stcs(out + j * NT, grad_vec<T, ENT>(g, x.v[j]));
    // the token's column, by the thread that has written its vector
    const int tv = g.token >= body ? (g.token - body) / N : -1;
    if (tv >= 0 && tv < p.count && tv % NT == tid) r.grad[g.token] = Vec<T>::narrow1(g.at_token);
  } else {
    const T* c = r.cache ? reinterpret_cast<const T*>(r.cache) : r.row + body;
    for (int i = tid; i < p.count * N; i += NT)
      r.grad[body + i] = Vec<T>::narrow1(body + i == g.token ? g.at_token : grad1<T, ENT>(g, c[i]));
  }
  if (p.edge_n)
    r.grad[p.edge_lo] =
        Vec<T>::narrow1(p.edge_lo == g.token ? g.at_token : grad1<T, ENT>(g, Vec<T>::narrow1(r.edge)));
}

// ---------------------------------------------------------------- host side

// How a row is split, and whether its parts stay in shared memory between the passes.
struct RowPlan {
  int size;     // CTAs a row
  int threads;  // 512, 256 or 128, 1024 of them a SM
  int kept;     // vectors of a part, if shared memory keeps them; 0: it does not
};

constexpr int ROW_SMS = 152;  // the device that this is written for
constexpr int ROW_SM_THREADS = 1024;

inline int64_t row_vectors(int V, int es) { return (static_cast<int64_t>(V) * es + 15) / 16; }
inline int64_t part_of(int64_t vecs, int size) { return (vecs + size - 1) / size; }

// Bytes of rows that may be in flight at once.  What a first pass has read, or a prefetch has brought, is there for the
// pass behind it as long as it fits L2 beside the gradient that is written.
constexpr int64_t ROW_FLIGHT = 62 << 20;

// Splits rows over more CTAs while the device is not full: few rows down to two vectors a thread, more
// of them for an even end, down to `least` vectors a thread.  Measured in bf16 at 50021 columns, a CTA a row against two:
// gradients from log-sum-exps 18.6, 17.0 us (500 rows) and 29.3, 25.0 (777), the policy loss 24.0, 23.9 and 35.6, 33.7, so
// they split from 8 vectors a thread; distillation with 64 entries 27.5, 32.0 and 41.5, 44.9, since each part goes through
// the whole list: from 16.
inline void fill_device(RowPlan& p, int64_t rows, int64_t vecs, int least) {
  const int slots = ROW_SMS * (ROW_SM_THREADS / p.threads);
  for (; p.size < ROW_MAX_CLUSTER; p.size *= 2) {
    const int64_t part = vecs / (2 * p.size);
    const bool few = rows * p.size < 2 * ROW_SMS && part >= 2 * p.threads;
    const bool uneven = rows * p.size < 2 * slots && part >= least * p.threads;
    if (!few && !uneven) break;
  }
}

// Rows that pass once, without a prefetch.  More threads a row shorten a CTA's chain, fewer leave less of a batch empty.
// Measured in bf16, by 512, 256 and 128 threads a CTA, one a row: 1536 rows of 201088 98, 96 and 109 us; 777 of 50021 18.2,
// 17.2, 15.1; 2000 of 32000 29, 24, 22; 4096 of 8192 33, 17, 14.5; 700 of 515 5.5, 3.5, 2.3; and 100 of 201088 by CTAs of 512
// two a row 10.0, of 256 four 9.4, of 128 eight 9.4.  (So the two borders lie high: 2 to 20 % behind the best.)
inline RowPlan plan_stream(int64_t rows, int V, int es) {
  const int64_t vecs = row_vectors(V, es);
  RowPlan p = {1, vecs >= 4096 ? 512 : vecs >= 1024 ? 256 : 128, 0};
  fill_device(p, rows, vecs, 8);
  return p;
}

// Rows that are prefetched, and kept or read again.  `beside`: bytes of shared memory of a CTA beside what is kept
// (negative: nothing is kept).  Measured for the policy loss in bf16, by 256 and 128 threads a CTA, one a row: 2000 rows of
// 32000 46, 54 us; 3000 of 16000 38.7, 35.7; 4096 of 8192 34, 26.6; 300 of 16000 (all at once) 7.2, 8.3; 700 of 515 5.9, 3.4.
// Bounded by ROW_FLIGHT, or split half as far: 1536 rows of 201088 200, 304; 400 62, 87; gradients from log-sum-exps, which
// read a row once, gain too, since a prefetch is then less far ahead of its use: 186, 225 and 51, 63.  Kept, or not: 300 rows
// of 16000 6.9, 7.2; 333 of 50021 19.6, 19.5.  (Whether a call's parts fit is counted of all of them, not of
// those that run at once: 4096 rows of 8192 would gain 0.7 of 26.6.)
inline RowPlan plan_rows(int64_t rows, int V, int es, int least, int beside) {
  const int64_t vecs = row_vectors(V, es);
  RowPlan p = {1, vecs >= 2048 || rows <= 4 * ROW_SMS ? 256 : 128, 0};
  const int slots = ROW_SMS * (ROW_SM_THREADS / p.threads);
  const auto flight = [&] {
    const int64_t at_once = slots / p.size;
    return (rows < at_once ? rows : at_once) * vecs * 16;
  };
  while (p.size < ROW_MAX_CLUSTER && flight() > ROW_FLIGHT) p.size *= 2;
  fill_device(p, rows, vecs, least);
  const int64_t part = part_of(vecs, p.size), a_sm = (rows * p.size + ROW_SMS - 1) / ROW_SMS;
  if (beside >= 0 && a_sm * (part * 16 + beside + 2048) <= ROW_SMEM) p.kept = static_cast<int>(part);
  return p;
}

// A cluster a row.  Shared memory beyond the default is asked for once a device.
template <auto KERNEL, typename A>
cudaError_t launch_rows(const RowPlan& p, int smem, int64_t rows, cudaStream_t stream, const A& a) {
  constexpr int DEVICES = 16;
  static std::atomic<bool> asked[DEVICES];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * p.size));
  cfg.blockDim = dim3(p.threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.size;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.size > 1 ? 2 : 1;
  if (smem > 32 * 1024) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= DEVICES || !asked[dev].load(std::memory_order_acquire))) {
      e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, ROW_SMEM);
      if (e == cudaSuccess && dev < DEVICES) asked[dev].store(true, std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, KERNEL, a);
}

// Bytes from a matrix's first element to its last.
inline int64_t extent(int64_t rows, int64_t ld, int V, int es) { return rows > 0 ? ((rows - 1) * ld + V) * es : 0; }

// Whether the gradient may be written: over the logits themselves in place, between their rows, or elsewhere.
inline bool grad_apart(const void* logits, int64_t ld, const void* grad, int64_t gld, int64_t rows, int V, int es) {
  if (!overlap(logits, extent(rows, ld, V, es), grad, extent(rows, gld, V, es))) return true;
  if (ld != gld) return rows <= 1 && logits == grad;
  if (logits == grad) return true;
  const int64_t d = (static_cast<const uint8_t*>(grad) - static_cast<const uint8_t*>(logits)) % (ld * es);
  const int64_t at = d < 0 ? d + ld * es : d;
  return at >= int64_t(V) * es && at + int64_t(V) * es <= ld * es;
}

}  // namespace tail
