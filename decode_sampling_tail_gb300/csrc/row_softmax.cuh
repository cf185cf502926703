// Row passes of the training operators on vocabulary logits (token_logprobs.cu, policy_loss.cu,
// preference_loss.cu, distill_topk.cu): a row's softmax statistics and its gradient, the row split over
// the CTAs of a cluster.
//
// Statistics.  With m the row's maximum and a_v = (z_v - m) log2(e) / T <= 0:
//   s = sum of 2^a_v over every column but one at the maximum,  u = sum of a_v 2^a_v  (fp32).
// One instance of the maximum stays out of s, since its weight 1 would swallow what the others add up to: with
// it apart, -log1p(s) is a likely token's log-probability and s / (1 + s) its distance from 1 to a few
// units of 2^-24 of themselves.  It costs a minimum a column: a running pair of maxima keeps the
// larger of each two values, and the smaller one goes into the sum, so that every value but the
// maxima enters exactly once.  The sums are taken 32 columns at a time against the maximum so far, so a change of
// it costs one multiplication a batch.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_common.h"
#include "common.cuh"

namespace tail {

constexpr int ROW_MAX_V = 1 << 20;      // columns
constexpr int ROW_MAX_CLUSTER = 8;      // CTAs a row, the portable cluster size
constexpr int ROW_SM_SMEM = 220 * 1024; // dynamic shared memory that the CTAs of an SM share out

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
  static __device__ __forceinline__ uint4 fill() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
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
  static __device__ __forceinline__ uint4 fill() {
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
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
  static __device__ __forceinline__ uint4 fill() {
    return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u);
  }
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
    if (ENT) u = mul2(fma2(s, make_float2(d, d), u), make_float2(c, c));
    s = mul2(s, make_float2(c, c));
    const float2 off = {-ref, -ref}, kk = {k, k};
#pragma unroll
    for (int i = 0; i < U * V::PAIRS; ++i) {
      float2 a = mul2(add2(V::widen(w[i]), off), kk);
      if (ENT) a.x = max_nan(a.x, -200.f), a.y = max_nan(a.y, -200.f);
      const float2 e = {ex2(a.x), ex2(a.y)};
      s = add2(s, e);
      if (ENT) u = fma2(e, a, u);
    }
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

__device__ __forceinline__ RowStat warp_merge(RowStat r, float k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    RowStat b;
    b.m = __shfl_xor_sync(0xffffffffu, r.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, r.s, o);
    b.u = __shfl_xor_sync(0xffffffffu, r.u, o);
    r = merge(r, b, k);
  }
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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Writes a word to the same shared variable of CTA `rank` of the cluster.
__device__ __forceinline__ void store_remote(float* mine, int rank, float v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

struct StatShared {
  RowStat warp[32];
  RowStat cta[ROW_MAX_CLUSTER];
};

// The statistics of all the cluster's threads, the same bits in each.  A cluster of more than one CTA has
// called cluster_arrive() once before: a CTA's shared memory may be written only when it has started.
__device__ __forceinline__ RowStat cluster_merge(RowStat r, float k, StatShared& sh, int rank, int size) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarp = blockDim.x >> 5;
  r = warp_merge(r, k);
  if (lane == 0) sh.warp[warp] = r;
  __syncthreads();
  if (warp == 0) {
    r = lane < nwarp ? sh.warp[lane] : no_stat();
    r = warp_merge(r, k);
  }
  if (size == 1) {
    if (threadIdx.x == 0) sh.cta[0] = r;
    __syncthreads();
    return sh.cta[0];
  }
  cluster_wait();
  if (warp == 0 && lane < size) {
    store_remote(&sh.cta[rank].m, lane, r.m);
    store_remote(&sh.cta[rank].s, lane, r.s);
    store_remote(&sh.cta[rank].u, lane, r.u);
  }
  cluster_arrive();
  cluster_wait();
  r = sh.cta[0];
  for (int i = 1; i < size; ++i) r = merge(r, sh.cta[i], k);
  return r;
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

// Puts the token's own value into the vector that holds it.
template <typename T>
__device__ __forceinline__ void put(uint4& v, int i, float x) {
  T* p = reinterpret_cast<T*>(&v);
#pragma unroll
  for (int j = 0; j < Vec<T>::N; ++j)
    if (j == i) p[j] = Vec<T>::narrow1(x);
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

// The gradient over this CTA's part of a row.  The first `cached` of its vectors are in shared memory
// (`cache`, written by the thread that reads them here, or by others before a barrier).  Rows whose gradient lies elsewhere
// in its 16-byte vectors are written column by column.
template <typename T, bool ENT>
__device__ __forceinline__ void grad_part(const RowGrad& g, const T* row, T* grad, const RowPart& p, const uint4* cache,
                                          int cached) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int body = p.head + p.first * N;  // the part's first column in a vector
  if (same_phase(row, grad)) {
    const uint4* in = reinterpret_cast<const uint4*>(row + p.head) + p.first;
    uint4* out = reinterpret_cast<uint4*>(grad + p.head) + p.first;
    const int tv = g.token >= body ? (g.token - body) / N : -1;
    constexpr int U = 4;
    for (int i0 = tid; i0 < p.count; i0 += U * nt) {
      uint4 z[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * nt;
        if (i < p.count) z[j] = i < cached ? cache[i] : __ldcg(in + i);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * nt;
        if (i >= p.count) continue;
        uint4 o = grad_vec<T, ENT>(g, z[j]);
        if (i == tv) put<T>(o, g.token - body - tv * N, g.at_token);
        __stcs(out + i, o);
      }
    }
  } else {
    const T* c = reinterpret_cast<const T*>(cache);
    for (int i = tid; i < p.count * N; i += nt) {
      const T z = i < cached * N ? c[i] : row[body + i];
      grad[body + i] = Vec<T>::narrow1(body + i == g.token ? g.at_token : grad1<T, ENT>(g, z));
    }
  }
  if (p.edge_n)
    grad[p.edge_lo] = Vec<T>::narrow1(p.edge_lo == g.token ? g.at_token : grad1<T, ENT>(g, row[p.edge_lo]));
}

// ---------------------------------------------------------------- statistics of a part

// Statistics over this CTA's part, straight from memory.
template <typename T, bool ENT>
__device__ __forceinline__ RowStat stat_part(const T* row, const RowPart& p, int from, float k, RowAcc<T, ENT>& acc) {
  constexpr int U = 32 / Vec<T>::N;  // 32 columns a batch
  const uint4* in = reinterpret_cast<const uint4*>(row + p.head) + p.first;
  for (int i0 = from + threadIdx.x; i0 < p.count; i0 += U * blockDim.x) {
    uint4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j * static_cast<int>(blockDim.x);
      v[j] = i < p.count ? __ldcg(in + i) : Vec<T>::fill();
    }
    acc.batch(v, k);
  }
  RowStat r = acc.done(k);
  if (p.edge_n) r = merge(r, stat_of(Vec<T>::widen1(row[p.edge_lo])), k);
  return r;
}

// Requests the part's first `cached` vectors into shared memory, each by the thread that uses it, as one group a batch of
// U vectors a thread; stat_cached takes them batch by batch as they arrive.
template <typename T>
__device__ __forceinline__ void fetch_part(const T* row, const RowPart& p, uint4* cache, int cached) {
  constexpr int U = 32 / Vec<T>::N;
  const uint4* in = reinterpret_cast<const uint4*>(row + p.head) + p.first;
  const int nt = blockDim.x;
  for (int b = 0; b < cached; b += U * nt) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = b + j * nt + static_cast<int>(threadIdx.x);
      if (i < cached) copy_async16(cache + i, in + i);
    }
    copy_commit();
  }
}

// `mask(i)`: the bits of vector i's columns that count as -inf.
template <typename T, bool ENT, typename Mask>
__device__ __forceinline__ RowStat stat_cached(const T* row, const RowPart& p, const uint4* cache, int cached, float k,
                                               Mask mask) {
  constexpr int U = 32 / Vec<T>::N;
  const uint4* in = reinterpret_cast<const uint4*>(row + p.head) + p.first;
  const int nt = blockDim.x;
  RowAcc<T, ENT> acc;
  int left = (cached + U * nt - 1) / (U * nt);
  for (int b = 0; b < p.count; b += U * nt) {
    if (left > 0) copy_wait(--left);
    uint4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = b + j * nt + static_cast<int>(threadIdx.x);
      v[j] = i < cached ? cache[i] : i < p.count ? __ldcg(in + i) : Vec<T>::fill();
      const uint32_t bits = i < p.count ? mask(i) : 0;
      if (bits) Vec<T>::mask(v[j], bits);
    }
    acc.batch(v, k);
  }
  return acc.done(k);
}

// ---------------------------------------------------------------- host side

struct RowPlan {
  int size;     // CTAs a row
  int threads;
  int cached;   // vectors of a part that shared memory holds
};

// How a row is split.  `fit`: bytes of the row that one CTA should hold at most (0: the row is not kept).
inline RowPlan plan_rows(int64_t rows, int V, int es, int64_t fit) {
  RowPlan p;
  const int64_t vecs = (static_cast<int64_t>(V) * es + 15) / 16;
  p.size = 1;
  while (p.size < ROW_MAX_CLUSTER && fit > 0 && (vecs + p.size - 1) / p.size * 16 > fit) p.size *= 2;
  // few rows: spread each over more SMs, as long as a part still has two vectors a thread
  while (p.size < ROW_MAX_CLUSTER && rows * p.size * 2 <= 2 * 152 && vecs / (2 * p.size) >= 1024) p.size *= 2;
  const int64_t part = (vecs + p.size - 1) / p.size;
  p.threads = part >= 2048 ? 512 : part >= 512 ? 256 : part >= 128 ? 128 : 64;
  p.cached = fit > 0 ? static_cast<int>(part * 16 <= fit ? part : fit / 16) : 0;
  return p;
}

template <typename A>
cudaError_t launch_rows(void (*kernel)(A), const RowPlan& p, int64_t rows, int smem, cudaStream_t stream, const A& a) {
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
  cfg.numAttrs = 2;
  if (smem > 48 * 1024 - 2048) {  // with the static part; idempotent, per device
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a);
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
