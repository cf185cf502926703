// A mixture-of-experts layer for a few tokens: arguments and device pieces
// (moe_layer.cu holds the kernels, moe_api.cu the entry points).
//
//   t = x * rsqrt(mean(x^2) + eps) * gamma
//   z = Wr t + br;  the topk experts of largest score, and the shared ones
//   a = act(W1[e] t + b1[e]);  y[slot] = W2[e] a + b2[e]
//   h = bf16(x + bf16(sum of routed w y + sum of shared y))   (moe.cuh)
//
// A few tokens select a few experts each, so the layer is a stream of weights:
// every selected expert's W1 and W2 once.  The matrix products run on mma.sync
// with 16 weight rows as the M side and up to 8 tokens as the N side; for so few
// columns the tensor pipe idles either way (8 tokens in bf16 need 0.18 of mma.sync's rate
// at full memory bandwidth; a tcgen05 tile would be 128 rows by at least 8 columns, its
// operands rounded to what one descriptor takes, its weights behind a barrier), and
// registers are fed without one.
//
// Weight fragments.  A lane (g = lane / 4, q = lane % 4) of an m16n8k16 product
// holds k slots {2q, 2q+1, 2q+8, 2q+9} of rows g and g + 8.  A sum does not mind
// the order of k, so lane q takes whole 16-byte pieces (8 bf16, or 32 4-bit
// values: one scale block) of each of its rows and feeds them as the slots of 2
// (8) products; its activations are the same columns.  The four lanes of a row
// copy 64 neighbouring bytes at a time, and nothing is shuffled.
//
// Each lane copies its own pieces, by cp.async, into its own places of a ring in
// shared memory and reads them back itself: no barrier guards the ring, any depth
// fits a loop that is not unrolled, and the bytes in flight hold no registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace tail {

constexpr int ML_FINISH = 4;  // warps that add the partial sums and finish the rows, besides the 12 main warps
constexpr int ML_MAX_WARPS = 16;
constexpr int ML_BUFS = 4;    // tiles whose partial sums may wait for a finishing warp
constexpr int ML_MAX_T = 64;
constexpr int ML_MAX_G = 16;  // tokens of one expert that share a pass over its weights
constexpr int ML_MAX_EXPERTS = 512;  // routed and shared together
constexpr int ML_MAX_TOPK = 16;
constexpr int ML_MAX_SHARED = 8;
constexpr int ML_MAX_DIM = 16384;

// Words the CTAs of one launch share; all zero between launches (the last CTA to leave clears them).
struct MoeControl {
  uint32_t ticket;   // next share of work
  uint32_t pad0[31];
  uint32_t done[3];  // finished shares of the router, the first and the second product
  uint32_t pad1[29];
  uint32_t left;     // CTAs that took their last ticket
  uint32_t pad2[31];
};

struct MoeLayerArgs {
  const uint16_t* x;      // [T][H] bf16
  const float* gamma;     // [H] or null: x is used as it is
  const uint16_t* wr;     // [E][H] bf16
  const float* br;        // [E] or null
  const uint8_t* w1;      // [n][N1][H]
  const uint8_t* s1;      // [n][N1][H / 32] scales, or null
  const float* b1;        // [n][N1] or null
  const uint8_t* w2;      // [n][H][I]
  const uint8_t* s2;
  const float* b2;        // [n][H] or null
  float* logits;          // [T][E]
  float2* stats;          // [T] 1 / rms and the largest |t|
  float* act;             // [T * S][I]
  uint32_t* amax;         // [T * S] largest |a|, as bits
  float* slots;           // [T * S][H]
  float* slot_w;          // [T][S]
  int32_t* ids;           // [T][S] or null
  uint16_t* h_out;        // [T][H] or null
  MoeControl* ctl;
  int* err;
  uint64_t timeout_ns;
  int T, H, I, N1, E, topk, nsh, S;
  int gated, interleaved, score;
  float alpha, beta, limit, route_scale, eps;
  int G;                  // tokens of one expert that share a pass over its weights
  int R;                  // activation rows in shared memory: G, or all T tokens (all_rows)
  int all_rows;           // the first product's rows are staged once, for every token
};

// ---------------------------------------------------------------- loads
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// One try at a phase of a barrier, suspended for up to 2 us: warps that poll in a loop took a sixth of
// the SM's issue slots from those that multiply.
__device__ __forceinline__ bool mbar_suspended_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(2000u)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// D (16x8 fp32) += A (16x16 fp16, row) * B (16x8 fp16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight 4-bit values (e2m1, low nibble first) times the scale pair: four fp16 pairs.
__device__ __forceinline__ void fp4_to_half(uint32_t w, uint32_t scale, uint32_t (&h)[4]) {
  asm("{\n.reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __hmul2(reinterpret_cast<const __half2&>(h[i]), reinterpret_cast<const __half2&>(scale));
    h[i] = reinterpret_cast<const uint32_t&>(v);
  }
}

// 2^(s - 127) of an e8m0 scale; 255 is NaN.
__device__ __forceinline__ float e8m0(int s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fc00000u : static_cast<uint32_t>(s) << 23);
}

// The power of two that brings amax into [2^12, 2^13), as the biased exponent of an fp32; 127 (one)
// for an amax that is not finite.  Its inverse has the exponent 254 - e.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23);
  return e >= 255 ? 127 : min(266 - e, 253);
}
__device__ __forceinline__ float pow2_field(int e) { return __uint_as_float(static_cast<uint32_t>(e) << 23); }

// ---------------------------------------------------------------- plan
// Which experts run, on which tokens: made by every CTA from the router's logits
// (the same integers in each), kept in shared memory.
struct MoePlan {
  uint16_t* pair_e;  // [pairs padded to 8] expert of pair t * S + s
  uint16_t* list;    // [pairs] pairs ordered by expert, then token
  uint32_t* unit;    // [<= pairs] expert | first list entry << 10 | entries << 21: one pass over an expert
  uint32_t* cnt;     // [ML_MAX_EXPERTS] pairs of each expert, then those before it
  uint32_t* red;     // [ML_MAX_WARPS]
  int nunits;
};
__host__ __device__ inline int plan_bytes(int pairs) {
  const int p8 = (pairs + 7) & ~7;
  return p8 * 2 * 2 + p8 * 4 + ML_MAX_EXPERTS * 4 + (ML_MAX_WARPS + 4) * 4;
}
__device__ __forceinline__ int unit_expert(uint32_t u) { return u & 1023; }
__device__ __forceinline__ int unit_first(uint32_t u) { return (u >> 10) & 2047; }
__device__ __forceinline__ int unit_size(uint32_t u) { return u >> 21; }

// What ranks an expert's logit: softmax: z with its bias; sigmoid: sigmoid(z) with its bias.
__device__ __forceinline__ float route_score(const MoeLayerArgs& a, float z) {
  return a.score ? __fdividef(1.0f, 1.0f + expf(-z)) : z;
}

// One warp: token t's experts, in falling order of the score; at most 32 * PER experts.
template <int PER>
__device__ __forceinline__ void route_token(const MoeLayerArgs& a, int t, uint16_t* pair_e) {
  const int lane = threadIdx.x & 31;
  const float* z = a.logits + static_cast<int64_t>(t) * a.E;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0u;  // below every score's key
    if (e < a.E) {
      const float v = __ldcg(z + e);
      key[i] = max(float_key(a.br ? route_score(a, v) + __ldg(a.br + e) : v), 1u);  // (0: some NaN's key)
    }
  }
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j < a.topk; ++j) {
    uint32_t best = 0u;
    int at = ML_MAX_EXPERTS - 1;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i * 32 + lane;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int e = __reduce_min_sync(0xffffffffu, best == top ? at : ML_MAX_EXPERTS - 1);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 32 + lane == e) key[i] = 0u;
    if (lane == j) mine = e;
  }
  if (lane < a.topk) pair_e[t * a.S + lane] = static_cast<uint16_t>(mine);
  if (lane < a.nsh) pair_e[t * a.S + a.topk + lane] = static_cast<uint16_t>(a.E + lane);
}

// One warp: token t's weights and ids to memory, its experts known.
__device__ __forceinline__ void write_routes(const MoeLayerArgs& a, int t, const uint16_t* pair_e) {
  const int lane = threadIdx.x & 31;
  float v = 0.f, top = -INFINITY;
  int e = 0;
  if (lane < a.topk) {
    e = pair_e[t * a.S + lane];
    v = __ldcg(a.logits + static_cast<int64_t>(t) * a.E + e);
    if (!a.score && a.br) v += __ldg(a.br + e);
    top = a.score ? fminf(v, 0.f) : v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // a share does not mind a common factor: exp(-top).  sigmoid(v) = exp(min(v, 0)) / (1 + exp(-|v|)), and scores
  // that all lie below the smallest fp32 number keep their ratios
  float w = 0.f;
  if (lane < a.topk)
    w = a.score ? __fdividef(expf(fminf(v, 0.f) - top), 1.0f + expf(-fabsf(v))) : expf(v - top);
  float sum = w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < a.topk) a.slot_w[t * a.S + lane] = a.route_scale * w / sum;
  if (lane < a.nsh) a.slot_w[t * a.S + a.topk + lane] = 1.0f;
  if (a.ids) {
    if (lane < a.topk) a.ids[t * a.S + lane] = e;
    if (lane < a.nsh) a.ids[t * a.S + a.topk + lane] = a.E + lane;
  }
}

// The whole CTA.
__device__ __forceinline__ void make_plan(const MoeLayerArgs& a, MoePlan& p) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nt = blockDim.x, nw = nt >> 5;
  const int pairs = a.T * a.S, p8 = (pairs + 7) & ~7;
#pragma unroll 1
  for (int i = tid; i < ML_MAX_EXPERTS; i += nt) p.cnt[i] = 0u;
  if (tid < p8 - pairs) p.pair_e[pairs + tid] = 0xffffu;
#pragma unroll 1
  for (int t = warp; t < a.T; t += nw) {
    if (a.E <= 128)
      route_token<4>(a, t, p.pair_e);
    else
      route_token<ML_MAX_EXPERTS / 32>(a, t, p.pair_e);
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < pairs; i += nt) atomicAdd(&p.cnt[p.pair_e[i]], 1u);
  __syncthreads();
  // the pairs (low half) and the units (high half) before each expert; a thread takes two experts
  constexpr int HALF = ML_MAX_EXPERTS / 2;
  uint32_t n0 = 0u, n1 = 0u;
  if (tid < HALF) {
    const uint2 n = reinterpret_cast<const uint2*>(p.cnt)[tid];
    n0 = n.x, n1 = n.y;
  }
  auto units = [&](uint32_t n) { return (n + a.G - 1) / a.G; };
  const uint32_t v0 = n0 | (units(n0) << 16), v = v0 + (n1 | (units(n1) << 16));
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) p.red[warp] = incl;
  __syncthreads();
  uint32_t before = incl - v, total = 0u;
#pragma unroll 1
  for (int w = 0; w < nw; ++w) {
    const uint32_t r = p.red[w];
    if (w < warp) before += r;
    total += r;
  }
  if (tid < HALF) {
    auto write_units = [&](uint32_t e, uint32_t n, uint32_t at) {
      p.cnt[e] = at & 0xffffu;
      uint32_t u = at >> 16;
#pragma unroll 1
      for (uint32_t f = 0; f < n; f += a.G, ++u)
        p.unit[u] = e | (((at & 0xffffu) + f) << 10) | (min(n - f, static_cast<uint32_t>(a.G)) << 21);
    };
    write_units(2 * tid, n0, before);
    write_units(2 * tid + 1, n1, before + v0);
  }
  p.nunits = static_cast<int>(total >> 16);
  __syncthreads();
  // a pair's place: the pairs of its expert before it
#pragma unroll 1
  for (int i = tid; i < pairs; i += nt) {
    const uint32_t e = p.pair_e[i], ee = e | (e << 16);
    uint32_t at = p.cnt[e];
    int j = 0;
#pragma unroll 1
    for (; j + 8 <= i; j += 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(p.pair_e + j);
      at += (__popc(__vcmpeq2(q.x, ee)) + __popc(__vcmpeq2(q.y, ee)) + __popc(__vcmpeq2(q.z, ee)) +
             __popc(__vcmpeq2(q.w, ee))) >> 4;
    }
#pragma unroll 1
    for (; j < i; ++j) at += p.pair_e[j] == e ? 1u : 0u;
    p.list[at] = static_cast<uint16_t>(i);
  }
  __syncthreads();
}

}  // namespace tail
