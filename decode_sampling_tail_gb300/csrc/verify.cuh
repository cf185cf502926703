// Pieces shared by the two forms of draft verification (verify_lists.cu,
// verify_logits.cu): sequence bounds, draft probabilities, warp sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "abi_common.h"
#include "common.cuh"
#include "fixed_exp.cuh"

namespace tail {

// Whether an output of n words meets another array of the call (rows or nseq + 1 words each): CTAs of one
// sequence read its drafts and uniforms while another writes its tokens.
inline bool meets(const void* out, int64_t n, const void* in, int64_t words) {
  return overlap(out, n * 4, in, words * 4);
}

constexpr int VERIFY_THREADS = 256;
constexpr int VERIFY_WARPS = VERIFY_THREADS / 32;

// The draft model's probabilities: [rows][ld] of dtype (0 fp32, 1 fp16, 2 bf16), or null (one-hot drafts).
struct DraftProbs {
  const void* p;
  int dtype;
  int64_t ld;
  int V;
};

// A probability: values outside [0, 1] count as the nearer end, NaN as 0.
__device__ __forceinline__ float as_prob(float v) { return fminf(fmaxf(v, 0.f), 1.f); }

__device__ __forceinline__ float draft_prob(const DraftProbs& q, int64_t row, int col) {
  if (col < 0 || col >= q.V) return 0.f;
  const int64_t i = row * q.ld + col;
  float v;
  if (q.dtype == 0)
    v = __ldg(static_cast<const float*>(q.p) + i);
  else if (q.dtype == 1)
    v = __half2float(static_cast<const __half*>(q.p)[i]);
  else
    v = __bfloat162float(static_cast<const __nv_bfloat16*>(q.p)[i]);
  return as_prob(v);
}

// Rows [lo, hi) of sequence s; bounds outside the call's rows are cut, a decreasing pair is empty.
__device__ __forceinline__ void sequence_rows(const int32_t* cu, int s, int rows, int& lo, int& hi) {
  lo = min(max(__ldg(cu + s), 0), rows);
  hi = min(max(__ldg(cu + s + 1), lo), rows);
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ int64_t warp_scan(int64_t v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// Launches with programmatic dependent launch: the kernel's start overlaps the end of the one before
// it, up to its pdl_wait.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(VERIFY_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A sequence's tokens around its settled row: the drafts before it, -1 behind it; its own token is
// written by whoever drew it.
__device__ __forceinline__ void write_sequence(int lo, int hi, int sel, const int32_t* drafts, int32_t* out_tokens,
                                               int32_t* out_count) {
  for (int r = lo + static_cast<int>(threadIdx.x); r < hi; r += blockDim.x)
    if (r != sel) out_tokens[r] = r < sel ? drafts[r] : -1;
  if (threadIdx.x == 0) *out_count = hi > lo ? sel - lo + 1 : 0;
}

}  // namespace tail
