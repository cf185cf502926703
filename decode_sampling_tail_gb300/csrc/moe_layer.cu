// The kernel of the mixture-of-experts layer for a few tokens (moe_layer.cuh
// states the formulas and the fragment layout).
//
// One launch, one CTA per SM, four stages: router logits; the first product and
// the activation; the second product; combine and residual.  A stage needs all of
// the one before, and the streams of two stages should not drain in between, so
// the CTAs stay: a stage is cut into one share per CTA, shares are taken in order
// from a ticket counter, and a CTA that ends a stage asks for its first weights of
// the next before it waits for the others.
//
// No CTA needs another to be resident: shares are handed out in stage order, so a
// share that a CTA waits on is held by a CTA that runs and, in its turn, waits on
// earlier stages only.  CTAs that start late find their shares done by others.
// Waits are bounded; one that runs out raises the error word, and the CTA leaves.
//
// Bound: bf16 by HBM, 4-bit weights by instructions.  Measured (copy rate 6.69 TB/s): bf16, 64 tokens over 128
// experts of 2880 x 5760 and 2880 x 2880, 5.54 GB: 849-887 us, 6.2-6.5 TB/s (0.93-0.98); 8 tokens over 64 experts
// and 2 shared, 737 MB: 121-126 us, 0.87-0.91; 5 tokens over 32 experts 0.88-0.92.  4 bits, 16 tokens over 128
// experts, 677 MB: 202-206 us, 0.50: a 2 KB k-step of a warp takes about 350 instructions (196 of them conversions,
// scalings and products), a scheduler's three main warps issue on 47 % of the cycles, and neither a deeper ring
// (3, 4, 5 or 6 steps: 204.8, 204.2, 205.4, 206.2 us) nor k-steps of 32 rows (211) move it.  One token, 54 MB:
// 35.4 us, a chain of stage latencies and of fetching code that runs once.
#include <math.h>

#include "internal.h"
#include "moe.cuh"
#include "moe_layer.cuh"
#include "moe_layer_internal.h"

namespace tail {

namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ void load_gamma(const float* gamma, int k, float (&g)[8]) {
  if (gamma == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.f;
    return;
  }
  const float4 a = __ldg(reinterpret_cast<const float4*>(gamma + k));
  const float4 b = __ldg(reinterpret_cast<const float4*>(gamma + k + 4));
  g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w, g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------- router
// The logits of experts [e0, e1) for every token, and per token in [t0, t1) 1 / rms, the largest |t| and its
// pairs' largest-activation words cleared.  The whole CTA; a warp a token, or several, K split, when there are
// fewer tokens than warps.  The norm factors out: z = (1 / rms) * sum(x gamma w), and gamma w is formed once, in
// shared memory (v: H floats).  Latency: 16 bytes a lane and step from L2, and the barriers between.
__device__ __forceinline__ void router_share(const MoeLayerArgs& a, int e0, int e1, int t0, int t1, float* v,
                                             float* s_part) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nt = blockDim.x, nw = nt >> 5;
#pragma unroll 1
  for (int e = e0; e <= e1; ++e) {
    const bool stat = e == e1;  // the last pass: statistics
    const int first = stat ? t0 : 0, n = (stat ? t1 : a.T) - first;
    if (n == 0) continue;
    const uint16_t* w = a.wr + static_cast<int64_t>(stat ? 0 : e) * a.H;
    __syncthreads();  // v and s_part are read by the pass before
#pragma unroll 1
    for (int k = tid * 8; k < a.H; k += nt * 8) {
      float wf[8], g[8];
      load_gamma(a.gamma, k, g);
      if (!stat) unpack8(__ldg(reinterpret_cast<const uint4*>(w + k)), wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = stat ? g[j] : g[j] * wf[j];
      *reinterpret_cast<float4*>(v + k) = make_float4(g[0], g[1], g[2], g[3]);
      *reinterpret_cast<float4*>(v + k + 4) = make_float4(g[4], g[5], g[6], g[7]);
    }
    __syncthreads();
    const int split = n >= nw ? 1 : 1 << (31 - __clz(nw / n));
    const int groups = nw / split, grp = warp / split, part = warp - grp * split;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += groups) {
      const bool live = grp < groups && i0 + grp < n;
      const int t = first + i0 + grp;
      float dot = 0.f, ss = 0.f;
      if (live) {
        const uint16_t* x = a.x + static_cast<int64_t>(t) * a.H;
#pragma unroll 4
        for (int k = (part * 32 + lane) * 8; k < a.H; k += split * 256) {
          float xf[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(x + k)), xf);
          const float4 p = *reinterpret_cast<const float4*>(v + k), q = *reinterpret_cast<const float4*>(v + k + 4);
          const float vf[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ss = fmaf(xf[j], xf[j], ss);
            if (stat) {
              const float m = fabsf(xf[j] * vf[j]);
              dot = m <= 3.402823466e38f ? fmaxf(dot, m) : INFINITY;
            } else {
              dot = fmaf(xf[j], vf[j], dot);
            }
          }
        }
        ss = warp_sum(ss);
        if (stat) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dot = fmaxf(dot, __shfl_xor_sync(0xffffffffu, dot, o));
        } else {
          dot = warp_sum(dot);
        }
      }
      __syncthreads();
      if (live && lane == 0) {
        s_part[2 * warp] = dot;
        s_part[2 * warp + 1] = ss;
      }
      __syncthreads();
      if (live && part == 0) {
        if (stat)
          for (int s = lane; s < a.S; s += 32) a.amax[t * a.S + s] = 0u;
        if (lane == 0) {
#pragma unroll 1
          for (int k = 1; k < split; ++k) {
            const float d = s_part[2 * (warp + k)];
            dot = stat ? fmaxf(dot, d) : dot + d;
            ss += s_part[2 * (warp + k) + 1];
          }
          const float r = a.gamma ? rsqrtf(__fdividef(ss, static_cast<float>(a.H)) + a.eps) : 1.0f;
          if (stat)
            a.stats[t] = make_float2(r, dot * r);
          else
            a.logits[static_cast<int64_t>(t) * a.E + e] = dot * r;
        }
      }
    }
  }
}

// ---------------------------------------------------------------- experts
// The two products of the experts have one form: rows of a weight [n][N][K], K contiguous, against
// up to 16 tokens' activations in shared memory.
//
// Work is cut into tiles of a unit (an expert and up to G of its tokens): RG subtiles of 16 * RT
// rows, whose K is split over MAIN / RG warps.  A share is a contiguous run of tiles.  Each main
// warp keeps DEPTH k-steps of 2 KB under way, across tile borders (12 warps of 4: 96 KB an SM); at
// the end of a tile it leaves its partial sums in shared memory and goes on.  A finishing warp adds
// them in a fixed order and finishes the rows: its chain of bias loads, sums and exponentials held up
// every warp of the CTA when a main warp did it between two barriers (bf16, 64 tokens over 128
// experts: 1640 us).
//
// Formats: BF16; MXFP4; MXFP4_WIDE, for rows that are whole pieces of 64 columns.
enum Format : int { BF16 = 0, MXFP4 = 1, MXFP4_WIDE = 2 };

template <int FMT>
struct Step {
  static constexpr bool FP4 = FMT != BF16;
  static constexpr int PIECES = FMT == MXFP4 ? 1 : 2;       // 16-byte pieces of a row that a lane takes
  static constexpr int PIECE_COLS = FP4 ? 32 : 8;
  static constexpr int COLS = 4 * PIECES * PIECE_COLS;      // columns of one k-step of a warp
};

struct Phase {
  const uint8_t* w;
  const uint8_t* s;
  const float* bias;
  int N, K;
  int row_bytes, scale_bytes;
  int a_mul, rt_step, b_step;  // rows from a lane's first to those of its other fragments (row_of)
  int w_rt, w_b, s_rt, s_b;    // the same steps in bytes of the weight and of its scales
  uintptr_t s_end;             // behind the last scale
  int nsub, tiles;             // subtiles and tiles of a unit
  int steps;                   // k-steps
  int pitch;                   // bytes of one activation row in shared memory
};

// A k-step's fragments in registers; a scale a word.
template <int FMT, int RT>
struct Frag {
  uint32_t w[RT][2][Step<FMT>::PIECES][4];
  uint32_t s[RT][2][Step<FMT>::PIECES];
};

// Bytes of one k-step of a warp in the ring.
template <int FMT, int RT>
__host__ __device__ constexpr int slot_bytes() {
  return RT * 2 * (Step<FMT>::PIECES * 512 + (Step<FMT>::FP4 ? 128 : 0));
}

// State of a CTA that outlives a share.
template <int MAIN>
struct Cta {
  MoePlan plan;
  const uint8_t* smem; // the dynamic shared memory
  uint32_t act;        // 2 R activation rows
  uint32_t ring;       // [MAIN][DEPTH] slots
  float4* red;         // [ML_BUFS][MAIN][RT * NACC][32]
  uint32_t full, empty;  // mbarriers [ML_BUFS]: partial sums written, and read
  uint32_t* top;         // [ML_MAX_G] all_rows: the largest |t| by which stage_all scaled each token's row, as bits
  volatile int* abort;   // a bounded wait ran out: no one waits any more
  uint32_t seq;        // tiles so far, over all shares
};

template <int MAIN>
__device__ __forceinline__ void main_warps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * MAIN) : "memory");
}

__device__ __forceinline__ void wait_or_abort(const MoeLayerArgs& a, volatile int* abort, uint32_t bar, uint32_t parity, int code) {
  if (*abort || mbar_suspended_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_suspended_wait(bar, parity)) {
    if (global_timer_ns() - t0 > a.timeout_ns) {
      raise_error(a.err, code);
      *abort = 1;
      return;
    }
  }
}

// The whole CTA: until `shares` shares of an earlier stage are done and their writes are visible.
__device__ __forceinline__ void wait_stage(const MoeLayerArgs& a, volatile int* abort, const uint32_t* done, uint32_t shares) {
  if (threadIdx.x == blockDim.x - 32 && !*abort) {  // a finishing warp's: no loads of its own to wait for
    uint32_t v;
    uint64_t t0 = 0;
    for (;;) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(done) : "memory");
      if (v >= shares) break;
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > a.timeout_ns) {
        raise_error(a.err, DEV_TIMEOUT_BARRIER);
        *abort = 1;
        break;
      }
    }
  }
  __syncthreads();
}

template <int FMT, int RT, int NB, int PHASE, int DEPTH, int MAIN>
struct Experts {
  static constexpr int NACC = NB == 4 ? 2 : 1;
  static constexpr int JOBS = RT * NACC;
  using S = Step<FMT>;
  static constexpr bool FP4 = S::FP4;
  static constexpr int PIECES = S::PIECES;
  static constexpr int SLOT = slot_bytes<FMT, RT>();

  const MoeLayerArgs& a;
  const Phase& ph;
  Cta<MAIN>& cta;
  const MoePlan& plan;
  uint32_t act;
  int ksplit, rg_warp, kw, RG;
  int lane, warp, g, q;

  __device__ __forceinline__ Experts(const MoeLayerArgs& a_, const Phase& ph_, Cta<MAIN>& c, int ks)
      : a(a_), ph(ph_), cta(c), plan(c.plan), act(c.act), ksplit(ks) {
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    g = lane >> 2;
    q = lane & 3;
    RG = MAIN / ksplit;
    rg_warp = warp / ksplit;
    kw = warp - rg_warp * ksplit;
  }

  __device__ __forceinline__ int64_t row_of(int sub) const {
    // first row (rt = 0, half 0) of this lane's fragment
    if (PHASE == 1 && a.gated) return static_cast<int64_t>(sub * 8 * RT + g) * ph.a_mul;
    return static_cast<int64_t>(sub) * 16 * RT + g;
  }

  // row `row` of the high (plane 0) or low (plane 1) parts
  __device__ __forceinline__ uint32_t act_row(int plane, int row) const {
    return act + static_cast<uint32_t>(plane * a.R + row) * ph.pitch;
  }
  // the row of a unit's token (any row past its tokens: those columns are not used)
  __device__ __forceinline__ int row_of_token(uint32_t unit, int tok) const {
    const int i = min(tok, unit_size(unit) - 1);
    return PHASE == 1 && a.all_rows ? plan.list[unit_first(unit) + i] / a.S : i;
  }

  // Eight activations v times mult into shared memory, split into a high and a low 16-bit part so that
  // the products carry them to about 2^-17 (bf16) or 2^-22 (fp16, scaled by a power of two a token; fp16's
  // smallest step is 2^-37 of the row's largest there).
  // What the four lanes of a row read together lies side by side.
  __device__ __forceinline__ void put8(int row, int k, const float (&v)[8], float mult) const {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (FP4) {
        const float x = v[2 * j] * mult, y = v[2 * j + 1] * mult;
        const __half2 h = __floats2half2_rn(x, y);
        const __half2 l = __floats2half2_rn(x - __low2float(h), y - __high2float(h));
        hi[j] = reinterpret_cast<const uint32_t&>(h);
        lo[j] = reinterpret_cast<const uint32_t&>(l);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        const __nv_bfloat162 l = __floats2bfloat162_rn(v[2 * j] - __low2float(h), v[2 * j + 1] - __high2float(h));
        hi[j] = reinterpret_cast<const uint32_t&>(h);
        lo[j] = reinterpret_cast<const uint32_t&>(l);
      }
    }
    int p = k / 8;
    if (FP4) {  // word w of block 4 j + q stands at (4 j + w, q)
      const int w = p & 3, block = p >> 2;
      p = (block & ~3) * 4 + w * 4 + (block & 3);
    }
    const uint32_t at = p * 16;
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(act_row(0, row) + at), "r"(hi[0]), "r"(hi[1]),
                 "r"(hi[2]), "r"(hi[3])
                 : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(act_row(1, row) + at), "r"(lo[0]), "r"(lo[1]),
                 "r"(lo[2]), "r"(lo[3])
                 : "memory");
  }

  // t of `token` at columns k .. k + 7, from its 1 / rms
  __device__ __forceinline__ void normed8(int token, int k, float r, float (&v)[8]) const {
    float gm[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(token) * a.H + k)), v);
    load_gamma(a.gamma, k, gm);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * r * gm[j];
  }

  // The main warps: the rows of a unit.
  __device__ __forceinline__ void stage(uint32_t unit) const {
    const int n = unit_size(unit), first = unit_first(unit);
    const int chunks = ph.steps * (S::COLS / 8);
#pragma unroll 1
    for (int row = 0; row < n; ++row) {  // a row at a time, all warps on it
      const int pair = plan.list[first + row];
      const int token = pair / a.S;
      float r = 1.f;
      uint32_t top = 0u;
      if (PHASE == 1) {
        const float2 st = __ldcg(a.stats + token);
        r = st.x;
        top = __float_as_uint(st.y);
      } else if (FP4) {
        top = __ldcg(a.amax + pair);
      }
#pragma unroll 1
      for (int c = warp * 32 + lane; c < chunks; c += 32 * MAIN) {
        const int k = c * 8;
        float v[8] = {};
        if (k < ph.K) {
          if (PHASE == 1) {
            normed8(token, k, r, v);
          } else {
            const float4* p = reinterpret_cast<const float4*>(a.act + static_cast<int64_t>(pair) * a.I + k);
            const float4 x = __ldcg(p), y = __ldcg(p + 1);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
          }
        }
        put8(row, k, v, FP4 ? pow2_field(scale_exponent(top)) : 1.f);
      }
    }
  }

  // The whole CTA, while the router's other shares finish: the first product's rows of every token, each
  // with a 1 / rms and a largest value formed here.
  __device__ __forceinline__ void stage_all(float* s_part) const {
    const int nw = blockDim.x >> 5;
    const int split = a.T >= nw ? 1 : 1 << (31 - __clz(nw / a.T));
    const int groups = nw / split, grp = warp / split, part = warp - grp * split;
    const int kpad = ph.steps * S::COLS;
#pragma unroll 1
    for (int i0 = 0; i0 < a.T; i0 += groups) {
      const int t = i0 + grp;
      const bool live = grp < groups && t < a.T;
      float ss = 0.f, mx = 0.f;
      if (live) {
#pragma unroll 4
        for (int k = (part * 32 + lane) * 8; k < a.H; k += split * 256) {
          float v[8], gm[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(t) * a.H + k)), v);
          load_gamma(a.gamma, k, gm);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ss = fmaf(v[j], v[j], ss);
            const float m = fabsf(v[j] * gm[j]);
            mx = m <= 3.402823466e38f ? fmaxf(mx, m) : INFINITY;
          }
        }
        ss = warp_sum(ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      }
      __syncthreads();
      if (live && lane == 0) {
        s_part[2 * warp] = mx;
        s_part[2 * warp + 1] = ss;
      }
      __syncthreads();
      if (!live) continue;
      mx = 0.f, ss = 0.f;
#pragma unroll 1
      for (int k = 0; k < split; ++k) {
        mx = fmaxf(mx, s_part[2 * (grp * split + k)]);
        ss += s_part[2 * (grp * split + k) + 1];
      }
      const float r = a.gamma ? rsqrtf(__fdividef(ss, static_cast<float>(a.H)) + a.eps) : 1.0f;
      // the products' scale is taken out again by this same value: another order of the sum of squares may
      // give another last bit, and next to a power of two another exponent
      const uint32_t top = __float_as_uint(mx * r);
      if (part == 0 && lane == 0) cta.top[t] = top;
      const float mult = FP4 ? pow2_field(scale_exponent(top)) : 1.f;
#pragma unroll 2
      for (int k = (part * 32 + lane) * 8; k < kpad; k += split * 256) {
        float v[8] = {};
        if (k < a.H) normed8(t, k, r, v);
        put8(t, k, v, mult);
      }
    }
    __syncthreads();
  }

  // Where the copies stand: DEPTH steps ahead of the products.
  struct Cursor {
    int u, tile;                // unit and tile in it
    int left;                   // tiles of the share that follow, this one included
    int i, nk;                  // k-step of the warp in the tile, and their number
    int step;                   // the same of the row
    const uint8_t* w[2 * RT];   // this lane's rows at the step
    const uint8_t* s[2 * RT];   // the word of the rows' scales that this lane copies
    uint32_t words;             // rows of which it copies one, a bit each
  };

  // Copies the next k-step into a slot; past the share, nothing.
  __device__ __forceinline__ void issue(Cursor& c, uint32_t slot) const {
    if (c.left > 0) {
      if (c.i == 0) {
        const int sub = c.tile * RG + rg_warp;  // past the last subtile: any rows, their sums are not used
        const int64_t row = static_cast<int64_t>(unit_expert(plan.unit[c.u])) * ph.N + row_of(sub < ph.nsub ? sub : 0);
        const uint8_t* w = ph.w + row * ph.row_bytes + kw * (PIECES * 64) + q * 16;
        const uint8_t* sc = ph.s + row * ph.scale_bytes + kw * (4 * PIECES);
        c.words = 0u;
        c.step = kw;
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
          c.w[r] = w + ((r >> 1) * ph.w_rt + (r & 1) * ph.w_b);
          if (FP4) {
            // a row's scales of a step, 4 * PIECES bytes, by the aligned words that hold them, lane q word q
            const uintptr_t p = reinterpret_cast<uintptr_t>(sc + ((r >> 1) * ph.s_rt + (r & 1) * ph.s_b));
            c.s[r] = reinterpret_cast<const uint8_t*>(p & ~static_cast<uintptr_t>(3)) + q * 4;
            if (q < PIECES || (q == PIECES && (p & 3) != 0)) c.words |= 1u << r;
          }
        }
      }
      const uint32_t dst = slot + lane * 16, to = slot + 2 * RT * PIECES * 512 + lane * 4;
      if ((c.step + 1) * S::COLS <= ph.K) {
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
#pragma unroll
          for (int j = 0; j < PIECES; ++j) copy16(dst + (r * PIECES + j) * 512, c.w[r] + j * 64);
          if (FP4 && (c.words >> r & 1u)) copy4(to + r * 128, c.s[r]);
        }
      } else if (c.step < ph.steps) {
        // the end of the rows: a piece past it repeats the step's first, and the activations it meets are
        // zero; words behind the last scale are not touched
        const int left = ph.K - c.step * S::COLS;  // columns
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
#pragma unroll
          for (int j = 0; j < PIECES; ++j)
            copy16(dst + (r * PIECES + j) * 512,
                   (j * 4 + q) * S::PIECE_COLS < left ? c.w[r] + j * 64 : c.w[r] - q * 16);
          if (FP4 && (c.words >> r & 1u) && reinterpret_cast<uintptr_t>(c.s[r]) < ph.s_end) copy4(to + r * 128, c.s[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r) {
        c.w[r] += ksplit * (PIECES * 64);
        if (FP4) c.s[r] += ksplit * (4 * PIECES);
      }
      c.step += ksplit;
      if (++c.i == c.nk) {
        c.i = 0;
        --c.left;
        if (++c.tile == ph.tiles) {
          c.tile = 0;
          ++c.u;
        }
      }
    }
    copies_commit();
  }

  // The oldest k-step's fragments; `low` are the two low bits of the rows' scale addresses (a step moves
  // them by whole words).
  __device__ __forceinline__ void take(Frag<FMT, RT>& f, uint32_t slot, const uint32_t (&low)[RT][2], int ks) const {
    const int blocks = ph.scale_bytes - ks * (4 * PIECES);  // of the row from this step on; a lane past them takes the first's
    copies_wait<DEPTH - 1>();
    if (FP4) __syncwarp();  // the scales were copied by the four lanes of a row together
#pragma unroll
    for (int r = 0; r < 2 * RT; ++r)
#pragma unroll
      for (int j = 0; j < PIECES; ++j) {
        uint32_t(&w)[4] = f.w[r >> 1][r & 1][j];
        lds128(slot + (r * PIECES + j) * 512 + lane * 16, w[0], w[1], w[2], w[3]);
        if (FP4)
          f.s[r >> 1][r & 1][j] = lds8(slot + 2 * RT * PIECES * 512 + r * 128 + g * 16 + low[r >> 1][r & 1] +
                                       (j * 4 + q < blocks ? j * 4 + q : 0));
      }
  }

  // Sums of a tile.  4-bit weights: d counts in units of 2^(ref - 127), acc in ones.
  struct Sums {
    float acc[RT][NACC][4];
    float d[FP4 ? RT : 1][FP4 ? NACC : 1][2][4];  // two chains of products each: one's latency under the other's
    int ref;
  };

  __device__ __forceinline__ void flush(Sums& t) const {
    if constexpr (FP4) {
      const float f = e8m0(t.ref);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int n = 0; n < NACC; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            t.acc[rt][n][j] = fmaf(t.d[rt][n][0][j] + t.d[rt][n][1][j], f, t.acc[rt][n][j]);
            t.d[rt][n][0][j] = t.d[rt][n][1][j] = 0.f;
          }
    }
  }

  // 16 bytes of activations; plain loads, which the compiler may move up past products
  __device__ __forceinline__ uint4 columns(uint32_t at) const {
    return *reinterpret_cast<const uint4*>(cta.smem + at);
  }

  // d += the fragment's products with its values times the scale pairs
  template <int N>
  __device__ __forceinline__ void products_fp4(const Frag<FMT, RT>& f, const uint32_t (&sc)[RT][2][PIECES], uint32_t at,
                                               const uint32_t (&bp)[NB], float (&d)[RT][NACC][2][4]) const {
#pragma unroll
    for (int i = 0; i < 4 * PIECES; ++i) {
      const int j = i / 4, w = i % 4;
      uint4 v[N];
#pragma unroll
      for (int b = 0; b < N; ++b) v[b] = columns(bp[b] + at + i * 64);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        uint32_t x[4], y[4];
        fp4_to_half(f.w[rt][0][j][w], sc[rt][0][j], x);
        fp4_to_half(f.w[rt][1][j][w], sc[rt][1][j], y);
#pragma unroll
        for (int b = 0; b < N; ++b) {
          mma_f16_16816(d[rt][b >> 1][0], x[0], y[0], x[1], y[1], v[b].x, v[b].y);
          mma_f16_16816(d[rt][b >> 1][1], x[2], y[2], x[3], y[3], v[b].z, v[b].w);
        }
      }
    }
  }

  // Adds the fragment's products with N n-tiles of 8 columns (N == 1: 4 high, 4 low columns).
  template <int N>
  __device__ __forceinline__ void products(const Frag<FMT, RT>& f, int ks, const uint32_t (&bp)[NB], Sums& t) const {
    const uint32_t at = ks * (S::COLS * 2);
    if constexpr (!FP4) {
#pragma unroll
      for (int b = 0; b < N; ++b)
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
          const uint4 v = columns(bp[b] + at + j * 64);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const uint32_t(&x)[4] = f.w[rt][0][j];
            const uint32_t(&y)[4] = f.w[rt][1][j];
            mma_bf16_16816(t.acc[rt][b >> 1], x[0], y[0], x[1], y[1], v.x, v.y);
            mma_bf16_16816(t.acc[rt][b >> 1], x[2], y[2], x[3], y[3], v.z, v.w);
          }
        }
    } else {
      // A block's scale relative to ref goes into its values: a power of two from 2^-8 to 2^7, so that
      // fp16 holds them exactly.  Trained weights stay in one such window for whole tiles; where they
      // leave it, ref moves, and blocks too far apart for any window take a pass for each window they fill.
      // (A block far below another may still be the whole sum: the other's activations may be zero.)
      if (__any_sync(0xffffffffu, outside(f, static_cast<uint32_t>(t.ref - 8)))) {
        flush(t);
        uint32_t todo = live(f);
        t.ref = window(f, todo) + 8;
        if (__any_sync(0xffffffffu, outside(f, static_cast<uint32_t>(t.ref - 8)))) {
          products_apart<N>(f, todo, at, bp, t);
          return;
        }
      }
      uint32_t sc[RT][2][PIECES];  // 2^(scale - ref), twice
      const uint32_t one = (15u - static_cast<uint32_t>(t.ref)) * 0x04000400u;
#pragma unroll
      for (int i = 0; i < 2 * RT * PIECES; ++i)
        sc[i / (2 * PIECES)][i / PIECES % 2][i % PIECES] = scale_of(f, i) * 0x04000400u + one;
      products_fp4<N>(f, sc, at, bp, t.d);
    }
  }

  // Blocks too far apart for one window, of which `todo` hold anything: the largest window's, then the rest.
  template <int N>
  __device__ __forceinline__ void products_apart(const Frag<FMT, RT>& f, uint32_t todo, uint32_t at,
                                                 const uint32_t (&bp)[NB], Sums& t) const {
#pragma unroll 1
    for (;;) {
      uint32_t sc[RT][2][PIECES];
      const uint32_t one = (15u - static_cast<uint32_t>(t.ref)) * 0x04000400u;
#pragma unroll
      for (int i = 0; i < 2 * RT * PIECES; ++i) {
        const uint32_t s = scale_of(f, i);
        const bool in = (todo >> i & 1u) && (s == 255u || s - static_cast<uint32_t>(t.ref - 8) <= 15u);
        sc[i / (2 * PIECES)][i / PIECES % 2][i % PIECES] = !in ? 0u : s == 255u ? 0x7e007e00u : s * 0x04000400u + one;
        if (in) todo &= ~(1u << i);
      }
      products_fp4<N>(f, sc, at, bp, t.d);
      flush(t);
      if (!__any_sync(0xffffffffu, todo != 0u)) break;
      t.ref = window(f, todo) + 8;  // takes the largest block left at least
    }
  }

  // block i of a lane's 2 * RT * PIECES
  static __device__ __forceinline__ uint32_t scale_of(const Frag<FMT, RT>& f, int i) {
    return f.s[i / (2 * PIECES)][i / PIECES % 2][i % PIECES];
  }

  // whether a scale of this lane lies outside [low, low + 15]
  static __device__ __forceinline__ bool outside(const Frag<FMT, RT>& f, uint32_t low) {
    uint32_t out = 0u;
#pragma unroll
    for (int i = 0; i < 2 * RT * PIECES; ++i) out |= scale_of(f, i) - low;
    return out > 15u;
  }

  // the blocks of this lane that hold a value other than 0 or a scale of NaN, a bit each
  static __device__ __forceinline__ uint32_t live(const Frag<FMT, RT>& f) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 2 * RT * PIECES; ++i) {
      const uint32_t(&w)[4] = f.w[i / (2 * PIECES)][i / PIECES % 2][i % PIECES];
      if (((w[0] | w[1] | w[2] | w[3]) & 0x77777777u) != 0u || scale_of(f, i) == 255u) m |= 1u << i;
    }
    return m;
  }

  // the lowest scale of the window for the warp's blocks `todo`: all of them, or the largest
  static __device__ __forceinline__ int window(const Frag<FMT, RT>& f, uint32_t todo) {
    uint32_t mx = 0u, mn = 255u;
#pragma unroll
    for (int i = 0; i < 2 * RT * PIECES; ++i) {
      const uint32_t s = scale_of(f, i);
      if ((todo >> i & 1u) && s != 255u) {
        mx = max(mx, s);
        mn = min(mn, s);
      }
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    mn = __reduce_min_sync(0xffffffffu, mn);
    return static_cast<int>(mn > mx ? 119u : mx - mn > 15u ? mx - 15u : min(mn, 239u));
  }

  __device__ __forceinline__ float glu(float gate, float up) const {
    if (a.limit > 0.f) {
      gate = gate > a.limit ? a.limit : gate;  // NaN stays
      up = up > a.limit ? a.limit : up < -a.limit ? -a.limit : up;
    }
    return __fdividef(gate, 1.0f + expf(-a.alpha * gate)) * (up + a.beta);
  }

  // One warp: the rows of subtile (rg, rt) for the tokens 8 * n .. of the unit.  `wait` is called once
  // the loads that need no partial sums are under way.
  template <typename Wait>
  __device__ __forceinline__ void finish(uint32_t unit, int tile_in_unit, int job, const float4* part, Wait wait) const {
    const int n = job % NACC, rt = (job / NACC) % RT, rg = job / (NACC * RT);
    const int sub = tile_in_unit * RG + rg;
    const int size = unit_size(unit), first = unit_first(unit), e = unit_expert(unit);
    const bool rows = sub < ph.nsub && n * 8 < size;
    const int64_t ra = row_of(sub) + rt * ph.rt_step, rb = ra + ph.b_step;
    const int tok0 = n * 8 + 2 * q;
    float ba = 0.f, bb = 0.f;
    uint32_t am[2] = {0u, 0u};
    int pair[2] = {0, 0};
    if (rows) {
      if (ph.bias) {
        const float* bias = ph.bias + static_cast<int64_t>(e) * ph.N;
        ba = __ldg(bias + ra);
        bb = __ldg(bias + rb);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (tok0 + j < size) {
          pair[j] = plan.list[first + tok0 + j];
          if (FP4)
            am[j] = PHASE == 2   ? __ldcg(a.amax + pair[j])
                    : a.all_rows ? cta.top[pair[j] / a.S]
                                 : __float_as_uint(__ldcg(&a.stats[pair[j] / a.S].y));
        }
    }
    wait();
    if (!rows) return;
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < ksplit; ++k) {
      const float4 p = part[((rg * ksplit + k) * JOBS + rt * NACC + n) * 32 + lane];
      c.x += p.x, c.y += p.y, c.z += p.z, c.w += p.w;
    }
    if (NB == 1 || size <= 4) {  // columns 0-3 high parts, 4-7 low parts
      c.x += __shfl_xor_sync(0xffffffffu, c.x, 2);
      c.y += __shfl_xor_sync(0xffffffffu, c.y, 2);
      c.z += __shfl_xor_sync(0xffffffffu, c.z, 2);
      c.w += __shfl_xor_sync(0xffffffffu, c.w, 2);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool live = tok0 + j < size;
      float va = j ? c.y : c.x, vb = j ? c.w : c.z;
      if (FP4) {
        const float inv = pow2_field(254 - scale_exponent(am[j]));
        va *= inv, vb *= inv;
      }
      va += ba, vb += bb;
      if (PHASE == 2) {
        if (live) {
          float* y = a.slots + static_cast<int64_t>(pair[j]) * a.H;
          y[ra] = va;
          y[rb] = vb;
        }
        continue;
      }
      float m;
      if (a.gated) {
        const float v = glu(va, vb);
        if (live) a.act[static_cast<int64_t>(pair[j]) * a.I + sub * 8 * RT + rt * 8 + g] = v;
        m = fabsf(v);
        if (!(m >= 0.f)) m = INFINITY;
      } else {
        va = va > 0.f ? va * va : va != va ? va : 0.f;
        vb = vb > 0.f ? vb * vb : vb != vb ? vb : 0.f;
        if (live) {
          a.act[static_cast<int64_t>(pair[j]) * a.I + ra] = va;
          a.act[static_cast<int64_t>(pair[j]) * a.I + rb] = vb;
        }
        m = va == va && vb == vb ? fmaxf(va, vb) : INFINITY;
      }
      if (FP4) {  // the largest of the row: a maximum does not depend on the order
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (live && g == 0) atomicMax(a.amax + pair[j], __float_as_uint(m));
      }
    }
  }

  __device__ __forceinline__ void aim_columns(uint32_t unit, uint32_t (&bp)[NB], int& nb) const {
    const int size = unit_size(unit);
    nb = NB == 1 || size <= 4 ? 1 : NB == 2 || size <= 8 ? 2 : NB;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      bp[b] = (nb == 1 ? act_row(g >> 2, row_of_token(unit, g & 3))
                       : act_row(b & 1, row_of_token(unit, (b >> 1) * 8 + g))) +
              q * 16 - smem_u32(cta.smem);
  }

  __device__ __forceinline__ float4* partial(uint32_t seq) const {
    return cta.red + (seq % ML_BUFS) * (MAIN * JOBS * 32);
  }

  // Tiles [lo, hi) on a finishing warp: every ML_FINISH-th of them.
  __device__ __forceinline__ void finish_share(int lo, int hi) const {
    int u = lo / ph.tiles, tile = lo - u * ph.tiles;
#pragma unroll 1
    for (int t = lo; t < hi; ++t) {
      const uint32_t s = cta.seq + (t - lo);
      if (static_cast<int>(s % ML_FINISH) == warp - MAIN) {
        const uint32_t unit = plan.unit[u];
#pragma unroll 1
        for (int job = 0; job < RG * JOBS; ++job)
          finish(unit, tile, job, partial(s), [&] {
            if (job == 0)
              wait_or_abort(a, cta.abort, cta.full + 8 * (s % ML_BUFS), (s / ML_BUFS) & 1, DEV_TIMEOUT_FULL);
          });
        __syncwarp();
        if (lane == 0) mbar_arrive(cta.empty + 8 * (s % ML_BUFS));
      }
      if (++tile == ph.tiles) {
        tile = 0;
        ++u;
      }
    }
  }

  // A tile's end: this warp's partial sums to the finishing warp.
  __device__ __forceinline__ void hand_over(uint32_t s, Sums& t) const {
    flush(t);
    if (s >= ML_BUFS)
      wait_or_abort(a, cta.abort, cta.empty + 8 * (s % ML_BUFS), (s / ML_BUFS - 1) & 1, DEV_TIMEOUT_EMPTY);
    float4* part = partial(s) + warp * JOBS * 32 + lane;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int m = 0; m < NACC; ++m) {
        part[(rt * NACC + m) * 32] = make_float4(t.acc[rt][m][0], t.acc[rt][m][1], t.acc[rt][m][2], t.acc[rt][m][3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) t.acc[rt][m][j] = 0.f;
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(cta.full + 8 * (s % ML_BUFS));
  }

  // Tiles [lo, hi) on a main warp; the copies of the first DEPTH steps are under way.
  __device__ __forceinline__ void main_share(int lo, int hi, Cursor& c, uint32_t ring) const {
    int u = lo / ph.tiles, tile = lo - u * ph.tiles;
    Sums t = {};
    t.ref = 127;
    uint32_t s = cta.seq;
    uint32_t bp[NB];
    int nb = 1, slot = 0;
#pragma unroll 1
    for (int n = lo; n < hi; ++n, ++s, ++tile) {
      if (tile == ph.tiles) {
        tile = 0;
        ++u;
      }
      if (n == lo || tile == 0) {  // another unit
        const uint32_t unit = plan.unit[u];
        if (!(PHASE == 1 && a.all_rows)) {
          main_warps_sync<MAIN>();  // the old unit's rows are not read any more
          stage(unit);
          main_warps_sync<MAIN>();
        }
        aim_columns(unit, bp, nb);
      }
      uint32_t low[RT][2] = {};
      if (FP4) {
        const int sub = tile * RG + rg_warp;
        const uint32_t row = static_cast<uint32_t>(row_of(sub < ph.nsub ? sub : 0));
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r)  // an expert's scales are whole words
          low[r >> 1][r & 1] = (row * ph.scale_bytes + (r >> 1) * ph.s_rt + (r & 1) * ph.s_b) & 3u;
      }
      int ks = kw;
#pragma unroll 1
      for (int i = 0; i < c.nk; ++i, ks += ksplit) {
        const uint32_t at = ring + slot * SLOT;
        Frag<FMT, RT> f;
        take(f, at, low, ks);
        if (ks < ph.steps) {
          if (NB == 1 || nb == 1)
            products<1>(f, ks, bp, t);
          else if (NB == 2 || nb == 2)
            products<NB < 2 ? 1 : 2>(f, ks, bp, t);
          else
            products<NB>(f, ks, bp, t);
        }
        if (FP4) __syncwarp();  // the scales have been read by every lane
        issue(c, at);
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
      }
      hand_over(s, t);
    }
  }

  // The whole CTA: tiles [lo, hi), once the stage before is done; the first copies start before.
  __device__ __forceinline__ void share(int lo, int hi, const uint32_t* done, uint32_t shares) {
    if (warp < MAIN) {
      Cursor c;
      c.u = lo / ph.tiles;
      c.tile = lo - c.u * ph.tiles;
      c.left = hi - lo;
      c.nk = (ph.steps + ksplit - 1) / ksplit;
      c.i = 0;
      const uint32_t ring = cta.ring + warp * (DEPTH * SLOT);
#pragma unroll 1
      for (int d = 0; d < DEPTH; ++d) issue(c, ring + d * SLOT);
      if (done) wait_stage(a, cta.abort, done, shares);
      main_share(lo, hi, c, ring);
    } else {
      if (done) wait_stage(a, cta.abort, done, shares);
      finish_share(lo, hi);
    }
    cta.seq += hi - lo;
  }
};

// h of token t at columns j and j + 1: the arithmetic of moe.cuh, a batch of slots' loads at a time.
__device__ __forceinline__ void combine2(const MoeLayerArgs& a, int t, int j) {
  constexpr int BATCH = 8;
  float r0 = 0.f, r1 = 0.f, s0 = 0.f, s1 = 0.f;
  const uint32_t x = *reinterpret_cast<const uint32_t*>(a.x + static_cast<int64_t>(t) * a.H + j);
  for (int b = 0; b < a.S; b += BATCH) {
    float2 y[BATCH];
    float w[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (b + i < a.S) {
        y[i] = __ldcg(reinterpret_cast<const float2*>(a.slots + static_cast<int64_t>(t * a.S + b + i) * a.H + j));
        w[i] = __ldcg(a.slot_w + t * a.S + b + i);
      }
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (b + i < a.S) {
        moe_accumulate(b + i, a.topk, w[i], y[i].x, r0, s0);
        moe_accumulate(b + i, a.topk, w[i], y[i].y, r1, s1);
      }
  }
  *reinterpret_cast<uint32_t*>(a.h_out + static_cast<int64_t>(t) * a.H + j) =
      moe_finish(x & 0xffffu, r0, s0) | (moe_finish(x >> 16, r1, s1) << 16);
}

template <int FMT, int RT, int NB, int DEPTH, int MAIN>
__global__ void __launch_bounds__(32 * (MAIN + ML_FINISH), 1)
    moe_layer_kernel(const __grid_constant__ MoeLayerArgs a, const __grid_constant__ Phase ph1,
                     const __grid_constant__ Phase ph2, int ksplit1, int ksplit2) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_bar[2 * ML_BUFS];
  __shared__ float s_part[2 * ML_MAX_WARPS];
  __shared__ uint32_t s_top[ML_MAX_G];
  __shared__ uint32_t s_ticket;
  __shared__ int s_abort;
  const int tid = threadIdx.x;
  const int pairs = a.T * a.S, p8 = (pairs + 7) & ~7;
  constexpr int THREADS = 32 * (MAIN + ML_FINISH);
  Cta<MAIN> cta;
  cta.plan.pair_e = reinterpret_cast<uint16_t*>(smem);
  cta.plan.list = cta.plan.pair_e + p8;
  cta.plan.unit = reinterpret_cast<uint32_t*>(cta.plan.list + p8);
  cta.plan.cnt = cta.plan.unit + p8;
  cta.plan.red = cta.plan.cnt + ML_MAX_EXPERTS;
  cta.plan.nunits = -1;
  cta.smem = smem;
  uint8_t* rows = smem + ((plan_bytes(pairs) + 127) & ~127);
  cta.act = smem_u32(rows);
  uint8_t* red = rows + ((2 * a.R * max(ph1.pitch, ph2.pitch) + 127) & ~127);
  cta.red = reinterpret_cast<float4*>(red);
  cta.ring = smem_u32(red) + ML_BUFS * MAIN * RT * (NB == 4 ? 2 : 1) * 512;
  cta.full = smem_u32(s_bar);
  cta.empty = cta.full + 8 * ML_BUFS;
  cta.top = s_top;
  cta.abort = &s_abort;
  cta.seq = 0;
  if (tid == 0) {
    for (int i = 0; i < ML_BUFS; ++i) {
      mbar_init(cta.full + 8 * i, MAIN);
      mbar_init(cta.empty + 8 * i, 1);
    }
    fence_mbar_init();
    s_abort = 0;
    pdl_wait();  // the run before may still use the shared words
    s_ticket = atomicAdd(&a.ctl->ticket, 1u);
  } else {
    pdl_wait();
  }
  __syncthreads();
  const uint32_t n = gridDim.x;
  uint32_t ticket = s_ticket;
  // the first of `total` things that belong to share k of n
  auto cut = [&](uint32_t total, uint32_t k) {
    const uint32_t q = total / n;
    return static_cast<int>(q * k + (total - q * n) * k / n);
  };
  auto begin_share = [&] {  // asks for the next share
    __syncthreads();
    if (tid == THREADS - 1) s_ticket = atomicAdd(&a.ctl->ticket, 1u);
  };
  // The tiles of a product; none without a plan.  Not by the word that a wait has run out: a warp that is ahead may
  // set it while another reads it, and all have to walk the same tiles between barriers.  After it has been set no
  // wait lasts, and what is left to do is done on whatever stands in the scratch.
  auto tiles_of = [&](const Phase& ph) { return static_cast<uint32_t>(max(cta.plan.nunits, 0) * ph.tiles); };
  auto end_share = [&](int stage) {  // counts this one as done, and goes to the next
    __syncthreads();
    if (tid == THREADS - 32 && stage < 3) {
      __threadfence();
      atomicAdd(&a.ctl->done[stage], 1u);
    }
    ticket = s_ticket;
  };

#pragma unroll 1
  while (ticket < n) {
    begin_share();
    const uint32_t r = n - 1 - ticket;  // the tokens' statistics go to the last shares first
    router_share(a, cut(a.E, ticket), cut(a.E, ticket + 1), cut(a.T, r), cut(a.T, r + 1), reinterpret_cast<float*>(rows),
                 s_part);
    end_share(0);
  }
  if (ticket < 3 * n) {
    if (a.all_rows && ticket < 2 * n) {
      __syncthreads();
      Experts<FMT, RT, NB, 1, DEPTH, MAIN>(a, ph1, cta, ksplit1).stage_all(s_part);
    }
    wait_stage(a, cta.abort, a.ctl->done, n);
    if (!s_abort) {
      make_plan(a, cta.plan);
      if (ticket == n && tid >= 32 * MAIN)
#pragma unroll 1
        for (int t = (tid >> 5) - MAIN; t < a.T; t += ML_FINISH) write_routes(a, t, cta.plan.pair_e);
    }
  }
#pragma unroll 1
  while (ticket < 2 * n) {
    begin_share();
    const uint32_t i = ticket - n, tiles = tiles_of(ph1);
    Experts<FMT, RT, NB, 1, DEPTH, MAIN>(a, ph1, cta, ksplit1).share(cut(tiles, i), cut(tiles, i + 1), nullptr, 0u);
    end_share(1);
  }
#pragma unroll 1
  while (ticket < 3 * n) {
    begin_share();
    const uint32_t i = ticket - 2 * n, tiles = tiles_of(ph2);
    Experts<FMT, RT, NB, 2, DEPTH, MAIN>(a, ph2, cta, ksplit2).share(cut(tiles, i), cut(tiles, i + 1), a.ctl->done + 1, n);
    end_share(2);
  }
#pragma unroll 1
  while (a.h_out && ticket < 4 * n) {
    begin_share();
    wait_stage(a, cta.abort, a.ctl->done + 2, n);
    const uint32_t i = ticket - 3 * n;
    const int half = a.H / 2;
    const int lo = cut(a.T * half, i), hi = cut(a.T * half, i + 1);
#pragma unroll 1
    for (int p = lo + tid; p < hi && !s_abort; p += THREADS) combine2(a, p / half, 2 * (p % half));
    end_share(3);
  }
  if (tid == THREADS - 32) {
    __threadfence();
    if (atomicAdd(&a.ctl->left, 1u) == n - 1) {  // every other CTA is past its last use of these words
      a.ctl->ticket = 0u;
      for (int k = 0; k < 3; ++k) a.ctl->done[k] = 0u;
      a.ctl->left = 0u;
    }
  }
}

// ---------------------------------------------------------------- host
constexpr int STATIC_SMEM = 512;  // at least moe_layer_kernel's __shared__ variables

// Main warps, steps in flight of each and 16-row groups a warp takes at a time, for a format and the
// number of n-tiles.
constexpr int MAIN_WARPS = 12;
constexpr int depth_of(int nb) { return nb == 4 ? 2 : 4; }
constexpr int groups_of(int fmt, int nb) { return fmt == MXFP4 && nb < 4 ? 2 : 1; }
int step_cols(int fmt) { return fmt == BF16 ? 64 : fmt == MXFP4 ? 128 : 256; }
int slot_of(int fmt, int rt) {
  return fmt == BF16 ? slot_bytes<BF16, 1>() : fmt == MXFP4_WIDE ? slot_bytes<MXFP4_WIDE, 1>() : rt * slot_bytes<MXFP4, 1>();
}
int columns_of(int G) { return G <= 4 ? 1 : G <= 8 ? 2 : 4; }

// An activation row: whole k-steps, and 64 bytes more so that two rows fill the 128 bytes of all banks.
int pitch_of(int fmt, int K) {
  const int cols = step_cols(fmt);
  return (K + cols - 1) / cols * cols * 2 + 64;
}

// Warps that split K: a divisor k of the main warps, and MAIN / k of them share a tile's rows.  The largest k that
// keeps 85 % of their k-steps busy: small tiles spread evenly over the SMs (bf16, 8 tokens over 66 experts: 165 us
// with 192 rows a tile, 136 with 48).  A 4-bit k-step holds four times the columns of a bf16 one, so that a warp
// would often meet one of a tile, and a tile costs it as much as a k-step: there k falls while a warp's run is
// below 6 k-steps and the units' tiles are at least 4 an SM (16 tokens over 128 experts of 2880 columns: k = 12, runs
// of one, 263 us; 6: 222; 4: 211; 2, runs of six: 204; 1: 212.  One token, four experts: k = 12 36.7 us; 6, the
// rule's: 35.4; 4: 38).  bf16 under the same rule: 5 tokens 129 -> 130 us, 64 tokens 870 -> 873.
int ksplit_of(int fmt, int rt, int K, int N, int units, int sms) {
  const int steps = (K + step_cols(fmt) - 1) / step_cols(fmt), main = MAIN_WARPS;
  int best = 0;
  for (int k = main; k >= 1; --k) {
    const int run = (steps + k - 1) / k;  // k-steps of a warp in a tile
    if (main % k != 0 || 100 * steps < 85 * run * k) continue;
    if (best != 0 && (fmt == BF16 || steps >= 6 * best ||
                      static_cast<int64_t>(units) * N < static_cast<int64_t>(4) * sms * 16 * rt * (main / k)))
      break;
    best = k;
  }
  return best;  // k = 1 keeps all of them busy
}

Phase make_phase(const MoeLayerArgs& a, int fmt, int nb, int phase, int ksplit) {
  Phase p;
  const bool gated = phase == 1 && a.gated;
  const int RT = groups_of(fmt, nb), RG = MAIN_WARPS / ksplit;
  p.w = phase == 1 ? a.w1 : a.w2;
  p.s = phase == 1 ? a.s1 : a.s2;
  p.bias = phase == 1 ? a.b1 : a.b2;
  p.N = phase == 1 ? a.N1 : a.H;
  p.K = phase == 1 ? a.H : a.I;
  p.row_bytes = fmt == BF16 ? p.K * 2 : p.K / 2;
  p.scale_bytes = p.K / 32;
  p.a_mul = gated && a.interleaved ? 2 : 1;
  p.rt_step = gated ? (a.interleaved ? 16 : 8) : 16;
  p.b_step = gated ? (a.interleaved ? 1 : a.I) : 8;
  p.w_rt = p.rt_step * p.row_bytes;
  p.w_b = p.b_step * p.row_bytes;
  p.s_rt = p.rt_step * p.scale_bytes;
  p.s_b = p.b_step * p.scale_bytes;
  p.s_end = reinterpret_cast<uintptr_t>(p.s) + static_cast<uintptr_t>(a.E + a.nsh) * p.N * p.scale_bytes;
  p.nsub = p.N / (16 * RT);
  p.tiles = (p.nsub + RG - 1) / RG;
  p.steps = (p.K + step_cols(fmt) - 1) / step_cols(fmt);
  p.pitch = pitch_of(fmt, p.K);
  return p;
}

template <int FMT, int NB>
cudaError_t launch_as(const MoeLayerArgs& a, const MoeLayerPlan& p, cudaStream_t stream) {
  const Phase ph1 = make_phase(a, FMT, NB, 1, p.ksplit1), ph2 = make_phase(a, FMT, NB, 2, p.ksplit2);
  auto f = moe_layer_kernel<FMT, groups_of(FMT, NB), NB, depth_of(NB), MAIN_WARPS>;
  const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(32 * (MAIN_WARPS + ML_FINISH));
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, a, ph1, ph2, p.ksplit1, p.ksplit2);
}

template <int FMT>
cudaError_t launch_columns(const MoeLayerArgs& a, const MoeLayerPlan& p, cudaStream_t s) {
  switch (p.columns) {
    case 1: return launch_as<FMT, 1>(a, p, s);
    case 2: return launch_as<FMT, 2>(a, p, s);
    default: return launch_as<FMT, 4>(a, p, s);
  }
}

}  // namespace

// Tokens a unit may hold and the shared memory, with activation rows of the wider of the two products.
MoeLayerPlan plan_moe_layer(int T, int topk, int nsh, int E, int H, int I, int N1, bool fp4, int max_smem, int num_sms) {
  MoeLayerPlan p;
  max_smem -= STATIC_SMEM;  // the limit counts the kernel's own variables too
  p.grid = num_sms;
  p.format = !fp4 ? BF16 : H % 64 == 0 && I % 64 == 0 ? MXFP4_WIDE : MXFP4;
  const int pitch = pitch_of(p.format, H > I ? H : I);
  const int fixed = ((plan_bytes(T * (topk + nsh)) + 127) & ~127) + 128;
  // room for the tokens that share an expert when they spread evenly, and three standard deviations
  const float mean = static_cast<float>(T) * topk / E;
  const float room = mean + 3.0f * sqrtf(mean);
  const int most = nsh > 0 ? ML_MAX_G : room <= 4.0f ? 4 : room <= 8.0f ? 8 : ML_MAX_G;
  auto fits = [&](int G, int columns) {
    const int rt = groups_of(p.format, columns);
    p.G = p.R = G;
    p.columns = columns;
    p.all_rows = T <= G;
    p.smem = fixed + 2 * G * pitch + ML_BUFS * MAIN_WARPS * rt * (columns == 4 ? 2 : 1) * 512 +
             MAIN_WARPS * depth_of(columns) * slot_of(p.format, rt);
    return p.smem <= max_smem;
  };
  p.ok = false;
  for (int G = T < most ? T : most; G >= 1 && !p.ok; --G) p.ok = fits(G, columns_of(G));
  // the widest rows of an odd number of 4-bit blocks: the form with the least shared memory besides them (two steps
  // of one 16-row group in flight, 80 KB, instead of four of two, 172 KB)
  for (int G = T < most ? T : most; G >= 1 && !p.ok; --G) p.ok = fits(G, 4);
  const int units = (T * topk < E ? T * topk : E) + nsh, rt = groups_of(p.format, p.columns);
  p.ksplit1 = ksplit_of(p.format, rt, H, N1, units, num_sms);
  p.ksplit2 = ksplit_of(p.format, rt, I, H, units, num_sms);
  return p;
}

cudaError_t launch_moe_layer(const MoeLayerArgs& a, const MoeLayerPlan& p, cudaStream_t s) {
  return p.format == BF16 ? launch_columns<BF16>(a, p, s)
         : p.format == MXFP4 ? launch_columns<MXFP4>(a, p, s)
                             : launch_columns<MXFP4_WIDE>(a, p, s);
}

}  // namespace tail
