// Kernels of the mixture-of-experts layer for a few tokens (moe_layer.cuh states
// the formulas and the fragment layout).
#include "internal.h"
#include "moe_layer.cuh"
#include "moe_layer_internal.h"

namespace tail {

namespace {

// ---------------------------------------------------------------- router
constexpr int ROUTER_THREADS = 256;
constexpr int ROUTER_WARPS = ROUTER_THREADS / 32;

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

// CTA e < E: the logits of expert e for every token, a warp a token.  CTA E + t: 1 / rms and the
// largest |t| of token t, and the largest-activation words of its pairs cleared.
__global__ void __launch_bounds__(ROUTER_THREADS) moe_router_kernel(const MoeLayerArgs a) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ float s_sum[ROUTER_WARPS], s_max[ROUTER_WARPS];
  if (static_cast<int>(blockIdx.x) < a.E) {
    const int e = blockIdx.x;
    const uint16_t* w = a.wr + static_cast<int64_t>(e) * a.H;
    for (int t = warp; t < a.T; t += ROUTER_WARPS) {
      const uint16_t* x = a.x + static_cast<int64_t>(t) * a.H;
      float dot = 0.f, ss = 0.f;
      for (int k = lane * 8; k < a.H; k += 256) {
        float xf[8], wf[8], g[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(x + k)), xf);
        unpack8(__ldg(reinterpret_cast<const uint4*>(w + k)), wf);
        load_gamma(a.gamma, k, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(xf[i], xf[i], ss);
          dot = fmaf(xf[i] * wf[i], g[i], dot);
        }
      }
      dot = warp_sum(dot);
      ss = warp_sum(ss);
      if (lane == 0) {
        const float r = a.gamma ? 1.0f / sqrtf(ss / static_cast<float>(a.H) + a.eps) : 1.0f;
        a.logits[static_cast<int64_t>(t) * a.E + e] = dot * r;
      }
    }
    return;
  }
  const int t = blockIdx.x - a.E;
  const uint16_t* x = a.x + static_cast<int64_t>(t) * a.H;
  float ss = 0.f, mx = 0.f;
  bool bad = false;
  for (int k = tid * 8; k < a.H; k += ROUTER_THREADS * 8) {
    float xf[8], g[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(x + k)), xf);
    load_gamma(a.gamma, k, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss = fmaf(xf[i], xf[i], ss);
      const float v = fabsf(xf[i] * g[i]);
      mx = fmaxf(mx, v);
      bad |= !(v <= 3.402823466e38f);
    }
  }
  if (bad) mx = INFINITY;
  ss = warp_sum(ss);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) {
    s_sum[warp] = ss;
    s_max[warp] = mx;
  }
  for (int s = tid; s < a.S; s += ROUTER_THREADS) a.amax[t * a.S + s] = 0u;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < ROUTER_WARPS; ++w) {
      ss += s_sum[w];
      mx = fmaxf(mx, s_max[w]);
    }
    const float r = a.gamma ? 1.0f / sqrtf(ss / static_cast<float>(a.H) + a.eps) : 1.0f;
    a.stats[t] = make_float2(r, mx * r);
  }
}

// ---------------------------------------------------------------- experts
// The two products of the experts have one form: rows of a weight [n][N][K], K contiguous, against
// up to 16 tokens' activations in shared memory.
//
// Work is cut into tiles of a unit (an expert and up to G of its tokens): RG subtiles of 16 * RT
// rows, whose K is split over 16 / RG warps.  A CTA takes a contiguous share of all tiles.  Each warp
// keeps the fragments of its next DEPTH k-steps in registers, across tile borders; at the end of a
// tile the warps' partial sums meet in shared memory (two buffers, one barrier a tile) and one warp a
// subtile adds them in a fixed order and finishes the rows while the others go on.
template <bool FP4>
struct Step {
  static constexpr int COLS = FP4 ? 128 : 64;     // columns of one k-step of a warp
  static constexpr int LANE_BYTES = FP4 ? 16 : 32;
  static constexpr int WORDS = LANE_BYTES / 4;
  static constexpr int STEP_BYTES = 4 * LANE_BYTES;
};

struct Phase {
  const uint8_t* w;
  const uint8_t* s;
  const float* bias;
  int N, K;
  int row_bytes, scale_bytes;
  int a_mul, rt_step, b_step;  // row of (subtile, rt, half, g): sub * a_mul * RT * .. (row_of)
  int nsub, tiles;             // subtiles and tiles of a unit
  int steps;                   // k-steps
  int pitch;                   // bytes of one activation row in shared memory
};

template <bool FP4, int RT>
struct Frag {
  uint32_t w[RT][2][Step<FP4>::WORDS];
  uint32_t s[RT][2];
};

template <bool FP4, int RT, int NB, int PHASE, int DEPTH>
struct Experts {
  static constexpr int NACC = NB == 4 ? 2 : 1;
  using S = Step<FP4>;

  const MoeLayerArgs& a;
  const Phase& ph;
  const MoePlan& plan;
  uint32_t act;        // shared memory: 2 G activation rows
  float4* red;         // [2][ML_WARPS][RT * NACC][32]
  int ksplit, rg_warp, kw, RG;
  int lane, warp, g, q;

  __device__ __forceinline__ int64_t row_of(int sub) const {
    // first row (rt = 0, half 0) of this lane's fragment
    if (PHASE == 1 && a.gated) return static_cast<int64_t>(sub * 8 * RT + g) * ph.a_mul;
    return static_cast<int64_t>(sub) * 16 * RT + g;
  }

  // the activation row of a token's high (plane 0) or low (plane 1) part
  __device__ __forceinline__ uint32_t act_row(int plane, int tok) const {
    return act + static_cast<uint32_t>(plane * a.G + min(tok, a.G - 1)) * ph.pitch;
  }

  // Activations of a unit into shared memory, split into a high and a low 16-bit part so that the
  // products carry them to about 2^-17 (bf16) or 2^-22 (fp16, scaled by a power of two a token).
  __device__ __forceinline__ void stage(uint32_t unit) const {
    const int n = unit_size(unit), first = unit_first(unit);
    const int kpad = ph.steps * S::COLS, chunks = kpad / 8;
    for (int i = threadIdx.x; i < n * chunks; i += ML_THREADS) {
      const int tok = i / chunks, k = (i - tok * chunks) * 8;
      const int pair = plan.list[first + tok];
      float v[8];
      float mult = 1.f;
      if (k >= ph.K) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
      } else if (PHASE == 1) {
        const int t = pair / a.S;
        const float2 st = __ldcg(a.stats + t);
        float gm[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(t) * a.H + k)), v);
        load_gamma(a.gamma, k, gm);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * st.x * gm[j];
        if (FP4) mult = pow2_field(scale_exponent(__float_as_uint(st.y)));
      } else {
        const float4* p = reinterpret_cast<const float4*>(a.act + static_cast<int64_t>(pair) * a.I + k);
        const float4 x = __ldcg(p), y = __ldcg(p + 1);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
        if (FP4) mult = pow2_field(scale_exponent(__ldcg(a.amax + pair)));
      }
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
          const __nv_bfloat162 l =
              __floats2bfloat162_rn(v[2 * j] - __low2float(h), v[2 * j + 1] - __high2float(h));
          hi[j] = reinterpret_cast<const uint32_t&>(h);
          lo[j] = reinterpret_cast<const uint32_t&>(l);
        }
      }
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(act_row(0, tok) + k * 2), "r"(hi[0]), "r"(hi[1]),
                   "r"(hi[2]), "r"(hi[3])
                   : "memory");
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(act_row(1, tok) + k * 2), "r"(lo[0]), "r"(lo[1]),
                   "r"(lo[2]), "r"(lo[3])
                   : "memory");
    }
  }

  struct Cursor {
    int tile, i;
    const uint8_t* w;  // null: no rows here for this warp
    const uint8_t* s;
  };

  __device__ __forceinline__ void aim(Cursor& c) const {
    const int u = c.tile / ph.tiles;
    const int sub = (c.tile - u * ph.tiles) * RG + rg_warp;
    c.w = nullptr;
    if (sub < ph.nsub) {
      const int64_t row = static_cast<int64_t>(unit_expert(plan.unit[u])) * ph.N + row_of(sub);
      c.w = ph.w + row * ph.row_bytes + q * S::LANE_BYTES;
      if (FP4) c.s = ph.s + row * ph.scale_bytes + q;
    }
  }

  __device__ __forceinline__ void load(Frag<FP4, RT>& f, Cursor& c, int nk) const {
    if (c.i == 0) aim(c);
    const int ks = kw + c.i * ksplit;
    const bool in = c.w != nullptr && ks * S::COLS + q * (S::COLS / 4) < ph.K;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t r = rt * ph.rt_step + h * ph.b_step;
        if (in) {
          ldg_stream(c.w + r * ph.row_bytes + ks * S::STEP_BYTES, f.w[rt][h]);
          if (FP4) f.s[rt][h] = __ldg(c.s + r * ph.scale_bytes + ks * 4);
        } else {
#pragma unroll
          for (int j = 0; j < S::WORDS; ++j) f.w[rt][h][j] = 0u;
          f.s[rt][h] = 0u;
        }
      }
    if (++c.i == nk) {
      c.i = 0;
      ++c.tile;
    }
  }

  // acc += the fragment's products; nb n-tiles of 8 columns (nb == 1: 4 high, 4 low columns)
  __device__ __forceinline__ void products(Frag<FP4, RT>& f, int ks, const uint32_t (&bp)[NB], int nb,
                                           float (&acc)[RT][NACC][4]) const {
    if constexpr (!FP4) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (b < nb) {
          uint32_t v[8];
          lds128(bp[b] + ks * 128, v[0], v[1], v[2], v[3]);
          lds128(bp[b] + ks * 128 + 16, v[4], v[5], v[6], v[7]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_bf16_16816(acc[rt][b >> 1], f.w[rt][0][2 * j], f.w[rt][1][2 * j], f.w[rt][0][2 * j + 1],
                             f.w[rt][1][2 * j + 1], v[2 * j], v[2 * j + 1]);
        }
      }
    } else {
      // Each lane's scale relative to the largest of the four blocks of its row goes into the values
      // (a power of two: exact), the largest itself into the fp32 sums.
      float d[RT][NACC][4];
      float fac[RT][2];
      uint32_t sc[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int n = 0; n < NACC; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) d[rt][n][j] = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int m = f.s[rt][h];
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
          sc[rt][h] = half_pow2(f.s[rt][h], m);
          fac[rt][h] = e8m0(m);
        }
      }
      const bool swap = q >= 2;  // lanes 2 and 3 take their words in another order: no two share banks
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int piece = swap ? w ^ 1 : w;
        uint32_t v[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (b < nb) lds128(bp[b] + ks * 256 + piece * 16, v[b][0], v[b][1], v[b][2], v[b][3]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          uint32_t x[4], y[4];
          fp4_to_half(swap ? f.w[rt][0][w ^ 1] : f.w[rt][0][w], sc[rt][0], x);
          fp4_to_half(swap ? f.w[rt][1][w ^ 1] : f.w[rt][1][w], sc[rt][1], y);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            if (b < nb) {
              mma_f16_16816(d[rt][b >> 1], x[0], y[0], x[1], y[1], v[b][0], v[b][1]);
              mma_f16_16816(d[rt][b >> 1], x[2], y[2], x[3], y[3], v[b][2], v[b][3]);
            }
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int n = 0; n < NACC; ++n) {
          acc[rt][n][0] = fmaf(d[rt][n][0], fac[rt][0], acc[rt][n][0]);
          acc[rt][n][1] = fmaf(d[rt][n][1], fac[rt][0], acc[rt][n][1]);
          acc[rt][n][2] = fmaf(d[rt][n][2], fac[rt][1], acc[rt][n][2]);
          acc[rt][n][3] = fmaf(d[rt][n][3], fac[rt][1], acc[rt][n][3]);
        }
    }
  }

  __device__ __forceinline__ float glu(float gate, float up) const {
    if (a.limit > 0.f) {
      gate = gate > a.limit ? a.limit : gate;  // NaN stays
      up = up > a.limit ? a.limit : up < -a.limit ? -a.limit : up;
    }
    return gate / (1.0f + expf(-a.alpha * gate)) * (up + a.beta);
  }

  // One warp: the rows of subtile (rg, rt) for the tokens 8 * n .. of the unit.
  __device__ __forceinline__ void finish(uint32_t unit, int tile_in_unit, int job, const float4* part) const {
    const int n = job % NACC, rt = (job / NACC) % RT, rg = job / (NACC * RT);
    const int sub = tile_in_unit * RG + rg;
    if (sub >= ph.nsub) return;
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < ksplit; ++k) {
      const float4 p = part[((rg * ksplit + k) * (RT * NACC) + rt * NACC + n) * 32 + lane];
      c.x += p.x, c.y += p.y, c.z += p.z, c.w += p.w;
    }
    const int size = unit_size(unit), first = unit_first(unit), e = unit_expert(unit);
    if (NB == 1 || size <= 4) {  // columns 0-3 high parts, 4-7 low parts
      c.x += __shfl_xor_sync(0xffffffffu, c.x, 2);
      c.y += __shfl_xor_sync(0xffffffffu, c.y, 2);
      c.z += __shfl_xor_sync(0xffffffffu, c.z, 2);
      c.w += __shfl_xor_sync(0xffffffffu, c.w, 2);
    }
    const int tok0 = n * 8 + 2 * q;
    const int64_t ra = row_of(sub) + rt * ph.rt_step, rb = ra + ph.b_step;
    const float* bias = ph.bias ? ph.bias + static_cast<int64_t>(e) * ph.N : nullptr;
    const float ba = bias ? __ldg(bias + ra) : 0.f, bb = bias ? __ldg(bias + rb) : 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tok = tok0 + j;
      const bool live = tok < size;
      const int pair = live ? plan.list[first + tok] : 0;
      float va = j ? c.y : c.x, vb = j ? c.w : c.z;
      if (FP4) {
        const uint32_t am = !live ? 0u
                            : PHASE == 1 ? __float_as_uint(__ldcg(&a.stats[pair / a.S].y))
                                         : __ldcg(a.amax + pair);
        const float inv = pow2_field(254 - scale_exponent(am));
        va *= inv, vb *= inv;
      }
      va += ba, vb += bb;
      if (PHASE == 2) {
        if (live) {
          float* y = a.slots + static_cast<int64_t>(pair) * a.H;
          y[ra] = va;
          y[rb] = vb;
        }
        continue;
      }
      float m;
      if (a.gated) {
        const float v = glu(va, vb);
        if (live) a.act[static_cast<int64_t>(pair) * a.I + sub * 8 * RT + rt * 8 + g] = v;
        m = fabsf(v);
        if (!(m >= 0.f)) m = INFINITY;
      } else {
        va = va > 0.f ? va * va : va != va ? va : 0.f;
        vb = vb > 0.f ? vb * vb : vb != vb ? vb : 0.f;
        if (live) {
          a.act[static_cast<int64_t>(pair) * a.I + ra] = va;
          a.act[static_cast<int64_t>(pair) * a.I + rb] = vb;
        }
        m = va == va && vb == vb ? fmaxf(va, vb) : INFINITY;
      }
      if (FP4) {  // the largest of the row: a maximum does not depend on the order
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (live && g == 0) atomicMax(a.amax + pair, __float_as_uint(m));
      }
    }
  }

  __device__ __forceinline__ void aim_columns(uint32_t unit, uint32_t (&bp)[NB], int& nb) const {
    const int size = unit_size(unit);
    nb = NB == 1 || size <= 4 ? 1 : NB == 2 || size <= 8 ? 2 : NB;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      bp[b] = (nb == 1 ? act_row(g >> 2, g & 3) : act_row(b & 1, (b >> 1) * 8 + g)) + q * (S::COLS / 4) * 2;
  }

  __device__ __forceinline__ void run(int lo, int hi) {
    if (lo >= hi) return;
    const int nk = (ph.steps + ksplit - 1) / ksplit;
    const int total = (hi - lo) * nk;
    Cursor c;
    c.tile = lo;
    c.i = 0;
    Frag<FP4, RT> f[DEPTH];
#pragma unroll
    for (int s = 0; s < DEPTH; ++s)
      if (s < total) load(f[s], c, nk);
    int u = lo / ph.tiles;
    int in_unit = lo - u * ph.tiles;
    uint32_t unit = plan.unit[u];
    stage(unit);
    __syncthreads();
    uint32_t bp[NB];
    int nb;
    aim_columns(unit, bp, nb);
    float acc[RT][NACC][4] = {};
    int i = 0, done = 0, turn = 0;
    for (int base = 0; base < total; base += DEPTH) {
#pragma unroll
      for (int s = 0; s < DEPTH; ++s) {
        if (base + s >= total) break;
        const int ks = kw + i * ksplit;
        if (ks < ph.steps) products(f[s], ks, bp, nb, acc);
        if (base + s + DEPTH < total) load(f[s], c, nk);
        if (++i == nk) {  // the tile's end
          i = 0;
          float4* part = red + (done & 1) * (ML_WARPS * RT * NACC * 32);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int n = 0; n < NACC; ++n) {
              part[(warp * (RT * NACC) + rt * NACC + n) * 32 + lane] =
                  make_float4(acc[rt][n][0], acc[rt][n][1], acc[rt][n][2], acc[rt][n][3]);
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[rt][n][j] = 0.f;
            }
          __syncthreads();
          const int jobs = RG * RT * NACC;
          for (int job = (warp - turn) & (ML_WARPS - 1); job < jobs; job += ML_WARPS)
            if (NACC == 1 || job % NACC == 0 || unit_size(unit) > 8) finish(unit, in_unit, job, part);
          turn += jobs;
          ++done;
          if (++in_unit == ph.tiles && lo + done < hi) {
            in_unit = 0;
            unit = plan.unit[++u];
            stage(unit);  // every warp is past the barrier: the old rows are not read any more
            __syncthreads();
            aim_columns(unit, bp, nb);
          }
        }
      }
    }
  }
};

template <bool FP4, int RT, int NB, int PHASE, int DEPTH>
__global__ void __launch_bounds__(ML_THREADS, 1) moe_experts_kernel(const MoeLayerArgs a, const Phase ph, int ksplit) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int pairs = a.T * a.S, p8 = (pairs + 7) & ~7;
  MoePlan plan;
  plan.pair_e = reinterpret_cast<uint16_t*>(smem);
  plan.list = plan.pair_e + p8;
  plan.unit = reinterpret_cast<uint32_t*>(plan.list + p8);
  plan.cnt = plan.unit + p8;
  plan.red = plan.cnt + ML_MAX_EXPERTS;
  make_plan(a, plan, PHASE == 1 && blockIdx.x == 0);
  uint8_t* act = smem + ((plan_bytes(pairs) + 127) & ~127);
  const int tid = threadIdx.x;
  Experts<FP4, RT, NB, PHASE, DEPTH> x{a, ph, plan};
  x.act = smem_u32(act);
  x.red = reinterpret_cast<float4*>(act + ((2 * a.G * ph.pitch + 127) & ~127));
  x.lane = tid & 31;
  x.warp = tid >> 5;
  x.g = x.lane >> 2;
  x.q = x.lane & 3;
  x.ksplit = ksplit;
  x.RG = ML_WARPS / ksplit;
  x.rg_warp = x.warp / ksplit;
  x.kw = x.warp - x.rg_warp * ksplit;
  const int64_t tiles = static_cast<int64_t>(plan.nunits) * ph.tiles;
  x.run(static_cast<int>(tiles * blockIdx.x / gridDim.x), static_cast<int>(tiles * (blockIdx.x + 1) / gridDim.x));
}

// ---------------------------------------------------------------- host
template <bool FP4, int RT>
Phase make_phase(const MoeLayerArgs& a, int phase, int ksplit) {
  Phase p;
  const bool gated = phase == 1 && a.gated;
  p.w = phase == 1 ? a.w1 : a.w2;
  p.s = phase == 1 ? a.s1 : a.s2;
  p.bias = phase == 1 ? a.b1 : a.b2;
  p.N = phase == 1 ? a.N1 : a.H;
  p.K = phase == 1 ? a.H : a.I;
  p.row_bytes = FP4 ? p.K / 2 : p.K * 2;
  p.scale_bytes = p.K / 32;
  p.a_mul = gated && a.interleaved ? 2 : 1;
  p.rt_step = gated ? (a.interleaved ? 16 : 8) : 16;
  p.b_step = gated ? (a.interleaved ? 1 : a.I) : 8;
  p.nsub = p.N / (16 * RT);
  const int RG = ML_WARPS / ksplit;
  p.tiles = (p.nsub + RG - 1) / RG;
  p.steps = (p.K + Step<FP4>::COLS - 1) / Step<FP4>::COLS;
  p.pitch = p.steps * Step<FP4>::COLS * 2 + (FP4 ? 32 : 16);
  return p;
}

int pitch_of(bool fp4, int K) {
  const int cols = fp4 ? 128 : 64;
  return (K + cols - 1) / cols * cols * 2 + (fp4 ? 32 : 16);
}

// Warps that split K: as many as leave every warp two k-steps.
int ksplit_of(bool fp4, int K) {
  const int steps = (K + (fp4 ? 127 : 63)) / (fp4 ? 128 : 64);
  int k = ML_WARPS;
  while (k > 1 && steps < 2 * k) k >>= 1;
  return k;
}

int columns_of(int G) { return G <= 4 ? 1 : G <= 8 ? 2 : 4; }

template <bool FP4, int RT, int NB, int DEPTH>
cudaError_t launch_experts(const MoeLayerArgs& a, int phase, int grid, int smem, int ksplit, cudaStream_t stream) {
  const Phase ph = make_phase<FP4, RT>(a, phase, ksplit);
  const void* f = phase == 1 ? reinterpret_cast<const void*>(moe_experts_kernel<FP4, RT, NB, 1, DEPTH>)
                             : reinterpret_cast<const void*>(moe_experts_kernel<FP4, RT, NB, 2, DEPTH>);
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<MoeLayerArgs*>(&a), const_cast<Phase*>(&ph), &ksplit};
  return cudaLaunchKernel(f, dim3(grid), dim3(ML_THREADS), args, smem, stream);
}

template <bool FP4>
cudaError_t launch_phase(const MoeLayerArgs& a, const MoeLayerPlan& p, int phase, cudaStream_t s) {
  const int ks = phase == 1 ? p.ksplit1 : p.ksplit2;
  switch (columns_of(a.G)) {
    case 1: return launch_experts<FP4, FP4 ? 2 : 1, 1, FP4 ? 3 : 4>(a, phase, p.grid, p.smem, ks, s);
    case 2: return launch_experts<FP4, FP4 ? 2 : 1, 2, FP4 ? 3 : 4>(a, phase, p.grid, p.smem, ks, s);
    default: return launch_experts<FP4, 1, 4, 4>(a, phase, p.grid, p.smem, ks, s);
  }
}

}  // namespace

// Tokens a unit may hold and the shared memory, for `pairs` pairs and activation rows of the wider
// of the two products.
MoeLayerPlan plan_moe_layer(int T, int S, int H, int I, bool fp4, int max_smem, int num_sms) {
  MoeLayerPlan p;
  p.grid = num_sms;
  const int pitch = pitch_of(fp4, H > I ? H : I);
  const int fixed = ((plan_bytes(T * S) + 127) & ~127) + 128;
  p.G = T < 16 ? T : 16;
  for (;; --p.G) {
    const int nb = columns_of(p.G);
    const int rt = fp4 && nb < 4 ? 2 : 1;
    const int red = 2 * ML_WARPS * rt * (nb == 4 ? 2 : 1) * 512;
    p.smem = fixed + 2 * p.G * pitch + red;
    if (p.smem <= max_smem || p.G == 1) break;
  }
  p.ok = p.smem <= max_smem;
  p.ksplit1 = ksplit_of(fp4, H);
  p.ksplit2 = ksplit_of(fp4, I);
  return p;
}

cudaError_t launch_moe_layer(const MoeLayerArgs& a, const MoeLayerPlan& p, bool fp4, cudaStream_t s) {
  moe_router_kernel<<<a.E + a.T, ROUTER_THREADS, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  for (int phase = 1; phase <= 2 && e == cudaSuccess; ++phase)
    e = fp4 ? launch_phase<true>(a, p, phase, s) : launch_phase<false>(a, p, phase, s);
  return e;
}

}  // namespace tail
