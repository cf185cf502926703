// Entry points of the mixture-of-experts layer: handle lifetime, argument checks,
// scratch and the launch.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <new>

#include "../../include/tail.h"
#include "abi_common.h"
#include "internal.h"
#include "moe_layer.cuh"
#include "moe_layer_internal.h"

using namespace tail;

struct tail_moe_s {
  tail_moe_config cfg;
  int device;
  int num_sms;
  int max_smem;
  int S, N1, n_all;
  uint8_t* scratch;
  int64_t scratch_bytes;
  // within scratch
  float* logits;
  float2* stats;
  float* act;
  uint32_t* amax;
  float* slots;
  float* slot_w;
  MoeControl* ctl;  // zero between launches
  int* err;
  uint64_t wait_limit_ns;
};

namespace {

bool valid(const tail_moe_config* c) {
  if (!c) return false;
  if (c->H < 1 || c->I < 1 || c->E < 1 || c->topk < 1 || c->topk > c->E || c->n_shared < 0) return false;
  if (c->t_max < 1 || !(c->eps >= 0.0f)) return false;
  if (c->weight_dtype != TAIL_BF16 && c->weight_dtype != TAIL_MXFP4) return false;
  if (c->act != TAIL_MOE_GLU && c->act != TAIL_MOE_RELU2) return false;
  if (c->score != TAIL_MOE_SOFTMAX && c->score != TAIL_MOE_SIGMOID) return false;
  if (!(c->act_limit >= 0.0f) || c->act_alpha != c->act_alpha || c->act_beta != c->act_beta) return false;
  return c->route_scale == c->route_scale;
}

bool supported(const tail_moe_config* c) {
  const int m = c->weight_dtype == TAIL_MXFP4 ? 32 : 16;
  return c->H % m == 0 && c->I % m == 0 && c->H <= ML_MAX_DIM && c->I <= ML_MAX_DIM && c->topk <= ML_MAX_TOPK &&
         c->n_shared <= ML_MAX_SHARED && c->E <= ML_MAX_EXPERTS - c->n_shared && c->t_max <= ML_MAX_T;
}

struct Span {
  const void* p;
  int64_t bytes;
};
bool meet(const Span& a, const Span& b) { return a.p && b.p && overlap(a.p, a.bytes, b.p, b.bytes); }

int64_t round256(int64_t v) { return (v + 255) & ~int64_t(255); }

}  // namespace

extern "C" {

int tail_moe_create(const tail_moe_config* cfg, int device, tail_moe_t** out) {
  if (!out) return TAIL_ERR_INVALID_ARG;
  *out = nullptr;
  if (!valid(cfg)) return TAIL_ERR_INVALID_ARG;
  if (!supported(cfg)) {
    set_last_error("tail_moe_create: H and I multiples of 16 (mxfp4: 32) up to 16384, E + n_shared <= 512, "
                   "topk <= 16, n_shared <= 8, t_max <= 64");
    return TAIL_ERR_UNSUPPORTED;
  }
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev) return TAIL_ERR_INVALID_ARG;
  DeviceGuard guard(device);
  if (!guard.ok) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
  cudaDeviceProp prop;
  cudaError_t e = cudaGetDeviceProperties(&prop, device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDeviceProperties");
  if (prop.major != 10 || prop.minor != 3) {
    set_last_error("tail_moe_create: built for sm_103a only");
    return TAIL_ERR_UNSUPPORTED;
  }
  tail_moe_t* m = new (std::nothrow) tail_moe_t();
  if (!m) return TAIL_ERR_OOM;
  memset(m, 0, sizeof(*m));
  m->cfg = *cfg;
  m->device = device;
  m->num_sms = prop.multiProcessorCount;
  m->max_smem = static_cast<int>(prop.sharedMemPerBlockOptin);
  m->S = cfg->topk + cfg->n_shared;
  m->N1 = cfg->act == TAIL_MOE_GLU ? 2 * cfg->I : cfg->I;
  m->n_all = cfg->E + cfg->n_shared;
  const int64_t T = cfg->t_max, pairs = T * m->S;
  const int64_t sizes[] = {T * cfg->E * 4, T * 8, pairs * cfg->I * 4, pairs * 4, pairs * cfg->H * 4, pairs * 4,
                           static_cast<int64_t>(sizeof(MoeControl)), 4};
  for (int64_t n : sizes) m->scratch_bytes += round256(n);
  e = cudaMalloc(reinterpret_cast<void**>(&m->scratch), static_cast<size_t>(m->scratch_bytes));
  if (e == cudaSuccess) e = cudaMemset(m->scratch, 0, static_cast<size_t>(m->scratch_bytes));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    if (m->scratch) cudaFree(m->scratch);
    delete m;
    return cuda_fail(e, "tail_moe_create: scratch allocation");
  }
  uint8_t* p = m->scratch;
  m->logits = reinterpret_cast<float*>(p);
  m->stats = reinterpret_cast<float2*>(p += round256(sizes[0]));
  m->act = reinterpret_cast<float*>(p += round256(sizes[1]));
  m->amax = reinterpret_cast<uint32_t*>(p += round256(sizes[2]));
  m->slots = reinterpret_cast<float*>(p += round256(sizes[3]));
  m->slot_w = reinterpret_cast<float*>(p += round256(sizes[4]));
  m->ctl = reinterpret_cast<MoeControl*>(p += round256(sizes[5]));
  m->err = reinterpret_cast<int*>(p += round256(sizes[6]));
  m->wait_limit_ns = DEFAULT_TIMEOUT_NS;
  *out = m;
  return TAIL_OK;
}

int tail_moe_run(tail_moe_t* m, const uint16_t* x, const float* gamma_opt, const uint16_t* router_w,
                 const float* router_bias_opt, const void* w1, const uint8_t* w1_scale, const float* b1_opt,
                 const void* w2, const uint8_t* w2_scale, const float* b2_opt, int32_t n_tokens,
                 uint16_t* out_hidden_opt, float* out_slots_opt, float* out_slot_w_opt, int32_t* out_ids_opt,
                 void* stream) {
  if (!m || n_tokens < 0 || n_tokens > m->cfg.t_max) return TAIL_ERR_INVALID_ARG;
  if (n_tokens == 0) return TAIL_OK;
  const tail_moe_config& c = m->cfg;
  const bool fp4 = c.weight_dtype == TAIL_MXFP4;
  if (!x || !router_w || !w1 || !w2 || (fp4 && (!w1_scale || !w2_scale))) return TAIL_ERR_INVALID_ARG;
  if (fp4 && (!aligned(w1_scale, 16) || !aligned(w2_scale, 16))) return TAIL_ERR_INVALID_ARG;
  if (!out_hidden_opt && !out_slots_opt) return TAIL_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(router_w, 16) || !aligned(gamma_opt, 16) || !aligned(w1, 32) || !aligned(w2, 32))
    return TAIL_ERR_INVALID_ARG;
  if (!aligned(router_bias_opt, 4) || !aligned(b1_opt, 4) || !aligned(b2_opt, 4) || !aligned(out_hidden_opt, 16) ||
      !aligned(out_slots_opt, 16) || !aligned(out_slot_w_opt, 4) || !aligned(out_ids_opt, 4))
    return TAIL_ERR_INVALID_ARG;
  // CTAs read inputs while others write outputs, so none may meet another; but x is read again where the slots are
  // combined, and h in place of x is an element-wise replacement
  const int64_t T = n_tokens, H = c.H, n1 = m->n_all * static_cast<int64_t>(m->N1), n2 = m->n_all * H;
  const Span in[] = {{x, T * H * 2},          {gamma_opt, H * 4},  {router_w, c.E * H * 2}, {router_bias_opt, c.E * 4LL},
                     {w1, fp4 ? n1 * H / 2 : n1 * H * 2},          {w1_scale, fp4 ? n1 * H / 32 : 0},
                     {b1_opt, n1 * 4},        {w2, fp4 ? n2 * c.I / 2 : n2 * c.I * 2},
                     {w2_scale, fp4 ? n2 * c.I / 32 : 0},          {b2_opt, n2 * 4}};
  const Span out[] = {{out_hidden_opt, T * H * 2},
                      {out_slots_opt, T * m->S * H * 4},
                      {out_slot_w_opt, T * m->S * 4},
                      {out_ids_opt, T * m->S * 4}};
  for (const Span& o : out) {
    for (const Span& i : in)
      if (meet(o, i) && !(o.p == out_hidden_opt && i.p == x && o.p == i.p)) return TAIL_ERR_INVALID_ARG;
    for (const Span* other = out; other < &o; ++other)
      if (meet(o, *other)) return TAIL_ERR_INVALID_ARG;
  }
  DeviceGuard guard(m->device);
  if (!guard.ok) return TAIL_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const MoeLayerPlan plan = plan_moe_layer(n_tokens, c.topk, c.n_shared, c.E, c.H, c.I, m->N1, fp4, m->max_smem,
                                           m->num_sms);
  if (!plan.ok) return TAIL_ERR_UNSUPPORTED;  // not reached within the limits of create
  MoeLayerArgs a;
  a.x = x;
  a.gamma = gamma_opt;
  a.wr = router_w;
  a.br = router_bias_opt;
  a.w1 = static_cast<const uint8_t*>(w1);
  a.s1 = w1_scale;
  a.b1 = b1_opt;
  a.w2 = static_cast<const uint8_t*>(w2);
  a.s2 = w2_scale;
  a.b2 = b2_opt;
  a.logits = m->logits;
  a.stats = m->stats;
  a.act = m->act;
  a.amax = m->amax;
  a.slots = out_slots_opt ? out_slots_opt : m->slots;
  a.slot_w = out_slot_w_opt ? out_slot_w_opt : m->slot_w;
  a.ids = out_ids_opt;
  a.T = n_tokens;
  a.H = c.H;
  a.I = c.I;
  a.N1 = m->N1;
  a.E = c.E;
  a.topk = c.topk;
  a.nsh = c.n_shared;
  a.S = m->S;
  a.gated = c.act == TAIL_MOE_GLU;
  a.interleaved = c.interleaved ? 1 : 0;
  a.score = c.score == TAIL_MOE_SIGMOID;
  a.alpha = c.act_alpha;
  a.beta = c.act_beta;
  a.limit = c.act_limit;
  a.route_scale = c.route_scale;
  a.eps = c.eps;
  a.G = plan.G;
  a.R = plan.R;
  a.all_rows = plan.all_rows;
  a.h_out = out_hidden_opt;
  a.ctl = m->ctl;
  a.err = m->err;
  a.timeout_ns = m->wait_limit_ns;
  const cudaError_t e = launch_moe_layer(a, plan, s);
  if (e != cudaSuccess) return cuda_fail(e, "tail_moe_run: kernel launch");
  return TAIL_OK;
}

int tail_moe_check(tail_moe_t* m) {
  if (!m) return TAIL_ERR_INVALID_ARG;
  DeviceGuard guard(m->device);
  if (!guard.ok) return TAIL_ERR_CUDA;
  cudaError_t e = cudaDeviceSynchronize();
  int code = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&code, m->err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && code != 0) e = cudaMemset(m->err, 0, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e, "tail_moe_check");
  return code != 0 ? TAIL_ERR_DEVICE : TAIL_OK;
}

int tail_moe_set_wait_limit(tail_moe_t* m, uint64_t ns) {
  if (!m) return TAIL_ERR_INVALID_ARG;
  m->wait_limit_ns = ns;
  return TAIL_OK;
}

int tail_moe_get_info(const tail_moe_t* m, int64_t* scratch_bytes) {
  if (!m || !scratch_bytes) return TAIL_ERR_INVALID_ARG;
  *scratch_bytes = m->scratch_bytes;
  return TAIL_OK;
}

void tail_moe_destroy(tail_moe_t* m) {
  if (!m) return;
  DeviceGuard guard(m->device);
  if (guard.ok) {
    cudaDeviceSynchronize();
    cudaFree(m->scratch);
    cudaGetLastError();
  }
  delete m;
}

}  // extern "C"
