// C entry points of the sequence-mixing operators declared in include/pnr.h: argument
// checks (before any HIP call) and the launches, nothing else.
#include <math.h>

#include "seq_ops.h"

using namespace pnr;

namespace {

int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return PNR_OK;
  return record_error(PNR_E_HIP, "%s failed: %s", what, hipGetErrorString(e));
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return PNR_OK;
  if (!ws) return record_error(PNR_E_WORKSPACE, "workspace is NULL (%zu bytes required)", need);
  if (reinterpret_cast<uintptr_t>(ws) % 256) return record_error(PNR_E_WORKSPACE, "workspace must be 256-byte aligned");
  if (have < need) return record_error(PNR_E_WORKSPACE, "workspace has %zu bytes, %zu required", have, need);
  return PNR_OK;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_dtype(int dtype) {
  if (dtype < PNR_F64 || dtype > PNR_BF16) return record_error(PNR_E_INVALID, "unknown dtype %d", dtype);
  if (dtype == PNR_F64) return record_error(PNR_E_UNSUPPORTED, "this operator supports f32 and bf16");
  return PNR_OK;
}

// Sizes and enums; `step`: T, the token strides and lens are not part of the request.
int validate(const pnr_linattn* d, bool step) {
  if (!d) return record_error(PNR_E_INVALID, "descriptor is NULL");
  if (d->B < 1 || d->H < 1 || d->H_kv < 1 || d->D_k < 1 || d->D_v < 1 || (!step && d->T < 0))
    return record_error(PNR_E_INVALID,
                        "sizes must satisfy B, H, H_kv, D_k, D_v >= 1 and T >= 0 (got B=%d T=%d H=%d H_kv=%d D_k=%d D_v=%d)",
                        d->B, d->T, d->H, d->H_kv, d->D_k, d->D_v);
  if (d->H % d->H_kv) return record_error(PNR_E_INVALID, "H_kv=%d must divide H=%d", d->H_kv, d->H);
  if (int rc = check_dtype(d->dtype)) return rc;
  if (d->decay != PNR_DECAY_HEAD && d->decay != PNR_DECAY_TOKEN)
    return record_error(PNR_E_INVALID, "unknown decay kind %d", d->decay);
  if (!isfinite((float)d->scale)) return record_error(PNR_E_INVALID, "scale must be finite, in fp32");
  for (int i = 0; i < 3; ++i)
    if ((!step || i != 1) && (d->q_stride[i] < 0 || d->k_stride[i] < 0 || d->v_stride[i] < 0))
      return record_error(PNR_E_INVALID, "strides must be >= 0");
  if (d->D_k > kMaxHeadDim || d->D_v > kMaxHeadDim)
    return record_error(PNR_E_UNSUPPORTED, "head sizes up to %d are supported (got D_k=%d D_v=%d)", kMaxHeadDim,
                        d->D_k, d->D_v);
  // a launch holds 2^32 threads, 512 a row and state head; 64 tokens of outputs span less than 2^31 bytes
  const double rows = (double)d->B * (step ? 1 : d->T);
  if (d->H > (1 << 15) || (double)d->B * d->H > 8.0e6 || rows * d->H * kMaxHeadDim > 4.0e18 || (!step && d->T > (1 << 30)))
    return record_error(PNR_E_INVALID, "problem too large for this library's index range");
  return PNR_OK;
}

LinAttn problem(const pnr_linattn* d, const void* q, const void* k, const void* v, const float* g) {
  LinAttn a{};
  a.B = d->B, a.T = d->T, a.H = d->H, a.Hkv = d->H_kv, a.Dk = d->D_k, a.Dv = d->D_v;
  a.bf16 = d->dtype == PNR_BF16;
  a.decay_token = d->decay == PNR_DECAY_TOKEN;
  a.scale = (float)d->scale;
  a.q = {q, d->q_stride[0], d->q_stride[1], d->q_stride[2]};
  a.k = {k, d->k_stride[0], d->k_stride[1], d->k_stride[2]};
  a.v = {v, d->v_stride[0], d->v_stride[1], d->v_stride[2]};
  a.g = g;
  a.lens = d->lens;
  return a;
}

// Pointers of the attention calls: natural alignment, inputs present.
int check_attn_inputs(const pnr_linattn* d, const void* q, const void* k, const void* v, const float* g) {
  const size_t es = d->dtype == PNR_BF16 ? 2 : 4;
  if (!q || !k || !v || !g) return record_error(PNR_E_INVALID, "q, k, v and log_decay must be non-NULL");
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(g, 4) || !aligned(d->lens, 4))
    return record_error(PNR_E_INVALID, "a pointer is not aligned to its element size");
  return PNR_OK;
}

int validate(const pnr_norm* d) {
  if (!d) return record_error(PNR_E_INVALID, "descriptor is NULL");
  if (d->N < 1 || d->C < 1 || d->L < 0 || d->groups < 1)
    return record_error(PNR_E_INVALID, "sizes must satisfy N, C, groups >= 1 and L >= 0 (got N=%d L=%d C=%d groups=%d)",
                        d->N, d->L, d->C, d->groups);
  if (d->C % d->groups) return record_error(PNR_E_INVALID, "groups=%d must divide C=%d", d->groups, d->C);
  if (int rc = check_dtype(d->dtype)) return rc;
  if (d->act < PNR_ACT_NONE || d->act > PNR_ACT_GELU) return record_error(PNR_E_INVALID, "unknown activation %d", d->act);
  if (!((float)d->eps > 0) || !isfinite((float)d->eps)) return record_error(PNR_E_INVALID, "eps must be finite and > 0, in fp32");
  // kernels and plans count a map's rows, two slabs of them ahead, and eight groups' channels in 32 bits; a launch
  // holds 2^32 threads, 64 a channel in the sums of the parameters' gradients
  if (d->L > (1 << 30) || d->C > (1 << 26)) return record_error(PNR_E_INVALID, "problem too large for this library's index range");
  // maps and wide groups take a block each at least
  const bool blocks = d->L != 1 || d->C / d->groups > 512;
  if ((double)d->N * d->L * d->C > 4.0e18 || (double)d->N * d->groups > (blocks ? 1.6e7 : 2.0e9))
    return record_error(PNR_E_INVALID, "problem too large for this library's index range");
  return PNR_OK;
}

Norm problem(const pnr_norm* d, const void* x, const float* weight, const float* bias, const void* gate) {
  Norm a{};
  a.N = d->N, a.L = d->L, a.C = d->C, a.groups = d->groups;
  a.bf16 = d->dtype == PNR_BF16;
  a.act = d->act;
  a.eps = (float)d->eps;
  a.lens = d->lens;
  a.x = x, a.weight = weight, a.bias = bias, a.gate = gate;
  return a;
}

int check_norm_inputs(const pnr_norm* d, const void* x, const float* weight, const float* bias, const void* gate) {
  const size_t es = d->dtype == PNR_BF16 ? 2 : 4;
  if (d->L > 0 && !x) return record_error(PNR_E_INVALID, "x must be non-NULL");
  if (!weight != !bias) return record_error(PNR_E_INVALID, "weight and bias are given together or not at all");
  if (!aligned(x, es) || !aligned(gate, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(d->lens, 4))
    return record_error(PNR_E_INVALID, "a pointer is not aligned to its element size");
  return PNR_OK;
}

}  // namespace

extern "C" {

size_t pnr_linattn_workspace_bytes(const pnr_linattn* desc) {
  if (validate(desc, false)) return 0;
  return linattn_workspace(problem(desc, nullptr, nullptr, nullptr, nullptr));
}

int pnr_linattn_forward(const pnr_linattn* desc, const void* q, const void* k, const void* v, const float* log_decay,
                        const float* state_in, void* o, float* state_out) {
  if (int rc = validate(desc, false)) return rc;
  if (desc->T > 0) {
    if (int rc = check_attn_inputs(desc, q, k, v, log_decay)) return rc;
    if (!o || !aligned(o, desc->dtype == PNR_BF16 ? 2 : 4)) return record_error(PNR_E_INVALID, "o is NULL or misaligned");
  }
  if (!aligned(state_in, 4) || !aligned(state_out, 4)) return record_error(PNR_E_INVALID, "a state pointer is misaligned");
  const LinAttn a = problem(desc, q, k, v, log_decay);
  if (int rc = check_workspace(desc->workspace, desc->workspace_bytes, linattn_workspace(a))) return rc;
  return hip_status(launch_linattn_forward(a, state_in, o, state_out, (char*)desc->workspace, (hipStream_t)desc->stream),
                    "linear attention");
}

int pnr_linattn_step(const pnr_linattn* desc, const void* q, const void* k, const void* v, const float* log_decay,
                     const float* state_in, const int32_t* slots, int n_slots, void* o, float* state_out) {
  if (int rc = validate(desc, true)) return rc;
  if (int rc = check_attn_inputs(desc, q, k, v, log_decay)) return rc;
  if (!o || !aligned(o, desc->dtype == PNR_BF16 ? 2 : 4)) return record_error(PNR_E_INVALID, "o is NULL or misaligned");
  if (!state_in || !state_out || !aligned(state_in, 4) || !aligned(state_out, 4))
    return record_error(PNR_E_INVALID, "state_in and state_out must be non-NULL and aligned");
  if (!aligned(slots, 4)) return record_error(PNR_E_INVALID, "slots is misaligned");
  if (n_slots < 1 || (!slots && n_slots < desc->B))
    return record_error(PNR_E_INVALID, "n_slots=%d: need >= 1, and >= B=%d without slots", n_slots, desc->B);
  return hip_status(launch_linattn_step(problem(desc, q, k, v, log_decay), state_in, slots, n_slots, o, state_out,
                                        (hipStream_t)desc->stream),
                    "linear attention step");
}

size_t pnr_linattn_workspace_bytes_backward(const pnr_linattn* desc) {
  if (validate(desc, false)) return 0;
  return linattn_workspace_backward(problem(desc, nullptr, nullptr, nullptr, nullptr));
}

int pnr_linattn_backward(const pnr_linattn* desc, const void* q, const void* k, const void* v, const float* log_decay,
                         const float* state_in, const void* grad_o, const float* grad_state_out, void* grad_q,
                         void* grad_k, void* grad_v, float* grad_log_decay, float* grad_state_in) {
  if (int rc = validate(desc, false)) return rc;
  const size_t es = desc->dtype == PNR_BF16 ? 2 : 4;
  if (desc->T > 0) {
    if (int rc = check_attn_inputs(desc, q, k, v, log_decay)) return rc;
    if (!grad_o) return record_error(PNR_E_INVALID, "grad_o must be non-NULL");
  }
  if (!aligned(grad_o, es) || !aligned(grad_q, es) || !aligned(grad_k, es) || !aligned(grad_v, es) ||
      !aligned(state_in, 4) || !aligned(grad_state_out, 4) || !aligned(grad_log_decay, 4) || !aligned(grad_state_in, 4))
    return record_error(PNR_E_INVALID, "a pointer is not aligned to its element size");
  const LinAttn a = problem(desc, q, k, v, log_decay);
  if (int rc = check_workspace(desc->workspace, desc->workspace_bytes, linattn_workspace_backward(a))) return rc;
  LinAttnGrads d{};
  d.go = {grad_o, (int64_t)a.T * a.H * a.Dv, (int64_t)a.H * a.Dv, a.Dv};
  d.gstate_out = grad_state_out;
  d.gq = grad_q, d.gk = grad_k, d.gv = grad_v;
  d.gg = grad_log_decay, d.gstate_in = grad_state_in;
  return hip_status(launch_linattn_backward(a, state_in, d, (char*)desc->workspace, (hipStream_t)desc->stream),
                    "linear attention backward");
}

size_t pnr_groupnorm_workspace_bytes(const pnr_norm* desc) {
  if (validate(desc)) return 0;
  return groupnorm_workspace(problem(desc, nullptr, nullptr, nullptr, nullptr));
}

int pnr_groupnorm(const pnr_norm* desc, const void* x, const float* weight, const float* bias, const void* gate,
                  void* y, float* mean, float* rstd) {
  if (int rc = validate(desc)) return rc;
  if (int rc = check_norm_inputs(desc, x, weight, bias, gate)) return rc;
  if ((desc->L > 0 && !y) || !aligned(y, desc->dtype == PNR_BF16 ? 2 : 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return record_error(PNR_E_INVALID, "an output is NULL or misaligned");
  const Norm a = problem(desc, x, weight, bias, gate);
  if (int rc = check_workspace(desc->workspace, desc->workspace_bytes, groupnorm_workspace(a))) return rc;
  return hip_status(launch_groupnorm(a, y, mean, rstd, (char*)desc->workspace, (hipStream_t)desc->stream), "group norm");
}

size_t pnr_groupnorm_workspace_bytes_backward(const pnr_norm* desc) {
  if (validate(desc)) return 0;
  return groupnorm_workspace_backward(problem(desc, nullptr, nullptr, nullptr, nullptr));
}

int pnr_groupnorm_backward(const pnr_norm* desc, const void* x, const float* weight, const float* bias,
                           const void* gate, const void* grad_y, const float* mean, const float* rstd, void* grad_x,
                           float* grad_weight, float* grad_bias, void* grad_gate) {
  if (int rc = validate(desc)) return rc;
  if (int rc = check_norm_inputs(desc, x, weight, bias, gate)) return rc;
  const size_t es = desc->dtype == PNR_BF16 ? 2 : 4;
  if ((desc->L > 0 && !grad_y) || !mean || !rstd)
    return record_error(PNR_E_INVALID, "grad_y, mean and rstd must be non-NULL");
  if (grad_gate && !gate) return record_error(PNR_E_INVALID, "grad_gate without a gate");
  if ((grad_weight || grad_bias) && !weight) return record_error(PNR_E_INVALID, "grad_weight or grad_bias without a weight");
  if (!aligned(grad_y, es) || !aligned(grad_x, es) || !aligned(grad_gate, es) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(grad_weight, 4) || !aligned(grad_bias, 4))
    return record_error(PNR_E_INVALID, "a pointer is not aligned to its element size");
  const Norm a = problem(desc, x, weight, bias, gate);
  if (int rc = check_workspace(desc->workspace, desc->workspace_bytes, groupnorm_workspace_backward(a))) return rc;
  return hip_status(launch_groupnorm_backward(a, grad_y, mean, rstd, grad_x, grad_weight, grad_bias, grad_gate,
                                              (char*)desc->workspace, (hipStream_t)desc->stream),
                    "group norm backward");
}

}  // extern "C"
