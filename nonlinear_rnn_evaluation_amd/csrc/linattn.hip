// Linear attention with per-head decay over whole sequences, and its gradients.
//
// Forward, for each batch row and state head: S_t = exp(g_t) S_{t-1} + k_t v_t^T,
// o_t = scale S_t^T q_t.  With D_t = dL/dS_t (D_T = grad_state_out + its token's term),
//   D_t = scale q_t do_t^T + exp(g_{t+1}) D_{t+1}
//   dq_t = scale S_t do_t,  dk_t = D_t v_t,  dv_t = D_t^T k_t,  dS_0 = exp(g_1) D_1
//   dg_t = <D_t, exp(g_t) S_{t-1}>, and  dg_t = q_t.dq_t - k_t.dk_t + dg_{t+1}
//   with dg_{T+1} = <grad_state_out, S_T>.
// All of o, dq, dk and dv are one recurrence in four roles:
//         queries   keys   values   direction
//   o     q         k      v        forward
//   dq    do        v      k        forward    (the state transposed)
//   dk    v         do     q        backward   (the state's gradient transposed)
//   dv    k         q      do       backward
#include "seq_ops.h"

namespace pnr {
namespace {

struct Role {
  LinAttn a;
  Rows q, k, v;              // queries, keys, values of this role (heads counted per state head below)
  int nq, nkv;               // heads of queries, and of keys and values, per state head
  int dk, dv;                // sizes of queries and keys, and of values
  bool transposed;           // the state buffers hold [dv, dk]
  bool reverse;
  float out_scale, kv_scale; // on the output, on k v^T
  const float* s_in;
  float* s_out;
  void* o;                   // [B, T, Hkv * nq, dv] contiguous
  Rows x;                    // the rows that dot products of the outputs are taken with, or p = nullptr
  double* dots;              // [B, T, Hkv]: sum over the nq outputs of out . x
  const float* s_dot;        // with dots: end_dot[b, h] = <last state, s_dot>
  double* end_dot;
};

template <bool kBf16>
__global__ void __launch_bounds__(256) recurrence_kernel(Role p) {
  using E = Elem<kBf16>;
  using T = typename E::type;
  const LinAttn& a = p.a;
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
  const int j = tid & 127, half = tid >> 7;
  const int n = row_len(a.lens, b, a.T);
  __shared__ float ks[128], qs[128];
  __shared__ double red[256];
  double s[64];
  const size_t sbase = ((size_t)b * a.Hkv + h) * p.dk * p.dv;
  auto at = [&](int r) { const int i = half * 64 + r; return sbase + (p.transposed ? (size_t)j * p.dk + i : (size_t)i * p.dv + j); };
#pragma unroll
  for (int r = 0; r < 64; ++r)
    s[r] = (p.s_in && half * 64 + r < p.dk && j < p.dv) ? p.s_in[at(r)] : 0.0f;
  for (int step = 0; step < a.T; ++step) {
    const int t = p.reverse ? a.T - 1 - step : step;
    T* out = (T*)p.o + (((size_t)b * a.T + t) * a.Hkv + h) * p.nq * p.dv;
    if (t >= n) {
      if (half == 0 && j < p.dv)
        for (int g = 0; p.o && g < p.nq; ++g) E::store(out + (size_t)g * p.dv + j, 0.0f);
      if (tid == 0 && p.dots) p.dots[((size_t)b * a.T + t) * a.Hkv + h] = 0.0;
      continue;
    }
    const double dec = exp((double)clamp_log_decay(a.g[(a.decay_token ? ((size_t)b * a.T + t) * a.Hkv : 0) + h]));
    if (!p.reverse)
#pragma unroll
      for (int r = 0; r < 64; ++r) s[r] *= dec;
    for (int g = 0; g < p.nkv; ++g) {
      const int64_t hh = (int64_t)h * p.nkv + g;
      const T* kp = (const T*)p.k.p + b * p.k.sb + t * p.k.st + hh * p.k.sh;
      const T* vp = (const T*)p.v.p + b * p.v.sb + t * p.v.st + hh * p.v.sh;
      __syncthreads();
      if (tid < 128) ks[tid] = tid < p.dk ? E::load(kp + tid) * p.kv_scale : 0.0f;
      __syncthreads();
      const float v = j < p.dv ? E::load(vp + j) : 0.0f;
#pragma unroll
      for (int r = 0; r < 64; ++r) s[r] = fma((double)ks[half * 64 + r], (double)v, s[r]);
    }
    double dot = 0.0;
    for (int g = 0; g < p.nq; ++g) {
      const int64_t hh = (int64_t)h * p.nq + g;
      const T* qp = (const T*)p.q.p + b * p.q.sb + t * p.q.st + hh * p.q.sh;
      __syncthreads();
      if (tid < 128) qs[tid] = tid < p.dk ? E::load(qp + tid) : 0.0f;
      __syncthreads();
      double acc = 0.0;
#pragma unroll
      for (int r = 0; r < 64; ++r) acc = fma((double)qs[half * 64 + r], s[r], acc);
      red[tid] = acc;
      __syncthreads();
      if (half == 0 && j < p.dv) {
        const double o = p.out_scale * (red[j] + red[128 + j]);
        if (p.o) E::store(out + (size_t)g * p.dv + j, (float)o);
        if (p.dots) dot += o * E::load((const T*)p.x.p + b * p.x.sb + t * p.x.st + hh * p.x.sh + j);
      }
    }
    if (p.dots) {
      __syncthreads();
      red[tid] = half == 0 ? dot : 0.0;
      __syncthreads();
      if (tid == 0) {
        double sum = 0.0;
        for (int i = 0; i < 128; ++i) sum += red[i];
        p.dots[((size_t)b * a.T + t) * a.Hkv + h] = sum;
      }
    }
    if (p.reverse)
#pragma unroll
      for (int r = 0; r < 64; ++r) s[r] *= dec;
  }
  double ed = 0.0;
#pragma unroll
  for (int r = 0; r < 64; ++r)
    if (half * 64 + r < p.dk && j < p.dv) {
      if (p.s_out) p.s_out[at(r)] = (float)s[r];
      if (p.s_dot) ed += s[r] * p.s_dot[at(r)];
    }
  if (p.end_dot) {
    __syncthreads();
    red[tid] = ed;
    __syncthreads();
    if (tid == 0) {
      double sum = 0.0;
      for (int i = 0; i < 256; ++i) sum += red[i];
      p.end_dot[(size_t)b * a.Hkv + h] = sum;
    }
  }
}

// dg_t = dg_{t+1} + q_t.dq_t - k_t.dk_t, a thread a row and state head
__global__ void decay_grad_kernel(LinAttn a, const double* qd, const double* kd, const double* end, float* gg, double* rows) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.B * a.Hkv) return;
  const int b = i / a.Hkv, h = i % a.Hkv;
  const int n = row_len(a.lens, b, a.T);
  double acc = end[i], sum = 0.0;
  for (int t = a.T - 1; t >= 0; --t) {
    const size_t at = ((size_t)b * a.T + t) * a.Hkv + h;
    if (t < n) acc += qd[at] - kd[at];
    const double v = t < n ? acc : 0.0;
    sum += v;
    if (a.decay_token) gg[at] = (float)v;
  }
  rows[i] = sum;
}

__global__ void sum_rows_kernel(const double* rows, int B, int Hkv, float* gg) {
  const int h = blockIdx.x * blockDim.x + threadIdx.x;
  if (h >= Hkv) return;
  double s = 0.0;
  for (int b = 0; b < B; ++b) s += rows[(size_t)b * Hkv + h];
  gg[h] = (float)s;
}

hipError_t run(const Role& p, hipStream_t st) {
  const dim3 grid(p.a.Hkv, p.a.B);
  if (p.a.bf16)
    recurrence_kernel<true><<<grid, 256, 0, st>>>(p);
  else
    recurrence_kernel<false><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

size_t linattn_workspace(const LinAttn&) { return 0; }

hipError_t launch_linattn_forward(const LinAttn& a, const float* state_in, void* o, float* state_out, char*,
                                  hipStream_t st) {
  Role p{};
  p.a = a;
  p.q = a.q, p.k = a.k, p.v = a.v;
  p.nq = a.H / a.Hkv, p.nkv = 1, p.dk = a.Dk, p.dv = a.Dv;
  p.out_scale = a.scale, p.kv_scale = 1.0f;
  p.s_in = state_in, p.s_out = state_out, p.o = o;
  return run(p, st);
}

size_t linattn_workspace_backward(const LinAttn& a) {
  return (2 * (size_t)a.B * a.T * a.Hkv + 2 * (size_t)a.B * a.Hkv) * 8;
}

hipError_t launch_linattn_backward(const LinAttn& a, const float* state_in, const LinAttnGrads& d, char* ws,
                                   hipStream_t st) {
  const int G = a.H / a.Hkv;
  double* qd = (double*)ws;
  double* kd = qd + (size_t)a.B * a.T * a.Hkv;
  double* end = kd + (size_t)a.B * a.T * a.Hkv;
  double* rows = end + (size_t)a.B * a.Hkv;
  Role p{};
  p.a = a;
  p.nq = G, p.nkv = 1, p.dk = a.Dv, p.dv = a.Dk, p.transposed = true;
  p.q = d.go, p.k = a.v, p.v = a.k;
  p.out_scale = a.scale, p.kv_scale = 1.0f;
  p.s_in = state_in, p.o = d.gq, p.x = a.q, p.dots = qd, p.s_dot = d.gstate_out, p.end_dot = end;
  hipError_t e = run(p, st);
  p.s_dot = nullptr, p.end_dot = nullptr;
  p.reverse = true, p.nq = 1, p.nkv = G, p.q = a.v, p.k = d.go, p.v = a.q;
  p.out_scale = 1.0f, p.kv_scale = a.scale;
  p.s_in = d.gstate_out, p.o = d.gk, p.x = a.k, p.dots = kd, p.s_out = d.gstate_in;
  if (e == hipSuccess) e = run(p, st);
  p.dots = nullptr, p.transposed = false, p.dk = a.Dk, p.dv = a.Dv, p.s_out = nullptr;
  p.q = a.k, p.k = a.q, p.v = d.go, p.o = d.gv;
  if (e == hipSuccess && d.gv) e = run(p, st);
  if (e == hipSuccess && d.gg) {
    decay_grad_kernel<<<(a.B * a.Hkv + 63) / 64, 64, 0, st>>>(a, qd, kd, end, d.gg, rows);
    if (!a.decay_token) sum_rows_kernel<<<(a.Hkv + 63) / 64, 64, 0, st>>>(rows, a.B, a.Hkv, d.gg);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace pnr
