// Group norm with an activation, channels last, and its gradients.
//   n = (x - mean) rstd,  z = n w + b,  y = act(z)  or  z act(gate)
//   dz = dy act'(z)  or  dy act(gate);   dgate = dy z act'(gate)
//   u = dz w,  dx = rstd (u - mean(u) - n mean(u n)),  dw = sum dz n,  db = sum dz
#include "seq_ops.h"

namespace pnr {
namespace {

__device__ __forceinline__ float sigmoid(float u) { return __builtin_amdgcn_rcpf(1.0f + __expf(-u)); }

// gelu(u) = u sigmoid(2 a), a = sqrt(2/pi) (u + 0.044715 u^3): 0.5 (1 + tanh a) = sigmoid(2 a)
__device__ __forceinline__ float gelu_arg(float u) { return 1.5957691216057308f * u * fmaf(0.044715f * u, u, 1.0f); }

__device__ __forceinline__ float act_value(int act, float u) {
  if (act == PNR_ACT_SILU) return u * sigmoid(u);
  if (act == PNR_ACT_GELU) return u * sigmoid(gelu_arg(u));
  return u;
}

// act(u) and act'(u)
__device__ __forceinline__ float act_grad(int act, float u, float& value) {
  if (act == PNR_ACT_NONE) {
    value = u;
    return 1.0f;
  }
  const float s = sigmoid(act == PNR_ACT_SILU ? u : gelu_arg(u));
  value = u * s;
  const float da = act == PNR_ACT_SILU ? 1.0f : 1.5957691216057308f * fmaf(0.134145f * u, u, 1.0f);
  return fmaf(value * da, 1.0f - s, s);
}

__device__ float block_sum(float v) {
  __shared__ float w[4];
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = v;
  __syncthreads();
  return w[0] + w[1] + w[2] + w[3];
}

template <bool kBf16>
__global__ void __launch_bounds__(256) norm_kernel(Norm a, void* y_, float* mean, float* rstd) {
  using E = Elem<kBf16>;
  using T = typename E::type;
  for (unsigned ng = blockIdx.x; ng < (unsigned)a.N * a.groups; ng += gridDim.x) {
  const int W = a.C / a.groups, g = ng % a.groups;
  const int n = ng / a.groups;
  const int len = row_len(a.lens, n, a.L);
  const size_t base = (size_t)n * a.L * a.C + (size_t)g * W;
  const T* x = (const T*)a.x + base;
  const T* gate = a.gate ? (const T*)a.gate + base : nullptr;
  T* y = (T*)y_ + base;
  const long cnt = (long)len * W;
  auto at = [&](long i) { return (size_t)(i / W) * a.C + i % W; };
  float s = 0.0f;
  for (long i = threadIdx.x; i < cnt; i += 256) s += E::load(x + at(i));
  const float m = cnt ? block_sum(s) / cnt : 0.0f;
  s = 0.0f;
  for (long i = threadIdx.x; i < cnt; i += 256) {
    const float d = E::load(x + at(i)) - m;
    s += d * d;
  }
  const float r = 1.0f / sqrtf((cnt ? block_sum(s) / cnt : 0.0f) + a.eps);
  if (threadIdx.x == 0) {
    if (mean) mean[ng] = m;
    if (rstd) rstd[ng] = r;
  }
  for (long i = threadIdx.x; i < (long)a.L * W; i += 256) {
    float v = 0.0f;
    if (i < cnt) {
      const int c = g * W + (int)(i % W);
      v = (E::load(x + at(i)) - m) * r;
      if (a.weight) v = fmaf(v, a.weight[c], a.bias[c]);
      v = gate ? v * act_value(a.act, E::load(gate + at(i))) : act_value(a.act, v);
    }
    E::store(y + at(i), v);
  }
  }
}

// dz and n of one element; with a gate also dgate
template <bool kBf16>
__device__ __forceinline__ void element_grad(const Norm& a, const void* gy, size_t at, int c, float m, float r,
                                             float& n, float& dz, float& dgate) {
  using E = Elem<kBf16>;
  using T = typename E::type;
  n = (E::load((const T*)a.x + at) - m) * r;
  const float z = a.weight ? fmaf(n, a.weight[c], a.bias[c]) : n;
  const float dy = E::load((const T*)gy + at);
  float val;
  if (a.gate) {
    const float d = act_grad(a.act, E::load((const T*)a.gate + at), val);
    dz = dy * val;
    dgate = dy * z * d;
  } else {
    dz = dy * act_grad(a.act, z, val);
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(256) norm_grad_kernel(Norm a, const void* gy, const float* mean, const float* rstd,
                                                        void* gx_, void* gg_) {
  using E = Elem<kBf16>;
  using T = typename E::type;
  for (unsigned ng = blockIdx.x; ng < (unsigned)a.N * a.groups; ng += gridDim.x) {
  const int W = a.C / a.groups, g = ng % a.groups;
  const int n = ng / a.groups;
  const int len = row_len(a.lens, n, a.L);
  const size_t base = (size_t)n * a.L * a.C + (size_t)g * W;
  const long cnt = (long)len * W;
  const float m = mean[ng], r = rstd[ng];
  float s1 = 0.0f, s2 = 0.0f;
  for (long i = threadIdx.x; i < cnt; i += 256) {
    float h, dz, dg;
    const int c = g * W + (int)(i % W);
    element_grad<kBf16>(a, gy, base + (size_t)(i / W) * a.C + i % W, c, m, r, h, dz, dg);
    const float u = a.weight ? dz * a.weight[c] : dz;
    s1 += u;
    s2 += u * h;
  }
  const float m1 = cnt ? block_sum(s1) / cnt : 0.0f, m2 = cnt ? block_sum(s2) / cnt : 0.0f;
  for (long i = threadIdx.x; i < (long)a.L * W; i += 256) {
    const size_t at = base + (size_t)(i / W) * a.C + i % W;
    float dx = 0.0f, dg = 0.0f;
    if (i < cnt) {
      float h, dz;
      const int c = g * W + (int)(i % W);
      element_grad<kBf16>(a, gy, at, c, m, r, h, dz, dg);
      const float u = a.weight ? dz * a.weight[c] : dz;
      dx = r * (u - m1 - h * m2);
    }
    if (gx_) E::store((T*)gx_ + at, dx);
    if (gg_) E::store((T*)gg_ + at, dg);
  }
  }
}

// dw and db: a block a channel, over all rows and positions
template <bool kBf16>
__global__ void __launch_bounds__(256) norm_param_kernel(Norm a, const void* gy, const float* mean, const float* rstd,
                                                         float* gw, float* gb) {
  const int c = blockIdx.x, g = c / (a.C / a.groups);
  float s1 = 0.0f, s2 = 0.0f;
  for (size_t i = threadIdx.x; i < (size_t)a.N * a.L; i += 256) {
    const int n = (int)(i / a.L);
    if ((int)(i % a.L) >= row_len(a.lens, n, a.L)) continue;
    float h, dz, dg;
    element_grad<kBf16>(a, gy, i * a.C + c, c, mean[(size_t)n * a.groups + g], rstd[(size_t)n * a.groups + g], h, dz, dg);
    s1 += dz * h;
    s2 += dz;
  }
  s1 = block_sum(s1), s2 = block_sum(s2);
  if (threadIdx.x == 0) {
    if (gw) gw[c] = s1;
    if (gb) gb[c] = s2;
  }
}

}  // namespace

size_t groupnorm_workspace(const Norm&) { return 0; }

hipError_t launch_groupnorm(const Norm& a, void* y, float* mean, float* rstd, char*, hipStream_t st) {
  const unsigned grid = (unsigned)a.N * a.groups < 65536u ? (unsigned)a.N * a.groups : 65536u;
  if (a.bf16)
    norm_kernel<true><<<grid, 256, 0, st>>>(a, y, mean, rstd);
  else
    norm_kernel<false><<<grid, 256, 0, st>>>(a, y, mean, rstd);
  return hipGetLastError();
}

size_t groupnorm_workspace_backward(const Norm&) { return 0; }

hipError_t launch_groupnorm_backward(const Norm& a, const void* gy, const float* mean, const float* rstd, void* gx,
                                     float* gw, float* gb, void* ggate, char*, hipStream_t st) {
  const unsigned grid = (unsigned)a.N * a.groups < 65536u ? (unsigned)a.N * a.groups : 65536u;
  if (a.bf16) {
    if (gx || ggate) norm_grad_kernel<true><<<grid, 256, 0, st>>>(a, gy, mean, rstd, gx, ggate);
    if (gw || gb) norm_param_kernel<true><<<a.C, 256, 0, st>>>(a, gy, mean, rstd, gw, gb);
  } else {
    if (gx || ggate) norm_grad_kernel<false><<<grid, 256, 0, st>>>(a, gy, mean, rstd, gx, ggate);
    if (gw || gb) norm_param_kernel<false><<<a.C, 256, 0, st>>>(a, gy, mean, rstd, gw, gb);
  }
  return hipGetLastError();
}

}  // namespace pnr
