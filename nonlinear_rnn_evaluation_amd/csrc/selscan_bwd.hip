// Gradients of the selective scan.  With gy = grad_y silu(z) and g_t = gy_t C_t + a_{t+1} g_{t+1}
// the gradient of h_t (a_t = exp(delta_t A)):
//   dC_t = sum_e gy h_t          dB_t = sum_e g delta u        q = sum_n g B_t
//   du = D gy + delta q          ddelta = u q + sum_n g a h_{t-1} A
//   dA = sum_t g a h_{t-1} delta      dD = sum_t gy u          dh_0 = a_1 g_1
// One thread a channel: a walk forwards that keeps every state, and one back.
#include <algorithm>

#include "seq_ops.h"

namespace pnr {
namespace {

struct BwdArgs {
  SelScan a;
  SelScanGrads d;
  const float* s_in;
  float *hist, *part, *pA, *pD, *pb;      // states [B, T, N, E]; sums of a tile, and of a row
  int tiles, per_group;                   // tiles of 64 channels: in all, a group
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

template <bool kBf16, int NP>
__global__ void __launch_bounds__(64) walk_kernel(BwdArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  const SelScan& a = p.a;
  const int b = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles, g = tile / p.per_group;
  const int W = a.E / a.G, w = tile % p.per_group * 64 + threadIdx.x;
  const bool live = w < W;
  const int e = g * W + (live ? w : 0), n = row_len(a.lens, b, a.T);
  float A[NP], h[NP], G[NP], gA[NP];
  const size_t at = ((size_t)b * a.E + e) * a.N;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    A[i] = i < a.N ? a.A[(size_t)e * a.N + i] : 0.0f;
    h[i] = i < a.N && p.s_in ? p.s_in[at + i] : 0.0f;
    G[i] = i < a.N && p.d.gstate_out ? p.d.gstate_out[at + i] : 0.0f;
    gA[i] = 0.0f;
  }
  const T* u = (const T*)a.u.p + b * a.u.sb + e;
  const T* dt = (const T*)a.dt.p + b * a.dt.sb + e;
  const T* z = a.z.p ? (const T*)a.z.p + b * a.z.sb + e : nullptr;
  const T* Bt = (const T*)a.Bt.p + b * a.Bt.sb + g * a.Bt.sh;
  const T* Ct = (const T*)a.Ct.p + b * a.Ct.sb + g * a.Ct.sh;
  const float D = a.D ? a.D[e] : 0.0f, bias = a.bias ? a.bias[e] : 0.0f;
  float* hist = p.hist + (size_t)b * a.T * a.N * a.E + e;
  for (int t = 0; t < n; ++t) {
    const float ut = El::load(u + t * a.u.st), raw = El::load(dt + t * a.dt.st) + bias;
    const float delta = a.softplus ? softplus(raw) : raw, du = delta * ut;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float Bv = i < a.N ? El::load(Bt + t * a.Bt.st + i) : 0.0f;
      if (i < a.N && live) hist[((size_t)t * a.N + i) * a.E] = h[i];
      h[i] = h[i] * __builtin_amdgcn_exp2f(delta * (A[i] * kLog2e)) + du * Bv;
    }
  }
  float gD = 0.0f, gb = 0.0f;
  for (int t = n - 1; t >= 0; --t) {
    const size_t o = ((size_t)b * a.T + t) * a.E + e;
    const float ut = El::load(u + t * a.u.st), raw = El::load(dt + t * a.dt.st) + bias;
    const float delta = a.softplus ? softplus(raw) : raw, du = delta * ut;
    float gy = live ? El::load((const T*)p.d.gy + o) : 0.0f;
    const float gy0 = gy, zt = z ? El::load(z + t * a.z.st) : 0.0f, sg = sigm(zt);
    if (z) gy *= zt * sg;
    float y = D * ut, q = 0.0f, gd = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (i >= a.N) break;
      const float Bv = El::load(Bt + t * a.Bt.st + i), Cv = El::load(Ct + t * a.Ct.st + i);
      const float hp = live ? hist[((size_t)t * a.N + i) * a.E] : 0.0f;
      const float dec = __builtin_amdgcn_exp2f(delta * (A[i] * kLog2e)), hn = hp * dec + du * Bv;
      y += Cv * hn;
      G[i] += gy * Cv;
      q += G[i] * Bv;
      const float dB = wave_sum(live ? G[i] * du : 0.0f), dC = wave_sum(live ? gy * hn : 0.0f);
      if (threadIdx.x == 0) {
        float* part = p.part + (((size_t)b * a.T + t) * p.tiles + tile) * 2 * a.N;
        part[i] = dB, part[a.N + i] = dC;
      }
      G[i] *= dec;
      gd += G[i] * hp * A[i];
      gA[i] += G[i] * hp * delta;
    }
    gd += ut * q;
    if (a.softplus) gd *= sigm(raw);
    gD += gy * ut, gb += gd;
    if (live) {
      if (p.d.gu) El::store((T*)p.d.gu + o, D * gy + delta * q);
      if (p.d.gdt) El::store((T*)p.d.gdt + o, gd);
      if (p.d.gz) El::store((T*)p.d.gz + o, gy0 * y * sg * (1.0f + zt * (1.0f - sg)));
    }
  }
  if (!live) return;
  for (int t = n; t < a.T; ++t) {
    const size_t o = ((size_t)b * a.T + t) * a.E + e;
    if (p.d.gu) El::store((T*)p.d.gu + o, 0.0f);
    if (p.d.gdt) El::store((T*)p.d.gdt + o, 0.0f);
    if (p.d.gz) El::store((T*)p.d.gz + o, 0.0f);
  }
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (i < a.N) {
      p.pA[at + i] = gA[i];
      if (p.d.gstate_in) p.d.gstate_in[at + i] = G[i];
    }
  p.pD[(size_t)b * a.E + e] = gD, p.pb[(size_t)b * a.E + e] = gb;
}

// The tiles' sums of dB and dC, in order.
template <bool kBf16>
__global__ void __launch_bounds__(64) token_kernel(BwdArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  const SelScan& a = p.a;
  for (int64_t row = blockIdx.x; row < (int64_t)a.B * a.T; row += gridDim.x) {
    const bool live = row % a.T < row_len(a.lens, (int)(row / a.T), a.T);
    for (int i = threadIdx.x; i < a.G * 2 * a.N; i += 64) {
      const int g = i / (2 * a.N), k = i % (2 * a.N);
      float s = 0.0f;
      if (live)
        for (int j = 0; j < p.per_group; ++j) s += p.part[((size_t)row * p.tiles + g * p.per_group + j) * 2 * a.N + k];
      T* out = (T*)(k < a.N ? p.d.gB : p.d.gC);
      if (out) El::store(out + ((size_t)row * a.G + g) * a.N + k % a.N, s);
    }
  }
}

__global__ void __launch_bounds__(256) row_kernel(const float* part, int rows, size_t n, float* out) {
  const size_t i = blockIdx.x * (size_t)256 + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
  for (int r = 0; r < rows; ++r) s += part[r * n + i];
  out[i] = s;
}

struct Layout {
  size_t hist, part, pA, pD, pb, bytes;
  int tiles, per_group;
};

Layout layout(const SelScan& a) {
  Layout l{};
  auto up = [](size_t v) { return (v * 4 + 255) / 256 * 256; };
  l.per_group = (a.E / a.G + 63) / 64;
  l.tiles = l.per_group * a.G;
  const size_t be = (size_t)a.B * a.E, bt = (size_t)a.B * a.T;
  l.part = l.hist + up(bt * a.E * a.N);
  l.pA = l.part + up(bt * l.tiles * 2 * a.N);
  l.pD = l.pA + up(be * a.N);
  l.pb = l.pD + up(be);
  l.bytes = l.pb + up(be);
  return l;
}

template <bool kBf16>
void launch(const BwdArgs& p, hipStream_t st) {
  const SelScan& a = p.a;
  const int blocks = a.B * p.tiles;
  if (a.N <= 4)
    walk_kernel<kBf16, 4><<<blocks, 64, 0, st>>>(p);
  else if (a.N <= 16)
    walk_kernel<kBf16, 16><<<blocks, 64, 0, st>>>(p);
  else
    walk_kernel<kBf16, 64><<<blocks, 64, 0, st>>>(p);
  if ((p.d.gB || p.d.gC) && a.T > 0)
    token_kernel<kBf16><<<(unsigned)std::min<int64_t>((int64_t)a.B * a.T, 1 << 20), 64, 0, st>>>(p);
  auto rows = [&](const float* part, size_t n, float* out) {
    if (out) row_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(part, a.B, n, out);
  };
  rows(p.pA, (size_t)a.E * a.N, p.d.gA);
  rows(p.pD, a.E, p.d.gD);
  rows(p.pb, a.E, p.d.gbias);
}

}  // namespace

size_t selscan_workspace_backward(const SelScan& a) { return layout(a).bytes; }

hipError_t launch_selscan_backward(const SelScan& a, const float* state_in, const SelScanGrads& d, char* ws,
                                   hipStream_t st) {
  const Layout l = layout(a);
  const BwdArgs p{a, d, state_in, (float*)(ws + l.hist), (float*)(ws + l.part), (float*)(ws + l.pA), (float*)(ws + l.pD),
                  (float*)(ws + l.pb), l.tiles, l.per_group};
  a.bf16 ? launch<true>(p, st) : launch<false>(p, st);
  return hipGetLastError();
}

}  // namespace pnr
