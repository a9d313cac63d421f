// Selective scan, one token for each running request:
//   h' = exp(delta A) h + delta u B,   y = (C . h' + D u) silu(z)
//
// The state is read and written once (8 bytes an element; the rest is a few per cent of that), so
// memory bounds a full batch and the launch a small one.  A channel's states lie in the registers
// of LPC neighbouring lanes, four consecutive ones each, and C . h' meets by shuffles.
#include "seq_ops.h"

namespace pnr {
namespace {

struct StepArgs {
  SelScan a;
  const float* s_in;
  float* s_out;
  const int32_t* slots;
  int n_slots;
  void* y;
};

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <bool kBf16, int LPC, bool kVec>
__global__ void __launch_bounds__(256) step_kernel(StepArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  const SelScan& a = p.a;
  constexpr int CH = 256 / LPC;              // channels of a block
  const int tiles = (a.E + CH - 1) / CH, b = blockIdx.x / tiles;
  const int e = blockIdx.x % tiles * CH + threadIdx.x / LPC, n0 = threadIdx.x % LPC * 4;
  if (e >= a.E) return;                      // a channel's lanes leave together
  const int slot = p.slots ? p.slots[b] : b;
  T* y = (T*)p.y + (size_t)b * a.E + e;
  if (slot < 0 || slot >= p.n_slots) {       // an idle row
    if (n0 == 0) El::store(y, 0.0f);
    return;
  }
  const size_t at = ((size_t)slot * a.E + e) * a.N + n0;
  f32x4 h{0, 0, 0, 0}, A{0, 0, 0, 0}, Bv{0, 0, 0, 0}, Cv{0, 0, 0, 0};
  if constexpr (kVec) {
    if (n0 < a.N) h = *(const f32x4*)(p.s_in + at), A = *(const f32x4*)(a.A + (size_t)e * a.N + n0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < a.N) h[i] = p.s_in[at + i], A[i] = a.A[(size_t)e * a.N + n0 + i];
  }
  const int g = e / (a.E / a.G);
  const T* Bt = (const T*)a.Bt.p + b * a.Bt.sb + g * a.Bt.sh + n0;
  const T* Ct = (const T*)a.Ct.p + b * a.Ct.sb + g * a.Ct.sh + n0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + i < a.N) Bv[i] = El::load(Bt + i), Cv[i] = El::load(Ct + i);
  const float u = El::load((const T*)a.u.p + b * a.u.sb + e);
  const float raw = El::load((const T*)a.dt.p + b * a.dt.sb + e) + (a.bias ? a.bias[e] : 0.0f);
  const float zt = a.z.p ? El::load((const T*)a.z.p + b * a.z.sb + e) : 0.0f;
  const float delta = a.softplus ? softplus(raw) : raw, du = delta * u;
  float acc = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + i < a.N) {
      h[i] = h[i] * __builtin_amdgcn_exp2f(delta * (A[i] * kLog2e)) + du * Bv[i];
      acc += h[i] * Cv[i];
    }
  if constexpr (kVec) {
    if (n0 < a.N) *(f32x4*)(p.s_out + at) = h;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < a.N) p.s_out[at + i] = h[i];
  }
#pragma unroll
  for (int d = 1; d < LPC; d <<= 1) acc += __shfl_xor(acc, d);
  if (n0 == 0) {
    acc += a.D ? a.D[e] * u : 0.0f;
    El::store(y, a.z.p ? acc * (zt * sigm(zt)) : acc);
  }
}

template <bool kBf16, bool kVec>
void launch(const StepArgs& p, hipStream_t st) {
  const SelScan& a = p.a;
  auto blocks = [&](int ch) { return dim3((unsigned)a.B * ((a.E + ch - 1) / ch)); };
  if (a.N <= 4)
    step_kernel<kBf16, 1, kVec><<<blocks(256), 256, 0, st>>>(p);
  else if (a.N <= 8)
    step_kernel<kBf16, 2, kVec><<<blocks(128), 256, 0, st>>>(p);
  else if (a.N <= 16)
    step_kernel<kBf16, 4, kVec><<<blocks(64), 256, 0, st>>>(p);
  else if (a.N <= 32)
    step_kernel<kBf16, 8, kVec><<<blocks(32), 256, 0, st>>>(p);
  else
    step_kernel<kBf16, 16, kVec><<<blocks(16), 256, 0, st>>>(p);
}

}  // namespace

hipError_t launch_selscan_step(const SelScan& a, const float* state_in, const int32_t* slots, int n_slots, void* y,
                               float* state_out, hipStream_t st) {
  const StepArgs p{a, state_in, state_out, slots, n_slots, y};
  const bool vec = a.N % 4 == 0 && ((uintptr_t)state_in | (uintptr_t)state_out | (uintptr_t)a.A) % 16 == 0;
  if (a.bf16)
    vec ? launch<true, true>(p, st) : launch<true, false>(p, st);
  else
    vec ? launch<false, true>(p, st) : launch<false, false>(p, st);
  return hipGetLastError();
}

}  // namespace pnr
