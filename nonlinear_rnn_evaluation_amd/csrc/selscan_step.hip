// Selective scan, one token for each running request:
//   h' = exp(delta A) h + delta u B,   y = (C . h' + D u) silu(z)
//
// The state is read and written once (8 bytes an element; the rest is a few per cent of that), so
// memory bounds a full batch and the launch a small one: 256 requests of 4096 x 16 take 35 us, 42
// with a pool that no cache holds (3.2 TB/s); one of 2048 x 16 takes 3.9.  A channel's states lie in the registers
// of LPC neighbouring lanes, four consecutive ones each, and C . h' meets by shuffles.
#include "selscan_tile.h"

namespace pnr {
namespace {

using namespace selscan;

struct StepArgs {
  SelScan a;
  const float* s_in;
  float* s_out;
  const int32_t* slots;
  int n_slots;
  void* y;
  bool whole;                // B and C are aligned to four values
};

// kEach channels a lane, 256 / LPC apart, all of whose states are asked for before the first is used.
template <bool kBf16, int LPC, bool kVec, int kEach>
__global__ void __launch_bounds__(256) step_kernel(StepArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  const SelScan& a = p.a;
  constexpr int CH = 256 / LPC;              // channels of a block at a time
  const int tiles = (a.E + CH * kEach - 1) / (CH * kEach), b = blockIdx.x / tiles;
  const int e0 = blockIdx.x % tiles * (CH * kEach) + threadIdx.x / LPC, n0 = threadIdx.x % LPC * 4;
  const int slot = p.slots ? p.slots[b] : b;
  T* y = (T*)p.y + (size_t)b * a.E;
  if (slot < 0 || slot >= p.n_slots) {       // an idle row
#pragma unroll
    for (int c = 0; c < kEach; ++c)
      if (n0 == 0 && e0 + c * CH < a.E) El::store(y + e0 + c * CH, 0.0f);
    return;
  }
  f32x4 h[kEach], A[kEach];
  float u[kEach], raw[kEach], zt[kEach];
#pragma unroll
  for (int c = 0; c < kEach; ++c) {
    const int e = min(e0 + c * CH, a.E - 1);            // a channel's lanes go together
    const size_t at = ((size_t)slot * a.E + e) * a.N + n0;
    h[c] = A[c] = f32x4{0, 0, 0, 0};
    if constexpr (kVec) {
      if (n0 < a.N) h[c] = *(const f32x4*)(p.s_in + at), A[c] = *(const f32x4*)(a.A + (size_t)e * a.N + n0);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0 + i < a.N) h[c][i] = p.s_in[at + i], A[c][i] = a.A[(size_t)e * a.N + n0 + i];
    }
    u[c] = El::load((const T*)a.u.p + b * a.u.sb + e);
    raw[c] = El::load((const T*)a.dt.p + b * a.dt.sb + e);
    zt[c] = a.z.p ? El::load((const T*)a.z.p + b * a.z.sb + e) : 0.0f;
  }
  int group = -1;
  f32x4 Bv{0, 0, 0, 0}, Cv{0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < kEach; ++c) {
    const int e = e0 + c * CH;
    if (e >= a.E) break;
    const int g = a.G == 1 ? 0 : e / (a.E / a.G);
    if (g != group) {
      group = g;
      const T* Bt = (const T*)a.Bt.p + b * a.Bt.sb + g * a.Bt.sh + n0;
      const T* Ct = (const T*)a.Ct.p + b * a.Ct.sb + g * a.Ct.sh + n0;
      if (kVec && p.whole) {                 // four values at once
        if (n0 < a.N) {
          T rb[4], rc[4];
          __builtin_memcpy(rb, __builtin_assume_aligned(Bt, sizeof(rb)), sizeof(rb));
          __builtin_memcpy(rc, __builtin_assume_aligned(Ct, sizeof(rc)), sizeof(rc));
#pragma unroll
          for (int i = 0; i < 4; ++i) Bv[i] = El::load(rb + i), Cv[i] = El::load(rc + i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < a.N) Bv[i] = El::load(Bt + i), Cv[i] = El::load(Ct + i);
      }
    }
    const float in = raw[c] + (a.bias ? a.bias[e] : 0.0f), delta = a.softplus ? softplus(in) : in, du = delta * u[c];
    float acc = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < a.N) {
        h[c][i] = h[c][i] * __builtin_amdgcn_exp2f(delta * exponent(A[c][i])) + du * Bv[i];
        acc += h[c][i] * Cv[i];
      }
    const size_t at = ((size_t)slot * a.E + e) * a.N + n0;
    if constexpr (kVec) {
      if (n0 < a.N) *(f32x4*)(p.s_out + at) = h[c];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0 + i < a.N) p.s_out[at + i] = h[c][i];
    }
#pragma unroll
    for (int d = 1; d < LPC; d <<= 1) acc += __shfl_xor(acc, d);
    if (n0 == 0) {
      acc += a.D ? a.D[e] * u[c] : 0.0f;
      El::store(y + e, a.z.p ? acc * (zt[c] * sigm(zt[c])) : acc);
    }
  }
}

template <bool kBf16, bool kVec, int LPC>
void launch_lanes(const StepArgs& p, hipStream_t st) {
  const SelScan& a = p.a;
  constexpr int CH = 256 / LPC;
  // bf16, us with one and with four channels a lane, pools that the last-level cache does not hold: 256 requests of
  // 4096 x 16 48 and 42, 512 of 1024 x 64 88 and 74, 16 of 4096 x 16 5.0 and 6.4 (too few blocks), and in one lane
  // a channel 256 of 8192 x 4 24 and 45 (its own four values and softplus come four times in a row).
  auto blocks = [&](int each) { return (unsigned)((int64_t)a.B * ((a.E + CH * each - 1) / (CH * each))); };
  if (LPC > 2 && blocks(4) >= 1024)
    step_kernel<kBf16, LPC, kVec, 4><<<blocks(4), 256, 0, st>>>(p);
  else
    step_kernel<kBf16, LPC, kVec, 1><<<blocks(1), 256, 0, st>>>(p);
}

template <bool kBf16, bool kVec>
void launch(const StepArgs& p, hipStream_t st) {
  const int N = p.a.N;
  if (N <= 4)
    launch_lanes<kBf16, kVec, 1>(p, st);
  else if (N <= 8)
    launch_lanes<kBf16, kVec, 2>(p, st);
  else if (N <= 16)
    launch_lanes<kBf16, kVec, 4>(p, st);
  else if (N <= 32)
    launch_lanes<kBf16, kVec, 8>(p, st);
  else
    launch_lanes<kBf16, kVec, 16>(p, st);
}

}  // namespace

hipError_t launch_selscan_step(const SelScan& a, const float* state_in, const int32_t* slots, int n_slots, void* y,
                               float* state_out, hipStream_t st) {
  const int es = a.bf16 ? 2 : 4;
  const bool whole = ((uintptr_t)a.Bt.p | (uintptr_t)a.Ct.p) % (4 * es) == 0 && (a.Bt.sb | a.Bt.sh | a.Ct.sb | a.Ct.sh) % 4 == 0;
  const StepArgs p{a, state_in, state_out, slots, n_slots, y, whole};
  const bool vec = a.N % 4 == 0 && ((uintptr_t)state_in | (uintptr_t)state_out | (uintptr_t)a.A) % 16 == 0;
  if (a.bf16)
    vec ? launch<true, true>(p, st) : launch<true, false>(p, st);
  else
    vec ? launch<false, true>(p, st) : launch<false, false>(p, st);
  return hipGetLastError();
}

}  // namespace pnr
