// Linear attention, one token for each running request:
//   S' = exp(g) S + k v^T,  o_h = scale S'^T q_h   for the H / H_kv query heads of a state.
//
// The state is read and written once (8 bytes an element; q, k, v and o are a few per cent
// of that), so memory bounds a full batch and the launch a small one.  A block takes one
// state head and 4 CW of its columns: a thread holds CW / 2 consecutive rows of four columns
// in registers, all asked for before the first is used.  Query heads go eight at a time:
// their sums over rows meet by shuffles, then over the waves in LDS.
#include "seq_ops.h"

namespace pnr {
namespace {

constexpr int kHeads = 8;        // query heads at a time

struct StepArgs {
  LinAttn a;
  const float* s_in;
  float* s_out;
  const int32_t* slots;
  int n_slots;
  void* o;
};

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <bool kBf16, int CW, bool kVec>
__global__ void __launch_bounds__(256) step_kernel(StepArgs p) {
  using E = Elem<kBf16>;
  using T = typename E::type;
  constexpr int RG = 256 / CW;               // row groups
  constexpr int R = kMaxHeadDim / RG;        // rows of a thread
  const LinAttn& a = p.a;
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  const int G = a.H / a.Hkv;
  const int tid = threadIdx.x, cw = tid % CW, i0 = tid / CW * R, wave = tid >> 6, lane = tid & 63;
  const int c0 = blockIdx.y * CW * 4, j0 = c0 + cw * 4;
  const int slot = p.slots ? p.slots[b] : b;
  T* o = (T*)p.o + ((size_t)b * a.H + (size_t)h * G) * a.Dv;
  if (slot < 0 || slot >= p.n_slots) {       // an idle row (uniform in the block)
    for (int i = tid; i < G * CW * 4; i += 256) {
      const int j = c0 + i % (CW * 4);
      if (j < a.Dv) E::store(o + (size_t)(i / (CW * 4)) * a.Dv + j, 0.0f);
    }
    return;
  }
  const size_t at = ((size_t)slot * a.Hkv + h) * a.Dk * a.Dv + (size_t)i0 * a.Dv + j0;
  f32x4 s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float* src = p.s_in + at + r * a.Dv;
    s[r] = f32x4{0, 0, 0, 0};
    if constexpr (kVec) {
      if (i0 + r < a.Dk && j0 < a.Dv) s[r] = *(const f32x4*)src;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i0 + r < a.Dk && j0 + c < a.Dv) s[r][c] = src[c];
    }
  }
  __shared__ alignas(16) float ks[kMaxHeadDim], qs[kHeads][kMaxHeadDim];
  __shared__ f32x4 part[kHeads][4][CW];
  const T* qp = (const T*)a.q.p + b * a.q.sb + (int64_t)h * G * a.q.sh;
  auto stage = [&](int g0, int heads) {
    for (int i = tid; i < heads * kMaxHeadDim; i += 256) {
      const int g = i / kMaxHeadDim, d = i % kMaxHeadDim;
      qs[g][d] = d < a.Dk ? E::load(qp + (g0 + g) * a.q.sh + d) : 0.0f;
    }
  };
  if (tid < kMaxHeadDim) ks[tid] = tid < a.Dk ? E::load((const T*)a.k.p + b * a.k.sb + h * a.k.sh + tid) : 0.0f;
  stage(0, min(G, kHeads));
  const T* vp = (const T*)a.v.p + b * a.v.sb + h * a.v.sh;
  f32x4 v;
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = j0 + c < a.Dv ? E::load(vp + j0 + c) : 0.0f;
  const float dec = expf(clamp_log_decay(a.g[(a.decay_token ? (size_t)b * a.Hkv : 0) + h]));
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    // rows behind the keys' end stay zero: zero times an infinite value would not be
    s[r] = i0 + r < a.Dk ? s[r] * dec + v * ks[i0 + r] : f32x4{0, 0, 0, 0};
    float* dst = p.s_out + at + r * a.Dv;
    if constexpr (kVec) {
      if (i0 + r < a.Dk && j0 < a.Dv) *(f32x4*)dst = s[r];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i0 + r < a.Dk && j0 + c < a.Dv) dst[c] = s[r][c];
    }
  }
  for (int g0 = 0; g0 < G; g0 += kHeads) {
    const int heads = min(G - g0, kHeads);
    if (g0) {
      __syncthreads();
      stage(g0, heads);
      __syncthreads();
    }
    for (int g = 0; g < heads; ++g) {
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < R; ++r) acc += s[r] * qs[g][i0 + r];
#pragma unroll
      for (int d = CW; d < 64; d <<= 1)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] += __shfl_xor(acc[c], d);
      if (lane < CW) part[g][wave][cw] = acc;
    }
    __syncthreads();
    for (int i = tid; i < heads * CW * 4; i += 256) {
      const int g = i / (CW * 4), j = i % (CW * 4);
      const float* w = (const float*)part[g];
      const float sum = (w[j] + w[CW * 4 + j]) + (w[CW * 8 + j] + w[CW * 12 + j]);
      if (c0 + j < a.Dv) E::store(o + (size_t)(g0 + g) * a.Dv + c0 + j, a.scale * sum);
    }
  }
}

template <bool kBf16, bool kVec, int CW>
void launch_columns(const StepArgs& p, hipStream_t st) {
  const LinAttn& a = p.a;
  step_kernel<kBf16, CW, kVec><<<dim3((unsigned)a.B * a.Hkv, (a.Dv + CW * 4 - 1) / (CW * 4)), 256, 0, st>>>(p);
}

// 128 columns a block keep sixteen loads of a thread in flight; where that leaves CUs without a
// block, 32 columns a block.  bf16, 32 query heads on 8 states of 128 x 128, 192 requests, in 128 and in 32
// columns: 48.8 us (4.2 TB/s) and 55.0, or 35.1 and 40.3 where the last-level cache still holds the pool
// from the call before; one request, 16 states of 64 x 64: 5.6 us and 4.6.
template <bool kBf16, bool kVec>
void launch(const StepArgs& p, hipStream_t st) {
  if ((int64_t)p.a.B * p.a.Hkv < 256)
    launch_columns<kBf16, kVec, 8>(p, st);
  else
    launch_columns<kBf16, kVec, 32>(p, st);
}

}  // namespace

hipError_t launch_linattn_step(const LinAttn& a, const float* state_in, const int32_t* slots, int n_slots, void* o,
                               float* state_out, hipStream_t st) {
  const StepArgs p{a, state_in, state_out, slots, n_slots, o};
  const bool vec = a.Dv % 4 == 0 && ((uintptr_t)state_in | (uintptr_t)state_out) % 16 == 0;
  if (a.bf16)
    vec ? launch<true, true>(p, st) : launch<true, false>(p, st);
  else
    vec ? launch<false, true>(p, st) : launch<false, false>(p, st);
  return hipGetLastError();
}

}  // namespace pnr
