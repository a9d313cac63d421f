// Linear attention, one token for each running request:
//   S' = exp(g) S + k v^T,  o_h = scale S'^T q_h   for the H / H_kv query heads of a state.
//
// The state is read and written once (8 bytes an element; q, k, v and o are a few per cent
// of that), so memory bounds a full batch and the launch a small one.  A block takes one
// state head and 4 * CW of its columns: a thread holds CW / 2 rows of four columns in
// registers, all loaded before the first is used, and the rows of a column meet in LDS.
#include "seq_ops.h"

namespace pnr {
namespace {

struct StepArgs {
  LinAttn a;
  const float* s_in;
  float* s_out;
  const int32_t* slots;
  int n_slots;
  void* o;
};

template <bool kBf16, int CW, bool kVec>
__global__ void __launch_bounds__(256) step_kernel(StepArgs p) {
  using E = Elem<kBf16>;
  using T = typename E::type;
  constexpr int RG = 256 / CW;               // row groups
  constexpr int R = kMaxHeadDim / RG;        // rows of a thread: row group + r * RG
  const LinAttn& a = p.a;
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  const int G = a.H / a.Hkv;
  const int cw = threadIdx.x % CW, rg = threadIdx.x / CW;
  const int j0 = (blockIdx.y * CW + cw) * 4;
  const int slot = p.slots ? p.slots[b] : b;
  T* o = (T*)p.o + ((size_t)b * a.H + (size_t)h * G) * a.Dv;
  if (slot < 0 || slot >= p.n_slots) {       // an idle row (uniform in the block)
    for (int i = threadIdx.x; i < G * CW * 4; i += 256) {
      const int j = blockIdx.y * CW * 4 + i % (CW * 4);
      if (j < a.Dv) E::store(o + (size_t)(i / (CW * 4)) * a.Dv + j, 0.0f);
    }
    return;
  }
  const size_t base = ((size_t)slot * a.Hkv + h) * a.Dk * a.Dv;
  float s[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = rg + r * RG;
    const float* src = p.s_in + base + (size_t)i * a.Dv + j0;
    if constexpr (kVec) {
      float4 w = make_float4(0, 0, 0, 0);
      if (i < a.Dk && j0 < a.Dv) w = *(const float4*)src;
      s[r][0] = w.x, s[r][1] = w.y, s[r][2] = w.z, s[r][3] = w.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) s[r][c] = (i < a.Dk && j0 + c < a.Dv) ? src[c] : 0.0f;
    }
  }
  const float dec = expf(clamp_log_decay(a.g[(a.decay_token ? (size_t)b * a.Hkv : 0) + h]));
  const T* kp = (const T*)a.k.p + b * a.k.sb + h * a.k.sh;
  const T* vp = (const T*)a.v.p + b * a.v.sb + h * a.v.sh;
  float v[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = j0 + c < a.Dv ? E::load(vp + j0 + c) : 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = rg + r * RG;
    const float ki = i < a.Dk ? E::load(kp + i) : 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) s[r][c] = fmaf(dec, s[r][c], ki * v[c]);
    float* dst = p.s_out + base + (size_t)i * a.Dv + j0;
    if constexpr (kVec) {
      if (i < a.Dk && j0 < a.Dv) *(float4*)dst = make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i < a.Dk && j0 + c < a.Dv) dst[c] = s[r][c];
    }
  }
  __shared__ float4 part[RG][CW];
  for (int g = 0; g < G; ++g) {
    const T* qp = (const T*)a.q.p + b * a.q.sb + (int64_t)(h * G + g) * a.q.sh;
    float acc[4] = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = rg + r * RG;
      const float qi = i < a.Dk ? E::load(qp + i) : 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = fmaf(qi, s[r][c], acc[c]);
    }
    part[rg][cw] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (threadIdx.x < CW * 4) {
      const int j = blockIdx.y * CW * 4 + threadIdx.x;
      float sum = 0.0f;
      for (int r = 0; r < RG; ++r) sum += ((const float*)part[r])[threadIdx.x];
      if (j < a.Dv) E::store(o + (size_t)g * a.Dv + j, a.scale * sum);
    }
    __syncthreads();
  }
}

template <bool kBf16, bool kVec>
void launch(const StepArgs& p, hipStream_t st) {
  const LinAttn& a = p.a;
  constexpr int CW = 32;
  step_kernel<kBf16, CW, kVec><<<dim3((unsigned)a.B * a.Hkv, (a.Dv + CW * 4 - 1) / (CW * 4)), 256, 0, st>>>(p);
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
