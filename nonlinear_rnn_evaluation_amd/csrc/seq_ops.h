// Internal interface of the sequence-mixing operators: linear attention with per-head
// decay (linattn*.hip), group norm with an activation (groupnorm.hip), the selective scan
// (selscan*.hip), the causal convolution (conv.hip) and 8-bit copies of activations
// (checkpoint.hip); their C entry points are in seq_api.hip.
#pragma once

#include "common.h"

namespace pnr {

// Records the text of the calling thread's last error (api.hip) and returns `code`.
int record_error(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

constexpr int kMaxHeadDim = 128;

// A [B, T, heads, D] operand: element strides between batch rows, tokens and heads.
struct Rows {
  const void* p;
  int64_t sb, st, sh;
};

// Device-side problem of the chunked linear attention (pnr_linattn without host fields).
struct LinAttn {
  int B, T, H, Hkv, Dk, Dv;
  int bf16;            // element type: 1 bf16, 0 fp32
  int decay_token;     // log_decay [B, T, Hkv] (1) or [Hkv] (0)
  float scale;
  Rows q, k, v;
  const float* g;
  const int32_t* lens;
};

struct LinAttnGrads {
  Rows go;                   // grad_o, contiguous
  const float* gstate_out;   // or nullptr
  void *gq, *gk, *gv;        // or nullptr
  float *gg, *gstate_in;     // or nullptr
};

size_t linattn_workspace(const LinAttn& a);
hipError_t launch_linattn_forward(const LinAttn& a, const float* state_in, void* o, float* state_out, char* ws,
                                  hipStream_t st);
size_t linattn_workspace_backward(const LinAttn& a);
hipError_t launch_linattn_backward(const LinAttn& a, const float* state_in, const LinAttnGrads& d, char* ws,
                                   hipStream_t st);
hipError_t launch_linattn_step(const LinAttn& a, const float* state_in, const int32_t* slots, int n_slots, void* o,
                               float* state_out, hipStream_t st);

struct Norm {
  int N, L, C, groups;
  int bf16, act;
  float eps;
  const int32_t* lens;
  const void* x;
  const float *weight, *bias;
  const void* gate;
};

size_t groupnorm_workspace(const Norm& a);
hipError_t launch_groupnorm(const Norm& a, void* y, float* mean, float* rstd, char* ws, hipStream_t st);
size_t groupnorm_workspace_backward(const Norm& a);
hipError_t launch_groupnorm_backward(const Norm& a, const void* gy, const float* mean, const float* rstd, void* gx,
                                     float* gw, float* gb, void* ggate, char* ws, hipStream_t st);

constexpr int kMaxStates = 64;    // of a channel of the selective scan
constexpr int kMaxTaps = 8;       // of the convolution
constexpr int kPackBlock = 32;    // values on one exponent in an 8-bit copy

// A [B, T, E] operand: element strides between batch rows and tokens.
struct Tokens {
  const void* p;
  int64_t sb, st;
};

// Device-side problem of the selective scan (pnr_selscan without host fields).
struct SelScan {
  int B, T, E, N, G;
  int bf16, softplus;
  Tokens u, dt, z;           // z.p may be nullptr
  Rows Bt, Ct;               // [B, T, G, N]
  const float *A, *D, *bias; // D, bias may be nullptr
  const int32_t* lens;
};

struct SelScanGrads {
  const void* gy;
  const float* gstate_out;   // or nullptr
  void *gu, *gdt, *gB, *gC, *gz;             // or nullptr
  float *gA, *gD, *gbias, *gstate_in;        // or nullptr
};

size_t selscan_workspace(const SelScan& a);
hipError_t launch_selscan_forward(const SelScan& a, const float* state_in, void* y, float* state_out, char* ws,
                                  hipStream_t st);
hipError_t launch_selscan_step(const SelScan& a, const float* state_in, const int32_t* slots, int n_slots, void* y,
                               float* state_out, hipStream_t st);
size_t selscan_workspace_backward(const SelScan& a);
hipError_t launch_selscan_backward(const SelScan& a, const float* state_in, const SelScanGrads& d, char* ws,
                                   hipStream_t st);

struct Conv {
  int B, T, E, W;
  int bf16, silu;
  Tokens x;
  const uint8_t* exps;       // x holds int8 codes on these exponents, or nullptr
  const float *weight, *bias;
  const int32_t* lens;
};

hipError_t launch_conv_forward(const Conv& a, const void* state_in, void* y, void* state_out, hipStream_t st);
hipError_t launch_conv_step(const Conv& a, const void* state_in, const int32_t* slots, int n_slots, void* y,
                            void* state_out, hipStream_t st);
size_t conv_workspace_backward(const Conv& a);
hipError_t launch_conv_backward(const Conv& a, const void* state_in, const void* gy, const void* gstate_out, void* gx,
                                float* gw, float* gb, void* gstate_in, char* ws, hipStream_t st);

hipError_t launch_checkpoint_pack(const Tokens& x, int B, int T, int E, int bf16, int8_t* codes, uint8_t* exps,
                                  hipStream_t st);
hipError_t launch_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows, int E, int bf16, void* x,
                                    hipStream_t st);

// ---- device helpers --------------------------------------------------------------------
__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Round to nearest, ties to even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  const __bf16 h = (__bf16)f;
  return __builtin_bit_cast(uint16_t, h);
}

// Two at once, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

template <bool kBf16>
struct Elem;
template <>
struct Elem<true> {
  using type = uint16_t;
  static __device__ __forceinline__ float load(const uint16_t* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ void store(uint16_t* p, float v) { *p = f32_to_bf16(v); }
};
template <>
struct Elem<false> {
  using type = float;
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// log(1 + e^x) without overflow and, where e^x is far below 1, without loss: to log(w) of the rounded
// w = 1 + e comes e - (w - 1), what the rounding took (over w, which is 1 where that counts).
__device__ __forceinline__ float softplus(float x) {
  const float e = fast_exp(-fabsf(x)), w = 1.0f + e;
  return fmaxf(x, 0.0f) + fmaf(__builtin_amdgcn_logf(w), kLn2, e - (w - 1.0f));
}

// What a code of an 8-bit copy counts on exponent byte s: 2^(s - 127), s >= 1; NaN on 255 (not finite).
__device__ __forceinline__ float unpack_step(int s) { return __uint_as_float(s == 255 ? 0x7fc00000u : (uint32_t)s << 23); }

__device__ __forceinline__ int row_len(const int32_t* lens, int b, int T) {
  if (!lens) return T;
  const int n = lens[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

// exp(g) of a log decay: below -104 it is 0 in fp32, so a larger drop (-inf included) is
// cut there and sums of log decays stay finite.  A NaN stays one.
constexpr float kLogDecayMin = -104.0f;
__device__ __forceinline__ float clamp_log_decay(float g) { return g < kLogDecayMin ? kLogDecayMin : g; }

}  // namespace pnr
