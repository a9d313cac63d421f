// Shared by the selective scan's kernels.  A channel's states lie in four lanes, so that what a token needs
// once a channel (its step width, softplus, gate) is computed by one of them and handed to the others by
// cross-lane operands.  Forwards (selscan_fwd.hip) the four are a quad, and each prepares one of
// four tokens; backwards (selscan_bwd.hip) a lane owns one of four channels.
#pragma once

#include "seq_ops.h"

namespace pnr {
namespace selscan {

// The value of another lane of the quad.
template <int kCtrl>
__device__ __forceinline__ float quad_perm(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kCtrl, 0xf, 0xf, true));
}

// A for exponents of 2, finite where A is: a step width of 0 leaves the state.
__device__ __forceinline__ float exponent(float A) {
  const float x = A * kLog2e;
  return x < -3e38f ? -3e38f : x > 3e38f ? 3e38f : x;
}

// A decay over a segment as a factor, and what it leaves of h with own added.  2^x alone may be beyond fp32 (states
// that grow): three factors reach from the least number beyond the largest, and a zero state stays zero.
__device__ __forceinline__ float factor(float x) { return __builtin_amdgcn_exp2f(x > 127.0f ? fminf(x, 381.0f) * (1.0f / 3.0f) : x); }
__device__ __forceinline__ float carried(float h, float x, float f, float own) { return fmaf(x > 127.0f ? h * f * f : h, f, own); }

// A buffer from p on, empty unless `there`: at kNowhere, or in an empty one, loads give zeros and writes
// are dropped.
constexpr int kNowhere = 0x7fffffff;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, bool there) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, there ? 0x7fffffff : 0, 0x00027000);
}
template <typename T>
__device__ __forceinline__ T load_buffer(__amdgpu_buffer_rsrc_t from, int at, int base) {
  if constexpr (sizeof(T) == 2)
    return __builtin_amdgcn_raw_buffer_load_b16(from, at, base, 0);
  else
    return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(from, at, base, 0));
}
template <bool kBf16>
__device__ __forceinline__ void store_buffer(float v, __amdgpu_buffer_rsrc_t to, int at, int base) {
  if constexpr (kBf16)
    __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v), to, at, base, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), to, at, base, 0);
}

// A token's step width, 0 for a token that is not there.  The softplus is taken in any case: a branch
// would part the tokens' instructions, which fill each other's gaps.
__device__ __forceinline__ float step_width(float raw, int soft, bool there) {
  float s = softplus(raw);
  asm volatile("" : "+v"(s));
  return there ? (soft ? s : raw) : 0.0f;
}

// silu(z), or 1 without a gate; no branch, for the same reason.
__device__ __forceinline__ float gate_of(float z, bool gated) {
  float s = z * sigm(z);
  asm volatile("" : "+v"(s));
  return gated ? s : 1.0f;
}

// R consecutive values of LDS.
template <int R>
__device__ __forceinline__ void read_states(const float* p, float (&v)[R]) {
  __builtin_memcpy(v, __builtin_assume_aligned(p, R >= 4 ? 16 : 4 * R), 4 * R);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// How time is cut: S segments of `len` tokens.
struct Segments {
  int S, len;
};

}  // namespace selscan
}  // namespace pnr
