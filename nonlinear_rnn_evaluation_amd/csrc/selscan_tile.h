// Shared by the selective scan's forward and backward kernels: how a wave holds channels and states,
// and how time is cut into segments.
//
// A wave owns 64 channels, one a lane, and all their states (N <= 4 R): lane l holds, for four
// channels, the R states that start at R ((l / 4) % 4).  Its slot r belongs to the channel of the
// lane 4 r places behind it in its row of 16, so that
//   - what a channel needs once a token (its step width, softplus, gate) is computed by one lane, and
//     a rotation of the row brings it to the three others that hold the rest of its states;
//   - a sum over a channel's states is one rotation and one addition a slot, and ends in the lane
//     that owns the channel.
// With one lane a channel and 16 states, a token's B and C would have to come to every lane
// (eight 16-byte reads of LDS instead of two), and a sum over channels would start from 64 lanes.
#pragma once

#include "seq_ops.h"

namespace pnr {
namespace selscan {

constexpr int kChannels = 64;     // of a wave
constexpr int kNarrow = 16;       // of a wave that holds one channel's states in a quad of lanes

// The value of the lane 4 r places away in the row of 16 (away<4 - r> undoes away<r>).
template <int r>
__device__ __forceinline__ float away(float x) {
  if constexpr (r % 4 == 0) return x;
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + 4 * (r % 4), 0xf, 0xf, true));
}
template <int r>
__device__ __forceinline__ int away(int x) {
  if constexpr (r % 4 == 0) return x;
  return __builtin_amdgcn_update_dpp(0, x, 0x120 + 4 * (r % 4), 0xf, 0xf, true);
}
__device__ __forceinline__ void to_slots(float x, float (&s)[4]) {
  s[0] = x, s[1] = away<1>(x), s[2] = away<2>(x), s[3] = away<3>(x);
}
// The sum of a channel's four partial sums, in its lane.
__device__ __forceinline__ float from_slots(const float (&s)[4]) {
  return (s[0] + away<3>(s[1])) + (away<2>(s[2]) + away<1>(s[3]));
}

template <int kCtrl>
__device__ __forceinline__ float quad_perm(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kCtrl, 0xf, 0xf, true));
}

// A for exponents of 2, finite where A is: a step width of 0 leaves the state.
__device__ __forceinline__ float exponent(float A) {
  const float x = A * kLog2e;
  return x < -3e38f ? -3e38f : x;
}

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

// Where a wave works: row b, group g, its first channel e0 (of E) and how many of 64 it has.
struct Tile {
  int b, g, e0, live;
};

// kW waves a block share a group's B and C, kCh channels each; `per_group` blocks a group.
template <int kW, int kCh>
__device__ __forceinline__ Tile tile_of(const SelScan& a, int64_t i, int per_group) {
  Tile t;
  const int W = a.E / a.G, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = (int)(i % per_group) * (kW * kCh) + wave * kCh;
  const int64_t rest = i / per_group;
  t.g = (int)(rest % a.G);
  t.b = (int)(rest / a.G);
  t.e0 = t.g * W + first;
  t.live = min(W - first, kCh);
  return t;
}

// Tokens of B and C that a block stages at a time.
template <int R>
constexpr int kStage = R <= 4 ? 32 : 16;

// Stages B and C of tokens t.. as fp32 [token][B, C][4 R], zeros beyond `end` and the states.  The
// values are fetched to registers first, so that they travel while the tile before is computed.
template <bool kBf16, int R, int kW, int kTok>
struct Stage {
  using El = Elem<kBf16>;
  using T = typename El::type;
  static constexpr int NP = 4 * R, kEach = (kTok * 2 * NP + kW * 64 - 1) / (kW * 64);
  T raw[kEach];
  const T *B, *C;
  int64_t bt, ct;
  int N;
  __device__ __forceinline__ void start(const SelScan& a, const Tile& w) {
    B = (const T*)a.Bt.p + w.b * a.Bt.sb + w.g * a.Bt.sh;
    C = (const T*)a.Ct.p + w.b * a.Ct.sb + w.g * a.Ct.sh;
    bt = a.Bt.st, ct = a.Ct.st, N = a.N;
  }
  __device__ __forceinline__ void fetch(int t, int end) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = threadIdx.x + k * kW * 64, n = i % NP, tok = t + i / (2 * NP);
      raw[k] = 0;
      if (i < kTok * 2 * NP && n < N && tok < end) raw[k] = i / NP % 2 ? C[tok * ct + n] : B[tok * bt + n];
    }
  }
  __device__ __forceinline__ void put(float* lds) const {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = threadIdx.x + k * kW * 64;
      if (i < kTok * 2 * NP) lds[i] = El::load(&raw[k]);
    }
  }
};

// R consecutive values of LDS.
template <int R>
__device__ __forceinline__ void read_states(const float* p, float (&v)[R]) {
  __builtin_memcpy(v, __builtin_assume_aligned(p, R >= 4 ? 16 : 4 * R), 4 * R);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// A token of the recurrence: h = exp2(d A) h + x B in each of four slots, B of this lane's states at
// p (LDS).  x B is an outer product of the channels of four neighbouring lanes and four states, which
// one matrix instruction adds to the decayed states: B's four values come from the four lanes, x
// from each.  It is exact as a fused multiplication and addition is.
template <int R>
__device__ __forceinline__ void advance(float (&h)[4][R], const float (&A)[4][R], const float (&d)[4], const float (&x)[4],
                                        const float* p, int lane) {
  if constexpr (R >= 4) {
    float b[R / 4];
#pragma unroll
    for (int m = 0; m < R / 4; ++m) b[m] = p[4 * m + (lane & 3)];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int m = 0; m < R / 4; ++m) {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = h[r][4 * m + i] * __builtin_amdgcn_exp2f(d[r] * A[r][4 * m + i]);
        v = __builtin_amdgcn_mfma_f32_4x4x1f32(b[m], x[r], v, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[r][4 * m + i] = v[i];
      }
  } else {
    float b[R];
    read_states<R>(p, b);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < R; ++i) h[r][i] = fmaf(h[r][i], __builtin_amdgcn_exp2f(d[r] * A[r][i]), x[r] * b[i]);
  }
}

// How time is cut: S segments of `len` tokens, a multiple of 32.
struct Segments {
  int S, len;
};

}  // namespace selscan
}  // namespace pnr
