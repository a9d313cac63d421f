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

// A for exponents of 2, finite where A is: a step width of 0 leaves the state.
__device__ __forceinline__ float exponent(float A) {
  const float x = A * kLog2e;
  return x < -3e38f ? -3e38f : x;
}

// Where a wave works: row b, group g, its first channel e0 (of E) and how many of 64 it has.
struct Tile {
  int b, g, e0, live;
};

// kW waves a block share a group's B and C; `per_group` blocks a group.
template <int kW>
__device__ __forceinline__ Tile tile_of(const SelScan& a, int64_t i, int per_group) {
  Tile t;
  const int W = a.E / a.G, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = (int)(i % per_group) * (kW * kChannels) + wave * kChannels;
  const int64_t rest = i / per_group;
  t.g = (int)(rest % a.G);
  t.b = (int)(rest / a.G);
  t.e0 = t.g * W + first;
  t.live = min(W - first, kChannels);
  return t;
}

// Tokens of B and C that a block stages at a time: 1024 values of both for up to 16 states a channel.
template <int R>
constexpr int kStage = R <= 4 ? 32 : 128 / R;

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

// How time is cut: S segments of `len` tokens, a multiple of 32.
struct Segments {
  int S, len;
};

}  // namespace selscan
}  // namespace pnr
