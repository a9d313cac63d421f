// Activations in 8 bits: 32 consecutive channels share the least power of two 2^e, e >= -126, of
// which the largest is at most 127, and a value is its nearest multiple.  Powers of two make every
// step but that rounding exact.
//
// Memory bounds both directions: 2 or 4 bytes and 33 / 32 of one an element.  Four lanes hold a
// block, eight values each, so that loads are 16 bytes wide and the largest value meets in a
// quad; operands off that alignment take a lane a value.
#include <algorithm>

#include "seq_ops.h"

namespace pnr {
namespace {

struct PackArgs {
  Tokens x;
  int64_t rows;
  int T, E, blocks;          // blocks: of 32 values in a row
  int8_t* codes;
  uint8_t* exps;
  void* out;                 // unpack
};

// The exponent byte of a block whose largest magnitude has the bits `m` (not finite: 255).
__device__ __forceinline__ int exponent_byte(uint32_t m) {
  if (m >= 0x7f800000u) return 255;
  // m = f 2^k, 1 <= f < 2: f <= 127 / 64 fits with 2^(k - 6), otherwise 2^(k - 5)
  return max((int)(m >> 23) - 6 + ((m & 0x7fffffu) > 0x7e0000u), 1);
}

// On the top exponent 2^122, 64 steps are beyond fp32's (and bf16's) largest value.
__device__ __forceinline__ int code_of(float x, int s) {
  const int q = s == 255 ? 0 : (int)rintf(ldexpf(x, 127 - s));
  return s == 249 ? min(max(q, -63), 63) : q;
}

// kV values a lane: 8 (four lanes a block) or 1 (32 lanes a block).
template <bool kBf16, int kV, bool kPack>
__global__ void __launch_bounds__(256) checkpoint_kernel(PackArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  constexpr int L = kPackBlock / kV;                       // lanes of a block
  const int per_row = p.blocks * L;
  const int64_t total = p.rows * per_row, padded = (total + 255) / 256 * 256;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < padded; i += (int64_t)gridDim.x * 256) {
    const int64_t row = min(i, total - 1) / per_row;       // a block's lanes stay together
    const int c = (int)(min(i, total - 1) % per_row), e = c * kV;
    const bool live = i < total && e < p.E;                // kV divides E or is 1
    const int64_t at = row * p.E + e, exp_at = row * p.blocks + c / L;
    if constexpr (kPack) {
      const T* x = (const T*)p.x.p + row / p.T * p.x.sb + row % p.T * p.x.st + e;
      float v[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) v[k] = 0.0f;
      if (live) {
        if constexpr (kV == 1) {
          v[0] = El::load(x);
        } else {
          T raw[kV];
          __builtin_memcpy(raw, __builtin_assume_aligned(x, 16), sizeof(raw));
#pragma unroll
          for (int k = 0; k < kV; ++k) v[k] = El::load(&raw[k]);
        }
      }
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < kV; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
#pragma unroll
      for (int d = 1; d < L; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
      const int s = exponent_byte(m);
      if (live) {
        int8_t q[kV];
#pragma unroll
        for (int k = 0; k < kV; ++k) q[k] = (int8_t)code_of(v[k], s);
        __builtin_memcpy(__builtin_assume_aligned(p.codes + at, kV), q, kV);
        if (c % L == 0) p.exps[exp_at] = (uint8_t)s;
      }
    } else if (live) {
      const float step = unpack_step(p.exps[exp_at]);
      int8_t q[kV];
      __builtin_memcpy(q, __builtin_assume_aligned(p.codes + at, kV), kV);
      T* out = (T*)p.out + at;
      T raw[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) El::store(&raw[k], q[k] * step);
      __builtin_memcpy(__builtin_assume_aligned(out, sizeof(T) * kV > 16 ? 16 : sizeof(T) * kV), raw, sizeof(raw));
    }
  }
}

template <bool kBf16, int kV, bool kPack>
void launch(const PackArgs& p, hipStream_t st) {
  const int64_t total = p.rows * p.blocks * (kPackBlock / kV);
  checkpoint_kernel<kBf16, kV, kPack><<<(unsigned)std::min<int64_t>((total + 255) / 256, 1 << 16), 256, 0, st>>>(p);
}

template <bool kPack>
hipError_t launch(const PackArgs& p, bool bf16, bool vec, hipStream_t st) {
  if (p.rows > 0) {
    if (bf16)
      vec ? launch<true, 8, kPack>(p, st) : launch<true, 1, kPack>(p, st);
    else
      vec ? launch<false, 8, kPack>(p, st) : launch<false, 1, kPack>(p, st);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_checkpoint_pack(const Tokens& x, int B, int T, int E, int bf16, int8_t* codes, uint8_t* exps,
                                  hipStream_t st) {
  const int es = bf16 ? 2 : 4;
  const PackArgs p{x, (int64_t)B * T, T, E, (E + kPackBlock - 1) / kPackBlock, codes, exps, nullptr};
  const bool vec = E % 8 == 0 && (uintptr_t)x.p % 16 == 0 && x.sb * es % 16 == 0 && x.st * es % 16 == 0 && (uintptr_t)codes % 8 == 0;
  return launch<true>(p, bf16, vec, st);
}

hipError_t launch_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows, int E, int bf16, void* x,
                                    hipStream_t st) {
  const PackArgs p{{}, rows, 1, E, (E + kPackBlock - 1) / kPackBlock, const_cast<int8_t*>(codes), const_cast<uint8_t*>(exps), x};
  const bool vec = E % 8 == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)codes % 8 == 0;
  return launch<false>(p, bf16, vec, st);
}

}  // namespace pnr
