// Activations in 8 bits: 32 consecutive channels share the least power of two 2^e, e >= -126, of
// which the largest is at most 127, and a value is its nearest multiple.  Powers of two make every
// step but that rounding exact.
//
// Memory bounds both directions: 2 or 4 bytes and 33 / 32 of one an element.  Four lanes hold a
// block, eight values each, so that loads are 16 bytes wide and the largest value meets in a
// quad; operands off that alignment take a lane a value.  16384 x 4096 bf16 pack in 43 us (4.7 TB/s) and
// unpack in 32 (6.3, partly from the last-level cache).  Rows and columns come from the launch: a division an
// item made packing 50 us, bound by issue.
#include <algorithm>

#include "seq_ops.h"

namespace pnr {
namespace {

struct PackArgs {
  Tokens x;
  int64_t rows;
  int T, E, blocks;          // blocks: of 32 values in a row
  bool even;                 // x's rows are x.st apart throughout
  int lanes, per_row;        // threads of a row (a power of two, at most 256); of them with work
  int col_blocks;
  int64_t row_blocks;        // of 256 / lanes rows
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

// The codes of kV values on exponent byte s.  x 2^(127 - s) is exact, and adding 3 2^22 rounds it to a whole
// number, ties to even, whose lowest byte is the code.
template <int kV>
__device__ __forceinline__ void codes_of(float (&v)[kV], int s, int8_t (&q)[kV]) {
  const float scale = __uint_as_float((uint32_t)(254 - s) << 23);
  if (s == 249) {            // on the top exponent 2^122, 64 steps are beyond fp32's (and bf16's) largest value
#pragma unroll
    for (int k = 0; k < kV; ++k) v[k] = fminf(fmaxf(v[k], -63.0f * 0x1p122f), 63.0f * 0x1p122f);
  }
#pragma unroll
  for (int k = 0; k < kV; ++k) q[k] = s == 255 ? (int8_t)0 : (int8_t)__float_as_uint(fmaf(v[k], scale, 12582912.0f));
}

// kV values a lane: 8 (four lanes a block) or 1 (32 lanes a block).
template <bool kBf16, int kV, bool kPack>
__global__ void __launch_bounds__(256) checkpoint_kernel(PackArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  constexpr int L = kPackBlock / kV;                       // lanes of a block
  const int per = 256 / p.lanes, c = blockIdx.x % p.col_blocks * p.lanes + (threadIdx.x & (p.lanes - 1)), e = c * kV;
  for (int64_t rb = blockIdx.x / p.col_blocks; rb < p.row_blocks; rb += gridDim.x / p.col_blocks) {
    const int64_t row = rb * per + threadIdx.x / p.lanes;
    const bool live = row < p.rows && e < p.E;             // kV divides E or is 1
    const int64_t at = row * p.E + e, exp_at = row * p.blocks + c / L;
    if constexpr (kPack) {
      float v[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) v[k] = 0.0f;
      if (live) {
        const T* x = (const T*)p.x.p + (p.even ? row * p.x.st : row / p.T * p.x.sb + row % p.T * p.x.st) + e;
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
        codes_of(v, s, q);
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
void launch(PackArgs p, hipStream_t st) {
  p.per_row = p.blocks * (kPackBlock / kV);                // whole blocks of 32: their lanes stay together
  p.lanes = kPackBlock / kV;
  while (p.lanes < 256 && p.lanes < p.per_row) p.lanes *= 2;
  p.col_blocks = (p.per_row + p.lanes - 1) / p.lanes;
  p.row_blocks = (p.rows + 256 / p.lanes - 1) / (256 / p.lanes);
  const int64_t most = std::max<int64_t>(1, (1 << 20) / p.col_blocks);
  checkpoint_kernel<kBf16, kV, kPack><<<(unsigned)(std::min(p.row_blocks, most) * p.col_blocks), 256, 0, st>>>(p);
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
  PackArgs p{};
  p.x = x, p.rows = (int64_t)B * T, p.T = T, p.E = E, p.blocks = (E + kPackBlock - 1) / kPackBlock;
  p.even = B == 1 || x.sb == (int64_t)T * x.st;
  p.codes = codes, p.exps = exps;
  const bool vec = E % 8 == 0 && (uintptr_t)x.p % 16 == 0 && x.sb * es % 16 == 0 && x.st * es % 16 == 0 && (uintptr_t)codes % 8 == 0;
  return launch<true>(p, bf16, vec, st);
}

hipError_t launch_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows, int E, int bf16, void* x,
                                    hipStream_t st) {
  PackArgs p{};
  p.rows = rows, p.E = E, p.blocks = (E + kPackBlock - 1) / kPackBlock;
  p.codes = const_cast<int8_t*>(codes), p.exps = const_cast<uint8_t*>(exps), p.out = x;
  const bool vec = E % 8 == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)codes % 8 == 0;
  return launch<false>(p, bf16, vec, st);
}

}  // namespace pnr
