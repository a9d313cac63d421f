// Activations in 8 bits: 32 consecutive channels share the least power of two 2^e, e >= -126, of
// which the largest is at most 127, and a value is its nearest multiple.  Powers of two make every
// step but that rounding exact.
//
// Memory bounds both directions: 2 or 4 bytes and 33 / 32 of one an element.  Four lanes hold a
// block, eight values each, so that loads are 16 bytes wide, on whatever address a row starts, and the
// largest value meets in a quad.  16384 x 4096 bf16 pack in 43 us (4.7 TB/s) and
// unpack in 32 (6.3, partly from the last-level cache).  Rows and columns come from the launch: a division an
// item made packing 50 us, bound by issue.
#include <algorithm>

#include "seq_ops.h"

namespace pnr {
namespace {

constexpr int kV = 8;        // values of a lane

struct PackArgs {
  Tokens x;
  int64_t rows;
  int T, E, blocks;          // blocks: of 32 values in a row
  bool even;                 // x's rows are x.st apart throughout
  int lanes;                 // threads of a row in a block: a power of two, at most 256
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

// The codes of a lane's values on exponent byte s.  x 2^(127 - s) is exact, and adding 3 2^22 rounds it to a whole
// number, ties to even, whose lowest byte is the code.
__device__ __forceinline__ void codes_of(float (&v)[kV], int s, int8_t (&q)[kV]) {
  const float scale = __uint_as_float((uint32_t)(254 - s) << 23);
  if (s == 249) {            // on the top exponent 2^122, 64 steps are beyond fp32's (and bf16's) largest value
#pragma unroll
    for (int k = 0; k < kV; ++k) v[k] = fminf(fmaxf(v[k], -63.0f * 0x1p122f), 63.0f * 0x1p122f);
  }
#pragma unroll
  for (int k = 0; k < kV; ++k) q[k] = s == 255 ? (int8_t)0 : (int8_t)__float_as_uint(fmaf(v[k], scale, 12582912.0f));
}

// Values between memory and a lane: eight at once, or the last few of a row.  kWhole: all rows are eights, aligned
// to 16 bytes or their own size.
template <bool kWhole, typename T>
__device__ __forceinline__ void load_some(const T* p, int n, T (&v)[kV]) {
  if (kWhole)
    __builtin_memcpy(v, __builtin_assume_aligned(p, sizeof(v) < 16 ? sizeof(v) : 16), sizeof(v));
  else if (n == kV)
    __builtin_memcpy(v, p, sizeof(v));
  else
#pragma unroll
    for (int k = 0; k < kV; ++k) v[k] = k < n ? p[k] : T(0);
}
template <bool kWhole, typename T>
__device__ __forceinline__ void store_some(T* p, int n, const T (&v)[kV]) {
  if (kWhole)
    __builtin_memcpy(__builtin_assume_aligned(p, sizeof(v) < 16 ? sizeof(v) : 16), v, sizeof(v));
  else if (n == kV)
    __builtin_memcpy(p, v, sizeof(v));
  else
#pragma unroll
    for (int k = 0; k < kV; ++k)
      if (k < n) p[k] = v[k];
}

template <bool kBf16, bool kPack, bool kWhole>
__global__ void __launch_bounds__(256) checkpoint_kernel(PackArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  constexpr int L = kPackBlock / kV;                       // lanes of a block
  const int per = 256 / p.lanes, c = blockIdx.x % p.col_blocks * p.lanes + (threadIdx.x & (p.lanes - 1)), e = c * kV;
  for (int64_t rb = blockIdx.x / p.col_blocks; rb < p.row_blocks; rb += gridDim.x / p.col_blocks) {
    const int64_t row = rb * per + threadIdx.x / p.lanes;
    const int n = row < p.rows ? min(kV, p.E - e) : 0;
    const bool live = n > 0;
    const int64_t at = row * p.E + e, exp_at = row * p.blocks + c / L;
    if constexpr (kPack) {
      float v[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) v[k] = 0.0f;
      if (live) {
        const T* x = (const T*)p.x.p + (p.even ? row * p.x.st : row / p.T * p.x.sb + row % p.T * p.x.st) + e;
        T raw[kV];
        load_some<kWhole>(x, n, raw);
#pragma unroll
        for (int k = 0; k < kV; ++k) v[k] = El::load(&raw[k]);
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
        store_some<kWhole>(p.codes + at, n, q);
        if (c % L == 0) p.exps[exp_at] = (uint8_t)s;
      }
    } else if (live) {
      const float step = unpack_step(p.exps[exp_at]);
      int8_t q[kV];
      load_some<kWhole>(p.codes + at, n, q);
      T raw[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) El::store(&raw[k], q[k] * step);
      store_some<kWhole>((T*)p.out + at, n, raw);
    }
  }
}

template <bool kBf16, bool kPack, bool kWhole>
void launch(PackArgs p, hipStream_t st) {
  const int per_row = p.blocks * (kPackBlock / kV);        // whole blocks of 32: their lanes stay together
  p.lanes = kPackBlock / kV;
  while (p.lanes < 256 && p.lanes < per_row) p.lanes *= 2;
  p.col_blocks = (per_row + p.lanes - 1) / p.lanes;
  p.row_blocks = (p.rows + 256 / p.lanes - 1) / (256 / p.lanes);
  const int64_t most = std::max<int64_t>(1, (1 << 20) / p.col_blocks);
  checkpoint_kernel<kBf16, kPack, kWhole><<<(unsigned)(std::min(p.row_blocks, most) * p.col_blocks), 256, 0, st>>>(p);
}

template <bool kPack>
hipError_t launch(const PackArgs& p, bool bf16, bool whole, hipStream_t st) {
  // 16384 x 4096 bf16, us in a loop over one tensor, as whole rows and as any others: packing 37 and 42, unpacking 33 and 41 (the few last values'
  // loads and stores are in everybody's way); a lane a value took 215 and 160 for 4095
  if (p.rows > 0) {
    if (bf16)
      whole ? launch<true, kPack, true>(p, st) : launch<true, kPack, false>(p, st);
    else
      whole ? launch<false, kPack, true>(p, st) : launch<false, kPack, false>(p, st);
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
  const bool whole = E % kV == 0 && (uintptr_t)x.p % 16 == 0 && x.sb * es % 16 == 0 && x.st * es % 16 == 0 && (uintptr_t)codes % kV == 0;
  return launch<true>(p, bf16, whole, st);
}

hipError_t launch_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows, int E, int bf16, void* x,
                                    hipStream_t st) {
  PackArgs p{};
  p.rows = rows, p.E = E, p.blocks = (E + kPackBlock - 1) / kPackBlock;
  p.codes = const_cast<int8_t*>(codes), p.exps = const_cast<uint8_t*>(exps), p.out = x;
  const bool whole = E % kV == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)codes % kV == 0;
  return launch<false>(p, bf16, whole, st);
}

}  // namespace pnr
