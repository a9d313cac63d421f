// The chunk kernel of the linear attention: device code shared by linattn_fwd.hip and
// linattn_bwd.hip.
//
// One recurrence in several roles.  With queries x, keys y, values z, tokens of a chunk
// 1..C, G_i = g_1 + ... + g_i and S the state at the chunk's start,
//   out_i = exp(G_i) S^T x_i + sum_{j <= i} exp(G_i - G_j) (x_i . y_j) z_j
//   S    <- exp(G_C) S + sum_j exp(G_C - G_j) y_j z_j^T
// and against time, S being what later chunks send back and H_i = g_{i+1} + ... + g_C,
//   out_i = exp(H_i) S^T x_i + sum_{j >= i} exp(H_i - H_j) (x_i . y_j) z_j
//   S    <- exp(G_C) S + sum_j exp(G_C - H_j) y_j z_j^T.
// Sums from the chunk's end, because a decay that is not finite then stays where it has a part.
//         x    y    z    direction   state
//   o     q    k    v    forward     S
//   dq    do   v    k    forward     S transposed
//   dk    v    do   q    backward    dL/dS transposed
//   dv    k    q    do   backward    dL/dS
#pragma once

#include "seq_ops.h"

namespace pnr {
namespace linattn {

constexpr int kChunk = 64;
constexpr int kWalk = 4;        // chunks between two exact values of <S, E>, from a segment's start on (see linattn_bwd.hip)

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

enum Kind {
  kOut,         // outputs
  kDotQ,        // dq, and from it u and b of the decay's gradient
  kDotK,        // dk, and from it c of the decay's gradient
};

// Segments with tokens of a row of n.  Those behind them have no sum, decay, entry state or crossing sum.
__device__ __forceinline__ int segments_of(int n, int seg_chunks) {
  const int64_t tokens = (int64_t)seg_chunks * kChunk;
  return (int)((n + tokens - 1) / tokens);
}

struct RoleArgs {
  LinAttn a;
  Rows x, y, z, e;       // queries, keys, values; the rows that the outputs' dot products are taken with
  int nq, nkv;           // heads of x, e and the outputs, and of y and z, per state head; one of them is 1
  int dk, dv;            // columns of x and y, and of z, e and the outputs
  int transposed;        // states are stored [dv][dk]
  int vec;               // rows of x, y, z, e may be read in 16-byte pieces, outputs written four at a time
  float p_scale, inter_scale, upd_scale;   // on scores, on S^T x, on y z^T
  const float* s_in;     // [B][Hkv][nseg] states at the segments' entry, or nullptr: zeros
  float* s_out;          // [B][Hkv][nseg] states at the segments' exit, or nullptr
  float* seg_decay;      // sum_kernel: [B][Hkv][nseg] the segment's whole decay
  void* o;
  float* u;              // [B][Hkv][T]: u + b (kDotQ), c (kDotK) of the decay's gradient
  float* b;              // [B][Hkv][chunks]: sums of b (kDotQ)
  int marks;             // kWalk chunks each that a segment has
  float* s_mid;          // kDotQ: [B][Hkv][nseg][marks - 1] states before all but the first of them, whole tiles in
                         // the order of their registers, written; kDotK: read; or nullptr
  float* x_end;          // kDotK: [B][Hkv][nseg][marks] <state after the last of these tokens, its gradient>, or nullptr
  const float* s_entry;  // ... that state at a segment's end, for all but the last: the next one's entry, [B][Hkv][nseg]
  const float* s_last;   // ... and after the last, [B][Hkv]
  float* x_first;        // kDotK: [B][Hkv] <state before the first token, its gradient>, or nullptr
  const float* s_first;  // ... that state
  int seg_chunks, nseg;
};

// ---- fragments ---------------------------------------------------------------------------
// An MFMA operand covers 16 rows (or columns) x 32 of the summed index: lane l holds row l & 15 and
// the eight summed indexes 8 g + e of its group g = l >> 4.  An accumulator tile holds rows
// 4 g + r.  So that the state, kept in accumulators, is an operand without leaving its registers,
// row m of its tile kt stands for row state_row(kt, m) of S: the eight values that a
// lane holds in tiles 2 k and 2 k + 1 are then rows 32 k + 8 g + 0 .. 7.
__device__ __forceinline__ int state_row(int kt, int m) { return kt / 2 * 32 + m / 4 * 8 + kt % 2 * 4 + m % 4; }

template <bool kBf16>
struct Mma;

template <>
struct Mma<true> {
  using Elt = uint16_t;
  using Frag = bf16x8;
  static constexpr int kPiece = 8;     // elements of a 16-byte piece
  static constexpr int kPadZ = 8;      // elements of padding a row: rows start 4 banks apart
  static __device__ __forceinline__ f32x4 mul(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ Frag rows(const Elt* p) { return *(const Frag*)p; }
  // Eight rows of one column: two transposing reads of 4 rows x 16 columns, for which lane i of a
  // group points at row i / 4 and the four columns from col0 + kStride (i % 4) on; lane l receives
  // column l of the 16.
  template <int kStride>
  static __device__ __forceinline__ Frag cols(const Elt* tile, int pitch, int row0, int col0, int lane) {
    const Elt* p = tile + (row0 + (lane >> 4) * 8 + ((lane >> 2) & 3)) * pitch + col0 + (lane & 3) * kStride;
    return cols_at(p, p + 4 * pitch);
  }
  static __device__ __forceinline__ Frag cols_at(const Elt* p, const Elt* four_rows_on) {
    using L = __attribute__((address_space(3))) s16x4;
    struct { s16x4 a, b; } w{__builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)p),
                             __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)four_rows_on)};
    return __builtin_bit_cast(Frag, w);
  }
  static __device__ __forceinline__ Frag none() { return Frag{}; }
};

template <>
struct Mma<false> {
  using Elt = float;
  struct Frag { float v[8]; };
  static constexpr int kPiece = 4;
  static constexpr int kPadZ = 4;
  static __device__ __forceinline__ f32x4 mul(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ Frag two(const float* p, const float* q) {
    Frag f;
    const float4 a = *(const float4*)p, b = *(const float4*)q;
    f.v[0] = a.x, f.v[1] = a.y, f.v[2] = a.z, f.v[3] = a.w;
    f.v[4] = b.x, f.v[5] = b.y, f.v[6] = b.z, f.v[7] = b.w;
    return f;
  }
  static __device__ __forceinline__ Frag rows(const Elt* p) { return two(p, p + 4); }
  template <int kStride>
  static __device__ __forceinline__ Frag cols(const Elt* tile, int pitch, int row0, int col0, int lane) {
    Frag f;
    const Elt* p = tile + (row0 + (lane >> 4) * 8) * pitch + col0 + ((lane >> 2) & 3) * kStride + (lane & 3);
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = p[e * pitch];
    return f;
  }
  static __device__ __forceinline__ Frag none() { return Frag{}; }
};

// Eight fp32 values as an operand: in fp32 as they are; in bf16 as the sum of kParts bf16 values,
// each the rounding of what the ones before it leave.  Two parts are good to 2^-17 of each value, and
// go where the result is rounded to bf16 afterwards (one part, 2^-9, made outputs off by 2.3e-3 of their norm
// where their own rounding is 1.7e-3); three are good to 2^-26, and go where a result in fp32 depends on
// them (two showed in such results: 2e-6 of a state).
template <bool kBf16, int kParts>
struct Split;
template <int kParts>
struct Split<true, kParts> {
  bf16x8 part[kParts];
  __device__ __forceinline__ Split() {}
  __device__ __forceinline__ explicit Split(float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        w[e / 2] = pack_bf16(v[e], v[e + 1]);
        if (k + 1 < kParts) {
          v[e] -= __uint_as_float(w[e / 2] << 16);
          v[e + 1] -= __uint_as_float(w[e / 2] & 0xffff0000u);
        }
      }
      __builtin_memcpy(&part[k], w, 16);
    }
  }
};
template <int kParts>
struct Split<false, kParts> {
  Mma<false>::Frag part[1];
  __device__ __forceinline__ Split() {}
  __device__ __forceinline__ explicit Split(float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[0].v[e] = v[e];
  }
};

// x of lane 63
__device__ __forceinline__ double wave_last(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return __builtin_bit_cast(double, (uint64_t)__builtin_amdgcn_readlane((uint32_t)(u >> 32), 63) << 32 |
                                        (uint32_t)__builtin_amdgcn_readlane((uint32_t)u, 63));
}

// The same number, as far as the compiler can tell computed anew: addresses made from it stay where
// they are used instead of being kept in registers over the whole loop.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// ---- tiles ---------------------------------------------------------------------------------
template <bool kBf16, int kCols, int kThreads>
struct Direct;

// 64 rows of keys in LDS, which are read by rows (scores) and by columns (the state's update).
template <bool kBf16, int kCols>
struct Keys;

// bf16: no padding; the 16-byte pieces of a row are permuted by the row so that neither 16 rows of one
// piece nor the four rows x four pieces of a transposing read meet in a bank.
template <int kCols>
struct Keys<true, kCols> {
  using M = Mma<true>;
  using Elt = M::Elt;
  static constexpr int kPerRow = kCols / M::kPiece, kSize = kChunk * kCols;
  static __device__ __forceinline__ int permute(int row) {
    return (kCols == 128 ? (row & 3) << 2 : (row & 2) << 1) | (row >> 2 & 3);
  }
  // first element of a row's piece; rows 16 apart are permuted alike
  static __device__ __forceinline__ int at(int row, int piece) { return (row * kPerRow + (piece ^ permute(row))) * M::kPiece; }
  static __device__ __forceinline__ M::Frag rows(const Elt* t, int row, int k, int g) {
    return M::rows(t + (at(row, g) ^ k * 32));
  }
  // rows 32 k + 8 g + 0 .. 7 of the columns that tile kt of the state stands for (see state_row)
  static __device__ __forceinline__ M::Frag cols(const Elt* t, int k, int kt, int lane) {
    const int row = (lane >> 4) * 8 + ((lane >> 2) & 3), first = at(row, lane & 3) ^ kt / 2 * 32;
    const Elt* p = t + k * 32 * kCols + kt % 2 * 4;
    return M::cols_at(p + first, p + (first ^ 8) + 4 * kCols);       // four rows on, the permutation differs by a piece
  }
};
template <int kCols>
struct Keys<false, kCols> {
  using M = Mma<false>;
  using Elt = M::Elt;
  static constexpr int kPitch = kCols + 4, kSize = kChunk * kPitch;
  static __device__ __forceinline__ int at(int row, int piece) { return row * kPitch + piece * M::kPiece; }
  static __device__ __forceinline__ M::Frag rows(const Elt* t, int row, int k, int g) {
    return M::rows(t + row * kPitch + k * 32 + g * 8);
  }
  static __device__ __forceinline__ M::Frag cols(const Elt* t, int k, int kt, int lane) {
    return M::cols<8>(t, kPitch, k * 32, state_row(kt, 0), lane);
  }
};

// A buffer from p on, of any length: offsets from kNowhere on lie behind its end, where loads give
// zeros and stores are dropped.
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, 0x7fffffff, 0x00027000);
}

// The rows of one batch row and head.
template <bool kBf16>
struct Source {
  using Elt = typename Mma<kBf16>::Elt;
  const Elt* p;
  int64_t st;
  uint32_t pitch;        // st in bytes, where 64 rows span less than 2^31 of them
  __device__ __forceinline__ Source(const Rows& r, int b, int h)
      : p((const Elt*)r.p + b * r.sb + h * r.sh), st(r.st), pitch((uint32_t)r.st * (uint32_t)sizeof(Elt)) {}
  __device__ __forceinline__ const Elt* at(int t) const { return p + t * st; }
};

// 64 rows x kCols of one operand on its way from memory to LDS: 16-byte pieces in registers.
template <bool kBf16, int kCols, int kThreads>
struct Stage {
  using M = Mma<kBf16>;
  using Elt = typename M::Elt;
  static constexpr int kPerRow = kCols / M::kPiece;
  static constexpr int kN = kChunk * kPerRow / kThreads;
  uint4 v[kN];

  // Rows t0 .. t0 + 63; rows at or past n and columns past `cols` are zeros.  kVec: every piece is
  // one aligned buffer load from a uniform base, and 64 rows span less than 2^31 bytes; a piece
  // that is not there gets an offset past the buffer's end, which reads as zeros without a branch.
  template <bool kVec>
  __device__ __forceinline__ void load(const Source<kBf16>& src, uint32_t off, int t0, int n, int cols) {
    constexpr int kStep = kThreads / kPerRow;            // rows between a thread's pieces
    const Elt* base = src.at(t0);
    if constexpr (kVec) {
      const __amdgpu_buffer_rsrc_t rsrc = buffer_at(base);
      if (t0 + kChunk <= n) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
          v[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, i * kStep * src.pitch, 0));
      } else {
        const int left = n - t0 - (int)fresh(threadIdx.x) / kPerRow;
#pragma unroll
        for (int i = 0; i < kN; ++i)
          v[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, left > i * kStep ? off : kNowhere, i * kStep * src.pitch, 0));
      }
    } else {
      const int tid = fresh(threadIdx.x), row = tid / kPerRow, c = (tid % kPerRow) * M::kPiece;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        Elt e[M::kPiece];
        const bool live = t0 + row + i * kStep < n;
        const Elt* from = base + (row + i * kStep) * src.st + c;
#pragma unroll
        for (int k = 0; k < M::kPiece; ++k) e[k] = live && c + k < cols ? from[k] : Elt(0);
        __builtin_memcpy(&v[i], e, 16);
      }
    }
  }
  // byte offset of a thread's first piece from its chunk's base
  static __device__ __forceinline__ uint32_t offset(uint32_t pitch, int cols) {
    const int tid = threadIdx.x, c = (tid % kPerRow) * M::kPiece;
    return c < cols ? tid / kPerRow * pitch + c * (uint32_t)sizeof(Elt) : kNowhere;
  }
  // rows `pitch` apart
  template <int kPitch>
  __device__ __forceinline__ void store(Elt* tile) const {
    const int tid = fresh(threadIdx.x);
    put<kPitch>(tile + (tid / kPerRow) * kPitch + (tid % kPerRow) * M::kPiece);
  }
  __device__ __forceinline__ void store_keys(Elt* tile) const {
    static_assert(!kBf16 || kThreads / kPerRow % 16 == 0, "one permutation for all of a thread's rows");
    const int tid = fresh(threadIdx.x);
    put<Keys<kBf16, kCols>::kSize / kChunk>(tile + Keys<kBf16, kCols>::at(tid / kPerRow, tid % kPerRow));
  }
  template <int kPitch>
  __device__ __forceinline__ void put(Elt* at) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) *(uint4*)(at + i * (kThreads / kPerRow) * kPitch) = v[i];
  }
  __device__ __forceinline__ void store_permuted(Elt* tile) const {      // as a Direct tile
    const int tid = fresh(threadIdx.x);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      *(uint4*)(tile + Direct<kBf16, kCols, kThreads>::at(tid / kPerRow + i * (kThreads / kPerRow), tid % kPerRow)) = v[i];
  }
};

// 64 rows x kCols without padding, the 16-byte pieces of a row permuted by the row so that 16 rows of
// one piece spread over the banks: the form that loads can fill without passing through
// registers, whose lanes write to consecutive addresses.
template <bool kBf16, int kCols, int kThreads>
struct Direct {
  using M = Mma<kBf16>;
  using Elt = typename M::Elt;
  static constexpr int kPerRow = kCols / M::kPiece;
  static constexpr int kStep = kThreads / kPerRow;       // rows between a thread's pieces, which one permutation serves
  static __device__ __forceinline__ int permute(int row) { return kPerRow >= 16 ? row & (kStep >= 16 ? 15 : 7) : row >> 1 & 7; }
  static_assert(kStep % (kPerRow < 16 || kStep >= 16 ? 16 : 8) == 0, "one permutation for all of a thread's rows");
  // first element of a row's piece
  static __device__ __forceinline__ int at(int row, int piece) { return (row * kPerRow + (piece ^ permute(row))) * M::kPiece; }
  static __device__ __forceinline__ typename M::Frag rows(const Elt* t, int row, int k, int g) {
    if constexpr (kBf16) return M::rows(t + at(row, k * 4 + g));
    else return M::two(t + at(row, k * 8 + g * 2), t + at(row, k * 8 + g * 2 + 1));
  }
  // rows t0 .. t0 + 63 as Stage::load takes them, straight to LDS; complete once vmcnt says so
  static __device__ __forceinline__ void load(const Source<kBf16>& src, uint32_t off, int t0, int n, Elt* tile, int wave) {
    const __amdgpu_buffer_rsrc_t rsrc = buffer_at(src.at(t0));
    const int left = t0 + kChunk <= n ? kChunk : n - t0 - (int)fresh(threadIdx.x) / kPerRow;
#pragma unroll
    for (int i = 0; i < kChunk / kStep; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(tile + (i * kThreads + wave * 64) * M::kPiece),
                                               16, left > i * kStep ? off : kNowhere, i * kStep * src.pitch, 0, 0);
  }
  static __device__ __forceinline__ uint32_t offset(uint32_t pitch, int cols) {
    const int tid = threadIdx.x, row = tid / kPerRow, c = ((tid % kPerRow) ^ permute(row)) * M::kPiece;
    return c < cols ? row * pitch + c * (uint32_t)sizeof(Elt) : kNowhere;
  }
};

// x of the lanes that a DPP move brings together, 0 where it brings nothing
template <int kCtrl, int kRows>
__device__ __forceinline__ double dpp_move(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, kRows, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, kRows, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// inclusive scan over the wave: within rows of 16 lanes, then across them
__device__ __forceinline__ double wave_scan(double x) {
  x += dpp_move<0x111, 0xf>(x);      // row_shr:1
  x += dpp_move<0x112, 0xf>(x);
  x += dpp_move<0x114, 0xf>(x);
  x += dpp_move<0x118, 0xf>(x);
  x += dpp_move<0x142, 0xa>(x);      // row_bcast:15 to rows 1 and 3
  x += dpp_move<0x143, 0xc>(x);      // row_bcast:31 to rows 2 and 3
  return x;
}

__device__ __forceinline__ float row16_sum(float v) {      // over the 16 lanes of a group
  v += __shfl_xor(v, 1);
  v += __shfl_xor(v, 2);
  v += __shfl_xor(v, 4);
  return v + __shfl_xor(v, 8);
}
__device__ __forceinline__ float group_sum(float v) {      // over the four groups
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// A chunk's weighted scores in LDS, row i of which may see column j <= i (j >= i against time).
template <bool kBf16, bool kReverse>
struct Scores;

// bf16: two parts, and of the 16 x 16 tiles only the ten on and before the diagonal.  16 rows of half a tile's
// columns, 16 bytes each, lie side by side in the banks.
template <bool kReverse>
struct Scores<true, kReverse> {
  using M = Mma<true>;
  using Elt = M::Elt;
  static constexpr int kParts = 2, kPart = 10 * 256, kSize = kParts * kPart;
  static __device__ __forceinline__ int tile(int it, int jt) {
    if (kReverse) it = 3 - it, jt = 3 - jt;
    return (it * (it + 1) / 2 + jt) * 256;
  }
  // columns j .. j + 3 of row i, within tile (it, jt)
  static __device__ __forceinline__ void put(Elt* p, int it, int jt, int i, int j, const float (&s)[4]) {
    if (kReverse ? jt < it : jt > it) return;
    Elt* at = p + tile(it, jt) + i * 16 + j;
    const uint2 hi = make_uint2(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]));
    *(uint2*)at = hi;
    *(uint2*)(at + kPart) = make_uint2(pack_bf16(s[0] - __uint_as_float(hi.x << 16), s[1] - __uint_as_float(hi.x & 0xffff0000u)),
                                       pack_bf16(s[2] - __uint_as_float(hi.y << 16), s[3] - __uint_as_float(hi.y & 0xffff0000u)));
  }
  // rows of tile row m, columns 32 k + 8 g + 0 .. 7: two tiles, one of which may be the one behind the diagonal
  static __device__ __forceinline__ M::Frag rows(const Elt* p, int part, int m, int k, int lane) {
    const int g = lane >> 4, half = g >> 1;
    const M::Frag f = M::rows(p + part * kPart + tile(m, 2 * k) + (kReverse ? -half : half) * 256 + (lane & 15) * 16 + (g & 1) * 8);
    if (m / 2 != k || m % 2 != (kReverse ? 1 : 0)) return f;
    return half == (kReverse ? 0 : 1) ? M::none() : f;
  }
  static __device__ __forceinline__ float value(const Elt* p, int i, int j) {
    const Elt* at = p + tile(i >> 4, j >> 4) + (i & 15) * 16 + (j & 15);
    return bf16_to_f32(at[0]) + bf16_to_f32(at[kPart]);
  }
};
// fp32: rows of 64 without padding, their 16-byte pieces permuted by the row so that 16 rows of one
// column spread over the banks.
template <bool kReverse>
struct Scores<false, kReverse> {
  using M = Mma<false>;
  using Elt = M::Elt;
  static constexpr int kParts = 1, kSize = kChunk * kChunk;
  static __device__ __forceinline__ int at(int i, int j) { return i * kChunk + (((j / 4) ^ (i & 15)) * 4) + j % 4; }
  static __device__ __forceinline__ void put(Elt* p, int it, int jt, int i, int j, const float (&s)[4]) {
    *(float4*)(p + at(it * 16 + i, jt * 16 + j)) = make_float4(s[0], s[1], s[2], s[3]);
  }
  static __device__ __forceinline__ M::Frag rows(const Elt* p, int, int m, int k, int lane) {
    const int i = m * 16 + (lane & 15), j = k * 32 + (lane >> 4) * 8;
    return M::two(p + at(i, j), p + at(i, j + 4));
  }
  static __device__ __forceinline__ float value(const Elt* p, int i, int j) { return p[at(i, j)]; }
};

// A chunk's weights.
struct alignas(16) Weights {
  float ghi[kChunk];                 // G, or H, in units of log2, as the sum of a float
  uint16_t glo[kChunk];              // ... and a bf16
  float upd[kChunk];                 // the weights of y z^T
  float total;                       // exp(G_C)
};

// S += Y^T (w Z) over the 32 tokens 32 k + 0 .. 31 of y, for 16 columns of Z held as an operand; kGroup row
// tiles at a time.
template <bool kBf16, int DK, int kGroup>
__device__ __forceinline__ void add_outer(f32x4 (&S)[DK / 16], const typename Mma<kBf16>::Frag& zf, const float* w,
                                          const typename Mma<kBf16>::Elt* y, int k, int lane) {
  using M = Mma<kBf16>;
  const float* wp = w + (lane >> 4) * 8;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (kBf16) v[e] = wp[e] * (float)zf[e]; else v[e] = wp[e] * zf.v[e];
  }
  const Split<kBf16, 3> wz(v);
#pragma unroll
  for (int kt = 0; kt < DK / 16; kt += kGroup) {
    typename M::Frag yf[kGroup];
#pragma unroll
    for (int q = 0; q < kGroup; ++q) yf[q] = Keys<kBf16, DK>::cols(y, k, kt + q, lane);
#pragma unroll
    for (int part = (kBf16 ? 3 : 1); part--;)
#pragma unroll
      for (int q = 0; q < kGroup; ++q) S[kt + q] = M::mul(yf[q], wz.part[part], S[kt + q]);
  }
}

// A block walks the chunks of one segment of one state head, with the state in accumulators: a wave
// holds 16 columns of S, all DK rows.  A chunk, in two halves with a barrier between them:
//   scores    P^T = Y X^T, two or four 16 x 16 tiles a wave, weighted, to LDS (in bf16: as two parts)
//   inter     O^T = S^T X^T, weighted; S enters as two bf16 parts, or as three where a dot product in
//             fp32 is taken from it
//   intra     O^T += Z^T P^T
//   update    S = exp(G_C) S + Y^T (w Z), w Z as three bf16 parts
// X and E are done with after the first half and are loaded straight into LDS during the second; Y
// and Z wait in registers.
//
// Measured, 16 heads of 128 x 128 in bf16 over 32768 tokens (kOut, 512 blocks, two a CU): 148 us for
// 575 MB, 3.9 TB/s; with one part each of scores and state, 134.  A chunk then cost a CU 4.2 us with two
// blocks (4.6 now) and 4.8 with one; left out one at a time, of those 4.2 the update was 1.1, the outputs
// 0.7, the loads 0.5, the scores 0.45, S^T X^T 0.4, Z^T P^T 0.2.  Matrix and vector instructions of a SIMD hardly overlap
// here (24 products and 96 fused multiply-adds, two waves each: 775 and 558 cycles alone, 1214
// together), so both are kept few.  32 columns a wave in half the waves, with half the reads of
// X and Y from LDS: 145 us where this took 137.
template <bool kBf16, int DK, int DV, bool kReverse, Kind kind, bool kVec>
__global__ void __launch_bounds__(DV * 4, kBf16 ? 4 : DV / 64) chunk_kernel(RoleArgs p) {
  using M = Mma<kBf16>;
  using Elt = typename M::Elt;
  using Frag = typename M::Frag;
  constexpr int kWaves = DV / 16, kThreads = kWaves * 64;
  constexpr int KT = DK / 16;               // row tiles of S
  constexpr int JT = 16 / kWaves;           // score tiles a wave takes of its query row tile
  constexpr int PV = DV + M::kPadZ;         // rows of Z in LDS
  using KY = Keys<kBf16, DK>;
  using SC = Scores<kBf16, kReverse>;
  constexpr bool kDots = kind == kDotQ || kind == kDotK;
  constexpr int kParts = kDots ? 3 : 2;     // of S
  // LDS (bf16, 128 x 128: two blocks a CU, also with the dot products' arrays).  Arrays of their own,
  // so that a read of one need not wait for loads on their way to another.
  __shared__ alignas(16) Elt lds_x[kChunk * DK];           // Direct
  __shared__ alignas(16) Elt lds_y[KY::kSize];
  __shared__ alignas(16) Elt lds_z[kChunk * PV];
  __shared__ alignas(16) Elt lds_e[kDots ? kChunk * DV : 1];          // Direct
  __shared__ alignas(16) Elt lds_p[SC::kSize];
  __shared__ Weights lds_w[2];                                        // this chunk's and the next one's
  __shared__ float lds_dot[kDots ? kWaves : 1][kChunk];               // the waves' parts of dot products and row sums
  __shared__ float lds_bsum[kDots ? kWaves : 1];
  __shared__ float lds_col[kind == kDotQ ? 10 : 1][16];               // column sums of the score tiles up to the diagonal

  const LinAttn& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l15 = lane & 15, g4 = (lane >> 4) * 4;
  const int seg = blockIdx.x % p.nseg;
  const int h = blockIdx.x / p.nseg % a.Hkv, b = blockIdx.x / p.nseg / a.Hkv;
  const int n = row_len(a.lens, b, a.T);
  const int c_lo = seg * p.seg_chunks, c_all = (a.T + kChunk - 1) / kChunk;
  const int c_hi = min(c_lo + p.seg_chunks, c_all);
  const int live = min(c_hi, (n + kChunk - 1) / kChunk);       // chunks c_lo .. live - 1 hold tokens
  const int nsub = p.nq > p.nkv ? p.nq : p.nkv;
  const size_t sbase = (size_t)blockIdx.x * p.dk * p.dv;
  const int col0 = wave * 16;                                  // the wave's first column
  const int it0 = wave / (kWaves / 4), jt0 = wave % (kWaves / 4) * JT;   // its score tiles

  const int count = live > c_lo ? (live - c_lo) * nsub : 0;
  const bool has_state = p.s_in && (count > 0 || p.s_out);     // a segment without tokens has no entry state

  f32x4 S[KT];
  auto s_at = [&](int kt, int r) {     // element (row, column) of accumulator register r
    const int i = state_row(kt, g4) + r, j = col0 + l15;
    return sbase + (p.transposed ? (size_t)j * p.dk + i : (size_t)i * p.dv + j);
  };
  auto s_in_range = [&](int kt, int r) { return state_row(kt, g4) + r < p.dk && col0 + l15 < p.dv; };
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S[kt][r] = (has_state && s_in_range(kt, r)) ? p.s_in[s_at(kt, r)] : 0.0f;

  // the loads of S end here: a wait for them inside the loop would wait for the tiles behind them
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
    asm volatile("" : "+v"(S[kt]));

  // the waves' parts of a sum go to lds_bsum, from where, after a barrier, thread 0 adds them
  auto share = [&](float s) {
    s = row16_sum(group_sum(s));
    if (lane == 0) lds_bsum[wave] = s;
  };
  auto shared = [&]() {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += lds_bsum[w];
    return s;
  };
  auto dot_state = [&](const float* other) {       // <S, other>, other a state at s_at
    float s = 0.0f;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (s_in_range(kt, r)) s += S[kt][r] * other[s_at(kt, r)];
    share(s);
  };
  const size_t s_size = (size_t)p.dk * p.dv;
  const int row = blockIdx.x / p.nseg;
  if constexpr (kind == kDotK) {
    if (p.x_end && count > 0) {
      dot_state(seg + 1 < segments_of(n, p.seg_chunks) ? p.s_entry + s_size : p.s_last - sbase + row * s_size);
      __syncthreads();
      if (tid == 0) p.x_end[(size_t)blockIdx.x * p.marks + (live - 1 - c_lo) / kWalk] = shared();
    }
  }

  using TX = Direct<kBf16, DK, kThreads>;
  using TE = Direct<kBf16, DV, kThreads>;
  Stage<kBf16, DK, kThreads> sx, sy;
  Stage<kBf16, DV, kThreads> sz, se;
  const uint32_t es = sizeof(Elt);
  const uint32_t off_x = kVec ? TX::offset((uint32_t)p.x.st * es, p.dk) : 0, off_e = kVec && kDots ? TE::offset((uint32_t)p.e.st * es, p.dv) : 0;
  const uint32_t off_y = kVec ? decltype(sy)::offset((uint32_t)p.y.st * es, p.dk) : 0, off_z = kVec ? decltype(sz)::offset((uint32_t)p.z.st * es, p.dv) : 0;
  // Lane l scans what G_l, or H_{63 - l}, has more than the lane before: the log decay of token l, or of token
  // 64 - l; against time, lane 0 holds token 0, which only the chunk's whole decay has.
  const int g_token = kReverse ? (lane ? kChunk - lane : 0) : lane, g_row = kReverse ? kChunk - 1 - lane : lane;
  float g_next = 0.0f;
  auto fetch = [&](int c, int sub) {
    const int t0 = c * kChunk;
    if (sub == 0 && wave == 0) {
      const int t = min(t0 + g_token, n - 1);
      g_next = a.g[a.decay_token ? ((size_t)b * a.T + t) * a.Hkv + h : (size_t)h];
    }
    if constexpr (!kVec)
      if (p.nq > 1 || sub == 0) {
        const int hh = h * p.nq + (p.nq > 1 ? sub : 0);
        sx.template load<kVec>(Source<kBf16>(p.x, b, hh), 0, t0, n, p.dk);
        if constexpr (kDots) se.template load<kVec>(Source<kBf16>(p.e, b, hh), 0, t0, n, p.dv);
      }
    if (p.nkv > 1 || sub == 0) {
      const int hh = h * p.nkv + (p.nkv > 1 ? sub : 0);
      sy.template load<kVec>(Source<kBf16>(p.y, b, hh), off_y, t0, n, p.dk);
      sz.template load<kVec>(Source<kBf16>(p.z, b, hh), off_z, t0, n, p.dv);
    }
  };

  // X and E are done with once the first half of a chunk is: aligned rows go straight to them then
  auto fetch_direct = [&](int c, int sub) {
    if constexpr (kVec)
      if (p.nq > 1 || sub == 0) {
        const int hh = h * p.nq + (p.nq > 1 ? sub : 0), t0 = c * kChunk;
        TX::load(Source<kBf16>(p.x, b, hh), off_x, t0, n, lds_x, wave);
        if constexpr (kDots) TE::load(Source<kBf16>(p.e, b, hh), off_e, t0, n, lds_e, wave);
      }
  };
  // Wave 0 turns the log decays that it fetched into a chunk's weights.  The scan is in 64 bits, because
  // differences of sums of log decays (each down to -104) are what counts.
  auto weigh = [&](int c, int slot) {
    const float g = c * kChunk + g_token < n ? clamp_log_decay(g_next) : 0.0f;
    const double x = wave_scan(kReverse && lane == 0 ? 0.0 : (double)g * 1.4426950408889634);
    double end = wave_last(x);
    if (kReverse) end += (double)__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(g))) * 1.4426950408889634;
    const float hi = (float)x;
    auto& w = lds_w[slot];
    w.ghi[g_row] = hi;
    w.glo[g_row] = f32_to_bf16((float)(x - (double)hi));
    w.upd[g_row] = __builtin_amdgcn_exp2f((float)(end - x)) * p.upd_scale;
    if (lane == 0) w.total = __builtin_amdgcn_exp2f((float)end);
  };
  if (count > 0) {
    fetch_direct(kReverse ? live - 1 : c_lo, 0);
    fetch(kReverse ? live - 1 : c_lo, 0);
    if (wave == 0) weigh(kReverse ? live - 1 : c_lo, 0);
  }
  float u_acc = 0.0f, b_acc = 0.0f;           // threads 0..63 (kDots): sums over the query heads
  f32x4 O[4];
  const f32x4 zero = {0, 0, 0, 0};

  for (int it = 0; it < count; ++it) {
    const int step = it / nsub, sub = it % nsub, c = kReverse ? live - 1 - step : c_lo + step, t0 = c * kChunk;
    const auto& wt = lds_w[step & 1];
    const bool last_sub = sub == nsub - 1;
    const bool new_x = p.nq > 1 || sub == 0, new_yz = p.nkv > 1 || sub == 0;
    // between two walks of kWalk chunks: S goes to s_mid, or meets the one that is there
    const int ahead = c + (kReverse ? 1 : 0) - c_lo;          // the segment's chunks before the state in S
    const bool mark = kDots && p.s_mid && it > 0 && sub == 0 && ahead % kWalk == 0;
    if constexpr (kDots)
      if (mark) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const __amdgpu_buffer_rsrc_t mid = buffer_at(p.s_mid + ((size_t)blockIdx.x * (p.marks - 1) + ahead / kWalk - 1) * (DK * DV));
        const uint32_t off = (uint32_t)fresh(tid) * 16;
        f32x4 dot = {0, 0, 0, 0};
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
          if constexpr (kind == kDotQ)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[kt]), mid, off, kt * kThreads * 16, 0);
          else
            dot += S[kt] * __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(mid, off, kt * kThreads * 16, 0));
        if constexpr (kind == kDotK) share((dot[0] + dot[1]) + (dot[2] + dot[3]));
      }
    __syncthreads();
    if constexpr (kind == kDotK)
      if (mark && tid == 0) p.x_end[(size_t)blockIdx.x * p.marks + ahead / kWalk - 1] = shared();
    if constexpr (!kVec)
      if (new_x) {
        sx.store_permuted(lds_x);
        if constexpr (kDots) se.store_permuted(lds_e);
      }
    if (new_yz) {
      sy.store_keys(lds_y);
      sz.template store<PV>(lds_z);
    }
    const int next_sub = last_sub ? 0 : sub + 1, next_c = last_sub ? (kReverse ? c - 1 : c + 1) : c;
    if constexpr (kVec) {
      // this thread's loads to LDS have landed; after the barrier, everyone's
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_s_waitcnt(0x0F70);
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
    }
    __syncthreads();

    {
      // ---- scores: lane column i, four rows j a register block
      const int ln = fresh(lane), l15 = ln & 15, g4 = (ln >> 4) * 4;
      const int i = it0 * 16 + l15;
      float row = 0.0f;
      if (kReverse ? jt0 + JT > it0 : jt0 <= it0) {       // some of the wave's tiles may see their keys
        f32x4 P[JT], A[JT];
#pragma unroll
        for (int k = 0; k < DK / 32; ++k) {
          const Frag xf = TX::rows(lds_x, i, k, g4 / 4);
#pragma unroll
          for (int q = 0; q < JT; ++q) P[q] = M::mul(KY::rows(lds_y, (jt0 + q) * 16 + l15, k, g4 / 4), xf, k ? P[q] : zero);
        }
        if constexpr (kind == kDotQ) {
#pragma unroll
          for (int k = 0; k < DV / 32; ++k) {
            const Frag ef = TE::rows(lds_e, i, k, g4 / 4);
#pragma unroll
            for (int q = 0; q < JT; ++q) A[q] = M::mul(M::rows(lds_z + ((jt0 + q) * 16 + l15) * PV + k * 32 + g4 * 2), ef, k ? A[q] : zero);
          }
        }
        const float gi = wt.ghi[i], gi_lo = bf16_to_f32(wt.glo[i]);
#pragma unroll
        for (int q = 0; q < JT; ++q) {
          const int jt = jt0 + q, j0 = jt * 16 + g4;
          float s[4] = {0, 0, 0, 0};
          if (kReverse ? jt >= it0 : jt <= it0) {
            const float4 gh = *(const float4*)&wt.ghi[j0];
            const uint2 gl = *(const uint2*)&wt.glo[j0];
            const float ghv[4] = {gh.x, gh.y, gh.z, gh.w};
            const float glv[4] = {__uint_as_float(gl.x << 16), __uint_as_float(gl.x & 0xffff0000u),
                                  __uint_as_float(gl.y << 16), __uint_as_float(gl.y & 0xffff0000u)};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float d = (gi - ghv[r]) + (gi_lo - glv[r]);
              s[r] = P[q][r] * (__builtin_amdgcn_exp2f(d) * p.p_scale);
            }
            if (jt == it0)
#pragma unroll
              for (int r = 0; r < 4; ++r) s[r] = (kReverse ? j0 + r >= i : j0 + r <= i) ? s[r] : 0.0f;
            if constexpr (kind == kDotQ) {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float t = j0 + r < i ? s[r] * A[q][r] : 0.0f;
                row += t;
                const float cs = row16_sum(t);
                if (l15 == 0) lds_col[it0 * (it0 + 1) / 2 + jt][g4 + r] = cs;
              }
            }
          }
          SC::put(lds_p, it0, jt, l15, g4, s);
        }
        if constexpr (kind == kDotQ) row = group_sum(row);
      }
      // ---- what the state gives: O^T = S^T X^T
      if (new_x) {
#pragma unroll
        for (int k = 0; k < DK / 32; ++k) {
          float v[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = S[2 * k][r], v[4 + r] = S[2 * k + 1][r];
          const Split<kBf16, kParts> sf(v);
          constexpr int MG = kDots ? 2 : 4;     // row tiles at a time: with dot products there is room for two
#pragma unroll
          for (int m0 = 0; m0 < 4; m0 += MG) {
            Frag xf[MG];
#pragma unroll
            for (int m = 0; m < MG; ++m) xf[m] = TX::rows(lds_x, (m0 + m) * 16 + l15, k, g4 / 4);
            // the smallest part first; products into one accumulator stand apart
#pragma unroll
            for (int q = (kBf16 ? kParts : 1); q--;)
#pragma unroll
              for (int m = 0; m < MG; ++m) O[m0 + m] = M::mul(sf.part[q], xf[m], k || q + 1 < (kBf16 ? kParts : 1) ? O[m0 + m] : zero);
          }
        }
        float sum = 0.0f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int t = m * 16 + l15;
          O[m] *= __builtin_amdgcn_exp2f(wt.ghi[t]) * p.inter_scale;
          if constexpr (kDots) {
            float d = 0.0f;
            const Elt* er = lds_e + TE::at(t, (col0 + g4) / M::kPiece) + (col0 + g4) % M::kPiece;
#pragma unroll
            for (int r = 0; r < 4; ++r) d += O[m][r] * Elem<kBf16>::load(er + r);
            d = group_sum(d);
            sum += d;
            if constexpr (kind == kDotQ) d += m == it0 ? row : 0.0f;
            if (lane < 16) lds_dot[wave][t] = d;
          }
        }
        if constexpr (kind == kDotQ) {
          sum = row16_sum(sum);
          if (lane == 0) lds_bsum[wave] = sum;
        }
      }
      // the next tiles are on their way during the rest of the chunk (asked for any earlier, they
      // would share the registers with the products above and spill)
      __builtin_amdgcn_sched_barrier(0);
      if (it + 1 < count) fetch(next_c, next_sub);
      __syncthreads();
      if (it + 1 < count) fetch_direct(next_c, next_sub);
    }

    // ---- the wave's columns of Z, all 64 rows
    const int lane2 = fresh(lane), l15 = lane2 & 15, g4 = (lane2 >> 4) * 4;
    Frag zf[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) zf[k] = M::template cols<4>(lds_z, PV, k * 32, col0, lane2);

    {
      // zero times every value: a NaN where one of them is none or infinite
      const f32x4 odd = M::mul(zf[1], M::none(), M::mul(zf[0], M::none(), zero));
      const float sum = (odd[0] + odd[1]) + (odd[2] + odd[3]);
      if (__all(sum == sum)) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int part = SC::kParts; part--;)
#pragma unroll
            for (int m = 0; m < 4; ++m)
              if (kReverse ? (k == 1 || m < 2) : (k == 0 || m >= 2))
                O[m] = M::mul(zf[k], SC::rows(lds_p, part, m, k, lane2), O[m]);
      } else {
        // an infinity or a NaN among the values reaches only the outputs that may see its token:
        // a zero score times it would not be zero, so masked products are left out one by one
#pragma unroll 1
        for (int j = 0; j < kChunk; ++j) {
          float z[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) z[r] = Elem<kBf16>::load(lds_z + j * PV + col0 + g4 + r);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int i = m * 16 + l15;
            if (kReverse ? j >= i : j <= i) {
              const float s = SC::value(lds_p, i, j);
#pragma unroll
              for (int r = 0; r < 4; ++r) O[m][r] = fmaf(s, z[r], O[m][r]);
            }
          }
        }
      }
      if constexpr (kDots) {
        if (tid < kChunk) {
          if (new_x) {
            float d = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) d += lds_dot[w][tid];
            if constexpr (kind == kDotQ) {
              const int jt = tid >> 4;
#pragma unroll
              for (int w = 0; w < 4; ++w)
                if (w >= jt) d -= lds_col[w * (w + 1) / 2 + jt][tid & 15];
#pragma unroll
              for (int w = 0; w < kWaves; ++w) b_acc += lds_bsum[w];
            }
            u_acc += d;
          }
          if (last_sub) {
            if (t0 + tid < a.T) p.u[((size_t)b * a.Hkv + h) * a.T + t0 + tid] = u_acc;
            if (kind == kDotQ && tid == 0) p.b[((size_t)b * a.Hkv + h) * c_all + c] = b_acc;
            u_acc = b_acc = 0.0f;
          }
        }
      }
      if ((p.nq > 1 || last_sub) && p.o) {
        const int oh = h * p.nq + (p.nq > 1 ? sub : 0), pitch = a.Hkv * p.nq * p.dv;
        Elt* out = (Elt*)p.o + ((size_t)b * a.T + t0) * pitch + (size_t)oh * p.dv;
        const __amdgpu_buffer_rsrc_t rsrc = buffer_at(out);
        const int ln = fresh(lane2), l15 = ln & 15, g4 = (ln >> 4) * 4;
        const uint32_t off = (uint32_t)(l15 * pitch + col0 + g4) * (uint32_t)sizeof(Elt);
        if (t0 + kChunk > n)                    // tokens behind the row's end
#pragma unroll
          for (int m = 0; m < 4; ++m)
            if (t0 + m * 16 + l15 >= n) O[m] = f32x4{0, 0, 0, 0};
        const int cols = p.dv - (col0 + g4), rows = a.T - t0 - l15;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int left = m * 16 < rows ? cols : 0;
          if constexpr (kVec) {
            const uint32_t at = left > 0 ? off : kNowhere, step = (uint32_t)(m * 16 * pitch) * es;
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
            if constexpr (kBf16)
              __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(O[m][0], O[m][1]), pack_bf16(O[m][2], O[m][3])}, rsrc, at, step, 0);
            else
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[m]), rsrc, at, step, 0);
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (r < left) Elem<kBf16>::store(out + (m * 16 + l15) * pitch + col0 + g4 + r, O[m][r]);
          }
        }
      }
    }

    // ---- the state's update, once for each pair of keys and values
    if (p.nkv > 1 || last_sub) {
      if (p.nkv == 1 || sub == 0) {
        const float total = wt.total;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] *= total;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) add_outer<kBf16, DK, kDots ? 2 : 4>(S, zf[k], wt.upd + k * 32, lds_y, k, lane2);
    }
    // the next chunk's weights, where no other wave waits for them
    if (last_sub && it + 1 < count && wave == 0) weigh(next_c, ~step & 1);
  }

  // ---- chunks without tokens: zeros
  {
    for (int c = max(live, c_lo); c < c_hi; ++c) {
      const int t0 = c * kChunk, rows = min(kChunk, a.T - t0);
      if (p.o)
        for (int q = tid; q < rows * p.nq * p.dv; q += kThreads) {
          const int t = t0 + q / (p.nq * p.dv), j = q % (p.nq * p.dv);
          ((Elt*)p.o)[(((size_t)b * a.T + t) * a.Hkv + h) * p.nq * p.dv + j] = Elt(0);
        }
      if constexpr (kDots)
        for (int t = tid; t < rows; t += kThreads) p.u[((size_t)b * a.Hkv + h) * a.T + t0 + t] = 0.0f;
      if (kind == kDotQ && tid == 0) p.b[((size_t)b * a.Hkv + h) * c_all + c] = 0.0f;
    }
  }
  if (p.s_out)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (s_in_range(kt, r)) p.s_out[s_at(kt, r)] = S[kt][r];
  if constexpr (kind == kDotK) {
    if (p.x_first && seg == 0) {
      __syncthreads();
      dot_state(p.s_first - sbase + row * s_size);
      __syncthreads();
      if (tid == 0) p.x_first[row] = shared();
    }
  }
}

// The sum of a segment alone, from a zero state, and the segment's decay: chunk_kernel's update, 128
// tokens a step (64 in fp32), because keys and values in flight are what bounds it: 16 heads of 128 x 128
// over 32768 tokens in 76 us, 3.9 TB/s; 64 x 64 heads 22 us where 64 tokens a step took 25.
template <bool kBf16, int DK, int DV, bool kReverse, bool kVec>
__global__ void __launch_bounds__(DV * 4, kBf16 ? 4 : DV / 64) sum_kernel(RoleArgs p) {
  using M = Mma<kBf16>;
  using Elt = typename M::Elt;
  using Frag = typename M::Frag;
  constexpr int kWaves = DV / 16, kThreads = kWaves * 64, KT = DK / 16;
  constexpr int kHalves = kBf16 ? 2 : 1, kStep = kHalves * kChunk;
  constexpr int PV = DV + M::kPadZ;
  using KY = Keys<kBf16, DK>;
  using SY = Stage<kBf16, DK, kThreads>;
  using SZ = Stage<kBf16, DV, kThreads>;
  __shared__ alignas(16) Elt lds_y[kHalves * KY::kSize];
  __shared__ alignas(16) Elt lds_z[kStep * PV];
  __shared__ alignas(16) float lds_upd[2][kStep];       // the weights of y z^T, of this step and the next
  __shared__ float lds_total[2];

  const LinAttn& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l15 = lane & 15, g4 = (lane >> 4) * 4;
  const int seg = blockIdx.x % p.nseg;
  const int h = blockIdx.x / p.nseg % a.Hkv, b = blockIdx.x / p.nseg / a.Hkv;
  const int first = seg * p.seg_chunks * kChunk;        // the segment's tokens: first .. n - 1
  const int n = min(row_len(a.lens, b, a.T), first + p.seg_chunks * kChunk);
  if (n <= first) return;
  const int steps = (n - first + kStep - 1) / kStep, count = steps * p.nkv;
  const int col0 = wave * 16;
  f32x4 S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) S[kt] = f32x4{0, 0, 0, 0};

  SY sy[kHalves];
  SZ sz[kHalves];
  float g_next[kHalves];
  const uint32_t es = sizeof(Elt);
  const uint32_t off_y = kVec ? SY::offset((uint32_t)p.y.st * es, p.dk) : 0, off_z = kVec ? SZ::offset((uint32_t)p.z.st * es, p.dv) : 0;
  auto start = [&](int step) { return first + (kReverse ? steps - 1 - step : step) * kStep; };
  auto fetch = [&](int step, int sub) {
    const int t0 = start(step), hh = h * p.nkv + sub;
    if (sub == 0 && wave == 0)
#pragma unroll
      for (int u = 0; u < kHalves; ++u) {
        const int t = min(t0 + u * kChunk + lane, n - 1);
        g_next[u] = a.g[a.decay_token ? ((size_t)b * a.T + t) * a.Hkv + h : (size_t)h];
      }
    const Source<kBf16> y(p.y, b, hh), z(p.z, b, hh);
#pragma unroll
    for (int u = 0; u < kHalves; ++u) {
      sy[u].template load<kVec>(y, off_y, t0 + u * kChunk, n, p.dk);
      sz[u].template load<kVec>(z, off_z, t0 + u * kChunk, n, p.dv);
    }
  };
  double seg_log = 0.0;                       // wave 0: log2 of the segment's decay
  auto weigh = [&](int step) {
    double x[kHalves], end = 0.0;
#pragma unroll
    for (int u = 0; u < kHalves; ++u) {
      const float g = start(step) + u * kChunk + lane < n ? clamp_log_decay(g_next[u]) : 0.0f;
      x[u] = end + wave_scan((double)g * 1.4426950408889634);
      end = wave_last(x[u]);
    }
#pragma unroll
    for (int u = 0; u < kHalves; ++u)
      lds_upd[step & 1][u * kChunk + lane] = __builtin_amdgcn_exp2f((float)(kReverse ? x[u] : end - x[u])) * p.upd_scale;
    if (lane == 0) lds_total[step & 1] = __builtin_amdgcn_exp2f((float)end);
    seg_log += end;
  };
  fetch(0, 0);
  if (wave == 0) weigh(0);
  for (int it = 0; it < count; ++it) {
    const int step = it / p.nkv, sub = it % p.nkv;
    const bool last_sub = sub == p.nkv - 1;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kHalves; ++u) {
      sy[u].store_keys(lds_y + u * KY::kSize);
      sz[u].template store<PV>(lds_z + u * kChunk * PV);
    }
    if (it + 1 < count) fetch(last_sub ? step + 1 : step, last_sub ? 0 : sub + 1);
    __syncthreads();
    if (sub == 0) {
      const float total = lds_total[step & 1];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) S[kt] *= total;
    }
    const int ln = fresh(lane);
#pragma unroll
    for (int k = 0; k < kStep / 32; ++k) {
      const Frag zf = M::template cols<4>(lds_z, PV, k * 32, col0, ln);
      add_outer<kBf16, DK, 4>(S, zf, lds_upd[step & 1] + k * 32, lds_y + k / 2 * KY::kSize, k % 2, ln);
    }
    // the next step's weights, where no other wave waits for them
    if (last_sub && it + 1 < count && wave == 0) weigh(step + 1);
  }
  const size_t base = (size_t)blockIdx.x * p.dk * p.dv;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = state_row(kt, g4) + r, j = col0 + l15;
      if (i < p.dk && j < p.dv) p.s_out[base + (size_t)i * p.dv + j] = S[kt][r];
    }
  if (tid == 0) p.seg_decay[blockIdx.x] = __builtin_amdgcn_exp2f((float)seg_log);
}

// The narrowest tiles that hold the head sizes, 64 or 128 columns, for the call's types.
template <class F>
hipError_t with_tiles(const RoleArgs& p, F f) {
  using std::integral_constant;
  auto sizes = [&](auto bf, auto vec) {
    if (p.dk > 64)
      return p.dv > 64 ? f(bf, vec, integral_constant<int, 128>{}, integral_constant<int, 128>{})
                       : f(bf, vec, integral_constant<int, 128>{}, integral_constant<int, 64>{});
    return p.dv > 64 ? f(bf, vec, integral_constant<int, 64>{}, integral_constant<int, 128>{})
                     : f(bf, vec, integral_constant<int, 64>{}, integral_constant<int, 64>{});
  };
  const std::true_type yes;
  const std::false_type no;
  if (p.a.bf16) return p.vec ? sizes(yes, yes) : sizes(yes, no);
  return p.vec ? sizes(no, yes) : sizes(no, no);
}

template <bool kReverse, Kind kind>
hipError_t run_role(const RoleArgs& p, hipStream_t st) {
  return with_tiles(p, [&](auto bf, auto vec, auto dk, auto dv) {
    constexpr int DV = decltype(dv)::value;
    chunk_kernel<decltype(bf)::value, decltype(dk)::value, DV, kReverse, kind, decltype(vec)::value>
        <<<(unsigned)p.a.B * p.a.Hkv * p.nseg, DV * 4, 0, st>>>(p);
    return hipGetLastError();
  });
}

template <bool kReverse>
hipError_t run_sum(const RoleArgs& p, hipStream_t st) {
  return with_tiles(p, [&](auto bf, auto vec, auto dk, auto dv) {
    constexpr int DV = decltype(dv)::value;
    sum_kernel<decltype(bf)::value, decltype(dk)::value, DV, kReverse, decltype(vec)::value>
        <<<(unsigned)p.a.B * p.a.Hkv * p.nseg, DV * 4, 0, st>>>(p);
    return hipGetLastError();
  });
}

inline bool rows_vec(const Rows& r, int cols, int bf16) {
  const int e = bf16 ? 8 : 4;
  return cols % e == 0 && r.sb % e == 0 && r.st % e == 0 && r.sh % e == 0 && (uintptr_t)r.p % 16 == 0 &&
         r.st < (1 << 22);
}

// ---- segments ------------------------------------------------------------------------------
struct Plan {
  int seg_chunks, nseg;
  size_t states;       // bytes of the segments' states
};

// Few rows and a long axis: the axis is cut into segments that run side by side, at the price of
// one more pass over the keys and values for the segments' own sums, and of the recurrence
// over the segments.  As many segments as fill the device (256 CUs, two blocks each of the widest
// bf16 tiles, one of fp32's), from the length on where that pays; one head's pass of 128 x 128 in us,
// whole | cut:
//            forward    bf16        fp32         backward   bf16         fp32
//   128 tokens       15 | 19     33 | 30                   65 | 71    120 | 103
//   192              19 | 19     46 | 30                   84 | 71    166 | 103
//   320              28 | 19     73 | 30                  122 | 72    259 | 104
//   4096            288 | 27    862 | 39                 1235 | 86   2988 | 118
// The other end, rows of 2048 tokens:
//            forward    bf16 128   bf16 64    fp32 128     backward   bf16 128   bf16 64    fp32 128
//   64 rows         152 | 79   115 | 41   442 | 179              653 | 271   508 | 136  1561 | 574
//   128             152 | 126  116 | 64   446 | 339              667 | 453   509 | 221  1573 | 1052
//   160             155 | 160  116 | 80                          672 | 552   513 | 286
//   192             159 | 206  116 | 104                         681 | 706   516 | 383
//   256             168 | 248  117 | 111                         706 | 818   518 | 416
// so from about 160 rows of wide bf16 heads on the rule cuts where the whole axis would be the faster.
inline Plan make_plan(const LinAttn& a, bool backward) {
  const int chunks = (a.T + kChunk - 1) / kChunk;
  const int64_t rows = (int64_t)a.B * a.Hkv;
  Plan p{chunks > 0 ? chunks : 1, 1, 0};
  const int64_t want = (a.bf16 ? 512 : 256) / rows;
  if (want >= 2 && chunks >= (backward || !a.bf16 ? 3 : 5)) {
    p.seg_chunks = (int)((chunks + want - 1) / want);
    p.nseg = (chunks + p.seg_chunks - 1) / p.seg_chunks;
  }
  p.states = ((size_t)rows * p.nseg * a.Dk * a.Dv * 4 + 255) / 256 * 256;
  return p;
}

// In place over the segments' own sums: entry states, and the last exit state.  `reverse` runs from
// the last segment to the first.  A row's segments without tokens are left alone.
struct ScanArgs {
  LinAttn a;
  int seg_chunks;
  float* seg;              // [rows][nseg][size]
  const float* decay;      // [rows][nseg]
  const float* s_in;       // [rows][size] or nullptr
  float* s_out;            // [rows][size] or nullptr
  int nseg, size, reverse;
};
hipError_t launch_scan(const ScanArgs* p, int count, int64_t rows, hipStream_t st);

}  // namespace linattn
}  // namespace pnr
