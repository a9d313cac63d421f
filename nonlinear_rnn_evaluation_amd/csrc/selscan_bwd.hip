// Gradients of the selective scan.  With gy = grad_y silu(z) and g_t = gy_t C_t + a_{t+1} g_{t+1}
// the gradient of h_t (a_t = exp(delta_t A)):
//   dC_t = sum_e gy h_t          dB_t = sum_e g delta u        q = sum_n g B_t
//   du = D gy + delta q          ddelta = u q + sum_n g a h_{t-1} A
//   dA = sum_t g a h_{t-1} delta      dD = sum_t gy u          dh_0 = a_1 g_1
//
// Keeping every state would cost 4 N bytes a channel and token, many times what the call reads, so
// they are made again, from coarse to fine:
//   local_kernel   a segment forwards from zeros: its state every 16 tokens (a chunk), and where time is
//                  cut the segment's sums for the recurrences of h and of g
//   join_kernel    those recurrences over a row's segments
//   walk_kernel    a segment's chunks, last to first: the chunk forwards once for the states
//                  every four tokens (LDS), each four forwards again with all states and
//                  decays in registers, and back through them
//   sum_kernel     what is summed over blocks
// Instruction issue bounds it: 10 slots a state and token before the walk, 24 in it (4.5 and 4.5 of them
// make states again).  bf16, 4 x 4096 tokens of 4096 channels x 16 states: 388, 15, 924 and 33 us.
// States every 8 tokens instead of 16 cost the walk 1290 us where 1030: each chunk starts with waits.
#include <algorithm>
#include <cmath>

#include "selscan_tile.h"

namespace pnr {
namespace {

using namespace selscan;

constexpr int R = 4;               // states of a channel in a lane: 16 in a wave
constexpr int kChannels = 64;      // of a wave
constexpr int kChunk = 16, kFour = 4;

// A wave owns 64 channels, one a lane, and 16 of their states: lane l holds, for four channels, the four
// states that start at 4 (l / 4 % 4).  Its slot r belongs to the channel of the lane 4 r places away in
// its row of 16, so that
//   - what a channel needs once a token is computed by one lane, and a rotation of the row brings it to
//     the three others that hold the rest of its states;
//   - a sum over a channel's states is one rotation and one addition a slot, and ends in the lane
//     that owns the channel;
//   - a sum over channels (dB, dC) starts from four of them in a lane: 22 slots a token for 16 states
//     of 64 channels.  With a channel a lane in a quad, as forwards, it would be four times that.

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

// A token of the recurrence: h = exp2(d A) h + x B in each of four slots, B of this lane's states at
// p (LDS).  x B is an outer product of the channels of four neighbouring lanes and four states, which
// one matrix instruction adds to the decayed states: B's four values come from the four lanes, x
// from each.  It is exact as a fused multiplication and addition is.
__device__ __forceinline__ void advance(float (&h)[4][R], const float (&A)[4][R], const float (&d)[4], const float (&x)[4],
                                        const float* p, int lane) {
  const float b = p[lane & 3];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    f32x4 v;
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = h[r][i] * __builtin_amdgcn_exp2f(d[r] * A[r][i]);
    v = __builtin_amdgcn_mfma_f32_4x4x1f32(b, x[r], v, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < R; ++i) h[r][i] = v[i];
  }
}

struct BwdArgs {
  SelScan a;
  SelScanGrads d;
  const float* s_in;
  Segments seg;
  int tiles, per_group;            // of 64 channels: in all, a group
  int NB, chunks;                  // blocks of 16 states; chunks of a row
  float *states, *reach;           // [B, chunks, E, 16 NB] and [B, chunks, E]: from the segment's start to the chunk's
  float *hs, *gs, *width;          // [B, S, E, 16 NB] twice, [B, S, E]
  float *part, *pA, *pD, *pb;      // [B, T, tiles, 2, 16 NB]; [B S, E, N], [B S, E], [B S, E]
};

// Where a wave works: row b, group g, its first channel e0 (of E) and how many of 64 it has.
struct Tile {
  int b, g, e0, live;
};

// What a wave knows of its place: the tile, its states and its lanes' channels.
struct Place {
  Tile w;
  int seg, lane, nq, e, n0;        // n0: this lane's first state
  int ch[4], off[4];               // the slots' channels (-1: none), and their states' offsets
  bool live;
};

template <int NB>
__device__ __forceinline__ Place place(const BwdArgs& p) {
  Place x;
  const int64_t per_seg = (int64_t)p.a.B * p.tiles;
  x.seg = (int)(blockIdx.x / per_seg);
  const int64_t i = blockIdx.x % per_seg;
  const int W = p.a.E / p.a.G, first = (int)(i % p.per_group) * kChannels;
  x.w.g = (int)(i / p.per_group % p.a.G), x.w.b = (int)(i / p.tiles);
  x.w.e0 = x.w.g * W + first, x.w.live = min(W - first, kChannels);
  x.lane = threadIdx.x & 63, x.nq = x.lane >> 2 & 3;
  x.live = x.lane < x.w.live;
  x.e = x.w.e0 + min(x.lane, x.w.live - 1);
  x.n0 = (NB > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 16 : 0) + x.nq * R;
  x.ch[0] = x.live ? x.e : -1, x.ch[1] = away<1>(x.ch[0]), x.ch[2] = away<2>(x.ch[0]), x.ch[3] = away<3>(x.ch[0]);
#pragma unroll
  for (int r = 0; r < 4; ++r) x.off[r] = x.ch[r] >= 0 ? (x.ch[r] * (16 * NB) + x.n0) * 4 : kNowhere;
  return x;
}

// A of a state that only fills a block of 16: decays are 1, and 0 at an infinite width, where 0 would make them
// NaN and the channel's sums with them.
constexpr float kNoState = -1.17549435e-38f;

__device__ __forceinline__ void load_A(const SelScan& a, const Place& x, float (&A)[4][R]) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < R; ++i) A[r][i] = x.ch[r] >= 0 && x.n0 + i < a.N ? exponent(a.A[(size_t)x.ch[r] * a.N + x.n0 + i]) : kNoState;
}

// Four states of each slot from, or to, [.., E, 16 NB] at row `row` of E channels.  A slot without a channel
// reads zeros and writes nowhere.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load_states(const float* p, size_t row, const BwdArgs& q, const Place& x, f32x4 (&h)[4]) {
  const __amdgpu_buffer_rsrc_t from = buffer_of(p + row * q.a.E * (16 * q.NB), true);
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = __builtin_bit_cast(f32x4, (u32x4)__builtin_amdgcn_raw_buffer_load_b128(from, x.off[r], 0, 0));
}
__device__ __forceinline__ void store_states(float* p, size_t row, const BwdArgs& q, const Place& x, const float (&h)[4][R]) {
  const __amdgpu_buffer_rsrc_t to = buffer_of(p + row * q.a.E * (16 * q.NB), true);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{h[r][0], h[r][1], h[r][2], h[r][3]}), to, x.off[r], 0, 0);
}

// B and C of a chunk, this wave's 16 states: [token][B, C][16], zeros beyond `end` and the states.  A lane
// takes every second token's B or C of one state; what is not there is read elsewhere and dropped.
template <bool kBf16>
struct Chunk {
  using El = Elem<kBf16>;
  using T = typename El::type;
  static constexpr int kEach = kChunk * 32 / 64;
  T raw[kEach];
  const T* from;
  int64_t st;
  int half;
  bool state;
  __device__ __forceinline__ void start(const SelScan& a, const Place& x) {
    const int n = (x.n0 & ~15) + (x.lane & 15);
    const Rows& r = x.lane >> 4 & 1 ? a.Ct : a.Bt;
    state = n < a.N;
    from = (const T*)r.p + x.w.b * r.sb + x.w.g * r.sh + (state ? n : 0);
    st = r.st, half = x.lane >> 5;
  }
  __device__ __forceinline__ void fetch(int t, int end) {       // end: of the row's segment, behind t
#pragma unroll
    for (int k = 0; k < kEach; ++k) raw[k] = from[min(t + 2 * k + half, end - 1) * st];
  }
  __device__ __forceinline__ void put(float* lds, int lane, int t, int end) const {
#pragma unroll
    for (int k = 0; k < kEach; ++k) lds[k * 64 + lane] = state && t + 2 * k + half < end ? El::load(&raw[k]) : 0.0f;
  }
};

// A [B, T, E] operand, by the lanes that own its channels: a buffer from a chunk's first token on, tokens as
// 32-bit offsets (the entry points keep wide strides away).  Lanes without a channel read zeros.
template <bool kBf16>
struct Operand {
  using T = typename Elem<kBf16>::type;
  const T* row;
  int64_t st;
  int off;
  bool given;
  __amdgpu_buffer_rsrc_t buf;
  __device__ __forceinline__ Operand(const void* p, int64_t sb, int64_t stride, const Place& x)
      : row((const T*)p + (p ? x.w.b * sb : 0)), st(stride), off(x.live ? x.e * (int)sizeof(T) : kNowhere), given(p) {}
  __device__ __forceinline__ void rebase(int t) { buf = buffer_of(row + (given ? t * st : 0), given); }
  __device__ __forceinline__ T get(int k) const { return load_buffer<T>(buf, off, k * (int)st * (int)sizeof(T)); }
  __device__ __forceinline__ void set(int k, bool there, float v) const {
    store_buffer<kBf16>(v, buf, there ? off : kNowhere, k * (int)st * (int)sizeof(T));
  }
};

template <bool kBf16, int NB, bool kCut>
__global__ void __launch_bounds__(NB * 64, 2) local_kernel(BwdArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  __shared__ alignas(16) float bc_all[NB][2][kChunk * 32];
  const SelScan& a = p.a;
  const Place x = place<NB>(p);
  const int n = row_len(a.lens, x.w.b, a.T), t0 = x.seg * p.seg.len, t1 = min(t0 + p.seg.len, n);
  if (t0 >= t1) return;
  const int sb = NB > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  float(*bc)[kChunk * 32] = bc_all[sb];
  float A[4][R], h[4][R] = {}, P[4][R], G[4][R] = {};
  load_A(a, x, A);
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < R; ++i) P[r][i] = 1.0f;
  const float bias = a.bias ? a.bias[x.e] : 0.0f;
  Operand<kBf16> u(a.u.p, a.u.sb, a.u.st, x), dt(a.dt.p, a.dt.sb, a.dt.st, x), z(kCut ? a.z.p : nullptr, a.z.sb, a.z.st, x),
      gy(p.d.gy, (int64_t)a.T * a.E, a.E, x);
  T ur[kFour], dr[kFour], zr[kFour], gr[kFour];
  int end = 0;                                   // of the row's segment, from the chunk's start
  auto fetch = [&](int k0) {                     // a token behind the end is the last one again
#pragma unroll
    for (int k = 0; k < kFour; ++k) {
      const int at = min(k0 + k, end - 1);
      ur[k] = u.get(at), dr[k] = dt.get(at);
      if (kCut) zr[k] = z.get(at), gr[k] = gy.get(at);
    }
  };
  auto rebase = [&](int t) {
    u.rebase(t), dt.rebase(t), end = t1 - t;
    if (kCut) z.rebase(t), gy.rebase(t);
  };
  float total = 0.0f;
  Chunk<kBf16> stage;
  stage.start(a, x);
  stage.fetch(t0, t1);
  rebase(t0);
  fetch(0);
  int buf = 0;
  for (int t = t0; t < t1; t += kChunk, buf ^= 1) {
    stage.put(bc[buf], x.lane, t, t1);
    const size_t row = (size_t)x.w.b * p.chunks + t / kChunk;
    if (t > t0) {
      store_states(p.states, row, p, x, h);
      if (sb == 0 && x.live) p.reach[row * a.E + x.e] = total;
    }
    if (!kCut && t + kChunk >= t1) break;        // the last chunk's end is nobody's start
    stage.fetch(min(t + kChunk, t1 - 1), t1);
    __builtin_amdgcn_wave_barrier();             // a wave reads what it staged itself
    for (int f = 0; f < kChunk && t + f < t1; f += kFour) {
      const int left = t1 - t - f;
      float uv[kFour], dv[kFour], zv[kFour], gv[kFour];
#pragma unroll
      for (int k = 0; k < kFour; ++k) {
        uv[k] = El::load(&ur[k]), dv[k] = El::load(&dr[k]);
        if (kCut) zv[k] = El::load(&zr[k]), gv[k] = El::load(&gr[k]);
      }
      if (f + kFour == kChunk) {
        rebase(min(t + kChunk, t1 - 1));
        fetch(0);
      } else {
        fetch(f + kFour);
      }
#pragma unroll
      for (int k = 0; k < kFour; ++k) {
        const bool there = k < left;
        const float delta = step_width(dv[k] + bias, a.softplus, x.live && there);
        total += delta;
        float d[4], s[4], g[4];
        to_slots(delta, d);
        to_slots(there ? delta * uv[k] : 0.0f, s);
        if (kCut) to_slots(there ? gv[k] * gate_of(zv[k], a.z.p) : 0.0f, g);
        const float* at = bc[buf] + (f + k) * 32 + x.nq * R + (x.lane & 3);
        const float b = at[0], c = at[16];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f32x4 v, w{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float dec = __builtin_amdgcn_exp2f(d[r] * A[r][i]);
            v[i] = h[r][i] * dec;
            P[r][i] *= dec;
          }
          v = __builtin_amdgcn_mfma_f32_4x4x1f32(b, s[r], v, 0, 0, 0);
          if (kCut) w = __builtin_amdgcn_mfma_f32_4x4x1f32(c, g[r], w, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            h[r][i] = v[i];
            if (kCut) {
              G[r][i] = fmaf(P[r][i], w[i], G[r][i]);
              asm volatile("" : "+v"(G[r][i]));     // here, not behind the loop's branches with all its factors waiting
            }
          }
        }
      }
    }
  }
  if (!kCut) return;
  const size_t row = (size_t)x.w.b * p.seg.S + x.seg;
  store_states(p.hs, row, p, x, h);
  store_states(p.gs, row, p, x, G);
  if (sb == 0 && x.live) p.width[row * a.E + x.e] = total;
}

// The recurrences over a row's segments: in place of a segment's sums its first state, and the gradient
// that reaches its last state from behind.  A thread a state; eight segments of each are asked for at once.
__device__ __forceinline__ void join_state(const BwdArgs& p, int s, int e, int b, int NP) {
  constexpr int kBatch = 8;
  const SelScan& a = p.a;
  const int n = row_len(a.lens, b, a.T), segs = (int)(((int64_t)n + p.seg.len - 1) / p.seg.len);
  const bool real = s < a.N;
  const float A = real ? exponent(a.A[(size_t)e * a.N + s]) : kNoState;
  const size_t at = ((size_t)b * a.E + e) * a.N + s, row = (size_t)b * p.seg.S * a.E + e;
  float h = real && p.s_in ? p.s_in[at] : 0.0f, g = real && p.d.gstate_out ? p.d.gstate_out[at] : 0.0f;
  if (p.seg.S > 1) {
    for (int k0 = 0; k0 < segs; k0 += kBatch) {      // h from the first segment on, g from the last
      float own[2][kBatch], d[2][kBatch];
      size_t r[2][kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int j = min(k0 + k, segs - 1);
        r[0][k] = row + (size_t)j * a.E, r[1][k] = row + (size_t)(segs - 1 - j) * a.E;
        own[0][k] = p.hs[r[0][k] * NP + s], d[0][k] = p.width[r[0][k]];
        own[1][k] = p.gs[r[1][k] * NP + s], d[1][k] = p.width[r[1][k]];
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < segs) {
          p.hs[r[0][k] * NP + s] = h;
          h = carried(h, d[0][k] * A, factor(d[0][k] * A), own[0][k]);
          p.gs[r[1][k] * NP + s] = g;
          g = carried(g, d[1][k] * A, factor(d[1][k] * A), own[1][k]);
        }
    }
    if (real && p.d.gstate_in) p.d.gstate_in[at] = g;
  } else {                                        // one segment: its walk goes on to the first state
    p.hs[row * NP + s] = h;
    p.gs[row * NP + s] = g;
    if (real && p.d.gstate_in && segs == 0) p.d.gstate_in[at] = g;
  }
}

__global__ void __launch_bounds__(256) join_kernel(BwdArgs p) {
  const int NP = 16 * p.NB, E = p.a.E;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < (int64_t)p.a.B * E * NP; i += (int64_t)gridDim.x * 256)
    join_state(p, (int)(i % NP), (int)(i / NP % E), (int)(i / NP / E), NP);
}

// Sums of dB and dC over the wave's channels (lane bits 0, 1, 4 and 5): the halves of the wave take one
// each, then rows of 16 and neighbouring lanes two states each.  Lane l ends with state
// 4 (l / 4 % 4) + (l / 16 % 2) + 2 (l % 2) of dB (l < 32) or dC.
__device__ __forceinline__ float over_channels(const float (&b)[R], const float (&c)[R], int lane) {
  float v[R], y[2];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(b[i]), __float_as_uint(c[i]), false, false);
    v[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), false, false);
    y[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  const bool odd = lane & 1;
  float o = (odd ? y[1] : y[0]) + quad_perm<0xb1>(odd ? y[0] : y[1]);
  o += quad_perm<0x4e>(o);
  return o;
}

template <bool kBf16, int NB>
__global__ void __launch_bounds__(NB * 64, 2) walk_kernel(BwdArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  constexpr int kFours = kChunk / kFour;
  __shared__ alignas(16) float bc_all[NB][kChunk * 32];
  __shared__ f32x4 mid_all[NB][kFours][4][64];
  __shared__ float sums[NB > 1 ? 2 : 1][NB > 1 ? NB : 1][3][NB > 1 ? kFour : 1][64];
  const SelScan& a = p.a;
  const SelScanGrads& d = p.d;
  const Place x = place<NB>(p);
  const int n = row_len(a.lens, x.w.b, a.T), t0 = x.seg * p.seg.len, tend = min(t0 + p.seg.len, a.T), t1 = min(tend, n);
  const int sb = NB > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  float* bc = bc_all[sb];
  auto& mid = mid_all[sb];
  const size_t seg_row = (size_t)x.w.b * p.seg.S + x.seg;
  T* gu = d.gu ? (T*)d.gu + (size_t)x.w.b * a.T * a.E : nullptr;
  T* gdt = d.gdt ? (T*)d.gdt + (size_t)x.w.b * a.T * a.E : nullptr;
  T* gz = d.gz ? (T*)d.gz + (size_t)x.w.b * a.T * a.E : nullptr;
  if (sb == 0 && x.live)
    for (int t = max(t0, t1); t < tend; ++t) {
      if (gu) El::store(gu + (size_t)t * a.E + x.e, 0.0f);
      if (gdt) El::store(gdt + (size_t)t * a.E + x.e, 0.0f);
      if (gz) El::store(gz + (size_t)t * a.E + x.e, 0.0f);
    }
  float A[4][R], g[4][R], dA[4][R] = {};
  float dD = 0.0f, db = 0.0f;
  if (t0 < t1) {
    load_A(a, x, A);
    f32x4 back[4];
    load_states(p.gs, seg_row, p, x, back);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < R; ++i) g[r][i] = back[r][i];
    const float bias = a.bias ? a.bias[x.e] : 0.0f, D = a.D ? a.D[x.e] : 0.0f;
    Operand<kBf16> u(a.u.p, a.u.sb, a.u.st, x), dt(a.dt.p, a.dt.sb, a.dt.st, x), z(a.z.p, a.z.sb, a.z.st, x),
        gy(d.gy, (int64_t)a.T * a.E, a.E, x), ou(d.gu, (int64_t)a.T * a.E, a.E, x), od(d.gdt, (int64_t)a.T * a.E, a.E, x),
        oz(d.gz, (int64_t)a.T * a.E, a.E, x);
    const bool gated = a.z.p;
    float* part = p.part + (((size_t)x.w.b * a.T) * p.tiles + x.w.g * p.per_group + (x.w.e0 - x.w.g * (a.E / a.G)) / kChannels) * 32 * NB;
    const int part_at = (x.lane & 2) ? kNowhere
                                     : ((x.lane >> 5) * 16 * NB + sb * 16 + x.nq * 4 + (x.lane >> 4 & 1) + 2 * (x.lane & 1)) * 4;
    const float* reach = p.reach + x.e;
    int turn = 0;
    T ur[kFour], dr[kFour], zr[kFour], gr[kFour];
    auto fetch = [&](int k0, int end) {          // a token behind the end is the last one again
#pragma unroll
      for (int k = 0; k < kFour; ++k) {
        const int at = min(k0 + k, end - 1);
        ur[k] = u.get(at), dr[k] = dt.get(at), zr[k] = z.get(at), gr[k] = gy.get(at);
      }
    };
    T us[kFour], ds[kFour];
    auto fetch_ahead = [&](int k0, int end) {
#pragma unroll
      for (int k = 0; k < kFour; ++k) us[k] = u.get(min(k0 + k, end - 1)), ds[k] = dt.get(min(k0 + k, end - 1));
    };
    auto begin = [&](int c, f32x4 (&own)[4], f32x4 (&entry)[4], float& added) {     // what a chunk starts from
      const int tc = t0 + c * kChunk, end = min(kChunk, t1 - tc);
      u.rebase(tc), dt.rebase(tc), z.rebase(tc), gy.rebase(tc);
      load_states(p.hs, seg_row, p, x, entry);
      const size_t row = (size_t)x.w.b * p.chunks + tc / kChunk;
      load_states(p.states, row, p, x, own);
      added = reach[row * a.E];
      fetch((end - 1) / kFour * kFour, end);
      fetch_ahead(0, end);
    };
    Chunk<kBf16> stage;
    const int last = (t1 - 1 - t0) / kChunk;
    stage.start(a, x);
    stage.fetch(t0 + last * kChunk, t1);
    for (int c = last; c >= 0; --c) {
      const int tc = t0 + c * kChunk, end = min(kChunk, t1 - tc), fours = (end + kFour - 1) / kFour;
      ou.rebase(tc), od.rebase(tc), oz.rebase(tc);
      const __amdgpu_buffer_rsrc_t out_part = buffer_of(part + (size_t)tc * p.tiles * 32 * NB, true);
      const int part_step = p.tiles * 32 * NB * 4;
      // the state at the chunk's start: the segment's, decayed, and what the segment added (the first chunk's
      // place in `states` and `reach` holds nothing)
      f32x4 own[4], entry[4];
      float h[4][R], w[4], added;
      begin(c, own, entry, added);
      to_slots(x.live && c > 0 ? added : 0.0f, w);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < R; ++i)
          h[r][i] = fmaf(entry[r][i], __builtin_amdgcn_exp2f(w[r] * A[r][i]), c > 0 ? own[r][i] : 0.0f);
      stage.put(bc, x.lane, tc, t1);
      if (c > 0) stage.fetch(tc - kChunk, t1);
      __builtin_amdgcn_wave_barrier();
      const float* lane_bc = bc + x.nq * R;
      auto keep = [&](int f) {
#pragma unroll
        for (int r = 0; r < 4; ++r) mid[f][r][x.lane] = f32x4{h[r][0], h[r][1], h[r][2], h[r][3]};
      };
      keep(0);
      // the states at each four's start
#pragma unroll 1
      for (int f = 0; f < fours - 1; ++f) {
        float uv[kFour], dv[kFour];
#pragma unroll
        for (int k = 0; k < kFour; ++k) uv[k] = El::load(&us[k]), dv[k] = El::load(&ds[k]);
        fetch_ahead((f + 1) * kFour, end);
#pragma unroll
        for (int k = 0; k < kFour; ++k) {
          const float delta = step_width(dv[k] + bias, a.softplus, x.live);
          float dl[4], s[4];
          to_slots(delta, dl);
          to_slots(delta * uv[k], s);
          advance(h, A, dl, s, lane_bc + (f * kFour + k) * 32, x.lane);
        }
        keep(f + 1);
      }
#pragma unroll 1
      for (int f = fours - 1; f >= 0; --f) {
        const int k0 = f * kFour;
        float uv[kFour], raw[kFour], zv[kFour], gv[kFour], delta[kFour];
#pragma unroll
        for (int k = 0; k < kFour; ++k) {
          const bool there = k0 + k < end;
          uv[k] = there ? El::load(&ur[k]) : 0.0f, raw[k] = El::load(&dr[k]) + bias, zv[k] = El::load(&zr[k]);
          gv[k] = there ? El::load(&gr[k]) : 0.0f, delta[k] = step_width(raw[k], a.softplus, x.live && there);
        }
        // forwards: states before each token, and decays
        float hist[kFour + 1][4][R], dec[kFour][4][R];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4 v = mid[f][r][x.lane];
#pragma unroll
          for (int i = 0; i < R; ++i) hist[0][r][i] = v[i];
        }
#pragma unroll
        for (int k = 0; k < kFour; ++k) {
          float dl[4], s[4];
          to_slots(delta[k], dl);
          to_slots(delta[k] * uv[k], s);
          const float b = lane_bc[(k0 + k) * 32 + (x.lane & 3)];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            f32x4 v;
#pragma unroll
            for (int i = 0; i < R; ++i) {
              dec[k][r][i] = __builtin_amdgcn_exp2f(dl[r] * A[r][i]);
              v[i] = hist[k][r][i] * dec[k][r][i];
            }
            v = __builtin_amdgcn_mfma_f32_4x4x1f32(b, s[r], v, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < R; ++i) hist[k + 1][r][i] = v[i];
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        // and back
        float ys[kFour], qs[kFour], ws[kFour];
        auto finish = [&](int k) {                // a token's gradients, from the sums over all states
          const bool there = k0 + k < end;
          const float sg = sigm(zv[k]), gated_gy = gated ? gv[k] * (zv[k] * sg) : gv[k];
          const float y = fmaf(D, uv[k], ys[k]), gd = fmaf(uv[k], qs[k], kLn2 * ws[k]);
          float slope = sigm(raw[k]);
          asm volatile("" : "+v"(slope));         // no branch between tokens
          const float gt = a.softplus ? gd * slope : gd;
          dD = fmaf(gated_gy, uv[k], dD);
          db += there ? gt : 0.0f;
          ou.set(k0 + k, there, fmaf(D, gated_gy, delta[k] * qs[k]));
          od.set(k0 + k, there, gt);
          oz.set(k0 + k, there, gv[k] * (sg * (1.0f + zv[k] * (1.0f - sg))) * y);   // a closed gate before anything large
        };
#pragma unroll
        for (int k = kFour - 1; k >= 0; --k) {
          const float* s = lane_bc + (k0 + k) * 32;
          float Bv[R], Cv[R], dl[4], xs[4], gs[4], ya[4], qa[4], wa[4], dB[R] = {}, dC[R] = {};
          read_states<R>(s, Bv);
          read_states<R>(s + 16, Cv);
          const float cl = s[16 + (x.lane & 3)];
          to_slots(delta[k], dl);
          to_slots(delta[k] * uv[k], xs);
          to_slots(gv[k] * gate_of(zv[k], gated), gs);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            f32x4 v{g[r][0], g[r][1], g[r][2], g[r][3]};
            v = __builtin_amdgcn_mfma_f32_4x4x1f32(cl, gs[r], v, 0, 0, 0);
            ya[r] = qa[r] = wa[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < R; ++i) g[r][i] = v[i];
          }
          if (k == 0) {                            // the four's first states, read again
            asm volatile("" ::: "memory");
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const f32x4 v = mid[f][r][x.lane];
#pragma unroll
              for (int i = 0; i < R; ++i) hist[0][r][i] = v[i];
            }
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const float hn = hist[k + 1][r][i], gn = g[r][i];
              ya[r] = fmaf(hn, Cv[i], ya[r]);
              dC[i] = fmaf(gs[r], hn, dC[i]);
              dB[i] = fmaf(xs[r], gn, dB[i]);
              qa[r] = fmaf(gn, Bv[i], qa[r]);
              g[r][i] = gn * dec[k][r][i];
              const float through = g[r][i] * hist[k][r][i];
              wa[r] = fmaf(through, A[r][i], wa[r]);
              dA[r][i] = fmaf(through, dl[r], dA[r][i]);
              asm volatile("" : "+v"(dA[r][i]));    // here, not behind the loop's branches, where 64 products wait for it
            }
          }
          if (k > 0 && k0 + k >= end) {            // behind the row's end, where the walk begins: a width of 0 times a
#pragma unroll                                     // state that need not be finite
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int i = 0; i < R; ++i) {
                dA[r][i] = 0.0f;
                asm volatile("" : "+v"(dA[r][i]));  // a branch: as selections the walk took 1.1 times as long
              }
          }
          ys[k] = from_slots(ya), qs[k] = from_slots(qa), ws[k] = from_slots(wa);
          const float o = over_channels(dB, dC, x.lane);
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o), out_part, k0 + k < end ? part_at : kNowhere, (k0 + k) * part_step, 0);
          if constexpr (NB == 1) finish(k);
          if (k == 1) fetch(f > 0 ? k0 - kFour : 0, end);     // three tokens' states and decays are done with
        }
        if constexpr (NB > 1) {
#pragma unroll
          for (int k = 0; k < kFour; ++k) sums[turn][sb][0][k][x.lane] = ys[k], sums[turn][sb][1][k][x.lane] = qs[k], sums[turn][sb][2][k][x.lane] = ws[k];
          __syncthreads();           // the turn before is read by all that met here
          if (sb == 0)
#pragma unroll
            for (int k = 0; k < kFour; ++k)
#pragma unroll
              for (int j = 1; j < NB; ++j)
                ys[k] += sums[turn][j][0][k][x.lane], qs[k] += sums[turn][j][1][k][x.lane], ws[k] += sums[turn][j][2][k][x.lane];
          turn ^= 1;
        }
        if constexpr (NB > 1)
          if (sb == 0)
#pragma unroll
            for (int k = 0; k < kFour; ++k) finish(k);
      }
    }
    if (p.seg.S == 1 && d.gstate_in)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (x.ch[r] >= 0 && x.n0 + i < a.N) d.gstate_in[((size_t)x.w.b * a.E + x.ch[r]) * a.N + x.n0 + i] = g[r][i];
  }
  // sums over the segment's tokens (zeros where it has none)
  if (p.pA)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (x.ch[r] >= 0 && x.n0 + i < a.N) p.pA[(seg_row * a.E + x.ch[r]) * a.N + x.n0 + i] = dA[r][i];
  if (sb == 0 && x.live) {
    if (p.pD) p.pD[seg_row * a.E + x.e] = dD;
    if (p.pb) p.pb[seg_row * a.E + x.e] = db;
  }
}

// What is summed over blocks of the walk, each value by one thread and in order: dB and dC of a token over the
// tiles (the first `token_blocks` blocks), and dA, dD and the bias's gradient over rows and segments.
template <bool kBf16>
__global__ void __launch_bounds__(256) sum_kernel(BwdArgs p, unsigned token_blocks) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  const SelScan& a = p.a;
  if (blockIdx.x >= token_blocks) {
    const size_t i = (blockIdx.x - token_blocks) * (size_t)256 + threadIdx.x, nA = (size_t)a.E * a.N;
    const bool inA = i < nA, inD = !inA && i < nA + a.E;
    if (i >= nA + 2 * (size_t)a.E) return;
    const float* part = inA ? p.pA : inD ? p.pD : p.pb;
    float* out = inA ? p.d.gA : inD ? p.d.gD : p.d.gbias;
    if (!out) return;
    const size_t n = inA ? nA : a.E, j = inA ? i : inD ? i - nA : i - nA - a.E;
    const int64_t rows = (int64_t)a.B * p.seg.S;
    float s = 0.0f;
#pragma unroll 8
    for (int64_t r = 0; r < rows; ++r) s += part[r * n + j];
    out[j] = s;
    return;
  }
  const int NP = 16 * p.NB;
  const int64_t total = (int64_t)a.B * a.T * a.G * 2 * NP;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < total; i += (int64_t)token_blocks * 256) {
    const int k = (int)(i % (2 * NP)), n = k % NP;
    const int64_t row = i / (2 * NP) / a.G;
    const int g = (int)(i / (2 * NP) % a.G);
    T* out = (T*)(k < NP ? p.d.gB : p.d.gC);
    if (n >= a.N || !out) continue;
    float s = 0.0f;
    if (row % a.T < row_len(a.lens, (int)(row / a.T), a.T)) {
      const float* part = p.part + ((size_t)row * p.tiles + g * p.per_group) * 2 * NP + k;
#pragma unroll 8
      for (int j = 0; j < p.per_group; ++j) s += part[(size_t)j * 2 * NP];
    }
    El::store(out + ((size_t)row * a.G + g) * a.N + n, s);
  }
}

struct Layout {
  size_t states, reach, hs, gs, width, part, pA, pD, pb, bytes;
  int tiles, per_group, NB, chunks;
  Segments seg;
};

Layout layout(const SelScan& a) {
  Layout l{};
  l.per_group = (a.E / a.G + kChannels - 1) / kChannels;
  l.tiles = l.per_group * a.G;
  l.NB = (a.N + 15) / 16;
  const int64_t waves = (int64_t)a.B * l.tiles * l.NB;
  int64_t S = 1;
  if (waves < 2048) S = std::min<int64_t>((a.T + kChunk - 1) / kChunk, (4096 + waves - 1) / waves);
  // us in one piece and cut, 1024 tokens in bf16: 16 states, 1024 waves 2082 and 1259, 1536 waves 2171 and 2001, 1984 waves 2399 and
  // 2388; 32 states (two waves a tile) 1024 waves 2210 and 1757; 64 states (one wave a SIMD has room) 1024 waves 1581 and 1704.
  // Few channels: the join's segments follow each other, as do a segment's tokens.  us with 2048 segments, with 512 and
  // with 128: 32768 tokens of 64 channels 422, 203 and 397; 8192 tokens with 512 and with 256: 133 and 107.
  S = std::min<int64_t>(S, (int64_t)std::sqrt(8.0 * a.T));
  S = std::max<int64_t>(S, 1);
  const int64_t len = std::max<int64_t>(kChunk, ((a.T + S - 1) / S + kChunk - 1) / kChunk * kChunk);
  l.seg = {(int)std::max<int64_t>(1, (a.T + len - 1) / len), (int)len};
  l.chunks = (a.T + kChunk - 1) / kChunk;
  size_t at = 0;
  auto take = [&](size_t floats) {
    const size_t here = at;
    at += (floats * 4 + 255) / 256 * 256;
    return here;
  };
  const size_t be = (size_t)a.B * a.E, NP = 16 * l.NB;
  l.states = take(be * l.chunks * NP);
  l.reach = take(be * l.chunks);
  l.hs = take(be * l.seg.S * NP), l.gs = take(be * l.seg.S * NP), l.width = take(be * l.seg.S);
  l.part = take((size_t)a.B * a.T * l.tiles * 2 * NP);
  l.pA = take(be * l.seg.S * a.N), l.pD = take(be * l.seg.S), l.pb = take(be * l.seg.S);
  l.bytes = at;
  return l;
}

template <bool kBf16, int NB>
void launch(const BwdArgs& p, hipStream_t st) {
  const SelScan& a = p.a;
  const unsigned blocks = (unsigned)((int64_t)a.B * p.tiles * p.seg.S);
  if (p.seg.S > 1)
    local_kernel<kBf16, NB, true><<<blocks, NB * 64, 0, st>>>(p);
  else if (a.T > kChunk)
    local_kernel<kBf16, NB, false><<<blocks, NB * 64, 0, st>>>(p);
  join_kernel<<<(unsigned)std::min<int64_t>(((int64_t)a.B * a.E * 16 * NB + 255) / 256, 1 << 22), 256, 0, st>>>(p);
  walk_kernel<kBf16, NB><<<blocks, NB * 64, 0, st>>>(p);
  const int64_t tokens = p.d.gB || p.d.gC ? (int64_t)a.B * a.T * a.G * 32 * NB : 0;
  const unsigned token_blocks = (unsigned)std::min<int64_t>((tokens + 255) / 256, 1 << 20);
  const unsigned row_blocks = p.pA || p.pD || p.pb ? (unsigned)(((int64_t)a.E * (a.N + 2) + 255) / 256) : 0;
  if (token_blocks + row_blocks) sum_kernel<kBf16><<<token_blocks + row_blocks, 256, 0, st>>>(p, token_blocks);
}

}  // namespace

size_t selscan_workspace_backward(const SelScan& a) { return layout(a).bytes; }

hipError_t launch_selscan_backward(const SelScan& a, const float* state_in, const SelScanGrads& d, char* ws,
                                   hipStream_t st) {
  const Layout l = layout(a);
  auto at = [&](size_t off) { return (float*)(ws + off); };
  const BwdArgs p{a, d, state_in, l.seg, l.tiles, l.per_group, l.NB, l.chunks, at(l.states), at(l.reach), at(l.hs), at(l.gs),
                  at(l.width), at(l.part), d.gA ? at(l.pA) : nullptr, d.gD ? at(l.pD) : nullptr, d.gbias ? at(l.pb) : nullptr};
  auto by_states = [&](auto bf16) {
    switch (l.NB) {
      case 1: return launch<bf16, 1>(p, st);
      case 2: return launch<bf16, 2>(p, st);
      case 3: return launch<bf16, 3>(p, st);
      default: return launch<bf16, 4>(p, st);
    }
  };
  a.bf16 ? by_states(std::true_type{}) : by_states(std::false_type{});
  return hipGetLastError();
}

}  // namespace pnr
