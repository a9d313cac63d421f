// Selective scan over whole sequences:
//   h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,   y_t = (C_t . h_t + D u_t) silu(z_t)
//
// The decay differs for every channel and state, so no product of chunks carries this; a state's
// token costs a multiplication for the exponent, 2^x (two issue slots), a multiplication and two
// fused ones: six slots.  For 16 states that is more time than its bytes take (184 us against 112
// for 32768 tokens of 2048 bf16 channels), and instruction issue bounds it.
//
// A quad of lanes holds a channel, so that what the states share (step width, gate, conversions)
// costs each lane a quarter, and four tokens go at once, so that their steps fill each other's
// gaps when a wave has its SIMD to itself.  9.2 slots a state and token; 4 x 4096 x 4096 x 16 in bf16 301 us, after
// 224 for the sums where time is cut, vector instructions issuing 98 and 92 % of the time (32768 x 2048 x 16: 93 and 87 %;
// rows that end early: 69 and 61 %, since every block cuts its row as a full one).  64 channels a wave with matrix
// instructions for the outer products, as backwards, came within 7 % of it and was slower for small calls.
#include <algorithm>
#include <cmath>

#include "selscan_tile.h"

namespace pnr {
namespace {

using namespace selscan;

struct FwdArgs {
  SelScan a;
  const float* s_in;
  void* y;
  float* s_out;
  Segments seg;
  int per_group;             // blocks of a group
  int64_t tiles;             // blocks of a segment
  float *sums, *width;       // [B, S, E, 4 R] states and [B, S, E] summed step widths of the segments
};

// Where a wave works: row b, group g, its first channel e0 (of E) and how many it has.
struct Tile {
  int b, g, e0, live;
};

// kW waves a block share a group's B and C, 16 channels each; `per_group` blocks a group.
constexpr int kChannels = 16;
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

// B and C of four tokens, this lane's states.
template <bool kOut, int R>
struct Four {
  float B[4][R], C[4][kOut ? R : 1];
  __device__ __forceinline__ void read(const float* s) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      read_states<R>(s + k * 8 * R, B[k]);
      if constexpr (kOut) read_states<R>(s + k * 8 * R + 4 * R, C[k]);
    }
  }
};

// Token k of a quad's four: the states of this lane, and (kOut) the channel's output in lane k.
template <int k, bool kOut, int R>
__device__ __forceinline__ void token(float delta, float x, float (&h)[R], const float (&A)[R], const Four<kOut, R>& f, float& o, int nq) {
  const float d = quad_perm<0x55 * k>(delta), xk = quad_perm<0x55 * k>(x);
  float acc = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    h[i] = fmaf(h[i], __builtin_amdgcn_exp2f(d * A[i]), xk * f.B[k][i]);
    if constexpr (kOut) acc = fmaf(h[i], f.C[k][i], acc);
  }
  if constexpr (kOut) {
    acc += quad_perm<0xb1>(acc);
    acc += quad_perm<0x4e>(acc);
    o = nq == k ? acc : o;
  }
}

// One segment of one block's channels.  kSum: from zeros, only the state at its end and the sum of its
// step widths; otherwise from the segment's first state to outputs.  A quad holds a channel, R
// states a lane.  Four tokens go at once: each lane of a quad prepares one of them (its step width,
// softplus, gate) and hands it to the others.
template <bool kBf16, int R, int kW, bool kSum>
__global__ void __launch_bounds__(kW * 64, 1) scan_kernel(FwdArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  constexpr int NP = 4 * R, kTok = kStage<R>;
  __shared__ alignas(16) float bc[2][kTok * 2 * NP];
  const SelScan& a = p.a;
  const int seg = (int)(blockIdx.x / p.tiles);
  const Tile w = tile_of<kW>(a, blockIdx.x % p.tiles, p.per_group);
  const int n = row_len(a.lens, w.b, a.T), t0 = seg * p.seg.len, tend = min(t0 + p.seg.len, a.T), t1 = min(tend, n);
  if (kSum && t0 >= t1) return;
  const int lane = threadIdx.x & 63, nq = lane & 3, c = lane >> 2, e = w.e0 + min(c, w.live - 1);
  const bool busy = w.live > 0, live = c < w.live, whole = p.seg.S == 1;
  const size_t mid = (((size_t)w.b * p.seg.S + seg) * a.E + e) * NP + nq * R, at = ((size_t)w.b * a.E + e) * a.N + nq * R;
  float A[R], h[R];
  if (busy) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool real = nq * R + i < a.N;
      A[i] = real ? exponent(a.A[(size_t)e * a.N + nq * R + i]) : 0.0f;
      h[i] = !kSum && whole && real && p.s_in ? p.s_in[at + i] : 0.0f;
    }
    if (!kSum && !whole) read_states<R>(p.sums + mid, h);
  }
  const float bias = busy && a.bias ? a.bias[e] : 0.0f, D = !kSum && busy && a.D ? a.D[e] : 0.0f;
  const T* u = (const T*)a.u.p + w.b * a.u.sb;
  const T* dt = (const T*)a.dt.p + w.b * a.dt.sb;
  const T* z = (const T*)a.z.p + (kSum || !a.z.p ? 0 : w.b * a.z.sb);
  const bool gated = !kSum && a.z.p;
  T* y = (T*)p.y + (size_t)w.b * a.T * a.E;
  float total = 0.0f;
  if (t0 < t1) {
    constexpr int kDepth = 4;                 // fours of tokens on their way from memory
    T ur[kDepth], dr[kDepth], zr[kDepth];
    // Operands as buffers from the tile's first token on, tokens as 32-bit offsets: a wave that runs alone
    // pays for every scalar instruction too (the plan keeps wide strides away).
    const int su = (int)a.u.st * (int)sizeof(T), sd = (int)a.dt.st * (int)sizeof(T), sz = (int)a.z.st * (int)sizeof(T),
              sy = a.E * (int)sizeof(T);
    const int ou = nq * su + e * (int)sizeof(T), od = nq * sd + e * (int)sizeof(T), oz = nq * sz + e * (int)sizeof(T),
              oy = nq * sy + e * (int)sizeof(T);
    __amdgpu_buffer_rsrc_t bu, bd, bz, by;
    int left = 0;                             // of the tile's tokens, this lane's from `left` on are not there
    auto rebase = [&](int tile) {
      bu = buffer_of(u + tile * a.u.st, true), bd = buffer_of(dt + tile * a.dt.st, true);
      bz = buffer_of(z + (kSum ? 0 : tile * a.z.st), gated), by = buffer_of(y + (int64_t)tile * a.E, true);
      left = t1 - tile - nq;
    };
    auto fetch = [&](int k, int i) {          // tokens k.. of the tile; zeros beyond the last token
      const bool there = k < left;
      ur[i] = load_buffer<T>(bu, there ? ou : kNowhere, k * su);
      dr[i] = load_buffer<T>(bd, there ? od : kNowhere, k * sd);
      if (!kSum) zr[i] = load_buffer<T>(bz, there ? oz : kNowhere, k * sz);
    };
    Stage<kBf16, R, kW, kTok> stage;
    stage.start(a, w);
    stage.fetch(t0, t1);
    // One wave a SIMD has nobody to fill its waits, so the steps of neighbouring fours overlap: while one
    // runs through the states, the next one's widths are made and the last one's outputs gated.
    float uv[2] = {}, zv[2] = {}, delta[2], x[2], done = 0.0f;
    auto widths = [&](int k, int i, int j) {
      uv[j] = El::load(&ur[i]), zv[j] = kSum ? 0.0f : El::load(&zr[i]);
      delta[j] = step_width(El::load(&dr[i]) + bias, a.softplus, k < left);
      x[j] = delta[j] * uv[j];
    };
    auto finish = [&](int k, int j, bool first) {           // the outputs of tokens k..k + 3
      const float o = fmaf(D, uv[j], done);
      store_buffer<kBf16>(o * gate_of(zv[j], gated), by, live && k < left && !first ? oy : kNowhere, first ? 0 : k * sy);
    };
    if (busy) {
      rebase(t0);
#pragma unroll
      for (int i = 0; i < kDepth; ++i) fetch(4 * i, i);
      widths(0, 0, 0);
      fetch(4 * kDepth, 0);
    }
    int buf = 0;
    for (int tile = t0; tile < t1; tile += kTok, buf ^= 1) {
      stage.put(bc[buf]);
      __syncthreads();
      if (tile + kTok < t1) stage.fetch(tile + kTok, t1);
      if (!busy) continue;
      if (tile > t0) {
        if (!kSum) finish(kTok - 4, 1, false);              // of the tile before
        rebase(tile);
      }
      Four<!kSum, R> f[2];
      const float* s = bc[buf] + nq * R;
      f[0].read(s);
      const int here = min(kTok, t1 - tile);
      for (int k0 = 0; k0 < here; k0 += 4 * kDepth) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
          const int k = k0 + 4 * i;
          if (k >= here) break;
          f[(i + 1) % 2].read(s + (k + 4 < kTok ? (k + 4) * 2 * NP : 0));
          float o = 0.0f;
          token<0, !kSum, R>(delta[i % 2], x[i % 2], h, A, f[i % 2], o, nq);
          if (!kSum) finish(k - 4, (i + 1) % 2, k == 0);
          token<1, !kSum, R>(delta[i % 2], x[i % 2], h, A, f[i % 2], o, nq);
          widths(k + 4, (i + 1) % kDepth, (i + 1) % 2);
          fetch(k + 4 + 4 * kDepth, (i + 1) % kDepth);
          token<2, !kSum, R>(delta[i % 2], x[i % 2], h, A, f[i % 2], o, nq);
          token<3, !kSum, R>(delta[i % 2], x[i % 2], h, A, f[i % 2], o, nq);
          if (kSum) total += delta[i % 2];
          done = o;
        }
      }
    }
    if (!kSum && busy) {
      const int k = ((t1 - 1 - t0) % kTok) / 4 * 4;
      k / 4 % 2 ? finish(k, 1, false) : finish(k, 0, false);
    }
  }
  if (!busy) return;
  if (kSum) {
#pragma unroll
    for (int i = 0; i < R; ++i) p.sums[mid + i] = h[i];
    total += quad_perm<0xb1>(total);
    total += quad_perm<0x4e>(total);
    if (live && nq == 0) p.width[((size_t)w.b * p.seg.S + seg) * a.E + e] = total;
    return;
  }
  if (live)
    for (int t = max(t0, t1) + nq; t < tend; t += 4) El::store(y + (size_t)t * a.E + e, 0.0f);
  if (whole && p.s_out && live)
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (nq * R + i < a.N) p.s_out[at + i] = h[i];
}

// The recurrence over a row's segments: each segment's first state in place of its sum, and the last
// state.  A thread a state; eight segments' sums are asked for before the first is used.
__device__ __forceinline__ void join_state(const FwdArgs& p, int s, int e, int b, int NP) {
  constexpr int kBatch = 8;
  const SelScan& a = p.a;
  const int n = row_len(a.lens, b, a.T), segs = (int)(((int64_t)n + p.seg.len - 1) / p.seg.len);
  const bool real = s < a.N;
  const float A = real ? exponent(a.A[(size_t)e * a.N + s]) : 0.0f;
  const size_t at = ((size_t)b * a.E + e) * a.N + s;
  float h = real && p.s_in ? p.s_in[at] : 0.0f;
  const size_t row = (size_t)b * p.seg.S * a.E + e;
  for (int k0 = 0; k0 < segs; k0 += kBatch) {
    float own[kBatch], d[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const size_t r = row + (size_t)min(k0 + k, segs - 1) * a.E;
      own[k] = p.sums[r * NP + s], d[k] = p.width[r];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k0 + k < segs) {
        p.sums[(row + (size_t)(k0 + k) * a.E) * NP + s] = h;
        h = carried(h, d[k] * A, factor(d[k] * A), own[k]);
      }
  }
  if (p.s_out && real) p.s_out[at] = h;
}

__global__ void __launch_bounds__(256) join_kernel(FwdArgs p, int NP) {
  const SelScan& a = p.a;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < (int64_t)a.B * a.E * NP; i += (int64_t)gridDim.x * 256)
    join_state(p, (int)(i % NP), (int)(i / NP % a.E), (int)(i / NP / a.E), NP);
}

int states_of(const SelScan& a) {
  int R = 1;
  while (4 * R < a.N) R *= 2;
  return R;
}

// How a call is cut: waves of a block, blocks of a group, segments.
struct Plan {
  int waves, per_group;
  Segments seg;
};

Plan plan_of(const SelScan& a) {
  Plan p{};
  const int W = a.E / a.G;
  p.waves = W <= kChannels ? 1 : 4;
  p.per_group = (W + p.waves * kChannels - 1) / (p.waves * kChannels);
  const int64_t waves = (int64_t)a.B * a.G * ((W + kChannels - 1) / kChannels);
  // One wave a SIMD goes through the tokens in one pass at 120 ns each; two passes over segments cost
  // twice the instructions, but many waves a SIMD fill each other's gaps.  bf16, 16 states, us in one
  // pass and in two over 12288 to 16384 waves: 1792 waves 672 and 825, 1536 waves 341 and 365 (2048
  // tokens), 1024 waves 520 and 483 (4096 tokens), 244 and 241 (2000), 256 waves 473 and 152, 128 waves
  // 4268 and 510 (32768).  A second pass and the join cost 8 us: 128 waves over 37 tokens 10.1 and 17.2.
  // Other counts of states, us in one pass and in two: 4 states, 2048 tokens, 1024 waves 179 and 134, 1536 waves 256
  // and 231; 32 states 768 waves 364 and 355, 1024 waves 369 and 464; 64 states (one wave a SIMD has room) 512 waves
  // 645 and 590, 768 waves 648 and 828, 1024 waves 654 and 1071, 1536 waves 1308 and 1579.  So from 32 states on two
  // passes cost up to 1.6 times one between 768 and 1280 waves.  fp32, 16 states: 1024 waves 283 and 268, 1536 356 and 393.
  // With row lengths some rows are expected to be short: what is cut behind their ends costs nothing, while in
  // one pass the longest row sets the time.  2000 tokens, rows half full, us in one pass and in two: 1024 waves 236 and
  // 183, 1792 waves 261 and 248, 2560 waves 295 and 368, 3840 waves 339 and 504; lengths that are all 2000: 1280 waves 332
  // and 301, 1792 waves 336 and 420, 3840 waves 576 and 863.  So the second pass is lost from some 2000 waves on.
  const int64_t enough = a.lens ? 4096 : 1280, target = a.lens ? 16384 : 12288;
  int64_t S = 1;
  if (waves < enough && a.T > 128) S = std::min<int64_t>((a.T + 31) / 32, (target + waves - 1) / waves);
  // Few channels: the join goes through S segments one after the other, at 0.12 us each, the passes through T / S
  // tokens at 0.24 us for both.  us with 1024 segments, with 256 and with 64: 32768 tokens of 64 channels 143, 64
  // and 113, of 256 channels 127, 106 and 130.
  S = std::min<int64_t>(S, (int64_t)std::sqrt(2.0 * a.T) + 1);
  const int64_t len = std::max<int64_t>(32, ((a.T + S - 1) / S + 31) / 32 * 32);
  p.seg = {(int)std::max<int64_t>(1, (a.T + len - 1) / len), (int)len};
  return p;
}

struct Layout {
  size_t sums, width, bytes;
};
Layout layout(const SelScan& a, const Segments& s) {
  Layout l{};
  if (s.S == 1) return l;
  auto up = [](size_t v) { return (v * 4 + 255) / 256 * 256; };
  l.width = up((size_t)a.B * s.S * a.E * 4 * states_of(a));
  l.bytes = l.width + up((size_t)a.B * s.S * a.E);
  return l;
}

template <bool kBf16, int R, int kW>
void launch_pass(const FwdArgs& p, hipStream_t st) {
  const unsigned blocks = (unsigned)(p.tiles * p.seg.S);
  if (p.seg.S > 1) {
    scan_kernel<kBf16, R, kW, true><<<blocks, kW * 64, 0, st>>>(p);
    join_kernel<<<(unsigned)std::min<int64_t>(((int64_t)p.a.B * p.a.E * 4 * R + 255) / 256, 1 << 22), 256, 0, st>>>(p, 4 * R);
  }
  scan_kernel<kBf16, R, kW, false><<<blocks, kW * 64, 0, st>>>(p);
}

template <bool kBf16, int R>
void launch_shape(const FwdArgs& p, const Plan& plan, hipStream_t st) {
  plan.waves == 1 ? launch_pass<kBf16, R, 1>(p, st) : launch_pass<kBf16, R, 4>(p, st);
}

template <bool kBf16>
void launch(const FwdArgs& p, const Plan& plan, hipStream_t st) {
  switch (states_of(p.a)) {
    case 1: return launch_shape<kBf16, 1>(p, plan, st);
    case 2: return launch_shape<kBf16, 2>(p, plan, st);
    case 4: return launch_shape<kBf16, 4>(p, plan, st);
    case 8: return launch_shape<kBf16, 8>(p, plan, st);
    default: return launch_shape<kBf16, 16>(p, plan, st);
  }
}

}  // namespace

size_t selscan_workspace(const SelScan& a) { return layout(a, plan_of(a).seg).bytes; }

hipError_t launch_selscan_forward(const SelScan& a, const float* state_in, void* y, float* state_out, char* ws,
                                  hipStream_t st) {
  const Plan plan = plan_of(a);
  FwdArgs p{a, state_in, y, state_out, plan.seg, plan.per_group};
  const Layout l = layout(a, p.seg);
  p.tiles = (int64_t)a.B * a.G * p.per_group;
  p.sums = (float*)(ws + l.sums), p.width = (float*)(ws + l.width);
  a.bf16 ? launch<true>(p, plan, st) : launch<false>(p, plan, st);
  return hipGetLastError();
}

}  // namespace pnr
