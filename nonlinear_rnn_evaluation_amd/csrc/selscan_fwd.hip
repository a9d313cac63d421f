// Selective scan over whole sequences:
//   h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,   y_t = (C_t . h_t + D u_t) silu(z_t)
//
// The decay differs for every channel and state, so no product of chunks carries this; a state's
// token costs a multiplication for the exponent, 2^x (two issue slots), a multiplication and two
// fused ones: six slots.  For 16 states that is an order more time than its bytes take, and
// instruction issue bounds it.
#include <algorithm>

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

// One segment of one block's channels.  kSum: from zeros, only the state at its end and the sum of
// its step widths; otherwise from the segment's first state to outputs.
template <bool kBf16, int R, int kW, bool kSum>
__global__ void __launch_bounds__(kW * 64) scan_kernel(FwdArgs p) {
  using El = Elem<kBf16>;
  using T = typename El::type;
  constexpr int NP = 4 * R, kTok = kStage<R>, kAhead = 8;
  __shared__ alignas(16) float bc[2][kTok * 2 * NP];
  const SelScan& a = p.a;
  const int seg = (int)(blockIdx.x / p.tiles);
  const Tile w = tile_of<kW>(a, blockIdx.x % p.tiles, p.per_group);
  const int n = row_len(a.lens, w.b, a.T), t0 = seg * p.seg.len, tend = min(t0 + p.seg.len, a.T), t1 = min(tend, n);
  const bool last = seg == p.seg.S - 1;
  if (kSum && t0 >= t1) return;                      // the join skips it
  const int lane = threadIdx.x & 63, nq = lane >> 2 & 3, e = w.e0 + min(lane, w.live - 1);
  const bool busy = w.live > 0, live = lane < w.live;
  float A[4][R], h[4][R];
  int ch[4] = {e, away<1>(e), away<2>(e), away<3>(e)};
  const bool whole = p.seg.S == 1;
  if (busy) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int s = nq * R + i;
        A[r][i] = s < a.N ? exponent(a.A[(size_t)ch[r] * a.N + s]) : 0.0f;
        h[r][i] = 0.0f;
        if (!kSum && whole && s < a.N && p.s_in) h[r][i] = p.s_in[((size_t)w.b * a.E + ch[r]) * a.N + s];
      }
    if (!kSum && !whole)
#pragma unroll
      for (int r = 0; r < 4; ++r) read_states<R>(p.sums + (((size_t)w.b * p.seg.S + seg) * a.E + ch[r]) * NP + nq * R, h[r]);
  }
  const float bias = busy && a.bias ? a.bias[e] : 0.0f, D = !kSum && busy && a.D ? a.D[e] : 0.0f;
  const T* u = (const T*)a.u.p + w.b * a.u.sb;
  const T* dt = (const T*)a.dt.p + w.b * a.dt.sb;
  const T* z = (const T*)a.z.p + (kSum || !a.z.p ? 0 : w.b * a.z.sb);
  const bool gated = !kSum && a.z.p;
  T* y = (T*)p.y + (size_t)w.b * a.T * a.E;
  float total = 0.0f;
  if (t0 < t1) {
    T ur[kAhead], dr[kAhead], zr[kAhead];
    auto fetch = [&](int t) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t at = min(t + k, t1 - 1);
        ur[k] = (u + at * a.u.st)[e];
        dr[k] = (dt + at * a.dt.st)[e];
        if (gated) zr[k] = (z + at * a.z.st)[e];
      }
    };
    Stage<kBf16, R, kW, kTok> stage;
    stage.start(a, w);
    stage.fetch(t0, t1);
    if (busy) fetch(t0);
    int buf = 0;
    for (int tile = t0; tile < t1; tile += kTok, buf ^= 1) {
      stage.put(bc[buf]);
      __syncthreads();           // the other buffer's readers are past it: they met here after reading
      if (tile + kTok < t1) stage.fetch(tile + kTok, t1);
      if (!busy) continue;
      const int stop = min(tile + kTok, t1);
      for (int t = tile; t < stop; t += kAhead) {
        float uv[kAhead], dv[kAhead], zv[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) uv[k] = El::load(&ur[k]), dv[k] = El::load(&dr[k]), zv[k] = gated ? El::load(&zr[k]) : 0.0f;
        if (t + kAhead < t1) fetch(t + kAhead);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (t + k >= stop) break;
          const float raw = dv[k] + bias, delta = a.softplus ? softplus(raw) : raw;
          float d[4], x[4], acc[4], Bv[R], Cv[R];
          to_slots(delta, d);
          to_slots(delta * uv[k], x);
          const float* s = bc[buf] + (t + k - tile) * 2 * NP + nq * R;
          read_states<R>(s, Bv);
          if (!kSum) read_states<R>(s + NP, Cv);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            acc[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
              h[r][i] = fmaf(h[r][i], __builtin_amdgcn_exp2f(d[r] * A[r][i]), x[r] * Bv[i]);
              if (!kSum) acc[r] = fmaf(h[r][i], Cv[i], acc[r]);
            }
          }
          if (kSum) {
            total += delta;
          } else {
            float o = fmaf(D, uv[k], from_slots(acc));
            if (gated) o *= zv[k] * sigm(zv[k]);
            if (live) El::store(y + (size_t)(t + k) * a.E + e, o);
          }
        }
      }
    }
  }
  if (!busy) return;
  if (kSum) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // a lane beyond the last channel repeats that channel's work and writes the same
      float* out = p.sums + (((size_t)w.b * p.seg.S + seg) * a.E + ch[r]) * NP + nq * R;
#pragma unroll
      for (int i = 0; i < R; ++i) out[i] = h[r][i];
    }
    if (live) p.width[((size_t)w.b * p.seg.S + seg) * a.E + e] = total;
    return;
  }
  if (live)
    for (int t = max(t0, t1); t < tend; ++t) El::store(y + (size_t)t * a.E + e, 0.0f);
  // cut time: the join wrote the last state
  if (whole && p.s_out)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (nq * R + i < a.N) p.s_out[((size_t)w.b * a.E + ch[r]) * a.N + nq * R + i] = h[r][i];
}

// The recurrence over a row's segments: each segment's first state in place of its sum, and the last
// state.  A thread a state.
__global__ void __launch_bounds__(256) join_kernel(FwdArgs p, int NP) {
  const SelScan& a = p.a;
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i >= (int64_t)a.B * a.E * NP) return;
  const int s = (int)(i % NP), e = (int)(i / NP % a.E), b = (int)(i / NP / a.E);
  const int n = row_len(a.lens, b, a.T), segs = (n + p.seg.len - 1) / p.seg.len;
  const bool real = s < a.N;
  const float A = real ? exponent(a.A[(size_t)e * a.N + s]) : 0.0f;
  const size_t at = ((size_t)b * a.E + e) * a.N + s;
  float h = real && p.s_in ? p.s_in[at] : 0.0f;
  const size_t row = (size_t)b * p.seg.S * a.E + e;
  for (int k = 0; k < segs; ++k) {
    float* sum = p.sums + (row + (size_t)k * a.E) * NP + s;
    const float own = *sum, d = p.width[row + (size_t)k * a.E];
    *sum = h;
    h = fmaf(h, __builtin_amdgcn_exp2f(d * A), own);
  }
  if (p.s_out && real) p.s_out[at] = h;
}

int states_of(const SelScan& a) {
  int R = 1;
  while (4 * R < a.N) R *= 2;
  return R;
}

int waves_of(const SelScan& a) { return a.E / a.G <= kChannels ? 1 : 4; }

int blocks_per_group(const SelScan& a) {
  const int ch = waves_of(a) * kChannels;
  return (a.E / a.G + ch - 1) / ch;
}

// One segment where the channels fill the device; otherwise enough of them to.
Segments segments_of(const SelScan& a) {
  const int64_t waves = (int64_t)a.B * a.G * ((a.E / a.G + kChannels - 1) / kChannels);
  const int most = (a.T + 63) / 64;                  // segments of 64 tokens at least
  int S = 1;
  if (waves < 768) S = (int)std::min<int64_t>(most, (4096 + waves - 1) / waves);
  S = std::max(S, 1);
  const int len = std::max(32, ((a.T + S - 1) / S + 31) / 32 * 32);
  return {std::max(1, (a.T + len - 1) / len), len};
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
    join_kernel<<<(unsigned)(((int64_t)p.a.B * p.a.E * 4 * R + 255) / 256), 256, 0, st>>>(p, 4 * R);
  }
  scan_kernel<kBf16, R, kW, false><<<blocks, kW * 64, 0, st>>>(p);
}

template <bool kBf16, int R>
void launch_waves(const FwdArgs& p, hipStream_t st) {
  waves_of(p.a) == 1 ? launch_pass<kBf16, R, 1>(p, st) : launch_pass<kBf16, R, 4>(p, st);
}

template <bool kBf16>
void launch(const FwdArgs& p, hipStream_t st) {
  switch (states_of(p.a)) {
    case 1: return launch_waves<kBf16, 1>(p, st);
    case 2: return launch_waves<kBf16, 2>(p, st);
    case 4: return launch_waves<kBf16, 4>(p, st);
    case 8: return launch_waves<kBf16, 8>(p, st);
    default: return launch_waves<kBf16, 16>(p, st);
  }
}

}  // namespace

size_t selscan_workspace(const SelScan& a) { return layout(a, segments_of(a)).bytes; }

hipError_t launch_selscan_forward(const SelScan& a, const float* state_in, void* y, float* state_out, char* ws,
                                  hipStream_t st) {
  FwdArgs p{a, state_in, y, state_out, segments_of(a), blocks_per_group(a)};
  const Layout l = layout(a, p.seg);
  p.tiles = (int64_t)a.B * a.G * p.per_group;
  p.sums = (float*)(ws + l.sums), p.width = (float*)(ws + l.width);
  a.bf16 ? launch<true>(p, st) : launch<false>(p, st);
  return hipGetLastError();
}

}  // namespace pnr
