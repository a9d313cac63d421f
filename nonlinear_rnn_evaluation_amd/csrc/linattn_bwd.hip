// Gradients of the linear attention.
//
// With D_t = dL/dS_t:  D_t = scale q_t do_t^T + exp(g_{t+1}) D_{t+1}, and
//   dq_t = scale S_t do_t,  dk_t = D_t v_t,  dv_t = D_t^T k_t,  dS_0 = exp(g_1) D_1:
// dq, dk and dv are the forward recurrence in other roles (linattn_tile.h).
//
// dg_t = <D_t, exp(g_t) S_{t-1}> is the sum of all products that cross from tokens before t to
// tokens from t on.  Inside a chunk of C tokens with the state S at its start and E what later
// chunks send back, it is
//   sum_{i >= t > j} W_ij + sum_{i >= t} b_i + sum_{j < t} c_j + exp(G_C) <S, E>,
//   W_ij = scale exp(G_i - G_j) (do_i . v_j)(q_i . k_j),  b_i = the part of q_i . dq_i that comes
//   from S,  c_j = the part of k_j . dk_j that comes from E.
// The last term follows from X = <S, E> behind the chunk: X - sum c, and X - sum c + sum b is <S, E> before
// it.  The rounding of these sums adds up along such a walk (as every token's does in the global form
// dg_t = dg_{t+1} + q_t . dq_t - k_t . dk_t), so X is taken from the states themselves every kWalk
// chunks, and what a walk misses of the value at its other end is spread over its chunks.  300 heads of 32 x 32
// over 4096 tokens in fp32, one walk a row: dg off by 1.7e-6 of its norm, more the earlier the token, and
// its sum over the tokens by 1.9e-5; walks of four chunks 3.5e-7 and 7.7e-7, for 1 % of a training pass.
//
// 4 x 16 heads of 128 x 128 over 4096 tokens in bf16: sums 42 and 45 us, scan 24, dq with u and b 144, dk
// with c 152, dv 94, dg 9 (10 % more on some boxes).  The dot products cost dq and dk their three-part S
// (two in dv), a fourth tile of rows and, dq, a second set of scores.
#include <algorithm>
#include <type_traits>

#include "linattn_tile.h"

namespace pnr {
namespace linattn {
namespace {

struct DecayArgs {
  LinAttn a;
  const float *u, *c;        // [B][Hkv][T]; u_t = b_t + sum_j W_tj - sum_i W_it
  const float* b;            // [B][Hkv][chunks]: sum b
  const float* x_end;        // [B][Hkv][nseg][marks]
  const float* x_first;      // [B][Hkv], or nullptr: zeros
  int seg_chunks, nseg, marks;
  float* gg;                 // [B][T][Hkv] (per token), or
  double* walk_sum;          // [B][Hkv][nseg][marks]
};

__device__ __forceinline__ float wave_suffix_sum(float v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const float y = __shfl_down(v, d);
    if (lane + d < 64) v += y;
  }
  return v;
}

// A wave a walk: up to kWalk chunks, from the last to the first.
__global__ void __launch_bounds__(256) decay_grad_kernel(DecayArgs p) {
  const LinAttn& a = p.a;
  const int lane = threadIdx.x & 63;
  const int64_t per_row = (int64_t)p.nseg * p.marks, walks = (int64_t)a.B * a.Hkv * per_row;
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < walks; w += (int64_t)gridDim.x * 4) {
    const int mark = w % p.marks, seg = w / p.marks % p.nseg, h = w / per_row % a.Hkv, b = w / per_row / a.Hkv;
    const int n = row_len(a.lens, b, a.T);
    const size_t row = (size_t)b * a.Hkv + h;
    const int chunks = (a.T + kChunk - 1) / kChunk, c_lo = seg * p.seg_chunks + mark * kWalk;
    const int c_hi = min(min(c_lo + kWalk, (seg + 1) * p.seg_chunks), chunks);
    const int live = min(c_hi, (n + kChunk - 1) / kChunk) - c_lo;       // chunks with tokens
    float us[kWalk], cs[kWalk], b_all[kWalk], before[kWalk];
#pragma unroll
    for (int j = 0; j < kWalk; ++j) {
      const int t = (c_lo + j) * kChunk + lane;
      const bool in = j < live && t < a.T;
      us[j] = in ? p.u[row * a.T + t] : 0.0f;
      cs[j] = in ? p.c[row * a.T + t] : 0.0f;
      b_all[j] = j < live ? p.b[row * chunks + c_lo + j] : 0.0f;
    }
    float x = live > 0 ? p.x_end[w] : 0.0f;
    const float x_start = live <= 0 ? 0.0f : c_lo > 0 ? p.x_end[w - 1] : p.x_first ? p.x_first[row] : 0.0f;
#pragma unroll
    for (int j = kWalk; j--;) {
      us[j] = wave_suffix_sum(us[j], lane);
      const float after = wave_suffix_sum(cs[j], lane), all = __shfl(after, 0);
      cs[j] = all - after;
      x -= all;
      before[j] = x;                                // exp(G_C) <S, E>
      x += b_all[j];
    }
    const float missed = live > 0 ? (x - x_start) / live : 0.0f;
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < kWalk; ++j) {
      const int t = (c_lo + j) * kChunk + lane;
      if (c_lo + j >= c_hi || t >= a.T) continue;
      const float g = a.g[a.decay_token ? ((size_t)b * a.T + t) * a.Hkv + h : (size_t)h];
      // a decay that forgets everything passes no gradient
      const float d = t < n && !(g <= kLogDecayMin) ? us[j] + cs[j] + (before[j] - missed * (live - j - 0.5f)) : 0.0f;
      if (p.gg) p.gg[((size_t)b * a.T + t) * a.Hkv + h] = d;
      sum += d;
    }
    if (p.walk_sum) {
#pragma unroll
      for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
      if (lane == 0) p.walk_sum[w] = sum;
    }
  }
}

__global__ void __launch_bounds__(64) decay_head_kernel(const double* walk_sum, int B, int Hkv, int64_t walks, float* gg) {
  const int h = blockIdx.x;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < B * walks; i += 64) s += walk_sum[((i / walks) * Hkv + h) * walks + i % walks];
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if (threadIdx.x == 0) gg[h] = (float)s;
}

struct BackwardLayout {
  Plan plan;
  int marks;
  size_t s = 0, e = 0, last = 0, decay = 0, u = 0, b = 0, c = 0, mid = 0, x_end = 0, x_first = 0, walk_sum = 0, total = 0;
};
BackwardLayout backward_layout(const LinAttn& a) {
  BackwardLayout l;
  l.plan = make_plan(a, true);
  l.marks = (l.plan.seg_chunks + kWalk - 1) / kWalk;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  const size_t rows = (size_t)a.B * a.Hkv, segs = rows * l.plan.nseg, tokens = rows * a.T * 4;
  if (l.plan.nseg > 1) l.s = take(l.plan.states), l.e = take(l.plan.states), l.decay = take(segs * 4);
  l.last = take(rows * a.Dk * a.Dv * 4);
  l.u = take(tokens), l.c = take(tokens);
  l.b = take(rows * ((a.T + kChunk - 1) / kChunk) * 4);
  const auto tile = [](int d) { return (size_t)(d > 64 ? 128 : 64); };
  l.mid = take(segs * (l.marks - 1) * tile(a.Dk) * tile(a.Dv) * 4);
  l.x_end = take(segs * l.marks * 4);
  l.x_first = take(rows * 4);
  l.walk_sum = take(segs * l.marks * 8);
  l.total = off;
  return l;
}

}  // namespace
}  // namespace linattn

using namespace linattn;

size_t linattn_workspace_backward(const LinAttn& a) { return backward_layout(a).total; }

hipError_t launch_linattn_backward(const LinAttn& a, const float* state_in, const LinAttnGrads& d, char* ws,
                                   hipStream_t st) {
  const BackwardLayout l = backward_layout(a);
  const int G = a.H / a.Hkv, nseg = l.plan.nseg;
  const int64_t rows = (int64_t)a.B * a.Hkv;
  float *S = (float*)(ws + l.s), *E = (float*)(ws + l.e), *last = (float*)(ws + l.last);
  float *u = (float*)(ws + l.u), *b = (float*)(ws + l.b), *c = (float*)(ws + l.c);
  hipError_t e = hipSuccess;

  RoleArgs base{};
  base.a = a;
  base.vec = rows_vec(a.q, a.Dk, a.bf16) && rows_vec(a.k, a.Dk, a.bf16) && rows_vec(a.v, a.Dv, a.bf16) &&
             rows_vec(d.go, a.Dv, a.bf16) && ((uintptr_t)d.gq | (uintptr_t)d.gk | (uintptr_t)d.gv) % 16 == 0;
  base.seg_chunks = l.plan.seg_chunks, base.nseg = nseg, base.marks = l.marks;
  float *x_end = (float*)(ws + l.x_end), *x_first = (float*)(ws + l.x_first);
  float* mid = d.gg && l.marks > 1 ? (float*)(ws + l.mid) : nullptr;
  base.p_scale = a.scale;
  // forward in time: keys k, values v; backward: keys q, values do, times the scale
  RoleArgs fwd = base, rev = base;
  fwd.nkv = 1, fwd.nq = G, fwd.inter_scale = a.scale, fwd.upd_scale = 1.0f;
  rev.nkv = G, rev.nq = 1, rev.inter_scale = 1.0f, rev.upd_scale = a.scale;
  fwd.s_in = state_in, rev.s_in = d.gstate_out;
  // states are needed at the segments' starts (forward in time) and ends (backward)
  const bool need_s = d.gq || d.gg, need_e = d.gk || d.gv || d.gg || d.gstate_in;
  if (nseg > 1) {
    ScanArgs sc[2];
    int count = 0;
    float* decay = (float*)(ws + l.decay);
    if (need_s) {
      RoleArgs p = fwd;
      p.y = a.k, p.z = a.v, p.dk = a.Dk, p.dv = a.Dv;
      p.s_out = S, p.seg_decay = decay;
      if ((e = run_sum<false>(p, st)) != hipSuccess) return e;
      sc[count++] = {a, l.plan.seg_chunks, S, decay, state_in, last, nseg, a.Dk * a.Dv, 0};
      fwd.s_in = S;
    }
    if (need_e) {
      RoleArgs p = rev;
      p.y = a.q, p.z = d.go, p.dk = a.Dk, p.dv = a.Dv;
      p.s_out = E, p.seg_decay = decay;
      if ((e = run_sum<true>(p, st)) != hipSuccess) return e;
      sc[count++] = {a, l.plan.seg_chunks, E, decay, d.gstate_out, d.gstate_in, nseg, a.Dk * a.Dv, 1};
      rev.s_in = E;
    }
    if (count && (e = launch_scan(sc, count, rows, st)) != hipSuccess) return e;
  }

  if (d.gq || d.gg) {
    RoleArgs p = fwd;
    p.x = d.go, p.y = a.v, p.z = a.k, p.e = a.q;
    p.dk = a.Dv, p.dv = a.Dk, p.transposed = 1;
    p.o = d.gq;
    p.u = u, p.b = b, p.s_mid = mid;
    if (nseg == 1) p.s_out = last;
    if ((e = run_role<false, kDotQ>(p, st)) != hipSuccess) return e;
  }
  const bool want_e = d.gstate_in && nseg == 1;
  if (d.gk || d.gg || want_e) {
    RoleArgs p = rev;
    p.x = a.v, p.y = d.go, p.z = a.q, p.e = a.k;
    p.dk = a.Dv, p.dv = a.Dk, p.transposed = 1;
    p.o = d.gk;
    p.u = c;
    p.s_mid = mid;
    if (d.gg) p.x_end = x_end, p.s_entry = S, p.s_last = last;
    if (d.gg && state_in) p.x_first = x_first, p.s_first = state_in;
    if (nseg == 1) p.s_out = d.gstate_in;
    if ((e = run_role<true, kDotK>(p, st)) != hipSuccess) return e;
  }
  if (d.gv) {
    RoleArgs p = rev;
    p.x = a.k, p.y = a.q, p.z = d.go;
    p.dk = a.Dk, p.dv = a.Dv;
    p.o = d.gv;
    if ((e = run_role<true, kOut>(p, st)) != hipSuccess) return e;
  }
  if (d.gg) {
    DecayArgs p{a, u, c, b, x_end, state_in ? x_first : nullptr, l.plan.seg_chunks, nseg, l.marks, nullptr, nullptr};
    if (a.decay_token) p.gg = d.gg; else p.walk_sum = (double*)(ws + l.walk_sum);
    const int64_t walks = (int64_t)nseg * l.marks, waves = rows * walks;
    decay_grad_kernel<<<(unsigned)std::min<int64_t>((waves + 3) / 4, 1 << 22), 256, 0, st>>>(p);
    if (!a.decay_token) decay_head_kernel<<<a.Hkv, 64, 0, st>>>(p.walk_sum, a.B, a.Hkv, walks, d.gg);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace pnr
