// Linear attention with per-head decay over whole sequences: the forward pass.
//
// One block a state head walks its chunks in order (linattn_tile.h).  Where that leaves most of
// the device idle, three launches: every segment's own sum (keys and values only), the
// recurrence over segments, and the outputs of all segments side by side.
#include <type_traits>

#include "linattn_tile.h"

namespace pnr {
namespace linattn {
namespace {

constexpr int kAhead = 4;

struct ScanPair {
  ScanArgs p[2];
};

// A thread an element of the state, over the row's segments in order: a read and a write of each one's
// state, bound by those bytes: 32 segments of 16 states of 128 x 128, 67 MB in 13 us, 5.1 TB/s.  The
// states and decays of the next kAhead segments are asked for before this kAhead's states are
// overwritten: a load behind the stores would wait for them (one segment at a time: 19 us; 2 or 8
// ahead: as 4).
__global__ void __launch_bounds__(256) scan_kernel(ScanPair pair) {
  const ScanArgs& p = pair.p[blockIdx.z];
  const int i = blockIdx.y * 256 + threadIdx.x;
  if (i >= p.size) return;
  const size_t row = blockIdx.x;
  float s = p.s_in ? p.s_in[row * p.size + i] : 0.0f;
  const int nseg = segments_of(row_len(p.a.lens, (int)(row / p.a.Hkv), p.a.T), p.seg_chunks);
  float* seg = p.seg + row * p.nseg * p.size + i;
  const float* dec = p.decay + row * p.nseg;
  auto at = [&](int k) { return p.reverse ? nseg - 1 - k : k; };
  float own[2][kAhead], d[2][kAhead];
  auto fetch = [&](int half, int k0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k0 + j < nseg) own[half][j] = seg[(size_t)at(k0 + j) * p.size], d[half][j] = dec[at(k0 + j)];
  };
  auto walk = [&](int half, int k0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k0 + j < nseg) {
        seg[(size_t)at(k0 + j) * p.size] = s;
        s = fmaf(d[half][j], s, own[half][j]);
      }
  };
  fetch(0, 0);
  for (int k0 = 0; k0 < nseg; k0 += 2 * kAhead) {
    fetch(1, k0 + kAhead);
    walk(0, k0);
    fetch(0, k0 + 2 * kAhead);
    walk(1, k0 + kAhead);
  }
  if (p.s_out) p.s_out[row * p.size + i] = s;
}

}  // namespace

hipError_t launch_scan(const ScanArgs* p, int count, int64_t rows, hipStream_t st) {
  ScanPair pair{};
  for (int i = 0; i < count; ++i) pair.p[i] = p[i];
  scan_kernel<<<dim3((unsigned)rows, (p[0].size + 255) / 256, count), 256, 0, st>>>(pair);
  return hipGetLastError();
}

}  // namespace linattn

using namespace linattn;

namespace {
struct ForwardLayout {
  Plan plan;
  size_t seg = 0, decay = 0, total = 0;
};
ForwardLayout forward_layout(const LinAttn& a) {
  ForwardLayout l;
  l.plan = make_plan(a, false);
  if (l.plan.nseg > 1) {
    l.decay = l.plan.states;
    l.total = l.decay + (size_t)a.B * a.Hkv * l.plan.nseg * 4;
  }
  return l;
}
}  // namespace

size_t linattn_workspace(const LinAttn& a) { return forward_layout(a).total; }

hipError_t launch_linattn_forward(const LinAttn& a, const float* state_in, void* o, float* state_out, char* ws,
                                  hipStream_t st) {
  const ForwardLayout l = forward_layout(a);
  RoleArgs p{};
  p.a = a;
  p.x = a.q, p.y = a.k, p.z = a.v;
  p.nq = a.H / a.Hkv, p.nkv = 1, p.dk = a.Dk, p.dv = a.Dv;
  p.vec = rows_vec(a.q, a.Dk, a.bf16) && rows_vec(a.k, a.Dk, a.bf16) && rows_vec(a.v, a.Dv, a.bf16) &&
          (uintptr_t)o % 16 == 0;
  p.p_scale = p.inter_scale = a.scale, p.upd_scale = 1.0f;
  p.o = o;
  p.seg_chunks = l.plan.seg_chunks, p.nseg = l.plan.nseg;
  if (l.plan.nseg == 1) {
    p.s_in = state_in, p.s_out = state_out;
    return run_role<false, kOut>(p, st);
  }
  float* seg = (float*)ws;
  float* decay = (float*)(ws + l.decay);
  RoleArgs s = p;
  s.s_out = seg, s.seg_decay = decay;
  hipError_t e = run_sum<false>(s, st);
  if (e != hipSuccess) return e;
  const ScanArgs sc{a, l.plan.seg_chunks, seg, decay, state_in, state_out, l.plan.nseg, a.Dk * a.Dv, 0};
  if ((e = launch_scan(&sc, 1, (int64_t)a.B * a.Hkv, st)) != hipSuccess) return e;
  p.s_in = seg;
  return run_role<false, kOut>(p, st);
}

}  // namespace pnr
