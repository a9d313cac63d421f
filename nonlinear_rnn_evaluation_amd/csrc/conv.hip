// Causal convolution along time, each channel by itself:
//   p_t = bias + sum_j w_j x_{t-W+1+j},  y = act(p)
// and its gradients, with g_t = grad_y act'(p_t):
//   dx_s = sum_j w_j g_{s+W-1-j},  dw_j = sum_t g_t x_{t-W+1+j},  db = sum_t g_t
//
// Memory bounds it: x in and y out.  A thread takes a few neighbouring channels and a run of
// tokens, and keeps the last W - 1 inputs (and, backwards, gradients) in registers, so that
// within a run everything is read once; W - 1 tokens are read again where runs meet.
#include <algorithm>

#include "seq_ops.h"

namespace pnr {
namespace {

constexpr int kRun = 32;           // tokens of a thread


struct ConvArgs {
  Conv a;
  int cols, lanes, runs;           // groups of channels; of them in a block's row of threads; runs of a row
  int64_t blocks;                  // of the whole problem
  int col_blocks, run_blocks;
  const void* s_in;
  void *y, *s_out;
  // backward
  const void *gy, *gs_out;
  void* gx;
  float* part;                     // [B * runs, W + 1, E]
};

// kV neighbouring values at row t of a [B, T, E] operand.
template <typename T, int kV>
__device__ __forceinline__ void load_values(const T* p, float (&v)[kV]) {
  T raw[kV];
  __builtin_memcpy(raw, __builtin_assume_aligned(p, sizeof(raw)), sizeof(raw));
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    if constexpr (sizeof(T) == 2)
      v[k] = bf16_to_f32(raw[k]);
    else
      v[k] = raw[k];
  }
}
template <typename T, int kV>
__device__ __forceinline__ void store_values(T* p, const float (&v)[kV]) {
  T raw[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) Elem<sizeof(T) == 2>::store(&raw[k], v[k]);
  __builtin_memcpy(__builtin_assume_aligned(p, sizeof(raw)), raw, sizeof(raw));
}

// The inputs of a row, from position -(W - 1) on: the state's before token 0.
template <typename T, int kV, bool kKept>
struct Inputs {
  const T* x;
  const int8_t* codes;
  const uint8_t* exps;
  const T* s;                      // state_in or nullptr
  int64_t st;
  int E, blocks, W;
  __device__ __forceinline__ void get(int t, float (&v)[kV]) const {
    if (t >= 0) {
      if constexpr (kKept) {
        int8_t q[kV];
        __builtin_memcpy(q, __builtin_assume_aligned(codes + (int64_t)t * E, kV), kV);
        const int e = exps[(int64_t)t * blocks];
#pragma unroll
        for (int k = 0; k < kV; ++k) v[k] = unpack_code(q[k], e);
      } else {
        load_values<T, kV>(x + t * st, v);
      }
    } else if (s) {
      load_values<T, kV>(s + (int64_t)(t + W - 1) * E, v);
    } else {
#pragma unroll
      for (int k = 0; k < kV; ++k) v[k] = 0.0f;
    }
  }
};

template <typename T, int kV, bool kKept>
__device__ __forceinline__ Inputs<T, kV, kKept> inputs(const Conv& a, const void* s_in, int b, int c) {
  Inputs<T, kV, kKept> in{};
  in.E = a.E, in.W = a.W, in.st = a.x.st, in.blocks = (a.E + kPackBlock - 1) / kPackBlock;
  in.s = s_in ? (const T*)s_in + (int64_t)b * (a.W - 1) * a.E + c : nullptr;
  if constexpr (kKept) {
    in.codes = (const int8_t*)a.x.p + b * a.x.sb + c;
    in.exps = a.exps + (int64_t)b * a.T * in.blocks + c / kPackBlock;
  } else {
    in.x = (const T*)a.x.p + b * a.x.sb + c;
  }
  return in;
}

// The work of a thread: its first channel, row and run; false where it has none.
struct Place {
  int b, run, c;
};
template <int kV>
__device__ __forceinline__ bool place(const ConvArgs& p, int64_t block, Place& w) {
  const int cb = (int)(block % p.col_blocks);
  const int64_t rest = block / p.col_blocks;
  const int per = 256 / p.lanes, col = cb * p.lanes + threadIdx.x % p.lanes;
  w.run = (int)(rest % p.run_blocks) * per + threadIdx.x / p.lanes;
  w.b = (int)(rest / p.run_blocks);
  w.c = col * kV;
  return col < p.cols && w.run < p.runs;
}

template <typename T, int kV, int W, bool kKept>
__global__ void __launch_bounds__(256) forward_kernel(ConvArgs p) {
  const Conv& a = p.a;
  for (int64_t block = blockIdx.x; block < p.blocks; block += gridDim.x) {
    Place w;
    if (!place<kV>(p, block, w)) continue;
    const int n = row_len(a.lens, w.b, a.T), t0 = w.run * kRun, t1 = min(t0 + kRun, a.T);
    const auto in = inputs<T, kV, kKept>(a, p.s_in, w.b, w.c);
    float wt[W][kV], bias[kV], x[W][kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      bias[k] = a.bias ? a.bias[w.c + k] : 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) wt[j][k] = a.weight[(int64_t)(w.c + k) * W + j];
    }
    T* y = (T*)p.y + (int64_t)w.b * a.T * a.E + w.c;
    const int end = min(t1, n);
    if (t0 < end)
#pragma unroll
      for (int j = 0; j < W - 1; ++j) in.get(t0 - (W - 1) + j, x[j]);
    for (int t = t0; t < end; ++t) {
      in.get(t, x[W - 1]);
      float o[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        float s = bias[k];
#pragma unroll
        for (int j = 0; j < W; ++j) s += wt[j][k] * x[j][k];
        o[k] = a.silu ? s * sigm(s) : s;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) x[j][k] = x[j + 1][k];
      }
      store_values<T, kV>(y + (int64_t)t * a.E, o);
    }
    float zero[kV] = {};
    for (int t = max(t0, end); t < t1; ++t) store_values<T, kV>(y + (int64_t)t * a.E, zero);
    if (p.s_out && w.run == 0) {           // the last W - 1 inputs, read again: at most seven tokens
      T* out = (T*)p.s_out + (int64_t)w.b * (W - 1) * a.E + w.c;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        float v[kV];
        in.get(n - (W - 1) + j, v);
        store_values<T, kV>(out + (int64_t)j * a.E, v);
      }
    }
  }
}

// SiLU's derivative.
__device__ __forceinline__ float silu_slope(float p) {
  const float s = sigm(p);
  return s * (1.0f + p * (1.0f - s));
}

template <typename T, int kV, int W, bool kKept>
__global__ void __launch_bounds__(256) backward_kernel(ConvArgs p) {
  const Conv& a = p.a;
  for (int64_t block = blockIdx.x; block < p.blocks; block += gridDim.x) {
    Place w;
    if (!place<kV>(p, block, w)) continue;
    const int n = row_len(a.lens, w.b, a.T), t0 = w.run * kRun, t1 = min(t0 + kRun, a.T);
    const auto in = inputs<T, kV, kKept>(a, p.s_in, w.b, w.c);
    float wt[W][kV], bias[kV], x[W][kV], g[W][kV], gw[W][kV], gb[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      bias[k] = a.bias ? a.bias[w.c + k] : 0.0f;
      gb[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) wt[j][k] = a.weight[(int64_t)(w.c + k) * W + j], g[j][k] = gw[j][k] = 0.0f;
    }
    const T* gy = (const T*)p.gy + (int64_t)w.b * a.T * a.E + w.c;
    const T* gs = p.gs_out ? (const T*)p.gs_out + (int64_t)w.b * (W - 1) * a.E + w.c : nullptr;
    T* gx = p.gx ? (T*)p.gx + (int64_t)w.b * a.T * a.E + w.c : nullptr;
    const int end = min(t1, n);
    if (t0 < end)
#pragma unroll
      for (int j = 0; j < W - 1; ++j) in.get(t0 - (W - 1) + j, x[j]);
    // token t closes the gradient of input t - W + 1
    for (int t = t0; t < (t0 < end ? end + W - 1 : t0); ++t) {
      const bool live = t < n;
      if (live) {
        in.get(t, x[W - 1]);
        load_values<T, kV>(gy + (int64_t)t * a.E, g[W - 1]);
      }
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        float s = bias[k];
#pragma unroll
        for (int j = 0; j < W; ++j) s += wt[j][k] * x[j][k];
        g[W - 1][k] = live ? (a.silu ? g[W - 1][k] * silu_slope(s) : g[W - 1][k]) : 0.0f;
        if (t < end) {
          gb[k] += g[W - 1][k];
#pragma unroll
          for (int j = 0; j < W; ++j) gw[j][k] += g[W - 1][k] * x[j][k];
        }
      }
      const int s = t - (W - 1);
      if (gx && s >= t0) {
        float o[kV];
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          o[k] = 0.0f;
#pragma unroll
          for (int j = 0; j < W; ++j) o[k] += wt[j][k] * g[W - 1 - j][k];
        }
        if (gs && t >= n) {
          float v[kV];
          load_values<T, kV>(gs + (int64_t)(t - n) * a.E, v);
#pragma unroll
          for (int k = 0; k < kV; ++k) o[k] += v[k];
        }
        store_values<T, kV>(gx + (int64_t)s * a.E, o);
      }
#pragma unroll
      for (int k = 0; k < kV; ++k)
#pragma unroll
        for (int j = 0; j < W - 1; ++j) x[j][k] = x[j + 1][k], g[j][k] = g[j + 1][k];
    }
    if (gx) {
      float zero[kV] = {};
      for (int t = max(t0, end); t < t1; ++t) store_values<T, kV>(gx + (int64_t)t * a.E, zero);
    }
    if (p.part) {
      float* part = p.part + ((int64_t)w.b * p.runs + w.run) * (W + 1) * a.E + w.c;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
#pragma unroll
        for (int j = 0; j < W; ++j) part[(int64_t)j * a.E + k] = gw[j][k];
        part[(int64_t)W * a.E + k] = gb[k];
      }
    }
  }
}

// The gradient of the inputs before the first: position i of the state meets tokens i - j, j <= i.
template <typename T, bool kKept>
__global__ void __launch_bounds__(256) state_kernel(ConvArgs p, T* gs_in) {
  const Conv& a = p.a;
  const int W = a.W;
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i >= (int64_t)a.B * (W - 1) * a.E) return;
  const int c = (int)(i % a.E), pos = (int)(i / a.E % (W - 1)), b = (int)(i / a.E / (W - 1));
  const int n = row_len(a.lens, b, a.T);
  const auto in = inputs<T, 1, kKept>(a, p.s_in, b, c);
  const float* wt = a.weight + (int64_t)c * W;
  float o = 0.0f;
  for (int t = 0; t <= min(pos, n - 1); ++t) {
    float s = a.bias ? a.bias[c] : 0.0f, v[1];
    for (int j = 0; j < W; ++j) {
      in.get(t - (W - 1) + j, v);
      s += wt[j] * v[0];
    }
    load_values<T, 1>((const T*)p.gy + ((int64_t)b * a.T + t) * a.E + c, v);
    o += wt[pos - t] * (a.silu ? v[0] * silu_slope(s) : v[0]);
  }
  if (p.gs_out && pos >= n) {
    float v[1];
    load_values<T, 1>((const T*)p.gs_out + ((int64_t)b * (W - 1) + pos - n) * a.E + c, v);
    o += v[0];
  }
  const float v[1] = {o};
  store_values<T, 1>(gs_in + i, v);
}

// The runs' sums, in order: out[e, j] (the weight) and out[e] (the bias).
__global__ void __launch_bounds__(256) sum_kernel(const float* part, int64_t runs, int E, int W, float* gw, float* gb) {
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i >= (int64_t)(W + 1) * E) return;
  const int c = (int)(i % E), j = (int)(i / E);
  float s = 0.0f;
  for (int64_t r = 0; r < runs; ++r) s += part[r * (W + 1) * E + i];
  if (j < W) {
    if (gw) gw[(int64_t)c * W + j] = s;
  } else if (gb) {
    gb[c] = s;
  }
}

template <typename T, int kV, bool kKept>
__global__ void __launch_bounds__(256) step_kernel(ConvArgs p, const int32_t* slots, int n_slots) {
  const Conv& a = p.a;
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i >= (int64_t)a.B * p.cols) return;
  const int b = (int)(i / p.cols), c = (int)(i % p.cols) * kV;
  const int slot = slots ? slots[b] : b;
  float o[kV] = {};
  if (slot >= 0 && slot < n_slots) {
    const T* s = (const T*)p.s_in + (int64_t)slot * (a.W - 1) * a.E + c;
    T* out = (T*)p.s_out + (int64_t)slot * (a.W - 1) * a.E + c;
    float x[kMaxTaps][kV];
    load_values<T, kV>((const T*)a.x.p + b * a.x.sb + c, x[kMaxTaps - 1]);
#pragma unroll
    for (int j = 1; j < kMaxTaps; ++j)         // x[7 - j]: the input j tokens back
      if (j < a.W) load_values<T, kV>(s + (int64_t)(a.W - 1 - j) * a.E, x[kMaxTaps - 1 - j]);
#pragma unroll
    for (int k = 0; k < kV; ++k) o[k] = a.bias ? a.bias[c + k] : 0.0f;
#pragma unroll
    for (int j = kMaxTaps - 1; j >= 0; --j)
      if (j < a.W) {
#pragma unroll
        for (int k = 0; k < kV; ++k) o[k] += a.weight[(int64_t)(c + k) * a.W + a.W - 1 - j] * x[kMaxTaps - 1 - j][k];
        if (j + 1 < a.W) store_values<T, kV>(out + (int64_t)(a.W - 2 - j) * a.E, x[kMaxTaps - 1 - j]);
      }
    if (a.silu)
#pragma unroll
      for (int k = 0; k < kV; ++k) o[k] *= sigm(o[k]);
  }
  store_values<T, kV>((T*)p.y + (int64_t)b * a.E + c, o);
}

ConvArgs arguments(const Conv& a, int kV) {
  ConvArgs p{};
  p.a = a;
  p.cols = a.E / kV;
  p.lanes = 1;
  while (p.lanes < 256 && p.lanes < p.cols) p.lanes *= 2;
  p.runs = std::max(1, (int)(((int64_t)a.T + kRun - 1) / kRun));
  p.col_blocks = (p.cols + p.lanes - 1) / p.lanes;
  const int per = 256 / p.lanes;
  p.run_blocks = (p.runs + per - 1) / per;
  p.blocks = (int64_t)a.B * p.run_blocks * p.col_blocks;
  return p;
}

constexpr int64_t kMaxBlocks = 1 << 22;
unsigned grid(int64_t blocks) { return (unsigned)std::min(blocks, kMaxBlocks); }

template <typename T, int kV, bool kKept, bool kBack>
hipError_t launch_taps(const ConvArgs& p, hipStream_t st) {
#define PNR_TAPS(w)                                                              \
  case w:                                                                        \
    if constexpr (kBack)                                                         \
      backward_kernel<T, kV, w, kKept><<<grid(p.blocks), 256, 0, st>>>(p);        \
    else                                                                         \
      forward_kernel<T, kV, w, kKept><<<grid(p.blocks), 256, 0, st>>>(p);         \
    break;
  switch (p.a.W) {
    PNR_TAPS(1) PNR_TAPS(2) PNR_TAPS(3) PNR_TAPS(4) PNR_TAPS(5) PNR_TAPS(6) PNR_TAPS(7) PNR_TAPS(8)
  }
#undef PNR_TAPS
  return hipGetLastError();
}

// Channels of a thread: 16 bytes of the element type (8 or 4), where every operand is aligned to them.
template <typename F>
hipError_t by_type(const Conv& a, bool vec, F&& f) {
  if (a.bf16) {
    if (a.exps) return vec ? f(uint16_t{}, std::integral_constant<int, 8>{}, std::true_type{}) : f(uint16_t{}, std::integral_constant<int, 1>{}, std::true_type{});
    return vec ? f(uint16_t{}, std::integral_constant<int, 8>{}, std::false_type{}) : f(uint16_t{}, std::integral_constant<int, 1>{}, std::false_type{});
  }
  if (a.exps) return vec ? f(float{}, std::integral_constant<int, 4>{}, std::true_type{}) : f(float{}, std::integral_constant<int, 1>{}, std::true_type{});
  return vec ? f(float{}, std::integral_constant<int, 4>{}, std::false_type{}) : f(float{}, std::integral_constant<int, 1>{}, std::false_type{});
}

bool vectors(const Conv& a, std::initializer_list<const void*> ptrs) {
  const int es = a.bf16 ? 2 : 4, v = 16 / es;
  bool ok = a.E % v == 0;
  if (a.exps)
    ok = ok && (uintptr_t)a.x.p % v == 0;
  else
    ok = ok && (uintptr_t)a.x.p % 16 == 0 && a.x.sb * es % 16 == 0 && a.x.st * es % 16 == 0;
  for (const void* p : ptrs) ok = ok && (uintptr_t)p % 16 == 0;
  return ok;
}

}  // namespace

hipError_t launch_conv_forward(const Conv& a, const void* state_in, void* y, void* state_out, hipStream_t st) {
  return by_type(a, vectors(a, {state_in, y, state_out}), [&](auto t, auto v, auto kept) {
    ConvArgs p = arguments(a, v);
    p.s_in = state_in, p.y = y, p.s_out = state_out;
    return launch_taps<decltype(t), v, kept, false>(p, st);
  });
}

hipError_t launch_conv_step(const Conv& a, const void* state_in, const int32_t* slots, int n_slots, void* y,
                            void* state_out, hipStream_t st) {
  return by_type(a, vectors(a, {state_in, y, state_out}), [&](auto t, auto v, auto kept) {
    ConvArgs p = arguments(a, v);
    p.s_in = state_in, p.y = y, p.s_out = state_out;
    if constexpr (!kept)
      step_kernel<decltype(t), v, false><<<(unsigned)(((int64_t)a.B * p.cols + 255) / 256), 256, 0, st>>>(p, slots, n_slots);
    return hipGetLastError();
  });
}

size_t conv_workspace_backward(const Conv& a) {
  const int64_t runs = std::max<int64_t>(1, ((int64_t)a.T + kRun - 1) / kRun);
  return ((size_t)a.B * runs * (a.W + 1) * a.E * 4 + 255) / 256 * 256;
}

hipError_t launch_conv_backward(const Conv& a, const void* state_in, const void* gy, const void* gstate_out, void* gx,
                                float* gw, float* gb, void* gstate_in, char* ws, hipStream_t st) {
  return by_type(a, vectors(a, {state_in, gy, gstate_out, gx}), [&](auto t, auto v, auto kept) {
    ConvArgs p = arguments(a, v);
    p.s_in = state_in, p.gy = gy, p.gs_out = gstate_out, p.gx = gx;
    p.part = gw || gb ? (float*)ws : nullptr;
    if (gx || p.part) {
      if (hipError_t e = launch_taps<decltype(t), v, kept, true>(p, st)) return e;
    }
    if (p.part)
      sum_kernel<<<(unsigned)(((int64_t)(a.W + 1) * a.E + 255) / 256), 256, 0, st>>>(p.part, (int64_t)a.B * p.runs, a.E, a.W, gw, gb);
    if (gstate_in && a.W > 1)
      state_kernel<decltype(t), kept><<<(unsigned)(((int64_t)a.B * (a.W - 1) * a.E + 255) / 256), 256, 0, st>>>(p, (decltype(t)*)gstate_in);
    return hipGetLastError();
  });
}

}  // namespace pnr
