// Causal convolution along time, each channel by itself:
//   p_t = bias + sum_j w_j x_{t-W+1+j},  y = act(p)
// and its gradients, with g_t = grad_y act'(p_t):
//   dx_s = sum_j w_j g_{s+W-1-j},  dw_j = sum_t g_t x_{t-W+1+j},  db = sum_t g_t
//
// Memory bounds it: x in and y out.  A thread takes a few neighbouring channels and a run of
// tokens, and keeps the last W - 1 inputs (and, backwards, gradients) in registers, so that
// within a run everything is read once; W - 1 tokens are read again where runs meet.
// 4 x 4096 x 4096 bf16, 4 taps, SiLU: forward 57 us (4.7 TB/s), gradients from an 8-bit copy 104 us
// (3.3 TB/s, issue 80 % of the time; 128 registers, four waves a SIMD) and 9 for the sums, as a profiler times the
// kernels; whole calls in a row take 52 and 105, and 112 for gradients from x itself.  Eight channels a
// thread took up to 1.4 times that.
#include <algorithm>
#include <type_traits>

#include "seq_ops.h"

namespace pnr {
namespace {

struct ConvArgs {
  Conv a;
  int cols, lanes, runs, run;      // groups of channels; of them in a block's row of threads; runs of a row; tokens of one
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
  __builtin_memcpy(raw, p, sizeof(raw));
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
  __builtin_memcpy(p, raw, sizeof(raw));
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
  // A token of the row as it lies in memory, and its values.
  struct Raw {
    std::conditional_t<kKept, int8_t, T> v[kV];
    uint8_t e;
  };
  __device__ __forceinline__ Raw raw(int t) const {
    Raw r;
    if constexpr (kKept) {
      __builtin_memcpy(r.v, codes + (int64_t)t * E, kV);
      r.e = exps[(int64_t)t * blocks];
    } else {
      __builtin_memcpy(r.v, x + t * st, sizeof(r.v));
      r.e = 0;
    }
    return r;
  }
  static __device__ __forceinline__ void values(const Raw& r, float (&v)[kV]) {
    const float step = kKept ? unpack_step(r.e) : 0.0f;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      if constexpr (kKept)
        v[k] = r.v[k] * step;
      else
        v[k] = Elem<sizeof(T) == 2>::load(&r.v[k]);
    }
  }
  __device__ __forceinline__ void get(int t, float (&v)[kV]) const {
    if (t >= 0) {
      values(raw(t), v);
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

// The work of a thread: its first channel, row and run; false where it has none.  A row's last thread goes back to
// the last kV channels, some of which its neighbour has too: both write the same values.
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
  w.c = min(col * kV, p.a.E - kV);
  return col < p.cols && w.run < p.runs;
}

// The taps of kV channels, which lie together, and their biases.
template <int kV, int W>
__device__ __forceinline__ void load_taps(const Conv& a, int c, float (&wt)[W][kV], float (&bias)[kV]) {
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    bias[k] = a.bias ? a.bias[c + k] : 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) wt[j][k] = a.weight[(int64_t)(c + k) * W + j];
  }
}

constexpr int kAhead = 2;          // tokens of a step; the next step's are asked for before it

template <typename T, int kV, int W, bool kKept>
__global__ void __launch_bounds__(256) forward_kernel(ConvArgs p) {
  const Conv& a = p.a;
  for (int64_t block = blockIdx.x; block < p.blocks; block += gridDim.x) {
    Place w;
    if (!place<kV>(p, block, w)) continue;
    const int n = row_len(a.lens, w.b, a.T), t0 = w.run * p.run, t1 = min(t0 + p.run, a.T);
    auto in = inputs<T, kV, kKept>(a, p.s_in, w.b, w.c);
    float wt[W][kV], bias[kV], x[W - 1 + kAhead][kV];
    load_taps<kV, W>(a, w.c, wt, bias);
    T* y = (T*)p.y + (int64_t)w.b * a.T * a.E + w.c;
    const int end = min(t1, n);
    if (t0 < end)
#pragma unroll
      for (int j = 0; j < W - 1; ++j) in.get(t0 - (W - 1) + j, x[j]);
    typename decltype(in)::Raw rx[kAhead];
    auto fetch = [&](int t) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) rx[i] = in.raw(min(t + i, end - 1));
    };
    if (t0 < end) fetch(t0);
    for (int t = t0; t < end; t += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) in.values(rx[i], x[W - 1 + i]);
      fetch(t + kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (t + i >= end) break;
        float o[kV];
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          float s = bias[k];
#pragma unroll
          for (int j = 0; j < W; ++j) s = fmaf(wt[j][k], x[i + j][k], s);
          o[k] = a.silu ? s * sigm(s) : s;
        }
        store_values<T, kV>(y + (int64_t)(t + i) * a.E, o);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int k = 0; k < kV; ++k) x[j][k] = x[j + kAhead][k];
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
    const int n = row_len(a.lens, w.b, a.T), t0 = w.run * p.run, t1 = min(t0 + p.run, a.T);
    auto in = inputs<T, kV, kKept>(a, p.s_in, w.b, w.c);
    float wt[W][kV], bias[kV], x[W - 1 + kAhead][kV], g[W - 1 + kAhead][kV], gw[W][kV], gb[kV];
    load_taps<kV, W>(a, w.c, wt, bias);
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      gb[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) gw[j][k] = 0.0f;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) g[j][k] = 0.0f;
    }
    const T* gy = (const T*)p.gy + (int64_t)w.b * a.T * a.E + w.c;
    const T* gs = p.gs_out ? (const T*)p.gs_out + (int64_t)w.b * (W - 1) * a.E + w.c : nullptr;
    T* gx = p.gx ? (T*)p.gx + (int64_t)w.b * a.T * a.E + w.c : nullptr;
    const int end = min(t1, n), stop = t0 < end ? end + W - 1 : t0;
    if (t0 < end)
#pragma unroll
      for (int j = 0; j < W - 1; ++j) in.get(t0 - (W - 1) + j, x[j]);
    // token t closes the gradient of input t - W + 1
    struct Values {
      T v[kV];
    };
    typename decltype(in)::Raw rx[kAhead];
    Values rg[kAhead];
    auto fetch = [&](int t) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = min(min(t + i, stop - 1), n - 1);
        rx[i] = in.raw(at);
        __builtin_memcpy(rg[i].v, gy + (int64_t)at * a.E, sizeof(T) * kV);
      }
    };
    if (t0 < stop) fetch(t0);
    for (int t = t0; t < stop; t += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        in.values(rx[i], x[W - 1 + i]);
#pragma unroll
        for (int k = 0; k < kV; ++k) g[W - 1 + i][k] = Elem<sizeof(T) == 2>::load(&rg[i].v[k]);
      }
      fetch(t + kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const bool live = t + i < min(stop, n), own = t + i < end;
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          float s = bias[k];
#pragma unroll
          for (int j = 0; j < W; ++j) s = fmaf(wt[j][k], x[i + j][k], s);
          const float gp = a.silu ? g[W - 1 + i][k] * silu_slope(s) : g[W - 1 + i][k];
          g[W - 1 + i][k] = live ? gp : 0.0f;
          if (own) {             // no product with zero: tokens behind the run may not be finite
            gb[k] += gp;
#pragma unroll
            for (int j = 0; j < W; ++j) gw[j][k] = fmaf(gp, x[i + j][k], gw[j][k]);
          }
        }
        const int s = t + i - (W - 1);
        if (gx && s >= t0 && t + i < stop) {
          float o[kV] = {};
#pragma unroll
          for (int j = 0; j < W; ++j)
            if (t + i - j < n)   // taps that met tokens
#pragma unroll
              for (int k = 0; k < kV; ++k) o[k] = fmaf(wt[j][k], g[i + W - 1 - j][k], o[k]);
          if (gs && t + i >= n) {
            float v[kV];
            load_values<T, kV>(gs + (int64_t)(t + i - n) * a.E, v);
#pragma unroll
            for (int k = 0; k < kV; ++k) o[k] += v[k];
          }
          store_values<T, kV>(gx + (int64_t)s * a.E, o);
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int k = 0; k < kV; ++k) x[j][k] = x[j + kAhead][k], g[j][k] = g[j + kAhead][k];
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

// The runs' sums: out[e, j] (the weight) and out[e] (the bias).  32 values a block, eight threads a value, which
// meet in order.
__global__ void __launch_bounds__(256) sum_kernel(const float* part, int64_t runs, int E, int W, float* gw, float* gb) {
  __shared__ float sums[8][32];
  const int col = threadIdx.x % 32, group = threadIdx.x / 32;
  const int64_t n = (int64_t)(W + 1) * E, i = blockIdx.x * (int64_t)32 + col;
  float s = 0.0f;
  if (i < n)
#pragma unroll 8
    for (int64_t r = group; r < runs; r += 8) s += part[r * n + i];
  sums[group][col] = s;
  __syncthreads();
  if (group || i >= n) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s += sums[k][col];
  const int c = (int)(i % E), j = (int)(i / E);
  if (j < W) {
    if (gw) gw[(int64_t)c * W + j] = s;
  } else if (gb) {
    gb[c] = s;
  }
}

template <typename T, int kV, int W>
__global__ void __launch_bounds__(256) step_kernel(ConvArgs p, const int32_t* slots, int n_slots) {
  const Conv& a = p.a;
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i >= (int64_t)a.B * p.cols) return;
  const int b = (int)(i / p.cols), c = (int)(i % p.cols) * kV;
  const int slot = slots ? slots[b] : b;
  float o[kV] = {};
  if (slot >= 0 && slot < n_slots) {
    const int64_t at = (int64_t)slot * (W - 1) * a.E + c;
    const T* s = (const T*)p.s_in + at;
    T* out = (T*)p.s_out + at;
    float wt[W][kV], bias[kV], x[W][kV];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_values<T, kV>(s + (int64_t)j * a.E, x[j]);
    load_values<T, kV>((const T*)a.x.p + b * a.x.sb + c, x[W - 1]);
    load_taps<kV, W>(a, c, wt, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_values<T, kV>(out + (int64_t)j * a.E, x[j + 1]);
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      float v = bias[k];
#pragma unroll
      for (int j = 0; j < W; ++j) v = fmaf(wt[j][k], x[j][k], v);
      o[k] = a.silu ? v * sigm(v) : v;
    }
  }
  store_values<T, kV>((T*)p.y + (int64_t)b * a.E + c, o);
}

// Tokens of a thread: long runs read few tokens twice and leave few partial sums, short ones fill the device.
// bf16, four taps, us with 16, 32 and 64 tokens: forward 8 x 2000 x 2048 19.4, 22 and 23; 4 x 4096 x 4096 forward 49, 52
// and 51, gradients from x 139, 112 and 112, from an 8-bit copy 133, 105 and 106 (with the sums over runs).
int run_of(const Conv& a) {
  int run = 32;
  while (run > 8 && (int64_t)a.B * ((a.T + run - 1) / run) * (a.E / 4 + 1) < 400000) run /= 2;
  return run;
}

ConvArgs arguments(const Conv& a, int kV) {
  ConvArgs p{};
  p.a = a;
  p.cols = (a.E + kV - 1) / kV;
  p.lanes = 1;
  while (p.lanes < 256 && p.lanes < p.cols) p.lanes *= 2;
  p.run = run_of(a);
  p.runs = std::max(1, (int)(((int64_t)a.T + p.run - 1) / p.run));
  p.col_blocks = (p.cols + p.lanes - 1) / p.lanes;
  const int per = 256 / p.lanes;
  p.run_blocks = (p.runs + per - 1) / per;
  p.blocks = (int64_t)a.B * p.run_blocks * p.col_blocks;
  return p;
}

constexpr int64_t kMaxBlocks = 1 << 22;
unsigned grid(int64_t blocks) { return (unsigned)std::min(blocks, kMaxBlocks); }

// f with the number of taps as a constant.
template <typename F>
hipError_t by_taps(int W, F&& f) {
  switch (W) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 5: f(std::integral_constant<int, 5>{}); break;
    case 6: f(std::integral_constant<int, 6>{}); break;
    case 7: f(std::integral_constant<int, 7>{}); break;
    default: f(std::integral_constant<int, 8>{}); break;
  }
  return hipGetLastError();
}

// f with the element type, the channels of a thread (four, on whatever address they start; with eight
// of them in bf16 the registers left one wave a SIMD: 84 us forward where 71, 222 backward where 156) and
// whether x is an 8-bit copy, as types.
template <typename F>
hipError_t by_type(const Conv& a, bool vec, F&& f) {
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;
  auto kept = [&](auto t, auto v) { return a.exps ? f(t, v, std::true_type{}) : f(t, v, std::false_type{}); };
  if (a.bf16) return vec ? kept(uint16_t{}, Four{}) : kept(uint16_t{}, One{});
  return vec ? kept(float{}, Four{}) : kept(float{}, One{});
}

// Whether a thread takes four channels: an 8-bit copy's last four have to share an exponent then.  4 x 4096 x 4095 bf16,
// us with four and with one a thread: forward 56 and 63, from an 8-bit copy 42 and 60, gradients 124 and 172, from the
// copy 115 and 172.
bool fours(const Conv& a) { return a.E >= 4 && (!a.exps || (a.E - 1) % kPackBlock >= 3); }

}  // namespace

hipError_t launch_conv_forward(const Conv& a, const void* state_in, void* y, void* state_out, hipStream_t st) {
  return by_type(a, fours(a), [&](auto t, auto v, auto kept) {
    ConvArgs p = arguments(a, v);
    p.s_in = state_in, p.y = y, p.s_out = state_out;
    return by_taps(a.W, [&](auto w) { forward_kernel<decltype(t), v, w, kept><<<grid(p.blocks), 256, 0, st>>>(p); });
  });
}

hipError_t launch_conv_step(const Conv& a, const void* state_in, const int32_t* slots, int n_slots, void* y,
                            void* state_out, hipStream_t st) {
  // pools may be updated in place, so no channel is two threads'
  return by_type(a, a.E % 4 == 0, [&](auto t, auto v, auto kept) {
    ConvArgs p = arguments(a, v);
    p.s_in = state_in, p.y = y, p.s_out = state_out;
    const unsigned blocks = (unsigned)(((int64_t)a.B * p.cols + 255) / 256);
    return by_taps(a.W, [&](auto w) {
      if constexpr (!kept) step_kernel<decltype(t), v, w><<<blocks, 256, 0, st>>>(p, slots, n_slots);
    });
  });
}

size_t conv_workspace_backward(const Conv& a) {
  const int run = run_of(a);
  const int64_t runs = std::max<int64_t>(1, ((int64_t)a.T + run - 1) / run);
  return ((size_t)a.B * runs * (a.W + 1) * a.E * 4 + 255) / 256 * 256;
}

hipError_t launch_conv_backward(const Conv& a, const void* state_in, const void* gy, const void* gstate_out, void* gx,
                                float* gw, float* gb, void* gstate_in, char* ws, hipStream_t st) {
  return by_type(a, fours(a), [&](auto t, auto v, auto kept) {
    ConvArgs p = arguments(a, v);
    p.s_in = state_in, p.gy = gy, p.gs_out = gstate_out, p.gx = gx;
    p.part = gw || gb ? (float*)ws : nullptr;
    if (gx || p.part) {
      const hipError_t e = by_taps(a.W, [&](auto w) { backward_kernel<decltype(t), v, w, kept><<<grid(p.blocks), 256, 0, st>>>(p); });
      if (e) return e;
    }
    if (p.part)
      sum_kernel<<<(unsigned)(((int64_t)(a.W + 1) * a.E + 31) / 32), 256, 0, st>>>(p.part, (int64_t)a.B * p.runs, a.E, a.W, gw, gb);
    if (gstate_in && a.W > 1)
      state_kernel<decltype(t), kept><<<(unsigned)(((int64_t)a.B * (a.W - 1) * a.E + 255) / 256), 256, 0, st>>>(p, (decltype(t)*)gstate_in);
    return hipGetLastError();
  });
}

}  // namespace pnr
