// Group norm with an activation, channels last, and its gradients.
//   n = (x - mean) rstd,  z = n w + b,  y = act(z)  or  z act(gate)
//   dz = dy act'(z)  or  dy act(gate);   dgate = dy z act'(gate)
//   u = dz w,  dx = rstd (u - mean(u) - n mean(u n)),  dw = sum dz n,  db = sum dz
//
// Two layouts of the work, both bound by memory:
//   tokens (L = 1, groups of up to some thousand channels): a group is one contiguous run that
//     1..64 lanes hold in registers, so x, the gate and dy are read once and the sums are wave
//     shuffles.  A thread keeps its channels over all its tokens: weight and bias are
//     loaded once, and dw and db are sums in registers until the block's end.
//   maps (L > 1, or wider groups): the rows of a map are cut into slabs of whole lines, a block
//     a slab and a range of channels: a pass for the sums, a pass for the outputs, which
//     finds x in the last-level cache where the tensor fits it.
// Variances come from deviations (two passes over registers, or running means that are joined by
// their counts), never from a difference of sums of squares.  All of it is fp32 up to
// the one rounding of each output.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "seq_ops.h"

namespace pnr {
namespace {

// ---- activations -----------------------------------------------------------------------------
__device__ __forceinline__ float sigmoid(float u) { return __builtin_amdgcn_rcpf(1.0f + __expf(-u)); }

// gelu(u) = u sigmoid(2 a), a = sqrt(2/pi) (u + 0.044715 u^3): 0.5 (1 + tanh a) = sigmoid(2 a)
__device__ __forceinline__ float gelu_arg(float u) { return 1.5957691216057308f * u * fmaf(0.044715f * u, u, 1.0f); }

template <int V>
__device__ __forceinline__ void act_values(int act, float (&u)[V]) {
  if (act == PNR_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] *= sigmoid(u[i]);
  } else if (act == PNR_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] *= sigmoid(gelu_arg(u[i]));
  }
}

// u -> act(u), d = act'(u)
template <int V>
__device__ __forceinline__ void act_grads(int act, float (&u)[V], float (&d)[V]) {
  if (act == PNR_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = sigmoid(u[i]);
      u[i] *= s;
      d[i] = fmaf(u[i], 1.0f - s, s);
    }
  } else if (act == PNR_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // from |u| = 16 on s is 0 or 1: cut there, the slope's cube stays finite under a factor of zero
      const float s = sigmoid(gelu_arg(u[i])), v = __builtin_amdgcn_fmed3f(u[i], -16.0f, 16.0f);
      const float da = 1.5957691216057308f * fmaf(0.134145f * v, v, 1.0f);
      u[i] *= s;
      d[i] = fmaf(v * s * da, 1.0f - s, s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 1.0f;
  }
}

// ---- pieces: V neighbouring channels, one 16-byte access (V = 8 bf16, 4 fp32) or one element -------
template <bool kBf16, bool kVec>
struct Piece {
  using E = Elem<kBf16>;
  using T = typename E::type;
  static constexpr int V = kVec ? (kBf16 ? 8 : 4) : 1;
  using Raw = typename std::conditional<kVec, uint4, T>::type;
  static __device__ __forceinline__ Raw raw(const void* p, size_t at) { return *(const Raw*)((const T*)p + at); }
  static __device__ __forceinline__ void load(const void* p, size_t at, float (&f)[V]) { unpack(raw(p, at), f); }
  static __device__ __forceinline__ void unpack(const Raw& w, float (&f)[V]) {
    if constexpr (!kVec) {
      f[0] = E::load(&w);
    } else {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kBf16) {
          f[2 * i] = __uint_as_float(u[i] << 16);
          f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        } else {
          f[i] = __uint_as_float(u[i]);
        }
      }
    }
  }
  static __device__ __forceinline__ void store(void* p, size_t at, const float (&f)[V]) {
    T* d = (T*)p + at;
    if constexpr (!kVec) {
      E::store(d, f[0]);
    } else {
      T v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (kBf16) v[i] = f32_to_bf16(f[i]); else v[i] = f[i];
      }
      uint4 w;
      __builtin_memcpy(&w, v, 16);
      *(uint4*)d = w;
    }
  }
};

template <int V>
__device__ __forceinline__ void load_params(const float* p, int c, float missing, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = p ? p[c + i] : missing;
}

// dy -> dz, and with a gate dgate -> gate; z -> unspecified
template <int V>
__device__ __forceinline__ void back_through_act(int act, bool gated, float (&dy)[V], float (&z)[V], float (&gate)[V]) {
  float d[V];
  if (gated) {
    act_grads(act, gate, d);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float a = gate[i];
      gate[i] = dy[i] * z[i] * d[i];
      dy[i] *= a;
    }
  } else {
    act_grads(act, z, d);
#pragma unroll
    for (int i = 0; i < V; ++i) dy[i] *= d[i];
  }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int d = 1; d < lanes; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// ---- tokens ------------------------------------------------------------------------------------
struct TokenPlan {
  int lanes;       // lanes a group
  int ppl;         // pieces a lane: 1, 2, 4 or 8; 0: the group is too wide
  int gb, nb;      // groups, and tokens, a block holds at a time
};
TokenPlan token_plan(int W, int groups, int V, int threads) {
  TokenPlan t{};
  const int pieces = (W + V - 1) / V;
  if (W % V || pieces > 512) return t;
  t.lanes = 1;
  while (t.lanes < pieces && t.lanes < 64) t.lanes *= 2;
  t.ppl = 1;
  while (t.ppl * t.lanes < pieces) t.ppl *= 2;
  t.gb = groups < threads / t.lanes ? groups : threads / t.lanes;
  t.nb = threads / (t.lanes * t.gb);
  return t;
}

struct TokenArgs {
  Norm a;
  TokenPlan t;
  void* y;                    // forward
  float *mean, *rstd;
  const void* gy;             // backward
  const float *mean_in, *rstd_in;
  void *gx, *ggate;
  float* part;                // [gridDim.x][2][C]: sums of dz n and of dz, or nullptr
};

// x and the gate are read once: 32768 tokens of 2048 channels in 16 groups, bf16 with a gate, 82 us
// for 403 MB, 4.9 TB/s (a copy's rate); 8 tokens 4.1 us, the launch and one trip to memory.
template <bool kBf16, bool kVec, int PPL>
__global__ void __launch_bounds__(256) token_kernel(TokenArgs p) {
  using P = Piece<kBf16, kVec>;
  constexpr int V = P::V;
  const Norm& a = p.a;
  const int W = a.C / a.groups, lanes = p.t.lanes;
  const int sub = threadIdx.x % lanes, slot = threadIdx.x / lanes;
  const int g = blockIdx.y * p.t.gb + slot % p.t.gb, ns = slot / p.t.gb;
  const bool mine = ns < p.t.nb && g < a.groups;
  const float inv = 1.0f / W;
  float w[PPL][V], b[PPL][V];
#pragma unroll
  for (int k = 0; k < PPL; ++k) {
    const int c = (sub + k * lanes) * V;
    const bool in = mine && c < W;
    load_params<V>(in ? a.weight : nullptr, g * W + c, 1.0f, w[k]);
    load_params<V>(in ? a.bias : nullptr, g * W + c, 0.0f, b[k]);
  }
  for (int64_t n0 = (int64_t)blockIdx.x * p.t.nb; n0 < a.N; n0 += (int64_t)gridDim.x * p.t.nb) {
    const int64_t n = n0 + ns;
    const bool there = mine && n < a.N, live = there && (!a.lens || a.lens[n] > 0);
    const size_t base = (size_t)n * a.C + (size_t)g * W;
    float x[PPL][V], gate[PPL][V];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      const int c = (sub + k * lanes) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) x[k][i] = gate[k][i] = 0.0f;
      if (live && c < W) {
        P::load(a.x, base + c, x[k]);
        if (a.gate) P::load(a.gate, base + c, gate[k]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) s += x[k][i];
    }
    const float mean = lanes_sum(s, lanes) * inv;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < PPL; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[k][i] -= mean;
        s += (sub + k * lanes) * V < W ? x[k][i] * x[k][i] : 0.0f;
      }
    const float rstd = 1.0f / sqrtf(fmaf(lanes_sum(s, lanes), inv, a.eps));
    if (there && sub == 0) {
      if (p.mean) p.mean[n * a.groups + g] = mean;
      if (p.rstd) p.rstd[n * a.groups + g] = rstd;
    }
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      const int c = (sub + k * lanes) * V;
      if (!there || c >= W) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) x[k][i] = fmaf(x[k][i] * rstd, w[k][i], b[k][i]);
      if (a.gate) {
        act_values(a.act, gate[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) x[k][i] *= gate[k][i];
      } else {
        act_values(a.act, x[k]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) x[k][i] = live ? x[k][i] : 0.0f;
      P::store(p.y, base + c, x[k]);
    }
  }
}

// The same tokens: 130 us for 671 MB, 5.2 TB/s.
template <bool kBf16, bool kVec, int PPL, int kThreads>
__global__ void __launch_bounds__(kThreads) token_grad_kernel(TokenArgs p) {
  using P = Piece<kBf16, kVec>;
  constexpr int V = P::V;
  const Norm& a = p.a;
  const int W = a.C / a.groups, lanes = p.t.lanes;
  const int sub = threadIdx.x % lanes, slot = threadIdx.x / lanes;
  const int g = blockIdx.y * p.t.gb + slot % p.t.gb, ns = slot / p.t.gb;
  const bool mine = ns < p.t.nb && g < a.groups;
  const float inv = 1.0f / W;
  float w[PPL][V], b[PPL][V], dw[PPL][V], db[PPL][V];
#pragma unroll
  for (int k = 0; k < PPL; ++k) {
    const int c = (sub + k * lanes) * V;
    const bool in = mine && c < W;
    load_params<V>(in ? a.weight : nullptr, g * W + c, 1.0f, w[k]);
    load_params<V>(in ? a.bias : nullptr, g * W + c, 0.0f, b[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = db[k][i] = 0.0f;
  }
  for (int64_t n0 = (int64_t)blockIdx.x * p.t.nb; n0 < a.N; n0 += (int64_t)gridDim.x * p.t.nb) {
    const int64_t n = n0 + ns;
    const bool there = mine && n < a.N, live = there && (!a.lens || a.lens[n] > 0);
    const size_t base = (size_t)n * a.C + (size_t)g * W;
    const float mean = live ? p.mean_in[n * a.groups + g] : 0.0f, rstd = live ? p.rstd_in[n * a.groups + g] : 0.0f;
    float h[PPL][V], gy[PPL][V], gate[PPL][V];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      const int c = (sub + k * lanes) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) h[k][i] = mean, gy[k][i] = gate[k][i] = 0.0f;
      if (live && c < W) {
        P::load(a.x, base + c, h[k]);
        P::load(p.gy, base + c, gy[k]);
        if (a.gate) P::load(a.gate, base + c, gate[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      float z[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[k][i] = (h[k][i] - mean) * rstd;
        z[i] = fmaf(h[k][i], w[k][i], b[k][i]);
      }
      back_through_act(a.act, a.gate != nullptr, gy[k], z, gate[k]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dw[k][i] = fmaf(gy[k][i], h[k][i], dw[k][i]);
        db[k][i] += gy[k][i];
        gy[k][i] *= w[k][i];
        s1 += gy[k][i];
        s2 = fmaf(gy[k][i], h[k][i], s2);
      }
    }
    s1 = lanes_sum(s1, lanes) * inv;
    s2 = lanes_sum(s2, lanes) * inv;
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      const int c = (sub + k * lanes) * V;
      if (!there || c >= W) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // a row without positions: zeros, also under a weight or a bias that is not finite
        h[k][i] = live ? rstd * (gy[k][i] - s1 - h[k][i] * s2) : 0.0f;
        gate[k][i] = live ? gate[k][i] : 0.0f;
      }
      if (p.gx) P::store(p.gx, base + c, h[k]);
      if (p.ggate) P::store(p.ggate, base + c, gate[k]);
    }
  }
  if (!p.part) return;
  // the block's tokens of a channel meet in LDS, in the order of their slots
  __shared__ float red[kThreads * V];
  float* out = p.part + (size_t)blockIdx.x * 2 * a.C;
  const int width = p.t.gb * lanes;            // threads that hold one token
#pragma unroll
  for (int k = 0; k < PPL; ++k)
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) red[threadIdx.x * V + i] = which ? db[k][i] : dw[k][i];
      __syncthreads();
      const int c = (sub + k * lanes) * V;
      if (mine && ns == 0 && c < W)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float s = 0.0f;
          for (int m = 0; m < p.t.nb; ++m) s += red[(threadIdx.x + m * width) * V + i];
          out[(size_t)which * a.C + g * W + c + i] = s;
        }
    }
}

// dw, db: sums of [rows][2][C] over the rows, added to what is there (more) or in its place; 32 channels a
// block, 32 runs of rows joined in order.
// 256 rows of 2048 channels: 4.8 us.
__global__ void __launch_bounds__(1024) param_sum_kernel(const float* part, int64_t rows, int C, bool more, float* gw, float* gb) {
  __shared__ float red[32][32];
  const int i = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  float s = 0.0f;
  if (i < 2 * C)
#pragma unroll 8
    for (int64_t r = run; r < rows; r += 32) s += part[r * 2 * C + i];
  red[run][threadIdx.x & 31] = s;
  __syncthreads();
  if (run == 0 && i < 2 * C) {
#pragma unroll
    for (int k = 1; k < 32; ++k) s += red[k][threadIdx.x];
    float* out = i < C ? gw + i : gb + (i - C);
    if (i < C ? gw : gb) *out = more ? *out + s : s;
  }
}

// ---- maps --------------------------------------------------------------------------------------
struct MapPlan {
  int tile;        // channels a block: whole groups, or (single) one wide group
  int single;
  int ct, rt;      // threads along channels and along rows
  int ctiles, nsplit, rows;   // blocks along channels and rows, rows a block
};
MapPlan map_plan(const Norm& a, int V) {
  MapPlan m{};
  const int W = a.C / a.groups;
  int lcm = W;
  while (lcm % V) lcm += W;                    // at most V steps
  m.single = lcm > 256 * V;
  if (m.single) {
    m.tile = W;
    m.ct = 256, m.rt = 1;
  } else {
    m.tile = 256 * V / lcm * lcm;
    if (m.tile > a.C) m.tile = a.C;
    m.ct = m.tile / V, m.rt = 256 / m.ct;
  }
  m.ctiles = (a.C + m.tile - 1) / m.tile;
  // about four blocks a CU, of eight rows a thread at least
  int64_t split = 1024 / ((int64_t)a.N * m.ctiles);
  const int64_t most = a.L / (8 * m.rt);
  if (split > most) split = most;
  if (split > 64) split = 64;
  if (split < 1) split = 1;
  m.rows = (int)((a.L + split - 1) / split);
  m.nsplit = m.rows > 0 ? (a.L - 1) / m.rows + 1 : 1;
  return m;
}
// a map's pieces must not straddle groups where a block holds a single wide one
bool map_vec(const Norm& a, int V) {
  const int W = a.C / a.groups;
  if (a.C % V) return false;
  int lcm = W;
  while (lcm % V) lcm += W;
  return lcm <= 256 * V || W % V == 0;
}

struct MapArgs {
  Norm a;
  MapPlan m;
  float2* stats;              // [N][nsplit][groups]: mean and sum of squared deviations of a slab
  void* y;
  float *mean, *rstd;
  const void* gy;
  const float *mean_in, *rstd_in;
  float* part;                // [N][nsplit][2][C]: sums of dz n and of dz over a slab
  float* chan;                // [N][2][C]: over a row; may be part where there is one slab
  float2* means;              // [N][groups]: mean(u n), mean(u)
  void *gx, *ggate;
};

struct MapBlock {
  int n, split, c0, cols, r0, r1, len;
};
__device__ __forceinline__ MapBlock map_block(const Norm& a, const MapPlan& m) {
  MapBlock k;
  const unsigned id = blockIdx.x;
  k.split = id % m.nsplit;
  k.c0 = id / m.nsplit % m.ctiles * m.tile;
  k.n = id / m.nsplit / m.ctiles;
  k.cols = min(m.tile, a.C - k.c0);
  k.len = row_len(a.lens, k.n, a.L);
  k.r0 = k.split * m.rows;
  k.r1 = min(k.r0 + m.rows, a.L);
  return k;
}

// rows of slab q that belong to the map
__device__ __forceinline__ float slab_rows(const MapBlock& k, const MapPlan& m, int q) {
  return (float)max(min((q + 1) * m.rows, k.len) - q * m.rows, 0);
}

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = lanes_sum(v, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

// 8 maps of 4096 x 320 in bf16, 32 groups: 10 us for 21 MB; too short to fill memory: two trips to it a
// thread, then the joins.
template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(256) map_stats_kernel(MapArgs p) {
  using P = Piece<kBf16, kVec>;
  constexpr int V = P::V;
  const Norm& a = p.a;
  const MapPlan& m = p.m;
  const MapBlock k = map_block(a, m);
  const int W = a.C / a.groups, r1 = min(k.r1, k.len);
  const int ct = threadIdx.x % m.ct, rt = threadIdx.x / m.ct;
  const void* x = a.x;
  const size_t base = (size_t)k.n * a.L * a.C + k.c0;
  __shared__ float2 part[256 * V];
  __shared__ float red[4];
  float2* out = p.stats + ((size_t)k.n * m.nsplit + k.split) * a.groups + k.c0 / W;
  // running mean and squared deviations of the thread's rows, channel by channel
  float mean[V], dev[V], all_mean = 0.0f, all_dev = 0.0f, all_count = 0.0f;
  for (int c = ct * V; c < k.cols; c += m.ct * V) {
    float count = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) mean[i] = dev[i] = 0.0f;
    if (rt < m.rt)
      for (int r = k.r0 + rt; r < r1; r += 8 * m.rt) {
        typename P::Raw w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = P::raw(x, base + (size_t)min(r + q * m.rt, r1 - 1) * a.C + c);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (r + q * m.rt < r1) {
            float f[V];
            P::unpack(w[q], f);
            count += 1.0f;
            const float inv = __builtin_amdgcn_rcpf(count);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float d = f[i] - mean[i];
              mean[i] = fmaf(d, inv, mean[i]);
              dev[i] = fmaf(d, f[i] - mean[i], dev[i]);
            }
          }
      }
    if (m.single && count > 0.0f) {
      // one group: join the channels as they come
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float total = all_count + count, d = mean[i] - all_mean, f = count / total;
        all_dev += dev[i] + d * d * all_count * f;
        all_mean = fmaf(d, f, all_mean);
        all_count = total;
      }
    }
  }
  if (m.single) {
    const float n = (float)(r1 > k.r0 ? r1 - k.r0 : 0) * W;
    const float gm = block_sum(all_mean * all_count, red) / fmaxf(n, 1.0f);
    const float d = all_mean - gm;
    const float gd = block_sum(all_dev + d * d * all_count, red);
    if (threadIdx.x == 0) *out = make_float2(gm, gd);
    return;
  }
  if (rt < m.rt && ct * V < k.cols)
#pragma unroll
    for (int i = 0; i < V; ++i) part[rt * m.tile + ct * V + i] = make_float2(mean[i], dev[i]);
  __syncthreads();
  // a channel's threads, joined by their counts of rows
  const int rows = r1 > k.r0 ? r1 - k.r0 : 0, ng = k.cols / W;
  for (int c = threadIdx.x; c < k.cols; c += 256) {
    float2 all = part[c];
    float count = (float)((rows + m.rt - 1) / m.rt);
    for (int r = 1; r < m.rt && r < rows; ++r) {
      const float more = (float)((rows - r + m.rt - 1) / m.rt), f = more / (count + more);
      const float2 e = part[r * m.tile + c];
      const float d = e.x - all.x;
      all.y += e.y + d * d * count * f;
      all.x = fmaf(d, f, all.x);
      count += more;
    }
    part[c] = all;
  }
  __syncthreads();
  // a group's channels, all of the same count
  int lanes = 64;
  while (lanes > 1 && lanes / 2 >= W) lanes /= 2;
  const int sub = threadIdx.x % lanes;
  for (int g0 = 0; g0 < ng; g0 += 256 / lanes) {
    const int g = g0 + threadIdx.x / lanes, at = min(g, ng - 1) * W;
    float s = 0.0f;
    for (int q = sub; q < W; q += lanes) s += part[at + q].x;
    const float gm = lanes_sum(s, lanes) / W;
    s = 0.0f;
    for (int q = sub; q < W; q += lanes) {
      const float2 e = part[at + q];
      s += e.y + rows * (e.x - gm) * (e.x - gm);
    }
    const float gd = lanes_sum(s, lanes);
    if (g < ng && sub == 0) out[g] = make_float2(gm, gd);
  }
}

// The same maps: 15 us for 42 MB, x out of the last-level cache.
template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(256) map_norm_kernel(MapArgs p) {
  using P = Piece<kBf16, kVec>;
  constexpr int V = P::V;
  const Norm& a = p.a;
  const MapPlan& m = p.m;
  const MapBlock k = map_block(a, m);
  const int W = a.C / a.groups, ng = k.cols / W;
  __shared__ float2 group[256 * V];            // mean and rstd
  // the slabs' means and deviations joined by their counts, several lanes a group
  int lanes = 64;
  while (lanes > 1 && (lanes / 2 >= m.nsplit || lanes * ng > 256)) lanes /= 2;
  const int sub = threadIdx.x % lanes;
  const float total = (float)k.len * W, inv = 1.0f / fmaxf(total, 1.0f);
  for (int g0 = 0; g0 < ng; g0 += 256 / lanes) {
    const int g = g0 + threadIdx.x / lanes;
    const float2* s = p.stats + (size_t)k.n * m.nsplit * a.groups + k.c0 / W + min(g, ng - 1);
    float mean = 0.0f, dev = 0.0f;
#pragma unroll 4
    for (int q = sub; q < m.nsplit; q += lanes) mean += slab_rows(k, m, q) * s[(size_t)q * a.groups].x;
    mean = lanes_sum(mean, lanes) * W * inv;
#pragma unroll 4
    for (int q = sub; q < m.nsplit; q += lanes) {
      const float2 e = s[(size_t)q * a.groups];
      const float rows = slab_rows(k, m, q), d = e.x - mean;
      dev += rows > 0.0f ? e.y + rows * W * d * d : 0.0f;
    }
    const float rstd = 1.0f / sqrtf(fmaf(lanes_sum(dev, lanes), inv, a.eps));
    if (g < ng && sub == 0) {
      group[g] = make_float2(mean, rstd);
      if (k.split == 0) {
        if (p.mean) p.mean[(size_t)k.n * a.groups + k.c0 / W + g] = mean;
        if (p.rstd) p.rstd[(size_t)k.n * a.groups + k.c0 / W + g] = rstd;
      }
    }
  }
  __syncthreads();
  const int ct = threadIdx.x % m.ct, rt = threadIdx.x / m.ct;
  if (rt >= m.rt) return;
  const size_t base = (size_t)k.n * a.L * a.C + k.c0;
  for (int c = ct * V; c < k.cols; c += m.ct * V) {
    float w[V], b[V], mean[V];
    load_params<V>(a.weight, k.c0 + c, 1.0f, w);
    load_params<V>(a.bias, k.c0 + c, 0.0f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 e = group[(c + i) / W];
      mean[i] = e.x;
      w[i] *= e.y;
    }
    constexpr int U = 4;                       // rows in flight
    for (int r = k.r0 + rt; r < k.r1; r += U * m.rt) {
      typename P::Raw w_x[U], w_g[U];
#pragma unroll
      for (int q = 0; q < U; ++q)
        if (r + q * m.rt < min(k.r1, k.len)) {
          const size_t at = base + (size_t)(r + q * m.rt) * a.C + c;
          w_x[q] = P::raw(a.x, at);
          if (a.gate) w_g[q] = P::raw(a.gate, at);
        }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        if (r + q * m.rt >= k.r1) continue;
        float f[V];
        if (r + q * m.rt < k.len) {
          P::unpack(w_x[q], f);
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = fmaf(f[i] - mean[i], w[i], b[i]);
          if (a.gate) {
            float gate[V];
            P::unpack(w_g[q], gate);
            act_values(a.act, gate);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] *= gate[i];
          } else {
            act_values(a.act, f);
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = 0.0f;
        }
        P::store(p.y, base + (size_t)(r + q * m.rt) * a.C + c, f);
      }
    }
  }
}

// Per channel, over a slab: sums of dz n and of dz (kSums); or the gradients of x and the gate.
// 3 maps of 1001 x 330 in fp32: 7.4 us and 7.9 us for 8 MB read and 8 read, 4 written, by single elements
// (rows of 330 are not aligned); launches as short as these are bound by their trips to memory.
template <bool kBf16, bool kVec, bool kSums>
__global__ void __launch_bounds__(256) map_grad_kernel(MapArgs p) {
  using P = Piece<kBf16, kVec>;
  constexpr int V = P::V;
  constexpr int U = 2;                         // rows in flight
  const Norm& a = p.a;
  const MapPlan& m = p.m;
  const MapBlock k = map_block(a, m);
  const int W = a.C / a.groups, r1 = kSums ? min(k.r1, k.len) : k.r1;
  const int ct = threadIdx.x % m.ct, rt = threadIdx.x / m.ct;
  const size_t base = (size_t)k.n * a.L * a.C + k.c0;
  __shared__ float red[kSums ? 256 * V : 1];
  for (int c0 = 0; c0 < k.cols; c0 += m.ct * V) {
    const int c = c0 + ct * V;
    const bool mine = rt < m.rt && c < k.cols;
    float w[V], b[V], mean[V], rstd[V], m1[V], m2[V], dw[V], db[V];
    load_params<V>(mine ? a.weight : nullptr, k.c0 + c, 1.0f, w);
    load_params<V>(mine ? a.bias : nullptr, k.c0 + c, 0.0f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const size_t g = (size_t)k.n * a.groups + (mine ? (k.c0 + c + i) / W : 0);
      mean[i] = p.mean_in[g];
      rstd[i] = p.rstd_in[g];
      dw[i] = db[i] = 0.0f;
      if constexpr (!kSums) {
        const float2 e = p.means[g];
        m2[i] = e.x, m1[i] = e.y;
      }
    }
    if (mine)
      for (int r = k.r0 + rt; r < r1; r += U * m.rt) {
        float x[U][V], gy[U][V], gate[U][V];
#pragma unroll
        for (int q = 0; q < U; ++q)
          if (r + q * m.rt < r1 && r + q * m.rt < k.len) {
            const size_t at = base + (size_t)(r + q * m.rt) * a.C + c;
            P::load(a.x, at, x[q]);
            P::load(p.gy, at, gy[q]);
            if (a.gate) P::load(a.gate, at, gate[q]);
          }
#pragma unroll
        for (int q = 0; q < U; ++q) {
          if (r + q * m.rt >= r1) continue;
          const size_t at = base + (size_t)(r + q * m.rt) * a.C + c;
          if (r + q * m.rt < k.len) {
            float z[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
              x[q][i] = (x[q][i] - mean[i]) * rstd[i];
              z[i] = fmaf(x[q][i], w[i], b[i]);
            }
            back_through_act(a.act, a.gate != nullptr, gy[q], z, gate[q]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              if constexpr (kSums) {
                dw[i] = fmaf(gy[q][i], x[q][i], dw[i]);
                db[i] += gy[q][i];
              } else {
                x[q][i] = rstd[i] * (gy[q][i] * w[i] - m1[i] - x[q][i] * m2[i]);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[q][i] = gate[q][i] = 0.0f;
          }
          if constexpr (!kSums) {
            if (p.gx) P::store(p.gx, at, x[q]);
            if (p.ggate) P::store(p.ggate, at, gate[q]);
          }
        }
      }
    if constexpr (kSums) {
      float* out = p.part + ((size_t)k.n * m.nsplit + k.split) * 2 * a.C + k.c0 + c;
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) red[threadIdx.x * V + i] = which ? db[i] : dw[i];
        __syncthreads();
        if (mine && rt == 0)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float s = 0.0f;
            for (int q = 0; q < m.rt; ++q) s += red[(threadIdx.x + q * m.ct) * V + i];
            out[(size_t)which * a.C + i] = s;
          }
      }
    }
  }
}

// A block a map and group: the slabs' sums of each channel, and from them the group's means.  32
// channels at a time, 8 runs of slabs joined in order.
__global__ void __launch_bounds__(256) map_means_kernel(MapArgs p) {
  const Norm& a = p.a;
  const int W = a.C / a.groups, g = blockIdx.x % a.groups, n = blockIdx.x / a.groups;
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  __shared__ float2 red[8][32];
  float2 group = make_float2(0.0f, 0.0f);
  for (int c0 = 0; c0 < W; c0 += 32) {
    const int c = g * W + c0 + lane;
    const bool in = c0 + lane < W;
    float2 s = make_float2(0.0f, 0.0f);
    if (in)
#pragma unroll 8
      for (int i = run; i < p.m.nsplit; i += 8) {
        const float* q = p.part + ((size_t)n * p.m.nsplit + i) * 2 * a.C + c;
        s.x += q[0];
        s.y += q[a.C];
      }
    __syncthreads();
    red[run][lane] = s;
    __syncthreads();
    if (run == 0 && in) {
#pragma unroll
      for (int k = 1; k < 8; ++k) s.x += red[k][lane].x, s.y += red[k][lane].y;
      p.chan[(size_t)n * 2 * a.C + c] = s.x;
      p.chan[(size_t)n * 2 * a.C + a.C + c] = s.y;
      const float w = a.weight ? a.weight[c] : 1.0f;
      group.x = fmaf(s.x, w, group.x);
      group.y = fmaf(s.y, w, group.y);
    }
  }
  if (threadIdx.x < 64) {
    const float inv = 1.0f / fmaxf((float)row_len(a.lens, n, a.L) * W, 1.0f);
    const float m2 = lanes_sum(group.x, 32) * inv, m1 = lanes_sum(group.y, 32) * inv;
    if (threadIdx.x == 0) p.means[blockIdx.x] = make_float2(m2, m1);
  }
}

// ---- launches --------------------------------------------------------------------------------
bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p % 16) return false;
  return true;
}

// The plan a call takes goes by sizes alone, so that a workspace is enough whatever the pointers: a
// misaligned call is the single-element form of the same plan's layout.
int vec_of(const Norm& a) { return a.bf16 ? 8 : 4; }

// Threads of a token gradient block of ppl pieces a lane: wide blocks leave fewer partial sums of dw
// and db (256 rows of them instead of 768: 5 us instead of 27 for 2048 channels); above two
// pieces a lane they do not have the registers.
constexpr int kGradThreads = 1024;
int grad_threads(int ppl) { return ppl <= 2 ? kGradThreads : 256; }

int token_blocks(const Norm& a, const TokenPlan& t, int per_cu) {
  const int by = (a.groups + t.gb - 1) / t.gb;
  const int64_t need = ((int64_t)a.N + t.nb - 1) / t.nb;
  int64_t bx = 256 * per_cu / by;
  if (bx < 64) bx = 64;
  return (int)(need < bx ? need : bx);
}

template <bool kBf16, bool kVec>
hipError_t run_tokens(const TokenArgs& p, bool grad, int bx, hipStream_t st) {
  const dim3 grid(bx, (p.a.groups + p.t.gb - 1) / p.t.gb);
  auto go = [&](auto ppl) {
    constexpr int K = decltype(ppl)::value;
    constexpr int kWide = K <= 2 ? kGradThreads : 256;
    if (grad)
      token_grad_kernel<kBf16, kVec, K, kWide><<<grid, kWide, 0, st>>>(p);
    else
      token_kernel<kBf16, kVec, K><<<grid, 256, 0, st>>>(p);
  };
  if (p.t.ppl == 1) go(std::integral_constant<int, 1>{});
  else if (p.t.ppl == 2) go(std::integral_constant<int, 2>{});
  else if (p.t.ppl == 4) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 8>{});
  return hipGetLastError();
}

hipError_t run_tokens(const TokenArgs& p, bool vec, bool grad, int bx, hipStream_t st) {
  if (p.a.bf16) return vec ? run_tokens<true, true>(p, grad, bx, st) : run_tokens<true, false>(p, grad, bx, st);
  return vec ? run_tokens<false, true>(p, grad, bx, st) : run_tokens<false, false>(p, grad, bx, st);
}

template <class F>
void with_types(bool bf16, bool vec, F f) {
  if (bf16)
    vec ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
  else
    vec ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Slabs for either access form, so that a workspace does not depend on alignment.
int most_splits(const Norm& a) {
  const int s1 = map_plan(a, 1).nsplit;
  const int sv = map_vec(a, vec_of(a)) ? map_plan(a, vec_of(a)).nsplit : 1;
  return s1 > sv ? s1 : sv;
}

// Maps whose slabs' results, `bytes` a map, a workspace holds at a time.  It stays bounded in the number of maps:
// short maps and wide groups would leave more than their own size (2 or 4 bytes a value, 8 a channel).
// 64 MB, or what eight blocks a CU take where that is more: gradients of 32768 tokens in one group of 8192 channels
// (bf16, a block a token) 1024, 2048 and all tokens at a time: 8.4, 5.4 and 6.8 ms.  32768 maps of 2 x 2048 in
// batches of 64 MB 1.73 ms, all at a time 1.97.
int64_t batch_maps(const Norm& a, size_t bytes) {
  const int V = vec_of(a);
  const int c1 = map_plan(a, 1).ctiles, cv = map_vec(a, V) ? map_plan(a, V).ctiles : c1;
  const int64_t n = (int64_t)(((size_t)64 << 20) / bytes), fill = 2048 / (c1 < cv ? c1 : cv);
  const int64_t most = n > fill ? n : fill;
  return most < 1 ? 1 : most < a.N ? most : a.N;
}
const void* at_map(const Norm& a, const void* p, int64_t n) {
  return p ? (const char*)p + n * a.L * a.C * (a.bf16 ? 2 : 4) : nullptr;
}
void* at_map(const Norm& a, void* p, int64_t n) { return (void*)at_map(a, (const void*)p, n); }
// the problem from map n on
Norm from_map(const Norm& a, int64_t n, int64_t count) {
  Norm b = a;
  b.N = (int)count;
  b.x = at_map(a, a.x, n), b.gate = at_map(a, a.gate, n);
  if (a.lens) b.lens = a.lens + n;
  return b;
}

struct TokenChoice {
  TokenPlan t;
  bool vec;
};
TokenChoice choose_tokens(const Norm& a, bool ok, bool grad) {
  const int W = a.C / a.groups, V = vec_of(a);
  if (a.L != 1) return {{}, false};
  auto plan = [&](int v) {
    const TokenPlan t = token_plan(W, a.groups, v, 256);
    return grad && t.ppl ? token_plan(W, a.groups, v, grad_threads(t.ppl)) : t;
  };
  if (ok) {
    const TokenPlan t = plan(V);
    if (t.ppl) return {t, true};
  }
  return {plan(1), false};
}
// blocks a CU of the token gradient: they bound the partial sums of dw and db
int grad_blocks_per_cu(int ppl) { return ppl <= 2 ? 1 : 3; }
constexpr int kMostGradBlocksPerCu = 3;

size_t stats_bytes(const Norm& a) { return (size_t)most_splits(a) * a.groups * sizeof(float2); }

}  // namespace

size_t groupnorm_workspace(const Norm& a) {
  if (choose_tokens(a, true, false).t.ppl && choose_tokens(a, false, false).t.ppl) return 0;
  return align256(batch_maps(a, stats_bytes(a)) * stats_bytes(a));
}

hipError_t launch_groupnorm(const Norm& a, void* y, float* mean, float* rstd, char* ws, hipStream_t st) {
  const bool ok = all_aligned({a.x, a.gate, y});
  const TokenChoice tc = choose_tokens(a, ok, false);
  if (tc.t.ppl) {
    TokenArgs p{};
    p.a = a, p.t = tc.t, p.y = y, p.mean = mean, p.rstd = rstd;
    return run_tokens(p, tc.vec, false, token_blocks(a, tc.t, 8), st);
  }
  const bool vec = ok && map_vec(a, vec_of(a));
  MapArgs p{};
  p.m = map_plan(a, vec ? vec_of(a) : 1), p.stats = (float2*)ws;
  const int64_t batch = batch_maps(a, stats_bytes(a));
  for (int64_t n = 0; n < a.N; n += batch) {
    p.a = from_map(a, n, batch < a.N - n ? batch : a.N - n);
    p.y = at_map(a, y, n), p.mean = mean ? mean + n * a.groups : nullptr, p.rstd = rstd ? rstd + n * a.groups : nullptr;
    const unsigned grid = (unsigned)p.a.N * p.m.ctiles * p.m.nsplit;
    with_types(a.bf16, vec, [&](auto b, auto v) {
      map_stats_kernel<decltype(b)::value, decltype(v)::value><<<grid, 256, 0, st>>>(p);
      map_norm_kernel<decltype(b)::value, decltype(v)::value><<<grid, 256, 0, st>>>(p);
    });
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

namespace {
struct GradLayout {
  size_t chan = 0, means = 0, total = 0;       // maps: part lies at 0
  int64_t batch = 0;
};
GradLayout grad_layout(const Norm& a) {
  GradLayout l;
  if (a.L == 1) l.total = align256((size_t)256 * kMostGradBlocksPerCu * 2 * a.C * 4);   // token form: partial sums
  if (choose_tokens(a, true, true).t.ppl && choose_tokens(a, false, true).t.ppl) return l;
  // where a map is one slab, the slab's sums are the map's
  const size_t row = (size_t)2 * a.C * 4, slabs = most_splits(a) > 1 ? most_splits(a) * row : 0, groups = a.groups * sizeof(float2);
  l.batch = batch_maps(a, slabs + row + groups);
  l.chan = align256(l.batch * slabs);
  l.means = l.chan + align256(l.batch * row);
  l.total = std::max(l.total, l.means + align256(l.batch * groups));
  return l;
}
}  // namespace

size_t groupnorm_workspace_backward(const Norm& a) { return grad_layout(a).total; }

hipError_t launch_groupnorm_backward(const Norm& a, const void* gy, const float* mean, const float* rstd, void* gx,
                                     float* gw, float* gb, void* ggate, char* ws, hipStream_t st) {
  const GradLayout l = grad_layout(a);
  const bool ok = all_aligned({a.x, a.gate, gy, gx, ggate}), params = gw || gb;
  const TokenChoice tc = choose_tokens(a, ok, true);
  const unsigned sum_blocks = (2 * (unsigned)a.C + 31) / 32;
  if (tc.t.ppl) {
    TokenArgs p{};
    p.a = a, p.t = tc.t, p.gy = gy, p.mean_in = mean, p.rstd_in = rstd, p.gx = gx, p.ggate = ggate;
    if (params) p.part = (float*)ws;
    const int bx = token_blocks(a, tc.t, grad_blocks_per_cu(tc.t.ppl));
    hipError_t e = run_tokens(p, tc.vec, true, bx, st);
    if (e != hipSuccess || !params) return e;
    param_sum_kernel<<<sum_blocks, 1024, 0, st>>>(p.part, bx, a.C, false, gw, gb);
    return hipGetLastError();
  }
  const bool vec = ok && map_vec(a, vec_of(a));
  MapArgs p{};
  p.m = map_plan(a, vec ? vec_of(a) : 1);
  p.part = (float*)ws, p.chan = (float*)(ws + l.chan), p.means = (float2*)(ws + l.means);
  for (int64_t n = 0; n < a.N; n += l.batch) {
    p.a = from_map(a, n, l.batch < a.N - n ? l.batch : a.N - n);
    p.gy = at_map(a, gy, n), p.mean_in = mean + n * a.groups, p.rstd_in = rstd + n * a.groups;
    p.gx = at_map(a, gx, n), p.ggate = at_map(a, ggate, n);
    const unsigned grid = (unsigned)p.a.N * p.m.ctiles * p.m.nsplit;
    with_types(a.bf16, vec, [&](auto b, auto v) {
      constexpr bool kB = decltype(b)::value, kV = decltype(v)::value;
      map_grad_kernel<kB, kV, true><<<grid, 256, 0, st>>>(p);
      map_means_kernel<<<(unsigned)p.a.N * a.groups, 256, 0, st>>>(p);
      if (gx || ggate) map_grad_kernel<kB, kV, false><<<grid, 256, 0, st>>>(p);
    });
    if (params) param_sum_kernel<<<sum_blocks, 1024, 0, st>>>(p.chan, p.a.N, a.C, n > 0, gw, gb);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace pnr
