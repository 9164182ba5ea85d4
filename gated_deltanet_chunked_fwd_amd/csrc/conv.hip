// The short causal convolution of a token mixer, per channel d:
//   z_t = bias + sum_w weight[d, w] x_{t - W + 1 + w},   y_t = silu(z_t) or z_t,
// inputs before a sequence's first token from its initial state (or zero).  Backward:
//   dz = dy silu'(z) (z formed again from x),  dx_s = sum_w weight[w] dz_{s + W - 1 - w},
//   dweight[w] = sum_t dz_t x_{t - W + 1 + w},  dbias = sum_t dz_t.
//
// Bound by memory.  A thread owns VEC channels (16 bytes) and a run of tokens, with the
// window of inputs (and, going back, of dz) in registers, so every input is read once
// but for W - 1 tokens at the run's edge, which come from the caches.
#include "mixer_device.h"
#include "mixer_launch.h"

namespace gdn {

struct ConvSeq {             // the sequence of one token
  int64_t n, start, end;     // tokens [start, end), flattened over the batch
};
__device__ __forceinline__ ConvSeq conv_seq(const ConvArgs& a, int64_t tok) {
  ConvSeq s;
  if (a.cu) {                // the last n with cu[n] <= tok, so cu[n + 1] > tok
    int lo = 0, hi = a.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= tok) lo = mid; else hi = mid - 1;
    }
    s.n = lo;
    s.start = a.cu[lo];
    s.end = a.cu[lo + 1];
  } else {
    s.n = tok / a.T;
    s.start = s.n * a.T;
    s.end = s.start + a.T;
  }
  return s;
}
__device__ __forceinline__ ConvSeq conv_seq_n(const ConvArgs& a, int64_t n) {
  ConvSeq s;
  s.n = n;
  s.start = a.cu ? (int64_t)a.cu[n] : n * a.T;
  s.end = a.cu ? (int64_t)a.cu[n + 1] : s.start + a.T;
  return s;
}

// The input at a token of the sequence, or before it (from the state).
template <typename E, int VEC, int W>
__device__ __forceinline__ void conv_input(const ConvArgs& a, const ConvSeq& s, int64_t tok, int64_t d, float (&v)[VEC]) {
  if (tok >= s.start) {
    load_vec<E, VEC>(reinterpret_cast<const E*>(a.x) + tok * a.x_stride + d, v);
  } else if (a.init) {
    load_vec<E, VEC>(reinterpret_cast<const E*>(a.init) + (s.n * (W - 1) + (W - 1 + tok - s.start)) * a.D + d, v);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.f;
  }
}

template <int VEC, int W>
struct ConvWeights {
  float w[W][VEC], bias[VEC];
  __device__ __forceinline__ void load(const ConvArgs& a, int64_t d) {
    float raw[VEC * W];
    load_params<VEC * W>(a.w, d * W, a.param_bf16, raw);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[j][i] = raw[i * W + j];
    if (a.bias) load_params<VEC>(a.bias, d, a.param_bf16, bias);
    else
#pragma unroll
      for (int i = 0; i < VEC; ++i) bias[i] = 0.f;
  }
};

// silu'(z) = s (1 + z (1 - s))
__device__ __forceinline__ float dsilu(float z) {
  const float s = sigmoid_f32(z);
  return s * (1.f + z * (1.f - s));
}

template <typename E, int VEC, int W>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, int run, int64_t main_items, int64_t items) {
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (item >= items) return;
  const int64_t DV = a.D / VEC, tokens = a.B * a.T;
  if (item >= main_items) {                // the last W - 1 inputs of every sequence
    const int64_t k = item - main_items;
    const int64_t d = k % DV * VEC, ni = k / DV;
    const ConvSeq s = conv_seq_n(a, ni / (W - 1));
    float v[VEC];
    conv_input<E, VEC, W>(a, s, s.end - (W - 1) + ni % (W - 1), d, v);
    store_vec<E, VEC>(reinterpret_cast<E*>(a.fin) + ni * a.D + d, v);
    return;
  }
  const int64_t d = item % DV * VEC;
  const int64_t t0 = item / DV * run, t1 = min(tokens, t0 + run);
  ConvWeights<VEC, W> cw;
  cw.load(a, d);
  ConvSeq s = conv_seq(a, t0);
  float x[W][VEC];
#pragma unroll
  for (int j = 0; j + 1 < W; ++j) conv_input<E, VEC, W>(a, s, t0 - (W - 1) + j, d, x[j]);
  for (int64_t t = t0; t < t1; ++t) {
    if (t >= s.end) {                      // the next sequence that has tokens
      s = conv_seq(a, t);
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) conv_input<E, VEC, W>(a, s, t - (W - 1) + j, d, x[j]);
    }
    load_vec<E, VEC>(reinterpret_cast<const E*>(a.x) + t * a.x_stride + d, x[W - 1]);
    float y[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float z = cw.bias[i];
#pragma unroll
      for (int j = 0; j < W; ++j) z += cw.w[j][i] * x[j][i];
      y[i] = a.silu ? z * sigmoid_f32(z) : z;
    }
    store_vec<E, VEC>(reinterpret_cast<E*>(a.y) + t * a.D + d, y);
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[j][i] = x[j + 1][i];
  }
}

// dz of one token, from memory (the edges of a run).
template <typename E, int VEC, int W>
__device__ __forceinline__ void conv_dz(const ConvArgs& a, const ConvWeights<VEC, W>& cw, const ConvSeq& s, int64_t t,
                                        int64_t d, float (&dz)[VEC]) {
  load_vec<E, VEC>(reinterpret_cast<const E*>(a.dy) + t * a.D + d, dz);
  if (!a.silu) return;
  float z[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) z[i] = cw.bias[i];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float x[VEC];
    conv_input<E, VEC, W>(a, s, t - (W - 1) + j, d, x);
#pragma unroll
    for (int i = 0; i < VEC; ++i) z[i] += cw.w[j][i] * x[i];
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) dz[i] *= dsilu(z[i]);
}

// Tokens last to first: a workgroup is CL channel lanes x 256 / CL runs of kConvRun tokens, whose
// shares of dweight and dbias it adds up in LDS and writes as one row of `part`.
constexpr int kConvRun = 16;
constexpr int kConvLanes = 64;
constexpr int kConvBlockTokens = kConvRun * (256 / kConvLanes);

template <typename E, int VEC, int W>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a) {
  __shared__ float red[256 / kConvLanes][VEC][kConvLanes];
  const int cl = threadIdx.x % kConvLanes, tr = threadIdx.x / kConvLanes;
  const int64_t DV = a.D / VEC, tokens = a.B * a.T;
  const int64_t cv = (int64_t)blockIdx.x * kConvLanes + cl;
  const bool on = cv < DV;
  const int64_t d = (on ? cv : 0) * VEC;
  const int64_t t0 = (int64_t)blockIdx.y * kConvBlockTokens + tr * kConvRun, t1 = min(tokens, t0 + kConvRun);
  float dw[W][VEC] = {}, db[VEC] = {};
  if (on && t0 < t1) {
    ConvWeights<VEC, W> cw;
    cw.load(a, d);
    ConvSeq s = conv_seq(a, t1 - 1);
    float dz[W][VEC];                      // dz[k] = dz_{t + k}, zero past the sequence's end
    float x[W][VEC];                       // x[j] = x_{t - W + 1 + j}
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) {      // after the shift below: dz[k + 1] = dz_{t1 + k}
      if (t1 + k < s.end) conv_dz<E, VEC, W>(a, cw, s, t1 + k, d, dz[k]);
      else
#pragma unroll
        for (int i = 0; i < VEC; ++i) dz[k][i] = 0.f;
    }
#pragma unroll
    for (int j = 1; j < W; ++j) conv_input<E, VEC, W>(a, s, t1 - 1 - (W - 1) + j, d, x[j - 1]);
    for (int64_t t = t1 - 1; t >= t0; --t) {
      if (t < s.start) {                   // an earlier sequence: nothing flows back into it
        s = conv_seq(a, t);
#pragma unroll
        for (int k = 0; k + 1 < W; ++k)
#pragma unroll
          for (int i = 0; i < VEC; ++i) dz[k][i] = 0.f;
#pragma unroll
        for (int j = 1; j < W; ++j) conv_input<E, VEC, W>(a, s, t - (W - 1) + j, d, x[j - 1]);
      }
#pragma unroll
      for (int j = W - 1; j > 0; --j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          x[j][i] = x[j - 1][i];
          dz[j][i] = dz[j - 1][i];
        }
      conv_input<E, VEC, W>(a, s, t - (W - 1), d, x[0]);
      load_vec<E, VEC>(reinterpret_cast<const E*>(a.dy) + t * a.D + d, dz[0]);
      float dx[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (a.silu) {
          float z = cw.bias[i];
#pragma unroll
          for (int j = 0; j < W; ++j) z += cw.w[j][i] * x[j][i];
          dz[0][i] *= dsilu(z);
        }
        float g = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          g += cw.w[j][i] * dz[W - 1 - j][i];
          dw[j][i] += dz[0][i] * x[j][i];
        }
        db[i] += dz[0][i];
        dx[i] = g;
      }
      if (a.dfin && t >= s.end - (W - 1)) {
        float f[VEC];
        load_vec<E, VEC>(reinterpret_cast<const E*>(a.dfin) + (s.n * (W - 1) + (t - (s.end - (W - 1)))) * a.D + d, f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dx[i] += f[i];
      }
      store_vec<E, VEC>(reinterpret_cast<E*>(a.dx) + t * a.D + d, dx);
    }
  }
  // the workgroup's shares, summed over its runs
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VEC; ++i) red[tr][i][cl] = j < W ? dw[j < W ? j : 0][i] : db[i];
    __syncthreads();
    if (on) {
      // (run, channel) pairs dealt over the runs' threads
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i % (256 / kConvLanes) == tr) {
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < 256 / kConvLanes; ++k) s += red[k][i][cl];
          a.part[((int64_t)blockIdx.y * (W + 1) + j) * a.D + d + i] = s;
        }
    }
  }
}

// Gradient of the initial state: the inputs before a sequence's first token.
template <typename E, int VEC, int W>
__global__ __launch_bounds__(256) void conv_dinit_kernel(ConvArgs a) {
  const int64_t DV = a.D / VEC;
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (item >= (int64_t)a.N * (W - 1) * DV) return;
  const int64_t d = item % DV * VEC, ni = item / DV;
  const ConvSeq s = conv_seq_n(a, ni / (W - 1));
  const int64_t i0 = ni % (W - 1), len = s.end - s.start;
  ConvWeights<VEC, W> cw;
  cw.load(a, d);
  float g[VEC] = {};
#pragma unroll
  for (int w = 0; w < W; ++w) {            // position i0 - (W - 1) meets dz_{i0 - w} with weight w
    if (i0 - w >= 0 && i0 - w < len) {
      float dz[VEC];
      conv_dz<E, VEC, W>(a, cw, s, s.start + i0 - w, d, dz);
#pragma unroll
      for (int i = 0; i < VEC; ++i) g[i] += cw.w[w][i] * dz[i];
    }
  }
  if (a.dfin && i0 >= len) {               // still among the last W - 1 inputs
    float f[VEC];
    load_vec<E, VEC>(reinterpret_cast<const E*>(a.dfin) + (s.n * (W - 1) + i0 - len) * a.D + d, f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] += f[i];
  }
  store_vec<E, VEC>(reinterpret_cast<E*>(a.dinit) + ni * a.D + d, g);
}

__global__ __launch_bounds__(1024) void conv_param_grads_kernel(ConvArgs a, int64_t rows) {
  const int64_t D = a.D;
  const int W = a.W;
  column_sums(a.part, rows, (int64_t)(W + 1) * D, [&](int64_t c, float v) {
    const int64_t j = c / D, d = c % D;
    void* p = j < W ? a.dw : a.dbias;
    if (!p) return;
    const int64_t at = j < W ? d * W + j : d;
    if (a.param_bf16) reinterpret_cast<bf16*>(p)[at] = (bf16)v;
    else reinterpret_cast<float*>(p)[at] = v;
  });
}

int64_t conv_bwd_blocks(int64_t tokens, int64_t D) {
  (void)D;
  return (tokens + kConvBlockTokens - 1) / kConvBlockTokens;
}

// 16-byte accesses need rows that start on 16 bytes: D and x's stride multiples of VEC
// (one channel per thread otherwise).
template <typename E>
static bool conv_vec(const ConvArgs& a) {
  constexpr int V = 16 / (int)sizeof(E);
  return a.D % V == 0 && a.x_stride % V == 0;
}

template <typename E, int VEC, int W>
static hipError_t conv_fwd_run(const ConvArgs& a, hipStream_t s) {
  const int64_t DV = a.D / VEC, tokens = a.B * a.T;
  // runs of 16 tokens read 3 / 16 of the inputs twice (from the caches); when they would not
  // give every CU work, shorter ones
  const int run = tokens * DV >= (int64_t)16 * 256 * 512 ? 16 : tokens * DV >= (int64_t)4 * 256 * 512 ? 8 : 4;
  const int64_t main_items = (tokens + run - 1) / run * DV;
  const int64_t items = main_items + (a.fin ? (int64_t)a.N * (W - 1) * DV : 0);
  const int64_t blocks = (items + 255) / 256;
  if (blocks == 0) return hipSuccess;
  if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  conv_fwd_kernel<E, VEC, W><<<(unsigned)blocks, 256, 0, s>>>(a, run, main_items, items);
  return hipGetLastError();
}
template <typename E, int VEC, int W>
static hipError_t conv_bwd_run(const ConvArgs& a, hipStream_t s) {
  const int64_t DV = a.D / VEC, tokens = a.B * a.T, rows = conv_bwd_blocks(tokens, a.D);
  const int64_t cb = (DV + kConvLanes - 1) / kConvLanes;
  if (rows > 65535 || cb > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  if (rows > 0) conv_bwd_kernel<E, VEC, W><<<dim3((unsigned)cb, (unsigned)rows), 256, 0, s>>>(a);
  if (a.dinit && a.N > 0) {
    const int64_t blocks = ((int64_t)a.N * (W - 1) * DV + 255) / 256;
    if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
    conv_dinit_kernel<E, VEC, W><<<(unsigned)blocks, 256, 0, s>>>(a);
  }
  const int64_t cols = (int64_t)(W + 1) * a.D;
  conv_param_grads_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, s>>>(a, rows);
  return hipGetLastError();
}
template <typename E, int VEC, bool BWD>
static hipError_t conv_taps(const ConvArgs& a, hipStream_t s) {
  switch (a.W) {
    case 2: return BWD ? conv_bwd_run<E, VEC, 2>(a, s) : conv_fwd_run<E, VEC, 2>(a, s);
    case 3: return BWD ? conv_bwd_run<E, VEC, 3>(a, s) : conv_fwd_run<E, VEC, 3>(a, s);
    case 4: return BWD ? conv_bwd_run<E, VEC, 4>(a, s) : conv_fwd_run<E, VEC, 4>(a, s);
    default: return hipErrorInvalidConfiguration;
  }
}
template <bool BWD>
static hipError_t conv_types(const ConvArgs& a, hipStream_t s) {
  if (a.bf16) return conv_vec<bf16>(a) ? conv_taps<bf16, 8, BWD>(a, s) : conv_taps<bf16, 1, BWD>(a, s);
  return conv_vec<float>(a) ? conv_taps<float, 4, BWD>(a, s) : conv_taps<float, 1, BWD>(a, s);
}
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s) { return conv_types<false>(a, s); }
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s) { return conv_types<true>(a, s); }

}  // namespace gdn
