// The short causal convolution of a token mixer, per channel d:
//   z_t = bias + sum_w weight[d, w] x_{t - W + 1 + w},   y_t = silu(z_t) or z_t,
// inputs before a sequence's first token from its initial state (or zero).  Backward:
//   dz = dy silu'(z) (z formed again from x),  dx_s = sum_w weight[w] dz_{s + W - 1 - w},
//   dweight[w] = sum_t dz_t x_{t - W + 1 + w},  dbias = sum_t dz_t.
//
// Bound by memory.  A thread owns VEC channels (16 bytes) and a run of tokens, with the
// window of inputs (and, going back, of dz) in registers, so every input is read once
// but for W - 1 tokens at the run's edge, which come from the caches.  bf16, W = 4:
// forward 4 x 4096 tokens of 6144 channels, 403 MB: 86 us (4.7 TB/s; a copy reaches 5.3).
// Backward of 12003 packed tokens of 2312 channels, 167 MB: 53 us, and 5 us for the second
// kernel, the sum of the weights' gradients.
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
// ... of a token that is the same for the whole wave (all 64 lanes call it): the lanes look
// at 64 places of the range that is left at once
__device__ __forceinline__ ConvSeq conv_seq_wave(const ConvArgs& a, int64_t tok) {
  if (!a.cu) return conv_seq(a, tok);
  const int lane = threadIdx.x & 63;
  int n = 0, size = a.N;                   // the first n with cu[n + 1] > tok, one of `size` from n on
  while (size > 1) {
    const int step = (size + 63) / 64;
    const int l = __builtin_ctzll(__ballot(a.cu[n + min((lane + 1) * step, size)] > tok));
    n += l * step;
    size = min(step, size - l * step);
  }
  ConvSeq s;
  s.n = n;
  s.start = a.cu[n];
  s.end = a.cu[n + 1];
  return s;
}
// The sequence with tokens in front of s (for the whole wave, as above), which has one.
__device__ __forceinline__ ConvSeq conv_seq_before(const ConvArgs& a, const ConvSeq& s) {
  if (!a.cu) return conv_seq(a, s.start - 1);
  const int lane = threadIdx.x & 63;
  for (int n = (int)s.n - 1;; n -= 64) {   // the last n with cu[n] < s.start
    const uint64_t hit = __ballot(a.cu[max(n - lane, 0)] < s.start);
    if (hit) {
      n -= __builtin_ctzll(hit);
      return {n, a.cu[n], s.start};
    }
  }
}
// The sequence of the token behind s, which is there: the next one, if not several are empty.
__device__ __forceinline__ ConvSeq conv_seq_behind(const ConvArgs& a, const ConvSeq& s) {
  if (a.cu) {
    for (int64_t n = s.n + 1; n <= s.n + 4; ++n) {
      const int64_t end = a.cu[n + 1];
      if (end > s.end) return {n, s.end, end};
    }
  }
  return conv_seq(a, s.end);
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
template <typename E>
__device__ __forceinline__ float dsilu(float z) {
  const float s = sigmoid<E>(z);
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
      s = conv_seq_behind(a, s);
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
      y[i] = a.silu ? z * sigmoid<E>(z) : z;
    }
    store_vec<E, VEC>(reinterpret_cast<E*>(a.y) + t * a.D + d, y);
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[j][i] = x[j + 1][i];
  }
}

// silu'(z) dy, or dy.
template <typename E, int VEC, int W>
__device__ __forceinline__ void conv_dz(const ConvWeights<VEC, W>& cw, const float (&x)[W][VEC], int silu, float (&dz)[VEC]) {
  if (!silu) return;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    float z = cw.bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) z += cw.w[j][i] * x[j][i];
    dz[i] *= dsilu<E>(z);
  }
}
// dz of one token, everything from memory.
template <typename E, int VEC, int W>
__device__ __forceinline__ void conv_dz_at(const ConvArgs& a, const ConvWeights<VEC, W>& cw, const ConvSeq& s, int64_t t,
                                           int64_t d, float (&dz)[VEC]) {
  float x[W][VEC];
#pragma unroll
  for (int j = 0; j < W; ++j) conv_input<E, VEC, W>(a, s, t - (W - 1) + j, d, x[j]);
  load_vec<E, VEC>(reinterpret_cast<const E*>(a.dy) + t * a.D + d, dz);
  conv_dz<E, VEC, W>(cw, x, a.silu, dz);
}

// Gradient of the initial state: the inputs before a sequence's first token.
template <typename E, int VEC, int W>
__device__ __forceinline__ void conv_dinit(const ConvArgs& a, int64_t item) {
  const int64_t DV = a.D / VEC;
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
      conv_dz_at<E, VEC, W>(a, cw, s, s.start + i0 - w, d, dz);
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

// Tokens last to first.  A workgroup is 64 channel lanes x 4 runs of kConvRun tokens (a wave
// each), whose shares of dweight and dbias it adds up in LDS and writes as one row of
// `part`.  Two channels a lane: with eight, the windows, weights and shares of W = 4 taps
// leave room for two waves per SIMD, too few to hide the loads.  Bound by the latency of a
// run's loads, all of which are issued ahead of their use: runs of 32 tokens take 75 us
// instead of 57, shorter ones read the window at their edge more often and make more
// shares.  The first workgroups form the gradient of the initial states (a chain of loads:
// last, they would be the tail).
constexpr int kConvRun = 16;
constexpr int kConvLanes = 64;
constexpr int kConvBlockTokens = kConvRun * (256 / kConvLanes);

template <typename E, int VEC, int W>
struct ConvBack {
  const ConvArgs& a;
  const uint32_t d;
  const bool on;                           // the lane has a channel (else it repeats the first one's work)
  ConvWeights<VEC, W> cw;
  float dw[W][VEC] = {}, db[VEC] = {};
  float dz[W][VEC];                        // dz[k] = dz_{t + k}, zero past the sequence's end
  float x[W][VEC];                         // x[j] = x_{t - W + 1 + j}

  __device__ __forceinline__ ConvBack(const ConvArgs& a_, uint32_t d_, bool on_) : a(a_), d(d_), on(on_) { cw.load(a, d); }
  __device__ __forceinline__ void shift() {
#pragma unroll
    for (int j = W - 1; j > 0; --j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        x[j][i] = x[j - 1][i];
        dz[j][i] = dz[j - 1][i];
      }
  }
  // one token with the window xw, its dy in dz[0]
  __device__ __forceinline__ void token(const float (&xw)[W][VEC], float (&dx)[VEC]) {
    conv_dz<E, VEC, W>(cw, xw, a.silu, dz[0]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float g = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        g += cw.w[j][i] * dz[W - 1 - j][i];
        dw[j][i] += dz[0][i] * xw[j][i];
      }
      db[i] += dz[0][i];
      dx[i] = g;
    }
  }
  __device__ __forceinline__ void store(int64_t t, const float (&dx)[VEC]) {
    if (on) store_vec<E, VEC>(reinterpret_cast<E*>(a.dx) + t * a.D + d, dx);
  }
  // a token's window with what lies before its sequence taken from the state
  __device__ __forceinline__ void patch(const ConvSeq& s, int64_t t, float (&xw)[W][VEC]) {
    if (t - (W - 1) >= s.start) return;
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
      if (t - (W - 1) + j < s.start) conv_input<E, VEC, W>(a, s, t - (W - 1) + j, d, xw[j]);
  }

  // Tokens [t0, t1) of a wave, last to first.  All inputs are read first, in one go, before
  // the sequence is known (rows past the batch's ends read its first or last token); the
  // window in registers then holds the batch's tokens whatever their sequence, and only
  // runs near a sequence's ends look at which of them are its own.
  __device__ __forceinline__ void run(int64_t t0, int64_t t1, int64_t tokens) {
    const E* xp = reinterpret_cast<const E*>(a.x);
    const E* yp = reinterpret_cast<const E*>(a.dy);
    auto in = [&](int64_t t) { return min(max(t, (int64_t)0), tokens - 1); };
    // inputs of tokens t1 + W - 2 down to t0 - (W - 1), dy of the same but the last W - 1
    Raw<E, VEC> ex[2 * W - 2], ey[W - 1], bx[kConvRun], by[kConvRun];
#pragma unroll
    for (int k = 0; k < 2 * W - 2; ++k) ex[k].load(xp + in(t1 - (W - 1) + k) * a.x_stride + d);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) ey[k].load(yp + in(t1 + k) * a.D + d);
#pragma unroll
    for (int k = 0; k < kConvRun; ++k) {     // token t1 - 1 - k: its oldest input and its dy
      bx[k].load(xp + in(t1 - 1 - k - (W - 1)) * a.x_stride + d);
      by[k].load(yp + in(t1 - 1 - k) * a.D + d);
    }
    ConvSeq s = conv_seq_wave(a, t1 - 1);
    const bool inner = t1 - t0 == kConvRun && t0 - (W - 1) >= s.start && t1 + (W - 1) <= s.end - (W - 1);
#pragma unroll
    for (int k = W - 2; k >= 0; --k) {       // dz of the W - 1 tokens behind the run
      float xe[W][VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        dz[k][i] = ey[k][i];
#pragma unroll
        for (int j = 0; j < W; ++j) xe[j][i] = ex[k + j][i];
      }
      if (!inner) patch(s, t1 + k, xe);
      conv_dz<E, VEC, W>(cw, xe, a.silu, dz[k]);
      if (!inner && t1 + k >= s.end)
#pragma unroll
        for (int i = 0; i < VEC; ++i) dz[k][i] = 0.f;
    }
#pragma unroll
    for (int j = 1; j < W; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[j - 1][i] = ex[j - 1][i];
    if (inner) {
#pragma unroll
      for (int k = 0; k < kConvRun; ++k) {
        shift();
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          x[0][i] = bx[k][i];
          dz[0][i] = by[k][i];
        }
        float dx[VEC];
        token(x, dx);
        store(t1 - 1 - k, dx);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < kConvRun; ++k) {
      const int64_t t = t1 - 1 - k;
      if (t >= t0) {
        if (t < s.start) {                   // an earlier sequence: nothing flows back into it
          s = conv_seq_before(a, s);
#pragma unroll
          for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) dz[j][i] = 0.f;
        }
        shift();
        float xe[W][VEC], dx[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          x[0][i] = bx[k][i];
          dz[0][i] = by[k][i];
#pragma unroll
          for (int j = 0; j < W; ++j) xe[j][i] = x[j][i];
        }
        patch(s, t, xe);
        token(xe, dx);
        if (a.dfin && t >= s.end - (W - 1)) {
          float f[VEC];
          load_vec<E, VEC>(reinterpret_cast<const E*>(a.dfin) + (s.n * (W - 1) + (t - (s.end - (W - 1)))) * a.D + d, f);
#pragma unroll
          for (int i = 0; i < VEC; ++i) dx[i] += f[i];
        }
        store(t, dx);
      }
    }
  }
};

template <typename E, int VEC, int W>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a, uint32_t extra, uint32_t cb) {
  __shared__ float red[256 / kConvLanes][VEC][kConvLanes];
  if (blockIdx.x < extra) {
    const int64_t items = (int64_t)a.N * (W - 1) * (a.D / VEC);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)extra * 256)
      conv_dinit<E, VEC, W>(a, i);
    return;
  }
  // (cb workgroups across the channels)
  const int64_t brow = (blockIdx.x - extra) / cb;
  const uint32_t bcol = (blockIdx.x - extra) % cb;
  // (a wave's run is uniform: its addresses are scalar but for the lane's channels)
  const int cl = threadIdx.x % kConvLanes, tr = __builtin_amdgcn_readfirstlane(threadIdx.x / kConvLanes);
  const int64_t DV = a.D / VEC, tokens = a.B * a.T;
  const int64_t cv = (int64_t)bcol * kConvLanes + cl;
  const bool on = cv < DV;
  const int64_t t0 = brow * kConvBlockTokens + tr * kConvRun, t1 = min(tokens, t0 + kConvRun);
  ConvBack<E, VEC, W> b(a, (uint32_t)(on ? cv : 0) * VEC, on);
  if (t0 < t1) b.run(t0, t1, tokens);
  // the workgroup's shares, summed over its runs
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VEC; ++i) red[tr][i][cl] = j < W ? b.dw[j < W ? j : 0][i] : b.db[i];
    __syncthreads();
    if (on) {
      // channels dealt over the runs' threads
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i % (256 / kConvLanes) == tr) {
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < 256 / kConvLanes; ++k) s += red[k][i][cl];
          a.part[(brow * (W + 1) + j) * a.D + b.d + i] = s;
        }
    }
  }
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

int64_t conv_bwd_rows(int64_t tokens) { return (tokens + kConvBlockTokens - 1) / kConvBlockTokens; }
// Workgroups for the initial states' gradients: more make further rounds.
constexpr int64_t kConvDinitBlocks = 1 << 14;
bool conv_bwd_fits(int64_t tokens, int64_t D, int W) {   // (a channel a lane: the most workgroups)
  return conv_bwd_rows(tokens) + 1 <= (kMaxDispatchItems / 256 - kConvDinitBlocks) / ((D + kConvLanes - 1) / kConvLanes) &&
         (W + 1) * D <= kMaxDispatchItems / 1024 * 32;
}

// Vector accesses need rows that start on a vector: D and x's stride multiples of VEC (one
// channel per thread otherwise).
static bool conv_vec(const ConvArgs& a, int v) { return a.D % v == 0 && a.x_stride % v == 0; }

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
  const int64_t DV = a.D / VEC, tokens = a.B * a.T, rows = conv_bwd_rows(tokens);
  const int64_t cb = (DV + kConvLanes - 1) / kConvLanes;
  const int64_t want = a.dinit ? ((int64_t)a.N * (W - 1) * DV + 255) / 256 : 0;
  const int64_t extra = want < kConvDinitBlocks ? want : kConvDinitBlocks, blocks = rows * cb + extra;
  if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  if (blocks > 0)
    conv_bwd_kernel<E, VEC, W><<<(unsigned)blocks, 256, 0, s>>>(a, (uint32_t)extra, (uint32_t)cb);
  const int64_t cols = (int64_t)(W + 1) * a.D;
  conv_param_grads_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, s>>>(a, rows);
  return hipGetLastError();
}
template <typename E, int VEC, int W, bool BWD>
static hipError_t conv_run(const ConvArgs& a, hipStream_t s) {
  if constexpr (BWD) return conv_bwd_run<E, VEC, W>(a, s);
  else return conv_fwd_run<E, VEC, W>(a, s);
}
template <typename E, int VEC, bool BWD>
static hipError_t conv_taps(const ConvArgs& a, hipStream_t s) {
  switch (a.W) {
    case 2: return conv_run<E, VEC, 2, BWD>(a, s);
    case 3: return conv_run<E, VEC, 3, BWD>(a, s);
    case 4: return conv_run<E, VEC, 4, BWD>(a, s);
    default: return hipErrorInvalidConfiguration;
  }
}
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s) {
  if (a.bf16) return conv_vec(a, 8) ? conv_taps<bf16, 8, false>(a, s) : conv_taps<bf16, 1, false>(a, s);
  return conv_vec(a, 4) ? conv_taps<float, 4, false>(a, s) : conv_taps<float, 1, false>(a, s);
}
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s) {
  if (a.bf16) return conv_vec(a, 2) ? conv_taps<bf16, 2, true>(a, s) : conv_taps<bf16, 1, true>(a, s);
  return conv_vec(a, 2) ? conv_taps<float, 2, true>(a, s) : conv_taps<float, 1, true>(a, s);
}

}  // namespace gdn
