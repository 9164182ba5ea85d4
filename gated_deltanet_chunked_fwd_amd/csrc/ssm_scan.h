// The selective state space scan on gfx950, as one kernel template:
//
//   out_j = alpha_j q_j h_j + D v_j,   h_j = exp(a_j) h_{j-1} + kappa_j k_j v_j^T
//
// with a [DK x DV] state h per (sequence, head).  The forward pass is the scan of
// (q, k, v) = (C, B, x); the backward pass is three more of the same form, dC from
// (dy, x, B) in order, dB from (x, dy, C) and du from (B, C, dy) last to first, so one
// kernel serves both and no per-chunk state goes through memory.
//
// In chunks of 64 steps, U the chunk-local inclusive cumsum of a and h the state before
// the chunk:
//   out = exp(U_j) q_j h + sum_{i <= j} (q_j . k_i) exp(U_j - U_i) kappa_i v_i
//   h  <- exp(U_63) h + sum_i k_i (exp(U_63 - U_i) kappa_i v_i)^T
// all four products on MFMA.  U is summed in fp64 and kept as a pair of floats: the
// differences U_j - U_i are small where they matter, U itself need not be.
//
// Last to first, step j of a chunk is its token 63 - j and a_j is the decay of the token
// after it (the adjoint of the forward scan); only the staging, the gates and the output
// addresses know about it.  Tokens past a sequence's end are steps with k = v = q = 0,
// a = 0.
//
// Precision.  bf16 tensors enter MFMA as they are; what is computed (the state, the
// decayed q k products, the decayed v) enters as a sum of bf16 terms: two for the
// outputs (17 bits, so that the output's own rounding is what is seen, and the gate
// gradients, long sums of flows that nearly cancel, keep about 1e-5), three for the
// state's update (24 bits: the final state is an fp32 result).  fp32 tensors use fp32
// MFMA throughout.
//
// Mapping.  One workgroup of 4 waves per (segment, head); a wave owns DV / 4 columns of
// the state for all DK rows, in registers, in tile order (gdn_device.h), so the state
// feeds the next product without leaving them.  Per chunk the workgroup stages q, k and
// v in LDS (the next chunk's global loads in flight meanwhile), splits the 10 lower
// tiles of q k^T over the waves, and each wave then runs its columns.  The outputs come
// out transposed (4 consecutive columns of one token per lane).
#pragma once
#include "gdn_device.h"
#include "mixer_launch.h"

namespace gdn {

// An MFMA operand as a sum of N terms of the tensors' type.
template <typename E, int N>
struct Terms;
template <int N>
struct Terms<float, N> {
  static constexpr int n = 1;
  f32x8 t[1];
  __device__ __forceinline__ void set(const f32x8& v) { t[0] = v; }
};
template <int N>
struct Terms<bf16, N> {
  static constexpr int n = N;
  bf16x8 t[N];
  __device__ __forceinline__ void set(const f32x8& v) {
    f32x8 r = v;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t[i][e] = (bf16)r[e];
        r[e] -= (float)t[i][e];
      }
    }
  }
};
__device__ __forceinline__ f32x8 join8(const f32x4& lo, const f32x4& hi) {
  f32x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = lo[i];
    r[4 + i] = hi[i];
  }
  return r;
}
__device__ __forceinline__ f32x8 widen(const bf16x8& v) {
  f32x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (float)v[i];
  return r;
}
__device__ __forceinline__ f32x8 widen(const f32x8& v) { return v; }

// Inclusive prefix sum of doubles over the wave (DPP moves of both halves).
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double x) {
  const uint64_t u = __double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
  return __longlong_as_double(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double readlane_f64(double x, int l) {
  const uint64_t u = __double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __longlong_as_double(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_scan_f64(double x) {
  x += dpp_f64<0x111>(x);
  x += dpp_f64<0x112>(x);
  x += dpp_f64<0x114>(x);
  x += dpp_f64<0x118>(x);
  const double r0 = readlane_f64(x, 15), r1 = readlane_f64(x, 31), r2 = readlane_f64(x, 47);
  const int row = (threadIdx.x & 63) >> 4;
  return x + (row == 0 ? 0.0 : row == 1 ? r0 : row == 2 ? r0 + r1 : r0 + r1 + r2);
}

// log(1 + exp(x)), x itself where the difference is below half an ulp.
__device__ __forceinline__ float softplus_f32(float x) { return x > 20.f ? x : log1pf(expf(x)); }

struct SsmHead {             // the gates' constants of one head
  float bias;
  double a2;                 // A log2(e)
  __device__ __forceinline__ void init(const SsmGates& g, int h) {
    bias = g.bias ? load_scalar(g.bias, h, g.param_bf16) : 0.f;
    a2 = (double)load_scalar(g.A, h, g.param_bf16) * 1.4426950408889634074;
  }
  __device__ __forceinline__ float delta(const SsmGates& g, float dt) const {
    return g.softplus ? softplus_f32(dt + bias) : dt + bias;
  }
};

struct SsmUnit {             // a (segment, head) unit of the launch
  int h, n, seg, segs;
  int64_t sg;                // global segment
  int64_t tok0;              // the sequence's first token
  int len, nch, c0, c1;      // the sequence's tokens and chunks; the segment's chunks
  int64_t chunk0;            // the sequence's first chunk over all sequences
  __device__ __forceinline__ void init(const SsmSeqs& q, int64_t unit) {
    h = (int)(unit % q.H);
    sg = unit / q.H;
    if (q.seg_off) {
      n = seq_of_chunk(sg, q.seg_off, q.N, 0);
      seg = (int)(sg - q.seg_off[n]);
      segs = q.seg_off[n + 1] - q.seg_off[n];
    } else {
      n = (int)(sg / q.segs);
      seg = (int)(sg - (int64_t)n * q.segs);
      segs = q.segs;
    }
    if (q.cu) {
      tok0 = q.cu[n];
      len = q.cu[n + 1] - q.cu[n];
      chunk0 = q.chunk_off ? q.chunk_off[n] : 0;
    } else {
      tok0 = (int64_t)n * q.T;
      len = (int)q.T;
      chunk0 = (int64_t)n * ((q.T + kChunk - 1) / kChunk);
    }
    nch = (len + kChunk - 1) / kChunk;
    c0 = seg * q.seg_chunks;
    c1 = min(nch, c0 + q.seg_chunks);
  }
};

// One chunk's rows of a tensor on their way from memory to LDS.
template <typename E, int W>
struct SsmTile {
  static constexpr int EPV = 16 / (int)sizeof(E), VPR = W / EPV, NV = kChunk * VPR / 256;
  u32x4 v[NV];
  // base: the sequence's first token (head offset applied); rows past the sequence's end
  // read the chunk's first token (zeroed in store)
  __device__ __forceinline__ void load(const E* base, int64_t stride, int c, int len, int rev, int tid) {
    const E* cb = base + (int64_t)c * kChunk * stride;
    const int lim = len - c * kChunk;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + 256 * j, r = i / VPR;
      const int t = rev ? kChunk - 1 - r : r;
      v[j] = *reinterpret_cast<const u32x4*>(cb + (int64_t)(t < lim ? t : 0) * stride + (i % VPR) * EPV);
    }
  }
  __device__ __forceinline__ void store(E* s, int ls, int c, int len, int rev, int tid) const {
    const int lim = len - c * kChunk;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + 256 * j, r = i / VPR;
      const int t = rev ? kChunk - 1 - r : r;
      *reinterpret_cast<u32x4*>(s + r * ls + (i % VPR) * EPV) = t < lim ? v[j] : zero;
    }
  }
};

__device__ __forceinline__ f32x4 load4(const bf16* p) {
  const bf16x4 b = *reinterpret_cast<const bf16x4*>(p);
  f32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (float)b[i];
  return r;
}
__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

template <typename E, int DK, int DV, bool STATE>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void ssm_scan_kernel(SsmScans args) {
  using M = Mma<E>;
  using frag = typename M::frag;
  constexpr bool BF = sizeof(E) == 2;
  constexpr int NC = DV / 64;              // 16-column tiles per wave
  constexpr int NKT = DK / 16, NKS = DK / 32;
  constexpr int KS = BF ? DK + 16 : DK + 4, VS = BF ? DV + 16 : DV + 4, CS = BF ? kChunk + 16 : kChunk + 4;
  constexpr int NP = BF ? 2 : 1;           // terms of the stored q k products

  __shared__ __align__(16) E sK[kChunk * KS];
  __shared__ __align__(16) E sV[kChunk * VS];
  __shared__ __align__(16) E sQ[STATE ? 8 : kChunk * KS];
  __shared__ __align__(16) E sP[STATE ? 1 : NP][STATE ? 8 : kChunk * CS];
  // gates of the chunk being computed and of the next one
  __shared__ __align__(16) float sUh[2][kChunk], sUl[2][kChunk], sKap[2][kChunk], sEU[2][kChunk], sWt[2][kChunk],
      sAl[2][kChunk], sDec[2];
  __shared__ float sDot[2][4][kChunk];

  const SsmSeqs& sq = args.seqs;
  const SsmGates& gt = args.gates;
  const SsmScan& a = args.s[blockIdx.y];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  SsmUnit u;
  u.init(sq, blockIdx.x);
  const int rev = a.rev;
  const int seg_in_order = rev ? u.segs - 1 - u.seg : u.seg;
  const bool last = seg_in_order == u.segs - 1;
  if (STATE && last) return;
  const int h = u.h, H = sq.H, len = u.len;
  const int64_t nh = (int64_t)u.n * H + h;
  const int64_t slot = u.sg * H + h;
  const int steps = max(0, u.c1 - u.c0);

  const E* kb = reinterpret_cast<const E*>(a.k.p) + u.tok0 * a.k.stride + (h / a.k.div) * DK;
  const E* vb = reinterpret_cast<const E*>(a.v.p) + u.tok0 * a.v.stride + (h / a.v.div) * DV;
  const E* qb = STATE ? nullptr : reinterpret_cast<const E*>(a.q.p) + u.tok0 * a.q.stride + (h / a.q.div) * DK;
  SsmHead hd;
  hd.init(gt, h);

  // ---- start state, tile order ----
  f32x4 st[NKT][NC];
  const int col0 = wave * 16 * NC + r16;   // this lane's first state column
  {
    const float* src = STATE ? nullptr : seg_in_order > 0 ? a.seg_start : a.h0;
    const int64_t off = (seg_in_order > 0 ? slot : nh) * (DK * DV);
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        const int row = prow(kt, 4 * q4), col = col0 + 16 * nc;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (src) {
          if (a.state_t) {
            v = *reinterpret_cast<const f32x4*>(src + off + (int64_t)col * DK + row);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = src[off + (int64_t)(row + i) * DV + col];
          }
        }
        st[kt][nc] = v;
      }
  }

  // ---- gates of one chunk, by one wave: lane = step ----
  float dt_own = 0.f, dt_dec = 0.f;        // raw dt of the step's token and of its decay's
  auto load_dt = [&](int c) {
    const int t = c * kChunk + (rev ? kChunk - 1 - lane : lane);
    const int64_t base = u.tok0 * H + h;
    dt_own = load_scalar(gt.dt, base + (int64_t)min(t, len - 1) * H, gt.dt_bf16);
    dt_dec = rev ? load_scalar(gt.dt, base + (int64_t)min(t + 1, len - 1) * H, gt.dt_bf16) : dt_own;
  };
  double seg_log2 = 0.0;
  auto gates = [&](int c, int b) {
    const int t = c * kChunk + (rev ? kChunk - 1 - lane : lane);
    const float del = t < len ? hd.delta(gt, dt_own) : 0.f;
    const float ddec = rev ? (t + 1 < len ? hd.delta(gt, dt_dec) : 0.f) : del;
    const double U = wave_scan_f64((double)ddec * hd.a2);
    const double end = readlane_f64(U, 63);
    const float kap = a.kappa_delta ? del : 1.f;
    const float hi = (float)U;
    sUh[b][lane] = hi;
    sUl[b][lane] = (float)(U - (double)hi);
    sKap[b][lane] = kap;
    sEU[b][lane] = __builtin_amdgcn_exp2f(hi);
    sWt[b][lane] = kap * __builtin_amdgcn_exp2f((float)(end - U));
    sAl[b][lane] = a.alpha_delta ? del : 1.f;
    if (lane == 0) sDec[b] = __builtin_amdgcn_exp2f((float)end);
    if (STATE) seg_log2 += end;
  };

  SsmTile<E, DK> tk;
  SsmTile<E, DV> tv;
  SsmTile<E, STATE ? 64 : DK> tq;
  auto chunk_of = [&](int i) { return rev ? u.c1 - 1 - i : u.c0 + i; };
  auto load_tiles = [&](int c) {
    tk.load(kb, a.k.stride, c, len, rev, tid);
    tv.load(vb, a.v.stride, c, len, rev, tid);
    if constexpr (!STATE) tq.load(qb, a.q.stride, c, len, rev, tid);
  };
  if (steps > 0) {
    load_tiles(chunk_of(0));
    if (wave == 3) {
      load_dt(chunk_of(0));
      gates(chunk_of(0), 0);
      if (steps > 1) load_dt(chunk_of(1));
    }
  }

  // adds the four waves' shares of a chunk's dots and stores them
  auto flush_dots = [&](int c) {
    if (tid < kChunk) {
      const int t = rev ? kChunk - 1 - tid : tid;
      const int64_t at = ((u.chunk0 + c) * H + h) * kChunk + t;
      a.dot_out[at] = (sDot[0][0][tid] + sDot[0][1][tid]) + (sDot[0][2][tid] + sDot[0][3][tid]);
      if (a.dot_skip)
        a.dot_skip[at] = (sDot[1][0][tid] + sDot[1][1][tid]) + (sDot[1][2][tid] + sDot[1][3][tid]);
    }
  };

  const float dskip = (!STATE && a.D) ? load_scalar(a.D, h, gt.param_bf16) : 0.f;
  for (int it = 0; it < steps; ++it) {
    const int c = chunk_of(it), b = it & 1;
    __syncthreads();                       // the previous chunk's tiles are done with
    tk.store(sK, KS, c, len, rev, tid);
    tv.store(sV, VS, c, len, rev, tid);
    if constexpr (!STATE) tq.store(sQ, KS, c, len, rev, tid);
    if constexpr (!STATE) {
      if (a.aux.p && it > 0) flush_dots(chunk_of(it - 1));
    }
    __syncthreads();
    if (it + 1 < steps) {
      load_tiles(chunk_of(it + 1));
      if (wave == 3) {
        gates(chunk_of(it + 1), b ^ 1);
        if (it + 2 < steps) load_dt(chunk_of(it + 2));
      }
    }

    f32x4 acc[4][NC];                      // out^T: columns (rows of the tile) x steps
    if constexpr (!STATE) {
      // ---- the lower tiles of (k q^T), decayed, to LDS as [step][key] ----
      // tile pair i of 10: (key tile, step tile), dealt round robin
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int pi = wave + 4 * i;
        if (pi < 10) {
          const int tt = pi < 1 ? 0 : pi < 3 ? 1 : pi < 6 ? 2 : 3;
          const int jt = pi - (tt * (tt + 1)) / 2;
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < NKS; ++s)
            p = M::run(lds_frag(sK, KS, 16 * jt + r16, 32 * s, q4), lds_frag(sQ, KS, 16 * tt + r16, 32 * s, q4), p);
          const int t = 16 * tt + r16, j0 = 16 * jt + 4 * q4;
          const float uh = sUh[b][t], ul = sUl[b][t];
          const f32x4 kh = *reinterpret_cast<const f32x4*>(&sUh[b][j0]);
          const f32x4 kl = *reinterpret_cast<const f32x4*>(&sUl[b][j0]);
          const f32x4 kp = *reinterpret_cast<const f32x4*>(&sKap[b][j0]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = __builtin_amdgcn_exp2f((uh - kh[e]) + (ul - kl[e])) * kp[e];
            p[e] = j0 + e <= t ? p[e] * w : 0.f;
          }
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            store4(&sP[n][t * CS + j0], p);
            if constexpr (BF) {
#pragma unroll
              for (int e = 0; e < 4; ++e) p[e] -= (float)(bf16)p[e];
            }
          }
        }
      }
      // zero tiles above the diagonal that a 32-wide contraction step reads
      if (wave < 2) {
        const int t = 32 * wave + r16, j0 = 32 * wave + 16 + 4 * q4;
        const f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NP; ++n) store4(&sP[n][t * CS + j0], z);
      }
      // ---- out^T = h^T q^T, decayed ----
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) acc[tt][nc] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < NKS; ++s) {
        Terms<E, 2> hs[NC];
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) hs[nc].set(join8(st[2 * s][nc], st[2 * s + 1][nc]));
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const frag qf = lds_frag(sQ, KS, 16 * tt + r16, 32 * s, q4);
#pragma unroll
          for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int n = 0; n < Terms<E, 2>::n; ++n) acc[tt][nc] = M::run(hs[nc].t[n], qf, acc[tt][nc]);
        }
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const float e = sEU[b][16 * tt + r16];
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[tt][nc][i] *= e;
      }
      __syncthreads();                     // sP
    }

    // ---- v^T operands; out^T += v^T p^T; the state's update ----
    const float dec = sDec[b];
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
      for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int i = 0; i < 4; ++i) st[kt][nc][i] *= dec;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      frag vf[NC];
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        const int cb = wave * 16 * NC + 16 * nc;
        vf[nc] = col_frag(sV, VS, 32 * s + 8 * q4, 32 * s + 8 * q4 + 4, cb + r16, cb + 4 * (r16 & 3));
      }
      if constexpr (!STATE) {
#pragma unroll
        for (int tt = 2 * s; tt < 4; ++tt)
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            const frag pf = lds_frag(sP[n], CS, 16 * tt + r16, 32 * s, q4);
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) acc[tt][nc] = M::run(vf[nc], pf, acc[tt][nc]);
          }
      }
      Terms<E, 3> wv[NC];
      {
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(&sWt[b][32 * s + 8 * q4]);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(&sWt[b][32 * s + 8 * q4 + 4]);
        const f32x8 w = join8(w0, w1);
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
          f32x8 x = widen(vf[nc]);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= w[e];
          wv[nc].set(x);
        }
      }
#pragma unroll
      for (int kt = 0; kt < NKT; ++kt) {
        const frag kf = col_frag(sK, KS, 32 * s + 8 * q4, 32 * s + 8 * q4 + 4, prow(kt, r16), prow(kt, 4 * (r16 & 3)));
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
          for (int n = 0; n < Terms<E, 3>::n; ++n) st[kt][nc] = M::run(kf, wv[nc].t[n], st[kt][nc]);
      }
    }

    if constexpr (!STATE) {
      // ---- outputs: lane = step 16 tt + r16, columns 4 q4 .. +3 of each tile ----
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int j = 16 * tt + r16;
        const int t = c * kChunk + (rev ? kChunk - 1 - j : j);
        const float al = sAl[b][j];
        float d0 = 0.f, d1 = 0.f;
        const bool ok = t < len;
        const int64_t tok = u.tok0 + (ok ? t : c * kChunk);
        const E* auxp = a.aux.p ? reinterpret_cast<const E*>(a.aux.p) + tok * a.aux.stride + (h / a.aux.div) * DV : nullptr;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
          const int col = wave * 16 * NC + 16 * nc + 4 * q4;
          f32x4 o = acc[tt][nc];
          const f32x4 v = load4(&sV[j * VS + col]);
          if (auxp) {
            const f32x4 x = load4(auxp + col);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              d0 += x[i] * o[i];
              d1 += x[i] * v[i];
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = o[i] * al + dskip * v[i];
          if (ok) {
            const int64_t at = (tok * H + h) * DV + col;
            if (BF && a.out_f32) *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at) = o;
            else store4(reinterpret_cast<E*>(a.out) + at, o);
          }
        }
        if (auxp) {
          d0 += __shfl_xor(d0, 16, 64);
          d0 += __shfl_xor(d0, 32, 64);
          d1 += __shfl_xor(d1, 16, 64);
          d1 += __shfl_xor(d1, 32, 64);
          if (q4 == 0) {
            sDot[0][wave][j] = ok ? d0 : 0.f;
            sDot[1][wave][j] = ok ? d1 : 0.f;
          }
        }
      }
    }
  }
  if constexpr (!STATE) {
    if (a.aux.p && steps > 0) {
      __syncthreads();
      flush_dots(chunk_of(steps - 1));
    }
  }

  // ---- the end state ----
  float* dst = STATE ? a.seg_state : (last ? a.hT : nullptr);
  if (dst) {
    float f = 1.f;
    if (!STATE && a.hT_decay && len > 0) {
      const float d = hd.delta(gt, load_scalar(gt.dt, u.tok0 * H + h, gt.dt_bf16));
      f = __builtin_amdgcn_exp2f((float)((double)d * hd.a2));
    }
    const int64_t off = (STATE ? slot : nh) * (DK * DV);
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        const int row = prow(kt, 4 * q4), col = col0 + 16 * nc;
        f32x4 v = st[kt][nc];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= f;
        if (a.state_t) {
          *reinterpret_cast<f32x4*>(dst + off + (int64_t)col * DK + row) = v;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[off + (int64_t)(row + i) * DV + col] = v[i];
        }
      }
  }
  if (STATE && wave == 3 && lane == 0) a.seg_decay[slot] = __builtin_amdgcn_exp2f((float)seg_log2);
}

template <typename E, int DK, int DV>
hipError_t run_ssm_scan(const SsmScans& a, int count, bool state_pass, hipStream_t s) {
  if (a.seqs.units == 0) return hipSuccess;
  if (a.seqs.units > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)a.seqs.units, (unsigned)count);
  if (state_pass) ssm_scan_kernel<E, DK, DV, true><<<grid, 256, 0, s>>>(a);
  else ssm_scan_kernel<E, DK, DV, false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <typename E>
hipError_t run_ssm_scan_dims(const SsmScans& a, int count, int dk, int dv, bool state_pass, hipStream_t s) {
  if (dk == 64 && dv == 64) return run_ssm_scan<E, 64, 64>(a, count, state_pass, s);
  if (dk == 64 && dv == 128) return run_ssm_scan<E, 64, 128>(a, count, state_pass, s);
  if (dk == 128 && dv == 64) return run_ssm_scan<E, 128, 64>(a, count, state_pass, s);
  if (dk == 128 && dv == 128) return run_ssm_scan<E, 128, 128>(a, count, state_pass, s);
  return hipErrorInvalidConfiguration;
}

}  // namespace gdn
