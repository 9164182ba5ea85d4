// Single-token steps for serving: the short convolution's, and the recurrences' (the
// gated delta rule and the selective state space step) on states kept in a pool of slots.
//
// Row i of a call works on slot slots[i] (or i).  Rows that name the same slot are
// applied in order, as one sequence's tokens: the first of them runs them all with the
// state in registers, the others exit.  A slot outside the pool reads and writes no
// state, and the row's output is zero.
#include "mixer_device.h"
#include "ssm_scan.h"

namespace gdn {

// Whether an earlier row than i names its slot (every thread of the workgroup calls it).
template <int NT>
__device__ __forceinline__ bool earlier_row(const int32_t* slots, int64_t i, int32_t slot) {
  int found = 0;
  for (int64_t j = threadIdx.x; j < i; j += NT) found |= slots[j] == slot;
  return __syncthreads_or(found);
}
// The next row after i that names the slot, or R.
template <int NT>
__device__ __forceinline__ int64_t later_row(const int32_t* slots, int64_t i, int64_t R, int32_t slot) {
  for (int64_t j0 = i + 1; j0 < R; j0 += NT) {
    const int64_t j = j0 + threadIdx.x;
    const bool hit = j < R && slots[j] == slot;
    __shared__ int first;
    if (threadIdx.x == 0) first = NT;
    __syncthreads();
    if (hit) atomicMin(&first, (int)threadIdx.x);
    __syncthreads();
    const int f = first;
    __syncthreads();
    if (f < NT) return j0 + f;
  }
  return R;
}

// ---- recurrences ---------------------------------------------------------------------
// delta rule:  h <- exp(g) h;  u = beta (v - k h);  h <- h + k u^T;  o = scale q h
// selective:   h <- exp(delta A) h + k (delta x)^T; o = q h + D x          (q = C, k = B)
// Bound by the state's bytes (read once, written once).  One workgroup of 256 threads
// per (row, head, BV value columns): a thread holds 4 columns of DK / (256 / (BV / 4))
// rows, so that k h and q h of the delta rule come from one reduction over the rows,
// q (h + k u^T) = q h + (q . k) u^T.  BV = 32 makes 64 workgroups of one row of 16 heads
// of 128 x 128 (4.4 us, latency) and keeps a workgroup's loads in flight together: 256
// such rows, 541 MB, take 110 us (4.9 TB/s; a copy reaches 5.3), 64 rows of the selective step
// 28 us (4.8 TB/s).
template <typename E, int DK, int BV, bool DELTA>
__global__ __launch_bounds__(256) void recurrent_step_kernel(StepArgs a) {
  constexpr int CL = BV / 4;               // lanes across the columns
  constexpr int RG = 256 / CL;             // row groups
  constexpr int RPT = DK / RG;             // rows per thread
  __shared__ float sq[DK], sk[DK];
  __shared__ __align__(16) float sA[4][BV], sB[4][BV];
  __shared__ float sS[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int ncb = a.dv / BV;
  const int cb = blockIdx.x % ncb;
  const int64_t rest = blockIdx.x / ncb;
  const int h = (int)(rest % a.H);
  int64_t row = rest / a.H;
  const int64_t slot = a.slots ? a.slots[row] : row;
  const int cl = tid % CL, rg = tid / CL;
  const int col = cb * BV + cl * 4;
  if (slot < 0 || slot >= a.S) {           // a padding row
    if (tid < CL) store4(reinterpret_cast<E*>(a.o) + (row * a.H + h) * a.dv + cb * BV + tid * 4, f32x4{0.f, 0.f, 0.f, 0.f});
    return;
  }
  if (a.slots && earlier_row<256>(a.slots, row, (int32_t)slot)) return;

  const int64_t base = (slot * a.H + h) * (int64_t)(DK * a.dv) + col;
  f32x4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    s[i] = *reinterpret_cast<const f32x4*>(a.state + base + (int64_t)(rg + i * RG) * a.dv);

  SsmHead hd;
  float dskip = 0.f;
  if (!DELTA) {
    hd.init(a.gates, h);
    if (a.D) dskip = load_scalar(a.D, h, a.gates.param_bf16);
  }
  const int hq = DELTA ? h : h / a.div, Hq = DELTA ? a.H : a.H / a.div;
  while (true) {
    const int64_t at = row * a.H + h;
    float dec, coef;                       // the state's decay; beta or delta
    if (DELTA) {
      dec = __builtin_amdgcn_exp2f(reinterpret_cast<const float*>(a.gate)[at] * 1.4426950408889634f);
      coef = load_scalar(a.beta, at, a.beta_bf16);
    } else {
      coef = hd.delta(a.gates, load_scalar(a.gate, at, a.gates.dt_bf16));
      dec = __builtin_amdgcn_exp2f((float)((double)coef * hd.a2));
    }
    const f32x4 v = load4(reinterpret_cast<const E*>(a.v) + at * a.dv + col);
    const E* qp = reinterpret_cast<const E*>(a.q) + (row * Hq + hq) * DK;
    const E* kp = reinterpret_cast<const E*>(a.k) + (row * Hq + hq) * DK;
    if (tid < DK) {
      sq[tid] = to_f32(qp[tid]);
      sk[tid] = to_f32(kp[tid]);
    }
    __syncthreads();
    f32x4 kh = {0.f, 0.f, 0.f, 0.f}, qh = kh;
    float qk = 0.f;
    if (DELTA) {
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float kr = sk[rg + i * RG], qr = sq[rg + i * RG];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][e] *= dec;
          kh[e] += kr * s[i][e];
          qh[e] += qr * s[i][e];
        }
        qk += kr * qr;
      }
    } else {
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float kr = sk[rg + i * RG] * coef, qr = sq[rg + i * RG];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][e] = s[i][e] * dec + kr * v[e];
          qh[e] += qr * s[i][e];
        }
      }
    }
    // over the wave's row groups (lanes of equal column), then over the waves
#pragma unroll
    for (int d = CL; d < 64; d <<= 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qh[e] += __shfl_xor(qh[e], d, 64);
        if (DELTA) kh[e] += __shfl_xor(kh[e], d, 64);
      }
      if (DELTA) qk += __shfl_xor(qk, d, 64);
    }
    if (lane < CL) {
      *reinterpret_cast<f32x4*>(&sA[wave][lane * 4]) = qh;
      if (DELTA) *reinterpret_cast<f32x4*>(&sB[wave][lane * 4]) = kh;
    }
    if (DELTA && lane == 0) sS[wave] = qk;
    __syncthreads();
    f32x4 u = {0.f, 0.f, 0.f, 0.f};
    if (DELTA) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = cl * 4 + e;
        u[e] = coef * (v[e] - ((sB[0][c] + sB[1][c]) + (sB[2][c] + sB[3][c])));
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] += sk[rg + i * RG] * u[e];
    }
    if (tid < CL) {                        // (their cl is tid)
      f32x4 o;
      const float kq = DELTA ? (sS[0] + sS[1]) + (sS[2] + sS[3]) : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = tid * 4 + e;
        const float q = (sA[0][c] + sA[1][c]) + (sA[2][c] + sA[3][c]);
        o[e] = DELTA ? a.scale * (q + kq * u[e]) : q + dskip * v[e];
      }
      store4(reinterpret_cast<E*>(a.o) + at * a.dv + col, o);
    }
    if (!a.slots) break;
    __syncthreads();                       // sq, sk, sA, sB are done with
    row = later_row<256>(a.slots, row, a.R, (int32_t)slot);
    if (row >= a.R) break;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    *reinterpret_cast<f32x4*>(a.state_out + base + (int64_t)(rg + i * RG) * a.dv) = s[i];
}

template <typename E, int DK, bool DELTA>
static hipError_t run_step(const StepArgs& a, hipStream_t s) {
  constexpr int BV = 32;
  const int64_t blocks = a.R * a.H * (a.dv / BV);
  if (blocks == 0) return hipSuccess;
  if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  recurrent_step_kernel<E, DK, BV, DELTA><<<(unsigned)blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_recurrent_step(const StepArgs& a, hipStream_t s) {
  if (a.delta_rule) {
    if (a.bf16) return a.dk == 64 ? run_step<bf16, 64, true>(a, s) : run_step<bf16, 128, true>(a, s);
    return a.dk == 64 ? run_step<float, 64, true>(a, s) : run_step<float, 128, true>(a, s);
  }
  if (a.bf16) return a.dk == 64 ? run_step<bf16, 64, false>(a, s) : run_step<bf16, 128, false>(a, s);
  return a.dk == 64 ? run_step<float, 64, false>(a, s) : run_step<float, 128, false>(a, s);
}

// ---- convolution ---------------------------------------------------------------------
// One thread per (row, channel), with a loop over the rows of a slot.  64 rows of 6144
// channels, 6 MB: 5.4 us, a launch and two dependent loads (slot, then state).
template <typename E, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepArgs a) {
  const int64_t nb = (a.D + 255) / 256;
  const int64_t d = (blockIdx.x % nb) * 256 + threadIdx.x;
  int64_t row = blockIdx.x / nb;
  const int64_t slot = a.slots ? a.slots[row] : row;
  if (slot < 0 || slot >= a.S) {
    if (d < a.D) reinterpret_cast<E*>(a.y)[row * a.D + d] = from_f32<E>(0.f);
    return;
  }
  if (a.slots && earlier_row<256>(a.slots, row, (int32_t)slot)) return;
  const bool on = d < a.D;
  float w[W], bias = 0.f;
  E st[W];                                 // the window, oldest first; st[W-1] the new input
  if (on) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = load_scalar(a.w, d * W + j, a.param_bf16);
    if (a.bias) bias = load_scalar(a.bias, d, a.param_bf16);
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) st[j + 1] = reinterpret_cast<const E*>(a.state)[(slot * (W - 1) + j) * a.D + d];
  }
  while (true) {
    if (on) {
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) st[j] = st[j + 1];
      st[W - 1] = reinterpret_cast<const E*>(a.x)[row * a.D + d];
      float z = bias;
#pragma unroll
      for (int j = 0; j < W; ++j) z += w[j] * to_f32(st[j]);
      if (a.silu) z *= sigmoid<E>(z);
      reinterpret_cast<E*>(a.y)[row * a.D + d] = from_f32<E>(z);
    }
    if (!a.slots) break;
    row = later_row<256>(a.slots, row, a.R, (int32_t)slot);
    if (row >= a.R) break;
  }
  if (on) {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) reinterpret_cast<E*>(a.state_out)[(slot * (W - 1) + j) * a.D + d] = st[j + 1];
  }
}

template <typename E>
static hipError_t run_conv_step(const ConvStepArgs& a, hipStream_t s) {
  const int64_t blocks = a.R * ((a.D + 255) / 256);
  if (blocks == 0) return hipSuccess;
  if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  if (a.W == 2) conv_step_kernel<E, 2><<<(unsigned)blocks, 256, 0, s>>>(a);
  else if (a.W == 3) conv_step_kernel<E, 3><<<(unsigned)blocks, 256, 0, s>>>(a);
  else conv_step_kernel<E, 4><<<(unsigned)blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t s) {
  return a.bf16 ? run_conv_step<bf16>(a, s) : run_conv_step<float>(a, s);
}

}  // namespace gdn
