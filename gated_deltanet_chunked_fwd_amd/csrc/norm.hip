// Layer norm of every row of x [rows, H, D] with each head's own weight and bias [H, D]
// (H = 1: the ordinary layer norm), and optionally a SiLU gate:
//   xh = (x - mean) rstd,   y = (xh w + b) silu(z)
// Backward, with the statistics the forward pass kept and dn = dy silu(z):
//   dx = rstd (dn w - mean_D(dn w) - xh mean_D(dn w xh)),   dz = dy (xh w + b) silu'(z),
//   dw = sum over rows of dn xh,   db = sum over rows of dn.
//
// Bound by memory: every tensor is read or written once.  A team of L lanes (within a
// wave, or the whole workgroup) holds one row in registers, K vectors of VEC elements a
// lane, so mean and variance are two passes over registers (no E[x^2] - E[x]^2, which
// loses the variance of rows far from zero).  Going back, a team keeps to one head and
// strides over the rows, with its share of dw and db in registers; one row of shares
// per team goes to memory (per workgroup where all its teams have the same head) and a
// second kernel adds them, in a fixed order.
#include "mixer_device.h"
#include "mixer_launch.h"

namespace gdn {

// Sum over a team's lanes, in every lane.
template <int L>
__device__ __forceinline__ float team_sum(float v, float* red) {
#pragma unroll
  for (int d = 1; d < (L < 64 ? L : 64); d <<= 1) v += __shfl_xor(v, d, 64);
  if constexpr (L == 256) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (red[0] + red[1]) + (red[2] + red[3]);
  }
  return v;
}

template <typename E, int VEC, int L, int K>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a) {
  __shared__ float red[4];
  const int lane = threadIdx.x % L;
  const int64_t row = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int D = a.D;
  if (row >= a.rows * a.H) return;         // (whole teams; a 256-lane team is never past the end)
  const E* xr = reinterpret_cast<const E*>(a.x) + row * D;
  float x[K][VEC], s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * L + lane) * VEC;
    if (c < D) load_vec<E, VEC>(xr + c, x[k]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if (c >= D) x[k][i] = 0.f;
      s += x[k][i];
    }
  }
  const float mean = team_sum<L>(s, red) / (float)D;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if ((k * L + lane) * VEC < D)
#pragma unroll
      for (int i = 0; i < VEC; ++i) v += (x[k][i] - mean) * (x[k][i] - mean);
  const float rstd = 1.f / sqrtf(team_sum<L>(v, red) / (float)D + a.eps);
  if (lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  const int64_t hoff = (row % a.H) * D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * L + lane) * VEC;
    if (c < D) {
      float w[VEC], b[VEC], z[VEC], y[VEC];
      if (a.w) load_params<VEC>(a.w, hoff + c, a.param_bf16, w);
      if (a.b) load_params<VEC>(a.b, hoff + c, a.param_bf16, b);
      if (a.gate) load_vec<E, VEC>(reinterpret_cast<const E*>(a.gate) + row * D + c, z);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float o = (x[k][i] - mean) * rstd;
        if (a.w) o *= w[i];
        if (a.b) o += b[i];
        if (a.gate) o *= z[i] * sigmoid_f32(z[i]);
        y[i] = o;
      }
      store_vec<E, VEC>(reinterpret_cast<E*>(a.y) + row * D + c, y);
    }
  }
}

template <typename E, int VEC, int L, int K>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormArgs a, int64_t strips, int shared_head) {
  constexpr int TEAMS = 256 / L;
  __shared__ float red[4];
  __shared__ float part[2][TEAMS > 1 ? L * K * VEC : 1];
  const int lane = threadIdx.x % L, team = threadIdx.x / L;
  const int64_t g = (int64_t)blockIdx.x * TEAMS + team;
  const int D = a.D, H = a.H;
  const int h = (int)(g % H);
  const int64_t strip = g / H;
  const int64_t hoff = (int64_t)h * D;
  const bool params = a.dw || a.db;
  float w[K][VEC], b[K][VEC], dw[K][VEC] = {}, db[K][VEC] = {};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * L + lane) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      w[k][i] = 1.f;
      b[k][i] = 0.f;
    }
    if (c < D && a.w) load_params<VEC>(a.w, hoff + c, a.param_bf16, w[k]);
    if (c < D && a.b) load_params<VEC>(a.b, hoff + c, a.param_bf16, b[k]);
  }
  // (teams past the last strip have no rows)
  for (int64_t t = strip < strips ? strip : a.rows; t < a.rows; t += strips) {
    const int64_t row = t * H + h;
    const float mean = a.mean_in[row], rstd = a.rstd_in[row];
    float xh[K][VEC], dn[K][VEC], s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * VEC;
      if (c < D) {
        float z[VEC];
        load_vec<E, VEC>(reinterpret_cast<const E*>(a.x) + row * D + c, xh[k]);
        load_vec<E, VEC>(reinterpret_cast<const E*>(a.dy) + row * D + c, dn[k]);
        if (a.gate) load_vec<E, VEC>(reinterpret_cast<const E*>(a.gate) + row * D + c, z);
#pragma unroll
        for (int i = 0; i < VEC; ++i) xh[k][i] = (xh[k][i] - mean) * rstd;
        if (a.gate) {
          float dz[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float sg = sigmoid_f32(z[i]);
            dz[i] = dn[k][i] * (xh[k][i] * w[k][i] + b[k][i]) * (sg * (1.f + z[i] * (1.f - sg)));
            dn[k][i] *= z[i] * sg;
          }
          store_vec<E, VEC>(reinterpret_cast<E*>(a.dgate) + row * D + c, dz);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          dw[k][i] += dn[k][i] * xh[k][i];
          db[k][i] += dn[k][i];
          dn[k][i] *= w[k][i];
          s0 += dn[k][i];
          s1 += dn[k][i] * xh[k][i];
        }
      }
    }
    const float m0 = team_sum<L>(s0, red) / (float)D;
    const float m1 = team_sum<L>(s1, red) / (float)D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * VEC;
      if (c < D) {
        float dx[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) dx[i] = rstd * (dn[k][i] - m0 - xh[k][i] * m1);
        store_vec<E, VEC>(reinterpret_cast<E*>(a.dx) + row * D + c, dx);
      }
    }
  }
  if (!params) return;
  if constexpr (TEAMS > 1) {
    if (shared_head) {                     // H == 1: the workgroup's teams share the columns
      for (int q = 0; q < TEAMS; ++q) {
        if (team == q) {
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const int at = (k * VEC + i) * L + lane;
              part[0][at] = q ? part[0][at] + dw[k][i] : dw[k][i];
              part[1][at] = q ? part[1][at] + db[k][i] : db[k][i];
            }
        }
        __syncthreads();
      }
      if (team != 0) return;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          dw[k][i] = part[0][(k * VEC + i) * L + lane];
          db[k][i] = part[1][(k * VEC + i) * L + lane];
        }
    }
  }
  const int64_t prow_ = shared_head ? blockIdx.x : strip;
  if (!shared_head && strip >= strips) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * L + lane) * VEC;
    if (c < D) {
      store_vec<float, VEC>(a.part + (prow_ * 2) * H * D + hoff + c, dw[k]);
      store_vec<float, VEC>(a.part + (prow_ * 2 + 1) * H * D + hoff + c, db[k]);
    }
  }
}

__global__ __launch_bounds__(1024) void norm_param_grads_kernel(NormArgs a, int64_t rows) {
  const int64_t HD = (int64_t)a.H * a.D;
  column_sums(a.part, rows, 2 * HD, [&](int64_t c, float v) {
    void* p = c < HD ? a.dw : a.db;
    if (!p) return;
    const int64_t at = c < HD ? c : c - HD;
    if (a.param_bf16) reinterpret_cast<bf16*>(p)[at] = (bf16)v;
    else reinterpret_cast<float*>(p)[at] = v;
  });
}

// A row's team: as many lanes as the row has vectors, up to a wave with four of them a
// lane, then the whole workgroup.
struct NormShape {
  int lanes, k;
};
static NormShape norm_shape(int D, int vec) {
  const int nv = (D + vec - 1) / vec;
  if (nv <= 8) return {8, 1};
  if (nv <= 16) return {16, 1};
  if (nv <= 32) return {32, 1};
  if (nv <= 64) return {64, 1};
  if (nv <= 128) return {64, 2};
  if (nv <= 256) return {64, 4};
  if (nv <= 1024) return {256, 4};
  if (nv <= 2048) return {256, 8};
  return {256, 32};                        // rows of at most kNormMaxWidth elements
}
static int norm_vec(int D, int is_bf16) { return D % (is_bf16 ? 8 : 4) == 0 ? (is_bf16 ? 8 : 4) : 1; }

// Strips of rows per head: enough teams for four workgroups per CU, and at least 16 rows
// a strip, so that the shares stay below a tenth of the traffic.
static int64_t norm_strips(int64_t rows, int H, int teams) {
  const int64_t want = (int64_t)4 * 256 * teams / H;
  const int64_t most = (rows + 15) / 16;
  int64_t s = want < most ? want : most;
  return s < 1 ? 1 : s;
}
int64_t norm_bwd_strips(int64_t rows, int H, int D, int is_bf16) {
  const NormShape n = norm_shape(D, norm_vec(D, is_bf16));
  const int teams = 256 / n.lanes;
  const int64_t s = norm_strips(rows, H, teams);
  return H == 1 ? (s + teams - 1) / teams : s;
}

template <typename E, int VEC, int L, int K, bool BWD>
static hipError_t norm_run(const NormArgs& a, hipStream_t s) {
  constexpr int TEAMS = 256 / L;
  if (!BWD) {
    const int64_t blocks = (a.rows * a.H + TEAMS - 1) / TEAMS;
    if (blocks == 0) return hipSuccess;
    if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
    norm_fwd_kernel<E, VEC, L, K><<<(unsigned)blocks, 256, 0, s>>>(a);
    return hipGetLastError();
  }
  const int shared_head = a.H == 1;
  int64_t strips = norm_strips(a.rows, a.H, TEAMS);
  if (shared_head) strips = (strips + TEAMS - 1) / TEAMS * TEAMS;   // whole workgroups
  const int64_t blocks = (strips * a.H + TEAMS - 1) / TEAMS;
  if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  norm_bwd_kernel<E, VEC, L, K><<<(unsigned)blocks, 256, 0, s>>>(a, strips, shared_head);
  if (a.dw || a.db) {
    const int64_t cols = (int64_t)2 * a.H * a.D;
    norm_param_grads_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, s>>>(a, shared_head ? blocks : strips);
  }
  return hipGetLastError();
}
template <typename E, int VEC, bool BWD>
static hipError_t norm_teams(const NormArgs& a, hipStream_t s) {
  const NormShape n = norm_shape(a.D, VEC);
  if (n.lanes == 8) return norm_run<E, VEC, 8, 1, BWD>(a, s);
  if (n.lanes == 16) return norm_run<E, VEC, 16, 1, BWD>(a, s);
  if (n.lanes == 32) return norm_run<E, VEC, 32, 1, BWD>(a, s);
  if (n.lanes == 64) {
    if (n.k == 1) return norm_run<E, VEC, 64, 1, BWD>(a, s);
    if (n.k == 2) return norm_run<E, VEC, 64, 2, BWD>(a, s);
    return norm_run<E, VEC, 64, 4, BWD>(a, s);
  }
  if (n.k == 4) return norm_run<E, VEC, 256, 4, BWD>(a, s);
  if constexpr (VEC <= 4)
    if (n.k == 8) return norm_run<E, VEC, 256, 8, BWD>(a, s);
  if constexpr (VEC == 1)
    if (a.D <= kNormMaxWidth) return norm_run<E, VEC, 256, 32, BWD>(a, s);
  return hipErrorInvalidConfiguration;
}
template <bool BWD>
static hipError_t norm_types(const NormArgs& a, hipStream_t s) {
  if (norm_vec(a.D, a.bf16) > 1)
    return a.bf16 ? norm_teams<bf16, 8, BWD>(a, s) : norm_teams<float, 4, BWD>(a, s);
  return a.bf16 ? norm_teams<bf16, 1, BWD>(a, s) : norm_teams<float, 1, BWD>(a, s);
}
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) { return norm_types<false>(a, s); }
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) { return norm_types<true>(a, s); }

}  // namespace gdn
