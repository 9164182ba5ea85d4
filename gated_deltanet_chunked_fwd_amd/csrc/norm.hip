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
//
// bf16: forward, gated, 16384 rows of 16 heads of 128, 203 MB: 42 us (4.8 TB/s; a copy reaches
// 5.3).  Backward of 16384 rows of 2048, 201 MB: 39 us, and 5 us for the second kernel.  fp32
// (8192 rows, as many bytes): 40 us and 40 in all.
#include <algorithm>

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
        if (a.gate) o *= z[i] * sigmoid<E>(z[i]);
        y[i] = o;
      }
      store_vec<E, VEC>(reinterpret_cast<E*>(a.y) + row * D + c, y);
    }
  }
}

// Two sums at once; a workgroup-wide team alternates between two buffers, so one barrier
// a call is enough.
template <int L>
__device__ __forceinline__ void team_sum2(float& u, float& v, float (*red)[2][4], int& turn) {
#pragma unroll
  for (int d = 1; d < (L < 64 ? L : 64); d <<= 1) {
    u += __shfl_xor(u, d, 64);
    v += __shfl_xor(v, d, 64);
  }
  if constexpr (L == 256) {
    float(*r)[4] = red[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
      r[0][threadIdx.x >> 6] = u;
      r[1][threadIdx.x >> 6] = v;
    }
    __syncthreads();
    u = (r[0][0] + r[0][1]) + (r[0][2] + r[0][3]);
    v = (r[1][0] + r[1][1]) + (r[1][2] + r[1][3]);
  }
}

template <typename E, int VEC, int L, int K>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormArgs a, int64_t strips, int shared_head) {
  constexpr int TEAMS = 256 / L;
  __shared__ float red[2][2][4];
  int turn = 0;
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
  // (teams past the last strip have no rows; the next row is read while this one is used)
  Raw<E, VEC> nx[K], ny[K], nz[K];
  float nmean = 0.f, nrstd = 0.f;
  auto load = [&](int64_t t) {
    const int64_t row = t * H + h;
    nmean = a.mean_in[row];
    nrstd = a.rstd_in[row];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * VEC;
      if (c < D) {
        nx[k].load(reinterpret_cast<const E*>(a.x) + row * D + c);
        ny[k].load(reinterpret_cast<const E*>(a.dy) + row * D + c);
        if (a.gate) nz[k].load(reinterpret_cast<const E*>(a.gate) + row * D + c);
      }
    }
  };
  const int64_t first = strip < strips ? strip : a.rows;
  if (first < a.rows) load(first);
  for (int64_t t = first; t < a.rows; t += strips) {
    const int64_t row = t * H + h;
    const float mean = nmean, rstd = nrstd;
    Raw<E, VEC> rx[K], ry[K], rz[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      rx[k] = nx[k];
      ry[k] = ny[k];
      rz[k] = nz[k];
    }
    if (t + strips < a.rows) load(t + strips);
    float xh[K][VEC], dn[K][VEC], s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * VEC;
      if (c < D) {
        float z[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          xh[k][i] = (rx[k][i] - mean) * rstd;
          dn[k][i] = ry[k][i];
          z[i] = rz[k][i];
        }
        if (a.gate) {
          float dz[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float sg = sigmoid<E>(z[i]);
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
    team_sum2<L>(s0, s1, red, turn);
    const float m0 = s0 / (float)D, m1 = s1 / (float)D;
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

// Going back a lane also holds its share of dw and db: rows of more than a vector a lane of
// a wave take the whole workgroup (16384 rows of 2048 bf16 elements: 39 us; a wave a row
// and four vectors a lane, at one or two waves per SIMD, 49 to 67 us).
static NormShape norm_bwd_shape(int D, int vec) {
  const NormShape n = norm_shape(D, vec);
  if (n.lanes < 64 || n.k == 1) return n;
  const int nv = (D + vec - 1) / vec;
  return {256, nv <= 256 ? 1 : n.k};
}
// Strips of rows per head, a team each, and rows of shares (H = 1: a workgroup's teams add
// theirs up): teams for four workgroups per CU, and at least 16 rows to a row of shares, so
// that these stay below a tenth of the traffic; at fewer rows, a row a team.
struct NormStrips {
  int64_t strips, shares;
};
static NormStrips norm_strips(int64_t rows, int H, int lanes) {
  const int teams = 256 / lanes;
  if (H == 1) {
    const int64_t few = std::min<int64_t>((rows + teams - 1) / teams, 256);
    const int64_t wgs = std::max<int64_t>(std::max<int64_t>(std::min<int64_t>(rows / 16, 4 * 256), few), 1);
    return {wgs * teams, wgs};
  }
  const int64_t want = (int64_t)4 * 256 * teams / H, most = (rows + 15) / 16;
  const int64_t s = std::max<int64_t>(std::min(want, most), 1);
  return {s, s};
}
int64_t norm_bwd_strips(int64_t rows, int H, int D, int is_bf16) {
  return norm_strips(rows, H, norm_bwd_shape(D, norm_vec(D, is_bf16)).lanes).shares;
}
// Forward, a team a row; going back the strips are fewer, and the sums take a workgroup of
// 1024 for 32 columns.
bool norm_fits(int64_t rows, int H, int D, int is_bf16) {
  const int64_t most = kMaxDispatchItems / 256 * (256 / norm_shape(D, norm_vec(D, is_bf16)).lanes);
  return H <= most && rows <= most / H && (int64_t)2 * H * D <= kMaxDispatchItems / 1024 * 32;
}

template <typename E, int VEC, int L, int K>
static hipError_t norm_fwd_run(const NormArgs& a, hipStream_t s) {
  constexpr int TEAMS = 256 / L;
  const int64_t blocks = (a.rows * a.H + TEAMS - 1) / TEAMS;
  if (blocks == 0) return hipSuccess;
  if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  norm_fwd_kernel<E, VEC, L, K><<<(unsigned)blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <typename E, int VEC, int L, int K>
static hipError_t norm_bwd_run(const NormArgs& a, hipStream_t s) {
  constexpr int TEAMS = 256 / L;
  const int shared_head = a.H == 1;
  const NormStrips st = norm_strips(a.rows, a.H, L);
  const int64_t blocks = (st.strips * a.H + TEAMS - 1) / TEAMS;
  if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  norm_bwd_kernel<E, VEC, L, K><<<(unsigned)blocks, 256, 0, s>>>(a, st.strips, shared_head);
  if (a.dw || a.db) {
    const int64_t cols = (int64_t)2 * a.H * a.D;
    norm_param_grads_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, s>>>(a, st.shares);
  }
  return hipGetLastError();
}
// The kernel of a row's shape; rows of at most kNormMaxWidth elements reach 1024 vectors of
// bf16, 2048 of fp32, 8192 single elements.
template <typename E, int VEC, bool BWD>
static hipError_t norm_teams(const NormArgs& a, hipStream_t s) {
  const NormShape n = BWD ? norm_bwd_shape(a.D, VEC) : norm_shape(a.D, VEC);
#define GDN_NORM(L, K)                                      \
  if (n.lanes == L && n.k == K) {                           \
    if constexpr (BWD) return norm_bwd_run<E, VEC, L, K>(a, s); \
    else return norm_fwd_run<E, VEC, L, K>(a, s);           \
  }
  GDN_NORM(8, 1)
  GDN_NORM(16, 1)
  GDN_NORM(32, 1)
  GDN_NORM(64, 1)
  if constexpr (BWD) {
    GDN_NORM(256, 1)
  } else {
    GDN_NORM(64, 2)
    GDN_NORM(64, 4)
  }
  GDN_NORM(256, 4)
  if constexpr (VEC <= 4) {
    GDN_NORM(256, 8)
  }
  if constexpr (VEC == 1) {
    if (a.D <= kNormMaxWidth) {
      GDN_NORM(256, 32)
    }
  }
#undef GDN_NORM
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
