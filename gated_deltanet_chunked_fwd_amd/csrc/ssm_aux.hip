// The selective scan's small kernels: the chain over segments, the gates' gradients and
// the sums over a group's heads.
#include "ssm_scan.h"

namespace gdn {

// The chunks and segments in front of every sequence of a packed batch, and behind the last:
// one workgroup, 1024 sequences a round.
__global__ __launch_bounds__(1024) void ssm_offsets_kernel(SsmSeqs q, int32_t* chunk_off, int32_t* seg_off) {
  __shared__ int sSum[2][16];
  const int tid = threadIdx.x, wave = tid >> 6;
  int c0 = 0, s0 = 0;
  for (int n0 = 0; n0 < q.N; n0 += 1024) {
    const int n = n0 + tid;
    const int nch = n < q.N ? (q.cu[n + 1] - q.cu[n] + kChunk - 1) / kChunk : 0;
    const int ns = n < q.N ? max(1, (nch + q.seg_chunks - 1) / q.seg_chunks) : 0;
    const int ic = wave_scan_i32(nch), is = wave_scan_i32(ns);
    if ((tid & 63) == 63) {
      sSum[0][wave] = ic;
      sSum[1][wave] = is;
    }
    __syncthreads();
    int cw = c0, sw = s0;                  // in front of the wave
    for (int w = 0; w < 16; ++w) {
      if (w < wave) {
        cw += sSum[0][w];
        sw += sSum[1][w];
      }
      c0 += sSum[0][w];
      s0 += sSum[1][w];
    }
    if (n < q.N) {
      chunk_off[n] = cw + ic - nch;
      seg_off[n] = sw + is - ns;
    }
    __syncthreads();
  }
  if (tid == 0) {
    chunk_off[q.N] = c0;
    seg_off[q.N] = s0;
  }
}

hipError_t launch_ssm_offsets(const SsmSeqs& q, int32_t* chunk_off, int32_t* seg_off, hipStream_t s) {
  ssm_offsets_kernel<<<1, 1024, 0, s>>>(q, chunk_off, seg_off);
  return hipGetLastError();
}

// One wave per (chunk, head), lane = step; blockIdx.y = 1: last to first (step j is token
// 63 - j and its decay the next token's, none behind the sequence's end).  Formed once here
// instead of by each of the scans' workgroups (whose softplus and fp64 sums were on their
// critical path): 5 us for 4 x 4096 tokens of 16 heads, and 17 MB for the scans to read.
__global__ __launch_bounds__(256) void ssm_gates_kernel(SsmSeqs q, SsmGates g, float* fwd, float* rev_out) {
  const int lane = threadIdx.x & 63, H = q.H;
  const uint32_t item = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t cg = item / (uint32_t)H;
  const int h = (int)(item % (uint32_t)H);
  if (cg >= q.chunks) return;
  const int rev = blockIdx.y;
  int64_t tok0;
  int len, c;
  if (q.cu) {
    const SsmSeq f = find_seq<false>(q, cg);
    tok0 = q.cu[f.n];
    len = q.cu[f.n + 1] - q.cu[f.n];
    c = (int)(cg - f.chunks);
  } else {
    const int64_t nch = (q.T + kChunk - 1) / kChunk;
    tok0 = cg / nch * q.T;
    len = (int)q.T;
    c = (int)(cg % nch);
  }
  SsmHead hd;
  hd.init(g, h);
  const int t = c * kChunk + (rev ? kChunk - 1 - lane : lane);
  const int64_t at = (tok0 + t) * H + h;
  const float del = t < len ? hd.delta(g, load_scalar(g.dt, at, g.dt_bf16)) : 0.f;
  float ddec = del;
  if (rev) {                 // the lane before holds the next token; the chunk's last one's is a chunk away
    ddec = __shfl_up(del, 1, 64);
    if (lane == 0) ddec = t + 1 < len ? hd.delta(g, load_scalar(g.dt, at + H, g.dt_bf16)) : 0.f;
  }
  // (a decay below 2^-4096 is zero in any type: clamped there, U keeps its precision, and its
  // differences are numbers, whatever came before in the chunk.  No delta, as behind the
  // sequence's end, is no decay, also of an infinite A.)
  const double step = ddec == 0.f ? 0.0 : (double)ddec * hd.a2;
  const double U = wave_scan_f64(step < -4096.0 ? -4096.0 : step);
  const double end = readlane_f64(U, 63);
  const float hi = (float)U;
  float* o = (rev ? rev_out : fwd) + (cg * H + h) * kGateFloats + lane;
  o[kGateU] = hi;
  o[kGateUlo] = (float)(U - (double)hi);
  o[kGateW] = (rev ? 1.f : del) * __builtin_amdgcn_exp2f((float)(end - U));
  o[kGateDelta] = del;
}

hipError_t launch_ssm_gates(const SsmSeqs& q, const SsmGates& g, float* fwd, float* rev, hipStream_t s) {
  const int64_t blocks = (q.chunks * q.H + 3) / 4;
  if (blocks == 0) return hipSuccess;
  if (blocks > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  ssm_gates_kernel<<<dim3((unsigned)blocks, rev ? 2 : 1), 256, 0, s>>>(q, g, fwd, rev);
  return hipGetLastError();
}

// Segments' end states (from a zero start) -> their start states, in place.  One thread
// per VEC state elements walks the segments of its (sequence, head), eight at a time, the
// next eight read ahead, so a long chain costs its bytes, not its latencies.  448 states
// of 64 KB: 10 us (5.7 TB/s).  VEC = 1 where VEC = 4 makes too few workgroups to hide the
// latency (4 heads of 256 segments: 22 us).
struct SsmMerges {
  SsmSeqs q;
  SsmMerge m[2];
};
template <int VEC>
__global__ __launch_bounds__(256) void ssm_merge_kernel(SsmMerges a, int elems) {
  typedef float vec __attribute__((ext_vector_type(VEC)));
  const SsmMerge& m = a.m[blockIdx.y];
  const uint32_t per = (uint32_t)elems / (256 * VEC);   // workgroups per (sequence, head)
  const uint32_t nh = blockIdx.x / per;
  const int H = a.q.H, n = __builtin_amdgcn_readfirstlane((int)(nh / H)), h = __builtin_amdgcn_readfirstlane((int)(nh % H));
  const int e = ((int)(blockIdx.x % per) * 256 + threadIdx.x) * VEC;
  int s0 = n * a.q.segs, segs = a.q.segs;
  if (a.q.cu) {
    if (a.q.chunk_off) {
      s0 = a.q.seg_off[n];
      segs = a.q.seg_off[n + 1] - s0;
    } else {                               // (up to 64 sequences, a lane each)
      const int l = threadIdx.x & 63;
      const int ns = l < a.q.N ? max(1, ((a.q.cu[l + 1] - a.q.cu[l] + kChunk - 1) / kChunk + a.q.seg_chunks - 1) / a.q.seg_chunks) : 0;
      s0 = __builtin_amdgcn_readlane(wave_scan_i32(ns) - ns, n);
      segs = __builtin_amdgcn_readlane(ns, n);
    }
  }
  constexpr int U = 8;
  const int64_t step = (int64_t)(m.rev ? -H : H);         // slots from a segment to the next in order
  const int64_t slot0 = ((int64_t)s0 + (m.rev ? segs - 1 : 0)) * H + h;
  vec s[U], t[U];
  float d[U], f[U];
  // (the last segment's end state was not formed: a segment before it is read instead)
  auto read = [&](int j0, vec (&x)[U], float (&y)[U]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t at = slot0 + min(j0 + i, max(segs - 2, 0)) * step;
      x[i] = *reinterpret_cast<const vec*>(m.state + at * elems + e);
      y[i] = m.decay[at];
    }
  };
  vec cur = 0.f;
  if (m.h0) cur = *reinterpret_cast<const vec*>(m.h0 + (int64_t)nh * elems + e);
  read(0, s, d);
  for (int j0 = 0; j0 < segs; j0 += U) {
    if (j0 + U < segs) read(j0 + U, t, f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (j0 + i < segs) {
        *reinterpret_cast<vec*>(m.state + (slot0 + (j0 + i) * step) * elems + e) = cur;
        cur = d[i] * cur + s[i];
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      s[i] = t[i];
      d[i] = f[i];
    }
  }
}

hipError_t launch_ssm_merge(const SsmSeqs& q, const SsmMerge* m, int count, int elems, hipStream_t s) {
  const int64_t nh = (int64_t)q.N * q.H;
  if (nh == 0) return hipSuccess;
  if (nh * (elems / 256) > kMaxDispatchItems / 256) return hipErrorInvalidConfiguration;
  SsmMerges a;
  a.q = q;
  for (int i = 0; i < 2; ++i) a.m[i] = m[i < count ? i : 0];
  // 16 bytes a thread, unless that leaves CUs without a workgroup
  if (nh * count * (elems / 1024) >= 512)
    ssm_merge_kernel<4><<<dim3((unsigned)(nh * (elems / 1024)), (unsigned)count), 256, 0, s>>>(a, elems);
  else
    ssm_merge_kernel<1><<<dim3((unsigned)(nh * (elems / 256)), (unsigned)count), 256, 0, s>>>(a, elems);
  return hipGetLastError();
}

__device__ __forceinline__ double wave_sum_f64(double x) { return readlane_f64(wave_scan_f64(x), 63); }

// Gradients of the gates of one (segment, head).  With m_t = C_t . dC_t - delta_t x_t . du_t
// (what of the flow from earlier to later tokens ends at t, less what starts there), the
// flow across the decay of token t is da_t = <h, dh> at the segment's end + sum_{r >= t} m_r:
// the sum runs over one segment only, so its rounding does not grow with the sequence.
// Sums in fp64; a wave takes a chunk.  Bound by its chain of loads: the unit, the two states
// of <h, dh>, the dots.  8192 packed tokens of 16 heads, segments of 5 chunks: 10 us with four
// waves or eight; 4 x 4096 tokens, segments of 8: 19 us with four, 17 with eight.
template <typename DOT, int NW>
__global__ __launch_bounds__(64 * NW) void ssm_gate_grads_kernel(SsmGateGrads a) {
  __shared__ double sRed[NW][3], sTot[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  SsmUnit u;
  u.init(a.seqs, blockIdx.x);
  const int h = u.h, H = a.seqs.H;
  const int64_t nh = (int64_t)u.n * H + h;
  const double A = (double)load_scalar(a.A, h, a.param_bf16);

  // <h, dh> at the segment's end
  double carry = 0.0;
  {
    const float *hp = nullptr, *gp = nullptr;
    double f = 1.0;
    if (u.seg + 1 < u.segs) {
      hp = a.hstart + ((u.sg + 1) * H + h) * a.elems;
      gp = a.gstart + (u.sg * H + h) * a.elems;
      // gp is the gradient behind the decay of the next segment's first token
      const float* gn = a.gates + ((u.chunk0 + u.c1) * H + h) * kGateFloats;
      f = exp2((double)gn[kGateU] + (double)gn[kGateUlo]);
    } else if (a.dhT) {
      hp = a.hT + nh * a.elems;
      gp = a.dhT + nh * a.elems;
    }
    if (hp) {
      double s = 0.0;
      for (int i = tid * 4; i < a.elems; i += 256 * NW) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(hp + i), y = *reinterpret_cast<const f32x4*>(gp + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) s += (double)x[k] * (double)y[k];
      }
      s = wave_sum_f64(s);
      if (lane == 0) sTot[wave] = s;
      __syncthreads();
      s = 0.0;
      for (int w = 0; w < NW; ++w) s += sTot[w];
      carry = f * s;
      __syncthreads();
    }
  }

  double pA = 0.0, pb = 0.0, pD = 0.0;
  for (int cg = u.c1 - 1; cg >= u.c0; cg -= NW) {
    const int c = cg - wave;
    const int t = c * kChunk + lane;
    const bool ok = c >= u.c0 && t < u.len;
    double m = 0.0, xdu = 0.0;
    float del = 0.f;
    int64_t tok = 0;
    if (ok) {
      tok = (u.tok0 + t) * H + h;
      del = a.gates[((u.chunk0 + c) * H + h) * kGateFloats + kGateDelta + lane];
      const int64_t at = ((u.chunk0 + c) * H + h) * kChunk + lane;
      xdu = (double)reinterpret_cast<const DOT*>(a.xdu)[at];
      m = (double)reinterpret_cast<const DOT*>(a.cdc)[at] - (double)del * xdu;
      if (a.dyx) pD += (double)reinterpret_cast<const DOT*>(a.dyx)[at];
    }
    const double incl = wave_scan_f64(m);
    const double tot = readlane_f64(incl, 63);
    if (lane == 0) sTot[wave] = tot;
    __syncthreads();
    double later = carry;
    for (int w = 0; w < wave; ++w) later += sTot[w];   // wave w holds a later chunk
    if (ok) {
      const double da = t > 0 || a.has_h0 ? later + (tot - incl + m) : 0.0;
      double g = xdu + A * da;
      if (a.softplus) g *= -expm1(-(double)del);   // softplus' = 1 - exp(-softplus)
      if (a.dt_bf16) reinterpret_cast<bf16*>(a.ddt)[tok] = (bf16)(float)g;
      else reinterpret_cast<float*>(a.ddt)[tok] = (float)g;
      pA += (double)del * da;
      pb += g;
    }
    for (int w = 0; w < NW; ++w) carry += sTot[w];
    __syncthreads();
  }
  pA = wave_sum_f64(pA);
  pb = wave_sum_f64(pb);
  pD = wave_sum_f64(pD);
  if (lane == 0) {
    sRed[wave][0] = pA;
    sRed[wave][1] = pb;
    sRed[wave][2] = pD;
  }
  __syncthreads();
  if (tid < 3) {
    double s = 0.0;
    for (int w = 0; w < NW; ++w) s += sRed[w][tid];
    a.part[((int64_t)blockIdx.x) * 3 + tid] = s;
  }
}

__device__ __forceinline__ void store_param(void* p, int i, float v, int is_bf16) {
  if (!p) return;
  if (is_bf16) reinterpret_cast<bf16*>(p)[i] = (bf16)v;
  else reinterpret_cast<float*>(p)[i] = v;
}

// Sums the segments' shares of one head's parameter gradients, in a fixed order.
__device__ __forceinline__ void sum_params(const SsmGateGrads& a, int h) {
  __shared__ double sRed[4][3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, H = a.seqs.H;
  const int64_t segs = a.seqs.units / H;
  double s[3] = {0.0, 0.0, 0.0};
  for (int64_t i = tid; i < segs; i += 256)
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += a.part[(i * H + h) * 3 + k];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    s[k] = wave_sum_f64(s[k]);
    if (lane == 0) sRed[wave][k] = s[k];
  }
  __syncthreads();
  if (tid < 3) {
    const float v = (float)((sRed[0][tid] + sRed[1][tid]) + (sRed[2][tid] + sRed[3][tid]));
    store_param(tid == 0 ? a.dA : tid == 1 ? a.dbias : a.dD, h, v, a.param_bf16);
  }
}

// The last sums: the parameters' gradients (the first H workgroups), and behind them the
// heads of each group of dB and dC, in [tokens, H, n] fp32 -> out [tokens, G, n], 16 bytes a
// thread.  Bound by memory: 8192 tokens of 16 heads and 2 groups, n = 128, 143 MB: 21 us
// (6.7 TB/s).
// In one launch since the first alone is a few workgroups waiting for memory.
template <typename E>
__global__ __launch_bounds__(256) void ssm_sums_kernel(SsmGateGrads a, SsmHeadSum b) {
  const uint32_t H = a.seqs.H;
  if (blockIdx.x < H) {
    sum_params(a, (int)blockIdx.x);
    return;
  }
  const uint32_t block = blockIdx.x - H, which = block >= b.blocks;
  const float* in = b.in[which];
  E* out = reinterpret_cast<E*>(b.out[which]);
  for (int64_t i = (int64_t)(block - which * b.blocks) * 256 + threadIdx.x; i < b.quads; i += (int64_t)b.blocks * 256) {
    const int64_t tg = i / b.n4;           // (token, group)
    const float* p = in + (tg * b.per * b.n4 + i % b.n4) * 4;
    f32x4 s = *reinterpret_cast<const f32x4*>(p);
    for (int k = 1; k < b.per; ++k) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p + (int64_t)k * b.n4 * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += x[e];
    }
    store4(out + i * 4, s);
  }
}

hipError_t launch_ssm_gate_grads(const SsmGateGrads& a, hipStream_t s) {
  if (a.seqs.units > kMaxDispatchItems / 512) return hipErrorInvalidConfiguration;
  if (a.seqs.units == 0) return hipSuccess;
  const bool wide = a.seqs.seg_chunks > 4;
  const unsigned n = (unsigned)a.seqs.units;
  if (a.dots_f64) {
    if (wide) ssm_gate_grads_kernel<double, 8><<<n, 512, 0, s>>>(a);
    else ssm_gate_grads_kernel<double, 4><<<n, 256, 0, s>>>(a);
  } else {
    if (wide) ssm_gate_grads_kernel<float, 8><<<n, 512, 0, s>>>(a);
    else ssm_gate_grads_kernel<float, 4><<<n, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_ssm_sums(const SsmGateGrads& a, const SsmHeadSum& heads, bool is_bf16, hipStream_t s) {
  SsmHeadSum b = heads;
  const int64_t want = (b.quads + 255) / 256;
  b.blocks = (uint32_t)(want < 4096 ? want : 4096);
  const unsigned grid = (unsigned)a.seqs.H + 2 * b.blocks;
  if (is_bf16) ssm_sums_kernel<bf16><<<grid, 256, 0, s>>>(a, b);
  else ssm_sums_kernel<float><<<grid, 256, 0, s>>>(a, b);
  return hipGetLastError();
}

hipError_t launch_ssm_scan(const SsmScans& a, int count, bool is_bf16, int dk, int dv, int mode,
                           hipStream_t s) {
  return is_bf16 ? launch_ssm_scan_bf16(a, count, dk, dv, mode, s)
                 : launch_ssm_scan_f32(a, count, dk, dv, mode, s);
}

}  // namespace gdn
