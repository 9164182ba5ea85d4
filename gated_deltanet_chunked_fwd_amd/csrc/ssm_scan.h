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
// decayed q k products, the decayed v) enters as a sum of bf16 terms.  The state's update
// takes three (24 bits: the final state is an fp32 result).  In the forward pass q k products
// and the state in the outputs take two (17 bits), 2^-8 of what the outputs are rounded to: y
// is then 1e-4 from fp32 arithmetic in the 2-norm, its own rounding being 1.7e-3 (with three
// for the products 2e-5, and 4 x 4096 tokens of 16 heads take 123 us instead of 111; with one
// for the state 4e-4, and where its products cancel 2^-8 of their sizes).  In the backward
// pass they take three: the gates' gradients are sums of flows hundreds of times their size,
// and with two terms ddt_bias was off by up to 2e-2 of itself (1300 tokens, 2 heads), now by
// 2e-3, and ddt by 1e-4, now 1e-5, which is what fp32 arithmetic leaves; up to 4% of the
// time.  fp32 tensors use fp32 MFMA, and their gradients fp64 MFMA with the q k products kept
// as doubles: with fp32 sums the error of dA and ddt_bias reached 9e-6 of them, now 6e-7 (2 x
// 777 tokens of 4 heads: 29 us instead of 16).
//
// Mapping.  One workgroup of DV / 16 waves per (segment, head); a wave owns 16 columns of
// the state for all DK rows, in registers, in tile order (gdn_device.h), so the state feeds
// the next product without leaving them.  Per chunk the workgroup stages q, k and v in LDS
// (the next chunk's global loads in flight meanwhile), splits the lower tiles of q k^T over
// the waves, and each wave then runs its columns.  A lane keeps a few LDS addresses, of which
// every read is a constant away.  The outputs come out transposed (4 consecutive columns of
// one token per lane).
//
// Bound, 4 x 4096 bf16 tokens of 16 heads, one group, n = p = 128 (176 MB, 53 GFLOP in
// bf16 terms): 70 us forward.  The loads and stores alone take 39 us, the arithmetic
// without them 68: reads of q and k from LDS by every wave, the splits into terms and the
// products.  With two workgroups per CU these hide each other, but what one wave does after
// the other shows.  Backward of the same: about 330 us for three scans.
#pragma once
#include <type_traits>

#include "gdn_device.h"
#include "mixer_launch.h"

namespace gdn {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// An MFMA operand as a sum of N terms of the tensors' type.
template <typename E, int N>
struct Terms;
template <int N>
struct Terms<float, N> {
  static constexpr int n = 1;
  f32x8 t[1];
  __device__ __forceinline__ void set(const f32x8& v) { t[0] = v; }
};
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
// Two floats rounded to bf16 in a dword, and what the rounding left (exact).
__device__ __forceinline__ uint32_t split2(float& x, float& y) {
  const uint32_t u = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
  x -= __uint_as_float(u << 16);
  y -= __uint_as_float(u & 0xffff0000u);
  return u;
}
template <int N>
struct Terms<bf16, N> {
  static constexpr int n = N;
  bf16x8 t[N];
  __device__ __forceinline__ void set(f32x8 r) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      u32x4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = r[2 * e], y = r[2 * e + 1];
        u[e] = split2(x, y);
        r[2 * e] = x;
        r[2 * e + 1] = y;
      }
      t[i] = __builtin_bit_cast(bf16x8, u);
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
// An operand with zeros for what is NaN or infinite.
template <typename F>
__device__ __forceinline__ F finite_only(F v) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (!(__builtin_fabsf((float)v[i]) < __builtin_inff())) v[i] = 0;
  return v;
}

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
  return x + ((row > 0 ? r0 : 0.0) + (row > 1 ? r1 : 0.0) + (row > 2 ? r2 : 0.0));
}
// Inclusive prefix sum of ints over the wave.
__device__ __forceinline__ int wave_scan_i32(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true);
  const int r0 = __builtin_amdgcn_readlane(x, 15), r1 = __builtin_amdgcn_readlane(x, 31);
  const int r2 = __builtin_amdgcn_readlane(x, 47);
  const int row = (threadIdx.x & 63) >> 4;
  return x + ((row > 0 ? r0 : 0) + (row > 1 ? r1 : 0) + (row > 2 ? r2 : 0));
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

__device__ __forceinline__ int64_t uniform64(int64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)x >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The sequence of a packed batch that owns item `at` of those it counts (its chunks, or its
// segments, at least one each), with what the sequences before it have of both.  Every
// lane of the wave calls it; the result is uniform.  Up to 64 sequences are counted on the
// spot, a lane each; more have tables (ssm_offsets_kernel), of which the lanes look at 64
// places of the range that is left at once (counted on the spot, 8000 sequences of 16 tokens
// of 8 heads, 64 x 64, took 2.8 ms, now 0.67; as batch rows they take 0.58).
struct SsmSeq {
  int n;
  int64_t chunks, segs;      // of the sequences before it
};
template <bool SEGS>
__device__ __forceinline__ SsmSeq find_seq(const SsmSeqs& q, int64_t at) {
  const int lane = threadIdx.x & 63;
  if (q.chunk_off) {
    const int32_t* off = SEGS ? q.seg_off : q.chunk_off;
    int n = 0, size = q.N;                 // the first n with off[n + 1] > at, one of `size` from n on
    while (size > 1) {
      const int step = (size + 63) / 64;
      const int l = __builtin_ctzll(__ballot(off[n + min((lane + 1) * step, size)] > at));
      n += l * step;
      size = min(step, size - l * step);
    }
    return {n, q.chunk_off[n], q.seg_off[n]};
  }
  const int nch = lane < q.N ? (q.cu[lane + 1] - q.cu[lane] + kChunk - 1) / kChunk : 0;
  const int ns = lane < q.N ? max(1, (nch + q.seg_chunks - 1) / q.seg_chunks) : 0;
  const int ic = wave_scan_i32(nch), is = wave_scan_i32(ns);
  const int l = __builtin_ctzll(__ballot((SEGS ? is : ic) > at));
  return {l, __builtin_amdgcn_readlane(ic - nch, l), __builtin_amdgcn_readlane(is - ns, l)};
}

struct SsmUnit {             // a (segment, head) unit of the launch
  int h, n, seg, segs;
  int64_t sg;                // global segment
  int64_t tok0;              // the sequence's first token
  int len, nch, c0, c1;      // the sequence's tokens and chunks; the segment's chunks
  int64_t chunk0;            // the sequence's first chunk over all sequences
  __device__ __forceinline__ void init(const SsmSeqs& q, uint32_t unit) {
    h = __builtin_amdgcn_readfirstlane((int)(unit % (uint32_t)q.H));
    sg = __builtin_amdgcn_readfirstlane((int)(unit / (uint32_t)q.H));
    if (q.cu) {
      const SsmSeq f = find_seq<true>(q, sg);
      n = f.n;
      seg = (int)(sg - f.segs);
      chunk0 = f.chunks;
      tok0 = q.cu[n];
      len = q.cu[n + 1] - q.cu[n];
    } else {
      n = (int)(sg / q.segs);
      seg = (int)(sg - (int64_t)n * q.segs);
      tok0 = (int64_t)n * q.T;
      len = (int)q.T;
      chunk0 = (int64_t)n * ((q.T + kChunk - 1) / kChunk);
    }
    // (one value for the workgroup: addresses formed from them stay in scalar registers)
    n = __builtin_amdgcn_readfirstlane(n);
    seg = __builtin_amdgcn_readfirstlane(seg);
    len = __builtin_amdgcn_readfirstlane(len);
    tok0 = uniform64(tok0);
    chunk0 = uniform64(chunk0);
    nch = (len + kChunk - 1) / kChunk;
    segs = max(1, (nch + q.seg_chunks - 1) / q.seg_chunks);
    c0 = seg * q.seg_chunks;
    c1 = min(nch, c0 + q.seg_chunks);
  }
};

// The gates of a (chunk, head), written by ssm_gates_kernel and read by the scans: four
// rows of 64 steps, U as two floats, the key's weight in the state behind the chunk, delta.
constexpr int kGateU = 0, kGateUlo = 64, kGateW = 128, kGateDelta = 192, kGateFloats = 256;

// Operands read from LDS at a lane's own address plus a constant: the addresses of a
// kernel's reads differ by constants from a few per-lane ones, which stay in registers.
template <typename E>
__device__ __forceinline__ typename Mma<E>::frag frag_at(const E* lane_base, int off) {
  return *reinterpret_cast<const typename Mma<E>::frag*>(lane_base + off);
}
// Transposed operand (col_frag) of the rows row, row + 1, .. and row + 16, ..: bf16 lanes
// address M[row + r16 / 4][four columns], fp32 lanes M[row][column].
__device__ __forceinline__ bf16x8 tr_frag_at(const bf16* lane_base, int off, int stride) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  typedef short i16x8 __attribute__((ext_vector_type(8)));
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_i16x4*)(__attribute__((address_space(3))) void*)(lane_base + off));
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_i16x4*)(__attribute__((address_space(3))) void*)(lane_base + off + 16 * stride));
  const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ f32x8 tr_frag_at(const float* lane_base, int off, int stride) {
  f32x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = lane_base[off + i * stride];
    r[4 + i] = lane_base[off + (16 + i) * stride];
  }
  return r;
}
// A lane's address for tr_frag_at: rows 4 q4 .. of a tile-order matrix, and the columns of
// its 16-lane group, four runs of four `run` apart.
template <typename E>
__device__ __forceinline__ const E* tr_base(const E* M, int stride, int col, int run, int r16, int q4) {
  return sizeof(E) == 2 ? M + (4 * q4 + (r16 >> 2)) * stride + col + run * (r16 & 3)
                        : M + 4 * q4 * stride + col + run * (r16 >> 2) + (r16 & 3);
}

// A chunk's rows of a token-major tensor as a buffer: `rows` rows of `bytes` from `base`.
// Reads past them give zero and writes are dropped, so a partial chunk needs no masks,
// and the number of memory operations of a step does not depend on it (their counters
// then let a wait for this step's loads leave its stores in flight).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_buffer(const void* base, int rows, uint32_t bytes) {
  const uint32_t size = (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)max(rows, 0) * bytes));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, size, 0x00027000);
}

// One chunk's rows of a tensor on their way from memory to LDS, NT threads.  TORD: rows
// are stored in tile order (gdn_device.h), which frees the transposed reads of bank
// conflicts.
template <typename E, int W, int NT, bool TORD>
struct SsmTile {
  static constexpr int EPV = 16 / (int)sizeof(E), VPR = W / EPV, NV = kChunk * VPR / NT;
  static_assert(NV * NT == kChunk * VPR && NT % VPR == 0, "a tile must split evenly over the threads");
  u32x4 v[NV];
  __device__ __forceinline__ void load(const E* base, int64_t stride, int c, int len, int rev, int tid) {
    const uint32_t rb = (uint32_t)stride * (uint32_t)sizeof(E);
    const __amdgpu_buffer_rsrc_t rs = chunk_buffer(base + (int64_t)c * kChunk * stride, min(kChunk, len - c * kChunk), rb);
    const int r0 = tid / VPR;
    const uint32_t o = (uint32_t)(rev ? kChunk - 1 - r0 : r0) * rb + (uint32_t)(tid % VPR) * 16u;
    const uint32_t step = rev ? 0u - (NT / VPR) * rb : (NT / VPR) * rb;
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, o + j * step, 0, 0));
  }
  __device__ __forceinline__ void store(E* s, int ls, int tid) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int r = (tid + NT * j) / VPR;
      *reinterpret_cast<u32x4*>(s + (TORD ? tord(r) : r) * ls + (tid % VPR) * EPV) = v[j];
    }
  }
  // whether an element is NaN or infinite: its exponent is the largest there is
  __device__ __forceinline__ bool not_finite() const {
    if constexpr (sizeof(E) == 2) {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 m = {0, 0};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[j][i] & 0x7fff7fffu));
      return m[0] >= 0x7f80 || m[1] >= 0x7f80;
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, v[j][i] & 0x7fffffffu);
      return m >= 0x7f800000u;
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

// One product of operands, added up in fp32 or fp64.  An fp64 product's result has row
// 4 i + q4 in a lane's element i, not 4 q4 + i: its first operand's lanes hold their rows
// in an order that makes up for it (wide_row).
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef double f64x8 __attribute__((ext_vector_type(8)));
template <typename M>
__device__ __forceinline__ f32x4 product(const typename M::frag& x, const typename M::frag& y, const f32x4& c) {
  return M::run(x, y, c);
}
template <typename M>
__device__ __forceinline__ f64x4 product(const f32x8& x, const f64x8& y, f64x4 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f64_16x16x4f64((double)x[e], y[e], c, 0, 0, 0);
  return c;
}
template <typename M>
__device__ __forceinline__ f64x4 product(const f32x8& x, const f32x8& y, f64x4 c) {
  return product<M>(x, __builtin_convertvector(y, f64x8), c);
}
__device__ __forceinline__ int wide_row(int r16) { return 4 * (r16 & 3) + (r16 >> 2); }

template <typename E, int DK, int DV, int MODE>
struct SsmCfg {
  static constexpr bool BF = sizeof(E) == 2;
  // a wave has one tile of 16 columns, so that four waves per SIMD cover each other's waits
  // (128 x 128 forward: 70 us against 76 with two tiles and half the waves; backward, whole
  // calls on one GPU in turn: 4 x 4096 tokens of 16 heads 466 us against 470, 9 x 4096 977
  // against 1024, 8 x 1024 224 against 237, 16 x 1024 432 against 414)
  static constexpr int NW = DV / 16;
  static constexpr int NT = 64 * NW;
  // waves per SIMD: what two workgroups per CU need (bf16; the LDS of fp32 tiles holds one)
  static constexpr int OCC = BF ? NW / 2 : NW / 4;
};

template <typename E, int DK, int DV, int MODE>
__global__ __launch_bounds__((SsmCfg<E, DK, DV, MODE>::NT), (SsmCfg<E, DK, DV, MODE>::OCC)) void ssm_scan_kernel(SsmScans args) {
  using M = Mma<E>;
  using frag = typename M::frag;
  using Cfg = SsmCfg<E, DK, DV, MODE>;
  constexpr bool BF = Cfg::BF, FWD = MODE == kScanForward, GRAD = MODE == kScanGrad;
  constexpr int NW = Cfg::NW, NT = Cfg::NT;
  constexpr int NKT = DK / 16, NKS = DK / 32;
  // gradients of fp32 tensors are summed in fp64
  constexpr bool WIDE = GRAD && !BF;
  using num = std::conditional_t<WIDE, double, float>;
  using num4 = std::conditional_t<WIDE, f64x4, f32x4>;
  // q k products in LDS: their bf16 terms; going back with equal widths fp32 numbers, split
  // when they are read, since three terms leave a CU of 128 x 128 one workgroup (64 x 64: 201
  // us instead of 221 for 4 x 4096 tokens of 16 heads; 128 x 64 packed, 8192 tokens, whose
  // eight waves would all split the same numbers: 222 instead of 211)
  constexpr bool SPLIT = GRAD && BF && DK == DV;
  using PE = std::conditional_t<WIDE, double, std::conditional_t<SPLIT, float, E>>;
  using pfrag = std::conditional_t<WIDE, f64x8, std::conditional_t<SPLIT, f32x8, frag>>;
  // row strides: 8 (mod 32) dwords keeps bf16 reads free of bank conflicts
  constexpr int KS = BF ? DK + 16 : DK + 4, VS = BF ? DV + 16 : DV + 4, CS = BF && !SPLIT ? kChunk + 16 : kChunk + 4;
  constexpr int NP = !BF || SPLIT ? 1 : GRAD ? 3 : 2;   // terms of the stored q k products
  constexpr int NH = GRAD ? 3 : 2;         // terms of the state in the outputs

  __shared__ __align__(16) E sK[kChunk * KS];            // rows in tile order
  __shared__ __align__(16) E sV[kChunk * VS];            // rows in tile order
  __shared__ __align__(16) E sQ[kChunk * KS];
  __shared__ __align__(16) PE sP[NP][kChunk * CS];
  __shared__ __align__(16) float sG[kGateFloats];
  __shared__ num sDot[2][GRAD ? NW : 1][GRAD ? kChunk : 1];
  // whether this chunk's (and, being cleared, the next one's) v has a value that is not finite.
  // The products with v are over whole tiles of keys, where a later key's weight of zero
  // would make a NaN of it: such values are left out of them and added key by key, so that no
  // output depends on later tokens.  (Forward only: gradients flow both ways.)
  __shared__ int sBad[2];

  const SsmSeqs& sq = args.seqs;
  const SsmScan& a = args.s[blockIdx.y];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int ra = WIDE ? wide_row(r16) : r16;   // the lane's row of a first operand
  SsmUnit u;
  u.init(sq, blockIdx.x);
  const int rev = FWD ? 0 : a.rev;
  const bool kdel = FWD || a.kappa_delta;
  const int seg_in_order = rev ? u.segs - 1 - u.seg : u.seg;
  const bool last = seg_in_order == u.segs - 1;
  const int h = u.h, H = sq.H, len = u.len;
  const int64_t nh = (int64_t)u.n * H + h;
  const int64_t slot = u.sg * H + h;
  const int steps = max(0, u.c1 - u.c0);

  auto row0 = [&](const SsmTensor& x, int width) {   // the head's row of the sequence's first token
    const int hx = __builtin_amdgcn_readfirstlane(h / x.div);
    return reinterpret_cast<const E*>(uniform64(reinterpret_cast<int64_t>(x.p))) + u.tok0 * x.stride + hx * width;
  };
  const E* kb = row0(a.k, DK);
  const E* vb = row0(a.v, DV);
  const E* qb = row0(a.q, DK);

  const int col0 = wave * 16;              // the wave's first state column
  // ---- start state, tile order ----
  f32x4 st[NKT];
  {
    const float* src = seg_in_order > 0 ? a.seg_start : a.h0;
    const int64_t off = (seg_in_order > 0 ? slot : nh) * (DK * DV);
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt) {
      const int row = prow(kt, 4 * q4), col = col0 + ra;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      if (src) {
        if (a.state_t) {
          v = *reinterpret_cast<const f32x4*>(src + off + (int64_t)col * DK + row);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = src[off + (int64_t)(row + i) * DV + col];
        }
      }
      st[kt] = v;
    }
  }

  const float* gb = a.gates + (u.chunk0 * H + h) * kGateFloats;
  float g = 0.f;
  SsmTile<E, DK, NT, true> tk;
  SsmTile<E, DV, NT, true> tv;
  SsmTile<E, DK, NT, false> tq;
  auto chunk_of = [&](int i) { return rev ? u.c1 - 1 - i : u.c0 + i; };
  auto load_tiles = [&](int c, int len, int tid) {
    tk.load(kb, a.k.stride, c, len, rev, tid);
    tq.load(qb, a.q.stride, c, len, rev, tid);
    tv.load(vb, a.v.stride, c, len, rev, tid);
    g = gb[(int64_t)c * H * kGateFloats + (tid & (kGateFloats - 1))];
  };
  if (steps > 0) load_tiles(chunk_of(0), len, tid);
  if (FWD && tid == 0) sBad[0] = 0;

  // adds the waves' shares of a chunk's dots and stores them
  auto flush_dots = [&](int c) {
    if (GRAD && tid < kChunk) {
      const int t = rev ? kChunk - 1 - tid : tid;
      const int64_t at = ((u.chunk0 + c) * H + h) * kChunk + t;
      num d0 = 0, d1 = 0;
#pragma unroll
      for (int w = 0; w < (GRAD ? NW : 1); ++w) {
        d0 += sDot[0][w][tid];
        d1 += sDot[1][w][tid];
      }
      reinterpret_cast<num*>(a.dot_out)[at] = d0;
      if (a.dot_skip) reinterpret_cast<num*>(a.dot_skip)[at] = d1;
    }
  };

  const float dskip = a.D ? load_scalar(a.D, h, args.param_bf16) : 0.f;
  // without alpha the skip is part of the step's own weight
  const float pskip = GRAD && a.alpha_delta ? 0.f : dskip;
  // the lane's addresses: rows of k, q and p, columns of k and v, gates of its step and of
  // its keys (tile order: columns prow(kt, .) are 32 (kt / 2) + 4 (kt % 2) + 8 (r16 / 4) + ..)
  const E* lK = sK + ra * KS + 8 * q4;
  const E* lQ = sQ + r16 * KS + 8 * q4;
  const PE* lP = sP[0] + r16 * CS + 8 * q4;
  const E* lKt = tr_base(sK, KS, 0, 8, r16, q4);
  const E* lVt = tr_base(sV, VS, col0, 4, ra, q4);
  const float* lGs = sG + r16;
  const float* lGk = sG + 8 * q4;
  for (int it = 0; it < steps; ++it) {
    const int c = chunk_of(it);
    // the lane's coordinates, opaque to the optimiser: LDS and output addresses are formed
    // again in every step, kept over the loop they spill
    int ln = lane, td = tid;
    asm volatile("" : "+v"(ln), "+v"(td));
    const int r16 = ln & 15, q4 = ln >> 4;
    __syncthreads();                       // the previous chunk's tiles are done with
    tk.store(sK, KS, td);
    tq.store(sQ, KS, td);
    tv.store(sV, VS, td);
    if constexpr (FWD) {
      if (td == 0) sBad[(it + 1) & 1] = 0;
      if (tv.not_finite()) sBad[it & 1] = 1;
    }
    if (NT == kGateFloats || wave < kGateFloats / 64) sG[td & (kGateFloats - 1)] = g;
    if constexpr (GRAD) {
      if (a.aux.p && it > 0) flush_dots(chunk_of(it - 1));
    }
    __syncthreads();
    num4 acc[4];                           // out^T: columns (rows of the tile) x steps
    {
      // ---- the tiles of (k q^T) with a key at or below a step, decayed, to LDS as [step][key] ----
      // key tiles are in tile order: 0 and 1 hold keys 0..31, so the 12 (key, step) tile
      // pairs are (0|1, 0|1) and (0..3, 2|3), dealt round robin
#pragma unroll
      for (int i = 0; i < (12 + NW - 1) / NW; ++i) {
        const int pi = wave + NW * i;
        if (pi < 12) {
          const int tt = pi < 4 ? pi >> 1 : 2 + ((pi - 4) >> 2);
          const int jt = pi < 4 ? pi & 1 : (pi - 4) & 3;
          frag kf[NKS], qf[NKS];
#pragma unroll
          for (int s = 0; s < NKS; ++s) {
            kf[s] = frag_at(lK, 16 * jt * KS + 32 * s);
            qf[s] = frag_at(lQ, 16 * tt * KS + 32 * s);
          }
          num4 pa = {0, 0, 0, 0}, pb = pa;   // (two chains: each waits for its last product)
#pragma unroll
          for (int s = 0; s < NKS; s += 2) {
            pa = product<M>(kf[s], qf[s], pa);
            pb = product<M>(kf[s + 1], qf[s + 1], pb);
          }
          num4 p;
          const int jb = 32 * (jt >> 1) + 4 * (jt & 1);   // keys jb + 8 q4 .. +3
          const int t = 16 * tt + r16, j0 = jb + 8 * q4;
          const float uh = lGs[kGateU + 16 * tt], ul = lGs[kGateUlo + 16 * tt];
          const f32x4 kh = *reinterpret_cast<const f32x4*>(lGk + kGateU + jb);
          const f32x4 kl = *reinterpret_cast<const f32x4*>(lGk + kGateUlo + jb);
          f32x4 kp = *reinterpret_cast<const f32x4*>(lGk + kGateDelta + jb);
          PE* pd = const_cast<PE*>(lP) + 16 * tt * CS + jb;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!kdel) kp[e] = 1.f;
            num x;
            if constexpr (WIDE)
              x = (pa[e] + pb[e]) * (double)kp[e] * exp2(((double)uh - (double)kh[e]) + ((double)ul - (double)kl[e]));
            else
              x = (pa[e] + pb[e]) * kp[e] * __builtin_amdgcn_exp2f((uh - kh[e]) + (ul - kl[e]));
            p[e] = j0 + e < t ? x : j0 + e == t ? x + pskip : 0;
          }
          if constexpr (BF && !SPLIT) {
#pragma unroll
            for (int n = 0; n < NP; ++n) {
              float p0 = p[0], p1 = p[1], p2 = p[2], p3 = p[3];
              u32x2 d;
              d[0] = split2(p0, p1);
              d[1] = split2(p2, p3);
              *reinterpret_cast<u32x2*>(pd + n * kChunk * CS) = d;
              p = f32x4{p0, p1, p2, p3};
            }
          } else {
            *reinterpret_cast<num4*>(pd) = p;
          }
        }
      }

      // ---- out^T = h^T q^T, decayed (the next operands are read while these are used) ----
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) acc[tt] = num4{0, 0, 0, 0};
      frag qf[2][4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) qf[0][tt] = frag_at(lQ, 16 * tt * KS);
#pragma unroll
      for (int s = 0; s < NKS; ++s) {
        if (s + 1 < NKS)
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) qf[(s + 1) & 1][tt] = frag_at(lQ, 16 * tt * KS + 32 * (s + 1));
        Terms<E, NH> hs;
        hs.set(join8(st[2 * s], st[2 * s + 1]));
#pragma unroll
        for (int n = 0; n < Terms<E, NH>::n; ++n)
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) acc[tt] = product<M>(hs.t[n], qf[s & 1][tt], acc[tt]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        num e;
        if constexpr (WIDE) e = exp2((double)lGs[kGateU + 16 * tt] + (double)lGs[kGateUlo + 16 * tt]);
        else e = __builtin_amdgcn_exp2f(lGs[kGateU + 16 * tt]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[tt][i] *= e;
      }
      __syncthreads();                     // sP
    }
    const int64_t tok0 = u.tok0 + c * kChunk;
    const int lim = min(kChunk, len - c * kChunk);
    // what the outputs are dotted with: ahead of the next tiles (loads come back in order)
    // where there are registers to hold it (64 columns: 56 -> 51 us; 128: spills)
    constexpr bool EARLY = GRAD && DV == 64;
    auto read_aux = [&](int tt) {
      const int j = 16 * tt + r16, t = rev ? kChunk - 1 - j : j;
      return load4(reinterpret_cast<const E*>(a.aux.p) + (tok0 + (t < lim ? t : 0)) * a.aux.stride +
                   (h / a.aux.div) * DV + col0 + 4 * q4);
    };
    f32x4 aux[EARLY ? 4 : 1];
    if constexpr (EARLY) {
      if (a.aux.p) {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) aux[tt] = read_aux(tt);
      }
    }
    // (behind the last chunk: buffers of no rows, which read nothing)
    load_tiles(chunk_of(min(it + 1, steps - 1)), it + 1 < steps ? len : 0, td);

    // ---- v^T operands; out^T += v^T p^T ----
    frag vf[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)            // tokens 32 s + 8 q4 + (0..3, 4..7): tile-order rows 32 s + 4 q4 and 16 further
      vf[s] = tr_frag_at(lVt, 32 * s * VS, VS);
    const bool bad = FWD && __builtin_amdgcn_readfirstlane(sBad[it & 1]) != 0;
    if (bad) {
#pragma unroll
      for (int s = 0; s < 2; ++s) vf[s] = finite_only(vf[s]);
    }
    if constexpr (SPLIT) {
#pragma unroll
      for (int k = 0; k < 6; ++k) {
        const int tt = k < 4 ? k : k - 2, half = k < 4 ? 0 : 1;
        Terms<E, 3> pt;
        pt.set(*reinterpret_cast<const pfrag*>(lP + 16 * tt * CS + 32 * half));
#pragma unroll
        for (int n = 0; n < 3; ++n) acc[tt] = product<M>(vf[half], pt.t[n], acc[tt]);
      }
    } else {
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        pfrag pf[6];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) pf[tt] = *reinterpret_cast<const pfrag*>(lP + (n * kChunk + 16 * tt) * CS);
#pragma unroll
        for (int tt = 2; tt < 4; ++tt) pf[2 + tt] = *reinterpret_cast<const pfrag*>(lP + (n * kChunk + 16 * tt) * CS + 32);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) acc[tt] = product<M>(vf[0], pf[tt], acc[tt]);
#pragma unroll
        for (int tt = 2; tt < 4; ++tt) acc[tt] = product<M>(vf[1], pf[2 + tt], acc[tt]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }

    {
      // ---- outputs: lane = step 16 tt + r16, columns 4 q4 .. +3 of each tile ----
      const bool wide = !BF || (GRAD && a.out_f32);
      const uint32_t ob = wide ? 4u : 2u;
      const __amdgpu_buffer_rsrc_t os =
          chunk_buffer(reinterpret_cast<char*>(a.out) + (tok0 * H + h) * DV * ob, lim, (uint32_t)(H * DV) * ob);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int j = 16 * tt + r16;
        const int t = rev ? kChunk - 1 - j : j;
        const bool ok = t < lim;
        num d0 = 0, d1 = 0;
        const int oc = col0 + 4 * q4;
        num4 o = acc[tt];
        if (GRAD && (a.aux.p || a.alpha_delta)) {
          const f32x4 v = load4(&sV[tord(j) * VS + oc]);
          if (a.aux.p) {
            const f32x4 x = EARLY ? aux[EARLY ? tt : 0] : read_aux(tt);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              d0 += x[i] * o[i];
              d1 += x[i] * v[i];
            }
          }
          if (a.alpha_delta) {
            const float al = sG[kGateDelta + j];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = o[i] * al + dskip * v[i];
          }
        }
        const uint32_t at = (uint32_t)t * (uint32_t)(H * DV) + oc;
        if (wide) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, __builtin_convertvector(o, f32x4)), os, at * 4u, 0, 0);
        } else {
          const bf16x4 d = __builtin_convertvector(o, bf16x4);
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, d), os, at * 2u, 0, 0);
        }
        if (GRAD && a.aux.p) {
          d0 += __shfl_xor(d0, 16, 64);
          d0 += __shfl_xor(d0, 32, 64);
          d1 += __shfl_xor(d1, 16, 64);
          d1 += __shfl_xor(d1, 32, 64);
          if (q4 == 0) {
            sDot[0][wave][j] = ok ? d0 : 0;
            sDot[1][wave][j] = ok ? d1 : 0;
          }
        }
      }
    }

    if (bad) {
      // outputs that meet a value that is not finite: what they get from those is all of them
      // (a lane's stores to one address stay in order)
#pragma unroll 1
      for (int tt = 0; tt < 4; ++tt) {
        const int j = 16 * tt + r16, oc = col0 + 4 * q4;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int k = 0; k <= j; ++k) {
          const f32x4 v = load4(&sV[tord(k) * VS + oc]);
          float pk = 0.f;
          for (int n = 0; n < NP; ++n) pk += (float)sP[n][j * CS + k];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(__builtin_fabsf(v[i]) < __builtin_inff())) o[i] += pk * v[i];
        }
        E* out = reinterpret_cast<E*>(a.out) + ((tok0 + j) * H + h) * DV + oc;
        for (int i = 0; i < 4; ++i)
          if (j < lim && !(__builtin_fabsf(o[i]) < __builtin_inff())) out[i] = from_f32<E>(o[i]);
      }
      // and the state takes all of v
#pragma unroll
      for (int s = 0; s < 2; ++s) vf[s] = tr_frag_at(lVt, 32 * s * VS, VS);
    }

    // ---- the state's update: groups of row tiles, the next group read while this is used ----
    const float dec = __builtin_amdgcn_exp2f(sG[kGateU + kChunk - 1]);
    constexpr int GK = 2, NG = NKT / GK;
    auto read_k = [&](int g, frag (&kf)[GK]) {   // group g of 2 NG: contraction step g / NG
      const int s = g / NG;
#pragma unroll
      for (int i = 0; i < GK; ++i) {
        const int kt = (g % NG) * GK + i;
        kf[i] = tr_frag_at(lKt, 32 * s * KS + 32 * (kt >> 1) + 4 * (kt & 1), KS);
      }
    };
    frag kf[2][GK];
    read_k(0, kf[0]);
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) st[kt][i] *= dec;
    Terms<E, 3> wv;
#pragma unroll
    for (int g = 0; g < 2 * NG; ++g) {
      if (g % NG == 0) {
        const int s = g / NG;
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(lGk + kGateW + 32 * s);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(lGk + kGateW + 32 * s + 4);
        const f32x8 w = join8(w0, w1);
        f32x8 x = widen(vf[s]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= w[e];
        wv.set(x);
      }
      if (g + 1 < 2 * NG) read_k(g + 1, kf[(g + 1) & 1]);
#pragma unroll
      for (int n = 0; n < Terms<E, 3>::n; ++n)
#pragma unroll
        for (int i = 0; i < GK; ++i)
          st[(g % NG) * GK + i] = M::run(kf[g & 1][i], wv.t[n], st[(g % NG) * GK + i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (GRAD) {
    if (a.aux.p && steps > 0) {
      __syncthreads();
      flush_dots(chunk_of(steps - 1));
    }
  }

  // ---- the end state ----
  float* dst = last ? a.hT : nullptr;
  if (dst) {
    float f = 1.f;
    if (GRAD && a.decay0 && len > 0) f = __builtin_amdgcn_exp2f(a.decay0[(u.chunk0 * H + h) * kGateFloats + kGateU]);
    const int64_t off = nh * (DK * DV);
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt) {
      const int row = prow(kt, 4 * q4), col = col0 + ra;
      f32x4 v = st[kt];
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
}

// The end state of each segment but a sequence's last (in scan order) from a zero start, and
// its decay.  S = sum_j k_j (exp(U_end - U_j) kappa_j v_j)^T over the whole segment is one
// long product, so the chunks are taken last to first with the decay to the segment's end
// in the weights: the state in registers is only ever added to.  All chunks count, however
// far they have decayed: a state of old inputs only, and a NaN in them, have to come out.
// 4 x 4096 bf16 tokens of 16 heads, n = p = 128, segments of 8 chunks: 33 us, for 104 MB.
// Three terms of v's weights make 25 GFLOP: MFMA 10 us, and as long again for the split
// into terms and the LDS reads.  131072 tokens of 4 heads: 78 us.
// Tiles are double-buffered in LDS, so a chunk is one barrier.
template <typename E, int DK, int DV>
__global__ __launch_bounds__(64 * (DV / 16), (SsmCfg<E, DK, DV, kScanState>::OCC)) void ssm_state_kernel(SsmScans args) {
  using M = Mma<E>;
  using frag = typename M::frag;
  using Cfg = SsmCfg<E, DK, DV, kScanState>;
  constexpr bool BF = Cfg::BF;
  constexpr int NT = Cfg::NT, NKT = DK / 16;
  constexpr int KS = BF ? DK + 16 : DK + 4, VS = BF ? DV + 16 : DV + 4;
  constexpr int NB = BF ? 2 : 1;           // fp32 tiles fit once
  __shared__ __align__(16) E sKb[NB][kChunk * KS];       // rows in tile order
  __shared__ __align__(16) E sVb[NB][kChunk * VS];
  __shared__ __align__(16) float sWt[2][kChunk];

  const SsmSeqs& sq = args.seqs;
  const SsmScan& a = args.s[blockIdx.y];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  SsmUnit u;
  u.init(sq, blockIdx.x);
  const int rev = a.rev;
  if ((rev ? u.segs - 1 - u.seg : u.seg) == u.segs - 1) return;
  const int h = u.h, H = sq.H, len = u.len;
  const int64_t slot = u.sg * H + h;
  const int steps = max(0, u.c1 - u.c0);
  auto row0 = [&](const SsmTensor& x, int width) {
    const int hx = __builtin_amdgcn_readfirstlane(h / x.div);
    return reinterpret_cast<const E*>(uniform64(reinterpret_cast<int64_t>(x.p))) + u.tok0 * x.stride + hx * width;
  };
  const E* kb = row0(a.k, DK);
  const E* vb = row0(a.v, DV);
  // step i of the walk is the segment's (steps - 1 - i)-th chunk in scan order
  auto chunk_of = [&](int i) { return rev ? u.c0 + i : u.c1 - 1 - i; };

  // a chunk's gates: one step's weight a thread, and the chunk's decay
  const float* gb = a.gates + (u.chunk0 * H + h) * kGateFloats;
  float wt = 0.f, eh = 0.f, el = 0.f;
  double log2_end = 0.0;                   // decay from the chunk's end to the segment's

  f32x4 st[NKT];
#pragma unroll
  for (int kt = 0; kt < NKT; ++kt) st[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
  SsmTile<E, DK, NT, true> tk;
  SsmTile<E, DV, NT, true> tv;
  auto load = [&](int i, int td) {
    tk.load(kb, a.k.stride, chunk_of(i), len, rev, td);
    tv.load(vb, a.v.stride, chunk_of(i), len, rev, td);
    const float* gc = gb + (int64_t)chunk_of(i) * H * kGateFloats;
    wt = gc[kGateW + (td & 63)];
    eh = gc[kGateU + kChunk - 1];
    el = gc[kGateUlo + kChunk - 1];
  };
  auto store = [&](int b, int td) {
    tk.store(sKb[BF ? b : 0], KS, td);
    tv.store(sVb[BF ? b : 0], VS, td);
    if (wave == 0) sWt[b][td] = wt * __builtin_amdgcn_exp2f((float)log2_end);
    log2_end += (double)eh + (double)el;
  };
  if (steps > 0) {
    load(0, tid);
    store(0, tid);
    if (steps > 1) load(1, tid);
  }
  __syncthreads();
  const E* lKt = tr_base(sKb[0], KS, 0, 8, r16, q4);
  const E* lVt = tr_base(sVb[0], VS, wave * 16, 4, r16, q4);
  const float* lW = sWt[0] + 8 * q4;
  for (int it = 0; it < steps; ++it) {
    const int b = it & 1, tb = BF ? b : 0;
    int td = tid;                          // (see ssm_scan_kernel)
    asm volatile("" : "+v"(td));
    const bool more = it + 1 < steps;
    if (BF && more) {
      store(b ^ 1, td);
      if (it + 2 < steps) load(it + 2, td);
    }
    const int kof = tb * kChunk * KS, vof = tb * kChunk * VS;
    constexpr int GK = 2, NG = NKT / GK;
    auto read_k = [&](int g, frag (&kf)[GK]) {
      const int s = g / NG;
#pragma unroll
      for (int i = 0; i < GK; ++i) {
        const int kt = (g % NG) * GK + i;
        kf[i] = tr_frag_at(lKt + kof, 32 * s * KS + 32 * (kt >> 1) + 4 * (kt & 1), KS);
      }
    };
    frag kf[2][GK], vf[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      vf[s] = tr_frag_at(lVt + vof, 32 * s * VS, VS);
    read_k(0, kf[0]);
    Terms<E, 3> wv;
#pragma unroll
    for (int g = 0; g < 2 * NG; ++g) {
      if (g % NG == 0) {
        const int s = g / NG;
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(lW + b * kChunk + 32 * s);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(lW + b * kChunk + 32 * s + 4);
        const f32x8 w = join8(w0, w1);
        f32x8 x = widen(vf[s]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= w[e];
        wv.set(x);
      }
      if (g + 1 < 2 * NG) read_k(g + 1, kf[(g + 1) & 1]);
#pragma unroll
      for (int n = 0; n < Terms<E, 3>::n; ++n)
#pragma unroll
        for (int i = 0; i < GK; ++i) st[(g % NG) * GK + i] = M::run(kf[g & 1][i], wv.t[n], st[(g % NG) * GK + i]);
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    if (!more) break;
    if (!BF) {                             // one buffer: the next chunk's tiles go where these were
      store(b ^ 1, td);
      if (it + 2 < steps) load(it + 2, td);
      __syncthreads();
    }
  }

  const int64_t off = slot * (DK * DV);
  const int col = wave * 16 + r16;
#pragma unroll
  for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
    for (int i = 0; i < 4; ++i) a.seg_state[off + (int64_t)(prow(kt, 4 * q4) + i) * DV + col] = st[kt][i];
  if (tid == 0) a.seg_decay[slot] = __builtin_amdgcn_exp2f((float)log2_end);
}

template <typename E, int DK, int DV>
hipError_t run_ssm_scan(const SsmScans& a, int count, int mode, hipStream_t s) {
  if (a.seqs.units == 0) return hipSuccess;
  if (a.seqs.units > kMaxDispatchItems / 512) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)a.seqs.units, (unsigned)count);
  if (mode == kScanState) ssm_state_kernel<E, DK, DV><<<grid, SsmCfg<E, DK, DV, kScanState>::NT, 0, s>>>(a);
  else if (mode == kScanForward)
    ssm_scan_kernel<E, DK, DV, kScanForward><<<grid, SsmCfg<E, DK, DV, kScanForward>::NT, 0, s>>>(a);
  else
    ssm_scan_kernel<E, DK, DV, kScanGrad><<<grid, SsmCfg<E, DK, DV, kScanGrad>::NT, 0, s>>>(a);
  return hipGetLastError();
}

template <typename E>
hipError_t run_ssm_scan_dims(const SsmScans& a, int count, int dk, int dv, int mode, hipStream_t s) {
  if (dk == 64 && dv == 64) return run_ssm_scan<E, 64, 64>(a, count, mode, s);
  if (dk == 64 && dv == 128) return run_ssm_scan<E, 64, 128>(a, count, mode, s);
  if (dk == 128 && dv == 64) return run_ssm_scan<E, 128, 64>(a, count, mode, s);
  if (dk == 128 && dv == 128) return run_ssm_scan<E, 128, 128>(a, count, mode, s);
  return hipErrorInvalidConfiguration;
}

}  // namespace gdn
