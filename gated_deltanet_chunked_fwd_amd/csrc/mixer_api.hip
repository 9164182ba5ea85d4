// C ABI of the operators around the delta rule: argument checks, workspace layout, the
// split of the selective scan and the launch sequences.  Contracts are in include/gdn.h.
#include <algorithm>
#include <climits>
#include <cmath>

#include "gdn.h"
#include "mixer_launch.h"

namespace {

using gdn::kChunk;

bool ok_type(int t) { return t == GDN_BF16 || t == GDN_F32; }
int type_bytes(int t) { return t == GDN_BF16 ? 2 : 4; }
bool mis(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
bool bad(const void* p) { return !p || mis(p); }
// a required pointer to `count` elements or rows (an empty tensor has no address)
bool bad(const void* p, int64_t count) { return count > 0 ? bad(p) : mis(p); }
// what the kernels take one element at a time needs no more than its type's alignment
bool mis_el(const void* p, int type) { return (reinterpret_cast<uintptr_t>(p) & (type_bytes(type) - 1)) != 0; }
bool bad_el(const void* p, int type, int64_t count = 1) { return (count > 0 && !p) || mis_el(p, type); }
bool mis_ints(const int32_t* p) { return (reinterpret_cast<uintptr_t>(p) & 3) != 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The sequence layout every shape struct shares.
int check_seqs(int64_t B, int64_t T, int64_t N, const int32_t* cu) {
  if (B < 1 || T < 0 || T > INT_MAX / 2 || B > INT_MAX / 2 || (T > 0 && B > INT64_C(0x7fffffffffff) / T)) return GDN_ERR_ARG;
  if (!cu) return N == B ? GDN_OK : GDN_ERR_ARG;
  if (B != 1 || N < 1 || N > INT_MAX / 2 || cu[0] != 0 || cu[N] != T) return GDN_ERR_ARG;
  for (int64_t n = 0; n < N; ++n)
    if (cu[n + 1] < cu[n]) return GDN_ERR_ARG;
  return GDN_OK;
}
// Device cu_seqlens come with their host copy, and the other way round.
bool cu_mismatch(const int32_t* dev, const int32_t* host) { return (dev != nullptr) != (host != nullptr) || mis_ints(dev); }

// ---- convolution ---------------------------------------------------------------------
int check_conv(const gdn_conv_shape* s) {
  if (!s || s->D < 1 || s->D > INT_MAX / 8) return GDN_ERR_ARG;
  if (const int rc = check_seqs(s->B, s->T, s->N, s->cu_seqlens_host)) return rc;
  if (s->x_stride != 0 && s->x_stride < s->D) return GDN_ERR_ARG;
  if (s->silu != 0 && s->silu != 1) return GDN_ERR_ARG;
  if (s->W < 2 || s->W > 4 || !ok_type(s->dtype) || !ok_type(s->param_dtype)) return GDN_ERR_UNSUPPORTED;
  // the forward's work-items: at most one per channel and 16 tokens, and the states' rows
  if (s->B * s->T / 16 + s->N * (s->W - 1) + 2 > (gdn::kMaxDispatchItems - 256) / s->D) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
gdn::ConvArgs conv_args(const void* x, const void* w, const void* bias, const void* init, const int32_t* cu,
                        const gdn_conv_shape* s) {
  gdn::ConvArgs a{};
  a.x = x;
  a.x_stride = s->x_stride ? s->x_stride : s->D;
  a.w = w;
  a.bias = bias;
  a.init = init;
  a.cu = cu;
  a.B = s->B;
  a.T = s->T;
  a.D = s->D;
  a.N = (int)s->N;
  a.W = (int)s->W;
  a.bf16 = s->dtype == GDN_BF16;
  a.param_bf16 = s->param_dtype == GDN_BF16;
  a.silu = s->silu;
  return a;
}

// ---- selective scan ------------------------------------------------------------------
int check_ssm(const gdn_ssm_shape* s) {
  if (!s || s->H < 1 || s->H > 65535 || s->G < 1 || s->H % s->G != 0 || s->reserved != 0) return GDN_ERR_ARG;
  if (const int rc = check_seqs(s->B, s->T, s->N, s->cu_seqlens_host)) return rc;
  if (s->N * s->H > INT_MAX / 2 || s->segment_chunks < 0) return GDN_ERR_ARG;
  if (s->dt_softplus != 0 && s->dt_softplus != 1) return GDN_ERR_ARG;
  if ((s->n != 64 && s->n != 128) || (s->p != 64 && s->p != 128)) return GDN_ERR_UNSUPPORTED;
  if (!ok_type(s->dtype) || !ok_type(s->dt_dtype) || !ok_type(s->param_dtype)) return GDN_ERR_UNSUPPORTED;
  const int64_t v = 16 / type_bytes(s->dtype);
  if (s->x_stride < 0 || s->b_stride < 0 || s->c_stride < 0) return GDN_ERR_ARG;
  if (s->x_stride % v || s->b_stride % v || s->c_stride % v) return GDN_ERR_ARG;
  // (the kernels' 32-bit byte offsets inside a chunk of 64 tokens)
  const int64_t widest = std::max(std::max(s->H * s->p, s->H * s->n), std::max(s->x_stride, std::max(s->b_stride, s->c_stride)));
  if (widest >= INT64_C(1) << 22) return GDN_ERR_UNSUPPORTED;
  if ((s->x_stride && s->x_stride < s->H * s->p) || (s->b_stride && s->b_stride < s->G * s->n) ||
      (s->c_stride && s->c_stride < s->G * s->n))
    return GDN_ERR_ARG;
  return GDN_OK;
}

struct SsmPlan {
  int64_t total_chunks = 0, max_chunks = 0;
  int seg_chunks = INT_MAX / 2;
  int64_t segs = 0, max_segs = 1;          // over all sequences; of the longest one
  // workspace offsets
  size_t gates[2] = {0, 0}, state[2] = {0, 0}, decay[2] = {0, 0}, hT = 0, cdc = 0, xdu = 0, dyx = 0, part = 0,
         dBp = 0, dCp = 0, offsets[2] = {0, 0}, bytes = 0;
};

int64_t ssm_chunks(const gdn_ssm_shape* s, int64_t n) {
  const int64_t len = s->cu_seqlens_host ? s->cu_seqlens_host[n + 1] - s->cu_seqlens_host[n] : s->T;
  return (len + kChunk - 1) / kChunk;
}

// Segments.  Units (a segment of a head) for two workgroups per CU (bf16; fp32 tiles leave
// room for one) and of equal length: L = ceil(chunks * H / units), at least kSsmMinChunks.  A
// segment costs a pass over its keys and values and its state's way through memory, so that
// a call with segments takes about 22 + 12 L us and one without 10 + 4 per chunk of its
// longest sequence: it is split if that one has kSsmSplitWorth[] L and kSsmSplitExtra chunks.
// Only the chunks count, not the sequences: short ones beside a long one do not keep it
// whole.  A split longest sequence has segments of equal length.  Measured (us, chunks per
// segment: time, - = unsplit; * = the rule), 128 x 128, 16 heads:
//   1 x 512 tokens                  *2: 31,  3: 35,  -: 38
//   1 x 256                          2: 30, *-: 23
//   4 x 4096                         4: 145, *8: 119, 16: 124, -: 253
//   9 x 4096                        18: 301, *22: 244, -: 275
//   16 x 4096                       16: 393, 32: 369, *-: 302
//   31 x 4096                       31: 795, 62: 1161, *-: 528
//   131072 tokens, 4 heads           8: 275, *16: 240, 32: 260
//   131072 tokens and 31 single ones 33: 817, *67: 806, -: 8056
//   fp32, 8 x 4096                  16: 592, *32: 601, -: 813
//   fp32, 12 x 4096                 24: 1060, 48: 1652, *-: 824
// Backward: no segments where the longest sequence has up to kSsmBwdSplitWorth L (three scans
// run side by side) and kSsmMaxBwdChunks chunks, the gates' gradients being sums of
// nearly cancelling flows over a segment, whose rounding grows with its length (1300 tokens, 2
// heads, bf16: dA off by 5e-3 of itself in one segment of 21 chunks; so a caller's longer
// segments are cut too), and one chunk for fp32 tensors, whose gradients are held to fp32 (2
// x 777 tokens, 4 heads: 53 us and an error of 3e-7 in dA; 2: 52, 7e-7; 4: 78, 2e-6).
//   8192 packed tokens, 128 x 64     4: 221, *5: 213, 6: 225, 8: 217, 16: 297
//   4 x 4096                         4: 527, *8: 457, 16: 482
//   16 x 1024                        4: 505, 8: 451, *-: 424
//   24 x 1024                        8: 668, 12: 822, *-: 570
//   8 x 256                          2: 102, *-: 72
//   1 x 384                         *2: 60, 3: 65, -: 68
constexpr int64_t kSsmMinChunks = 2;
constexpr int64_t kSsmSplitWorth[2] = {2, 3}, kSsmSplitExtra[2] = {0, 2};   // fp32, bf16
constexpr int64_t kSsmBwdSplitWorth = 5;
constexpr int64_t kSsmMaxBwdChunks = 16;

SsmPlan plan_ssm(const gdn_ssm_shape* s, bool bwd) {
  SsmPlan P;
  for (int64_t n = 0; n < s->N; ++n) {
    const int64_t c = ssm_chunks(s, n);
    P.total_chunks += c;
    P.max_chunks = std::max(P.max_chunks, c);
  }
  const bool is_bf16 = s->dtype == GDN_BF16;
  int64_t L = INT_MAX / 2;
  if (s->segment_chunks > 0) {
    L = bwd ? std::min<int64_t>(s->segment_chunks, kSsmMaxBwdChunks) : s->segment_chunks;
  } else {
    const int64_t units = (int64_t)gdn::device_cus() * (is_bf16 ? 2 : 1), work = P.total_chunks * s->H;
    const int64_t even = std::max(kSsmMinChunks, (work + units - 1) / units);
    if (bwd) {
      if (P.max_chunks * units > kSsmBwdSplitWorth * work) L = even;
      L = std::min(L, is_bf16 ? kSsmMaxBwdChunks : (int64_t)1);
    } else if (P.max_chunks >= kSsmSplitWorth[is_bf16] * even + kSsmSplitExtra[is_bf16]) {
      const int64_t parts = P.max_chunks / even;
      L = (P.max_chunks + parts - 1) / parts;
    }
  }
  P.seg_chunks = (int)std::min<int64_t>(L, INT_MAX / 2);
  for (int64_t n = 0; n < s->N; ++n) {
    const int64_t g = std::max<int64_t>(1, (ssm_chunks(s, n) + P.seg_chunks - 1) / P.seg_chunks);
    P.segs += g;
    P.max_segs = std::max(P.max_segs, g);
  }
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += up256(bytes);
    return o;
  };
  if (s->cu_seqlens_host && s->N > gdn::kSsmCounted)
    for (size_t& o : P.offsets) o = take((s->N + 1) * 4);
  const size_t state = (size_t)(s->n * s->p) * 4;
  const bool split = P.max_segs > 1;
  for (int i = 0; i < (bwd ? 2 : 1); ++i) P.gates[i] = take((size_t)P.total_chunks * s->H * 1024);
  if (split)
    for (int i = 0; i < (bwd ? 2 : 1); ++i) {
      P.state[i] = take(P.segs * s->H * state);
      P.decay[i] = take(P.segs * s->H * 4);
    }
  if (bwd) {
    P.hT = take(s->N * s->H * state);
    const size_t dots = (size_t)P.total_chunks * s->H * kChunk * (is_bf16 ? 4 : 8);
    P.cdc = take(dots);
    P.xdu = take(dots);
    P.dyx = take(dots);
    P.part = take(P.segs * s->H * 3 * 8);
    if (s->G < s->H) {
      const size_t per_head = (size_t)(s->B * s->T) * s->H * s->n * 4;
      P.dBp = take(per_head);
      P.dCp = take(per_head);
    }
  }
  P.bytes = at;
  return P;
}
// Grids of one workgroup per (segment, head), in work-items.
int check_plan(const SsmPlan& P, const gdn_ssm_shape* s) {
  return P.segs * s->H > gdn::kMaxDispatchItems / 512 || P.total_chunks * s->H > gdn::kMaxDispatchItems / 64 - 4 || s->N * s->H * (s->n * s->p / 256) > gdn::kMaxDispatchItems / 256
             ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

// (and enqueues the tables of many packed sequences)
hipError_t ssm_seqs(const gdn_ssm_shape* s, const SsmPlan& P, const int32_t* cu, char* ws, hipStream_t stream, gdn::SsmSeqs* out) {
  gdn::SsmSeqs q{};
  q.cu = cu;
  q.T = s->T;
  q.N = (int)s->N;
  q.H = (int)s->H;
  q.seg_chunks = P.seg_chunks;
  q.segs = cu ? 1 : (int)P.max_segs;
  q.units = P.segs * s->H;
  q.chunks = P.total_chunks;
  hipError_t rc = hipSuccess;
  if (cu && s->N > gdn::kSsmCounted) {
    int32_t* chunk_off = reinterpret_cast<int32_t*>(ws + P.offsets[0]);
    int32_t* seg_off = reinterpret_cast<int32_t*>(ws + P.offsets[1]);
    rc = gdn::launch_ssm_offsets(q, chunk_off, seg_off, stream);
    q.chunk_off = chunk_off;
    q.seg_off = seg_off;
  }
  *out = q;
  return rc;
}
gdn::SsmGates ssm_gates(const gdn_ssm_shape* s, const void* dt, const void* A, const void* bias) {
  gdn::SsmGates g{};
  g.dt = dt;
  g.A = A;
  g.bias = bias;
  g.dt_bf16 = s->dt_dtype == GDN_BF16;
  g.param_bf16 = s->param_dtype == GDN_BF16;
  g.softplus = s->dt_softplus;
  return g;
}

// ---- norm ----------------------------------------------------------------------------
int check_norm(const gdn_norm_shape* s) {
  if (!s || s->rows < 0 || s->H < 1 || s->D < 1 || s->reserved != 0 || s->H > INT_MAX / 8) return GDN_ERR_ARG;
  if (!(s->eps > 0.f) || !std::isfinite(s->eps)) return GDN_ERR_ARG;
  if (s->D > gdn::kNormMaxWidth || !ok_type(s->dtype) || !ok_type(s->param_dtype)) return GDN_ERR_UNSUPPORTED;
  if (!gdn::norm_fits(s->rows, (int)s->H, (int)s->D, s->dtype == GDN_BF16)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
gdn::NormArgs norm_args(const gdn_norm_shape* s) {
  gdn::NormArgs a{};
  a.rows = s->rows;
  a.H = (int)s->H;
  a.D = (int)s->D;
  a.bf16 = s->dtype == GDN_BF16;
  a.param_bf16 = s->param_dtype == GDN_BF16;
  a.eps = s->eps;
  return a;
}

int launched(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

}  // namespace

extern "C" {

int gdn_conv_fwd(const void* x, const void* weight, const void* bias, const void* initial_state,
                 const int32_t* cu_seqlens, void* y, void* final_state, const gdn_conv_shape* shape,
                 hipStream_t stream) {
  if (const int rc = check_conv(shape)) return rc;
  const int64_t tokens = shape->B * shape->T;
  if (bad(x, tokens) || bad(weight) || mis(bias) || mis(initial_state) || bad(y, tokens) || mis(final_state))
    return GDN_ERR_ARG;
  if (cu_mismatch(cu_seqlens, shape->cu_seqlens_host)) return GDN_ERR_ARG;
  gdn::ConvArgs a = conv_args(x, weight, bias, initial_state, cu_seqlens, shape);
  a.y = y;
  a.fin = final_state;
  return launched(gdn::launch_conv_fwd(a, stream));
}

int gdn_conv_bwd_workspace_bytes(const gdn_conv_shape* shape, size_t* bytes) {
  if (const int rc = check_conv(shape)) return rc;
  if (!bytes) return GDN_ERR_ARG;
  if (!gdn::conv_bwd_fits(shape->B * shape->T, shape->D, (int)shape->W)) return GDN_ERR_UNSUPPORTED;
  *bytes = up256((size_t)gdn::conv_bwd_rows(shape->B * shape->T) * (shape->W + 1) * shape->D * 4 + 4);
  return GDN_OK;
}

int gdn_conv_bwd(const void* x, const void* weight, const void* bias, const void* initial_state,
                 const int32_t* cu_seqlens, const void* dy, const void* d_final_state, void* dx, void* dweight,
                 void* dbias, void* d_initial_state, const gdn_conv_shape* shape, void* workspace,
                 size_t workspace_bytes, hipStream_t stream) {
  size_t need = 0;
  if (const int rc = gdn_conv_bwd_workspace_bytes(shape, &need)) return rc;
  const int64_t tokens = shape->B * shape->T;
  if (bad(x, tokens) || bad(weight) || mis(bias) || mis(initial_state) || bad(dy, tokens) || mis(d_final_state) ||
      bad(dx, tokens) ||
      bad(dweight) || mis(dbias) || mis(d_initial_state) || (dbias && !bias))
    return GDN_ERR_ARG;
  if (cu_mismatch(cu_seqlens, shape->cu_seqlens_host)) return GDN_ERR_ARG;
  if (bad(workspace) || workspace_bytes < need) return GDN_ERR_WORKSPACE;
  gdn::ConvArgs a = conv_args(x, weight, bias, initial_state, cu_seqlens, shape);
  a.dy = dy;
  a.dfin = d_final_state;
  a.dx = dx;
  a.dw = dweight;
  a.dbias = dbias;
  a.dinit = d_initial_state;
  a.part = static_cast<float*>(workspace);
  return launched(gdn::launch_conv_bwd(a, stream));
}

int gdn_conv_step(const void* x, const void* weight, const void* bias, const void* state, const int32_t* slots,
                  void* y, void* state_out, const gdn_conv_shape* shape, hipStream_t stream) {
  if (!shape || shape->T != 1 || shape->cu_seqlens_host || shape->x_stride != 0 || shape->N < 1) return GDN_ERR_ARG;
  gdn_conv_shape rows = *shape;            // (N counts slots here)
  rows.N = rows.B;
  if (const int rc = check_conv(&rows)) return rc;
  if (bad(x) || bad(weight) || mis(bias) || bad(state) || mis_ints(slots) || bad(y) || bad(state_out)) return GDN_ERR_ARG;
  if (!slots && shape->B > shape->N) return GDN_ERR_ARG;
  if (shape->N > INT_MAX || shape->B * ((shape->D + 255) / 256) > gdn::kMaxDispatchItems / 256) return GDN_ERR_UNSUPPORTED;
  gdn::ConvStepArgs a{};
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.state = state;
  a.slots = slots;
  a.y = y;
  a.state_out = state_out;
  a.R = shape->B;
  a.S = shape->N;
  a.D = shape->D;
  a.W = (int)shape->W;
  a.bf16 = shape->dtype == GDN_BF16;
  a.param_bf16 = shape->param_dtype == GDN_BF16;
  a.silu = shape->silu;
  return launched(gdn::launch_conv_step(a, stream));
}

int gdn_ssm_fwd_workspace_bytes(const gdn_ssm_shape* shape, size_t* bytes) {
  if (const int rc = check_ssm(shape)) return rc;
  if (!bytes) return GDN_ERR_ARG;
  const SsmPlan P = plan_ssm(shape, false);
  if (const int rc = check_plan(P, shape)) return rc;
  *bytes = P.bytes;
  return GDN_OK;
}

int gdn_ssm_fwd(const void* x, const void* dt, const void* A, const void* Bm, const void* Cm, const void* D,
                const void* dt_bias, const float* initial_state, const int32_t* cu_seqlens, void* y,
                float* final_state, const gdn_ssm_shape* shape, void* workspace, size_t workspace_bytes,
                hipStream_t stream) {
  if (const int rc = check_ssm(shape)) return rc;
  const int64_t tokens = shape->B * shape->T;
  const int et = shape->dt_dtype, ep = shape->param_dtype;
  if (bad(x, tokens) || bad_el(dt, et, tokens) || bad_el(A, ep) || bad(Bm, tokens) || bad(Cm, tokens) || mis_el(D, ep) ||
      mis_el(dt_bias, ep) || mis(initial_state) || bad(y, tokens) || mis(final_state))
    return GDN_ERR_ARG;
  if (cu_mismatch(cu_seqlens, shape->cu_seqlens_host)) return GDN_ERR_ARG;
  const SsmPlan P = plan_ssm(shape, false);
  if (const int rc = check_plan(P, shape)) return rc;
  if (P.bytes && (bad(workspace) || workspace_bytes < P.bytes)) return GDN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  const bool split = P.max_segs > 1;
  const int is_bf16 = shape->dtype == GDN_BF16, n = (int)shape->n, p = (int)shape->p, div = (int)(shape->H / shape->G);
  gdn::SsmScans a{};
  if (ssm_seqs(shape, P, cu_seqlens, ws, stream, &a.seqs) != hipSuccess) return GDN_ERR_HIP;
  a.param_bf16 = shape->param_dtype == GDN_BF16;
  float* gates = reinterpret_cast<float*>(ws + P.gates[0]);
  if (gdn::launch_ssm_gates(a.seqs, ssm_gates(shape, dt, A, dt_bias), gates, nullptr, stream) != hipSuccess)
    return GDN_ERR_HIP;
  gdn::SsmScan& s = a.s[0];
  s.gates = gates;
  s.q = {Cm, shape->c_stride ? shape->c_stride : shape->G * n, div};
  s.k = {Bm, shape->b_stride ? shape->b_stride : shape->G * n, div};
  s.v = {x, shape->x_stride ? shape->x_stride : shape->H * p, 1};
  s.kappa_delta = 1;
  s.D = D;
  s.h0 = initial_state;
  s.out = y;
  s.out_f32 = !is_bf16;
  s.hT = final_state;
  if (split) {
    s.seg_state = reinterpret_cast<float*>(ws + P.state[0]);
    s.seg_decay = reinterpret_cast<float*>(ws + P.decay[0]);
    s.seg_start = s.seg_state;
    if (gdn::launch_ssm_scan(a, 1, is_bf16, n, p, gdn::kScanState, stream) != hipSuccess) return GDN_ERR_HIP;
    const gdn::SsmMerge m = {s.seg_state, s.seg_decay, initial_state, 0};
    if (gdn::launch_ssm_merge(a.seqs, &m, 1, n * p, stream) != hipSuccess) return GDN_ERR_HIP;
  }
  return launched(gdn::launch_ssm_scan(a, 1, is_bf16, n, p, gdn::kScanForward, stream));
}

int gdn_ssm_bwd_workspace_bytes(const gdn_ssm_shape* shape, size_t* bytes) {
  if (const int rc = check_ssm(shape)) return rc;
  if (!bytes) return GDN_ERR_ARG;
  const SsmPlan P = plan_ssm(shape, true);
  if (const int rc = check_plan(P, shape)) return rc;
  *bytes = P.bytes;
  return GDN_OK;
}

int gdn_ssm_bwd(const void* x, const void* dt, const void* A, const void* Bm, const void* Cm, const void* D,
                const void* dt_bias, const float* initial_state, const int32_t* cu_seqlens, const void* dy,
                const float* d_final_state, void* dx, void* ddt, void* dA, void* dB, void* dC, void* dD,
                void* d_dt_bias, float* d_initial_state, const gdn_ssm_shape* shape, void* workspace,
                size_t workspace_bytes, hipStream_t stream) {
  if (const int rc = check_ssm(shape)) return rc;
  const int64_t tokens = shape->B * shape->T;
  const int et = shape->dt_dtype, ep = shape->param_dtype;
  if (bad(x, tokens) || bad_el(dt, et, tokens) || bad_el(A, ep) || bad(Bm, tokens) || bad(Cm, tokens) || mis_el(D, ep) ||
      mis_el(dt_bias, ep) || mis(initial_state) || bad(dy, tokens) || mis(d_final_state) || bad(dx, tokens) ||
      bad_el(ddt, et, tokens) || bad_el(dA, ep) || bad(dB, tokens) || bad(dC, tokens) || mis_el(dD, ep) ||
      mis_el(d_dt_bias, ep) || mis(d_initial_state))
    return GDN_ERR_ARG;
  if (cu_mismatch(cu_seqlens, shape->cu_seqlens_host)) return GDN_ERR_ARG;
  const SsmPlan P = plan_ssm(shape, true);
  if (const int rc = check_plan(P, shape)) return rc;
  if (bad(workspace) || workspace_bytes < P.bytes) return GDN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  const bool split = P.max_segs > 1;
  const int is_bf16 = shape->dtype == GDN_BF16, n = (int)shape->n, p = (int)shape->p, div = (int)(shape->H / shape->G);
  const gdn::SsmTensor tx = {x, shape->x_stride ? shape->x_stride : shape->H * p, 1};
  const gdn::SsmTensor tb = {Bm, shape->b_stride ? shape->b_stride : shape->G * n, div};
  const gdn::SsmTensor tc = {Cm, shape->c_stride ? shape->c_stride : shape->G * n, div};
  const gdn::SsmTensor ty = {dy, shape->H * p, 1};
  float* hstate = split ? reinterpret_cast<float*>(ws + P.state[0]) : nullptr;
  float* gstate = split ? reinterpret_cast<float*>(ws + P.state[1]) : nullptr;
  float* hdecay = split ? reinterpret_cast<float*>(ws + P.decay[0]) : nullptr;
  float* gdecay = split ? reinterpret_cast<float*>(ws + P.decay[1]) : nullptr;
  gdn::SsmScans a{};
  if (ssm_seqs(shape, P, cu_seqlens, ws, stream, &a.seqs) != hipSuccess) return GDN_ERR_HIP;
  a.param_bf16 = shape->param_dtype == GDN_BF16;
  float* gfwd = reinterpret_cast<float*>(ws + P.gates[0]);
  float* grev = reinterpret_cast<float*>(ws + P.gates[1]);
  if (gdn::launch_ssm_gates(a.seqs, ssm_gates(shape, dt, A, dt_bias), gfwd, grev, stream) != hipSuccess)
    return GDN_ERR_HIP;
  if (split) {                             // the states at every segment's start, both ways
    gdn::SsmScan& f = a.s[0];
    f.gates = gfwd;
    f.k = tb;
    f.v = tx;
    f.kappa_delta = 1;
    f.seg_state = hstate;
    f.seg_decay = hdecay;
    gdn::SsmScan& r = a.s[1];
    r.gates = grev;
    r.k = tc;
    r.v = ty;
    r.rev = 1;
    r.seg_state = gstate;
    r.seg_decay = gdecay;
    if (gdn::launch_ssm_scan(a, 2, is_bf16, n, p, gdn::kScanState, stream) != hipSuccess) return GDN_ERR_HIP;
    const gdn::SsmMerge m[2] = {{hstate, hdecay, initial_state, 0}, {gstate, gdecay, d_final_state, 1}};
    if (gdn::launch_ssm_merge(a.seqs, m, 2, n * p, stream) != hipSuccess) return GDN_ERR_HIP;
  }
  const bool sums = shape->G < shape->H;   // dB, dC per head first, then summed over a group's heads
  float* dBp = sums ? reinterpret_cast<float*>(ws + P.dBp) : nullptr;
  float* dCp = sums ? reinterpret_cast<float*>(ws + P.dCp) : nullptr;
  void* cdc = ws + P.cdc;
  void* xdu = ws + P.xdu;
  void* dyx = ws + P.dyx;
  float* hT = d_final_state ? reinterpret_cast<float*>(ws + P.hT) : nullptr;
  gdn::SsmScan du{}, dc{}, db{};
  du.gates = grev;
  du.q = tb;
  du.k = tc;
  du.v = ty;
  du.aux = tx;
  du.rev = 1;
  du.alpha_delta = 1;
  du.D = D;
  du.h0 = d_final_state;
  du.seg_start = gstate;
  du.out = dx;
  du.out_f32 = !is_bf16;
  du.hT = d_initial_state;
  du.decay0 = gfwd;
  du.dot_out = xdu;
  du.dot_skip = dD ? dyx : nullptr;
  dc.gates = gfwd;
  dc.q = ty;
  dc.k = tx;
  dc.v = tb;
  dc.aux = tc;
  dc.kappa_delta = 1;
  dc.h0 = initial_state;
  dc.seg_start = hstate;
  dc.state_t = 1;
  dc.out = sums ? static_cast<void*>(dCp) : dC;
  dc.out_f32 = sums || !is_bf16;
  dc.hT = hT;
  dc.dot_out = cdc;
  db.gates = grev;
  db.q = tx;
  db.k = ty;
  db.v = tc;
  db.rev = 1;
  db.alpha_delta = 1;
  db.h0 = d_final_state;
  db.seg_start = gstate;
  db.state_t = 1;
  db.out = sums ? static_cast<void*>(dBp) : dB;
  db.out_f32 = sums || !is_bf16;
  a.s[0] = dc;
  a.s[1] = db;
  a.s[2] = du;
  if (n == p) {
    if (gdn::launch_ssm_scan(a, 3, is_bf16, n, n, gdn::kScanGrad, stream) != hipSuccess) return GDN_ERR_HIP;
  } else {
    if (gdn::launch_ssm_scan(a, 2, is_bf16, p, n, gdn::kScanGrad, stream) != hipSuccess) return GDN_ERR_HIP;
    a.s[0] = du;
    if (gdn::launch_ssm_scan(a, 1, is_bf16, n, p, gdn::kScanGrad, stream) != hipSuccess) return GDN_ERR_HIP;
  }
  gdn::SsmGateGrads g{};
  g.seqs = a.seqs;
  g.gates = gfwd;
  g.A = A;
  g.dt_bf16 = shape->dt_dtype == GDN_BF16;
  g.param_bf16 = a.param_bf16;
  g.softplus = shape->dt_softplus;
  g.cdc = cdc;
  g.xdu = xdu;
  g.dots_f64 = !is_bf16;
  g.dyx = dD ? dyx : nullptr;
  g.hstart = hstate;
  g.gstart = gstate;
  g.hT = hT;
  g.dhT = d_final_state;
  g.has_h0 = initial_state != nullptr;
  g.elems = n * p;
  g.ddt = ddt;
  g.part = reinterpret_cast<double*>(ws + P.part);
  g.dA = dA;
  g.dbias = d_dt_bias;
  g.dD = dD;
  if (gdn::launch_ssm_gate_grads(g, stream) != hipSuccess) return GDN_ERR_HIP;
  gdn::SsmHeadSum heads{};
  if (sums) heads = {{dBp, dCp}, {dB, dC}, tokens * shape->G * (n / 4), div, n / 4, 0};
  return launched(gdn::launch_ssm_sums(g, heads, is_bf16, stream));
}

int gdn_ssm_step(const void* x, const void* dt, const void* A, const void* Bm, const void* Cm, const void* D,
                 const void* dt_bias, const float* state, const int32_t* slots, void* y, float* state_out,
                 const gdn_ssm_shape* shape, hipStream_t stream) {
  if (!shape || shape->T != 1 || shape->cu_seqlens_host || shape->N < 1 || shape->x_stride || shape->b_stride ||
      shape->c_stride)
    return GDN_ERR_ARG;
  gdn_ssm_shape rows = *shape;             // (N counts slots here)
  rows.N = rows.B;
  if (const int rc = check_ssm(&rows)) return rc;
  const int ep = shape->param_dtype;
  if (bad(x) || bad_el(dt, shape->dt_dtype) || bad_el(A, ep) || bad(Bm) || bad(Cm) || mis_el(D, ep) || mis_el(dt_bias, ep) ||
      bad(state) || mis_ints(slots) || bad(y) || bad(state_out))
    return GDN_ERR_ARG;
  if (!slots && shape->B > shape->N) return GDN_ERR_ARG;
  if (shape->N > INT_MAX || shape->B * shape->H > gdn::kMaxDispatchItems / 256 / 4) return GDN_ERR_UNSUPPORTED;
  gdn::StepArgs a{};
  a.q = Cm;
  a.k = Bm;
  a.v = x;
  a.gate = dt;
  a.gates = ssm_gates(shape, dt, A, dt_bias);
  a.D = D;
  a.state = state;
  a.slots = slots;
  a.o = y;
  a.state_out = state_out;
  a.R = shape->B;
  a.S = shape->N;
  a.H = (int)shape->H;
  a.div = (int)(shape->H / shape->G);
  a.dk = (int)shape->n;
  a.dv = (int)shape->p;
  a.bf16 = shape->dtype == GDN_BF16;
  return launched(gdn::launch_recurrent_step(a, stream));
}

int gdn_delta_step(const void* q, const void* k, const void* v, const float* g, const void* beta,
                   const float* state, const int32_t* slots, float scale, void* o, float* state_out,
                   const gdn_shape* shape, hipStream_t stream) {
  if (!shape || shape->B < 1 || shape->B > INT_MAX / 2 || shape->T != 1 || shape->H < 1 || shape->H > 65535 ||
      shape->N < 1 || shape->cu_seqlens_host || !std::isfinite(scale))
    return GDN_ERR_ARG;
  if ((shape->dk != 64 && shape->dk != 128) || (shape->dv != 64 && shape->dv != 128) || !ok_type(shape->qkv_dtype) ||
      !ok_type(shape->beta_dtype))
    return GDN_ERR_UNSUPPORTED;
  if (bad(q) || bad(k) || bad(v) || bad_el(g, GDN_F32) || bad_el(beta, shape->beta_dtype) || bad(state) || mis_ints(slots) ||
      bad(o) || bad(state_out))
    return GDN_ERR_ARG;
  if (!slots && shape->B > shape->N) return GDN_ERR_ARG;
  if (shape->N > INT_MAX || shape->B * shape->H > gdn::kMaxDispatchItems / 256 / 4) return GDN_ERR_UNSUPPORTED;
  gdn::StepArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.gate = g;
  a.beta = beta;
  a.state = state;
  a.slots = slots;
  a.o = o;
  a.state_out = state_out;
  a.R = shape->B;
  a.S = shape->N;
  a.H = (int)shape->H;
  a.div = 1;
  a.dk = (int)shape->dk;
  a.dv = (int)shape->dv;
  a.bf16 = shape->qkv_dtype == GDN_BF16;
  a.beta_bf16 = shape->beta_dtype == GDN_BF16;
  a.scale = scale;
  a.delta_rule = 1;
  return launched(gdn::launch_recurrent_step(a, stream));
}

int gdn_norm_fwd(const void* x, const void* weight, const void* bias, const void* gate, void* y, float* mean,
                 float* rstd, const gdn_norm_shape* shape, hipStream_t stream) {
  if (const int rc = check_norm(shape)) return rc;
  if (bad(x, shape->rows) || mis(weight) || mis(bias) || mis(gate) || bad(y, shape->rows) ||
      mis_el(mean, GDN_F32) || mis_el(rstd, GDN_F32))
    return GDN_ERR_ARG;
  gdn::NormArgs a = norm_args(shape);
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.gate = gate;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return launched(gdn::launch_norm_fwd(a, stream));
}

int gdn_norm_bwd_workspace_bytes(const gdn_norm_shape* shape, size_t* bytes) {
  if (const int rc = check_norm(shape)) return rc;
  if (!bytes) return GDN_ERR_ARG;
  *bytes = up256((size_t)gdn::norm_bwd_strips(shape->rows, (int)shape->H, (int)shape->D, shape->dtype == GDN_BF16) * 2 *
                 shape->H * shape->D * 4);
  return GDN_OK;
}

int gdn_norm_bwd(const void* x, const void* weight, const void* bias, const void* gate, const float* mean,
                 const float* rstd, const void* dy, void* dx, void* dweight, void* dbias, void* dgate,
                 const gdn_norm_shape* shape, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  size_t need = 0;
  if (const int rc = gdn_norm_bwd_workspace_bytes(shape, &need)) return rc;
  const int64_t rows = shape->rows;
  if (bad(x, rows) || mis(weight) || mis(bias) || mis(gate) || bad_el(mean, GDN_F32, rows) ||
      bad_el(rstd, GDN_F32, rows) || bad(dy, rows) ||
      bad(dx, rows) || mis(dweight) || mis(dbias) || mis(dgate) || (rows > 0 && (gate != nullptr) != (dgate != nullptr)))
    return GDN_ERR_ARG;
  if ((dweight || dbias) && (bad(workspace) || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  gdn::NormArgs a = norm_args(shape);
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.gate = gate;
  a.dy = dy;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.dgate = dgate;
  a.part = static_cast<float*>(workspace);
  return launched(gdn::launch_norm_bwd(a, stream));
}

}  // extern "C"
