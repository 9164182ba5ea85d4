// Internal host-side launch interface of the operators around the delta rule: the short
// convolution, the selective scan, the heads' norm and the single-token steps.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_launch.h"

namespace gdn {

// ---- selective scan (ssm_scan.h, ssm_aux.hip) --------------------------------------

// The sequences and their split, shared by every launch of one call.
struct SsmSeqs {
  const int32_t* cu;         // device cu_seqlens or null
  int64_t T;                 // tokens per batch row (dense)
  int N, H;
  int seg_chunks;            // chunks per segment
  int segs;                  // dense: segments per sequence
  int64_t units;             // segments over all sequences x H
  int64_t chunks;            // chunks over all sequences
  const int32_t* chunk_off;  // [N + 1] chunks, and segments, in front of each sequence; null up
  const int32_t* seg_off;    // to kSsmCounted of them, or dense
};
constexpr int kSsmCounted = 64;            // (a lane each)
hipError_t launch_ssm_offsets(const SsmSeqs& q, int32_t* chunk_off, int32_t* seg_off, hipStream_t s);

// The gates: delta = softplus(dt + dt_bias) (or without the softplus), a = delta A.
struct SsmGates {
  const void* dt;
  const void* A;
  const void* bias;          // or null
  int dt_bf16, param_bf16, softplus;
};
// The scans' gates of every (chunk, head), in order (fwd) and, if rev is not null, last to
// first: [chunks, H, 256] floats each (ssm_scan.h).
hipError_t launch_ssm_gates(const SsmSeqs& q, const SsmGates& g, float* fwd, float* rev, hipStream_t s);

// A token-major tensor [tokens, heads, width] as the scan reads it: head h's row of
// token t starts at t * stride + (h / div) * width.
struct SsmTensor {
  const void* p;
  int64_t stride;
  int div;
};

// One scan: out_j = alpha_j q_j h_j + D v_j, h_j = exp(a_j) h_{j-1} + kappa_j k_j v_j^T,
// over a sequence's tokens in order, or last to first (rev; then step j applies the
// decay of the token after its own, so that the scan is the adjoint of the forward one).
struct SsmScan {
  const float* gates;        // launch_ssm_gates' output in the scan's direction
  SsmTensor q, k, v;
  SsmTensor aux;             // p == null: no dots; else dots with the output before alpha
  int rev;
  int kappa_delta;           // kappa = delta (else 1)
  int alpha_delta;           // alpha = delta (else 1)
  const void* D;             // skip weights [H] or null
  const float* h0;           // [N, H] states before the first step, or null (zero)
  const float* seg_start;    // [segments, H] states, or null: a segment's own start
  int state_t;               // the stored states are [DV, DK], not [DK, DV]
  void* out;                 // token-major [tokens, H, DV]
  int out_f32;               // out is fp32 (else the tensors' type)
  float* hT;                 // [N, H] states after the last step, or null
  const float* decay0;       // null, or the gates in order: hT times exp(a) of the first token
  void* dot_out;             // [chunks, H, 64] aux . (q h), or null; fp64 of fp32 tensors, else fp32
  void* dot_skip;            // [chunks, H, 64] aux . v, or null
  float* seg_state;          // state pass: [segments, H] end states from a zero start
  float* seg_decay;          // state pass: [segments, H] decay over the segment
};
struct SsmScans {
  SsmSeqs seqs;
  int param_bf16;            // D
  SsmScan s[3];
};

// What a launch does: only the segments' end states and decays, of every segment but each
// sequence's last in scan order; the forward scan (in order, kappa = delta, alpha = 1, no
// dots, outputs in the tensors' type); or any scan of the backward pass.
enum { kScanState = 0, kScanForward = 1, kScanGrad = 2 };
// count scans (blockIdx.y); dk, dv in {64, 128}.
hipError_t launch_ssm_scan(const SsmScans& a, int count, bool bf16, int dk, int dv, int mode,
                           hipStream_t s);
hipError_t launch_ssm_scan_bf16(const SsmScans& a, int count, int dk, int dv, int mode, hipStream_t s);
hipError_t launch_ssm_scan_f32(const SsmScans& a, int count, int dk, int dv, int mode, hipStream_t s);

// Turns the segments' end states into their start states, in place: a chain over each
// sequence's segments (last to first for rev) from h0 (null: zero).
struct SsmMerge {
  float* state;              // [segments, H, n, p]
  const float* decay;        // [segments, H]
  const float* h0;           // [N, H, n, p] or null
  int rev;
};
hipError_t launch_ssm_merge(const SsmSeqs& q, const SsmMerge* m, int count, int elems, hipStream_t s);

// Gradients of the gates from the scans' dots.
struct SsmGateGrads {
  SsmSeqs seqs;
  const float* gates;        // in order
  const void* A;
  int dt_bf16, param_bf16, softplus;
  const void* cdc;           // [chunks, H, 64] C . dC, fp64 or fp32
  const void* xdu;           // [chunks, H, 64] x . du
  const void* dyx;           // [chunks, H, 64] dy . x, or null (no D)
  int dots_f64;
  const float* hstart;       // [segments, H, n, p] (more than one segment somewhere) or null
  const float* gstart;       // the reverse scan's segment starts
  const float* hT;           // [N, H, n, p] final states, null without dhT
  const float* dhT;
  int has_h0;                // without a start state nothing crosses a sequence's first decay
  int elems;
  void* ddt;                 // dt's type
  double* part;              // [segments, H, 3]: dA, ddt_bias, dD
  void* dA;                  // the parameters' type; any may be null
  void* dbias;
  void* dD;
};
hipError_t launch_ssm_gate_grads(const SsmGateGrads& a, hipStream_t s);
// out [tokens, G, n] (E) = sum over each group's heads of in [tokens, H, n] fp32, twice.
struct SsmHeadSum {
  const float* in[2];
  void* out[2];
  int64_t quads;             // tokens * G * n / 4; 0: nothing to sum
  int per, n4;               // heads of a group, n / 4
  uint32_t blocks;           // (set by the launch) workgroups per tensor
};
// The parameters' gradients from the segments' shares, and the sums over heads.
hipError_t launch_ssm_sums(const SsmGateGrads& a, const SsmHeadSum& heads, bool is_bf16, hipStream_t s);

// ---- short convolution (conv.hip) --------------------------------------------------
struct ConvArgs {
  const void* x;
  int64_t x_stride;
  const void* w;             // [D, W]
  const void* bias;          // or null
  const void* init;          // [N, W-1, D] or null
  const int32_t* cu;
  void* y;
  void* fin;                 // [N, W-1, D] or null
  int64_t B, T, D;           // packed: B = 1
  int N, W, bf16, param_bf16, silu;
  // backward
  const void* dy;
  const void* dfin;          // or null
  void* dx;
  void* dw;
  void* dbias;               // or null
  void* dinit;               // or null
  float* part;               // [blocks, W + 1, D]
};
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s);
// Token blocks of the backward (rows of its partial sums).
int64_t conv_bwd_rows(int64_t tokens);
bool conv_bwd_fits(int64_t tokens, int64_t D, int W);   // every launch's workgroups in one dispatch

// ---- single-token steps (step.hip) -------------------------------------------------
struct ConvStepArgs {
  const void* x;             // [R, D]
  const void* w;
  const void* bias;
  const void* state;         // [S, W-1, D]
  const int32_t* slots;      // [R] or null: row i uses slot i
  void* y;
  void* state_out;
  int64_t R, S, D;
  int W, bf16, param_bf16, silu;
};
hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t s);

struct StepArgs {
  const void* q;             // [R, Gq, dk]
  const void* k;
  const void* v;             // [R, H, dv]
  const void* gate;          // delta rule: g fp32 [R, H]; selective: dt
  const void* beta;          // delta rule
  SsmGates gates;            // selective
  const void* D;             // selective: skip weights or null
  const float* state;        // [S, H, dk, dv]
  const int32_t* slots;
  void* o;
  float* state_out;
  int64_t R, S;
  int H, div, dk, dv, bf16, beta_bf16;
  float scale;
  int delta_rule;
};
hipError_t launch_recurrent_step(const StepArgs& a, hipStream_t s);

// ---- norm (norm.hip) ---------------------------------------------------------------
struct NormArgs {
  const void* x;
  const void* gate;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  int64_t rows;              // tokens
  int H, D;
  int bf16, param_bf16;
  float eps;
  // backward
  const void* dy;
  const float* mean_in;
  const float* rstd_in;
  void* dx;
  void* dgate;
  void* dw;
  void* db;
  float* part;               // [strips, 2, H, D]
};
constexpr int kNormMaxWidth = 8192;   // elements of a row that a workgroup holds
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s);
int64_t norm_bwd_strips(int64_t rows, int H, int D, int bf16);
bool norm_fits(int64_t rows, int H, int D, int bf16);   // every launch's workgroups in one dispatch

}  // namespace gdn
