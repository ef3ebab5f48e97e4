// gdn_block.hpp -- internal interface of the kernels around a recurrent layer's
// state update: the root-mean-square norm, the short convolution and the
// selective state space scan.  Arguments arrive validated (block_api.cpp).
// Strides are distances between rows, in elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

struct NormArgs {
  const void* x;
  const void* residual;  // may be NULL
  const void* weight;
  void* out;    // rows of the input's type, or codes
  void* sum;    // x + residual; NULL without a residual
  float* scale;  // of the codes
  long long xs, rs;
  float eps;
  int T, C;
  bool f32, w_f32;  // float32 rows, float32 weights; otherwise bf16
  int fmt;          // of the codes; -1: rows of the input's type
  int block;        // columns to a scale, 0: a whole row
  void* stream;
};
hipError_t launch_rms_norm(const NormArgs& a);

struct NormBwdArgs {
  const void* sum;
  const void* weight;
  const void* grad_out;
  const void* grad_sum;  // may be NULL
  void* grad_x;
  void* grad_weight;
  float* ws;
  long long ss, gs, gss;
  float eps;
  int T, C;
  bool f32, w_f32;
  void* stream;
};
size_t rms_norm_bwd_workspace_bytes(int T, int C, bool f32);
hipError_t launch_rms_norm_bwd(const NormBwdArgs& a);

struct ConvArgs {
  const void* x;
  const void* weight;
  const void* bias;  // may be NULL
  const int* cu;
  const void* state;  // may be NULL
  void* out;
  void* state_final;  // may be NULL
  long long xs;
  int T, R, C, W;
  bool f32, w_f32, silu, zero_rest;
  void* stream;
};
hipError_t launch_short_conv(const ConvArgs& a);

struct ConvBwdArgs {
  const void* x;
  const void* weight;
  const void* bias;
  const void* grad_out;
  const int* cu;
  const void* state;
  const void* grad_state_final;
  void* grad_x;
  void* grad_weight;
  void* grad_bias;   // may be NULL
  void* grad_state;  // may be NULL
  float* ws;
  long long xs, gs;
  int T, R, C, W;
  bool f32, w_f32, silu, zero_rest;
  void* stream;
};
size_t short_conv_bwd_workspace_bytes(int T, int C, int W);
hipError_t launch_short_conv_bwd(const ConvBwdArgs& a);

struct ConvStepArgs {
  const void* x;
  const void* weight;
  const void* bias;
  void* state;
  void* out;
  long long xs;
  int R, C, W;
  bool f32, w_f32, silu;
  void* stream;
};
hipError_t launch_short_conv_step(const ConvStepArgs& a);

// Types and sizes of a scan: H heads of P channels read G groups of B and C of N
// values.  dt is float32 or bf16, and so are the parameters.
struct ScanShape {
  int T, R, H, P, G, N;
  bool dt_f32, p_f32;
};

struct ScanArgs {
  const void* x;
  const void* dt;
  const void* a;
  const void* B;
  const void* C;
  const void* D;     // may be NULL
  const void* bias;  // may be NULL
  const int* cu;
  const float* S0;  // may be NULL
  void* out;
  float* S_final;  // may be NULL
  float* ws;
  long long xs, dts, bs, cs;
  ScanShape n;
  bool zero_rest;
  void* stream;
};
size_t ssm_scan_workspace_bytes(int T, int H, int P, int G, int N);
hipError_t launch_ssm_scan(const ScanArgs& a);

struct ScanBwdArgs {
  const void* x;
  const void* dt;
  const void* a;
  const void* B;
  const void* C;
  const void* D;
  const void* bias;
  const void* grad_out;
  const int* cu;
  const float* S0;
  const float* grad_S_final;  // may be NULL
  void* grad_x;
  void* grad_dt;
  void* grad_a;
  void* grad_B;
  void* grad_C;
  void* grad_D;     // may be NULL
  void* grad_bias;  // may be NULL
  float* grad_S0;   // may be NULL
  void* ws;
  long long xs, dts, bs, cs, gs, gxs, gbs, gcs;
  ScanShape n;
  bool zero_rest;
  void* stream;
};
size_t ssm_scan_bwd_workspace_bytes(int T, int R, int H, int P, int G, int N);
hipError_t launch_ssm_scan_bwd(const ScanBwdArgs& a);

struct ScanStepArgs {
  const void* x;
  const void* dt;
  const void* a;
  const void* B;
  const void* C;
  const void* D;
  const void* bias;
  float* S;
  void* out;
  long long xs, dts, bs, cs;
  ScanShape n;
  void* stream;
};
hipError_t launch_ssm_step(const ScanStepArgs& a);

}  // namespace gdn
