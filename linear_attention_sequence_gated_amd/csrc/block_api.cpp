// block_api.cpp -- the C ABI of what stands around a recurrent layer's state
// update (declared in include/gdn.h): validates every argument before anything is
// enqueued, then launches.
#include <stdint.h>

#include <cmath>
#include <initializer_list>

#include "../../include/gdn.h"
#include "gdn_block.hpp"

namespace {

template <int N> bool all_aligned(const void* const (&ptrs)[N]) {
  for (const void* p : ptrs)
    if (p && (reinterpret_cast<uintptr_t>(p) & 15u)) return false;
  return true;
}

// Whether a buffer that one workgroup reads is one that another writes: states before
// and behind a call, or rows and results of a convolution.
bool same(const void* read, const void* written) { return read && read == written; }

// Whether any result is any of what is read; if_any: rows (states), which a call without
// tokens (sequences) does not read.
bool in_place(std::initializer_list<const void*> read, std::initializer_list<const void*> written) {
  for (const void* r : read)
    for (const void* w : written)
      if (same(r, w)) return true;
  return false;
}
const void* if_any(int n, const void* p) { return n ? p : nullptr; }

// Whether a norm's result, whose rows are C apart, begins where rows do that lie
// elsewhere: the threads that write a row have read the same values of the rows then
// only if these are C apart too.
bool elsewhere(const void* rows, long long stride, const void* result, int T, int C) {
  return T > 1 && stride != C && same(rows, result);
}

int status(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

bool known_dtype(int d) { return d == GDN_F32 || d == GDN_BF16 || d == GDN_C64; }

// Types of rows and of parameters: bf16 or float32; float32 rows have float32
// parameters.
int types(int dtype, int param_dtype) {
  if (!known_dtype(dtype) || !known_dtype(param_dtype)) return GDN_ERR_DTYPE;
  if (dtype == GDN_C64 || param_dtype == GDN_C64 || (dtype == GDN_F32 && param_dtype != GDN_F32)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// A row stride: room for the row, 16-byte aligned rows, no offset past 2^62.
bool stride_ok(long long s, long long row) { return s >= row && s % 8 == 0 && s < (1LL << 32); }

// Rows of a norm: their pieces fit a workgroup's registers.
int norm_shape(int T, int C, int dtype) {
  if (T < 0 || C <= 0 || T >= (1 << 24)) return GDN_ERR_SHAPE;
  return C % 8 == 0 && C <= 16384 && dtype != GDN_C64 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

// Sizes of a convolution, which keep its launches under 2^32 work-items.
int conv_shape(int T, int R, int C, int W) {
  if (T < 0 || R < 0 || C <= 0 || W <= 0 || R >= (1 << 20) || T >= (1 << 28)) return GDN_ERR_SHAPE;
  if ((long long)T * C >= (1LL << 34) || (long long)R * C >= (1LL << 31)) return GDN_ERR_SHAPE;
  return C % 8 == 0 && C <= 65536 && W >= 2 && W <= 4 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

int norm(const void* x, const void* residual, const void* weight, void* out, void* sum, float* scale, float eps,
         long long xs, long long rs, int T, int C, int fmt, int block, int dtype, int weight_dtype, void* stream) {
  if (const int s = types(dtype, weight_dtype)) return s;
  if (const int s = norm_shape(T, C, dtype)) return s;
  if (!std::isfinite(eps) || eps < 0.f || !stride_ok(xs, C) || (residual && !stride_ok(rs, C))) return GDN_ERR_SHAPE;
  if (T == 0) return GDN_OK;
  if (!x || !weight || !out || (residual && !sum) || (fmt >= 0 && !scale)) return GDN_ERR_NULL;
  const void* ptrs[] = {x, residual, weight, out, sum, scale};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  const void* results[] = {out, residual ? sum : nullptr};
  for (const void* r : results)
    if (elsewhere(x, xs, r, T, C) || elsewhere(residual, rs, r, T, C)) return GDN_ERR_UNSUPPORTED;
  if (same(out, results[1])) return GDN_ERR_UNSUPPORTED;
  if (fmt >= 0 && (same(x, out) || same(residual, out) || same(x, scale) || same(residual, scale))) return GDN_ERR_UNSUPPORTED;
  return status(gdn::launch_rms_norm({x, residual, weight, out, sum, scale, xs, rs, eps, T, C, dtype == GDN_F32,
                                      weight_dtype == GDN_F32, fmt, block, stream}));
}

// Sizes and types of a scan.  64 rows of x, B and C, the most that a buffer
// resource covers, stay inside 32-bit byte offsets.
int scan_shape(int T, int R, int H, int P, int G, int N) {
  if (T < 0 || R < 0 || H <= 0 || P <= 0 || G <= 0 || N <= 0 || H % G || T >= (1 << 26) || R >= (1 << 20)) return GDN_ERR_SHAPE;
  if (H >= (1 << 16) || (long long)T * H >= (1LL << 31) || (long long)R * H >= (1LL << 22)) return GDN_ERR_SHAPE;
  return (P == 64 || P == 128) && (N == 64 || N == 128) ? GDN_OK : GDN_ERR_UNSUPPORTED;
}
bool near_ok(long long s, long long row) { return stride_ok(s, row) && s < (1LL << 24); }
// dt and the parameters of heads may begin anywhere, as columns of a projection do.
bool params_aligned(std::initializer_list<const void*> ptrs, int dtype) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % (dtype == GDN_F32 ? 4 : 2)) return false;
  return true;
}
int scan_types(int dtype, int dt_dtype, int param_dtype) {
  for (const int d : {dtype, dt_dtype, param_dtype})
    if (!known_dtype(d)) return GDN_ERR_DTYPE;
  return dtype == GDN_BF16 && dt_dtype != GDN_C64 && param_dtype != GDN_C64 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int gdn_rms_norm(const void* x, const void* residual, const void* weight, void* out, void* sum, float eps,
                 long long x_stride, long long residual_stride, int T, int C, int dtype, int weight_dtype, void* stream) {
  return norm(x, residual, weight, out, sum, nullptr, eps, x_stride, residual_stride, T, C, -1, 0, dtype, weight_dtype, stream);
}

int gdn_rms_norm_quant(const void* x, const void* residual, const void* weight, void* codes, float* scale, void* sum,
                       float eps, long long x_stride, long long residual_stride, int T, int C, int block, int dtype,
                       int weight_dtype, int format, void* stream) {
  if (format != GDN_CACHE_I8 && format != GDN_CACHE_E4M3) return GDN_ERR_DTYPE;
  if (block < 0) return GDN_ERR_SHAPE;
  if (block != 0 && (block != 128 || C % 128)) return GDN_ERR_UNSUPPORTED;
  return norm(x, residual, weight, codes, sum, scale, eps, x_stride, residual_stride, T, C, format, block, dtype, weight_dtype,
              stream);
}

size_t gdn_rms_norm_bwd_workspace_bytes(int T, int C, int dtype) {
  return types(dtype, GDN_F32) || norm_shape(T, C, dtype) ? 0 : gdn::rms_norm_bwd_workspace_bytes(T, C, dtype == GDN_F32);
}

int gdn_rms_norm_bwd(const void* sum, const void* weight, const void* grad_out, const void* grad_sum, void* grad_x,
                     void* grad_weight, float eps, long long sum_stride, long long grad_out_stride,
                     long long grad_sum_stride, int T, int C, int dtype, int weight_dtype, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (const int s = types(dtype, weight_dtype)) return s;
  if (const int s = norm_shape(T, C, dtype)) return s;
  if (!std::isfinite(eps) || eps < 0.f || !stride_ok(sum_stride, C) || !stride_ok(grad_out_stride, C)) return GDN_ERR_SHAPE;
  if (grad_sum && !stride_ok(grad_sum_stride, C)) return GDN_ERR_SHAPE;
  if (!weight || !grad_weight || (T && (!sum || !grad_out || !grad_x))) return GDN_ERR_NULL;
  const void* ptrs[] = {sum, weight, grad_out, grad_sum, grad_x, grad_weight, workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  const size_t need = gdn::rms_norm_bwd_workspace_bytes(T, C, dtype == GDN_F32);
  if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  if (elsewhere(sum, sum_stride, grad_x, T, C) || elsewhere(grad_out, grad_out_stride, grad_x, T, C) ||
      elsewhere(grad_sum, grad_sum_stride, grad_x, T, C))
    return GDN_ERR_UNSUPPORTED;
  return status(gdn::launch_rms_norm_bwd({sum, weight, grad_out, grad_sum, grad_x, grad_weight, static_cast<float*>(workspace),
                                          sum_stride, grad_out_stride, grad_sum_stride, eps, T, C, dtype == GDN_F32,
                                          weight_dtype == GDN_F32, stream}));
}

int gdn_short_conv(const void* x, const void* weight, const void* bias, const int* cu_seqlens, const void* state, void* out,
                   void* state_final, long long x_stride, int T, int R, int C, int W, int dtype, int weight_dtype,
                   int silu, int zero_rest, void* stream) {
  if (const int s = types(dtype, weight_dtype)) return s;
  if (const int s = conv_shape(T, R, C, W)) return s;
  if (!stride_ok(x_stride, C)) return GDN_ERR_SHAPE;
  if (T == 0 && (R == 0 || !state_final)) return GDN_OK;
  if (!weight || !cu_seqlens || (T && (!x || !out))) return GDN_ERR_NULL;
  const void* ptrs[] = {x, weight, bias, cu_seqlens, state, out, state_final};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  if (in_place({if_any(T, x), if_any(R, state)}, {out, state_final})) return GDN_ERR_UNSUPPORTED;
  return status(gdn::launch_short_conv({x, weight, bias, cu_seqlens, state, out, state_final, x_stride, T, R, C, W,
                                        dtype == GDN_F32, weight_dtype == GDN_F32, silu != 0, zero_rest != 0, stream}));
}

size_t gdn_short_conv_bwd_workspace_bytes(int T, int C, int W) {
  return conv_shape(T, 0, C, W) ? 0 : gdn::short_conv_bwd_workspace_bytes(T, C, W);
}

int gdn_short_conv_bwd(const void* x, const void* weight, const void* bias, const void* grad_out, const int* cu_seqlens,
                       const void* state, const void* grad_state_final, void* grad_x, void* grad_weight, void* grad_bias,
                       void* grad_state, long long x_stride, long long grad_out_stride, int T, int R, int C, int W,
                       int dtype, int weight_dtype, int silu, int zero_rest, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (const int s = types(dtype, weight_dtype)) return s;
  if (const int s = conv_shape(T, R, C, W)) return s;
  if (!stride_ok(x_stride, C) || !stride_ok(grad_out_stride, C)) return GDN_ERR_SHAPE;
  if (!weight || !cu_seqlens || !grad_weight || (T && (!x || !grad_out || !grad_x))) return GDN_ERR_NULL;
  const void* ptrs[] = {x, weight, bias, grad_out, cu_seqlens, state, grad_state_final, grad_x, grad_weight, grad_bias, grad_state,
                        workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  const size_t need = gdn::short_conv_bwd_workspace_bytes(T, C, W);
  if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  if (in_place({if_any(T, x), if_any(T, grad_out), if_any(R, state), if_any(R, grad_state_final)}, {grad_x, grad_state}))
    return GDN_ERR_UNSUPPORTED;
  return status(gdn::launch_short_conv_bwd({x, weight, bias, grad_out, cu_seqlens, state, grad_state_final, grad_x, grad_weight,
                                            grad_bias, grad_state, static_cast<float*>(workspace), x_stride, grad_out_stride,
                                            T, R, C, W, dtype == GDN_F32, weight_dtype == GDN_F32, silu != 0, zero_rest != 0,
                                            stream}));
}

int gdn_short_conv_step(const void* x, const void* weight, const void* bias, void* state, void* out, long long x_stride,
                        int R, int C, int W, int dtype, int weight_dtype, int silu, void* stream) {
  if (const int s = types(dtype, weight_dtype)) return s;
  if (const int s = conv_shape(R, R, C, W)) return s;
  if (!stride_ok(x_stride, C)) return GDN_ERR_SHAPE;
  if (R == 0) return GDN_OK;
  if (!x || !weight || !state || !out) return GDN_ERR_NULL;
  const void* ptrs[] = {x, weight, bias, state, out};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  if (in_place({x, state}, {out}) || same(x, state)) return GDN_ERR_UNSUPPORTED;
  return status(gdn::launch_short_conv_step({x, weight, bias, state, out, x_stride, R, C, W, dtype == GDN_F32,
                                             weight_dtype == GDN_F32, silu != 0, stream}));
}

size_t gdn_ssm_scan_workspace_bytes(int T, int H, int P, int G, int N) {
  return scan_shape(T, 0, H, P, G, N) ? 0 : gdn::ssm_scan_workspace_bytes(T, H, P, G, N);
}

int gdn_ssm_scan(const void* x, const void* dt, const void* a, const void* B, const void* C, const void* D,
                 const void* dt_bias, const int* cu_seqlens, const float* S0, void* out, float* S_final, long long x_stride,
                 long long dt_stride, long long B_stride, long long C_stride, int T, int R, int H, int P, int G, int N,
                 int dtype, int dt_dtype, int param_dtype, int zero_rest, void* workspace, size_t workspace_bytes,
                 void* stream) {
  if (const int s = scan_types(dtype, dt_dtype, param_dtype)) return s;
  if (const int s = scan_shape(T, R, H, P, G, N)) return s;
  if (!near_ok(x_stride, (long long)H * P) || !near_ok(B_stride, (long long)G * N) || !near_ok(C_stride, (long long)G * N))
    return GDN_ERR_SHAPE;
  if (dt_stride < H || dt_stride >= (1LL << 32)) return GDN_ERR_SHAPE;
  if (T == 0 && (R == 0 || !S_final)) return GDN_OK;
  if (!a || !cu_seqlens || (T && (!x || !dt || !B || !C || !out))) return GDN_ERR_NULL;
  const void* ptrs[] = {x, B, C, cu_seqlens, S0, out, S_final, workspace};
  if (!all_aligned(ptrs) || !params_aligned({dt}, dt_dtype) || !params_aligned({a, D, dt_bias}, param_dtype)) return GDN_ERR_ALIGN;
  const size_t need = gdn::ssm_scan_workspace_bytes(T, H, P, G, N);
  if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  if (in_place({if_any(T, x), if_any(T, dt), if_any(T, B), if_any(T, C), if_any(R, S0)}, {out, S_final})) return GDN_ERR_UNSUPPORTED;
  return status(gdn::launch_ssm_scan({x, dt, a, B, C, D, dt_bias, cu_seqlens, S0, out, S_final, static_cast<float*>(workspace),
                                      x_stride, dt_stride, B_stride, C_stride,
                                      {T, R, H, P, G, N, dt_dtype == GDN_F32, param_dtype == GDN_F32}, zero_rest != 0, stream}));
}

size_t gdn_ssm_scan_bwd_workspace_bytes(int T, int R, int H, int P, int G, int N) {
  return scan_shape(T, R, H, P, G, N) ? 0 : gdn::ssm_scan_bwd_workspace_bytes(T, R, H, P, G, N);
}

int gdn_ssm_scan_bwd(const void* x, const void* dt, const void* a, const void* B, const void* C, const void* D,
                     const void* dt_bias, const void* grad_out, const int* cu_seqlens, const float* S0,
                     const float* grad_S_final, void* grad_x, void* grad_dt, void* grad_a, void* grad_B, void* grad_C,
                     void* grad_D, void* grad_dt_bias, float* grad_S0, long long x_stride, long long dt_stride,
                     long long B_stride, long long C_stride, long long grad_out_stride, long long grad_x_stride,
                     long long grad_B_stride, long long grad_C_stride, int T, int R, int H, int P, int G, int N, int dtype,
                     int dt_dtype, int param_dtype, int zero_rest, void* workspace, size_t workspace_bytes, void* stream) {
  if (const int s = scan_types(dtype, dt_dtype, param_dtype)) return s;
  if (const int s = scan_shape(T, R, H, P, G, N)) return s;
  for (const long long s : {x_stride, grad_out_stride, grad_x_stride})
    if (!near_ok(s, (long long)H * P)) return GDN_ERR_SHAPE;
  for (const long long s : {B_stride, C_stride, grad_B_stride, grad_C_stride})
    if (!near_ok(s, (long long)G * N)) return GDN_ERR_SHAPE;
  if (dt_stride < H || dt_stride >= (1LL << 32)) return GDN_ERR_SHAPE;
  if (!a || !cu_seqlens || !grad_a || (T && (!x || !dt || !B || !C || !grad_out || !grad_x || !grad_dt || !grad_B || !grad_C)))
    return GDN_ERR_NULL;
  const void* ptrs[] = {x, B, C, grad_out, cu_seqlens, S0, grad_S_final, grad_x, grad_dt, grad_B, grad_C, grad_S0, workspace};
  if (!all_aligned(ptrs) || !params_aligned({dt}, dt_dtype) ||
      !params_aligned({a, D, dt_bias, grad_a, grad_D, grad_dt_bias}, param_dtype))
    return GDN_ERR_ALIGN;
  const size_t need = gdn::ssm_scan_bwd_workspace_bytes(T, R, H, P, G, N);
  if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  if (in_place({if_any(T, x), if_any(T, dt), if_any(T, B), if_any(T, C), if_any(T, grad_out), if_any(R, S0), if_any(R, grad_S_final)},
               {grad_x, grad_dt, grad_B, grad_C, grad_S0}))
    return GDN_ERR_UNSUPPORTED;
  return status(gdn::launch_ssm_scan_bwd({x, dt, a, B, C, D, dt_bias, grad_out, cu_seqlens, S0, grad_S_final, grad_x, grad_dt,
                                          grad_a, grad_B, grad_C, grad_D, grad_dt_bias, grad_S0, workspace, x_stride, dt_stride,
                                          B_stride, C_stride, grad_out_stride, grad_x_stride, grad_B_stride, grad_C_stride,
                                          {T, R, H, P, G, N, dt_dtype == GDN_F32, param_dtype == GDN_F32}, zero_rest != 0,
                                          stream}));
}

int gdn_ssm_step(const void* x, const void* dt, const void* a, const void* B, const void* C, const void* D,
                 const void* dt_bias, float* S, void* out, long long x_stride, long long dt_stride, long long B_stride,
                 long long C_stride, int R, int H, int P, int G, int N, int dtype, int dt_dtype, int param_dtype,
                 void* stream) {
  if (const int s = scan_types(dtype, dt_dtype, param_dtype)) return s;
  if (const int s = scan_shape(0, R, H, P, G, N)) return s;
  if (!stride_ok(x_stride, (long long)H * P) || !stride_ok(B_stride, (long long)G * N) || !stride_ok(C_stride, (long long)G * N))
    return GDN_ERR_SHAPE;
  if (dt_stride < H || dt_stride >= (1LL << 32)) return GDN_ERR_SHAPE;
  if (R == 0) return GDN_OK;
  if (!x || !dt || !a || !B || !C || !S || !out) return GDN_ERR_NULL;
  const void* ptrs[] = {x, B, C, S, out};
  if (!all_aligned(ptrs) || !params_aligned({dt}, dt_dtype) || !params_aligned({a, D, dt_bias}, param_dtype)) return GDN_ERR_ALIGN;
  if (in_place({x, dt, B, C, S}, {out}) || in_place({x, dt, B, C}, {S})) return GDN_ERR_UNSUPPORTED;
  return status(gdn::launch_ssm_step({x, dt, a, B, C, D, dt_bias, S, out, x_stride, dt_stride, B_stride, C_stride,
                                      {R, R, H, P, G, N, dt_dtype == GDN_F32, param_dtype == GDN_F32}, stream}));
}

}  // extern "C"
