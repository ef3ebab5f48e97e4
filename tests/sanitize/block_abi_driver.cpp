// Host-only driver for the sanitizer test of the entry points around a recurrent
// layer: arguments that fail validation, the empty calls and workspace sizes up to
// the limits.  No call reaches a kernel.
#include <climits>
#include <cmath>
#include <cstdio>
#include <initializer_list>

#include "gdn.h"

static int failures = 0;

static void expect(const char* what, int got, int want) {
  if (got != want) {
    std::fprintf(stderr, "%s: status %d, expected %d\n", what, got, want);
    ++failures;
  }
}

alignas(16) static unsigned char buf[4096];
static void* const A = buf;
static int* const I = reinterpret_cast<int*>(buf);
static void* const U = buf + 1;  // misaligned
static float* const F = reinterpret_cast<float*>(buf);
constexpr int bf = GDN_BF16, f32 = GDN_F32;

static int norm(const void* x, float eps, long long stride, int T, int C, int dtype, int wdtype) {
  return gdn_rms_norm(x, A, A, A, A, eps, stride, stride, T, C, dtype, wdtype, nullptr);
}
static int quant(const void* x, long long stride, int T, int C, int block, int fmt) {
  return gdn_rms_norm_quant(x, A, A, A, F, A, 1e-6f, stride, stride, T, C, block, bf, bf, fmt, nullptr);
}
static int norm_bwd(const void* s, long long stride, int T, int C, void* ws, size_t bytes) {
  return gdn_rms_norm_bwd(s, A, A, A, A, A, 1e-6f, stride, stride, stride, T, C, bf, bf, ws, bytes, nullptr);
}
static int conv(const void* x, long long stride, int T, int R, int C, int W, int dtype, int wdtype) {
  return gdn_short_conv(x, A, A, I, A, A, A, stride, T, R, C, W, dtype, wdtype, 1, 1, nullptr);
}
static int conv_bwd(const void* x, long long stride, int T, int R, int C, int W, void* ws, size_t bytes) {
  return gdn_short_conv_bwd(x, A, A, A, I, A, A, A, A, A, A, stride, stride, T, R, C, W, bf, bf, 1, 1, ws, bytes, nullptr);
}
static int conv_step(const void* x, long long stride, int R, int C, int W) {
  return gdn_short_conv_step(x, A, A, A, A, stride, R, C, W, bf, bf, 1, nullptr);
}
static int scan(const void* x, long long xs, long long dts, long long bs, int T, int R, int H, int P, int G, int N, int dtype, void* ws,
                size_t bytes) {
  return gdn_ssm_scan(x, A, A, A, A, A, A, I, F, A, F, xs, dts, bs, bs, T, R, H, P, G, N, dtype, bf, f32, 1, ws, bytes, nullptr);
}
static int scan_bwd(const void* x, long long xs, long long dts, long long bs, int T, int R, int H, int P, int G, int N, void* ws,
                    size_t bytes) {
  return gdn_ssm_scan_bwd(x, A, A, A, A, A, A, A, I, F, F, A, A, A, A, A, A, A, F, xs, dts, bs, bs, xs, xs, bs, bs, T, R, H, P, G, N, bf,
                          bf, f32, 1, ws, bytes, nullptr);
}
static int step(const void* x, long long xs, long long dts, long long bs, int R, int H, int P, int G, int N) {
  return gdn_ssm_step(x, A, A, A, A, A, A, F, A, xs, dts, bs, bs, R, H, P, G, N, bf, bf, f32, nullptr);
}

int main() {
  expect("norm dtype", norm(A, 1e-6f, 256, 4, 256, 9, bf), GDN_ERR_DTYPE);
  expect("norm weights", norm(A, 1e-6f, 256, 4, 256, f32, bf), GDN_ERR_UNSUPPORTED);
  expect("norm rows", norm(A, 1e-6f, 256, INT_MAX, 256, bf, bf), GDN_ERR_SHAPE);
  expect("norm columns", norm(A, 1e-6f, LLONG_MAX, 4, INT_MAX, bf, bf), GDN_ERR_UNSUPPORTED);
  expect("norm eps", norm(A, NAN, 256, 4, 256, bf, bf), GDN_ERR_SHAPE);
  expect("norm stride", norm(A, 0.f, LLONG_MIN, 4, 256, bf, bf), GDN_ERR_SHAPE);
  expect("norm null", norm(nullptr, 0.f, 256, 4, 256, bf, bf), GDN_ERR_NULL);
  expect("norm align", norm(U, 0.f, 256, 4, 256, bf, bf), GDN_ERR_ALIGN);
  expect("norm nothing", norm(nullptr, 0.f, 256, 0, 256, bf, bf), GDN_OK);
  expect("quant format", quant(A, 256, 4, 256, 128, 5), GDN_ERR_DTYPE);
  expect("quant block", quant(A, 256, 4, 256, INT_MIN, GDN_CACHE_I8), GDN_ERR_SHAPE);
  expect("quant blocks", quant(A, 256, 4, 256, INT_MAX, GDN_CACHE_I8), GDN_ERR_UNSUPPORTED);
  expect("quant null", quant(nullptr, 256, 4, 256, 0, GDN_CACHE_E4M3), GDN_ERR_NULL);
  expect("norm bwd rows", norm_bwd(A, 256, INT_MIN, 256, A, 0), GDN_ERR_SHAPE);
  expect("norm bwd workspace", norm_bwd(A, 256, 40, 256, A, 16), GDN_ERR_WORKSPACE);
  expect("norm bwd align", norm_bwd(A, 256, 40, 256, U, 1 << 30), GDN_ERR_ALIGN);
  for (int T : {INT_MIN, -1, 0, 1, 1000, (1 << 24) - 1, 1 << 24, INT_MAX})
    for (int C : {-8, 0, 8, 4096, 16384, INT_MAX})
      for (int d : {bf, f32, 9}) (void)gdn_rms_norm_bwd_workspace_bytes(T, C, d);

  expect("conv dtype", conv(A, 64, 4, 2, 64, 4, bf, 9), GDN_ERR_DTYPE);
  expect("conv rows", conv(A, 64, INT_MAX, 2, 64, 4, bf, bf), GDN_ERR_SHAPE);
  expect("conv sequences", conv(A, 64, 4, INT_MAX, 64, 4, bf, bf), GDN_ERR_SHAPE);
  expect("conv values", conv(A, 65536, (1 << 28) - 1, 2, 65536, 4, bf, bf), GDN_ERR_SHAPE);
  expect("conv channels", conv(A, INT_MAX, 1, 0, INT_MAX, 4, bf, bf), GDN_ERR_UNSUPPORTED);
  expect("conv taps", conv(A, 64, 4, 2, 64, INT_MAX, bf, bf), GDN_ERR_UNSUPPORTED);
  expect("conv stride", conv(A, LLONG_MAX, 4, 2, 64, 4, bf, bf), GDN_ERR_SHAPE);
  expect("conv null", conv(nullptr, 64, 4, 2, 64, 4, bf, bf), GDN_ERR_NULL);
  expect("conv align", conv(U, 64, 4, 2, 64, 4, bf, bf), GDN_ERR_ALIGN);
  expect("conv nothing", conv(nullptr, 64, 0, 0, 64, 4, bf, bf), GDN_OK);
  expect("conv bwd workspace", conv_bwd(A, 64, 400, 2, 64, 4, A, 16), GDN_ERR_WORKSPACE);
  expect("conv bwd stride", conv_bwd(A, 60, 400, 2, 64, 4, A, 16), GDN_ERR_SHAPE);
  expect("conv step sequences", conv_step(A, 64, INT_MIN, 64, 4), GDN_ERR_SHAPE);
  expect("conv step nothing", conv_step(nullptr, 64, 0, 64, 4), GDN_OK);
  for (int T : {-1, 0, 1, 1000, 1 << 20, (1 << 28) - 1, INT_MAX})
    for (int C : {-8, 0, 8, 4096, 65536, INT_MAX})
      for (int W : {0, 2, 4, INT_MAX}) (void)gdn_short_conv_bwd_workspace_bytes(T, C, W);

  expect("scan dtype", scan(A, 256, 4, 128, 90, 2, 4, 64, 2, 64, 9, A, 0), GDN_ERR_DTYPE);
  expect("scan f32", scan(A, 256, 4, 128, 90, 2, 4, 64, 2, 64, f32, A, 0), GDN_ERR_UNSUPPORTED);
  expect("scan rows", scan(A, 256, 4, 128, INT_MAX, 2, 4, 64, 2, 64, bf, A, 0), GDN_ERR_SHAPE);
  expect("scan heads", scan(A, LLONG_MAX, 4, 128, 90, 2, INT_MAX, 64, 1, 64, bf, A, 0), GDN_ERR_SHAPE);
  expect("scan groups", scan(A, 256, 4, 128, 90, 2, 4, 64, INT_MAX, 64, bf, A, 0), GDN_ERR_SHAPE);
  expect("scan states", scan(A, 512, 8, 128, 90, (1 << 20) - 1, 8, 64, 2, 64, bf, A, 0), GDN_ERR_SHAPE);
  expect("scan size", scan(A, 256, 4, 128, 90, 2, 4, INT_MAX, 2, 64, bf, A, 0), GDN_ERR_UNSUPPORTED);
  expect("scan stride", scan(A, 1LL << 24, 4, 128, 90, 2, 4, 64, 2, 64, bf, A, 0), GDN_ERR_SHAPE);
  expect("scan stride of dt", scan(A, 256, LLONG_MIN, 128, 90, 2, 4, 64, 2, 64, bf, A, 0), GDN_ERR_SHAPE);
  expect("scan null", scan(nullptr, 256, 4, 128, 90, 2, 4, 64, 2, 64, bf, A, 0), GDN_ERR_NULL);
  expect("scan align", scan(U, 256, 4, 128, 90, 2, 4, 64, 2, 64, bf, A, 0), GDN_ERR_ALIGN);
  expect("scan workspace", scan(A, 256, 4, 128, 900, 2, 4, 64, 2, 64, bf, A, 16), GDN_ERR_WORKSPACE);
  expect("scan bwd stride", scan_bwd(A, 256, 4, 1LL << 24, 90, 2, 4, 64, 2, 64, A, 0), GDN_ERR_SHAPE);
  expect("scan bwd workspace", scan_bwd(A, 256, 4, 128, 90, 2, 4, 64, 2, 64, A, 16), GDN_ERR_WORKSPACE);
  expect("step sequences", step(A, 256, 4, 128, INT_MAX, 4, 64, 2, 64), GDN_ERR_SHAPE);
  expect("step null", step(nullptr, 256, 4, 128, 3, 4, 64, 2, 64), GDN_ERR_NULL);
  expect("step nothing", step(nullptr, 256, 4, 128, 0, 4, 64, 2, 64), GDN_OK);
  for (int T : {-1, 0, 1, 65, 4096, 1 << 20, (1 << 26) - 1, INT_MAX})
    for (int R : {-1, 0, 1, 4095, (1 << 20) - 1, INT_MAX})
      for (int H : {-1, 0, 1, 24, 70, 256, 4097, (1 << 16) - 1, INT_MAX})
        for (int G : {1, 2, 5, 256, (1 << 16) - 1})
          for (int P : {64, 128, INT_MAX}) {
            (void)gdn_ssm_scan_workspace_bytes(T, H, P, G, 128);
            (void)gdn_ssm_scan_bwd_workspace_bytes(T, R, H, P, G, 128);
          }

  if (failures) {
    std::fprintf(stderr, "%d checks failed\n", failures);
    return 1;
  }
  std::printf("recurrent block abi driver: all checks passed\n");
  return 0;
}
