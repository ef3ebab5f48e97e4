// Host-only driver for the sanitizer test of the attention layer's entry points:
// arguments that fail validation, the empty calls and workspace sizes up to the
// limits.  No call reaches a kernel.
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
static int* const U = reinterpret_cast<int*>(buf + 4);  // misaligned
static float* const F = reinterpret_cast<float*>(buf);

static int tables(int* seq, int R, int width, int n_free, int bt, int nb, int T) {
  return gdn_block_tables(seq, I, I, I, I, I, I, I, R, width, n_free, bt, nb, T, nullptr);
}
static int append(const void* k, long long stride, int T, int H, int D, int bt, int nb, int dtype, int fmt) {
  return gdn_cache_append(k, A, I, A, A, F, F, stride, stride, T, H, D, bt, nb, dtype, fmt, nullptr);
}
static int decode(const void* q, float scale, long long qs, int R, int Hq, int H, int D, int bt, int nb, int width,
                  int dtype, int fmt, void* ws, size_t bytes) {
  return gdn_attn_decode(q, A, A, F, F, I, I, A, F, scale, qs, R, Hq, H, D, bt, nb, width, dtype, fmt, ws, bytes, nullptr);
}
static int prompt(const void* q, float scale, long long qs, long long ks, int T, int R, int Hq, int H, int D, int dtype) {
  return gdn_attn_prompt(q, A, A, I, A, F, scale, qs, ks, ks, T, R, Hq, H, D, dtype, 0, nullptr);
}
static int bwd(const void* q, float scale, long long qs, long long ks, int T, int R, int Hq, int H, int D, int dtype,
               void* ws, size_t bytes) {
  return gdn_attn_prompt_bwd(q, A, A, A, F, A, I, A, A, A, scale, qs, ks, ks, qs, qs, ks, ks, T, R, Hq, H, D, dtype, 0, ws,
                             bytes, nullptr);
}

int main() {
  expect("tables shape", tables(I, -1, 8, 10, 16, 64, 100), GDN_ERR_SHAPE);
  expect("tables most requests", tables(I, INT_MAX, 8, 10, 16, 64, 100), GDN_ERR_SHAPE);
  expect("tables width", tables(I, 4, INT_MAX, 10, 16, 64, 100), GDN_ERR_SHAPE);
  expect("tables blocks", tables(I, 4, 8, 10, 16, INT_MAX, 100), GDN_ERR_SHAPE);
  expect("tables slots", tables(I, 4, 8, 10, 16, 64, INT_MAX), GDN_ERR_SHAPE);
  expect("tables block size", tables(I, 4, 8, 10, INT_MAX, 0, 100), GDN_ERR_SHAPE);
  expect("tables block of 48", tables(I, 4, 8, 10, 48, 64, 100), GDN_ERR_UNSUPPORTED);
  expect("tables null", tables(nullptr, 4, 8, INT_MAX, 16, 64, 100), GDN_ERR_NULL);
  expect("tables align", tables(U, 4, 8, 10, 16, 64, 100), GDN_ERR_ALIGN);

  expect("append dtype", append(A, 256, 10, 4, 64, 16, 64, 9, GDN_CACHE_I8), GDN_ERR_DTYPE);
  expect("append format", append(A, 256, 10, 4, 64, 16, 64, GDN_BF16, 2), GDN_ERR_DTYPE);
  expect("append f32", append(A, 256, 10, 4, 64, 16, 64, GDN_F32, GDN_CACHE_I8), GDN_ERR_UNSUPPORTED);
  expect("append heads", append(A, 256, 10, INT_MAX, 64, 16, 64, GDN_BF16, GDN_CACHE_I8), GDN_ERR_SHAPE);
  expect("append tokens", append(A, 256, INT_MAX, 4, 64, 16, 64, GDN_BF16, GDN_CACHE_I8), GDN_ERR_SHAPE);
  expect("append stride", append(A, LLONG_MAX, 10, 4, 64, 16, 64, GDN_BF16, GDN_CACHE_I8), GDN_ERR_SHAPE);
  expect("append stride down", append(A, LLONG_MIN, 10, 4, 64, 16, 64, GDN_BF16, GDN_CACHE_I8), GDN_ERR_SHAPE);
  expect("append null", append(nullptr, 256, 10, 4, 64, 16, 64, GDN_BF16, GDN_CACHE_I8), GDN_ERR_NULL);
  expect("append align", append(U, 256, 10, 4, 64, 16, 64, GDN_BF16, GDN_CACHE_I8), GDN_ERR_ALIGN);
  expect("append nothing", append(nullptr, 256, 0, 4, 64, 16, 64, GDN_BF16, GDN_CACHE_E4M3), GDN_OK);

  const int i8 = GDN_CACHE_I8, bf = GDN_BF16;
  expect("decode dtype", decode(A, 1.f, 512, 3, 8, 4, 64, 16, 64, 72, 9, i8, A, 0), GDN_ERR_DTYPE);
  expect("decode format", decode(A, 1.f, 512, 3, 8, 4, 64, 16, 64, 72, bf, -1, A, 0), GDN_ERR_DTYPE);
  expect("decode width", decode(A, 1.f, 512, 3, 8, 4, 64, 128, 64, INT_MAX, bf, i8, A, 0), GDN_ERR_SHAPE);
  expect("decode tokens", decode(A, 1.f, 512, 1, 8, 4, 64, 16, 64, INT_MAX / 16, bf, i8, A, 0), GDN_ERR_SHAPE);
  expect("decode rows", decode(A, 1.f, 512, 1 << 19, 64, 4, 64, 16, 64, 1, bf, i8, A, 0), GDN_ERR_SHAPE);
  expect("decode scale", decode(A, NAN, 512, 3, 8, 4, 64, 16, 64, 72, bf, i8, A, 0), GDN_ERR_SHAPE);
  expect("decode stride", decode(A, 1.f, LLONG_MAX, 3, 8, 4, 64, 16, 64, 72, bf, i8, A, 0), GDN_ERR_SHAPE);
  expect("decode null", decode(nullptr, 1.f, 512, 3, 8, 4, 64, 16, 64, 72, bf, i8, A, 0), GDN_ERR_NULL);
  expect("decode align", decode(U, 1.f, 512, 3, 8, 4, 64, 16, 64, 72, bf, i8, A, 0), GDN_ERR_ALIGN);
  expect("decode workspace", decode(A, 1.f, 512, 3, 8, 4, 64, 16, 64, 72, bf, i8, A, 16), GDN_ERR_WORKSPACE);
  expect("decode nothing", decode(nullptr, 1.f, 512, 0, 8, 4, 64, 16, 64, 72, bf, i8, nullptr, 0), GDN_OK);
  for (int R : {-1, 0, 1, 3, 300, (1 << 20) - 1, INT_MAX})
    for (int H : {-1, 0, 1, 8, (1 << 20) - 1, INT_MAX})
      for (int bt : {0, 16, 128, INT_MAX})
        for (int width : {-1, 0, 1, 70, 100000, (INT_MAX - 4096) / 128, INT_MAX})
          for (int g : {1, 3, 17, INT_MAX}) {
            const long long Hq = (long long)H * g;
            (void)gdn_attn_decode_workspace_bytes(R, Hq > INT_MAX ? INT_MAX : (int)Hq, H, 64, bt, width);
          }

  expect("prompt dtype", prompt(A, 1.f, 512, 256, 100, 3, 8, 4, 64, 9), GDN_ERR_DTYPE);
  expect("prompt f32", prompt(A, 1.f, 512, 256, 100, 3, 8, 4, 64, GDN_F32), GDN_ERR_UNSUPPORTED);
  expect("prompt rows", prompt(A, 1.f, 512, 256, INT_MAX, 3, 8, 4, 64, bf), GDN_ERR_SHAPE);
  expect("prompt sequences", prompt(A, 1.f, 512, 256, 100, INT_MAX, 8, 4, 64, bf), GDN_ERR_SHAPE);
  expect("prompt heads", prompt(A, 1.f, 512, 256, 100, 3, INT_MIN, INT_MIN, 64, bf), GDN_ERR_SHAPE);
  expect("prompt scale", prompt(A, INFINITY, 512, 256, 100, 3, 8, 4, 64, bf), GDN_ERR_SHAPE);
  expect("prompt stride", prompt(A, 1.f, 512, LLONG_MAX, 100, 3, 8, 4, 64, bf), GDN_ERR_SHAPE);
  expect("prompt null", prompt(nullptr, 1.f, 512, 256, 100, 3, 8, 4, 64, bf), GDN_ERR_NULL);
  expect("prompt align", prompt(U, 1.f, 512, 256, 100, 3, 8, 4, 64, bf), GDN_ERR_ALIGN);
  expect("prompt nothing", prompt(nullptr, 1.f, 512, 256, 0, 3, 8, 4, 64, bf), GDN_OK);

  expect("bwd dtype", bwd(A, 1.f, 512, 256, 100, 3, 8, 4, 64, 9, A, 0), GDN_ERR_DTYPE);
  expect("bwd scale", bwd(A, NAN, 512, 256, 100, 3, 8, 4, 64, bf, A, 0), GDN_ERR_SHAPE);
  expect("bwd stride", bwd(A, 1.f, 1LL << 24, 256, 100, 3, 8, 4, 64, bf, A, 0), GDN_ERR_SHAPE);
  expect("bwd null", bwd(nullptr, 1.f, 512, 256, 100, 3, 8, 4, 64, bf, A, 0), GDN_ERR_NULL);
  expect("bwd align", bwd(A, 1.f, 512, 256, 100, 3, 8, 4, 64, bf, U, 1 << 30), GDN_ERR_ALIGN);
  expect("bwd workspace", bwd(A, 1.f, 512, 256, 100, 3, 8, 4, 64, bf, A, 16), GDN_ERR_WORKSPACE);
  expect("bwd nothing", bwd(nullptr, 1.f, 512, 256, 0, 3, 8, 4, 64, bf, nullptr, 0), GDN_OK);
  for (int T : {-1, 0, 1, 31, 1000, 1 << 20, (1 << 28) - 1, INT_MAX})
    for (int H : {-1, 0, 1, 8, (1 << 20) - 1, INT_MAX})
      for (int g : {1, 4, 6, 64})
        for (int D : {0, 64, 128}) {
          const long long Hq = (long long)H * g;
          (void)gdn_attn_prompt_bwd_workspace_bytes(T, Hq > INT_MAX ? INT_MAX : (int)Hq, H, D);
        }

  if (failures) {
    std::fprintf(stderr, "%d checks failed\n", failures);
    return 1;
  }
  std::printf("attention abi driver: all checks passed\n");
  return 0;
}
