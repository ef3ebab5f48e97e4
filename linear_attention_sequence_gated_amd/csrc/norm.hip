// norm.hip -- root-mean-square norm of rows, with the residual's addition, an
// output in 8 bits with scales, and its gradients.
//
//   s = round(x + r) (a number of the rows' type: what the next block reads),
//   y = s w / sqrt(mean(s^2) + eps)
//
// and, for g the gradient of y and h that of s from elsewhere, with
// n = s / sqrt(mean(s^2) + eps):
//
//   gs = (w g - n mean(w g n)) / sqrt(mean(s^2) + eps) + h,   gw = sum over rows of g n.
//
// Bound by memory: every row is read once into registers, reduced there, and
// written once.  A row is taken by one wave where its pieces are at most two to
// a lane (1024 columns of bf16), otherwise by a workgroup (by_width).  All arithmetic
// is float32.  With codes, 9869 rows of 2048 bf16 values with the residual: 24.4 us,
// 5.8 TB/s; 16384 rows of 768 forward in 19 us (5.3 TB/s), their gradients in 18.5,
// and 4 for the sum of the shares; six rows: 2.8 us.
#include "gdn.h"
#include "gdn_block.hpp"
#include "gdn_rows.hpp"

namespace gdn {
namespace {

using namespace rows;

// Sum over the LR lanes that share a row (a wave, or the workgroup's four).
template <int LR> __device__ __forceinline__ float row_sum(float x, float* red) {
  x = wave_sum(x);
  if constexpr (LR > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = red[0] + red[1] + red[2] + red[3];
  }
  return x;
}

constexpr int kSame = -1;

// Codes of a piece: y / scale, rounded to nearest even, of the magnitude that the
// format ends with at most.  NaN stays NaN in e4m3 and is zero in int8, where the
// scale carries it.
template <int FMT, int N> __device__ __forceinline__ void put_codes(void* out, long long at, const float (&y)[N], float inv) {
  unsigned w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    float z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = y[4 * i + e] * inv;
      const float most = FMT == GDN_CACHE_I8 ? 127.f : 448.f;
      z[e] = v != v ? v : fminf(fmaxf(v, -most), most);
    }
    if constexpr (FMT == GDN_CACHE_I8) {
      w[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[i] |= ((unsigned)(z[e] != z[e] ? 0 : (int)rintf(z[e])) & 0xffu) << (8 * e);
    } else {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
      w[i] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], lo, true);
    }
  }
  unsigned* p = reinterpret_cast<unsigned*>(static_cast<char*>(out) + at);
  if constexpr (N == 8) *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
  else *p = w[0];
}

// out and sum may be the rows of x or residual: a lane reads its pieces of a row, and
// all pieces of both, before it writes the same ones.
template <bool F32, int LR, int K, int FMT>
__global__ __launch_bounds__(256) void norm_kernel(const void* x, const void* residual, const void* __restrict__ weight,
                                                   void* out, void* sum, float* __restrict__ scale, long long xs,
                                                   long long rs, float eps, int T, int C, bool w_f32, int block) {
  constexpr int PE = kPiece<F32>;
  __shared__ float red[4];
  const int row = blockIdx.x * (256 / LR) + threadIdx.x / LR, lane = threadIdx.x % LR, np = C / PE;
  if (row >= T) return;  // whole waves, or the whole workgroup

  u32x4 a[K], b[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int p = k * LR + lane;
    a[k] = u32x4{0, 0, 0, 0};
    if (p < np) a[k] = piece<F32>(x, (long long)row * xs, p);
  }
  if (residual) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = k * LR + lane;
      b[k] = u32x4{0, 0, 0, 0};
      if (p < np) b[k] = piece<F32>(residual, (long long)row * rs, p);
    }
  }
  float s[K][PE], sq = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int p = k * LR + lane;
    unpack<F32>(a[k], s[k]);
    if (residual) {
      float r[PE];
      unpack<F32>(b[k], r);
#pragma unroll
      for (int e = 0; e < PE; ++e) s[k][e] += r[e];
      const u32x4 w = pack<F32>(s[k]);
      if (p < np) put<F32>(sum, (long long)row * C, p, w);
      unpack<F32>(w, s[k]);
    }
#pragma unroll
    for (int e = 0; e < PE; ++e) sq = __builtin_fmaf(s[k][e], s[k][e], sq);
  }
  const float var = row_sum<LR>(sq, red) / (float)C + eps;
  const float rstd = 1.f / sqrtf(var);

  float y[K][PE];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int p = k * LR + lane;
    float w[PE];
    if (p < np) params<PE>(weight, w_f32, (long long)p * PE, w);
    else {
#pragma unroll
      for (int e = 0; e < PE; ++e) w[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < PE; ++e) y[k][e] = s[k][e] * rstd * w[e];
  }
  if constexpr (FMT == kSame) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = k * LR + lane;
      if (p < np) put<F32>(out, (long long)row * C, p, pack<F32>(y[k]));
    }
  } else {
    constexpr float kInvMost = 1.f / (FMT == GDN_CACHE_I8 ? 127.f : 448.f);
    constexpr float kSmallest = 0x1p-100f;
    constexpr int LB = 128 / PE;  // lanes to a block of 128 columns
    unsigned m[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      m[k] = 0;
#pragma unroll
      for (int e = 0; e < PE; ++e) m[k] = max(m[k], __builtin_bit_cast(unsigned, y[k][e]) & 0x7fffffffu);
    }
    if (block) {
#pragma unroll
      for (int k = 0; k < K; ++k) m[k] = lanes_max<LB>(m[k]);
    } else {
#pragma unroll
      for (int k = 1; k < K; ++k) m[0] = max(m[0], m[k]);
      m[0] = lanes_max<64>(m[0]);
      if constexpr (LR > 64) {
        __shared__ unsigned most[4];
        if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = m[0];
        __syncthreads();
        m[0] = max(max(most[0], most[1]), max(most[2], most[3]));
      }
#pragma unroll
      for (int k = 1; k < K; ++k) m[k] = m[0];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = k * LR + lane;
      const float top = __builtin_bit_cast(float, m[k]) * kInvMost;
      const float sc = top < kSmallest ? kSmallest : top;  // NaN stays
      if (p < np) put_codes<FMT, PE>(out, (long long)row * C + (long long)p * PE, y[k], 1.f / sc);
      if (block ? p < np && p % LB == 0 : p == 0) scale[block ? (long long)row * (C / 128) + p / LB : row] = sc;
    }
  }
}

// ---------------------------------------------------------------- gradients
// Rows are dealt to the waves (workgroups) in turn; each keeps its share of gw in
// registers over its rows.  The shares are added in a fixed order by a second
// launch, so that a call's results are the same every time.  grad_x may be the rows of
// any of the three that are read.
template <bool F32, int LR, int K>
__global__ __launch_bounds__(256) void norm_bwd_kernel(const void* sum, const void* __restrict__ weight,
                                                       const void* grad_out, const void* grad_sum, void* grad_x,
                                                       float* __restrict__ ws, long long ss, long long gs,
                                                       long long gss, float eps, int T, int C, bool w_f32) {
  constexpr int PE = kPiece<F32>, G = 256 / LR;
  __shared__ float red[4];
  const int lane = threadIdx.x % LR, np = C / PE;
  const int first = blockIdx.x * G + threadIdx.x / LR, step = gridDim.x * G;

  float w[K][PE], gw[K][PE];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int p = k * LR + lane;
#pragma unroll
    for (int e = 0; e < PE; ++e) w[k][e] = gw[k][e] = 0.f;
    if (p < np) params<PE>(weight, w_f32, (long long)p * PE, w[k]);
  }
  for (int row = first; row < T; row += step) {  // the same number of rounds in every lane of a row's group
    u32x4 a[K], b[K], c[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = k * LR + lane;
      a[k] = b[k] = c[k] = u32x4{0, 0, 0, 0};
      if (p < np) {
        a[k] = piece<F32>(sum, (long long)row * ss, p);
        b[k] = piece<F32>(grad_out, (long long)row * gs, p);
        if (grad_sum) c[k] = piece<F32>(grad_sum, (long long)row * gss, p);
      }
    }
    float sq = 0.f, dot = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s[PE], g[PE];
      unpack<F32>(a[k], s);
      unpack<F32>(b[k], g);
#pragma unroll
      for (int e = 0; e < PE; ++e) {
        sq = __builtin_fmaf(s[e], s[e], sq);
        dot = __builtin_fmaf(g[e] * w[k][e], s[e], dot);
      }
    }
    const float rstd = 1.f / sqrtf(row_sum<LR>(sq, red) / (float)C + eps);
    const float along = row_sum<LR>(dot, red) * rstd / (float)C * rstd;  // mean(w g n) / |.|, of s
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = k * LR + lane;
      float s[PE], g[PE], h[PE], o[PE];
      unpack<F32>(a[k], s);
      unpack<F32>(b[k], g);
      unpack<F32>(c[k], h);
#pragma unroll
      for (int e = 0; e < PE; ++e) {
        gw[k][e] = __builtin_fmaf(g[e], s[e] * rstd, gw[k][e]);
        o[e] = __builtin_fmaf(rstd, g[e] * w[k][e] - s[e] * along, h[e]);
      }
      if (p < np) put<F32>(grad_x, (long long)row * C, p, pack<F32>(o));
    }
  }
  if constexpr (G > 1) {
    // the waves' shares through LDS, one piece of each lane at a time
    __shared__ float part[G][64 * PE];
    const int wave = threadIdx.x / 64;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < PE; ++e) part[wave][lane * PE + e] = gw[k][e];
      __syncthreads();
      for (int i = threadIdx.x; i < 64 * PE; i += 256) {
        const int col = k * 64 * PE + i;
        float t = part[0][i];
#pragma unroll
        for (int v = 1; v < G; ++v) t += part[v][i];
        if (col < C) ws[(long long)blockIdx.x * C + col] = t;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = k * LR + lane;
      if (p < np)
#pragma unroll
        for (int e = 0; e < PE; ++e) ws[(long long)blockIdx.x * C + p * PE + e] = gw[k][e];
    }
  }
}

// Sums of n rows of C numbers: 32 columns to a workgroup, 32 threads to a column.
__global__ __launch_bounds__(1024) void shares_kernel(const float* __restrict__ ws, void* __restrict__ out, int n, int C,
                                                      bool f32) {
  __shared__ float part[32][33];
  const int c = threadIdx.x % 32, r = threadIdx.x / 32, col = blockIdx.x * 32 + c;
  float t = 0.f;
  if (col < C) {
#pragma unroll 8
    for (int i = r; i < n; i += 32) t += ws[(long long)i * C + col];
  }
  part[r][c] = t;
  __syncthreads();
  if (r == 0 && col < C) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) all += part[i][c];
    put_param(out, f32, col, all);
  }
}

// Lanes to a row and pieces to a lane that hold C columns: a wave up to two pieces a
// lane, then the workgroup; with few rows, whose time is one row's, from more than one
// piece on.  A wave with four pieces a lane against the workgroup, 2048 columns of bf16:
// 3.5 and 2.5 us for 64 rows, 22.2 and 22.1 for 16384; gradients 40.8 and 37.0.  With
// two, 768 columns: 2.7 and 2.4 us for 6 rows, 3.3 and 3.4 for 2048, 10.4 and 13.6 for
// 16384; gradients 19.5 and 29.7.  Eight float32 pieces a lane leave one wave to a SIMD:
// 4096 rows of 8192 with the residual take 239 us, 2048 of 16384, as many bytes with
// sixteen, 110 (bf16: 40 and 44).
template <bool F32, class F> hipError_t by_width(int pieces, bool few, F f) {
  using pipe::ic;
  if (pieces <= 64) return f(ic<64>{}, ic<1>{});
  if (pieces <= 128 && !few) return f(ic<64>{}, ic<2>{});
  if (pieces <= 256) return f(ic<256>{}, ic<1>{});
  if (pieces <= 512) return f(ic<256>{}, ic<2>{});
  if (pieces <= 1024) return f(ic<256>{}, ic<4>{});
  if constexpr (F32)
    if (pieces > 2048) return f(ic<256>{}, ic<16>{});
  return f(ic<256>{}, ic<8>{});
}

// Workgroups of the gradients, each of which writes a share of C numbers.  With 512, 1024
// and 2048 at most: 16384 rows of 768 in bf16 21.4, 22.2 and 25.8 us, in float32 37.7, 34.5
// and 37.8; one row at a time, 4096 of 4096 in bf16 26.6, 28.6 and 34.9, 1464 of 8192 24.6,
// 30.7 and 39.0 (256: 26.0), 4096 of 8192 in float32 107, 112 and 125.
int bwd_blocks(int T, int C, bool f32) {
  const int group = C / (f32 ? 4 : 8) <= 128 ? 4 : 1;  // rows to a workgroup
  const int most = 1024;
  const int need = (T + group - 1) / group;
  return need < most ? need : most;
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a) {
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  auto run = [&](auto f32, auto fmt) {
    return by_width<decltype(f32)::value>(a.C / kPiece<decltype(f32)::value>, a.T <= 1024, [&](auto lr, auto k) {
      constexpr int rows_wg = 256 / decltype(lr)::value;
      hipLaunchKernelGGL((norm_kernel<decltype(f32)::value, decltype(lr)::value, decltype(k)::value, decltype(fmt)::value>),
                         dim3((a.T + rows_wg - 1) / rows_wg), dim3(256), 0, st, a.x, a.residual, a.weight, a.out, a.sum,
                         a.scale, a.xs, a.rs, a.eps, a.T, a.C, a.w_f32, a.block);
      return hipGetLastError();
    });
  };
  auto typed = [&](auto fmt) { return a.f32 ? run(std::true_type{}, fmt) : run(std::false_type{}, fmt); };
  if (a.fmt == GDN_CACHE_I8) return typed(pipe::ic<GDN_CACHE_I8>{});
  if (a.fmt == GDN_CACHE_E4M3) return typed(pipe::ic<GDN_CACHE_E4M3>{});
  return typed(pipe::ic<kSame>{});
}

size_t rms_norm_bwd_workspace_bytes(int T, int C, bool f32) { return (size_t)bwd_blocks(T, C, f32) * C * sizeof(float); }

hipError_t launch_rms_norm_bwd(const NormBwdArgs& a) {
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  const int blocks = bwd_blocks(a.T, a.C, a.f32);
  if (blocks) {
    auto run = [&](auto f32) {
      return by_width<decltype(f32)::value>(a.C / kPiece<decltype(f32)::value>, false, [&](auto lr, auto k) {
        hipLaunchKernelGGL((norm_bwd_kernel<decltype(f32)::value, decltype(lr)::value, decltype(k)::value>), dim3(blocks),
                           dim3(256), 0, st, a.sum, a.weight, a.grad_out, a.grad_sum, a.grad_x, a.ws, a.ss, a.gs, a.gss,
                           a.eps, a.T, a.C, a.w_f32);
        return hipGetLastError();
      });
    };
    if (const hipError_t e = a.f32 ? run(std::true_type{}) : run(std::false_type{})) return e;
  }
  hipLaunchKernelGGL(shares_kernel, dim3((a.C + 31) / 32), dim3(1024), 0, st, a.ws, a.grad_weight, blocks, a.C, a.w_f32);
  return hipGetLastError();
}

}  // namespace gdn
