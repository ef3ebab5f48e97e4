// ssm_step.hip -- one token for each of R sequences of the selective state space
// scan: S <- 2^g S + d B x^T, y = S^T C + D x, in place on S [R, H, N, P] float32.
//
// Bound by memory: a state is read once and written once, in 16-byte pieces that do
// not stay in the caches.  A workgroup takes a strip of 64 columns; a thread four of
// them in N / 16 consecutive rows, so that its parts of B and C are one load each.
// 256 sequences, 24 heads of 64, N = 128: 64.5 us, 6.3 TB/s.
#include "gdn_scan.hpp"

namespace gdn {
namespace {

using namespace scan;
typedef float f32x4v __attribute__((ext_vector_type(4)));

template <int N>
__global__ __launch_bounds__(256) void step_kernel(const void* __restrict__ x, const void* __restrict__ dt,
                                                   const void* __restrict__ a, const void* __restrict__ B,
                                                   const void* __restrict__ C, const void* __restrict__ D,
                                                   const void* __restrict__ bias, float* __restrict__ S,
                                                   void* __restrict__ out, long long xs, long long dts, long long bs,
                                                   long long cs, int H, int P, int G, bool dt_f32, bool p_f32) {
  constexpr int M = N / 16;
  __shared__ float part[4][64];
  const int t = threadIdx.x, cg = t % 16, rg = t / 16, spp = P / 64;
  const int r = blockIdx.x / (H * spp), strip = blockIdx.x % (H * spp), head = strip / spp, group = head / (H / G);
  const int col = (strip % spp) * 64 + 4 * cg;
  float* s = S + (((long long)r * H + head) * N + rg * M) * P + col;
  f32x4v v[M];
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4v*>(s + (long long)m * P));
  float b[M], c[M];
  params<M>(B, false, (long long)r * bs + group * N + rg * M, b);
  params<M>(C, false, (long long)r * cs + group * N + rg * M, c);
  float xv[4];
  params<4>(x, false, (long long)r * xs + head * P + col, xv);
  const float z = dt_at(dt, dt_f32, (long long)r * dts + head) + (bias ? param(bias, p_f32, head) : 0.f);
  const float delta = softplus(z), keep = exp2_(log2_keep(param(a, p_f32, head), delta));
  f32x4v y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const float db = delta * b[m];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[m][e] = __builtin_fmaf(db, xv[e], v[m][e] * keep);
      y[e] = __builtin_fmaf(c[m], v[m][e], y[e]);
    }
    __builtin_nontemporal_store(v[m], reinterpret_cast<f32x4v*>(s + (long long)m * P));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] += __shfl_xor(y[e], 16);
    y[e] += __shfl_xor(y[e], 32);
  }
  if (t % 64 < 16)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[t / 64][4 * cg + e] = y[e];
  __syncthreads();
  if (t < 64) {
    const long long at = ((long long)r * H + head) * P + (strip % spp) * 64 + t;
    const float xt = (float)static_cast<const __bf16*>(x)[(long long)r * xs + head * P + (strip % spp) * 64 + t];
    const float sum = part[0][t] + part[1][t] + part[2][t] + part[3][t];
    static_cast<__bf16*>(out)[at] = (__bf16)(D ? __builtin_fmaf(param(D, p_f32, head), xt, sum) : sum);
  }
}

}  // namespace

hipError_t launch_ssm_step(const ScanStepArgs& a) {
  const ScanShape& n = a.n;
  auto go = [&](auto nn) {
    hipLaunchKernelGGL((step_kernel<decltype(nn)::value>), dim3(n.R * n.H * (n.P / 64)), dim3(256), 0,
                       static_cast<hipStream_t>(a.stream), a.x, a.dt, a.a, a.B, a.C, a.D, a.bias, a.S, a.out, a.xs, a.dts, a.bs,
                       a.cs, n.H, n.P, n.G, n.dt_f32, n.p_f32);
    return hipGetLastError();
  };
  return n.N == 64 ? go(pipe::ic<64>{}) : go(pipe::ic<128>{});
}

}  // namespace gdn
