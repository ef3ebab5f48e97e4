// short_conv.hip -- depthwise causal convolution of W = 2 to 4 taps over packed
// sequences, with SiLU, a carried state, its gradients and its single-token step.
//
// With z the inputs of a sequence behind the W - 1 rows of its state (zeros
// without one), p_t = b + sum_j w_j z_{t + j} (z_{t + W - 1} is x_t) and
// y = silu(p) or p.  The state afterwards is the last W - 1 rows of z.
// Gradients, with q_t = g_t silu'(p_t):
//
//   gz_s = sum_j w_j q_{s - j},   gw_j = sum_t q_t z_{t + j},   gb = sum_t q_t.
//
// Bound by memory.  A thread takes four channels and walks down a run of rows with the
// taps' rows in registers, so that each row is read once but for W - 1 rows ahead of a
// run (and, for the gradients, behind it); a wave's rows are 256 consecutive channels.
// Which rows are whose is looked up once per workgroup, while rows are on their way.
// All arithmetic is float32.  In the gradients' loop, of 1660 vector instructions for 24
// values a lane, 450 move rows along, 190 ask whose a row is, 48 are transcendental.
#include "gdn_block.hpp"
#include "gdn_rows.hpp"

namespace gdn {
namespace {

using namespace rows;
using pipe::ic;

// The taps and the bias of a thread's channels.
template <bool F32, int W, int PE = kPiece<F32>> struct Taps {
  typedef PieceOf<F32, PE> Piece;
  float w[PE * W], b[PE];
  __device__ __forceinline__ void load(const void* weight, const void* bias, bool w_f32, int p) {
    params<PE * W>(weight, w_f32, (long long)p * PE * W, w);
#pragma unroll
    for (int e = 0; e < PE; ++e) b[e] = 0.f;
    if (bias) params<PE>(bias, w_f32, (long long)p * PE, b);
  }
  // b + sum_j w_j z_j
  __device__ __forceinline__ void sum(const typename Piece::Word (&z)[W], float (&p)[PE]) const {
#pragma unroll
    for (int e = 0; e < PE; ++e) p[e] = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float f[PE];
      Piece::unpack(z[j], f);
#pragma unroll
      for (int e = 0; e < PE; ++e) p[e] = __builtin_fmaf(w[e * W + j], f[e], p[e]);
    }
  }
};

// Row `back` rows before the first of sequence s, from its state; zeros without one.
template <bool F32, int W, int PE = kPiece<F32>>
__device__ __forceinline__ typename PieceOf<F32, PE>::Word before(const void* state, int s, int back, int C, int p) {
  if (!state) return PieceOf<F32, PE>::zero();
  return PieceOf<F32, PE>::get(state, ((long long)s * (W - 1) + W - 1 - back) * C, p);
}

// Channels to a thread that walks down rows: with eight, taps and rows (and the
// gradients' shares) left half as many waves to a SIMD.  8 x 2048 rows of 2304 in bf16:
// 39 us for 42, 3.9 TB/s.
constexpr int kRunPiece = 4;

// -------------------------------------------------------------------- forward
// A workgroup: 64 pieces of the channels, four runs of L rows.  The workgroups
// behind the last run write the states, one sequence each.
template <bool F32, int W, int L>
__global__ __launch_bounds__(256) void conv_kernel(const void* __restrict__ x, const void* __restrict__ weight,
                                                   const void* __restrict__ bias, const int* __restrict__ cu,
                                                   const void* __restrict__ state, void* __restrict__ out,
                                                   void* __restrict__ state_final, long long xs, int T, int R, int C,
                                                   bool w_f32, bool silu_on, bool zero_rest, int runs) {
  constexpr int PE = kRunPiece, NR = 4 * L;
  typedef PieceOf<F32, PE> Piece;
  typedef typename Piece::Word Word;
  __shared__ int window[kWindow], seq[NR], beg[NR], end[NR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int p = blockIdx.y * 64 + lane, np = C / PE;

  if ((int)blockIdx.x >= runs) {  // states
    const int s = blockIdx.x - runs;
    const Span sp = span_of(cu, T, s);
    if (p < np && wave < W - 1) {
      const int row = sp.end - (W - 1) + wave;
      const Word z = row >= sp.beg ? Piece::get(x, (long long)row * xs, p) : before<F32, W, PE>(state, s, sp.beg - row, C, p);
      Piece::put(state_final, ((long long)s * (W - 1) + wave) * C, p, z);
    }
    return;
  }

  // the rows are on their way while it is found out whose they are
  const int r0 = blockIdx.x * NR, first = r0 + wave * L;
  Word rows_in[L + W - 1];
#pragma unroll
  for (int i = 0; i < L + W - 1; ++i) {
    const int row = first + i - (W - 1);
    rows_in[i] = Piece::zero();
    if (row >= 0 && row < T && p < np) rows_in[i] = Piece::get(x, (long long)row * xs, p);
  }
  find_seqs<NR, 256>(cu, R, T, r0, window, seq, beg, end);
  if (p >= np) return;
  Taps<F32, W, PE> taps;
  taps.load(weight, bias, w_f32, p);
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int row = first + i;
    if (row >= T) break;
    const int b = __builtin_amdgcn_readfirstlane(beg[wave * L + i]);
    if (b < 0) {
      if (zero_rest) Piece::put(out, (long long)row * C, p, Piece::zero());
      continue;
    }
    Word z[W];
#pragma unroll
    for (int j = 0; j < W; ++j) z[j] = rows_in[i + j];
    if (row - b < W - 1) {
      const int s = __builtin_amdgcn_readfirstlane(seq[wave * L + i]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        if (row - (W - 1) + j < b) z[j] = before<F32, W, PE>(state, s, b - (row - (W - 1) + j), C, p);
    }
    float y[PE];
    taps.sum(z, y);
    if (silu_on) {
#pragma unroll
      for (int e = 0; e < PE; ++e) y[e] = silu(y[e]);
    }
    Piece::put(out, (long long)row * C, p, Piece::pack(y));
  }
}

// ------------------------------------------------------------------ gradients
// q of row t, from the rows z that its taps see.
constexpr int kMostRun = 64;
template <bool F32, int W>
__device__ __forceinline__ void slope(const Taps<F32, W, kRunPiece>& taps, const typename PieceOf<F32, kRunPiece>::Word (&z)[W],
                                      const typename PieceOf<F32, kRunPiece>::Word& g, bool silu_on, float (&q)[kRunPiece]) {
  PieceOf<F32, kRunPiece>::unpack(g, q);
  if (!silu_on) return;
  float p[kRunPiece];
  taps.sum(z, p);
#pragma unroll
  for (int e = 0; e < kRunPiece; ++e) q[e] *= silu_slope(p[e]);
}

// A workgroup: 64 pieces of the channels, four runs of L rows, one after the
// other's in each wave; shares of gw and gb are added over the waves through LDS
// and written to ws [runs][W + 1][C].  The workgroups behind the last run take the
// gradients of the states, one sequence each.
template <bool F32, int W>
__global__ __launch_bounds__(256) void conv_bwd_kernel(const void* __restrict__ x, const void* __restrict__ weight,
                                                       const void* __restrict__ bias, const void* __restrict__ grad_out,
                                                       const int* __restrict__ cu, const void* __restrict__ state,
                                                       const void* __restrict__ grad_state_final,
                                                       void* __restrict__ grad_x, void* __restrict__ grad_state,
                                                       float* __restrict__ ws, long long xs, long long gs, int T, int R,
                                                       int C, bool w_f32, bool silu_on, bool zero_rest, int runs, int L) {
  constexpr int PE = kRunPiece, M = 4 * kMostRun + W - 1;
  typedef PieceOf<F32, PE> Piece;
  typedef typename Piece::Word Word;
  __shared__ int window[kWindow], seq[M], beg[M], end[M];
  __shared__ float part[4][64 * PE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int p = blockIdx.y * 64 + lane, np = C / PE;
  const bool here = p < np;
  const int pc = here ? p : np - 1;  // lanes behind the last channel read it and write nothing

  if ((int)blockIdx.x >= runs) {  // states
    const int s = blockIdx.x - runs;
    if (!here || wave) return;
    const Span sp = span_of(cu, T, s);
    const int n = sp.end - sp.beg;
    Taps<F32, W, PE> taps;
    taps.load(weight, bias, w_f32, p);
    float acc[W - 1][PE];
#pragma unroll
    for (int m = 0; m < W - 1; ++m) {
#pragma unroll
      for (int e = 0; e < PE; ++e) acc[m][e] = 0.f;
      // row m of the state is row m - n of the state afterwards, where the sequence is that short
      if (grad_state_final && m >= n) Piece::unpack(Piece::get(grad_state_final, ((long long)s * (W - 1) + m - n) * C, p), acc[m]);
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
      if (t >= n) break;
      Word z[W];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int back = W - 1 - t - j;
        z[j] = back > 0 ? before<F32, W, PE>(state, s, back, C, p) : Piece::get(x, (long long)(sp.beg - back) * xs, p);
      }
      float q[PE];
      slope<F32, W>(taps, z, Piece::get(grad_out, (long long)(sp.beg + t) * gs, p), silu_on, q);
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        if (t + j < W - 1)
#pragma unroll
          for (int e = 0; e < PE; ++e) acc[t + j][e] = __builtin_fmaf(taps.w[e * W + j], q[e], acc[t + j][e]);
    }
#pragma unroll
    for (int m = 0; m < W - 1; ++m) Piece::put(grad_state, ((long long)s * (W - 1) + m) * C, p, Piece::pack(acc[m]));
    return;
  }

  const int r0 = blockIdx.x * 4 * L;
  find_seqs<M, 256>(cu, R, T, r0, window, seq, beg, end);
  Taps<F32, W, PE> taps;
  taps.load(weight, bias, w_f32, pc);
  const int first = wave * L;  // of r0
  float gw[W][PE], gb[PE];
#pragma unroll
  for (int e = 0; e < PE; ++e) {
    gb[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) gw[j][e] = 0.f;
  }
  auto row_of = [&](const void* base, long long stride, int i) {
    const int row = r0 + i;
    return row >= 0 && row < T ? Piece::get(base, (long long)row * stride, pc) : Piece::zero();
  };
  // zs: the rows t - W + 1 .. t;  qs: q of rows t - W + 1 .. t, whose first is s
  Word zs[W];
  float qs[W][PE];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    zs[j + 1] = row_of(x, xs, first + j - (W - 1));
#pragma unroll
    for (int e = 0; e < PE; ++e) qs[j + 1][e] = 0.f;
  }
  constexpr int U = 6;  // rows whose loads are issued together: 72 us (see bwd_run) for 75 with four, 83 with eight
  for (int i0 = 0; i0 < L + W - 1; i0 += U) {
    Word xn[U], gn[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      xn[u] = gn[u] = Piece::zero();
      if (i0 + u < L + W - 1) {
        xn[u] = row_of(x, xs, first + i0 + u);
        gn[u] = row_of(grad_out, gs, first + i0 + u);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;  // of the wave's rows; the last W - 1 are the next wave's, for their q alone
      if (i >= L + W - 1) break;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        zs[j] = zs[j + 1];
#pragma unroll
        for (int e = 0; e < PE; ++e) qs[j][e] = qs[j + 1][e];
      }
      zs[W - 1] = xn[u];
      const int row = r0 + first + i;
      const int b = __builtin_amdgcn_readfirstlane(beg[first + i]);
      if (b < 0) {
#pragma unroll
        for (int e = 0; e < PE; ++e) qs[W - 1][e] = 0.f;
      } else {
        Word z[W];
#pragma unroll
        for (int j = 0; j < W; ++j) z[j] = zs[j];
        if (row - b < W - 1) {
          const int s = __builtin_amdgcn_readfirstlane(seq[first + i]);
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
            if (row - (W - 1) + j < b) z[j] = before<F32, W, PE>(state, s, b - (row - (W - 1) + j), C, pc);
        }
        slope<F32, W>(taps, z, gn[u], silu_on, qs[W - 1]);
        if (i < L) {
#pragma unroll
          for (int j = 0; j < W; ++j) {
            float f[PE];
            Piece::unpack(z[j], f);
#pragma unroll
            for (int e = 0; e < PE; ++e) gw[j][e] = __builtin_fmaf(qs[W - 1][e], f[e], gw[j][e]);
          }
#pragma unroll
          for (int e = 0; e < PE; ++e) gb[e] += qs[W - 1][e];
        }
      }
      // row s = i - (W - 1) has all of the q that it gives to
      const int is = i - (W - 1), s_row = r0 + first + is;
      if (is < 0 || s_row >= T) continue;
      const int sb = __builtin_amdgcn_readfirstlane(beg[first + is]);
      if (sb < 0) {
        if (zero_rest && here) Piece::put(grad_x, (long long)s_row * C, p, Piece::zero());
        continue;
      }
      const int se = __builtin_amdgcn_readfirstlane(end[first + is]);
      float o[PE];
#pragma unroll
      for (int e = 0; e < PE; ++e) o[e] = 0.f;
      if (grad_state_final && se - s_row <= W - 1) {
        const int s = __builtin_amdgcn_readfirstlane(seq[first + is]);
        Piece::unpack(Piece::get(grad_state_final, ((long long)s * (W - 1) + W - 1 - (se - s_row)) * C, pc), o);
      }
#pragma unroll
      for (int k = 0; k < W; ++k)
        if (s_row + k < se)
#pragma unroll
          for (int e = 0; e < PE; ++e) o[e] = __builtin_fmaf(taps.w[e * W + W - 1 - k], qs[k][e], o[e]);
      if (here) Piece::put(grad_x, (long long)s_row * C, p, Piece::pack(o));
    }
  }
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < PE; ++e) part[wave][lane * PE + e] = j < W ? gw[j < W ? j : 0][e] : gb[e];
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * PE; i += 256) {
      const int col = blockIdx.y * 64 * PE + i;
      if (col < C) ws[((long long)blockIdx.x * (W + 1) + j) * C + col] = part[0][i] + part[1][i] + part[2][i] + part[3][i];
    }
  }
}

// gw [C][W] and gb [C] from n shares: 32 columns of the (W + 1) C to a workgroup.
__global__ __launch_bounds__(1024) void conv_shares_kernel(const float* __restrict__ ws, void* __restrict__ gw,
                                                           void* __restrict__ gb, int n, int C, int W, bool f32) {
  __shared__ float part[32][33];
  const int c = threadIdx.x % 32, r = threadIdx.x / 32, cols = C * (W + 1), col = blockIdx.x * 32 + c;
  float t = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int i = r; i < n; i += 32) t += ws[(long long)i * cols + col];
  }
  part[r][c] = t;
  __syncthreads();
  if (r == 0 && col < cols) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) all += part[i][c];
    const int j = col / C, ch = col % C;
    if (j < W) put_param(gw, f32, (long long)ch * W + j, all);
    else if (gb) put_param(gb, f32, ch, all);
  }
}

// ------------------------------------------------------------ single tokens
template <bool F32, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(const void* __restrict__ x, const void* __restrict__ weight,
                                                        const void* __restrict__ bias, void* __restrict__ state,
                                                        void* __restrict__ out, long long xs, int R, int C, bool w_f32,
                                                        bool silu_on) {
  constexpr int PE = kPiece<F32>;
  const int p = blockIdx.y * 64 + (threadIdx.x & 63), r = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (p >= C / PE || r >= R) return;
  u32x4 z[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) z[j] = piece<F32>(state, ((long long)r * (W - 1) + j) * C, p);
  z[W - 1] = piece<F32>(x, (long long)r * xs, p);
  Taps<F32, W> taps;
  taps.load(weight, bias, w_f32, p);
  float y[PE];
  taps.sum(z, y);
  if (silu_on) {
#pragma unroll
    for (int e = 0; e < PE; ++e) y[e] = silu(y[e]);
  }
  put<F32>(out, (long long)r * C, p, pack<F32>(y));
#pragma unroll
  for (int j = 0; j < W - 1; ++j) put<F32>(state, ((long long)r * (W - 1) + j) * C, p, z[j + 1]);
}

// Calls f with the type and the taps as constants.
template <class F> hipError_t by_form(bool f32, int W, F f) {
  if (f32) {
    if (W == 2) return f(std::true_type{}, ic<2>{});
    if (W == 3) return f(std::true_type{}, ic<3>{});
    return f(std::true_type{}, ic<4>{});
  }
  if (W == 2) return f(std::false_type{}, ic<2>{});
  if (W == 3) return f(std::false_type{}, ic<3>{});
  return f(std::false_type{}, ic<4>{});
}

int column_groups(int C, int piece) { return (C / piece + 63) / 64; }

// Rows to a wave's run in the gradients: as many as let all workgroups, four to a CU,
// run at once (8 x 2048 rows of 2304: 72 us, 3.1 TB/s; with 32 rows, 1152 workgroups, 80),
// between 8 and kMostRun; with more rows than that, 40 (bf16, with 24, 32, 40 and 64 rows:
// 32768 rows of 2304 147, 142, 147 and 157 us, 131072 500, 487, 476 and 475, 16384 of 8192
// 255, 234, 239 and 230).
int bwd_run(int T, int C) {
  const int groups = 1024 / column_groups(C, kRunPiece);
  const int L = groups ? (int)(((long long)T + 4 * groups - 1) / (4 * groups)) : kMostRun + 1;
  return L < 8 ? 8 : L <= kMostRun ? L : 40;
}
int bwd_runs(int T, int C) {
  const int rows = 4 * bwd_run(T, C);
  return (T + rows - 1) / rows;
}

}  // namespace

hipError_t launch_short_conv(const ConvArgs& a) {
  const int cols = column_groups(a.C, kRunPiece);
  return by_form(a.f32, a.W, [&](auto f32, auto w) {
    auto go = [&](auto l) {
      constexpr int rows_wg = 4 * decltype(l)::value;
      const int runs = (a.T + rows_wg - 1) / rows_wg, blocks = runs + (a.state_final ? a.R : 0);
      if (!blocks) return hipSuccess;
      hipLaunchKernelGGL((conv_kernel<decltype(f32)::value, decltype(w)::value, decltype(l)::value>), dim3(blocks, cols),
                         dim3(256), 0, static_cast<hipStream_t>(a.stream), a.x, a.weight, a.bias, a.cu, a.state, a.out,
                         a.state_final, a.xs, a.T, a.R, a.C, a.w_f32, a.silu, a.zero_rest, runs);
      return hipGetLastError();
    };
    // short runs where there are few rows to share out: with two rows and with eight, 64 rows of 1792 in bf16 3.4 and
    // 5.3 us, 1400 5.0 and 6.5, 3000 8.2 and 8.4; beyond that eight read less twice
    return (long long)a.T * cols < 4 * 8 * 512 ? go(ic<2>{}) : go(ic<8>{});
  });
}

size_t short_conv_bwd_workspace_bytes(int T, int C, int W) { return (size_t)bwd_runs(T, C) * (W + 1) * C * sizeof(float); }

hipError_t launch_short_conv_bwd(const ConvBwdArgs& a) {
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  const int cols = column_groups(a.C, kRunPiece), runs = bwd_runs(a.T, a.C), blocks = runs + (a.grad_state ? a.R : 0);
  if (blocks) {
    const hipError_t e = by_form(a.f32, a.W, [&](auto f32, auto w) {
      hipLaunchKernelGGL((conv_bwd_kernel<decltype(f32)::value, decltype(w)::value>), dim3(blocks, cols), dim3(256),
                         0, st, a.x, a.weight, a.bias, a.grad_out, a.cu, a.state, a.grad_state_final, a.grad_x,
                         a.grad_state, a.ws, a.xs, a.gs, a.T, a.R, a.C, a.w_f32, a.silu, a.zero_rest, runs, bwd_run(a.T, a.C));
      return hipGetLastError();
    });
    if (e) return e;
  }
  const int n = a.C * (a.W + 1);
  hipLaunchKernelGGL(conv_shares_kernel, dim3((n + 31) / 32), dim3(1024), 0, st, a.ws, a.grad_weight, a.grad_bias, runs, a.C,
                     a.W, a.w_f32);
  return hipGetLastError();
}

hipError_t launch_short_conv_step(const ConvStepArgs& a) {
  return by_form(a.f32, a.W, [&](auto f32, auto w) {
    hipLaunchKernelGGL((conv_step_kernel<decltype(f32)::value, decltype(w)::value>), dim3((a.R + 3) / 4, column_groups(a.C, a.f32 ? 4 : 8)),
                       dim3(256), 0, static_cast<hipStream_t>(a.stream), a.x, a.weight, a.bias, a.state, a.out, a.xs, a.R,
                       a.C, a.w_f32, a.silu);
    return hipGetLastError();
  });
}

}  // namespace gdn
