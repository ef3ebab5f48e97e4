// ssm_scan.hip -- selective state space scan over packed sequences.
//
// For each head, with d_t = softplus(dt_t + bias), a state S of N x P:
//
//   S_t = 2^(g_t) S_{t-1} + d_t B_t x_t^T,   y_t = S_t^T C_t + D x_t,   g_t = a d_t log2(e).
//
// Rows are taken in pieces of up to 64 of one sequence.  With G_i the sum of g over
// the piece's rows up to i,
//
//   Y = (C B^T o L) X + 2^G C S,   L_ij = 2^(G_i - G_j) d_j for i >= j,
//   S' = 2^(G_n) S + sum_j 2^(G_n - G_j) d_j B_j x_j^T,
//
// all of it products of matrices.  A workgroup walks down a segment of rows with
// the states of NS strips of 64 channels in its accumulators; a wave has 32 columns
// of one.  Segments are cut by rows, whatever the sequences, so that the workgroups
// are alike; where there are several, a first launch finds what each leaves in the
// state that crosses its end, a second one adds these up along the sequences.
//
// Where numbers are rounded: C B^T o L and the state, as it enters the product with
// C, to bf16 (2^-9 of each term); what goes into the state is kept in three bf16
// parts, 2^-25 of each term, since the state is a result and is carried on.
#include "gdn_scan.hpp"

namespace gdn {
namespace {

using namespace scan;
using tile::operand;
using tile::zero16;

constexpr int kStrips = 2;  // strips to a workgroup
constexpr int kThreads = 128 * kStrips, kWaves = 2 * kStrips;
constexpr int kParts = 3;

struct ScanParams {
  const void* x;
  const void* dt;
  const void* a;
  const void* B;
  const void* C;
  const void* D;
  const void* bias;
  const int* cu;
  const float* S0;
  void* out;
  float* S_final;
  float* ws;
  long long xs, dts, bs, cs;
  int T, R, H, P, G, seg, nseg;
  bool dt_f32, p_f32, zero_rest;
};

// The workspace: the states of [segments - 1][strips][N][64], then what each segment
// keeps (see join).
template <int N, bool OUT>
__global__ __launch_bounds__(kThreads) void scan_kernel(ScanParams p) {
  constexpr int NT = N / 32;
  constexpr int kTile = Q * N, kX = Q * 128 * (kStrips / 2);
  constexpr int kBuf = (OUT ? 2 : 1) * kTile + kX;
  __shared__ __attribute__((aligned(1024))) __bf16 buf[2][kBuf];
  __shared__ Steps st_all[kWaves];
  __shared__ int window[kWindow];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5, col = lane & 31;
  Steps& st = st_all[wave];

  const Strips sp = strips(p.H, p.P, p.G, kStrips);
  const int group = blockIdx.x / sp.sets, set = blockIdx.x % sp.sets, seg = blockIdx.y;
  const int in_group = set * kStrips, here = min(kStrips, sp.per_group - in_group);
  const int strip0 = group * sp.per_group + in_group;
  const bool mine = wave / 2 < here;  // otherwise the wave follows the first strip and writes nothing
  const int strip = strip0 + (mine ? wave / 2 : 0);
  const int spp = p.P / 64, head = strip / spp, hcol = (strip % spp) * 64 + (wave & 1) * 32;  // of the head
  const int nstrips = p.H * spp;
  const float a = param(p.a, p.p_f32, head), bias = p.bias ? param(p.bias, p.p_f32, head) : 0.f;

  const Offsets cu = offsets<kThreads>(p.cu, p.R, window);
  const int s0 = seg * p.seg, s1 = min(s0 + p.seg, p.T);
  float* const local = p.ws;
  float* const kept = p.ws + (size_t)(p.nseg - 1) * nstrips * N * 64;
  auto state_at = [&](const float* base, int seq) { return base + (((long long)seq * p.H + head) * N) * p.P + hcol; };
  auto slot = [&](int s) { return local + ((size_t)s * nstrips + strip) * N * 64 + (wave & 1) * 32; };

  f32x16 S[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) S[t] = zero16();
  Walk<false> walk;
  walk.init(cu, p.R, p.T, s0, s1);
  float whole = 0.f;  // log2 of what the segment keeps of a state (not OUT)
  bool fresh = false;
  if constexpr (OUT) {
    // rows of no sequence, and the states of sequences without rows
    const int lead = p.R ? min(max(cu(0), 0), p.T) : p.T, tail = p.R ? min(max(cu(p.R), 0), p.T) : p.T;
    if (p.zero_rest) {
      auto zero = [&](int r0, int r1) {
        for (int i = threadIdx.x; i < (r1 - r0) * here * 8; i += kThreads)
          *reinterpret_cast<u32x4*>(static_cast<__bf16*>(p.out) + (long long)(r0 + i / (here * 8)) * p.H * p.P + strip0 * 64 +
                                    i % (here * 8) * 8) = u32x4{0, 0, 0, 0};
      };
      if (s0 < lead) zero(s0, min(lead, s1));
      if (tail < s1) zero(max(tail, s0), s1);
    }
    if (p.S_final && mine) {
      const int k0 = seg ? cu.below(p.R, s0) : 0, k1 = seg == p.nseg - 1 ? p.R : cu.below(p.R, s1);
      for (int r = k0; r < k1; ++r) {
        const int b = min(max(cu(r), 0), p.T);
        if (min(cu(r + 1), p.T) > b) continue;
        float* dst = p.S_final + (((long long)r * p.H + head) * N) * p.P + hcol;
        const float* src = p.S0 ? state_at(p.S0, r) : nullptr;
        for (int n = half; n < N; n += 2) dst[(long long)n * p.P + col] = src ? src[(long long)n * p.P + col] : 0.f;
      }
    }
    if (seg && walk.goes_on()) load_state<NT>(S, slot(seg - 1), 64);
  } else {
    // only the sequence that crosses the segment's end
    const int r = walk.rend - 1;
    const int b = r >= 0 ? min(max(cu(r), 0), p.T) : p.T, e = r >= 0 ? min(cu(r + 1), p.T) : 0;
    if (e <= s1 || b >= s1) {
      if (threadIdx.x < here) kept[(size_t)seg * nstrips + strip0 + threadIdx.x] = kNone;
      return;
    }
    walk.r = r, walk.beg = b, walk.pos = max(b, s0), walk.end = e;
    fresh = b >= s0;
  }

  // staging: rows of C, B and x
  tile::Stage<N, Q, kWaves> sc, sb;
  tile::Stage<128, Q, kWaves> sx;
  if constexpr (OUT) sc.init(p.cs, wave);
  sb.init(p.bs, wave);
  sx.init(p.xs, wave);
  const __bf16* xg = static_cast<const __bf16*>(p.x) + strip0 * 64;
  const __bf16* bg = static_cast<const __bf16*>(p.B) + group * N;
  const __bf16* cg = static_cast<const __bf16*>(p.C) + group * N;
  auto stage = [&](int b, const Piece& pc) {
    if constexpr (OUT) sc.load(buf[b] + kTile + kX, tile::rows_rsrc(cg, p.cs, pc.row, pc.n, N), wave);
    sb.load(buf[b], tile::rows_rsrc(bg, p.bs, pc.row, pc.n, N), wave);
    sx.load(buf[b] + kTile, tile::rows_rsrc(xg, p.xs, pc.row, pc.n, 64 * here), wave);
  };
  auto raw_dt = [&](const Piece& pc) {
    return lane < pc.n ? dt_at(p.dt, p.dt_f32, (long long)(pc.row + lane) * p.dts + head) + bias : 0.f;
  };
  const int rb = tile::row_base<N>(lane), cb = col_base_state<N>(lane), xb = tile::col_base<128>(lane);
  const float dskip = OUT && p.D ? param(p.D, p.p_f32, head) : 0.f;

  Piece cur, nxt;
  bool more = walk.next(cur);
  float z = 0.f;
  if (more) {
    stage(0, cur);
    z = raw_dt(cur);
  }
  for (int b = 0; more; b ^= 1) {
    tile::staged_barrier();  // this piece's rows are here, and the other buffer is free
    more = walk.next(nxt);
    float z_next = 0.f;
    if (more) {
      stage(b ^ 1, nxt);
      z_next = raw_dt(nxt);
    }
    if (cur.first) {
      if (p.S0) load_state<NT>(S, state_at(p.S0, cur.seq), p.P);
      else {
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] = zero16();
      }
    }
    const float total = steps(st, z, a, lane < cur.n);
    whole += total;
    const __bf16 *Bt = buf[b], *Xt = buf[b] + kTile, *Ct = buf[b] + kTile + kX;
    const int xcol = wave;  // 32-column block of the tile of x
    u32x4 xf[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) xf[k] = tile::col_frag<128>(Xt, xb, 16 * k, xcol);

    if constexpr (OUT) {
      f32x16 y[2] = {zero16(), zero16()}, m[3] = {zero16(), zero16(), zero16()};
#pragma unroll
      for (int ks = 0; ks < N / 16; ++ks) {
        const u32x4 c0 = tile::row_frag<N>(Ct, rb, 0, ks), c1 = tile::row_frag<N>(Ct, rb, 32, ks);
        const u32x4 b0 = tile::row_frag<N>(Bt, rb, 0, ks), b1 = tile::row_frag<N>(Bt, rb, 32, ks);
        const u32x4 s = operand(S[ks / 2], ks % 2);
        m[0] = tile::mma(b0, c0, m[0]);
        m[1] = tile::mma(b0, c1, m[1]);
        m[2] = tile::mma(b1, c1, m[2]);
        y[0] = tile::mma(s, c0, y[0]);
        y[1] = tile::mma(s, c1, y[1]);
      }
      const float g0 = st.G[col], g1 = st.G[32 + col], g31 = st.G[31];
      const float k0 = exp2_(g0), k1 = exp2_(g1), off = exp2_(g1 - g31);
#pragma unroll
      for (int e = 0; e < 16; ++e) y[0][e] *= k0, y[1][e] *= k1;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 ua = *reinterpret_cast<const float4*>(st.u + 8 * q + 4 * half);
        const float4 ub = *reinterpret_cast<const float4*>(st.u + 32 + 8 * q + 4 * half);
        const float4 v = *reinterpret_cast<const float4*>(st.v + 8 * q + 4 * half);
        const float fa[4] = {ua.x, ua.y, ua.z, ua.w}, fb[4] = {ub.x, ub.y, ub.z, ub.w}, fv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool seen = 8 * q + 4 * half + j <= col;
          m[0][4 * q + j] *= seen ? exp2_(g0 + fa[j]) : 0.f;
          m[2][4 * q + j] *= seen ? exp2_(g1 + fb[j]) : 0.f;
          m[1][4 * q + j] *= off * fv[j];
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        y[0] = tile::mma(xf[k], operand(m[0], k), y[0]);
        y[1] = tile::mma(xf[k], operand(m[1], k), y[1]);
        y[1] = tile::mma(xf[2 + k], operand(m[2], k), y[1]);
      }
      // y tile: columns are rows of the piece, elements channels 8 q + 4 half + j
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const int i = 32 * it + col;
        if (mine && i < cur.n) {
          __bf16* o = static_cast<__bf16*>(p.out) + (long long)(cur.row + i) * p.H * p.P + strip * 64 + (wave & 1) * 32 + 4 * half;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x2 xv = pipe::ld4(Xt + pipe::row_off<128>(i, xcol * 32 + 8 * q + 4 * half));
            u32x2 w;
            w[0] = pipe::cvt2(__builtin_fmaf(dskip, pipe::lo_f(xv[0]), y[it][4 * q]), __builtin_fmaf(dskip, pipe::hi_f(xv[0]), y[it][4 * q + 1]));
            w[1] = pipe::cvt2(__builtin_fmaf(dskip, pipe::lo_f(xv[1]), y[it][4 * q + 2]), __builtin_fmaf(dskip, pipe::hi_f(xv[1]), y[it][4 * q + 3]));
            *reinterpret_cast<u32x2*>(o + 8 * q) = w;
          }
        }
      }
    }

    // the state behind the piece
    const float keep = exp2_(total);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) S[t][e] *= keep;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      Split<kParts> xw;
      xw.make(xf[k], st.w + 16 * k + 4 * half, st.w + 16 * k + 8 + 4 * half);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const u32x4 bt = tile::col_frag<N>(Bt, cb, 16 * k, t);
#pragma unroll
        for (int q = 0; q < kParts; ++q) S[t] = tile::mma(bt, xw.part[q], S[t]);
      }
    }
    if constexpr (OUT) {
      if (cur.last && p.S_final && mine) store_state<NT>(S, const_cast<float*>(state_at(p.S_final, cur.seq)), p.P);
    }
    cur = nxt;
    z = z_next;
  }
  if constexpr (!OUT) {
    if (mine) {
      store_state<NT>(S, slot(seg), 64);
      if (threadIdx.x % 128 == 0) kept[(size_t)seg * nstrips + strip] = fresh ? kFresh : whole;
    }
  }
}

template <int N> __global__ __launch_bounds__(256) void join_kernel(float* ws, int nstrips, int slots) {
  join<N>(ws, nstrips, slots, blockIdx.y, (blockIdx.x * 256 + threadIdx.x) * 4, false);
}

// Rows to a segment: enough workgroups for the CUs, and at least four pieces each.
int segment_rows(int T, int H, int P, int G) {
  const int sets = G * strips(H, P, G, kStrips).sets;
  const int want = sets >= 256 ? 1 : 256 / sets;
  const int pieces = (T + Q - 1) / Q;
  int per = (pieces + want - 1) / want;
  if (per < 4) per = 4;
  return per * Q;
}
int segments(int T, int seg) { return T > seg ? (T + seg - 1) / seg : 1; }

}  // namespace

size_t ssm_scan_workspace_bytes(int T, int H, int P, int G, int N) {
  const size_t slots = segments(T, segment_rows(T, H, P, G)) - 1, nstrips = (size_t)H * (P / 64);
  return slots * nstrips * (N * 64 + 1) * sizeof(float);
}

hipError_t launch_ssm_scan(const ScanArgs& a) {
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  const ScanShape& n = a.n;
  const int seg = segment_rows(n.T, n.H, n.P, n.G), nseg = segments(n.T, seg);
  const int sets = n.G * strips(n.H, n.P, n.G, kStrips).sets, nstrips = n.H * (n.P / 64);
  const ScanParams p = {a.x, a.dt, a.a, a.B, a.C, a.D, a.bias, a.cu, a.S0, a.out, a.S_final, a.ws, a.xs, a.dts, a.bs, a.cs,
                        n.T, n.R, n.H, n.P, n.G, seg, nseg, n.dt_f32, n.p_f32, a.zero_rest};
  auto go = [&](auto nn) {
    constexpr int N = decltype(nn)::value;
    if (nseg > 1) {
      hipLaunchKernelGGL((scan_kernel<N, false>), dim3(sets, nseg - 1), dim3(kThreads), 0, st, p);
      if (const hipError_t e = hipGetLastError()) return e;
      hipLaunchKernelGGL((join_kernel<N>), dim3(N * 64 / 1024, nstrips), dim3(256), 0, st, a.ws, nstrips, nseg - 1);
      if (const hipError_t e = hipGetLastError()) return e;
    }
    hipLaunchKernelGGL((scan_kernel<N, true>), dim3(sets, nseg), dim3(kThreads), 0, st, p);
    return hipGetLastError();
  };
  return n.N == 64 ? go(pipe::ic<64>{}) : go(pipe::ic<128>{});
}

}  // namespace gdn
