// ssm_scan_bwd.hip -- gradients of the selective state space scan.
//
// With the notation of ssm_scan.hip, h = grad_out, Z the gradient of the state behind
// a piece, and, for i >= j of the piece's rows,
//
//   M_ij = (C_i.B_j) L_ij,  W_ij = (h_i.x_j) L_ij,  E_ij = (h_i.x_j) M_ij,
//
//   gx_j = sum_i M_ij h_i + 2^(G_n - G_j) d_j Z^T B_j + D h_j,
//   gC_i = sum_j W_ij B_j + 2^(G_i) S h_i,     gB_j = sum_i W_ij C_i + 2^(G_n - G_j) d_j Z x_j,
//   Z'   = 2^(G_n) Z + sum_i 2^(G_i) C_i h_i^T.
//
// The gradient of the log decay of row t is what crosses it: of the terms from a row
// j < t, or the state before, to a row i >= t, or the state behind,
//
//   gg_t = sum_{i >= t > j} E_ij + sum_{i >= t} R_i + sum_{j < t} Q_j + 2^(G_n) <Z, S>,
//   R_i = C_i . (2^(G_i) S h_i),   Q_j = B_j . (2^(G_n - G_j) d_j Z x_j),
//
// which is added up from terms of their own sign, but for the first sum: that is
// the rows' sums of E less the columns', over rows from t on, of float32 products
// that were never rounded to fewer bits.  The gradient of d_j is a gg_j +
// (sum_{i >= j} E_ij + Q_j) / d_j.
//
// Launches.  (1) Where there are several segments of rows, each one's share in the
// state and in Z at its border, and (2) their sum along the sequences.  (3) The states
// before each piece of 64 rows and Z behind it, walked down and up the segments, to
// memory in bf16: as such they enter every product below.  (4) All gradients, a
// workgroup to 64 rows and a run of strips of one group: gB and gC are summed over the
// strips in its accumulators.  (5) Sums over the runs of strips where there are
// several, and over rows for a, D and the bias.  All sums are made in a fixed order.
#include "gdn_scan.hpp"

namespace gdn {
namespace {

using namespace scan;
using tile::operand;
using tile::zero16;

struct BwdParams {
  const void* x;
  const void* dt;
  const void* a;
  const void* B;
  const void* C;
  const void* D;
  const void* bias;
  const void* go;
  const int* cu;
  const float* S0;
  const float* gSf;
  void* gx;
  void* gdt;
  void* ga;
  void* gB;
  void* gC;
  void* gD;
  void* gbias;
  float* gS0;
  float* seg_ws[2];    // shares of the segments: states, and gradients of states
  __bf16* states[2];   // [pieces][strips][N][64]
  float* shares;       // [gB, gC][runs][T][G][N], where runs > 1
  float* heads;        // [64-row blocks][H][3]: of a, D, bias
  long long xs, dts, bs, cs, gs, gxs, gbs, gcs;
  int T, R, H, P, G, seg, nseg, runs, run_strips;
  bool dt_f32, p_f32, zero_rest;
};

// ---------------------------------------------------------------- states
// A workgroup: one strip, one segment; blockIdx.z: states downwards, or their
// gradients upwards.  A wave has 32 n and 64 channels (N = 64: 32 of them) of
// the transposed state: its lanes the n, its elements the channels, eight in a row to
// a lane, so that a row of the stored state is written in 16-byte pieces.  What the
// rows add is weighted on the side of B (C), in PARTS bf16 parts.
template <int N, bool LOCAL, int PARTS>
__global__ __launch_bounds__(256) void states_kernel(BwdParams p) {
  constexpr int NP = N == 128 ? 2 : 1;  // tiles of 32 channels to a wave
  __shared__ __attribute__((aligned(1024))) __bf16 buf[2][Q * N + Q * 64];
  __shared__ Steps st_all[4];
  __shared__ int window[kWindow];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5, col = lane & 31;
  const int nt = N == 128 ? wave : wave & 1, pt0 = N == 128 ? 0 : wave >> 1;
  Steps& st = st_all[wave];
  const int strip = blockIdx.x, spp = p.P / 64, head = strip / spp, hcol = (strip % spp) * 64, group = head / (p.H / p.G);
  const int nstrips = p.H * spp;
  const bool up = blockIdx.z != 0;
  const int seg = LOCAL && up ? blockIdx.y + 1 : blockIdx.y;
  const float a = param(p.a, p.p_f32, head), bias = p.bias ? param(p.bias, p.p_f32, head) : 0.f;
  const Offsets cu = offsets<256>(p.cu, p.R, window);
  const int s0 = seg * p.seg, s1 = min(s0 + p.seg, p.T);
  float* const shares = p.seg_ws[up];
  float* const kept = shares + (size_t)(p.nseg - 1) * nstrips * N * 64;

  f32x16 S[NP];
#pragma unroll
  for (int t = 0; t < NP; ++t) S[t] = zero16();
  const int n = 32 * nt + col;
  // rows of a state in float32: the lane's n, channels of a wave's tiles
  auto load = [&](const float* src, long long stride) {
#pragma unroll
    for (int t = 0; t < NP; ++t)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float4* q = reinterpret_cast<const float4*>(src + n * stride + 32 * (pt0 + t) + 16 * b + 8 * half);
        const float4 u = q[0], v = q[1];
        S[t][8 * b] = u.x, S[t][8 * b + 1] = u.y, S[t][8 * b + 2] = u.z, S[t][8 * b + 3] = u.w;
        S[t][8 * b + 4] = v.x, S[t][8 * b + 5] = v.y, S[t][8 * b + 6] = v.z, S[t][8 * b + 7] = v.w;
      }
  };
  auto store = [&](float* dst, long long stride) {
#pragma unroll
    for (int t = 0; t < NP; ++t)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float4* q = reinterpret_cast<float4*>(dst + n * stride + 32 * (pt0 + t) + 16 * b + 8 * half);
        q[0] = make_float4(S[t][8 * b], S[t][8 * b + 1], S[t][8 * b + 2], S[t][8 * b + 3]);
        q[1] = make_float4(S[t][8 * b + 4], S[t][8 * b + 5], S[t][8 * b + 6], S[t][8 * b + 7]);
      }
  };
  auto of_seq = [&](long long r) { return ((r * p.H + head) * N) * p.P + hcol; };
  auto slot = [&](int s) { return shares + ((size_t)s * nstrips + strip) * N * 64; };

  Walk<true> down;
  WalkBack back;
  down.init(cu, p.R, p.T, s0, s1);
  back.init(cu, p.R, p.T, s0, s1);
  float whole = 0.f;
  bool fresh = false;
  if constexpr (LOCAL) {
    // only the sequence that crosses the border: the segment's end, or, upwards, its beginning
    bool crosses;
    if (up) {
      const int r = cu.below(p.R, s0) - 1;
      const int b = r >= 0 ? min(max(cu(r), 0), p.T) : p.T, e = r >= 0 ? min(cu(r + 1), p.T) : 0;
      crosses = b < s0 && e > s0;
      back.r = back.rlow = r;
      if (crosses) back.take(s1);
      fresh = e <= s1;
    } else {
      const int r = down.rend - 1;
      const int b = r >= 0 ? min(max(cu(r), 0), p.T) : p.T, e = r >= 0 ? min(cu(r + 1), p.T) : 0;
      crosses = e > s1 && b < s1;
      down.r = r, down.beg = b, down.pos = max(b, s0), down.end = e;
      fresh = b >= s0;
    }
    if (!crosses) {
      if (threadIdx.x == 0) kept[(size_t)blockIdx.y * nstrips + strip] = kNone;
      return;
    }
  } else if (up) {
    if (p.gS0) {  // sequences without rows
      const int k0 = seg ? cu.below(p.R, s0) : 0, k1 = seg == p.nseg - 1 ? p.R : cu.below(p.R, s1);
      for (int r = k0; r < k1; ++r) {
        const int b = min(max(cu(r), 0), p.T);
        if (min(cu(r + 1), p.T) > b) continue;
        for (int i = threadIdx.x; i < N * 64; i += 256) {
          const long long at = of_seq(r) + (long long)(i / 64) * p.P + i % 64;
          p.gS0[at] = p.gSf ? p.gSf[at] : 0.f;
        }
      }
    }
    if (back.r >= back.rlow && back.pos > max(back.beg, s0) && back.end > s1) load(slot(seg), 64);
  } else if (seg && down.goes_on()) {
    load(slot(seg - 1), 64);
  }

  Stage<N, Q, 4> sk;
  Stage<64, Q, 4> sv;
  const __bf16* kg = (up ? static_cast<const __bf16*>(p.C) : static_cast<const __bf16*>(p.B)) + group * N;
  const __bf16* vg = (up ? static_cast<const __bf16*>(p.go) : static_cast<const __bf16*>(p.x)) + strip * 64;
  const long long ks = up ? p.cs : p.bs, vs = up ? p.gs : p.xs;
  sk.init(ks, wave);
  sv.init(vs, wave);
  auto stage = [&](int b, const Piece& pc) {
    sk.load(buf[b], source(kg, ks, pc.row, pc.n, N), wave);
    sv.load(buf[b] + Q * N, source(vg, vs, pc.row, pc.n, 64), wave);
  };
  auto raw_dt = [&](const Piece& pc) {
    return lane < pc.n ? dt_at(p.dt, p.dt_f32, (long long)(pc.row + lane) * p.dts + head) + bias : 0.f;
  };
  auto next = [&](Piece& pc) { return up ? back.next(pc) : down.next(pc); };
  const int kb = tile::col_base<N>(lane), vb = col_base_state<64>(lane);

  Piece cur, nxt;
  bool more = next(cur);
  float z = 0.f;
  if (more) {
    stage(0, cur);
    z = raw_dt(cur);
  }
  for (int b = 0; more; b ^= 1) {
    tile::staged_barrier();
    more = next(nxt);
    float z_next = 0.f;
    if (more) {
      stage(b ^ 1, nxt);
      z_next = raw_dt(nxt);
    }
    if (up ? cur.last : cur.first) {
      const float* src = up ? p.gSf : p.S0;
      if (src) load(src + of_seq(cur.seq), p.P);
      else {
#pragma unroll
        for (int t = 0; t < NP; ++t) S[t] = zero16();
      }
    }
    if constexpr (!LOCAL) {
      __bf16* dst = p.states[up] + (((long long)piece_id(cur) * nstrips + strip) * N + n) * 64 + 32 * pt0 + 8 * half;
#pragma unroll
      for (int t = 0; t < NP; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(dst + 32 * t + 16 * i) = operand(S[t], i);
    }
    const float total = steps(st, z, a, lane < cur.n);
    whole += total;
    if (up) {
      st.w[lane] = exp2_(st.G[lane]);
      pipe::issue_fence();
    }
    const __bf16 *Kt = buf[b], *Vt = buf[b] + Q * N;
    const float keep = exp2_(total);
#pragma unroll
    for (int t = 0; t < NP; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) S[t][e] *= keep;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      Split<PARTS> kw;
      kw.make(tile::col_frag<N>(Kt, kb, 16 * k, nt), st.w + 16 * k + 4 * half, st.w + 16 * k + 8 + 4 * half);
#pragma unroll
      for (int t = 0; t < NP; ++t) {
        const u32x4 v = tile::col_frag<64>(Vt, vb, 16 * k, pt0 + t);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) S[t] = tile::mma(v, kw.part[q], S[t]);
      }
    }
    if constexpr (!LOCAL) {
      if (up && cur.first && p.gS0) store(p.gS0 + of_seq(cur.seq), p.P);
    }
    cur = nxt;
    z = z_next;
  }
  if constexpr (LOCAL) {
    store(slot(blockIdx.y), 64);
    if (threadIdx.x == 0) kept[(size_t)blockIdx.y * nstrips + strip] = fresh ? kFresh : whole;
  }
}

template <int N> __global__ __launch_bounds__(256) void join_both_kernel(float* down, float* up, int nstrips, int slots) {
  const bool back = blockIdx.z != 0;
  join<N>(back ? up : down, nstrips, slots, blockIdx.y, (blockIdx.x * 256 + threadIdx.x) * 4, back);
}

// -------------------------------------------------------------- gradients
// Sums of 16 elements over the 32 lanes of each half: lane l gets that of element l % 16.
__device__ __forceinline__ float column_sums(f32x16 v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1, n = 8; n; d *= 2, n /= 2) {
    const bool odd = lane & d;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float mine = odd ? v[2 * i + 1] : v[2 * i], other = odd ? v[2 * i] : v[2 * i + 1];
      v[i] = mine + __shfl_xor(other, d);
    }
  }
  return v[0] + __shfl_xor(v[0], 16);
}

__device__ __forceinline__ float dot2(unsigned a, unsigned b, float c) {
  return __builtin_fmaf(pipe::lo_f(a), pipe::lo_f(b), __builtin_fmaf(pipe::hi_f(a), pipe::hi_f(b), c));
}

template <int N> struct GradLds {
  __bf16 C[Q * N], B[Q * N];
  struct {
    __bf16 S[N * 64], Z[N * 64], x[Q * 64], h[Q * 64];
  } strip[2];
  __bf16 M[Q * Q], W[Q * Q];  // [i][j]
  Steps st[4];
  float er[Q], er1[32], ec[Q], ec1[32], ed[Q], hx[Q];  // sums of E by rows and columns, its diagonal; h.x
  float R[N / 32][Q], Qs[N / 32][Q], zs[4];
  int window[kWindow];
};

template <int N>
__global__ __launch_bounds__(256) void grad_kernel(BwdParams p) {
  constexpr int NR = N == 128 ? 2 : 1;  // tiles of 32 rows to a wave
  __shared__ __attribute__((aligned(1024))) GradLds<N> L;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5, col = lane & 31;
  const int nt = N == 128 ? wave : wave & 1, rt0 = N == 128 ? 0 : wave >> 1;
  const int group = blockIdx.y / p.runs, run = blockIdx.y % p.runs;
  const int spp = p.P / 64, per_group = p.H / p.G * spp, nstrips = p.H * spp;
  const int strip0 = group * per_group + run * p.run_strips;
  const int strips_here = min(p.run_strips, per_group - run * p.run_strips);
  const int c0 = blockIdx.x * Q, c1 = min(c0 + Q, p.T);
  Steps& st = L.st[wave];
  const Offsets cu = offsets<256>(p.cu, p.R, L.window);

  const bool one_run = p.runs == 1;
  const long long share = (long long)p.T * p.G * N;
  float* const shareB = p.shares + (long long)run * share;
  float* const shareC = shareB + p.runs * share;
  float* const heads = p.heads + (long long)blockIdx.x * p.H * 3;

  {  // rows of no sequence, and the heads' sums
    const int lead = p.R ? min(max(cu(0), 0), p.T) : p.T, tail = p.R ? min(max(cu(p.R), 0), p.T) : p.T;
    auto zero = [&](int r0, int r1) {
      for (int r = r0 + (int)(threadIdx.x / 64); r < r1; r += 4) {
        if (p.zero_rest) {
          for (int i = lane; i < strips_here * 8; i += 64)
            *reinterpret_cast<u32x4*>(static_cast<__bf16*>(p.gx) + r * p.gxs + strip0 * 64 + i * 8) = u32x4{0, 0, 0, 0};
          for (int i = lane; i < strips_here / spp; i += 64) put_param(p.gdt, p.dt_f32, (long long)r * p.H + strip0 / spp + i, 0.f);
        }
        for (int i = lane; i < N; i += 64) {
          const long long at = ((long long)r * p.G + group) * N + i;
          if (!one_run) shareB[at] = shareC[at] = 0.f;
          else if (p.zero_rest) {
            static_cast<__bf16*>(p.gB)[r * p.gbs + group * N + i] = (__bf16)0.f;
            static_cast<__bf16*>(p.gC)[r * p.gcs + group * N + i] = (__bf16)0.f;
          }
        }
      }
    };
    zero(c0, min(lead, c1));
    zero(max(tail, c0), c1);
  }

  Stage<N, Q, 4> sc, sb;
  Stage<64, Q, 4> sx, sh;
  Stage<64, N, 4> ss;
  sc.init(p.cs, wave);
  sb.init(p.bs, wave);
  sx.init(p.xs, wave);
  sh.init(p.gs, wave);
  ss.init(64, wave);
  const int rbn = tile::row_base<N>(lane), rb64 = tile::row_base<64>(lane);
  const int cbn = col_base8<N>(lane), cb64 = col_base8<64>(lane);

  Walk<true> walk;
  walk.init(cu, p.R, p.T, c0, c1);
  Piece pc;
  bool later = false;  // than the first piece of these rows
  for (; walk.next(pc); later = true) {
    __syncthreads();  // the piece before is done with its buffers
    auto stage = [&](int b, int strip) {
      const long long at = ((long long)piece_id(pc) * nstrips + strip) * N * 64;
      ss.load(L.strip[b].S, source(p.states[0] + at, 64, 0, N, 64), wave);
      ss.load(L.strip[b].Z, source(p.states[1] + at, 64, 0, N, 64), wave);
      sx.load(L.strip[b].x, source(static_cast<const __bf16*>(p.x) + strip * 64, p.xs, pc.row, pc.n, 64), wave);
      sh.load(L.strip[b].h, source(static_cast<const __bf16*>(p.go) + strip * 64, p.gs, pc.row, pc.n, 64), wave);
    };
    sc.load(L.C, source(static_cast<const __bf16*>(p.C) + group * N, p.cs, pc.row, pc.n, N), wave);
    sb.load(L.B, source(static_cast<const __bf16*>(p.B) + group * N, p.bs, pc.row, pc.n, N), wave);
    stage(0, strip0);

    f32x16 gB[NR], gC[NR], cb = zero16();
#pragma unroll
    for (int t = 0; t < NR; ++t) gB[t] = gC[t] = zero16();
    // tiles of the triangle: (rows i, rows j) of wave 0, 1, 2: (0, 0), (1, 1), (1, 0)
    const int it = wave == 0 ? 0 : 1, jt = wave == 1 ? 1 : 0;
    // of wave 3's rows, over the strips of a head
    float z = 0.f, a = 0.f, total = 0.f, sum_a = 0.f, sum_q = 0.f, sum_d = 0.f, sum_k = 0.f, sum_hx = 0.f;

    for (int s = 0; s < strips_here; ++s) {
      const int strip = strip0 + s, head = strip / spp, b = s & 1;
      tile::staged_barrier();
      if (s + 1 < strips_here) stage(b ^ 1, strip + 1);
      if (strip % spp == 0) {
        a = param(p.a, p.p_f32, head);
        z = lane < pc.n ? dt_at(p.dt, p.dt_f32, (long long)(pc.row + lane) * p.dts + head) + (p.bias ? param(p.bias, p.p_f32, head) : 0.f) : 0.f;
        total = steps(st, z, a, lane < pc.n);
        sum_a = sum_q = sum_d = sum_k = sum_hx = 0.f;
      }
      const __bf16 *St = L.strip[b].S, *Zt = L.strip[b].Z, *Xt = L.strip[b].x, *Ht = L.strip[b].h;
      if (s == 0 && wave < 3) {
#pragma unroll
        for (int k = 0; k < N / 16; ++k)
          cb = tile::mma(tile::row_frag<N>(L.B, rbn, 32 * jt, k), tile::row_frag<N>(L.C, rbn, 32 * it, k), cb);
      }
      // M, W and the sums of E: tiles with rows j as elements, rows i as lanes
      if (wave < 3) {
        f32x16 w = zero16(), m = cb, e;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w = tile::mma(tile::row_frag<64>(Xt, rb64, 32 * jt, k), tile::row_frag<64>(Ht, rb64, 32 * it, k), w);
        const float gi = st.G[32 * it + col], off = exp2_(gi - st.G[31]);
        float row = 0.f, diag = 0.f, hx = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 f4 = *reinterpret_cast<const float4*>((wave == 2 ? st.v : st.u + 32 * jt) + 8 * q + 4 * half);
          const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 4 * q + j, at = 8 * q + 4 * half + j;
            const float l = wave == 2 ? off * f[j] : at <= col ? exp2_(gi + f[j]) : 0.f;
            m[i] *= l;
            const float x = w[i] * m[i];
            if (wave < 2) {
              if (at == col) diag += x, hx += w[i];
              e[i] = at < col ? x : 0.f;
            } else {
              e[i] = x;
            }
            row += e[i];
            w[i] *= l;
          }
          *reinterpret_cast<u32x2*>(L.M + pipe::row_off<64>(32 * it + col, 32 * jt + 8 * q + 4 * half)) =
              u32x2{pipe::cvt2(m[4 * q], m[4 * q + 1]), pipe::cvt2(m[4 * q + 2], m[4 * q + 3])};
          *reinterpret_cast<u32x2*>(L.W + pipe::row_off<64>(32 * it + col, 32 * jt + 8 * q + 4 * half)) =
              u32x2{pipe::cvt2(w[4 * q], w[4 * q + 1]), pipe::cvt2(w[4 * q + 2], w[4 * q + 3])};
        }
        row = tile::sum_halves(row);
        const float column = column_sums(e);
        const int ej = 8 * ((lane & 15) / 4) + 4 * half + (lane & 3);
        if (wave < 2) {
          diag = tile::sum_halves(diag), hx = tile::sum_halves(hx);
          if (half == 0) L.er[32 * it + col] = row, L.ed[32 * it + col] = diag, L.hx[32 * it + col] = hx;
          if (col < 16) L.ec[32 * jt + ej] = column;
        } else {
          if (half == 0) L.er1[col] = row;
          if (col < 16) L.ec1[ej] = column;
        }
      }
      {  // <Z, S>
        float dot = 0.f;
        const u32x4* s4 = reinterpret_cast<const u32x4*>(St) + threadIdx.x;
        const u32x4* z4 = reinterpret_cast<const u32x4*>(Zt) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < N * 64 / 8 / 256; ++i) {
          const u32x4 u = s4[i * 256], v = z4[i * 256];
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = dot2(u[e], v[e], dot);
        }
        dot = wave_sum(dot);
        if (lane == 0) L.zs[wave] = dot;
      }
      lds_barrier();

      // gC and gB: tiles of n by rows
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        const int rt = rt0 + t, row = 32 * rt + col;
        f32x16 uc = zero16(), ub = zero16();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uc = tile::mma(tile::row_frag<64>(St, rb64, 32 * nt, k), tile::row_frag<64>(Ht, rb64, 32 * rt, k), uc);
          ub = tile::mma(tile::row_frag<64>(Zt, rb64, 32 * nt, k), tile::row_frag<64>(Xt, rb64, 32 * rt, k), ub);
        }
        const float kc = exp2_(st.G[row]), kb = st.w[row];
        float r = 0.f, q = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = pipe::row_off<N>(row, 32 * nt + 8 * i + 4 * half);
          const u32x2 cv = pipe::ld4(L.C + at), bv = pipe::ld4(L.B + at);
          const float cf[4] = {pipe::lo_f(cv[0]), pipe::hi_f(cv[0]), pipe::lo_f(cv[1]), pipe::hi_f(cv[1])};
          const float bf[4] = {pipe::lo_f(bv[0]), pipe::hi_f(bv[0]), pipe::lo_f(bv[1]), pipe::hi_f(bv[1])};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float vc = uc[4 * i + j] * kc, vb = ub[4 * i + j] * kb;
            r = __builtin_fmaf(vc, cf[j], r);
            q = __builtin_fmaf(vb, bf[j], q);
            gC[t][4 * i + j] += vc;
            gB[t][4 * i + j] += vb;
          }
        }
        r = tile::sum_halves(r), q = tile::sum_halves(q);
        if (half == 0) L.R[nt][row] = r, L.Qs[nt][row] = q;
        // gC_i += sum over j <= i;  gB_j += sum over i >= j
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < 2 * rt + 2)
            gC[t] = tile::mma(col_frag8<N>(L.B, cbn, 16 * k, nt), tile::row_frag<64>(L.W, rb64, 32 * rt, k), gC[t]);
          if (k >= 2 * rt)
            gB[t] = tile::mma(col_frag8<N>(L.C, cbn, 16 * k, nt), col_frag8<64>(L.W, cb64, 16 * k, rt), gB[t]);
        }
      }
      {  // gx: a wave's tile of 32 channels by 32 rows
        const int pt = wave & 1, rt = wave >> 1, row = 32 * rt + col;
        f32x16 u = zero16();
#pragma unroll
        for (int k = 0; k < N / 16; ++k)
          u = tile::mma(col_frag8<64>(Zt, cb64, 16 * k, pt), tile::row_frag<N>(L.B, rbn, 32 * rt, k), u);
        const float kb = st.w[row], dskip = p.D ? param(p.D, p.p_f32, head) : 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] *= kb;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k >= 2 * rt) u = tile::mma(col_frag8<64>(Ht, cb64, 16 * k, pt), col_frag8<64>(L.M, cb64, 16 * k, rt), u);
        if (row < pc.n) {
          __bf16* o = static_cast<__bf16*>(p.gx) + (long long)(pc.row + row) * p.gxs + strip * 64 + 32 * pt + 4 * half;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x2 hv = pipe::ld4(Ht + pipe::row_off<64>(row, 32 * pt + 8 * q + 4 * half));
            u32x2 w;
            w[0] = pipe::cvt2(__builtin_fmaf(dskip, pipe::lo_f(hv[0]), u[4 * q]), __builtin_fmaf(dskip, pipe::hi_f(hv[0]), u[4 * q + 1]));
            w[1] = pipe::cvt2(__builtin_fmaf(dskip, pipe::lo_f(hv[1]), u[4 * q + 2]), __builtin_fmaf(dskip, pipe::hi_f(hv[1]), u[4 * q + 3]));
            *reinterpret_cast<u32x2*>(o + 8 * q) = w;
          }
        }
      }
      lds_barrier();
      if (wave == 3) {  // sums by rows, a lane each; the next strip's are written behind the next barrier
        float r = 0.f, q = 0.f;
#pragma unroll
        for (int i = 0; i < N / 32; ++i) r += L.R[i][lane], q += L.Qs[i][lane];
        const float er = L.er[lane] + (lane >= 32 ? L.er1[lane & 31] : 0.f);
        const float ec = L.ec[lane] + (lane < 32 ? L.ec1[lane & 31] : 0.f);
        sum_a += (er - ec) + r;
        sum_q += q;
        sum_d += ec + L.ed[lane] + q;
        sum_k += L.zs[0] + L.zs[1] + L.zs[2] + L.zs[3];
        sum_hx += L.hx[lane];
        if (strip % spp == spp - 1) {
          const float behind = __shfl(pipe::wave_prefix_sum(__shfl(sum_a, 63 - lane)), 63 - lane);
          const float upto = __shfl(pipe::wave_prefix_sum(sum_q), (lane + 63) & 63);
          const float gg = behind + (lane ? upto : 0.f) + exp2_(total) * sum_k;
          const float delta = softplus(z), sig = logistic(z);
          const bool in = lane < pc.n;
          const float gz = in ? (delta > 0.f ? sum_d * (sig / delta) : 0.f) + a * gg * sig : 0.f;
          if (in) put_param(p.gdt, p.dt_f32, (long long)(pc.row + lane) * p.H + head, gz);
          const float ga = wave_sum(in ? gg * delta : 0.f), gD = wave_sum(in ? sum_hx : 0.f), gb = wave_sum(gz);
          if (lane == 0) {
            float* o = heads + head * 3;
            o[0] = later ? o[0] + ga : ga, o[1] = later ? o[1] + gD : gD, o[2] = later ? o[2] + gb : gb;
          }
        }
      }
    }
    // gB and gC: lanes are rows, elements n = 32 nt + 8 q + 4 half + j
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      const int row = 32 * (rt0 + t) + col;
      if (row >= pc.n) continue;
      const long long r = pc.row + row;
      const int n = group * N + 32 * nt + 4 * half;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (one_run) {
          *reinterpret_cast<u32x2*>(static_cast<__bf16*>(p.gB) + r * p.gbs + n + 8 * q) =
              u32x2{pipe::cvt2(gB[t][4 * q], gB[t][4 * q + 1]), pipe::cvt2(gB[t][4 * q + 2], gB[t][4 * q + 3])};
          *reinterpret_cast<u32x2*>(static_cast<__bf16*>(p.gC) + r * p.gcs + n + 8 * q) =
              u32x2{pipe::cvt2(gC[t][4 * q], gC[t][4 * q + 1]), pipe::cvt2(gC[t][4 * q + 2], gC[t][4 * q + 3])};
        } else {
          const long long at = r * p.G * N + n + 8 * q;
          *reinterpret_cast<float4*>(shareB + at) = make_float4(gB[t][4 * q], gB[t][4 * q + 1], gB[t][4 * q + 2], gB[t][4 * q + 3]);
          *reinterpret_cast<float4*>(shareC + at) = make_float4(gC[t][4 * q], gC[t][4 * q + 1], gC[t][4 * q + 2], gC[t][4 * q + 3]);
        }
      }
    }
  }
  if (!later)
    for (int i = threadIdx.x; i < strips_here / spp * 3; i += 256) heads[strip0 / spp * 3 + i] = 0.f;
}

// The first H blocks: a head's sums over the blocks of rows.  Those behind: gB and gC
// from the runs' shares, four values to a thread; rows of no sequence hold zeros there
// and are left out unless they are to be zero.
__global__ __launch_bounds__(256) void sums_kernel(BwdParams p, int blocks, int N) {
  if ((int)blockIdx.x < p.H) {
    if (blockIdx.y) return;
    __shared__ float part[3][4];
    const int head = blockIdx.x;
    float s[3] = {0.f, 0.f, 0.f};
    for (int i = threadIdx.x; i < blocks; i += 256)
#pragma unroll
      for (int k = 0; k < 3; ++k) s[k] += p.heads[((long long)i * p.H + head) * 3 + k];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      s[k] = wave_sum(s[k]);
      if ((threadIdx.x & 63) == 0) part[k][threadIdx.x >> 6] = s[k];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      float t[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) t[k] = part[k][0] + part[k][1] + part[k][2] + part[k][3];
      put_param(p.ga, p.p_f32, head, t[0]);
      if (p.gD) put_param(p.gD, p.p_f32, head, t[1]);
      if (p.gbias) put_param(p.gbias, p.p_f32, head, t[2]);
    }
    return;
  }
  const long long row_n = (long long)p.G * N, all = (long long)p.T * row_n;
  const long long i = ((long long)(blockIdx.x - p.H) * 256 + threadIdx.x) * 4;
  if (i >= all) return;
  const long long r = i / row_n;
  if (!p.zero_rest) {
    const int lead = p.R ? min(max(p.cu[0], 0), p.T) : p.T, tail = p.R ? min(max(p.cu[p.R], 0), p.T) : p.T;
    if (r < lead || r >= tail) return;
  }
  const float* src = p.shares + (blockIdx.y ? p.runs * all : 0) + i;
  float4 s = *reinterpret_cast<const float4*>(src);
#pragma unroll 4
  for (int k = 1; k < p.runs; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(src + k * all);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  __bf16* o = blockIdx.y ? static_cast<__bf16*>(p.gC) + r * p.gcs + i % row_n : static_cast<__bf16*>(p.gB) + r * p.gbs + i % row_n;
  *reinterpret_cast<u32x2*>(o) = u32x2{pipe::cvt2(s.x, s.y), pipe::cvt2(s.z, s.w)};
}

// How the work is cut, and where the parts of the workspace lie (bytes).
struct Plan {
  int seg, nseg, runs, run_strips, blocks;
  size_t share, states, heads, shares, total;  // of one direction's segments; of one of the two states; behind both
};
Plan plan(int T, int R, int H, int P, int G, int N) {
  Plan w;
  const int nstrips = H * (P / 64), spp = P / 64;
  w.blocks = (T + Q - 1) / Q;
  // segments: workgroups for every CU three times over, both directions counted, of at least four pieces
  const int want = nstrips >= 384 ? 1 : 384 / nstrips;
  int per = (w.blocks + want - 1) / want;
  if (per < 4) per = 4;
  w.seg = per * Q;
  w.nseg = T > w.seg ? (T + w.seg - 1) / w.seg : 1;
  // runs of strips: the fewest rounds of workgroups over the CUs, weighed by their length
  const int heads = H / G, base = w.blocks * G;
  long long best = -1;
  for (int n = 1; n <= heads; ++n) {
    const int len = (heads + n - 1) / n;
    if ((heads + len - 1) / len != n) continue;
    const long long cost = ((long long)base * n + 255) / 256 * (len * spp + 2);
    if (best < 0 || cost < best) best = cost, w.runs = n, w.run_strips = len * spp;
  }
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  w.share = up((size_t)(w.nseg - 1) * nstrips * (N * 64 + 1) * sizeof(float));
  w.states = up((size_t)(w.blocks + R) * nstrips * N * 64 * sizeof(__bf16));
  w.heads = up((size_t)w.blocks * H * 3 * sizeof(float));
  w.shares = w.runs > 1 ? 2 * (size_t)w.runs * T * G * N * sizeof(float) : 0;
  w.total = 2 * w.share + 2 * w.states + w.heads + w.shares;
  return w;
}

}  // namespace

size_t ssm_scan_bwd_workspace_bytes(int T, int R, int H, int P, int G, int N) { return plan(T, R, H, P, G, N).total; }

hipError_t launch_ssm_scan_bwd(const ScanBwdArgs& a) {
  hipStream_t stream = static_cast<hipStream_t>(a.stream);
  const ScanShape& n = a.n;
  const Plan w = plan(n.T, n.R, n.H, n.P, n.G, n.N);
  char* ws = static_cast<char*>(a.ws);
  const int nstrips = n.H * (n.P / 64);
  BwdParams p = {a.x, a.dt, a.a, a.B, a.C, a.D, a.bias, a.grad_out, a.cu, a.S0, a.grad_S_final, a.grad_x, a.grad_dt, a.grad_a,
                 a.grad_B, a.grad_C, a.grad_D, a.grad_bias, a.grad_S0,
                 {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + w.share)},
                 {reinterpret_cast<__bf16*>(ws + 2 * w.share), reinterpret_cast<__bf16*>(ws + 2 * w.share + w.states)},
                 reinterpret_cast<float*>(ws + 2 * w.share + 2 * w.states + w.heads),
                 reinterpret_cast<float*>(ws + 2 * w.share + 2 * w.states), a.xs, a.dts, a.bs, a.cs, a.gs, a.gxs, a.gbs, a.gcs,
                 n.T, n.R, n.H, n.P, n.G, w.seg, w.nseg, w.runs, w.run_strips, n.dt_f32, n.p_f32, a.zero_rest};
  auto go = [&](auto nn, auto parts) {
    constexpr int N = decltype(nn)::value, PARTS = decltype(parts)::value;
    if (w.nseg > 1) {
      hipLaunchKernelGGL((states_kernel<N, true, PARTS>), dim3(nstrips, w.nseg - 1, 2), dim3(256), 0, stream, p);
      if (const hipError_t e = hipGetLastError()) return e;
      hipLaunchKernelGGL((join_both_kernel<N>), dim3(N * 64 / 1024, nstrips, 2), dim3(256), 0, stream, p.seg_ws[0], p.seg_ws[1],
                         nstrips, w.nseg - 1);
      if (const hipError_t e = hipGetLastError()) return e;
    }
    hipLaunchKernelGGL((states_kernel<N, false, PARTS>), dim3(nstrips, w.nseg, 2), dim3(256), 0, stream, p);
    if (const hipError_t e = hipGetLastError()) return e;
    if (w.blocks) {
      hipLaunchKernelGGL((grad_kernel<N>), dim3(w.blocks, n.G * w.runs), dim3(256), 0, stream, p);
      if (const hipError_t e = hipGetLastError()) return e;
    }
    const long long values = w.runs > 1 ? (long long)n.T * n.G * N : 0;
    hipLaunchKernelGGL(sums_kernel, dim3(n.H + (unsigned)((values + 1023) / 1024), values ? 2 : 1), dim3(256), 0, stream, p,
                       w.blocks, N);
    return hipGetLastError();
  };
  // Two parts leave 2^-17 of each term in states that are stored as bf16; the gradient of S0 is a float32 result.
  auto typed = [&](auto nn) { return a.grad_S0 ? go(nn, pipe::ic<3>{}) : go(nn, pipe::ic<2>{}); };
  return n.N == 64 ? typed(pipe::ic<64>{}) : typed(pipe::ic<128>{});
}

}  // namespace gdn
