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
// Where numbers are rounded: C B^T o L, and the state as it enters the product with C, are
// taken in two bf16 parts (2^-17 of each term), so that the result is off by its own
// rounding alone (1.66e-3 in norm; with one part of the state and of the weights between the
// halves of a piece it was 1.8e-3, 2.4e-3 where most of it comes from the state, in 94.7
// and 205 us for 99.5 and 216 of the two cases below).  What goes into the state is taken
// in three parts, 2^-25, since the state is a result and is carried on.
//
// 8 x 2048 rows, 24 heads of 64, N = 128: 28 us for the segments' ends, 72 for the rest,
// 0.13 PFLOP/s of the formulas' own work; 1 x 16384, 32 heads of 128: 60 + 12 + 150.  What
// bounds it is the chain of a piece (9 us for four strips), beside which nothing runs on a
// CU, since LDS holds one workgroup: the matrix unit is 0.22 to 0.30 busy, the vector unit
// 0.41 to 0.56.  Scalars that do not fit are kept in lanes (47 to 59 of them).
#include "gdn_scan.hpp"

namespace gdn {
namespace {

using namespace scan;
using tile::zero16;

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
  int T, R, H, P, G, seg, nseg, idle;  // idle: segments without rows behind the others (see Idle)
  bool dt_f32, p_f32, zero_rest, joined;
};

// A workgroup's part of the work: those of a segment, which read the same rows of B and
// C, are neighbours.  Segments without rows are behind all others.
struct Where {
  int seg, group, set;
};
__device__ __forceinline__ Where where(const ScanParams& p, const Strips& sp, int segs) {
  const int per = p.G * sp.sets, all = per * segs;
  const int id = (int)blockIdx.x < all ? neighbours(blockIdx.x, all) : blockIdx.x;
  return {id / per, id % per / sp.sets, id % sp.sets};
}

// Where four values (j a multiple of 4) of a row i of C B^T lie in LDS: 16-byte pieces
// are moved by the row, so that neither 16 rows' nor 16 pieces' meet in a bank.
__device__ __forceinline__ int cb_off(int i, int j) { return i * Q + ((j / 4) ^ (i & 15)) * 4; }

// The state S of 32 columns (block xcol of the rows Xt) behind a piece of rows of B and
// x.  between(k), k = 0 to 3: what else is to be issued behind the products of 16 rows.
template <int N, class F>
__device__ __forceinline__ void add_piece(f32x16 (&S)[N / 32], const __bf16* Bt, const __bf16* Xt, int xcol, int cb, int xb,
                                          const Steps& st, int half, F between) {
  constexpr int NT = N / 32;
  const float keep = exp2_(st.total);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) S[t][e] *= keep;
  // each 16 rows' operands are read beside the products of the 16 before
  u32x4 bt[2][NT], xk[2];
  xk[0] = tile::col_frag<128>(Xt, xb, 0, xcol);
#pragma unroll
  for (int t = 0; t < NT; ++t) bt[0][t] = tile::col_frag<N>(Bt, cb, 0, t);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    Split<kParts> xw;
    xw.make(xk[k & 1], st.w + 16 * k + 4 * half, st.w + 16 * k + 8 + 4 * half);
    if (k < 3) {
      xk[(k + 1) & 1] = tile::col_frag<128>(Xt, xb, 16 * (k + 1), xcol);
#pragma unroll
      for (int t = 0; t < NT; ++t) bt[(k + 1) & 1][t] = tile::col_frag<N>(Bt, cb, 16 * (k + 1), t);
    }
#pragma unroll
    for (int q = 0; q < kParts; ++q)
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t] = tile::mma(bt[k & 1][t], xw.part[q], S[t]);
    between(k);
  }
}

// What each segment leaves in the state of the sequence that crosses its end.  As
// many waves more as strips bring the rows of the piece to come and compute its steps,
// one strip's each, so that the others have nothing but their products to wait for.
template <int N, int NS>
__global__ __launch_bounds__(192 * NS, 1) void ends_kernel(ScanParams p) {
  constexpr int NT = N / 32, kTile = Q * N, kBuf = kTile + Q * 64 * NS;
  __shared__ __attribute__((aligned(1024))) __bf16 buf[2][kBuf];
  __shared__ Steps st_all[2][NS];
  __shared__ int window[kWindow];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const bool helper = wave >= 2 * NS;
  const int mine_of = helper ? wave - 2 * NS : wave / 2;  // strip of the set
  const Strips sp = strips(p.H, p.P, p.G, NS);
  const Where wg = where(p, sp, p.nseg - 1);
  const int group = wg.group, set = wg.set, seg = wg.seg;
  const int here = min(NS, sp.per_group - set * NS), strip0 = group * sp.per_group + set * NS;
  const bool mine = mine_of < here;
  const int strip = strip0 + (mine ? mine_of : 0), spp = p.P / 64, head = strip / spp, hcol = (strip % spp) * 64 + (wave & 1) * 32;
  const int nstrips = p.H * spp;

  const Offsets cu = offsets<192 * NS>(p.cu, p.R, window);
  const int s0 = seg * p.seg, s1 = min(s0 + p.seg, p.T);
  float* const kept = p.ws + (size_t)(p.nseg - 1) * nstrips * N * 64;
  Walk<false> walk;
  walk.init(cu, p.R, p.T, s0, s1);
  const int r = walk.rend - 1;
  const int b0 = r >= 0 ? min(max(cu(r), 0), p.T) : p.T, e0 = r >= 0 ? min(cu(r + 1), p.T) : 0;
  if (e0 <= s1 || b0 >= s1) {
    if ((int)threadIdx.x < here) kept[(size_t)seg * nstrips + strip0 + threadIdx.x] = kNone;
    return;
  }
  walk.r = r, walk.beg = b0, walk.pos = max(b0, s0), walk.end = e0;

  Piece cur, nxt, nx2;
  bool more = walk.next(cur), more2 = more && walk.next(nxt);
  if (!more2) nxt.row = nxt.n = 0;
  if (helper) {
    Stage<N, Q, NS> sb;
    Stage<128, Q, NS> sx;  // two strips at a time
    sb.init(p.bs, mine_of);
    sx.init(p.xs, mine_of);
    const __bf16* xg = static_cast<const __bf16*>(p.x) + strip0 * 64;
    const __bf16* bg = static_cast<const __bf16*>(p.B) + group * N;
    const float a = param(p.a, p.p_f32, head), bias = p.bias ? param(p.bias, p.p_f32, head) : 0.f;
    auto stage = [&](int b, const Piece& pc) {
      sb.load(buf[b], source(bg, p.bs, pc.row, pc.n, N), mine_of);
#pragma unroll
      for (int i = 0; i < NS / 2; ++i)
        if (2 * i < here)
          sx.load(buf[b] + kTile + i * Q * 128, source(xg + 128 * i, p.xs, pc.row, pc.n, 64 * min(2, here - 2 * i)), mine_of);
    };
    auto ask = [&](const Piece& pc) { return lane < pc.n ? dt_bits(p.dt, p.dt_f32, (long long)(pc.row + lane) * p.dts + head) : 0u; };
    auto take = [&](int b, unsigned bits, const Piece& pc) { steps(st_all[b][mine_of], dt_of(bits, p.dt_f32) + bias, a, lane < pc.n); };
    unsigned bits = ask(cur), ahead = ask(nxt);
    if (more) take(0, bits, cur), stage(0, cur);
    bits = ahead;
    for (int b = 0; more; b ^= 1) {
      tile::staged_barrier();
      bits = arrived(bits);
      const bool more3 = more2 && walk.next(nx2);
      if (!more3) nx2.row = nx2.n = 0;
      ahead = ask(nx2);
      if (more2) stage(b ^ 1, nxt), take(b ^ 1, bits, nxt);
      bits = ahead;
      nxt = nx2;
      more = more2, more2 = more3;
    }
    return;
  }

  f32x16 S[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) S[t] = zero16();
  const int cb = col_base_state<N>(lane), xb = tile::col_base<128>(lane);
  float whole = 0.f;  // log2 of what the segment keeps of a state
  for (int b = 0; more; b ^= 1) {
    tile::staged_barrier();
    const bool more3 = more2 && walk.next(nx2);
    if (cur.first && p.S0) load_state<NT>(S, p.S0 + (((long long)cur.seq * p.H + head) * N) * p.P + hcol, p.P);
    const Steps& st = st_all[b][wave / 2];
    whole += st.total;
    add_piece<N>(S, buf[b], buf[b] + kTile + wave / 4 * Q * 128, wave % 4, cb, xb, st, half, [](int) {});
    cur = nxt, nxt = nx2;
    more = more2, more2 = more3;
  }
  if (mine) {
    f32x4* at = reinterpret_cast<f32x4*>(p.ws + ((size_t)seg * nstrips + strip) * N * 64 + (wave & 1) * N * 32) + lane;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) at[(4 * t + q) * 64] = f32x4{S[t][4 * q], S[t][4 * q + 1], S[t][4 * q + 2], S[t][4 * q + 3]};
    if (threadIdx.x % 128 == 0) kept[(size_t)seg * nstrips + strip] = b0 >= s0 ? kFresh : whole;
  }
}

template <int N, int NS>
__global__ __launch_bounds__(128 * NS, NS == 4 ? 2 : 1) void scan_kernel(ScanParams p) {
  constexpr int NT = N / 32, kThreads = 128 * NS, kWaves = 2 * NS;
  constexpr int kTile = Q * N, kX = Q * 64 * NS;
  constexpr int kBuf = 2 * kTile + kX;
  __shared__ __attribute__((aligned(1024))) __bf16 buf[2][kBuf];
  __shared__ Steps st_all[NS];
  __shared__ __attribute__((aligned(1024))) float cbs[Q * Q];  // C B^T: [i][j], see cb_off
  __shared__ __attribute__((aligned(16))) __bf16 yts[N == 64 ? NS * 64 * 32 : 8];
  __shared__ int window[kWindow];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5, col = lane & 31;

  const Strips sp = strips(p.H, p.P, p.G, NS);
  const Where wg = where(p, sp, p.nseg);
  const int group = wg.group, set = wg.set, seg = wg.seg;
  const int in_group = set * NS, here = min(NS, sp.per_group - in_group);
  const int strip0 = group * sp.per_group + in_group;
  const bool mine = wave / 2 < here;  // otherwise the wave follows the first strip and writes nothing
  const int strip = strip0 + (mine ? wave / 2 : 0);
  const int spp = p.P / 64, head = strip / spp, hcol = (strip % spp) * 64 + (wave & 1) * 32;  // of the head
  const int nstrips = p.H * spp;
  const float a = param(p.a, p.p_f32, head), bias = p.bias ? param(p.bias, p.p_f32, head) : 0.f;

  const Offsets cu = offsets<kThreads>(p.cu, p.R, window);
  const int s0 = min(seg * p.seg, p.T), s1 = min(s0 + p.seg, p.T);
  float* const local = p.ws;
  float* const kept = p.ws + (size_t)(p.nseg - 1) * nstrips * N * 64;
  auto state_at = [&](const float* base, int seq) { return base + (((long long)seq * p.H + head) * N) * p.P + hcol; };
  // a slot holds the accumulators as they are, four values of each lane together
  auto slot = [&](int s) { return reinterpret_cast<f32x4*>(local + ((size_t)s * nstrips + strip) * N * 64 + (wave & 1) * N * 32) + lane; };

  f32x16 S[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) S[t] = zero16();
  Walk<false> walk;
  walk.init(cu, p.R, p.T, s0, s1);
  const bool goes_on = seg && walk.goes_on();

  // staging: rows of C, B and x
  Stage<N, Q, kWaves> sc, sb;
  Stage<128, Q, kWaves> sx;  // two strips at a time
  sc.init(p.cs, wave);
  sb.init(p.bs, wave);
  sx.init(p.xs, wave);
  const __bf16* xg = static_cast<const __bf16*>(p.x) + strip0 * 64;
  const __bf16* bg = static_cast<const __bf16*>(p.B) + group * N;
  const __bf16* cg = static_cast<const __bf16*>(p.C) + group * N;
  // One of the kLoads parts of a piece's staging: they are spread over the work on the piece before, since the loads of
  // eight waves in a row wait for each other.
  constexpr int kLx = decltype(sx)::LOADS, kLb = decltype(sb)::LOADS, kLoads = NS / 2 * kLx + 2 * kLb;
  auto stage = [&](int b, const Piece& pc, int i) {
    if (i < NS / 2 * kLx) {
      const int pair = i / kLx;
      if (2 * pair < here)
        sx.load_one(buf[b] + kTile + pair * Q * 128,
                    source(xg + 128 * pair, p.xs, pc.row, pc.n, 64 * min(2, here - 2 * pair)), wave, i % kLx);
    } else if (i < NS / 2 * kLx + kLb) {
      sb.load_one(buf[b], source(bg, p.bs, pc.row, pc.n, N), wave, i - NS / 2 * kLx);
    } else {
      sc.load_one(buf[b] + kTile + kX, source(cg, p.cs, pc.row, pc.n, N), wave, i - NS / 2 * kLx - kLb);
    }
  };
  auto raw_dt = [&](const Piece& pc) {
    return lane < pc.n ? dt_at(p.dt, p.dt_f32, (long long)(pc.row + lane) * p.dts + head) + bias : 0.f;
  };
  const int rb = tile::row_base<N>(lane), cb = col_base_state<N>(lane), xb = tile::col_base<128>(lane);
  const float dskip = p.D ? param(p.D, p.p_f32, head) : 0.f;

  Piece cur, nxt;
  bool more = walk.next(cur);
  float z0 = 0.f;
  // One wave of a strip computes its steps: waves 0, 3, 5 and 6, one on each SIMD.
  const bool steps_mine = wave % 2 == ((wave / 2 ^ wave / 4) & 1);
  if (more) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) stage(0, cur, i);
    if (steps_mine) z0 = raw_dt(cur);
  }
  {
    if (goes_on) {  // the state at the border, added up here where that was not done before
      float f = 1.f;
      for (int k = seg - 1;; --k) {
        const f32x4* at = slot(k);
        const float keeps = p.joined ? kFresh : kept[(size_t)k * nstrips + strip];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 v = at[(4 * t + q) * 64];
#pragma unroll
            for (int j = 0; j < 4; ++j) S[t][4 * q + j] = __builtin_fmaf(f, v[j], S[t][4 * q + j]);
          }
        if (keeps == kFresh || k == 0) break;
        f *= exp2_(keeps);
      }
    }
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
      const Idle of = idle_of(seg, p.nseg, p.idle);
      for (int r = of.first; r < p.R; r += of.step) {
        const int b = min(max(cu(r), 0), p.T);
        if (min(cu(r + 1), p.T) > b) continue;
        // by 64 rows, whose loads are issued together; addresses are computed here
        const int lane = tile::fresh(threadIdx.x & 63), step = tile::fresh(8 * p.P);
        const long long at = (((long long)r * p.H + head) * N + lane / 8) * p.P + hcol + lane % 8 * 4;
        const float* from = p.S0 + at;
        float* to = p.S_final + at;
#pragma unroll 1
        for (int n = 0; n < N; n += 64) {
          f32x4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i, from += step) v[i] = p.S0 ? *reinterpret_cast<const f32x4*>(from) : pipe::zero4();
#pragma unroll
          for (int i = 0; i < 8; ++i, to += step) *reinterpret_cast<f32x4*>(to) = v[i];
        }
      }
    }
  }
  float z = z0;
  for (int b = 0; more; b ^= 1) {
    tile::staged_barrier();  // this piece's rows are here, and the other buffer is free
    z = arrived(z);
    more = walk.next(nxt);
    if (!more) nxt.row = nxt.n = 0;
    const float z_next = steps_mine ? raw_dt(nxt) : 0.f;
    auto stage_some = [&](int part) {  // of four
      if (more)
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (i * 4 / kLoads == part) stage(b ^ 1, nxt, i);
    };
    if (cur.first) {
      if (p.S0) load_state<NT>(S, state_at(p.S0, cur.seq), p.P);
      else {
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] = zero16();
      }
    }
    Steps& st = st_all[wave / 2];
    const __bf16 *Bt = buf[b], *Xt = buf[b] + kTile + wave / 4 * Q * 128, *Ct = buf[b] + kTile + kX;
    const int xcol = wave % 4;  // 32-column block of the pair of strips

    if (steps_mine) steps(st, z, a, lane < cur.n);
    f32x16 y[2] = {zero16(), zero16()};
    float k0 = 0.f, k1 = 0.f;  // of the lane's two rows
    {
      // C B^T, once for all strips: the ten 16 x 16 blocks at or under the diagonal, rows j by lanes i, by the waves that
      // have no steps to compute
      const int lane = tile::fresh(threadIdx.x & 63);
#pragma unroll 1
      for (int tile = steps_mine ? 10 : NS == 4 ? (wave < 3 ? wave - 1 : wave < 7 ? 2 : 3) : wave - 1; tile < 10; tile += NS) {
        const int ib = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, jb = tile - ib * (ib + 1) / 2;
        f32x4 acc = pipe::zero4();
#pragma unroll
        for (int ks = 0; ks < N / 32; ++ks)
          acc = pipe::mma32(*reinterpret_cast<const u32x4*>(Bt + pipe::row_off<N>(16 * jb + lane % 16, 32 * ks + lane / 16 * 8)),
                            *reinterpret_cast<const u32x4*>(Ct + pipe::row_off<N>(16 * ib + lane % 16, 32 * ks + lane / 16 * 8)), acc);
        *reinterpret_cast<f32x4*>(cbs + cb_off(16 * ib + lane % 16, 16 * jb + lane / 16 * 4)) = acc;
      }
#pragma unroll
      for (int ks = 0; ks < N / 16; ++ks) {
        const Two s = two_parts(S[ks / 2], ks % 2);
        const u32x4 c0 = tile::row_frag<N>(Ct, rb, 0, ks), c1 = tile::row_frag<N>(Ct, rb, 32, ks);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          y[0] = tile::mma(s.part[q], c0, y[0]);
          y[1] = tile::mma(s.part[q], c1, y[1]);
        }
      }
    }
    lds_barrier();
    k0 = st.G[col], k1 = st.G[32 + col];
    auto state = [&] { add_piece<N>(S, Bt, Xt, xcol, cb, xb, st, half, stage_some); };
    auto result = [&] {
      // addresses and masks are computed here, not kept over the loop
      const int lane = tile::fresh(threadIdx.x & 63), half = lane >> 5, col = lane & 31;
      const unsigned seen = col < 4 * half ? 0u : 0xffffffffu >> (31 - (col - 4 * half));  // bit 8 q + j: row 8 q + 4 half + j <= col
      const float g0 = k0, g1 = k1, off = exp2_(g1 - st.G[31]);
      const float f0 = exp2_(g0), f1 = exp2_(g1);
#pragma unroll
      for (int e = 0; e < 16; ++e) y[0][e] *= f0, y[1][e] *= f1;
      // the weights of rows: tiles of rows j (elements) by rows i (lanes), 16 rows j at a time, as operands
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float f[3][8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j0 = 16 * k + 8 * u + 4 * half;
          const float4 ua = *reinterpret_cast<const float4*>(st.u + j0), ub = *reinterpret_cast<const float4*>(st.u + 32 + j0);
          const float4 v = *reinterpret_cast<const float4*>(st.v + j0);
          const f32x4 c00 = *reinterpret_cast<const f32x4*>(cbs + cb_off(col, j0));
          const f32x4 c10 = *reinterpret_cast<const f32x4*>(cbs + cb_off(32 + col, j0));
          const f32x4 c11 = *reinterpret_cast<const f32x4*>(cbs + cb_off(32 + col, 32 + j0));
          const float fa[4] = {ua.x, ua.y, ua.z, ua.w}, fb[4] = {ub.x, ub.y, ub.z, ub.w}, fv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // blocks over the diagonal hold anything: left out by bits
            const int in = (int)(seen << (31 - (8 * (2 * k + u) + j))) >> 31;
            f[0][4 * u + j] = __builtin_bit_cast(float, __builtin_bit_cast(int, c00[j] * exp2_(g0 + fa[j])) & in);
            f[1][4 * u + j] = c10[j] * (off * fv[j]);
            f[2][4 * u + j] = __builtin_bit_cast(float, __builtin_bit_cast(int, c11[j] * exp2_(g1 + fb[j])) & in);
          }
        }
        u32x4 w[3], rest[3];
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[i][e] = pipe::cvt2(f[i][2 * e], f[i][2 * e + 1]);
            rest[i][e] = pipe::cvt2(f[i][2 * e] - pipe::lo_f(w[i][e]), f[i][2 * e + 1] - pipe::hi_f(w[i][e]));
          }
        const u32x4 x0 = tile::col_frag<128>(Xt, xb, 16 * k, xcol), x1 = tile::col_frag<128>(Xt, xb, 32 + 16 * k, xcol);
        y[0] = tile::mma(x0, w[0], y[0]);
        y[1] = tile::mma(x0, w[1], y[1]);
        y[0] = tile::mma(x0, rest[0], y[0]);
        y[1] = tile::mma(x0, rest[1], y[1]);
        y[1] = tile::mma(x1, w[2], y[1]);
        y[1] = tile::mma(x1, rest[2], y[1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      // y: columns are rows of the piece, elements channels 8 q + 4 half + j.  Added to D x, and by 32 rows through a part
      // of LDS that is this wave's alone, where C was, to memory in pieces of 16 bytes.
      char* const yt = reinterpret_cast<char*>(N == 128 ? const_cast<__bf16*>(Ct) : yts) + wave * 2048;
      const int hp = p.H * p.P;
      __bf16* o = static_cast<__bf16*>(p.out) + (long long)(cur.row + lane / 4) * hp + strip * 64 + (wave & 1) * 32 + lane % 4 * 8;
#pragma unroll
      for (int it = 0; it < 2; ++it) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const u32x2 xv = pipe::ld4(Xt + pipe::row_off<128>(32 * it + col, xcol * 32 + 8 * q + 4 * half));
          u32x2 w;
          w[0] = pipe::cvt2(__builtin_fmaf(dskip, pipe::lo_f(xv[0]), y[it][4 * q]), __builtin_fmaf(dskip, pipe::hi_f(xv[0]), y[it][4 * q + 1]));
          w[1] = pipe::cvt2(__builtin_fmaf(dskip, pipe::lo_f(xv[1]), y[it][4 * q + 2]), __builtin_fmaf(dskip, pipe::hi_f(xv[1]), y[it][4 * q + 3]));
          *reinterpret_cast<u32x2*>(yt + col * 64 + ((q ^ (col >> 1 & 3)) * 16 + half * 8)) = w;
        }
        pipe::issue_fence();
        const int left = mine ? cur.n - 32 * it - lane / 4 : 0;
#pragma unroll
        for (int r = 0; r < 2; ++r, o += 16 * hp) {
          const int row = 16 * r + lane / 4;
          const u32x4 v = *reinterpret_cast<const u32x4*>(yt + row * 64 + (lane % 4 ^ (row >> 1 & 3)) * 16);
          if (16 * r < left) *reinterpret_cast<u32x4*>(o) = v;
        }
        pipe::issue_fence();
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // The waves of a SIMD take the two in different orders, so that one's products run beside the other's arithmetic.
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      if (i == wave / (kWaves / 2)) result();
      else state();
    }
    if (cur.last && p.S_final && mine) store_state<NT>(S, const_cast<float*>(state_at(p.S_final, cur.seq)), p.P);
    cur = nxt;
    z = z_next;
  }
}

template <int N> __global__ __launch_bounds__(256) void join_kernel(float* ws, int nstrips, int slots) {
  join<N>(ws, nstrips, slots, blockIdx.y, (blockIdx.x * 256 + threadIdx.x) * 4, false);
}

// How the work is cut.  Strips to a workgroup: four, so that eight waves share C B^T
// and its operands, where that still leaves a workgroup for every second CU; otherwise
// two, whose four waves are done sooner (24 heads of 64, N = 128, with four and with two:
// 8 x 2048 rows 89 and 104 us, 1 x 16384 97 and 110; 1 x 2048 57 and 45, 131 24 and 21).
// Rows to a segment: a workgroup to each CU,
// none waiting, and at least four pieces.
struct Cut {
  int ns, sets, seg, nseg;
};
Cut cut(int T, int H, int P, int G) {
  Cut c;
  const int pieces = (T + Q - 1) / Q;
  for (c.ns = 4;; c.ns = 2) {
    c.sets = G * strips(H, P, G, c.ns).sets;
    const int want = c.sets >= 256 ? 1 : 256 / c.sets;
    int per = (pieces + want - 1) / want;
    if (per < 4) per = 4;
    c.seg = per * Q;
    c.nseg = T > c.seg ? (T + c.seg - 1) / c.seg : 1;
    if (c.ns == 2 || (H / G * (P / 64) > 2 && c.sets * c.nseg >= 128)) return c;
  }
}
// Whether a launch of its own adds the segments up: a workgroup that does it for itself reads all those before it in its
// sequence, half of a sequence's on average (24 heads of 64, with the launch and without: 8 x 2048 rows 95 and 88 us, 1 x 16384 97 and 119).
bool joins(int T, int R, int seg) { return (long long)T > 8LL * seg * (R > 1 ? R : 1); }

}  // namespace

// The workspace: the states of [segments - 1][strips][N][64], then what each segment
// keeps (see join).
size_t ssm_scan_workspace_bytes(int T, int H, int P, int G, int N) {
  const size_t slots = cut(T, H, P, G).nseg - 1, nstrips = (size_t)H * (P / 64);
  return slots * nstrips * (N * 64 + 1) * sizeof(float);
}

hipError_t launch_ssm_scan(const ScanArgs& a) {
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  const ScanShape& n = a.n;
  const Cut c = cut(n.T, n.H, n.P, n.G);
  const int nseg = c.nseg, nstrips = n.H * (n.P / 64);
  const int idle = a.S_final ? idle_segments(n.R, 256 / c.sets - nseg) : 0;  // one workgroup to a CU
  const ScanParams p = {a.x, a.dt, a.a, a.B, a.C, a.D, a.bias, a.cu, a.S0, a.out, a.S_final, a.ws, a.xs, a.dts, a.bs, a.cs,
                        n.T, n.R, n.H, n.P, n.G, c.seg, nseg, idle, n.dt_f32, n.p_f32, a.zero_rest, joins(n.T, n.R, c.seg)};
  auto go = [&](auto nn, auto per) {
    constexpr int N = decltype(nn)::value, NS = decltype(per)::value;
    if (nseg > 1) {
      hipLaunchKernelGGL((ends_kernel<N, NS>), dim3(c.sets * (nseg - 1)), dim3(192 * NS), 0, st, p);
      if (const hipError_t e = hipGetLastError()) return e;
      if (p.joined) {
        hipLaunchKernelGGL((join_kernel<N>), dim3(N * 64 / 1024, nstrips), dim3(256), 0, st, a.ws, nstrips, nseg - 1);
        if (const hipError_t e = hipGetLastError()) return e;
      }
    }
    hipLaunchKernelGGL((scan_kernel<N, NS>), dim3(c.sets * (nseg + idle)), dim3(128 * NS), 0, st, p);
    return hipGetLastError();
  };
  auto sized = [&](auto nn) { return c.ns == 4 ? go(nn, pipe::ic<4>{}) : go(nn, pipe::ic<2>{}); };
  return n.N == 64 ? sized(pipe::ic<64>{}) : sized(pipe::ic<128>{});
}

}  // namespace gdn
