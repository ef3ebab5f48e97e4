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
// memory in bf16: as such they enter every product below.  (M, and W summed over a run's
// heads in float32, are taken in two bf16 parts: x's, B's and C's gradients are 1.7e-3 off,
// of which their own rounding is 1.66e-3; with one part, and W rounded for each head, 2.3e-3,
// and 6.7e-3 where heads cancel.  Those of a and dt_bias, for which <Z, S> is taken of two
// states as stored, are 1e-4 to 1e-3 off in float32, up to 4e-3 where their rows' terms
// cancel; states in two parts would be 400 MB more to move at the 8 x 2048 rows below, and
// no LDS is left for them at N = 128.)  (4) All gradients, a
// workgroup to 64 rows and a run of strips of one group: gB and gC are summed over the
// strips in its accumulators.  (5) Sums over the runs of strips where there are
// several, and over rows for a, D and the bias.  All sums are made in a fixed order.
// 8 x 2048 rows, 24 heads of 64, N = 128: 5 + 5 + 85 + 128 + 5 us; 13 sequences of up to
// 1201 rows, 16 heads of 128, N = 64: 26 + 5 + 50 + 129 + 5.
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
  int T, R, H, P, G, seg, nseg, idle, runs, run_strips;
  bool dt_f32, p_f32, zero_rest;
};

// ---------------------------------------------------------------- states
// A stored state: 16-byte pieces of eight channels.  That of row n, channels 8 c on, is
// the one of this number.
__device__ __forceinline__ int state_piece(int n, int c) { return (n / 32 * 4 + c / 2) * 64 + (c & 1) * 32 + n % 32; }

// A workgroup: 64 n of one strip, one segment; states downwards, or their
// gradients upwards.  Two waves have 32 n and 64 channels each of the transposed
// state: their lanes the n, their elements the channels, eight in a row to a lane: a
// 16-byte piece of the stored state.  Stored are a wave's pieces as they are, 1 KB at a
// time (see state_piece).  What the rows add is weighted on the side of B (C), in PARTS
// bf16 parts, once.  A third wave brings the rows of the piece after next, and a fourth
// computes the next one's steps, so that the two have nothing but their products to
// wait for.  The states go to memory: 8 x 2048 rows x 24 strips, N = 128, write 201 MB
// and read 194 in 85 us; 13 sequences of up to 1201 rows x 32 strips, N = 64, took 55 us
// with a piece's rows one piece ahead and four waves of 32 x 32, now 50.
constexpr int kStateThreads = 256, kHalf = 64;  // n to a workgroup
template <int N, bool LOCAL, int PARTS>
__global__ __launch_bounds__(kStateThreads, 3) void states_kernel(BwdParams p) {
  constexpr int NP = 2, kParts = N / kHalf;  // tiles of 32 channels to a wave; workgroups to a strip
  __shared__ __attribute__((aligned(1024))) __bf16 buf[3][Q * kHalf + Q * 64];
  __shared__ Steps st_two[2];
  __shared__ int window[kWindow];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5, col = lane & 31;
  const int spp = p.P / 64, nstrips = p.H * spp, per = nstrips * kParts, slots = p.nseg - LOCAL;
  // the two halves of a strip, which read the same x, lie nstrips apart: on one XCD where that is a multiple of eight
  const bool up = (int)blockIdx.x >= per * slots;  // and behind those, segments without rows
  const int id = blockIdx.x - up * per * slots, seg0 = id / per;
  const int strip = id % nstrips, n0 = id % per / nstrips * kHalf, nt = n0 / 32 + (wave & 1), head = strip / spp;
  const int hcol = (strip % spp) * 64, group = head / (p.H / p.G);
  const int seg = LOCAL && up ? seg0 + 1 : seg0;
  const float a = param(p.a, p.p_f32, head), bias = p.bias ? param(p.bias, p.p_f32, head) : 0.f;
  const Offsets cu = offsets<kStateThreads>(p.cu, p.R, window);
  const int s0 = min(seg * p.seg, p.T), s1 = min(s0 + p.seg, p.T);
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
        const float4* q = reinterpret_cast<const float4*>(src + n * stride + 32 * t + 16 * b + 8 * half);
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
        float4* q = reinterpret_cast<float4*>(dst + n * stride + 32 * t + 16 * b + 8 * half);
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
      if (threadIdx.x == 0 && n0 == 0) kept[(size_t)seg0 * nstrips + strip] = kNone;
      return;
    }
  } else if (up) {
    if (p.gS0) {  // sequences without rows
      const Idle of = idle_of(seg, p.nseg, p.idle);
      for (int r = of.first; r < p.R; r += of.step) {
        const int b = min(max(cu(r), 0), p.T);
        if (min(cu(r + 1), p.T) > b) continue;
        constexpr int K = kHalf * 16 / kStateThreads;
        const long long at = of_seq(r) + (long long)(n0 + (int)threadIdx.x / 16) * p.P + threadIdx.x % 16 * 4;
        f32x4 v[K];
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = p.gSf ? *reinterpret_cast<const f32x4*>(p.gSf + at + i * (kStateThreads / 16) * p.P) : pipe::zero4();
#pragma unroll
        for (int i = 0; i < K; ++i) *reinterpret_cast<f32x4*>(p.gS0 + at + i * (kStateThreads / 16) * p.P) = v[i];
      }
    }
    if (seg >= p.nseg) return;
    if (back.r >= back.rlow && back.pos > max(back.beg, s0) && back.end > s1) load(slot(seg), 64);
  } else if (seg && down.goes_on()) {
    load(slot(seg - 1), 64);
  }

  StageWave<kHalf> sk;
  StageWave<64> sv;
  const __bf16* kg = (up ? static_cast<const __bf16*>(p.C) : static_cast<const __bf16*>(p.B)) + group * N + n0;
  const __bf16* vg = (up ? static_cast<const __bf16*>(p.go) : static_cast<const __bf16*>(p.x)) + strip * 64;
  const long long ks = up ? p.cs : p.bs, vs = up ? p.gs : p.xs;
  sk.init(ks), sv.init(vs);
  const bool loads = wave == 2, steps_mine = wave == 3;
  auto raw_dt = [&](const Piece& pc) { return lane < pc.n ? dt_bits(p.dt, p.dt_f32, (long long)(pc.row + lane) * p.dts + head) : 0u; };
  auto take_steps = [&](int b, unsigned bits, const Piece& pc) {
    Steps& st = st_two[b];
    steps(st, dt_of(bits, p.dt_f32) + bias, a, lane < pc.n);
    if (up) {  // what a row adds is weighted by the decays up to it
      st.w[lane] = exp2_(st.G[lane]);
      pipe::issue_fence();
    }
  };
  auto next = [&](Piece& pc) {
    const bool some = up ? back.next(pc) : down.next(pc);
    if (!some) pc.row = pc.n = 0;
    return some;
  };
  const int kb = tile::col_base<kHalf>(lane), vb = col_base_state<64>(lane);
  auto stage = [&](int b, const Piece& pc) {
    sk.template load<Q>(buf[b], source(kg, ks, pc.row, pc.n, kHalf), 0);
    sv.template load<Q>(buf[b] + Q * kHalf, source(vg, vs, pc.row, pc.n, 64), 0);
  };

  Piece cur, nxt, nx2;
  bool more = next(cur), more2 = more && next(nxt);
  if (!more2) nxt.row = nxt.n = 0;
  if (loads) {
    tile::wait_all_but<0>();  // counted below are staged loads alone
    if (more) stage(0, cur);
    if (more2) stage(1, nxt);
    for (int to = 2; more; to = to == 2 ? 0 : to + 1) {
      // this piece's rows are here; the next one's, the latest loads, may be on their way
      if (more2) loads_barrier<(Q * kHalf + Q * 64) / 512>();
      else loads_barrier<0>();
      const bool more3 = more2 && next(nx2);
      if (more3) stage(to, nx2);
      cur = nxt, nxt = nx2, more = more2, more2 = more3;
    }
    return;
  }
  if (steps_mine) {
    unsigned bits = raw_dt(nxt);
    if (more) take_steps(0, raw_dt(cur), cur);
    for (int b = 0; more; b ^= 1) {
      lds_barrier();
      const bool more3 = more2 && next(nx2);
      if (!more3) nx2.row = nx2.n = 0;
      const unsigned after = raw_dt(nx2);
      if (more2) take_steps(b ^ 1, bits, nxt);
      bits = after;
      cur = nxt, nxt = nx2, more = more2, more2 = more3;
    }
    return;
  }
  for (int b = 0, at = 0; more; b ^= 1, at = at == 2 ? 0 : at + 1) {
    lds_barrier();
    const bool more3 = more2 && next(nx2);
    const Steps& st = st_two[b];
    if (up ? cur.last : cur.first) {
      const float* src = up ? p.gSf : p.S0;
      if (src) load(src + of_seq(cur.seq), p.P);
      else {
#pragma unroll
        for (int t = 0; t < NP; ++t) S[t] = zero16();
      }
    }
    if constexpr (!LOCAL) {
      u32x4* dst = reinterpret_cast<u32x4*>(p.states[up] + ((long long)piece_id(cur) * nstrips + strip) * N * 64) + nt * 256 + lane;
#pragma unroll
      for (int t = 0; t < NP; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) dst[(2 * t + i) * 64] = operand(S[t], i);
    }
    const float total = st.total;
    whole += total;
    const __bf16 *Kt = buf[at], *Vt = buf[at] + Q * kHalf;
    const float keep = exp2_(total);
#pragma unroll
    for (int t = 0; t < NP; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) S[t][e] *= keep;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      Split<PARTS> kw;
      kw.make(tile::col_frag<kHalf>(Kt, kb, 16 * k, wave), st.w + 16 * k + 4 * half, st.w + 16 * k + 8 + 4 * half);
#pragma unroll
      for (int t = 0; t < NP; ++t) {
        const u32x4 v = tile::col_frag<64>(Vt, vb, 16 * k, t);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) S[t] = tile::mma(v, kw.part[q], S[t]);
      }
    }
    if constexpr (!LOCAL) {
      if (up && cur.first && p.gS0) store(p.gS0 + of_seq(cur.seq), p.P);
    }
    cur = nxt, nxt = nx2, more = more2, more2 = more3;
  }
  if constexpr (LOCAL) {
    store(slot(seg0), 64);
    if (threadIdx.x == 0 && n0 == 0) kept[(size_t)seg0 * nstrips + strip] = fresh ? kFresh : whole;
  }
}

template <int N> __global__ __launch_bounds__(256) void join_both_kernel(float* down, float* up, int nstrips, int slots) {
  const bool back = blockIdx.z != 0;
  join<N>(back ? up : down, nstrips, slots, blockIdx.y, (blockIdx.x * 256 + threadIdx.x) * 4, back);
}

// -------------------------------------------------------------- gradients
template <int CTRL> __device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
// Sums of four elements over the 16 lanes of a row of lanes: lane l gets that of element l % 4.
__device__ __forceinline__ float column_sums(const f32x4& v) {
  const int lane = threadIdx.x & 63;
  const bool b0 = lane & 1, b1 = lane & 2;
  const float p = (b0 ? v[1] : v[0]) + dpp<0xB1>(b0 ? v[0] : v[1]), q = (b0 ? v[3] : v[2]) + dpp<0xB1>(b0 ? v[2] : v[3]);  // quad_perm [1, 0, 3, 2]
  float r = (b1 ? q : p) + dpp<0x4E>(b1 ? p : q);  // quad_perm [2, 3, 0, 1]
  r += dpp<0x128>(r);  // row_ror:8
  return r + dpp<0x124>(r);  // row_ror:4
}
// Sum over the four rows of 16 lanes, in each.
__device__ __forceinline__ float row_sums(float x) {
  int u = __builtin_bit_cast(int, x), w = u;
  asm("" : "+v"(w));
  const auto r = __builtin_amdgcn_permlane16_swap(u, w, false, false);
  return tile::sum_halves(__builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]));
}

__device__ __forceinline__ float dot2(unsigned a, unsigned b, float c) {
  return __builtin_fmaf(pipe::lo_f(a), pipe::lo_f(b), __builtin_fmaf(pipe::hi_f(a), pipe::hi_f(b), c));
}

constexpr int kFew = 64;        // offsets kept in LDS; more are read from memory
constexpr int kMostHeads = 64;  // to a run
constexpr int kGradWaves = 8, kGradThreads = 64 * kGradWaves;
constexpr int kBlockWaves = 5, kSteps = 5, kLoads = 6, kSums = 7;  // waves and their parts

template <int N> struct GradLds {
  __bf16 C[Q * N], B[Q * N];
  struct {
    __bf16 S[N * 64], Z[N * 64], x[Q * 64], h[Q * 64];
  } strip[2];
  __bf16 M[2][Q * Q];              // [i][j], in two parts; at the end W, summed over the strips
  Steps st[2];
  // sums of E over the columns and rows of each 16 x 16 block, its diagonal; h.x; shares of <Z, S>
  struct {
    float er[10][16], ec[10][16], ed[Q], hx[Q], zs[kGradThreads], R[N / 32][Q], Qs[N / 32][Q];
  } sums[2];
  struct {
    float a, bias, D;
  } heads[kMostHeads];  // of the run
  int window[kFew];
};

// A workgroup: 64 rows, a run of strips of one group, one after the other, with the
// next one's operands on their way to LDS.  For each strip, behind a barrier:
//   - five waves: M, W and the sums of E, in the ten blocks of 16 x 16 at or under the
//     diagonal (M goes to LDS as operands in two bf16 parts, W is summed over the strips in
//     their registers); the sixth: the steps of the next head;
//     the seventh: the next strip's loads; the eighth: the sums by rows of the
//     strip before;
//   - each wave: the states' products for a tile of gC and of gB (N = 64: of one of
//     them), 32 n x 32 rows, which stay in its accumulators over the strips, and of gx,
//     32 channels x 16 rows;
//   - behind a second barrier, the products with M, and gx to memory.
// Behind the last strip W, in two parts, takes M's place for its products with C and B.
// A strip takes some 5 us: the vector unit is 0.32 busy, LDS 0.25, the matrix unit 0.09.
// (With W's products in every strip it was 5.1, without the loads 4.6, without the states'
// products 4.3, without M, W and E the same.)  The waves wait 0.62 of the time, mostly at the two barriers, with one workgroup to a CU.  Pointers, strides and
// resources are live in every wave over the whole walk: 351 scalars (N = 64: 283) are kept in
// lanes, and the loop over the pieces has some 600 reads of these.
template <int N>
__global__ __launch_bounds__(kGradThreads, 2) void grad_kernel(BwdParams p) {
  __shared__ __attribute__((aligned(1024))) GradLds<N> L;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5, col = lane & 31;
  const int g16 = lane >> 4, c16 = lane & 15;
  const int nt = N == 128 ? wave & 3 : wave & 1, rt = N == 128 ? wave >> 2 : (wave >> 1) & 1;
  const bool do_c = N == 128 || wave < 4, do_b = N == 128 || wave >= 4;
  const int group = blockIdx.y / p.runs, run = blockIdx.y % p.runs;
  const int shift = p.P / 128, spp = 1 << shift;  // P is 64 or 128
  const int per_group = p.H / p.G * spp, nstrips = p.H * spp;
  const int strip0 = group * per_group + run * p.run_strips;
  const int strips_here = min(p.run_strips, per_group - run * p.run_strips);
  const int c0 = blockIdx.x * Q, c1 = min(c0 + Q, p.T);
  Offsets cu = {p.cu, nullptr};
  if (p.R < kFew) {
    if ((int)threadIdx.x <= p.R) L.window[threadIdx.x] = p.cu[threadIdx.x];
    cu.window = L.window;
  }
  // the blocks over the diagonal that operands of 32 rows reach stay zero
  for (int i = threadIdx.x; i < 2 * 16 * 2; i += kGradThreads) {
    const int r = i / 32 * 32 + i / 2 % 16, at = pipe::row_off<64>(r, i / 32 * 32 + 16 + i % 2 * 8);
    *reinterpret_cast<u32x4*>(L.M[0] + at) = *reinterpret_cast<u32x4*>(L.M[1] + at) = u32x4{0, 0, 0, 0};
  }
  for (int i = threadIdx.x; i < strips_here >> shift; i += kGradThreads) {
    const int head = (strip0 >> shift) + i;
    L.heads[i] = {param(p.a, p.p_f32, head), p.bias ? param(p.bias, p.p_f32, head) : 0.f, p.D ? param(p.D, p.p_f32, head) : 0.f};
  }
  __syncthreads();

  const bool one_run = p.runs == 1;
  const long long share = (long long)p.T * p.G * N;
  float* const shareB = p.shares + (long long)run * share;
  float* const shareC = shareB + p.runs * share;
  float* const heads = p.heads + (long long)blockIdx.x * p.H * 3;

  {  // rows of no sequence
    const int lead = p.R ? min(max(cu(0), 0), p.T) : p.T, tail = p.R ? min(max(cu(p.R), 0), p.T) : p.T;
    auto zero = [&](int r0, int r1) {
      for (int r = r0 + wave; r < r1; r += kGradWaves) {
        if (p.zero_rest) {
          for (int i = lane; i < strips_here * 8; i += 64)
            *reinterpret_cast<u32x4*>(static_cast<__bf16*>(p.gx) + r * p.gxs + strip0 * 64 + i * 8) = u32x4{0, 0, 0, 0};
          for (int i = lane; i < (strips_here >> shift); i += 64) put_param(p.gdt, p.dt_f32, (long long)r * p.H + (strip0 >> shift) + i, 0.f);
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

  Stage<N, Q, kGradWaves> sc, sb;
  StageWave<64> sx, sh;
  sc.init(p.cs, wave);
  sb.init(p.bs, wave);
  sx.init(p.xs), sh.init(p.gs);
  unsigned state_off[2];  // of the lane's pieces of rows 0 to 7 and 8 to 15 in the swizzled tile
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 8 * i + lane / 8;
    state_off[i] = state_piece(r, (pipe::row_off<64>(r, 8 * (lane % 8)) - r * 64) / 8) * 16;
  }
  const int rb64 = tile::row_base<64>(lane), cb64 = col_base8<64>(lane), cbn = col_base8<N>(lane);
  // operands of 16 rows (columns) for the products of 16 x 16 x 32: rows r0 + l % 16, values k0 + 8 (l / 16) on
  auto rows16 = [&](const __bf16* t, auto d, int r0, int k0) {
    return *reinterpret_cast<const u32x4*>(t + pipe::row_off<decltype(d)::value>(r0 + c16, k0 + 8 * g16));
  };
  // columns n0 + l % 16, rows k0 + 8 (l / 16) on
  auto cols16 = [&](const __bf16* t, int k0, int n0) {
    const int r = k0 + 8 * g16 + (c16 >> 2), e = n0 + 4 * (c16 & 3);
    return pipe::pair(pipe::ld4_tr(t + pipe::row_off<64>(r, e)), pipe::ld4_tr(t + pipe::row_off<64>(r + 4, e)));
  };

  Walk<true> walk;
  walk.init(cu, p.R, p.T, c0, c1);
  Piece pc;
  bool later = false;  // than the first piece of these rows
  for (; walk.next(pc); later = true) {
    __syncthreads();  // the piece before is done with its buffers
    const long long at = ((long long)piece_id(pc) * nstrips + strip0) * N * 64;
    // all strips of the run: what is ahead counts against the end
    const Source from_s = source(p.states[0] + at, 64, 0, N * strips_here, 64), from_z = source(p.states[1] + at, 64, 0, N * strips_here, 64);
    const Source from_x = source(static_cast<const __bf16*>(p.x) + strip0 * 64, p.xs, pc.row, pc.n, 64 * strips_here);
    const Source from_h = source(static_cast<const __bf16*>(p.go) + strip0 * 64, p.gs, pc.row, pc.n, 64 * strips_here);
    auto stage = [&](int s) {  // by one wave: others would wait in line with their loads
      auto& to = L.strip[s & 1];
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {  // 8 rows at a time: 16 rows further is 256 bytes, 32 rows 4 KB
        const int ahead = s * N * 128 + i / 4 * 4096 + (i / 2 & 1) * 256;
        load_piece(to.S + i * 512, from_s, state_off[i & 1], ahead);
        load_piece(to.Z + i * 512, from_z, state_off[i & 1], ahead);
      }
      sx.load<Q>(to.x, from_x, s * 128);
      sh.load<Q>(to.h, from_h, s * 128);
    };
    sc.load(L.C, source(static_cast<const __bf16*>(p.C) + group * N, p.cs, pc.row, pc.n, N), wave);
    sb.load(L.B, source(static_cast<const __bf16*>(p.B) + group * N, p.bs, pc.row, pc.n, N), wave);
    if (wave == kLoads) stage(0);

    // dt of the rows, a lane each: of the present and the next head (sums), of the next and the one behind that (steps)
    auto ask = [&](int head) {
      head = min(head, (strip0 + strips_here - 1) >> shift);
      return lane < pc.n ? dt_bits(p.dt, p.dt_f32, (long long)(pc.row + lane) * p.dts + head) : 0u;
    };
    auto z_of = [&](unsigned bits, int head) { return dt_of(bits, p.dt_f32) + L.heads[head - (strip0 >> shift)].bias; };
    auto a_of = [&](int head) { return L.heads[head - (strip0 >> shift)].a; };
    unsigned now = 0, next = 0;
    float total = 0.f;  // log2 of what the rows keep of a state, of the strip before
    float sum_a = 0.f, sum_q = 0.f, sum_d = 0.f, sum_k = 0.f, sum_hx = 0.f;  // of its rows, over the strips of a head
    // Sums by rows of a strip, a lane each, when all of its parts are there.
    auto by_rows = [&](int s) {
      const int strip = strip0 + s, head = strip >> shift;
      const auto& u = L.sums[s & 1];
      if ((strip & (spp - 1)) == 0) sum_a = sum_q = sum_d = sum_k = sum_hx = 0.f;
      float r = 0.f, q = 0.f, er = 0.f, ec = 0.f;
#pragma unroll
      for (int i = 0; i < N / 32; ++i) r += u.R[i][lane], q += u.Qs[i][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i <= g16) er += u.er[g16 * (g16 + 1) / 2 + i][c16];
        if (i >= g16) ec += u.ec[i * (i + 1) / 2 + g16][c16];
      }
      sum_a += (er - ec) + r;
      sum_q += q;
      sum_d += ec + u.ed[lane] + q;
#pragma unroll
      for (int i = 0; i < kGradWaves; ++i) sum_k += u.zs[64 * i + lane];
      sum_hx += u.hx[lane];
      if ((strip & (spp - 1)) == spp - 1) {
        const float behind = __shfl(pipe::wave_prefix_sum(__shfl(sum_a, 63 - lane)), 63 - lane);
        const float upto = __shfl(pipe::wave_prefix_sum(sum_q), (lane + 63) & 63);
        const float gg = behind + (lane ? upto : 0.f) + exp2_(total) * wave_sum(sum_k);
        const float z = z_of(now, head), a = a_of(head), delta = softplus(z), sig = logistic(z);
        const bool in = lane < pc.n;
        const float gz = in ? (delta > 0.f ? sum_d * (sig / delta) : 0.f) + a * gg * sig : 0.f;
        if (in) put_param(p.gdt, p.dt_f32, (long long)(pc.row + lane) * p.H + head, gz);
        const float ga = wave_sum(in ? gg * delta : 0.f), gD = wave_sum(in ? sum_hx : 0.f), gb = wave_sum(gz);
        if (lane == 0) {
          float* o = heads + head * 3;
          o[0] = later ? o[0] + ga : ga, o[1] = later ? o[1] + gD : gD, o[2] = later ? o[2] + gb : gb;
        }
      }
    };
    const int head0 = strip0 >> shift;
    if (wave == kSums) {
      now = ask(head0), next = ask(head0 + 1);
    } else if (wave == kSteps) {
      const unsigned first = ask(head0);
      now = ask(head0 + 1), next = ask(head0 + 2);
      steps(L.st[0], z_of(first, head0), a_of(head0), lane < pc.n);
    }

    f32x16 gB = zero16(), gC = zero16();
    f32x4 cb[2], wsum[2];  // C B^T of the wave's blocks, and W over the strips
    // the wave's n-th block of 16 x 16, ib >= jb
    auto block_of = [&](int n, int& ib, int& jb) {
      const int t = wave + n * kBlockWaves;
      ib = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3, jb = t - ib * (ib + 1) / 2;
    };
    auto put_parts = [&](int ib, int jb, const f32x4& v) {
      const int at = pipe::row_off<64>(16 * ib + c16, 16 * jb + 4 * g16);
      const u32x2 hi = pipe::cvt4(v);
      *reinterpret_cast<u32x2*>(L.M[0] + at) = hi;
      *reinterpret_cast<u32x2*>(L.M[1] + at) = pipe::cvt4(f32x4{v[0] - pipe::lo_f(hi[0]), v[1] - pipe::hi_f(hi[0]), v[2] - pipe::lo_f(hi[1]),
                                                                v[3] - pipe::hi_f(hi[1])});
    };

    for (int s = 0; s < strips_here; ++s) {
      const int strip = strip0 + s, head = strip >> shift, b = s & 1;
      tile::staged_barrier();
      now = arrived(now), next = arrived(next);
      unsigned after = next;
      if (wave == kSums ? s && (strip & (spp - 1)) == 0 : wave == kSteps && ((strip + 1) & (spp - 1)) == 0)
        after = ask(wave == kSums ? head + 1 : head + 3);
      if (wave == kLoads && s + 1 < strips_here) stage(s + 1);
      const Steps& st = L.st[(head - (strip0 >> shift)) & 1];
      const __bf16 *St = L.strip[b].S, *Zt = L.strip[b].Z, *Xt = L.strip[b].x, *Ht = L.strip[b].h;
      auto& sums = L.sums[b];
      if (wave < kBlockWaves) {
        // two blocks, one's steps between the other's: rows j as elements 4 g16 + r, rows i as lanes
        int ib[2], jb[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) block_of(n, ib[n], jb[n]);
        if (s == 0) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            cb[n] = wsum[n] = pipe::zero4();
#pragma unroll
            for (int k = 0; k < N / 32; ++k)
              cb[n] = pipe::mma32(rows16(L.B, pipe::ic<N>{}, 16 * jb[n], 32 * k), rows16(L.C, pipe::ic<N>{}, 16 * ib[n], 32 * k), cb[n]);
          }
        }
        f32x4 w[2], x[2];
        float row[2], column[2], diagonal[2], hx[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          w[n] = pipe::zero4();
#pragma unroll
          for (int k = 0; k < 2; ++k)
            w[n] = pipe::mma32(rows16(Xt, pipe::ic<64>{}, 16 * jb[n], 32 * k), rows16(Ht, pipe::ic<64>{}, 16 * ib[n], 32 * k), w[n]);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const bool off = ib[n] != jb[n];
          const float gi = st.G[16 * ib[n] + c16];
          const float4 u4 = *reinterpret_cast<const float4*>(st.u + 16 * jb[n] + 4 * g16);
          const float u[4] = {u4.x, u4.y, u4.z, u4.w};
          f32x4 m, e;
          hx[n] = c16 & 2 ? (c16 & 1 ? w[n][3] : w[n][2]) : (c16 & 1 ? w[n][1] : w[n][0]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 4 * g16 + r;  // against lane c16 where rows i and j are the same ones
            const float l = off || j <= c16 ? exp2_(gi + u[r]) : 0.f;
            m[r] = cb[n][r] * l;
            x[n][r] = w[n][r] * m[r];
            e[r] = off || j < c16 ? x[n][r] : 0.f;
            wsum[n][r] = __builtin_fmaf(w[n][r], l, wsum[n][r]);
          }
          diagonal[n] = c16 & 2 ? (c16 & 1 ? x[n][3] : x[n][2]) : (c16 & 1 ? x[n][1] : x[n][0]);
          put_parts(ib[n], jb[n], m);
          row[n] = row_sums(((e[0] + e[1]) + e[2]) + e[3]);
          column[n] = column_sums(e);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int t = wave + n * kBlockWaves;
          if (g16 == 0) sums.er[t][c16] = row[n];
          if (c16 < 4) sums.ec[t][4 * g16 + c16] = column[n];
          if (ib[n] == jb[n] && g16 == c16 / 4) sums.ed[16 * ib[n] + c16] = diagonal[n], sums.hx[16 * ib[n] + c16] = hx[n];
        }
      } else if (wave == kSums) {
        if (s) {
          by_rows(s - 1);
          if ((strip & (spp - 1)) == 0) now = next, next = after;
        }
        total = st.total;
      }
      if (wave == kSteps && ((strip + 1) & (spp - 1)) == 0 && s + 1 < strips_here) {
        steps(L.st[(head + 1 - (strip0 >> shift)) & 1], z_of(now, head + 1), a_of(head + 1), lane < pc.n);
        now = next, next = after;
      }
      {  // <Z, S>
        float dot = 0.f;
        const u32x4* s4 = reinterpret_cast<const u32x4*>(St) + threadIdx.x;
        const u32x4* z4 = reinterpret_cast<const u32x4*>(Zt) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < N * 64 / 8 / kGradThreads; ++i) {
          const u32x4 u = s4[i * kGradThreads], v = z4[i * kGradThreads];
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = dot2(u[e], v[e], dot);
        }
        sums.zs[threadIdx.x] = dot;
      }
      const int pt = wave & 1, rb = wave >> 1;
      f32x4 u[2] = {pipe::zero4(), pipe::zero4()};
      {  // gx: 32 channels by 16 rows, as two tiles of 16
#pragma unroll
        for (int k = 0; k < N / 32; ++k) {
          const u32x4 rows = rows16(L.B, pipe::ic<N>{}, 16 * rb, 32 * k);
#pragma unroll
          for (int i = 0; i < 2; ++i) u[i] = pipe::mma32(cols16(Zt, 32 * k, 32 * pt + 16 * i), rows, u[i]);
        }
        const float kb = st.w[16 * rb + c16];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) u[i][e] *= kb;
      }
      // gC and gB: elements n, lanes rows
      const int row = 32 * rt + col;
      auto inter = [&](f32x16& acc, const __bf16* states, const __bf16* rows, float scale, const __bf16* with, float* out) {
        f32x16 u = zero16();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          u = tile::mma(tile::row_frag<64>(states, rb64, 32 * nt, k), tile::row_frag<64>(rows, rb64, 32 * rt, k), u);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u32x2 v = pipe::ld4(with + pipe::row_off<N>(row, 32 * nt + 8 * i + 4 * half));
          const float f[4] = {pipe::lo_f(v[0]), pipe::hi_f(v[0]), pipe::lo_f(v[1]), pipe::hi_f(v[1])};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sum = __builtin_fmaf(u[4 * i + j], f[j], sum);
            acc[4 * i + j] = __builtin_fmaf(u[4 * i + j], scale, acc[4 * i + j]);
          }
        }
        sum = tile::sum_halves(sum) * scale;
        if (half == 0) out[row] = sum;
      };
      if (do_c) inter(gC, St, Ht, exp2_(st.G[row]), L.C, sums.R[nt]);
      if (do_b) inter(gB, Zt, Xt, st.w[row], L.B, sums.Qs[nt]);
      lds_barrier();

      {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (k >= rb / 2) {
            const u32x4 m0 = cols16(L.M[0], 32 * k, 16 * rb), m1 = cols16(L.M[1], 32 * k, 16 * rb);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const u32x4 h = cols16(Ht, 32 * k, 32 * pt + 16 * i);
              u[i] = pipe::mma32(h, m0, u[i]);
              u[i] = pipe::mma32(h, m1, u[i]);
            }
          }
        const float dskip = L.heads[head - (strip0 >> shift)].D;
        __bf16* const mine = L.strip[b].S + wave * 512;  // S has been used: on the way to memory
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const u32x2 hv = pipe::ld4(Ht + pipe::row_off<64>(16 * rb + c16, 32 * pt + 16 * i + 4 * g16));
          u32x2 w;
          w[0] = pipe::cvt2(__builtin_fmaf(dskip, pipe::lo_f(hv[0]), u[i][0]), __builtin_fmaf(dskip, pipe::hi_f(hv[0]), u[i][1]));
          w[1] = pipe::cvt2(__builtin_fmaf(dskip, pipe::lo_f(hv[1]), u[i][2]), __builtin_fmaf(dskip, pipe::hi_f(hv[1]), u[i][3]));
          *reinterpret_cast<u32x2*>(mine + c16 * 32 + 16 * i + 4 * g16) = w;
        }
        pipe::issue_fence();
        const int row = 16 * rb + lane / 4;
        const u32x4 v = *reinterpret_cast<const u32x4*>(mine + lane * 8);
        if (row < pc.n)
          *reinterpret_cast<u32x4*>(static_cast<__bf16*>(p.gx) + (long long)(pc.row + row) * p.gxs + strip * 64 + 32 * pt + lane % 4 * 8) = v;
      }
    }
    lds_barrier();  // the last M has been used
    if (wave < kBlockWaves) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        int ib, jb;
        block_of(n, ib, jb);
        put_parts(ib, jb, wsum[n]);
      }
    } else if (wave == kSums) {
      by_rows(strips_here - 1);
    }
    lds_barrier();
    if (do_c)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < 2 * rt + 2) {
          const u32x4 b = col_frag8<N>(L.B, cbn, 16 * k, nt);
#pragma unroll
          for (int q = 0; q < 2; ++q) gC = tile::mma(b, tile::row_frag<64>(L.M[q], rb64, 32 * rt, k), gC);
        }
    if (do_b)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k >= 2 * rt) {
          const u32x4 c = col_frag8<N>(L.C, cbn, 16 * k, nt);
#pragma unroll
          for (int q = 0; q < 2; ++q) gB = tile::mma(c, col_frag8<64>(L.M[q], cb64, 16 * k, rt), gB);
        }

    // gB and gC: lanes are rows, elements n = 32 nt + 8 q + 4 half + j
    const int row = 32 * rt + col;
    if (row < pc.n) {
      const long long r = pc.row + row;
      const int n = group * N + 32 * nt + 4 * half;
      auto put = [&](const f32x16& v, void* rows, long long stride, float* shares) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (one_run)
            *reinterpret_cast<u32x2*>(static_cast<__bf16*>(rows) + r * stride + n + 8 * q) =
                u32x2{pipe::cvt2(v[4 * q], v[4 * q + 1]), pipe::cvt2(v[4 * q + 2], v[4 * q + 3])};
          else
            *reinterpret_cast<f32x4*>(shares + r * p.G * N + n + 8 * q) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        }
      };
      if (do_b) put(gB, p.gB, p.gbs, shareB);
      if (do_c) put(gC, p.gC, p.gcs, shareC);
    }
  }
  if (!later)
    for (int i = threadIdx.x; i < (strips_here >> shift) * 3; i += kGradThreads) heads[(strip0 >> shift) * 3 + i] = 0.f;
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
  // segments: three workgroups for every two CUs, both directions counted, of at least four pieces; where the sequences
  // would be as long as each other and as a number of pieces, whole ones, whose states need not be joined
  const int want = nstrips >= 192 ? 1 : 192 / nstrips;
  int per = (w.blocks + want - 1) / want;
  if (want > 1 && R > 1 && T % R == 0 && T / R % Q == 0 && 2 * (T / R) >= per * Q && T / R <= 2 * per * Q) per = T / R / Q;
  if (per < 4) per = 4;
  w.seg = per * Q;
  w.nseg = T > w.seg ? (T + w.seg - 1) / w.seg : 1;
  // runs of strips: the fewest rounds of workgroups over the CUs, weighed by their length
  const int heads = H / G, base = w.blocks * G;
  long long best = -1;
  const int few = (heads + kMostHeads - 1) / kMostHeads;
  for (int n = few; n <= heads && n < few + 1024; ++n) {
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
  const int nstrips = n.H * (n.P / 64), per = nstrips * (n.N / kHalf);
  const int idle = a.grad_S0 ? idle_segments(n.R, 768 / per - 2 * w.nseg) : 0;  // three workgroups to a CU
  BwdParams p = {a.x, a.dt, a.a, a.B, a.C, a.D, a.bias, a.grad_out, a.cu, a.S0, a.grad_S_final, a.grad_x, a.grad_dt, a.grad_a,
                 a.grad_B, a.grad_C, a.grad_D, a.grad_bias, a.grad_S0,
                 {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + w.share)},
                 {reinterpret_cast<__bf16*>(ws + 2 * w.share), reinterpret_cast<__bf16*>(ws + 2 * w.share + w.states)},
                 reinterpret_cast<float*>(ws + 2 * w.share + 2 * w.states + w.heads),
                 reinterpret_cast<float*>(ws + 2 * w.share + 2 * w.states), a.xs, a.dts, a.bs, a.cs, a.gs, a.gxs, a.gbs, a.gcs,
                 n.T, n.R, n.H, n.P, n.G, w.seg, w.nseg, idle, w.runs, w.run_strips, n.dt_f32, n.p_f32, a.zero_rest};
  auto go = [&](auto nn, auto parts) {
    constexpr int N = decltype(nn)::value, PARTS = decltype(parts)::value;
    if (w.nseg > 1) {
      hipLaunchKernelGGL((states_kernel<N, true, PARTS>), dim3(per * (w.nseg - 1) * 2), dim3(kStateThreads), 0, stream, p);
      if (const hipError_t e = hipGetLastError()) return e;
      hipLaunchKernelGGL((join_both_kernel<N>), dim3(N * 64 / 1024, nstrips, 2), dim3(256), 0, stream, p.seg_ws[0], p.seg_ws[1],
                         nstrips, w.nseg - 1);
      if (const hipError_t e = hipGetLastError()) return e;
    }
    hipLaunchKernelGGL((states_kernel<N, false, PARTS>), dim3(per * (w.nseg * 2 + idle)), dim3(kStateThreads), 0, stream, p);
    if (const hipError_t e = hipGetLastError()) return e;
    if (w.blocks) {
      hipLaunchKernelGGL((grad_kernel<N>), dim3(w.blocks, n.G * w.runs), dim3(kGradThreads), 0, stream, p);
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
