// attn_prompt.hip -- causal attention over packed prompts, forward.
//
// For row i and the keys j of its sequence up to itself,
//   s_ij = scale q_i.k_j,   o_i = sum_j e^(s_ij) v_j / sum_j e^(s_ij),   lse_i = log sum_j e^(s_ij),
// in one pass over the keys with a running maximum m and sum.  The maximum in
// use is renewed only once a score lies 2^8 above it: sums and weights are then
// at most 2^8, which float32 and bf16 hold as well as 1, and most tiles skip the
// rescaling of the accumulators.
//
// A workgroup takes 128 rows of one head, a wave 32 of them; S^T = K Q^T and
// O^T = V^T P^T by 32x32x16 products, so that a row is a lane's column: its
// maximum and sum take one exchange of half-waves, and the weights, rounded to
// bf16 (2^-8 of each, the operands' own precision; in two parts, the rounded and what
// the rounding leaves, 18 to 35 % more time), go from accumulator to operand in place.  K and V are staged in LDS by direct loads, one tile ahead,
// and read there by rows (K) and transposed (V).  Rows are cut into tiles where
// they lie, whatever sequences they belong to: tiles that some row sees in part
// are masked, those that all rows see whole are not.  The workgroups of the
// heads that share keys are neighbours.
//
// What bounds it is the matrix and the vector unit together: 32 keys of a wave's
// 32 rows are 4 D / 32 products of 32 cycles and 16 lanes' exponentials, with as
// many multiply-adds, sums and maxima.  1 x 16384 x 16/4 x 64 takes 578 to 605 us, 910
// to 950 TFLOP/s of the 1600 that the largest library products reach here; 8 x 2048 x
// 12/4 x 64 71 to 79 us (a fifth of the CUs' time goes by waiting for the longest
// tiles); 1 x 16384 x 16/4 x 128 1030 to 1130 us, 970 to 1060 TFLOP/s.  Without the softmax the same
// loop reaches 1190, without the reads of LDS 1215.  Two tiles of rows to a wave,
// the next scores beside the softmax, eight waves, orders set by hand and other
// wave priorities were all slower or the same.
#include "../../include/gdn.h"
#include "gdn_attn.hpp"
#include "gdn_launch.hpp"
#include "gdn_tile.hpp"

namespace gdn {
namespace {

using namespace tile;

constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;
constexpr float kLowest = -3e38f;  // running maximum before the first token
constexpr float kSlack = 8.f;      // the maximum in use may lie this far (powers of two) below the true one

// What a wave carries over the keys: lane l has row l % 32, its output columns
// as in the accumulators; m is shared by the two lanes of a row, l is the lane's
// own part.
template <int D> struct Rows {
  f32x16 o[D / 32];
  float m, l;
  __device__ __forceinline__ void clear() {
    m = kLowest;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = zero16();
  }
};

// One staged tile of 32 NH keys; MASKED: only keys from .. upto (less 4 hl) of it
// are seen by the lane's row.
// keys_done() is called when the keys have been read, values_due() before the values are.
template <int D, int NH, bool MASKED, class F, class G>
__device__ __forceinline__ void take_keys(Rows<D>& x, const __bf16* kt, const __bf16* vt, int kb0, int vb0,
                                          const u32x4 (&q)[D / 16], float c, int from, int upto, F keys_done, G values_due) {
  constexpr int KS = D / 16, DT = D / 32;
  const int kb = fresh(kb0), vb = fresh(vb0);
  f32x16 s[NH];
#pragma unroll
  for (int n = 0; n < NH; ++n) {
    s[n] = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) s[n] = mma(row_frag<D>(kt, kb, 32 * n, ks), q[ks], s[n]);
  }
  keys_done();
  if constexpr (MASKED) {
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      const unsigned seen = bits(from - 32 * n, upto - 32 * n);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[n][e] = where_seen<false>(s[n][e], seen, e);
    }
  }
  float top = s[0][0];
#pragma unroll
  for (int n = 0; n < NH; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, s[n][e]);
  top = max_halves(top) * c;
  if (__any(top > x.m + kSlack)) {
    const float to = fmaxf(x.m, top), f = __builtin_amdgcn_exp2f(x.m - to);
    x.m = to;
    x.l *= f;
#pragma unroll
    for (int i = 0; i < DT; ++i) x.o[i] *= f;
  }
  u32x4 p[2 * NH];
  float sum = 0.f;
#pragma unroll
  for (int n = 0; n < NH; ++n) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      s[n][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][e], c, -x.m));
      sum += s[n][e];
    }
    p[2 * n] = operand(s[n], 0);
    p[2 * n + 1] = operand(s[n], 1);
  }
  x.l += sum;
  values_due();
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int b = 0; b < 2 * NH; ++b) x.o[i] = mma(col_frag<D>(vt, vb, 16 * b, i), p[b], x.o[i]);
}

// Where rows lo .. hi - 1 of V hold values that are not finite.
template <int D, int N, int NT>
__device__ __forceinline__ void mark_values(Marks<D, N>& up, Marks<D, N>& down, const void* v, long long stride, int lo,
                                            int hi, int r0) {
  up.template clear<NT>();
  down.template clear<NT>();
  __syncthreads();
  up.template look<NT, Kind::up>(v, stride, lo, hi, r0);
  down.template look<NT, Kind::down>(v, stride, lo, hi, r0);
  __syncthreads();
}
__device__ __forceinline__ float with_infinities(float x, bool up, bool down) {
  if (up) x += INFINITY;
  if (down) x -= INFINITY;
  return x;
}

// NW / KP waves of a workgroup take 32 rows each; KP = 2: the others the same rows
// and the second half of each tile's keys, added at the end.  That halves a row's
// chain of tiles for twice the reads of keys (1 x 5000 x 16/4 x 128 140 us for 174,
// 2 x 2000 55 for 75, 1 x 8000 319 for 301).
template <int D, int NW, int KP> __global__ __launch_bounds__(64 * NW, D == 64 ? 4 : KP == 1 ? 3 : 2) void attn_prompt_kernel(PromptArgs a) {
  // keys of a staged tile: 64 at D = 64, where 125 registers let four workgroups
  // share a CU (578 us for 1 x 16384 x 16/4 x 64; with 32 keys 620); 32 at
  // D = 128, where that takes 158 registers and three workgroups a CU (67.7 us for
  // 13 prompts of up to 1201 rows x 16/4 x 128; with 64 keys and two 70.5)
  constexpr int kN = D == 64 ? 64 : 32 * KP, NH = kN / 32 / KP;
  constexpr int RW = NW / KP, BM = 32 * RW, NT = 64 * NW, KS = D / 16, DT = D / 32;
  __shared__ union alignas(16) {
    struct {
      __bf16 k[2][kN * D], v[2][kN * D];
    } staged;
    float part[KP == 2 ? RW : 1][32][D + 4];
  } mem;
  auto &kt = mem.staged.k, &vt = mem.staged.v;
  __shared__ float ml[2][BM];
  __shared__ int begs[BM], window[kWindow], ranges[3][NW], bad[2][NW];
  __shared__ Marks<D, BM> up, down;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  const int tiles = (a.T + BM - 1) / BM;
  // the tiles with the most keys (of a long sequence: the last) first, all heads of a tile side by side
  const int rank = blockIdx.x / a.Hq, hq = blockIdx.x - rank * a.Hq;
  int tile = tiles - 1 - rank;
  if (a.by_length) tile = tile_by_length<BM, NT, false>(a.cu, a.R, a.T, tiles, rank, window, reinterpret_cast<int*>(kt));
  const int r0 = tile * BM, kvh = hq / (a.Hq / a.Hkv);

  // queries: operands for the wave's rows
  const int part = wave / RW, ko = 32 * NH * part, w0 = r0 + (wave - part * RW) * 32, row = w0 + (lane & 31);
  u32x4 q[KS];
  find_rows<BM, NT>(a.cu, a.R, a.T, r0, window, begs, nullptr, [&] {
    const __hip_bfloat16* src =
        static_cast<const __hip_bfloat16*>(a.q) + (long long)min(row, a.T - 1) * a.qs + (long long)hq * D + 8 * hl;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks] = *reinterpret_cast<const u32x4*>(src + 16 * ks);
  });
  // the keys that the tile's rows see, and the last beginning of a sequence among them
  const int beg = begs[row - r0];
  int lowest = beg < 0 ? a.T : beg, highest = lowest, last = beg < 0 ? -1 : row + 1;
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    lowest = min(lowest, __shfl_xor(lowest, d));
    highest = max(highest, __shfl_xor(highest, d));
    last = max(last, __shfl_xor(last, d));
  }
  if (lane == 0) {
    ranges[0][wave] = lowest;
    ranges[1][wave] = highest;
    ranges[2][wave] = last;
  }
  __syncthreads();
  int first = a.T, latest = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    first = min(first, ranges[0][w]);
    latest = max(latest, ranges[1][w]);
    last = max(last, ranges[2][w]);
  }
  lowest = __builtin_amdgcn_readfirstlane(lowest);  // of the wave's rows
  highest = __builtin_amdgcn_readfirstlane(highest);
  first = __builtin_amdgcn_readfirstlane(first);
  latest = __builtin_amdgcn_readfirstlane(latest);
  last = __builtin_amdgcn_readfirstlane(last);
  if (last < 0) {  // no row of the tile is in a sequence
    if (a.zero_rest) {
      zero_rows<D>(static_cast<__bf16*>(a.out) + (long long)hq * D, (long long)a.Hq * D, r0, min(BM, a.T - r0), NT);
      for (int i = tid; i < BM && r0 + i < a.T; i += NT) a.lse[(size_t)hq * a.T + r0 + i] = 0.f;
    }
    return;
  }

  // a scale of zero stays just above it, so that masked scores, -infinity, keep
  // a weight of zero; for a negative one the queries' signs are turned
  const float c = fmaxf(__builtin_fabsf(a.scale) * kLog2e, 1e-37f);
  const unsigned flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) q[ks] ^= flip;
  const int from = beg - 4 * hl, upto = beg < 0 ? -8 : row - 4 * hl;  // the keys that the lane's row sees, less 4 hl

  Rows<D> x;
  x.clear();

  const int kb0 = row_base<D>(lane), vb0 = col_base<D>(lane);
  Stage<D, kN, NW> sk, sv;
  sk.init(a.ks, wave);
  sv.init(a.vs, wave);
  const __hip_bfloat16* kp = static_cast<const __hip_bfloat16*>(a.k) + (long long)kvh * D;
  const __hip_bfloat16* vp = static_cast<const __hip_bfloat16*>(a.v) + (long long)kvh * D;
  auto stage = [&](int buf, int kv) {
    const int n = min(kN, last - kv);
    sk.load(kt[buf], rows_rsrc(kp, a.ks, kv, n, D), wave);
    sv.load(vt[buf], rows_rsrc(vp, a.vs, kv, n, D), wave);
  };
  // the tiles whose non-finite values were left out: some row may not see them,
  // and its weight of zero must not meet them; they are added to the rows that
  // see them when all is written
  int dirty_lo = last, dirty_hi = 0;
  stage(0, first);
  int buf = 0, kv = first;
  auto next = [&] {
    const bool masked = kv + kN - 1 > r0 || kv < latest || kv + kN > last;  // for some wave
    if (masked) {
      wait_staged();
      const bool ok = Stage<D, kN, NW>::scrub(vt[buf], wave);
      if (lane == 0) bad[buf][wave] = !ok;
    }
    staged_barrier();
    if (masked && !all_clean(bad[buf])) {
      dirty_lo = min(dirty_lo, kv);
      dirty_hi = kv + kN;
    }
    if (kv + kN < last) stage(buf ^ 1, kv + kN);
  };
  // where the tiles that the wave's rows see whole end (a wave none of whose rows is
  // in a sequence may lie behind the last tile: it takes no more than the others,
  // with whom it shares the barriers)
  const int whole = min(w0 + 1, last);
  // tiles of which some row misses some key, at both ends of the range, and
  // those between, which all rows see whole (loops apart: one loop with both
  // bodies takes more registers than there are)
  auto edge = [&](int end) {
    for (; kv < end; kv += kN, buf ^= 1) {
      next();
      const int at = kv + ko;
      if (at <= w0 + 31 && at + 32 * NH > lowest) take_keys<D, NH, true>(x, kt[buf] + ko * D, vt[buf] + ko * D, kb0, vb0, q, c, from - at, upto - at, [] {}, [] {});
    }
  };
  edge(min(highest, last));
  for (; kv + kN <= whole; kv += kN, buf ^= 1) {
    next();
    take_keys<D, NH, false>(x, kt[buf] + ko * D, vt[buf] + ko * D, kb0, vb0, q, c, 0, 0, [] {}, [] {});
  }
  edge(last);
  if (dirty_hi) mark_values<D, BM, NT>(up, down, vp, a.vs, dirty_lo, min(dirty_hi, last), r0);

  float z = sum_halves(x.l);
  if constexpr (KP == 2) {  // the second half of each tile's keys, handed to the waves of the first
    const int r = row - r0;
    __syncthreads();
    if (part) {
      if (hl == 0) {
        ml[0][r] = x.m;
        ml[1][r] = z;
      }
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<f32x4*>(&mem.part[r / 32][r % 32][32 * i + 8 * e + 4 * hl]) =
              f32x4{x.o[i][4 * e], x.o[i][4 * e + 1], x.o[i][4 * e + 2], x.o[i][4 * e + 3]};
    }
    __syncthreads();
    if (part) return;
    const float m = fmaxf(x.m, ml[0][r]), f = __builtin_amdgcn_exp2f(x.m - m), g = __builtin_amdgcn_exp2f(ml[0][r] - m);
    x.m = m;
    z = z * f + ml[1][r] * g;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(&mem.part[r / 32][r % 32][32 * i + 8 * e + 4 * hl]);
#pragma unroll
        for (int j = 0; j < 4; ++j) x.o[i][4 * e + j] = x.o[i][4 * e + j] * f + y[j] * g;
      }
  }
  const bool rest = beg < 0 && row < a.T && a.zero_rest;
  if (beg < 0 && !rest) return;
  const float inv = rest ? 0.f : 1.f / z;
  __bf16* dst = static_cast<__bf16*>(a.out) + ((size_t)row * a.Hq + hq) * D;
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<u32x2*>(dst + 32 * i + 8 * e + 4 * hl) =
          pipe::cvt4(f32x4{x.o[i][4 * e] * inv, x.o[i][4 * e + 1] * inv, x.o[i][4 * e + 2] * inv, x.o[i][4 * e + 3] * inv});
  if (hl == 0) a.lse[(size_t)hq * a.T + row] = rest ? 0.f : (x.m + __builtin_amdgcn_logf(z)) * kLn2;
  if (rest || !dirty_hi) return;
  const int lo = max(beg - r0, 0), hi = row - r0 + 1;
  for (int w = 0; w < DT; ++w) {
    const unsigned u = up.columns(w, lo, hi, beg < r0), n = down.columns(w, lo, hi, beg < r0);
    if (u | n)
      for (int d = 4 * hl; d < 32; d += 8)  // the entries that this lane stored
        for (int i = d; i < d + 4; ++i) dst[32 * w + i] = (__bf16)with_infinities((float)dst[32 * w + i], u >> i & 1, n >> i & 1);
  }
}

// Few rows: a workgroup takes 32 rows of one head and its waves every NW-th tile
// of their keys, each staging its own and waiting for nobody; what they have is
// joined through LDS at the end.  A row's chain of tiles is a quarter as long for
// four times the reads of keys: 1 x 1000 x 16/4 x 128 15.6 us for 36.2, 1 x 2500
// x 12/4 x 64 25 for 50, 1 x 131 5.2 for 6.6; 8 x 2048 112 for 75.
template <int D, int NW> __global__ __launch_bounds__(64 * NW, D == 64 ? 4 : 2) void attn_prompt_split_kernel(PromptArgs a) {
  constexpr int kN = 32, NT = 64 * NW, KS = D / 16, DT = D / 32, LD = D + 4;
  __shared__ union alignas(16) {
    __bf16 staged[NW][2][kN * D];
    float part[NW][32][LD];
  } mem;
  auto& part = mem.part;
  __shared__ float ml[NW][2][32];
  __shared__ int begs[32], window[kWindow], dirty[2][NW];
  __shared__ Marks<D, 32> up, down;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  const int tiles = (a.T + 31) / 32;
  const int rank = blockIdx.x / a.Hq, hq = blockIdx.x - rank * a.Hq;
  const int r0 = (tiles - 1 - rank) * 32, kvh = hq / (a.Hq / a.Hkv);

  const int row = r0 + (lane & 31);
  u32x4 q[KS];
  find_rows<32, NT>(a.cu, a.R, a.T, r0, window, begs, nullptr, [&] {
    const __hip_bfloat16* src =
        static_cast<const __hip_bfloat16*>(a.q) + (long long)min(row, a.T - 1) * a.qs + (long long)hq * D + 8 * hl;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks] = *reinterpret_cast<const u32x4*>(src + 16 * ks);
  });
  const int beg = begs[row - r0];
  const KeyRange range = key_range(beg, row, a.T);
  const int first = range.first, latest = range.latest, last = range.last;
  if (last < 0) {  // no row of the tile is in a sequence
    if (a.zero_rest) {
      zero_rows<D>(static_cast<__bf16*>(a.out) + (long long)hq * D, (long long)a.Hq * D, r0, min(32, a.T - r0), NT);
      if (tid < 32 && r0 + tid < a.T) a.lse[(size_t)hq * a.T + r0 + tid] = 0.f;
    }
    return;
  }
  const float c = fmaxf(__builtin_fabsf(a.scale) * kLog2e, 1e-37f);
  const unsigned flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) q[ks] ^= flip;
  const int from = beg - 4 * hl, upto = beg < 0 ? -8 : row - 4 * hl;

  Rows<D> x;
  x.clear();
  const int kb0 = row_base<D>(lane), vb0 = col_base<D>(lane);
  Stage<D, kN, 1> sk, sv;
  sk.init(a.ks, 0);
  sv.init(a.vs, 0);
  const __hip_bfloat16* kp = static_cast<const __hip_bfloat16*>(a.k) + (long long)kvh * D;
  const __hip_bfloat16* vp = static_cast<const __hip_bfloat16*>(a.v) + (long long)kvh * D;
  // one buffer each: the next keys are on their way while the values are used,
  // the next values while the keys are, so that more workgroups share a CU
  __bf16 *kt = mem.staged[wave][0], *vt = mem.staged[wave][1];
  auto stage_keys = [&](int kv) { sk.load(kt, rows_rsrc(kp, a.ks, kv, min(kN, last - kv), D), 0); };
  auto stage_values = [&](int kv) { sv.load(vt, rows_rsrc(vp, a.vs, kv, min(kN, last - kv), D), 0); };
  constexpr int kLoads = Stage<D, kN, 1>::LOADS;
  int dirty_lo = last, dirty_hi = 0, kv = first + kN * wave;
  if (kv < last) {
    stage_keys(kv);
    stage_values(kv);
  }
  for (; kv < last; kv += kN * NW) {
    const int to = kv + kN * NW;
    wait_all_but<kLoads>();
    auto keys_done = [&] {
      if (to < last) {
        wait_read();
        stage_keys(to);
      }
    };
    auto values_due = [&] {
      if (to < last) wait_all_but<kLoads>();
      else wait_all_but<0>();
    };
    if (kv + kN - 1 > r0 || kv < latest || kv + kN > last) {
      take_keys<D, 1, true>(x, kt, vt, kb0, vb0, q, c, from - kv, upto - kv, keys_done, [&] {
        values_due();
        if (!Stage<D, kN, 1>::scrub(vt, 0)) {
          dirty_lo = min(dirty_lo, kv);
          dirty_hi = kv + kN;
        }
      });
    } else {
      take_keys<D, 1, false>(x, kt, vt, kb0, vb0, q, c, 0, 0, keys_done, values_due);
    }
    if (to < last) {
      wait_read();
      stage_values(to);
    }
  }

  const float z = sum_halves(x.l);
  if (lane < 32) {
    ml[wave][0][lane] = x.m;
    ml[wave][1][lane] = z;
  }
  if (lane == 0) {
    dirty[0][wave] = dirty_lo;
    dirty[1][wave] = dirty_hi;
  }
  __syncthreads();
  {
    float M = ml[0][0][lane & 31];
#pragma unroll
    for (int w = 1; w < NW; ++w) M = fmaxf(M, ml[w][0][lane & 31]);
    const float f = __builtin_amdgcn_exp2f(x.m - M);
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(&part[wave][lane & 31][32 * i + 8 * e + 4 * hl]) =
            f32x4{x.o[i][4 * e] * f, x.o[i][4 * e + 1] * f, x.o[i][4 * e + 2] * f, x.o[i][4 * e + 3] * f};
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    dirty_lo = min(dirty_lo, dirty[0][w]);
    dirty_hi = max(dirty_hi, dirty[1][w]);
  }
  if (dirty_hi) mark_values<D, 32, NT>(up, down, vp, a.vs, dirty_lo, min(dirty_hi, last), r0);
  for (int i = tid; i < 32 * (D / 4); i += NT) {
    const int r = i / (D / 4), d = i % (D / 4) * 4, b = begs[r];
    if (r0 + r >= a.T || (b < 0 && !a.zero_rest)) continue;
    float M = ml[0][0][r], L = 0.f;
#pragma unroll
    for (int w = 1; w < NW; ++w) M = fmaxf(M, ml[w][0][r]);
    f32x4 o = pipe::zero4();
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      L += ml[w][1][r] * __builtin_amdgcn_exp2f(ml[w][0][r] - M);
      o += *reinterpret_cast<const f32x4*>(&part[w][r][d]);
    }
    o *= 1.f / L;
    if (dirty_hi && b >= 0) {
      const int lo = max(b - r0, 0);
      const unsigned u = up.columns(d / 32, lo, r + 1, b < r0), n = down.columns(d / 32, lo, r + 1, b < r0);
      for (int j = 0; j < 4; ++j) o[j] = with_infinities(o[j], u >> (d % 32 + j) & 1, n >> (d % 32 + j) & 1);
    }
    if (b < 0) o = pipe::zero4();
    *reinterpret_cast<u32x2*>(static_cast<__bf16*>(a.out) + ((size_t)(r0 + r) * a.Hq + hq) * D + d) = pipe::cvt4(o);
    if (d == 0) a.lse[(size_t)hq * a.T + r0 + r] = b < 0 ? 0.f : (M + __builtin_amdgcn_logf(L)) * kLn2;
  }
}

template <int D> hipError_t launch(const PromptArgs& a) {
  constexpr int NW = 4;
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  if (split_keys(a.T, a.R, a.Hq, D)) {
    const dim3 grid((unsigned)((a.T + 31) / 32 * a.Hq));
    if constexpr (D == 64)
      // few workgroups with long chains: eight waves (1 x 600 x 12/4 x 64 6.9 us for
      // 8.3 with four, 4 x 512 13.3 for 10.3)
      if (grid.x <= 512 && a.T >= 256LL * a.R) return launch_kernel(attn_prompt_split_kernel<D, 8>, grid, dim3(512), st, a);
    return launch_kernel(attn_prompt_split_kernel<D, 4>, grid, dim3(256), st, a);
  }
  if constexpr (D == 128)
    if (split_halves(a.T, a.R, a.Hq)) {
      PromptArgs b = a;
      b.by_length = false;
      return launch_kernel(attn_prompt_kernel<D, NW, 2>, dim3((unsigned)((a.T + 63) / 64 * a.Hq)), dim3(64 * NW), st, b);
    }
  const unsigned tiles = (unsigned)((a.T + 32 * NW - 1) / (32 * NW));
  return launch_kernel(attn_prompt_kernel<D, NW, 1>, dim3(tiles * a.Hq), dim3(64 * NW), st, a);
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& args) {
  PromptArgs a = args;
  a.by_length = rank_tiles(a.T, a.R, a.Hq);
  return a.D == 64 ? launch<64>(a) : launch<128>(a);
}

}  // namespace gdn
