// attn_prompt_bwd.hip -- gradients of causal attention over packed prompts.
//
// With p_ij = exp(scale q_i.k_j - lse_i) for the keys j that row i attends to,
//   delta_i = do_i . o_i,     dv_j = sum_i p_ij do_i,
//   ds_ij = p_ij (do_i . v_j - delta_i),
//   dq_i = scale sum_j ds_ij k_j,     dk_j = scale sum_i ds_ij q_i,
// dk and dv summed over the query heads that share key head j's.
//
// One launch by tiles of rows for dq (three products for a pair of tiles), one
// by tiles of keys for dk and dv (four), each of which owns the sums it writes,
// so that their order is fixed.  The probabilities are computed in both; the
// first launch leaves lse (times log2 e) and -delta, which the second's products
// start from, in the workspace.  Where there are few keys to share out, the
// query heads of a key head are shared out too, and a third launch adds their
// sums.  (Five products in one launch, dq added up with atomics, would read and
// exponentiate half as often but make the order of dq's sums one of arrival.)
//
// p and ds are rounded to bf16 where they enter a product, 2^-8 of each; for dq, ds
// is taken in two parts, the rounded and what the rounding left (2^-16 of it):
// with one, dq's relative error is 2.5e-3, half as much again as that of rounding
// the result (1.7e-3), with two 1.9e-3, for a fourth product in place of three (4
// to 8 % of the time of forward and gradients).  dk has 2.4e-3 and dv 2.3e-3 with one:
// two for both of them are six products for four, 15 to 26 % of the gradients' time.
//
// Bound by the matrix and the vector unit together, as the forward: 8 x 2048 x
// 12 x 64 takes 125 us for dq and 149 for dk and dv, 2 x 4096 x 16/4 x 128
// with the forward 735 to 775 us, 620 to 650 TFLOP/s.  Packed sequences of many
// lengths are bound by the longest workgroups: of the time of dk and dv of 13
// documents of up to 1201 rows x 16/4 x 128, 146 us, the CUs are busy 0.70.
#include <algorithm>

#include "../../include/gdn.h"
#include "gdn_attn.hpp"
#include "gdn_launch.hpp"
#include "gdn_tile.hpp"

namespace gdn {
namespace {

using namespace tile;

constexpr float kLog2e = 1.44269504088896f;
constexpr int kN = 64;  // rows of a staged tile

// acc[t] += (columns 32 t of a staged tile, rows r0 .. r0 + 15)^T w, as kept in
// acc's registers.
template <int D>
__device__ __forceinline__ void add_columns(f32x16 (&acc)[D / 32], const __bf16* tile, int base, int r0, const u32x4& w) {
#pragma unroll
  for (int t = 0; t < D / 32; ++t) acc[t] = mma(col_frag<D>(tile, base, r0, t), w, acc[t]);
}

template <int D> __device__ __forceinline__ void store_rows(__bf16* dst, const f32x16 (&acc)[D / 32], float f, int hl) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<u32x2*>(dst + 32 * i + 8 * e + 4 * hl) =
          pipe::cvt4(f32x4{acc[i][4 * e] * f, acc[i][4 * e + 1] * f, acc[i][4 * e + 2] * f, acc[i][4 * e + 3] * f});
}

// What scrubbing left out of a gradient row: NaN into those of its columns 32 w ..
// whose bit is set.  Each lane sees to the entries that it stored.
template <class T> __device__ __forceinline__ void spoil(T* dst, int w, unsigned columns, int hl) {
  if (columns)
    for (int d = 4 * hl; d < 32; d += 8)
      for (int i = d; i < d + 4; ++i)
        if (columns >> i & 1) dst[32 * w + i] = (T)__builtin_nanf("");
}

// Which of rows lo .. hi - 1 of K hold values that are not finite.
template <int D, int N, int NT>
__device__ __forceinline__ void mark_keys(Marks<D, N>& marks, const void* k, long long stride, int lo, int hi, int r0) {
  marks.template clear<NT>();
  __syncthreads();
  marks.template look<NT, Kind::not_finite>(k, stride, lo, hi, r0);
  __syncthreads();
}

// The waves' sums of 32 rows (a lane's row: l % 32), one beside the other in LDS,
// and what they add up to.  The first begins and ends with a barrier.
template <int D, int NW> using Parts = float[NW][32][D + 4];
template <int D, int NW>
__device__ __forceinline__ void join_rows(Parts<D, NW>& part, const f32x16 (&acc)[D / 32], int wave, int lane) {
  __syncthreads();
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<f32x4*>(&part[wave][lane & 31][32 * i + 8 * e + 4 * (lane >> 5)]) =
          f32x4{acc[i][4 * e], acc[i][4 * e + 1], acc[i][4 * e + 2], acc[i][4 * e + 3]};
  __syncthreads();
}
template <int D, int NW> __device__ __forceinline__ f32x4 joined(const Parts<D, NW>& part, int r, int d) {
  f32x4 o = *reinterpret_cast<const f32x4*>(&part[0][r][d]);
#pragma unroll
  for (int w = 1; w < NW; ++w) o += *reinterpret_cast<const f32x4*>(&part[w][r][d]);
  return o;
}

// ---------------------------------------------------------------------- dq
// do . o of a row, of which each half-wave holds half of do as operands.
template <int D>
__device__ __forceinline__ float delta_of(const PromptBwdArgs& a, int row, int hq, const u32x4 (&g)[D / 16], int hl) {
  const __bf16* op = static_cast<const __bf16*>(a.out) + ((long long)row * a.Hq + hq) * D + 8 * hl;
  float delta = 0.f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const u32x4 o = *reinterpret_cast<const u32x4*>(op + 16 * ks);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      delta = __builtin_fmaf(pipe::lo_f(g[ks][e]), pipe::lo_f(o[e]), delta);
      delta = __builtin_fmaf(pipe::hi_f(g[ks][e]), pipe::hi_f(o[e]), delta);
    }
  }
  return sum_halves(delta);
}

// 32 keys, rows n0 .. of the staged K and V, for a wave's 32 rows, of which the
// lane's sees keys from .. upto (less 4 hl) if MASKED; values_done() is called
// when V has been read.  GLDS: do comes from LDS, gt, not from g.
template <int D, bool MASKED, bool GLDS, class F>
__device__ __forceinline__ void dq_tile(f32x16 (&dq)[D / 32], float& rest, const __bf16* K, const __bf16* V, int rb, int cb,
                                        int n0, const u32x4 (&q)[D / 16], const u32x4 (&g)[D / 16], const __bf16* gt, int gb, float c, float lse2,
                                        float delta, int from, int upto, F values_done) {
  const unsigned seen = bits(from, upto);
  f32x16 s = zero16(), dp = zero16();
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    s = mma(row_frag<D>(K, rb, n0, ks), q[ks], s);
    dp = mma(row_frag<D>(V, rb, n0, ks), GLDS ? row_frag<D>(gt, gb, 0, ks) : g[ks], dp);
  }
  values_done();
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -lse2));
    s[e] = p * (dp[e] - delta);
    if constexpr (MASKED) s[e] = where_seen<true>(s[e], seen, e);
    rest += s[e];
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const u32x4 hi = operand(s, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[8 * b + 2 * i] -= pipe::lo_f(hi[i]);
      s[8 * b + 2 * i + 1] -= pipe::hi_f(hi[i]);
    }
    const u32x4 lo = operand(s, b);
#pragma unroll
    for (int t = 0; t < D / 32; ++t) {
      const u32x4 k = col_frag<D>(K, cb, n0 + 16 * b, t);
      dq[t] = mma(k, lo, mma(k, hi, dq[t]));
    }
  }
}

template <int D, int NW> __global__ __launch_bounds__(64 * NW, 2) void attn_dq_kernel(PromptBwdArgs a) {
  constexpr int BM = 32 * NW, NT = 64 * NW, KS = D / 16;
  __shared__ alignas(16) __bf16 kt[2][kN * D], vt[2][kN * D];
  __shared__ int begs[BM], window[kWindow], ranges[3][NW], dirty;  // dirty: a tile held values that are not finite
  __shared__ Marks<D, BM> marks;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  const int tiles = (a.T + BM - 1) / BM;
  const int rank = blockIdx.x / a.Hq, hq = blockIdx.x - rank * a.Hq;
  int tile = tiles - 1 - rank;
  if (a.by_length) tile = tile_by_length<BM, NT, false>(a.cu, a.R, a.T, tiles, rank, window, reinterpret_cast<int*>(kt));
  const int r0 = tile * BM, kvh = hq / (a.Hq / a.Hkv);

  const int w0 = r0 + wave * 32, row = w0 + (lane & 31), at = min(row, a.T - 1);
  const float c = a.scale * kLog2e;
  u32x4 q[KS], g[KS];
  if (tid == 0) dirty = 0;
  find_rows<BM, NT>(a.cu, a.R, a.T, r0, window, begs, nullptr, [&] {
    const __bf16* qp = static_cast<const __bf16*>(a.q) + (long long)at * a.qs + (long long)hq * D + 8 * hl;
    const __bf16* gp = static_cast<const __bf16*>(a.grad_out) + (long long)at * a.gos + (long long)hq * D + 8 * hl;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[ks] = *reinterpret_cast<const u32x4*>(qp + 16 * ks);
      g[ks] = *reinterpret_cast<const u32x4*>(gp + 16 * ks);
    }
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
    if (a.zero_rest) zero_rows<D>(static_cast<__bf16*>(a.grad_q) + (long long)hq * D, a.gqs, r0, min(BM, a.T - r0), NT);
    return;
  }

  const float delta = delta_of<D>(a, at, hq, g, hl);
  const float lse2 = a.lse[(size_t)hq * a.T + at] * kLog2e;

  f32x16 dq[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) dq[i] = zero16();
  const int rb0 = row_base<D>(lane), cb0 = col_base<D>(lane);
  Stage<D, kN, NW> sk, sv;
  sk.init(a.ks, wave);
  sv.init(a.vs, wave);
  const __bf16* kp = static_cast<const __bf16*>(a.k) + (long long)kvh * D;
  const __bf16* vp = static_cast<const __bf16*>(a.v) + (long long)kvh * D;
  auto stage = [&](int buf, int kv) {
    const int n = min(kN, last - kv);
    sk.load(kt[buf], rows_rsrc(kp, a.ks, kv, n, D), wave);
    sv.load(vt[buf], rows_rsrc(vp, a.vs, kv, n, D), wave);
  };
  const int from = beg - 4 * hl, upto = beg < 0 ? -8 : row - 4 * hl;  // the keys that the lane's row sees
  // delta comes from the rounded output.  The ds of a row add up to zero, but for
  // that rounding: what they add up to is its error, and the second launch gets
  // delta without it.
  float rest = 0.f;
  int buf = 0, kv = first;
  auto step = [&](auto masked_, const __bf16* K, const __bf16* V) {
    constexpr bool MASKED = decltype(masked_)::value;
    const int rb = fresh(rb0), cb = fresh(cb0);
#pragma unroll 1
    for (int n = 0; n < 2; ++n)
      dq_tile<D, MASKED, false>(dq, rest, K, V, rb, cb, 32 * n, q, g, nullptr, 0, c, lse2, delta, from - kv - 32 * n, upto - kv - 32 * n, [] {});
  };
  stage(0, first);
  auto next = [&] {
    const bool masked = kv + kN - 1 > r0 || kv < latest || kv + kN > last;  // for some wave
    if (masked) {
      wait_staged();
      const bool ok = Stage<D, kN, NW>::scrub(kt[buf], wave);
      if (lane == 0 && !ok) dirty = 1;
    }
    staged_barrier();
    if (kv + kN < last) stage(buf ^ 1, kv + kN);
  };
  const int whole = min(w0 + 1, last);  // waves behind the last tile take no more than the others
  // tiles of which some row misses some key, at both ends, and those between
  auto edge = [&](int end) {
    for (; kv < end; kv += kN, buf ^= 1) {
      next();
      if (kv <= w0 + 31 && kv + kN > lowest) step(std::true_type{}, kt[buf], vt[buf]);
    }
  };
  edge(min(highest, last));
  for (; kv + kN <= whole; kv += kN, buf ^= 1) {
    next();
    step(std::false_type{}, kt[buf], vt[buf]);
  }
  edge(last);
  const float off = sum_halves(rest);
  if (beg >= 0 && hl == 0) {
    a.ws[(size_t)hq * a.T + row] = lse2;
    a.ws[(size_t)(a.Hq + hq) * a.T + row] = -(delta + off);
  }
  const bool outside = beg < 0 && row < a.T && a.zero_rest;
  if (beg >= 0 || outside)
    store_rows<D>(static_cast<__bf16*>(a.grad_q) + (long long)row * a.gqs + (long long)hq * D, dq, outside ? 0.f : a.scale, hl);
  __syncthreads();
  if (dirty) {  // a key that is not finite spoils the weights of all rows that see it
    mark_keys<D, BM, NT>(marks, kp, a.ks, first, last, r0);
    if (beg >= 0 && marks.any(max(beg - r0, 0), row - r0 + 1, beg < r0))
      for (int w = 0; w < D / 32; ++w)
        spoil(static_cast<__bf16*>(a.grad_q) + (long long)row * a.gqs + (long long)hq * D, w, ~0u, hl);
  }
}

// Few rows, as in the forward: a workgroup takes 32 rows and its waves every
// NW-th tile of 32 keys, each staging its own; their sums are added at the end.
// With the same for dk and dv: forward and gradients of 1 x 1000 x 12/4 x 64 41 us
// for 76, 1 x 2500 x 16/4 x 128 217 for 297.
template <int D, int NW> __global__ __launch_bounds__(64 * NW, 2) void attn_dq_split_kernel(PromptBwdArgs a) {
  constexpr int NT = 64 * NW, KS = D / 16, LD = D + 4;
  __shared__ union alignas(16) {
    __bf16 staged[NW][2][32 * D];
    float part[NW][32][LD];
  } mem;
  constexpr bool GLDS = D == 128;  // do, the same rows for all waves, from LDS: there are no registers for it
  __shared__ alignas(16) __bf16 gt[GLDS ? 32 * D : 8];
  __shared__ float rests[NW][32];
  __shared__ int begs[32], window[kWindow], dirty[2][NW];
  __shared__ Marks<D, 32> marks;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  const int tiles = (a.T + 31) / 32;
  const int rank = blockIdx.x / a.Hq, hq = blockIdx.x - rank * a.Hq;
  const int r0 = (tiles - 1 - rank) * 32, kvh = hq / (a.Hq / a.Hkv);

  const int row = r0 + (lane & 31), at = min(row, a.T - 1);
  const float c = a.scale * kLog2e;
  u32x4 q[KS], g[KS];
  find_rows<32, NT>(a.cu, a.R, a.T, r0, window, begs, nullptr, [&] {
    const __bf16* qp = static_cast<const __bf16*>(a.q) + (long long)at * a.qs + (long long)hq * D + 8 * hl;
    const __bf16* gp = static_cast<const __bf16*>(a.grad_out) + (long long)at * a.gos + (long long)hq * D + 8 * hl;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[ks] = *reinterpret_cast<const u32x4*>(qp + 16 * ks);
      g[ks] = *reinterpret_cast<const u32x4*>(gp + 16 * ks);
    }
  });
  const int beg = begs[row - r0];
  const KeyRange range = key_range(beg, row, a.T);
  const int first = range.first, latest = range.latest, last = range.last;
  if (last < 0) {  // no row of the tile is in a sequence
    if (a.zero_rest) zero_rows<D>(static_cast<__bf16*>(a.grad_q) + (long long)hq * D, a.gqs, r0, min(32, a.T - r0), NT);
    return;
  }
  const float delta = delta_of<D>(a, at, hq, g, hl), lse2 = a.lse[(size_t)hq * a.T + at] * kLog2e;

  if constexpr (GLDS) {
    Stage<D, 32, NW> sg;
    sg.init(a.gos, wave);
    sg.load(gt, rows_rsrc(static_cast<const __bf16*>(a.grad_out) + (long long)hq * D, a.gos, r0, min(32, a.T - r0), D), wave);
    staged_barrier();
  }
  f32x16 dq[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) dq[i] = zero16();
  const int rb0 = row_base<D>(lane), cb0 = col_base<D>(lane);
  Stage<D, 32, 1> sk, sv;
  sk.init(a.ks, 0);
  sv.init(a.vs, 0);
  const __bf16* kp = static_cast<const __bf16*>(a.k) + (long long)kvh * D;
  const __bf16* vp = static_cast<const __bf16*>(a.v) + (long long)kvh * D;
  __bf16 *kt = mem.staged[wave][0], *vt = mem.staged[wave][1];
  const int from = beg - 4 * hl, upto = beg < 0 ? -8 : row - 4 * hl;
  float rest = 0.f;
  int dirty_lo = last, dirty_hi = 0, kv = first + 32 * wave;
  auto stage_keys = [&](int kv) { sk.load(kt, rows_rsrc(kp, a.ks, kv, min(32, last - kv), D), 0); };
  auto stage_values = [&](int kv) { sv.load(vt, rows_rsrc(vp, a.vs, kv, min(32, last - kv), D), 0); };
  if (kv < last) {
    stage_keys(kv);
    stage_values(kv);
  }
  for (; kv < last; kv += 32 * NW) {
    const int to = kv + 32 * NW, rb = fresh(rb0), cb = fresh(cb0);
    wait_staged();
    auto values_done = [&] {
      if (to < last) {
        wait_read();
        stage_values(to);
      }
    };
    if (kv + 31 > r0 || kv < latest || kv + 32 > last) {
      if (!Stage<D, 32, 1>::scrub(kt, 0)) {
        dirty_lo = min(dirty_lo, kv);
        dirty_hi = kv + 32;
      }
      dq_tile<D, true, GLDS>(dq, rest, kt, vt, rb, cb, 0, q, g, gt, rb, c, lse2, delta, from - kv, upto - kv, values_done);
    } else {
      dq_tile<D, false, GLDS>(dq, rest, kt, vt, rb, cb, 0, q, g, gt, rb, c, lse2, delta, 0, 0, values_done);
    }
    if (to < last) {
      wait_read();
      stage_keys(to);
    }
  }
  const float off = sum_halves(rest);
  if (hl == 0) rests[wave][lane] = off;
  if (lane == 0) {
    dirty[0][wave] = dirty_lo;
    dirty[1][wave] = dirty_hi;
  }
  join_rows<D, NW>(mem.part, dq, wave, lane);
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    dirty_lo = min(dirty_lo, dirty[0][w]);
    dirty_hi = max(dirty_hi, dirty[1][w]);
  }
  if (wave == 0 && hl == 0 && beg >= 0) {
    float more = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) more += rests[w][lane];
    a.ws[(size_t)hq * a.T + row] = lse2;
    a.ws[(size_t)(a.Hq + hq) * a.T + row] = -(delta + more);
  }
  if (dirty_hi) mark_keys<D, 32, NT>(marks, kp, a.ks, dirty_lo, min(dirty_hi, last), r0);
  for (int i = tid; i < 32 * (D / 4); i += NT) {
    const int r = i / (D / 4), d = i % (D / 4) * 4, b = begs[r];
    if (r0 + r >= a.T || (b < 0 && !a.zero_rest)) continue;
    f32x4 o = joined<D, NW>(mem.part, r, d) * (b < 0 ? 0.f : a.scale);
    if (b < 0) o = pipe::zero4();
    if (dirty_hi && b >= 0 && marks.any(max(b - r0, 0), r + 1, b < r0)) o += __builtin_nanf("");
    *reinterpret_cast<u32x2*>(static_cast<__bf16*>(a.grad_q) + (long long)(r0 + r) * a.gqs + (long long)hq * D + d) = pipe::cvt4(o);
  }
}

// ------------------------------------------------------------------ dk, dv
// A workgroup's part: a tile of keys of one key head, and of the query heads
// that share it all (shares = 1) or an equal share.  Shares write float32 sums
// to the workspace, [share][dk, dv][T][Hkv][D], which a last launch adds.
struct Share {
  int tile, kvh, h0, heads, at;
};
__device__ __forceinline__ Share share_of(const PromptBwdArgs& a) {
  // the first tiles of a long sequence meet the most rows
  const int per = a.Hkv * a.shares, tile = blockIdx.x / per, x = blockIdx.x - tile * per;
  const int heads = a.Hq / per;
  return {tile, x / a.shares, x * heads, heads, x % a.shares};
}
__host__ __device__ inline size_t sums_at(int T, int Hq) { return ((size_t)2 * T * Hq + 3) / 4 * 4; }  // behind lse, delta
__device__ __forceinline__ float* sums_row(const PromptBwdArgs& a, int D, int at, bool values, int row, int kvh) {
  return a.ws + sums_at(a.T, a.Hq) + ((((size_t)at * 2 + values) * a.T + row) * a.Hkv + kvh) * D;
}

template <int D>
__device__ __forceinline__ void write_grad(const PromptBwdArgs& a, const Share& sh, bool values, int key, int end,
                                           const f32x16 (&acc)[D / 32], float f, int hl) {
  if (a.shares > 1) {
    if (end < 0) return;
    float* dst = sums_row(a, D, sh.at, values, key, sh.kvh);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(dst + 32 * i + 8 * e + 4 * hl) =
            f32x4{acc[i][4 * e] * f, acc[i][4 * e + 1] * f, acc[i][4 * e + 2] * f, acc[i][4 * e + 3] * f};
    return;
  }
  const bool rest = end < 0 && key < a.T && a.zero_rest;
  if (end >= 0 || rest)
    store_rows<D>(static_cast<__bf16*>(values ? a.grad_v : a.grad_k) + (long long)key * (values ? a.gvs : a.gks) + (long long)sh.kvh * D,
                  acc, rest ? 0.f : f, hl);
}

// Which rows of q and of do, of the share's heads, hold values that are not finite.
// Those of q spoil the weights of their keys, dk and dv whole; those of do dk whole
// and dv where they are.
template <int D, int N> struct RowMarks {
  Marks<D, N> q, g;
  template <int NT> __device__ __forceinline__ void look(const PromptBwdArgs& a, const Share& sh, int r0, int last) {
    q.template clear<NT>();
    g.template clear<NT>();
    __syncthreads();
    for (int h = sh.h0; h < sh.h0 + sh.heads; ++h) {
      q.template look<NT, Kind::not_finite>(static_cast<const __bf16*>(a.q) + (long long)h * D, a.qs, r0, last, r0);
      g.template look<NT, Kind::not_finite>(static_cast<const __bf16*>(a.grad_out) + (long long)h * D, a.gos, r0, last, r0);
    }
    __syncthreads();
  }
  // Columns 32 w .. of dk (of dv) that the rows from lo to hi - 1 (from r0), and with
  // `others` those behind the tile, spoil.
  __device__ __forceinline__ unsigned columns(bool values, int w, int lo, int hi, bool others) const {
    if (q.any(lo, hi, others)) return ~0u;
    if (values) return g.columns(w, lo, hi, others);
    return g.any(lo, hi, others) ? ~0u : 0u;
  }
};
template <int D, int N>
__device__ __forceinline__ void spoil_grad(const PromptBwdArgs& a, const Share& sh, const RowMarks<D, N>& marks, bool values,
                                           int key, int r0, int end, int hl) {
  for (int w = 0; w < D / 32; ++w) {
    const unsigned m = marks.columns(values, w, key - r0, min(end - r0, N), end > r0 + N);
    if (a.shares > 1)
      spoil(sums_row(a, D, sh.at, values, key, sh.kvh), w, m, hl);
    else
      spoil(static_cast<__bf16*>(values ? a.grad_v : a.grad_k) + (long long)key * (values ? a.gvs : a.gks) + (long long)sh.kvh * D, w, m, hl);
  }
}

// Adds the shares of kSumRows keys of one key head, in their order.  The sums are
// read before it is known which rows are in a sequence: those of the others are
// what the workspace held, and left out.
constexpr int kSumRows = 8;
template <int D> __global__ __launch_bounds__(256) void attn_dkv_sum_kernel(PromptBwdArgs a) {
  constexpr int kItems = 2 * kSumRows * (D / 4) / 256;
  static_assert(kItems * 256 == 2 * kSumRows * (D / 4), "");
  __shared__ int begs[kSumRows], window[kWindow];
  const int tile = blockIdx.x / a.Hkv, kvh = blockIdx.x - tile * a.Hkv;
  auto place = [&](int n, bool& values, int& i, int& d) {
    const int x = threadIdx.x + 256 * n;
    values = x >= kSumRows * (D / 4);
    i = x % (kSumRows * (D / 4)) / (D / 4);
    d = x % (D / 4) * 4;
  };
  f32x4 sum[kItems];
  find_rows<kSumRows, 256>(a.cu, a.R, a.T, tile * kSumRows, window, begs, nullptr, [&] {
#pragma unroll
    for (int n = 0; n < kItems; ++n) sum[n] = pipe::zero4();
#pragma unroll 2
    for (int s = 0; s < a.shares; ++s)
#pragma unroll
      for (int n = 0; n < kItems; ++n) {
        bool values;
        int i, d;
        place(n, values, i, d);
        sum[n] += *reinterpret_cast<const f32x4*>(sums_row(a, D, s, values, min(tile * kSumRows + i, a.T - 1), kvh) + d);
      }
  });
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    bool values;
    int i, d;
    place(n, values, i, d);
    const int row = tile * kSumRows + i;
    const bool in = begs[i] >= 0;
    if (row >= a.T || (!in && !a.zero_rest)) continue;
    *reinterpret_cast<u32x2*>(static_cast<__bf16*>(values ? a.grad_v : a.grad_k) + (long long)row * (values ? a.gvs : a.gks) +
                              (long long)kvh * D + d) = pipe::cvt4(in ? sum[n] : pipe::zero4());
  }
}

// 32 rows, n0 .. of the staged Q and dO with their lse and -delta, for a wave's
// 32 keys: k their operands, v those of V or (VLDS) vt its rows from v0 on; the lane's key is seen by rows
// from .. upto (less 4 hl) if MASKED.
template <int D, bool MASKED, bool VLDS>
__device__ __forceinline__ void dkv_tile(f32x16 (&dk)[D / 32], f32x16 (&dv)[D / 32], const __bf16* Q, const __bf16* O,
                                         const float* lt, const float* dt, int rb, int cb, int n0,
                                         const u32x4 (&k)[D / 16], const u32x4 (&v)[D / 16], const __bf16* vt, int v0, float c, int from, int upto, int hl) {
  const unsigned seen = bits(from, upto);
  f32x16 s = zero16(), dp;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) s = mma(row_frag<D>(Q, rb, n0, ks), k[ks], s);
#pragma unroll
  for (int e4 = 0; e4 < 4; ++e4) {
    const f32x4 d = *reinterpret_cast<const f32x4*>(&dt[n0 + 8 * e4 + 4 * hl]);
#pragma unroll
    for (int j = 0; j < 4; ++j) dp[4 * e4 + j] = d[j];
  }
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
    dp = mma(row_frag<D>(O, rb, n0, ks), VLDS ? row_frag<D>(vt, rb, v0, ks) : v[ks], dp);
#pragma unroll
  for (int e4 = 0; e4 < 4; ++e4) {
    const f32x4 l = *reinterpret_cast<const f32x4*>(&lt[n0 + 8 * e4 + 4 * hl]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * e4 + j;
      s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -l[j]));
      dp[e] = s[e] * dp[e];
      if constexpr (MASKED) {
        s[e] = where_seen<true>(s[e], seen, e);
        dp[e] = where_seen<true>(dp[e], seen, e);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    add_columns<D>(dv, O, cb, n0 + 16 * b, operand(s, b));
    add_columns<D>(dk, Q, cb, n0 + 16 * b, operand(dp, b));
  }
}

// One wave to 32 keys, rows in tiles of NR.  At D = 64 a wave holds K and V of
// its keys as operands beside both accumulators (243 registers).  At D = 128
// that would be 192 registers before the first score: V stays in LDS (VLDS),
// which takes tiles of half as many rows, and every tile goes through the masked
// body, since two bodies of this size take more registers than there are (256
// with one; a bit mask per score costs less than a spill, whose reload waits for
// the loads that stage the next tile).  Two waves that share the work of 32 keys
// and hand the scores over through LDS took 260 us where this takes 146 (13
// documents of up to 1201 rows, 16/4 heads of 128).
template <int D, int NW, int NR, bool VLDS> __global__ __launch_bounds__(64 * NW, 2) void attn_dkv_kernel(PromptBwdArgs a) {
  constexpr int BN = 32 * NW, NT = 64 * NW, KS = D / 16;
  __shared__ alignas(16) __bf16 qt[2][NR * D], gt[2][NR * D];
  __shared__ alignas(16) float lt[2][64], dt[2][64];
  __shared__ alignas(16) __bf16 vt[VLDS ? BN * D : 8];
  __shared__ int begs[BN], ends[BN], window[kWindow], most[2][NW], dirty;  // dirty: a tile held values that are not finite
  __shared__ RowMarks<D, BN> marks;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  // the first tiles of a long sequence meet the most rows
  Share sh = share_of(a);
  if (a.keys_by_length)
    sh.tile = tile_by_length<BN, NT, true>(a.cu, a.R, a.T, (a.T + BN - 1) / BN, sh.tile, window, reinterpret_cast<int*>(qt));
  const int r0 = sh.tile * BN, kvh = sh.kvh, h0 = sh.h0, heads = sh.heads;

  if (tid == 0) dirty = 0;
  find_rows<BN, NT>(a.cu, a.R, a.T, r0, window, begs, ends, [] {});
  int last = -1, soonest = a.T;  // the rows behind the last that attend to the tile's keys: the most, the least
  for (int i = tid; i < BN; i += NT) {
    last = max(last, ends[i]);
    soonest = min(soonest, ends[i]);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    last = max(last, __shfl_xor(last, d));
    soonest = min(soonest, __shfl_xor(soonest, d));
  }
  if (lane == 0) {
    most[0][wave] = last;
    most[1][wave] = soonest;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    last = max(last, most[0][w]);
    soonest = min(soonest, most[1][w]);
  }
  last = __builtin_amdgcn_readfirstlane(last);
  soonest = __builtin_amdgcn_readfirstlane(soonest);
  if (last < 0) {
    if (a.zero_rest && a.shares == 1) {
      zero_rows<D>(static_cast<__bf16*>(a.grad_k) + (long long)kvh * D, a.gks, r0, min(BN, a.T - r0), NT);
      zero_rows<D>(static_cast<__bf16*>(a.grad_v) + (long long)kvh * D, a.gvs, r0, min(BN, a.T - r0), NT);
    }
    return;
  }

  const int w0 = r0 + wave * 32, key = w0 + (lane & 31), end = ends[key - r0];
  const int at = min(key, a.T - 1);
  const float c = a.scale * kLog2e;
  u32x4 k[KS], v[KS];
  {
    const __bf16* kp = static_cast<const __bf16*>(a.k) + (long long)at * a.ks + (long long)kvh * D + 8 * hl;
    const __bf16* vp = static_cast<const __bf16*>(a.v) + (long long)at * a.vs + (long long)kvh * D + 8 * hl;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      k[ks] = *reinterpret_cast<const u32x4*>(kp + 16 * ks);
      if (!VLDS) v[ks] = *reinterpret_cast<const u32x4*>(vp + 16 * ks);
    }
  }
  int lowest = end, highest = end;  // the range of end over the wave's keys
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    lowest = min(lowest, __shfl_xor(lowest, d));
    highest = max(highest, __shfl_xor(highest, d));
  }
  lowest = __builtin_amdgcn_readfirstlane(lowest);
  highest = __builtin_amdgcn_readfirstlane(highest);

  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) dk[i] = dv[i] = zero16();
  const int rb0 = row_base<D>(lane), cb0 = col_base<D>(lane);
  Stage<D, NR, NW> sq, sg;
  sq.init(a.qs, wave);
  sg.init(a.gos, wave);
  const __bf16* qp = static_cast<const __bf16*>(a.q);
  const __bf16* gp = static_cast<const __bf16*>(a.grad_out);
  auto stage = [&](int buf, int hq, int i0) {
    const int n = min(NR, last - i0);
    sq.load(qt[buf], rows_rsrc(qp + (long long)hq * D, a.qs, i0, n, D), wave);
    sg.load(gt[buf], rows_rsrc(gp + (long long)hq * D, a.gos, i0, n, D), wave);
    if (wave == 0) stage_words(lt[buf], pipe::make_rsrc(a.ws + (size_t)hq * a.T + i0, n * 4));
    if (wave == 1) stage_words(dt[buf], pipe::make_rsrc(a.ws + (size_t)(a.Hq + hq) * a.T + i0, n * 4));
  };
  // a tile of rows that the wave's keys may be seen by
  auto step = [&](auto masked_, int buf, int i1) {
    constexpr bool MASKED = decltype(masked_)::value;
    const int rb = fresh(rb0), cb = fresh(cb0);
    const __bf16 *Q = qt[buf], *O = gt[buf];
    const int from = key - i1 - 4 * hl, upto = end - 1 - i1 - 4 * hl;  // the rows that see the lane's key
#pragma unroll MASKED ? 1 : NR / 32
    for (int n = 0; n < NR / 32; ++n) {
      dkv_tile<D, MASKED, VLDS>(dk, dv, Q, O, lt[buf], dt[buf], rb, cb, 32 * n, k,
                          v, vt, 32 * wave, c, from - 32 * n, upto - 32 * n, hl);
    }
  };
  if constexpr (VLDS) {
    Stage<D, BN, NW> sv;
    sv.init(a.vs, wave);
    sv.load(vt, rows_rsrc(static_cast<const __bf16*>(a.v) + (long long)kvh * D, a.vs, r0, min(BN, a.T - r0), D), wave);
  }
  stage(0, h0, r0);
  int buf = 0;
  for (int head = 0; head < heads; ++head) {
    int i1 = r0;
    auto next = [&] {
      const bool masked = i1 < r0 + BN - 1 || i1 + NR > soonest;  // for some wave
      if (masked) {
        wait_staged();
        const bool q_ok = Stage<D, NR, NW>::scrub(qt[buf], wave), g_ok = Stage<D, NR, NW>::scrub(gt[buf], wave);
        if (lane == 0 && !(q_ok && g_ok)) dirty = 1;
      }
      staged_barrier();
      if (i1 + NR < last) stage(buf ^ 1, h0 + head, i1 + NR);
      else if (head + 1 < heads) stage(buf ^ 1, h0 + head + 1, r0);
    };
    // tiles of which some row misses some key, at both ends, and those between
    auto edge = [&](int stop) {
      for (; i1 < stop; i1 += NR, buf ^= 1) {
        next();
        if (i1 + NR - 1 >= w0 && i1 < highest) step(std::true_type{}, buf, i1);
      }
    };
    if constexpr (!VLDS) {
      edge(min(w0 + 31, last));
      for (; i1 + NR <= lowest; i1 += NR, buf ^= 1) {
        next();
        step(std::false_type{}, buf, i1);
      }
    }
    edge(last);
  }
  write_grad<D>(a, sh, false, key, end, dk, a.scale, hl);
  write_grad<D>(a, sh, true, key, end, dv, 1.f, hl);
  __syncthreads();
  if (dirty) {
    marks.template look<NT>(a, sh, r0, last);
    for (int values = 0; values < 2 && end >= 0; ++values) spoil_grad<D, BN>(a, sh, marks, values, key, r0, end, hl);
  }
}

// Few keys: a workgroup takes 32 of one key head, and its waves every NW-th tile
// of 32 rows of the share's query heads, one head after the other.
template <int D, int NW> __global__ __launch_bounds__(64 * NW, 2) void attn_dkv_split_kernel(PromptBwdArgs a) {
  constexpr int NT = 64 * NW, KS = D / 16;
  constexpr bool VLDS = D == 128;
  __shared__ union alignas(16) {
    __bf16 staged[NW][2][32 * D];
    Parts<D, NW> part;
  } mem;
  __shared__ alignas(16) float lt[NW][64], dt[NW][64];
  __shared__ alignas(16) __bf16 vt[VLDS ? 32 * D : 8];
  __shared__ int begs[32], ends[32], window[kWindow], dirty[NW];
  __shared__ RowMarks<D, 32> marks;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  const Share sh = share_of(a);
  const int r0 = sh.tile * 32, kvh = sh.kvh;
  find_rows<32, NT>(a.cu, a.R, a.T, r0, window, begs, ends, [] {});
  const int key = r0 + (lane & 31), end = ends[lane & 31], at = min(key, a.T - 1);
  int last = end, soonest = end;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    last = max(last, __shfl_xor(last, d));
    soonest = min(soonest, __shfl_xor(soonest, d));
  }
  last = __builtin_amdgcn_readfirstlane(last);
  soonest = __builtin_amdgcn_readfirstlane(soonest);
  if (last < 0) {
    if (a.zero_rest && a.shares == 1) {
      zero_rows<D>(static_cast<__bf16*>(a.grad_k) + (long long)kvh * D, a.gks, r0, min(32, a.T - r0), NT);
      zero_rows<D>(static_cast<__bf16*>(a.grad_v) + (long long)kvh * D, a.gvs, r0, min(32, a.T - r0), NT);
    }
    return;
  }
  const float c = a.scale * kLog2e;
  u32x4 k[KS], v[KS];
  {
    const __bf16* kp = static_cast<const __bf16*>(a.k) + (long long)at * a.ks + (long long)kvh * D + 8 * hl;
    const __bf16* vp = static_cast<const __bf16*>(a.v) + (long long)at * a.vs + (long long)kvh * D + 8 * hl;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      k[ks] = *reinterpret_cast<const u32x4*>(kp + 16 * ks);
      if (!VLDS) v[ks] = *reinterpret_cast<const u32x4*>(vp + 16 * ks);
    }
  }
  if constexpr (VLDS) {
    Stage<D, 32, NW> sv;
    sv.init(a.vs, wave);
    sv.load(vt, rows_rsrc(static_cast<const __bf16*>(a.v) + (long long)kvh * D, a.vs, r0, min(32, a.T - r0), D), wave);
    staged_barrier();
  }
  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) dk[i] = dv[i] = zero16();
  const int rb0 = row_base<D>(lane), cb0 = col_base<D>(lane);
  Stage<D, 32, 1> sq, sg;
  sq.init(a.qs, 0);
  sg.init(a.gos, 0);
  auto stage = [&](int head, int i1) {
    const int n = min(32, last - i1), hq = sh.h0 + head;
    sq.load(mem.staged[wave][0], rows_rsrc(static_cast<const __bf16*>(a.q) + (long long)hq * D, a.qs, i1, n, D), 0);
    sg.load(mem.staged[wave][1], rows_rsrc(static_cast<const __bf16*>(a.grad_out) + (long long)hq * D, a.gos, i1, n, D), 0);
    stage_words(lt[wave], pipe::make_rsrc(a.ws + (size_t)hq * a.T + i1, n * 4));
    stage_words(dt[wave], pipe::make_rsrc(a.ws + (size_t)(a.Hq + hq) * a.T + i1, n * 4));
  };
  const int nt = (last - r0 + 31) / 32;  // tiles of rows to a head
  bool bad = false;
  int head = wave / nt, i = wave - head * nt;
  __bf16 *Q = mem.staged[wave][0], *O = mem.staged[wave][1];
  if (head < sh.heads) stage(head, r0 + 32 * i);
  while (head < sh.heads) {
    const int i1 = r0 + 32 * i, rb = fresh(rb0), cb = fresh(cb0);
    for (i += NW; i >= nt && head < sh.heads; i -= nt) ++head;
    wait_staged();
    if (VLDS || i1 < r0 + 31 || i1 + 32 > soonest) {
      if (i1 < r0 + 31 || i1 + 32 > soonest) {
        const bool q_ok = Stage<D, 32, 1>::scrub(Q, 0), g_ok = Stage<D, 32, 1>::scrub(O, 0);
        bad |= !(q_ok && g_ok);
      }
      dkv_tile<D, true, VLDS>(dk, dv, Q, O, lt[wave], dt[wave], rb, cb, 0, k, v, vt, 0, c, key - i1 - 4 * hl,
                              end - 1 - i1 - 4 * hl, hl);
    } else {
      dkv_tile<D, false, VLDS>(dk, dv, Q, O, lt[wave], dt[wave], rb, cb, 0, k, v, vt, 0, c, 0, 0, hl);
    }
    if (head < sh.heads) {
      wait_read();
      stage(head, r0 + 32 * i);
    }
  }
  if (lane == 0) dirty[wave] = bad;
  __syncthreads();
  const bool any = !all_clean(dirty);
  if (any) marks.template look<NT>(a, sh, r0, last);
  for (int values = 0; values < 2; ++values) {
    if (values) join_rows<D, NW>(mem.part, dv, wave, lane);
    else join_rows<D, NW>(mem.part, dk, wave, lane);
    for (int x = tid; x < 32 * (D / 4); x += NT) {
      const int r = x / (D / 4), d = x % (D / 4) * 4, e = ends[r];
      if (r0 + r >= a.T || (e < 0 && (!a.zero_rest || a.shares > 1))) continue;
      f32x4 o = joined<D, NW>(mem.part, r, d) * (values ? 1.f : a.scale);
      if (e < 0) o = pipe::zero4();
      if (any && e >= 0) {
        const unsigned m = marks.columns(values, d / 32, r, min(e - r0, 32), e > r0 + 32);
        for (int j = 0; j < 4; ++j)
          if (m >> (d % 32 + j) & 1) o[j] = __builtin_nanf("");
      }
      if (a.shares > 1)
        *reinterpret_cast<f32x4*>(sums_row(a, D, sh.at, values, r0 + r, kvh) + d) = o;
      else
        *reinterpret_cast<u32x2*>(static_cast<__bf16*>(values ? a.grad_v : a.grad_k) +
                                  (long long)(r0 + r) * (values ? a.gvs : a.gks) + (long long)kvh * D + d) = pipe::cvt4(o);
    }
  }
}

// Shares of the query heads that read one key head: as few as give the CUs
// kEnough tiles of keys to choose from (the first tiles of a sequence meet many
// more rows than its last, so few tiles leave most CUs waiting for the longest),
// at most one head each.  (13 documents of up to 1201 rows x 16/4 x 128, forward and
// gradients: 331 us with two shares, 335 with four; 1 x 1000 x 16/4 x 128, in
// small tiles, 67 for 74 with 256.)  No shares where all heads together are a few
// small tiles to a wave: 4 x 128 x 12/4 x 64 19.4 us for 20.7.
constexpr int kEnough = 600, kEnoughSplit = 512;
int shares_of(int T, int R, int Hq, int Hkv, int D) {
  const int G = Hq / Hkv;
  const bool split = split_keys(T, R, Hq, D);
  if (split && (long long)G * T <= 512LL * std::max(R, 1)) return 1;
  const long long tiles = split ? ((long long)T + 31) / 32 * Hkv : ((long long)T + 127) / 128 * Hkv;
  for (int s = 1; s < G; ++s)
    if (G % s == 0 && tiles * s >= (split ? kEnoughSplit : kEnough)) return s;
  return G;
}

template <int D> hipError_t launch(const PromptBwdArgs& a, bool split) {
  const unsigned tiles = (unsigned)((a.T + 127) / 128), fine = (unsigned)((a.T + 31) / 32);
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  hipError_t e;
  if (split) e = launch_kernel(attn_dq_split_kernel<D, 4>, dim3(fine * a.Hq), dim3(256), st, a);
  else e = launch_kernel(attn_dq_kernel<D, 4>, dim3(tiles * a.Hq), dim3(256), st, a);
  if (e != hipSuccess) return e;
  const dim3 grid((split ? fine : tiles) * a.Hkv * a.shares);
  if (split) e = launch_kernel(attn_dkv_split_kernel<D, 4>, grid, dim3(256), st, a);
  else if constexpr (D == 64) e = launch_kernel(attn_dkv_kernel<D, 4, 64, false>, grid, dim3(256), st, a);
  else e = launch_kernel(attn_dkv_kernel<D, 4, 32, true>, grid, dim3(256), st, a);
  if (e != hipSuccess || a.shares == 1) return e;
  return launch_kernel(attn_dkv_sum_kernel<D>, dim3((unsigned)((a.T + kSumRows - 1) / kSumRows) * a.Hkv), dim3(256), st, a);
}

}  // namespace

size_t attn_prompt_bwd_workspace_bytes(int T, int Hq, int Hkv, int D) {
  // the most that any number of sequences takes
  const int shares = std::max(shares_of(T, 1, Hq, Hkv, D), shares_of(T, T + 1, Hq, Hkv, D));
  const size_t sums = shares > 1 ? (size_t)shares * 2 * T * Hkv * D : 0;
  return (sums_at(T, Hq) + sums) * sizeof(float);
}

hipError_t launch_attn_prompt_bwd(const PromptBwdArgs& args) {
  PromptBwdArgs a = args;
  const bool split = split_keys(a.T, a.R, a.Hq, a.D);
  a.shares = shares_of(a.T, a.R, a.Hq, a.Hkv, a.D);
  a.by_length = rank_tiles(a.T, a.R, a.Hq);
  a.keys_by_length = rank_tiles(a.T, a.R, a.Hkv * a.shares);
  return a.D == 64 ? launch<64>(a, split) : launch<128>(a, split);
}

}  // namespace gdn
