// attn_prompt_bwd.hip -- gradients of causal attention over packed prompts.
//
// With p_ij = exp(scale q_i.k_j - lse_i) for the keys j that row i attends to,
//   delta_i = do_i . o_i,     dv_j = sum_i p_ij do_i,
//   ds_ij = p_ij (do_i . v_j - delta_i),
//   dq_i = scale sum_j ds_ij k_j,     dk_j = scale sum_i ds_ij q_i,
// dk and dv summed over the query heads that share key head j's.
//
// Two launches, each of which owns the gradients it writes, so that nothing is
// added through memory and the order of every sum is fixed: one per tile of
// rows for dq (three products for a pair of tiles), one per tile of keys for dk
// and dv (four).  The probabilities are computed in both; the first launch
// leaves lse and delta, in powers of two, in the workspace for the second.
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
// acc's registers.  Where the tile is not clean (a value that no weight may
// meet is not finite, see masked tiles) its non-finite values count as zero and
// as NaN where a weight other than zero meets them.
template <int D>
__device__ __forceinline__ void add_columns(f32x16 (&acc)[D / 32], const __bf16* tile, int base, int r0, const u32x4& w,
                                            bool clean) {
#pragma unroll
  for (int t = 0; t < D / 32; ++t) {
    const u32x4 f = col_frag<D>(tile, base, r0, t);
    if (clean) {
      acc[t] = mma(f, w, acc[t]);
    } else {
      acc[t] = mma(pick(f, 0), w, acc[t]);
      const u32x4 size{w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu, w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu};
      f32x16 bad = zero16();
#pragma unroll
      for (int kind = 1; kind < 4; ++kind) bad = mma(pick(f, kind), size, bad);
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[t][e] = bad[e] > 0.f ? __builtin_nanf("") : acc[t][e];
    }
  }
}

template <int D> __device__ __forceinline__ void store_rows(__bf16* dst, const f32x16 (&acc)[D / 32], float f, int hl) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<u32x2*>(dst + 32 * i + 8 * e + 4 * hl) =
          pipe::cvt4(f32x4{acc[i][4 * e] * f, acc[i][4 * e + 1] * f, acc[i][4 * e + 2] * f, acc[i][4 * e + 3] * f});
}

// ---------------------------------------------------------------------- dq
template <int D, int NW> __global__ __launch_bounds__(64 * NW, 2) void attn_dq_kernel(PromptBwdArgs a) {
  constexpr int BM = 32 * NW, NT = 64 * NW, KS = D / 16;
  __shared__ __bf16 kt[2][kN * D], vt[2][kN * D];
  __shared__ int begs[BM], window[BM + 1], lows[NW];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  const int tiles = (a.T + BM - 1) / BM;
  const int rank = blockIdx.x / a.Hq, hq = blockIdx.x - rank * a.Hq;
  const int r0 = (tiles - 1 - rank) * BM, kvh = hq / (a.Hq / a.Hkv);

  find_rows<BM, NT>(a.cu, a.R, a.T, r0, window, begs, nullptr);
  int first = a.T;
  for (int i = tid; i < BM; i += NT)
    if (begs[i] >= 0) first = min(first, begs[i]);
#pragma unroll
  for (int d = 32; d; d >>= 1) first = min(first, __shfl_xor(first, d));
  if (lane == 0) lows[wave] = first;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) first = min(first, lows[w]);
  first = __builtin_amdgcn_readfirstlane(first);
  if (first >= a.T) return;
  const int last = min(r0 + BM, a.T);

  const int w0 = r0 + wave * 32, row = w0 + (lane & 31), beg = begs[row - r0];
  const int at = min(row, a.T - 1);
  const float c = a.scale * kLog2e;
  u32x4 q[KS], g[KS];
  float delta = 0.f;
  {
    const __bf16* qp = static_cast<const __bf16*>(a.q) + (long long)at * a.qs + (long long)hq * D + 8 * hl;
    const __bf16* gp = static_cast<const __bf16*>(a.grad_out) + (long long)at * a.gos + (long long)hq * D + 8 * hl;
    const __bf16* op = static_cast<const __bf16*>(a.out) + ((long long)at * a.Hq + hq) * D + 8 * hl;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[ks] = *reinterpret_cast<const u32x4*>(qp + 16 * ks);
      g[ks] = *reinterpret_cast<const u32x4*>(gp + 16 * ks);
      const u32x4 o = *reinterpret_cast<const u32x4*>(op + 16 * ks);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        delta = __builtin_fmaf(pipe::lo_f(g[ks][e]), pipe::lo_f(o[e]), delta);
        delta = __builtin_fmaf(pipe::hi_f(g[ks][e]), pipe::hi_f(o[e]), delta);
      }
    }
  }
  delta = sum_halves(delta);
  const float lse2 = a.lse[(size_t)hq * a.T + at] * kLog2e;
  if (beg >= 0 && hl == 0) {
    a.ws[(size_t)hq * a.T + row] = lse2;
    a.ws[(size_t)(a.Hq + hq) * a.T + row] = delta;
  }
  int lowest = beg < 0 ? a.T : beg, highest = lowest;
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    lowest = min(lowest, __shfl_xor(lowest, d));
    highest = max(highest, __shfl_xor(highest, d));
  }
  lowest = __builtin_amdgcn_readfirstlane(lowest);
  highest = __builtin_amdgcn_readfirstlane(highest);

  f32x16 dq[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) dq[i] = zero16();
  const int rb = row_base<D>(lane), cb = col_base<D>(lane);
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
  stage(0, first);
  int buf = 0;
  for (int kv = first; kv < last; kv += kN, buf ^= 1) {
    staged_barrier();
    if (kv + kN < last) stage(buf ^ 1, kv + kN);
    if (kv > w0 + 31 || kv + kN <= lowest) continue;
    const bool masked = kv + kN - 1 > w0 || kv < highest || kv + kN > last;
    const bool clean = !masked || clean_tile<D, kN>(kt[buf]);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        s = mma(row_frag<D>(kt[buf], rb, 32 * n, ks), q[ks], s);
        dp = mma(row_frag<D>(vt[buf], rb, 32 * n, ks), g[ks], dp);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -lse2));
        s[e] = p * (dp[e] - delta);
      }
      if (masked) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int key = kv + 32 * n + 8 * (e / 4) + 4 * hl + e % 4;
          s[e] = beg >= 0 && key >= beg && key <= row ? s[e] : 0.f;
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) add_columns<D>(dq, kt[buf], cb, 32 * n + 16 * b, operand(s, b), clean);
    }
  }
  if (beg >= 0) store_rows<D>(static_cast<__bf16*>(a.grad_q) + (long long)row * a.gqs + (long long)hq * D, dq, a.scale, hl);
}

// ------------------------------------------------------------------ dk, dv
template <int D, int NW> __global__ __launch_bounds__(64 * NW, 2) void attn_dkv_kernel(PromptBwdArgs a) {
  constexpr int BN = 32 * NW, NT = 64 * NW, KS = D / 16;
  __shared__ __bf16 qt[2][kN * D], gt[2][kN * D];
  __shared__ float lt[2][kN], dt[2][kN];
  __shared__ int begs[BN], ends[BN], window[BN + 1], most[NW];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  // the first tiles of a long sequence meet the most rows
  const int rank = blockIdx.x / a.Hkv, kvh = blockIdx.x - rank * a.Hkv;
  const int r0 = rank * BN, G = a.Hq / a.Hkv;

  find_rows<BN, NT>(a.cu, a.R, a.T, r0, window, begs, ends);
  int last = -1;  // the row behind the last that attends to a key of the tile
  for (int i = tid; i < BN; i += NT) last = max(last, ends[i]);
#pragma unroll
  for (int d = 32; d; d >>= 1) last = max(last, __shfl_xor(last, d));
  if (lane == 0) most[wave] = last;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) last = max(last, most[w]);
  last = __builtin_amdgcn_readfirstlane(last);
  if (last < 0) return;

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
      v[ks] = *reinterpret_cast<const u32x4*>(vp + 16 * ks);
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
  const int rb = row_base<D>(lane), cb = col_base<D>(lane);
  Stage<D, kN, NW> sq, sg;
  sq.init(a.qs, wave);
  sg.init(a.gos, wave);
  const __bf16* qp = static_cast<const __bf16*>(a.q);
  const __bf16* gp = static_cast<const __bf16*>(a.grad_out);
  auto stage = [&](int buf, int hq, int i0) {
    const int n = min(kN, last - i0);
    sq.load(qt[buf], rows_rsrc(qp + (long long)hq * D, a.qs, i0, n, D), wave);
    sg.load(gt[buf], rows_rsrc(gp + (long long)hq * D, a.gos, i0, n, D), wave);
    if (wave == 0) stage_words(lt[buf], pipe::make_rsrc(a.ws + (size_t)hq * a.T + i0, n * 4));
    if (wave == 1) stage_words(dt[buf], pipe::make_rsrc(a.ws + (size_t)(a.Hq + hq) * a.T + i0, n * 4));
  };
  const int steps = (last - r0 + kN - 1) / kN, total = steps * G;
  stage(0, kvh * G, r0);
  int buf = 0, head = 0, i0 = r0;
  for (int it = 0; it < total; ++it, buf ^= 1) {
    staged_barrier();
    int nh = head, ni = i0 + kN;
    if (ni >= last) {
      nh = head + 1;
      ni = r0;
    }
    if (it + 1 < total) stage(buf ^ 1, kvh * G + nh, ni);
    const int i1 = i0;
    head = nh;
    i0 = ni;
    if (i1 + kN - 1 < w0 || i1 >= highest) continue;
    const bool masked = i1 < w0 + 31 || i1 + kN > lowest;
    const bool clean = !masked || (clean_tile<D, kN>(qt[buf]) && clean_tile<D, kN>(gt[buf]));
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        s = mma(row_frag<D>(qt[buf], rb, 32 * n, ks), k[ks], s);
        dp = mma(row_frag<D>(gt[buf], rb, 32 * n, ks), v[ks], dp);
      }
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const f32x4 l = *reinterpret_cast<const f32x4*>(&lt[buf][32 * n + 8 * e4 + 4 * hl]);
        const f32x4 d = *reinterpret_cast<const f32x4*>(&dt[buf][32 * n + 8 * e4 + 4 * hl]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * e4 + j;
          s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -l[j]));
          dp[e] = s[e] * (dp[e] - d[j]);
        }
      }
      if (masked) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int i = i1 + 32 * n + 8 * (e / 4) + 4 * hl + e % 4;
          const bool seen = i >= key && i < end;
          s[e] = seen ? s[e] : 0.f;
          dp[e] = seen ? dp[e] : 0.f;
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        add_columns<D>(dv, gt[buf], cb, 32 * n + 16 * b, operand(s, b), clean);
        add_columns<D>(dk, qt[buf], cb, 32 * n + 16 * b, operand(dp, b), clean);
      }
    }
  }
  if (end >= 0) {
    store_rows<D>(static_cast<__bf16*>(a.grad_k) + (long long)key * a.gks + (long long)kvh * D, dk, a.scale, hl);
    store_rows<D>(static_cast<__bf16*>(a.grad_v) + (long long)key * a.gvs + (long long)kvh * D, dv, 1.f, hl);
  }
}

template <int D> hipError_t launch(const PromptBwdArgs& a) {
  constexpr int NW = 4;
  const unsigned tiles = (unsigned)((a.T + 32 * NW - 1) / (32 * NW));
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  const hipError_t e = launch_kernel(attn_dq_kernel<D, NW>, dim3(tiles * a.Hq), dim3(64 * NW), st, a);
  if (e != hipSuccess) return e;
  return launch_kernel(attn_dkv_kernel<D, NW>, dim3(tiles * a.Hkv), dim3(64 * NW), st, a);
}

}  // namespace

size_t attn_prompt_bwd_workspace_bytes(int T, int Hq) { return ((size_t)2 * T * Hq * sizeof(float) + 15) / 16 * 16; }

hipError_t launch_attn_prompt_bwd(const PromptBwdArgs& a) { return a.D == 64 ? launch<64>(a) : launch<128>(a); }

}  // namespace gdn
