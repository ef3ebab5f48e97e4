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
// bf16 (2^-8 of each, the operands' own precision), go from accumulator to
// operand in place.  K and V are staged in LDS by direct loads, one tile ahead,
// and read there by rows (K) and transposed (V).  Rows are cut into tiles where
// they lie, whatever sequences they belong to: tiles that some row sees in part
// are masked, those that all rows see whole are not.  The workgroups of the
// heads that share keys are neighbours.
//
// What bounds it is the matrix and the vector unit together: 32 keys of a wave's
// 32 rows are 4 D / 32 products of 32 cycles and 16 lanes' exponentials, with as
// many multiply-adds, sums and maxima.  1 x 16384 x 16/4 x 64 takes 578 us, 950
// TFLOP/s of the 1600 that the largest library products reach here; 8 x 2048 x
// 12/4 x 64 70 us; 1 x 16384 x 16/4 x 128 1030 us, 1060 TFLOP/s.  Without the softmax the same
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

template <int D, int NW> __global__ __launch_bounds__(64 * NW, D == 64 ? 4 : 3) void attn_prompt_kernel(PromptArgs a) {
  // keys of a staged tile: 64 at D = 64, where 125 registers let four workgroups
  // share a CU (578 us for 1 x 16384 x 16/4 x 64; with 32 keys 620); 32 at
  // D = 128, where that takes 158 registers and three workgroups a CU (67.7 us for
  // 13 prompts of up to 1201 rows x 16/4 x 128; with 64 keys and two 70.5)
  constexpr int kN = D == 64 ? 64 : 32, NH = kN / 32;
  constexpr int BM = 32 * NW, NT = 64 * NW, KS = D / 16, DT = D / 32;
  __shared__ alignas(16) __bf16 kt[2][kN * D], vt[2][kN * D];
  __shared__ int begs[BM], window[kWindow], ranges[3][NW], bad[2][NW];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  const int tiles = (a.T + BM - 1) / BM;
  // the tiles with the most keys (of a long sequence: the last) first, all heads of a tile side by side
  const int rank = blockIdx.x / a.Hq, hq = blockIdx.x - rank * a.Hq;
  int tile = tiles - 1 - rank;
  if (a.by_length) tile = tile_by_length<BM, NT, false>(a.cu, a.R, a.T, tiles, rank, window, reinterpret_cast<int*>(kt));
  const int r0 = tile * BM, kvh = hq / (a.Hq / a.Hkv);

  // queries: operands for the wave's rows
  const int w0 = r0 + wave * 32, row = w0 + (lane & 31);
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

  f32x16 o[DT];
  float m = kLowest, l = 0.f;
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zero16();

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
  // one tile of keys; MASKED: some of its keys are not seen by some of the rows
  auto step = [&](auto masked_, int buf, int kv) {
    constexpr bool MASKED = decltype(masked_)::value;
    const int kb = fresh(kb0), vb = fresh(vb0);
    f32x16 s[NH];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      s[n] = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) s[n] = mma(row_frag<D>(kt[buf], kb, 32 * n, ks), q[ks], s[n]);
    }
    if constexpr (MASKED) {
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        const unsigned seen = bits(from - kv - 32 * n, upto - kv - 32 * n);
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
    if (__any(top > m + kSlack)) {
      const float to = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i] *= f;
    }
    u32x4 p[2 * NH];
    float sum = 0.f;
#pragma unroll
    for (int n = 0; n < NH; ++n) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[n][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][e], c, -m));
        sum += s[n][e];
      }
      p[2 * n] = operand(s[n], 0);
      p[2 * n + 1] = operand(s[n], 1);
    }
    l += sum;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int b = 0; b < 2 * NH; ++b) o[i] = mma(col_frag<D>(vt[buf], vb, 16 * b, i), p[b], o[i]);
  };
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
  // tiles of which some row misses some key, at both ends of the range, and
  // those between, which all rows see whole (loops apart: one loop with both
  // bodies takes more registers than there are)
  auto edge = [&](int end) {
    for (; kv < end; kv += kN, buf ^= 1) {
      next();
      if (kv <= w0 + 31 && kv + kN > lowest) step(std::true_type{}, buf, kv);
    }
  };
  edge(min(highest, last));
  for (; kv + kN - 1 <= w0; kv += kN, buf ^= 1) {
    next();
    step(std::false_type{}, buf, kv);
  }
  edge(last);

  const float z = sum_halves(l);
  const bool rest = beg < 0 && row < a.T && a.zero_rest;
  if (beg < 0 && !rest) return;
  const float inv = rest ? 0.f : 1.f / z;
  __bf16* dst = static_cast<__bf16*>(a.out) + ((size_t)row * a.Hq + hq) * D;
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<u32x2*>(dst + 32 * i + 8 * e + 4 * hl) =
          pipe::cvt4(f32x4{o[i][4 * e] * inv, o[i][4 * e + 1] * inv, o[i][4 * e + 2] * inv, o[i][4 * e + 3] * inv});
  if (hl == 0) a.lse[(size_t)hq * a.T + row] = rest ? 0.f : (m + __builtin_amdgcn_logf(z)) * kLn2;
  if (rest) return;
  for (int key = max(beg, dirty_lo); key <= row && key < dirty_hi; ++key) {
    const __bf16* src = static_cast<const __bf16*>(a.v) + (long long)key * a.vs + (long long)kvh * D;
    for (int d = 4 * hl; d < D; d += 8)  // the entries that this lane stored
      for (int i = 0; i < 4; ++i) {
        const float x = (float)src[d + i];
        if (!__builtin_isfinite(x)) dst[d + i] = (__bf16)((float)dst[d + i] + x);
      }
  }
}

template <int D> hipError_t launch(const PromptArgs& a) {
  constexpr int NW = 4;
  const unsigned tiles = (unsigned)((a.T + 32 * NW - 1) / (32 * NW));
  return launch_kernel(attn_prompt_kernel<D, NW>, dim3(tiles * a.Hq), dim3(64 * NW), static_cast<hipStream_t>(a.stream), a);
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& args) {
  PromptArgs a = args;
  a.by_length = rank_tiles(a.T, a.R, a.Hq);
  return a.D == 64 ? launch<64>(a) : launch<128>(a);
}

}  // namespace gdn
