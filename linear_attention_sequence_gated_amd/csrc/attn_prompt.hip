// attn_prompt.hip -- causal attention over packed prompts, forward.
#include "../../include/gdn.h"
#include "gdn_attn.hpp"
#include "gdn_launch.hpp"
#include "gdn_tile.hpp"

namespace gdn {
namespace {

using namespace tile;

constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;
constexpr float kLowest = -1e30f;  // running maximum before the first token
constexpr float kSlack = 8.f;      // the maximum in use may lie this far (powers of two) below the true one
constexpr int kN = 64;             // keys of a tile

template <int D, int QT, int NW> struct Fwd {
  static constexpr int BM = 32 * QT * NW, NT = 64 * NW, KS = D / 16, DT = D / 32;
  struct Lds {
    __bf16 k[2][kN * D];
    __bf16 v[2][kN * D];
    int beg[BM];
    int window[kWindow];
    int lo[NW], hi[NW];
  };
};

template <int D, int QT, int NW>
__global__ __launch_bounds__(64 * NW, QT == 2 && D == 128 ? 1 : 2) void attn_prompt_kernel(PromptArgs a) {
  using F = Fwd<D, QT, NW>;
  constexpr int BM = F::BM, NT = F::NT, KS = F::KS, DT = F::DT;
  __shared__ typename F::Lds lds;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hl = lane >> 5;
  const int tiles = (a.T + BM - 1) / BM;
  // the tiles with the most keys of a long sequence first, all heads of a tile side by side
  const int rank = blockIdx.x / a.Hq, hq = blockIdx.x - rank * a.Hq;
  const int r0 = (tiles - 1 - rank) * BM, kvh = hq / (a.Hq / a.Hkv);

  // queries: operands for the wave's rows, on their way while the sequences are found
  const int w0 = r0 + wave * 32 * QT;
  u32x4 q[QT][KS];
  int row[QT], beg[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    row[t] = w0 + 32 * t + (lane & 31);
    const __hip_bfloat16* src =
        static_cast<const __hip_bfloat16*>(a.q) + (long long)min(row[t], a.T - 1) * a.qs + (long long)hq * D + 8 * hl;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[t][ks] = *reinterpret_cast<const u32x4*>(src + 16 * ks);
  }
  find_rows<BM, NT>(a.cu, a.R, a.T, r0, lds.window, lds.beg, nullptr);
  int first = a.T, last = -1;  // the keys that the tile's rows see
  for (int i = tid; i < BM; i += NT)
    if (lds.beg[i] >= 0) {
      first = min(first, lds.beg[i]);
      last = max(last, r0 + i + 1);
    }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    first = min(first, __shfl_xor(first, d));
    last = max(last, __shfl_xor(last, d));
  }
  if (lane == 0) {
    lds.lo[wave] = first;
    lds.hi[wave] = last;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    first = min(first, lds.lo[w]);
    last = max(last, lds.hi[w]);
  }
  first = __builtin_amdgcn_readfirstlane(first);
  last = __builtin_amdgcn_readfirstlane(last);
  if (last < 0) {  // no row of the tile is in a sequence
    if (a.zero_rest) zero_rows<D>(static_cast<__bf16*>(a.out) + (long long)hq * D, (long long)a.Hq * D, r0, min(BM, a.T - r0), NT);
    if (a.zero_rest)
      for (int i = tid; i < BM && r0 + i < a.T; i += NT) a.lse[(size_t)hq * a.T + r0 + i] = 0.f;
    return;
  }

  int lowest = a.T, highest = -1;  // the range of beg over the wave's rows
  // a scale of zero stays just above it, so that masked scores, -infinity, keep
  // a weight of zero; for a negative one the queries' signs are turned
  const float c = fmaxf(__builtin_fabsf(a.scale) * kLog2e, 1e-37f);
  const unsigned flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    beg[t] = lds.beg[row[t] - r0];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[t][ks] ^= flip;
    lowest = min(lowest, beg[t] < 0 ? a.T : beg[t]);
    highest = max(highest, beg[t] < 0 ? a.T : beg[t]);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    lowest = min(lowest, __shfl_xor(lowest, d));
    highest = max(highest, __shfl_xor(highest, d));
  }
  lowest = __builtin_amdgcn_readfirstlane(lowest);
  highest = __builtin_amdgcn_readfirstlane(highest);

  int from[QT], upto[QT];  // the keys that the lane's row sees, less 4 hl
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    from[t] = beg[t] - 4 * hl;
    upto[t] = beg[t] < 0 ? -8 : row[t] - 4 * hl;
  }
  f32x16 o[QT][DT];
  float m[QT], l[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    m[t] = kLowest;
    l[t] = 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[t][i] = zero16();
  }

  const int kb = row_base<D>(lane), vb = col_base<D>(lane);
  Stage<D, kN, NW> sk, sv;
  sk.init(a.ks, wave);
  sv.init(a.vs, wave);
  const __hip_bfloat16* kp = static_cast<const __hip_bfloat16*>(a.k) + (long long)kvh * D;
  const __hip_bfloat16* vp = static_cast<const __hip_bfloat16*>(a.v) + (long long)kvh * D;
  auto stage = [&](int buf, int kv) {
    const int n = min(kN, last - kv);
    sk.load(lds.k[buf], rows_rsrc(kp, a.ks, kv, n, D), wave);
    sv.load(lds.v[buf], rows_rsrc(vp, a.vs, kv, n, D), wave);
  };
  int dirty_lo = last, dirty_hi = 0;  // the tiles with non-finite values that were left out
  // one tile of keys; MASKED: some of its keys are not seen by some of the rows
  auto step = [&](auto masked_, const __bf16* K, const __bf16* V, int kv) {
    constexpr bool MASKED = decltype(masked_)::value;
    f32x16 s[QT][2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int t = 0; t < QT; ++t) s[t][n] = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const u32x4 f = row_frag<D>(K, kb, 32 * n, ks);
#pragma unroll
        for (int t = 0; t < QT; ++t) s[t][n] = mma(f, q[t][ks], s[t][n]);
      }
    }
    u32x4 p[QT][4];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      if constexpr (MASKED) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int key = 32 * n + 8 * (e / 4) + e % 4;  // from kv + 4 hl on
            s[t][n][e] = key >= from[t] - kv && key <= upto[t] - kv ? s[t][n][e] : -INFINITY;
          }
      }
      float top = s[t][0][0];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[t][n][e]);
      top = max_halves(top) * c;
      if (__any(top > m[t] + kSlack)) {
        const float to = fmaxf(m[t], top), f = __builtin_amdgcn_exp2f(m[t] - to);
        m[t] = to;
        l[t] *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i) o[t][i] *= f;
      }
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][n][e], c, -m[t]));
          s[t][n][e] = x;
          sum += x;
        }
        p[t][2 * n] = operand(s[t][n], 0);
        p[t][2 * n + 1] = operand(s[t][n], 1);
      }
      l[t] += sum;
    }
    bool clean = true;
    if constexpr (MASKED) clean = clean_tile<D, kN>(V);
    if (clean) {
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const u32x4 f = col_frag<D>(V, vb, 16 * b, i);
#pragma unroll
          for (int t = 0; t < QT; ++t) o[t][i] = mma(f, p[t][b], o[t][i]);
        }
    } else {
      // values that some row does not see must not reach its sums: they are left
      // out here, and added to the rows that see them when all is written
      dirty_lo = min(dirty_lo, kv);
      dirty_hi = kv + kN;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const u32x4 f = finite_only(col_frag<D>(V, vb, 16 * b, i));
#pragma unroll
          for (int t = 0; t < QT; ++t) o[t][i] = mma(f, p[t][b], o[t][i]);
        }
    }
  };
  stage(0, first);
  int buf = 0;
  int kv = first;
  auto next = [&] {
    staged_barrier();
    if (kv + kN < last) stage(buf ^ 1, kv + kN);
  };
  // tiles of which some row misses some key, at both ends of the range, and
  // those between, which all rows see whole (loops apart: one loop with both
  // bodies takes more registers than there are)
  auto edge = [&](int end) {
    for (; kv < end; kv += kN, buf ^= 1) {
      next();
      if (kv <= w0 + 32 * QT - 1 && kv + kN > lowest) step(std::true_type{}, lds.k[buf], lds.v[buf], kv);
    }
  };
  edge(min(highest, last));
  for (; kv + kN - 1 <= w0; kv += kN, buf ^= 1) {
    next();
    step(std::false_type{}, lds.k[buf], lds.v[buf], kv);
  }
  edge(last);

#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const float z = sum_halves(l[t]);
    const bool rest = beg[t] < 0 && row[t] < a.T && a.zero_rest;
    const float inv = rest ? 0.f : 1.f / z;
    if (beg[t] >= 0 || rest) {
      __bf16* dst = static_cast<__bf16*>(a.out) + ((size_t)row[t] * a.Hq + hq) * D + 4 * hl;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<u32x2*>(dst + 32 * i + 8 * e) = pipe::cvt4(
              f32x4{o[t][i][4 * e] * inv, o[t][i][4 * e + 1] * inv, o[t][i][4 * e + 2] * inv, o[t][i][4 * e + 3] * inv});
      if (hl == 0) a.lse[(size_t)hq * a.T + row[t]] = rest ? 0.f : (m[t] + __builtin_amdgcn_logf(z)) * kLn2;
    }
  }  if (dirty_hi == 0) return;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    if (beg[t] < 0) continue;
    __bf16* dst = static_cast<__bf16*>(a.out) + ((size_t)row[t] * a.Hq + hq) * D;
    for (int key = max(beg[t], dirty_lo); key <= row[t] && key < dirty_hi; ++key) {
      const __bf16* src = static_cast<const __bf16*>(a.v) + (long long)key * a.vs + (long long)kvh * D;
      for (int d = 4 * hl; d < D; d += 8)  // the entries that this lane stored
        for (int i = 0; i < 4; ++i) {
          const float x = (float)src[d + i];
          if (!__builtin_isfinite(x)) dst[d + i] = (__bf16)((float)dst[d + i] + x);
        }
    }
  }
}

template <int D, int QT, int NW> hipError_t launch(const PromptArgs& a) {
  constexpr int BM = Fwd<D, QT, NW>::BM;
  const unsigned tiles = (unsigned)((a.T + BM - 1) / BM);
  return launch_kernel(attn_prompt_kernel<D, QT, NW>, dim3(tiles * a.Hq), dim3(64 * NW), static_cast<hipStream_t>(a.stream), a);
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& a) {
  return a.D == 64 ? launch<64, 1, 4>(a) : launch<128, 1, 4>(a);
}

}  // namespace gdn
