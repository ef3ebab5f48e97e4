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
    int window[BM + 1];
    int lo[NW];
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

  find_rows<BM, NT>(a.cu, a.R, a.T, r0, lds.window, lds.beg, nullptr);
  int first = a.T;  // first key that any row of the tile sees
  for (int i = tid; i < BM; i += NT)
    if (lds.beg[i] >= 0) first = min(first, lds.beg[i]);
#pragma unroll
  for (int d = 32; d; d >>= 1) first = min(first, __shfl_xor(first, d));
  if (lane == 0) lds.lo[wave] = first;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) first = min(first, lds.lo[w]);
  first = __builtin_amdgcn_readfirstlane(first);
  if (first >= a.T) return;  // no row of the tile is in a sequence
  const int last = min(r0 + BM, a.T);

  // queries: operands for the wave's rows, their sign turned for a negative scale
  const int w0 = r0 + wave * 32 * QT;
  u32x4 q[QT][KS];
  int row[QT], beg[QT];
  int lowest = a.T, highest = -1;  // the range of beg over the wave's rows
  const float c = __builtin_fabsf(a.scale) * kLog2e;
  const unsigned flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    row[t] = w0 + 32 * t + (lane & 31);
    beg[t] = lds.beg[row[t] - r0];
    const __hip_bfloat16* src =
        static_cast<const __hip_bfloat16*>(a.q) + (long long)min(row[t], a.T - 1) * a.qs + (long long)hq * D + 8 * hl;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[t][ks] = *reinterpret_cast<const u32x4*>(src + 16 * ks);
      q[t][ks] ^= flip;
    }
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
  stage(0, first);
  int buf = 0;
  for (int kv = first; kv < last; kv += kN, buf ^= 1) {
    staged_barrier();
    if (kv + kN < last) stage(buf ^ 1, kv + kN);
    if (kv > w0 + 32 * QT - 1 || kv + kN <= lowest) continue;  // nothing of it is seen by the wave's rows
    const bool masked = kv + kN - 1 > w0 || kv < highest || kv + kN > last;
    const __bf16 *K = lds.k[buf], *V = lds.v[buf];
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
      if (masked) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int key = kv + 32 * n + 8 * (e / 4) + 4 * hl + e % 4;
            const bool seen = beg[t] >= 0 && key >= beg[t] && key <= row[t];
            s[t][n][e] = seen ? s[t][n][e] : -INFINITY;
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
          float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][n][e], c, -m[t]));
          if (masked) x = s[t][n][e] == -INFINITY ? 0.f : x;
          s[t][n][e] = x;
          sum += x;
        }
        p[t][2 * n] = operand(s[t][n], 0);
        p[t][2 * n + 1] = operand(s[t][n], 1);
      }
      l[t] += sum;
    }
    bool clean = true;
    if (masked) {  // values that no row sees must not reach the sums, whatever they are
      unsigned w = 0;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const u32x4 f = col_frag<D>(V, vb, 16 * b, i);
          w = worst(worst(w, f[0]), f[1]);
          w = worst(worst(w, f[2]), f[3]);
        }
      clean = __all(finite(w));
    }
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
      // finite values as ever; the others through the sum of the weights that meet them
#pragma unroll 1
      for (int kind = 0; kind < 4; ++kind)
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int t = 0; t < QT; ++t) {
            f32x16 x = kind ? zero16() : o[t][i];
#pragma unroll
            for (int b = 0; b < 4; ++b) x = mma(pick(col_frag<D>(V, vb, 16 * b, i), kind), p[t][b], x);
            const float bad = kind == 1 ? INFINITY : kind == 2 ? -INFINITY : __builtin_nanf("");
#pragma unroll
            for (int e = 0; e < 16; ++e) o[t][i][e] = kind == 0 ? x[e] : x[e] > 0.f ? o[t][i][e] + bad : o[t][i][e];
          }
    }
  }

#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const float z = sum_halves(l[t]), inv = 1.f / z;
    if (beg[t] >= 0) {
      __bf16* dst = static_cast<__bf16*>(a.out) + ((size_t)row[t] * a.Hq + hq) * D + 4 * hl;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<u32x2*>(dst + 32 * i + 8 * e) = pipe::cvt4(
              f32x4{o[t][i][4 * e] * inv, o[t][i][4 * e + 1] * inv, o[t][i][4 * e + 2] * inv, o[t][i][4 * e + 3] * inv});
      if (hl == 0) a.lse[(size_t)hq * a.T + row[t]] = (m[t] + __builtin_amdgcn_logf(z)) * kLn2;
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
