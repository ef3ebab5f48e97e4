// attn_decode.hip -- attention of one new token per request over the 8-bit
// paged cache.
//
// For a request's n tokens and one key head, with codes kc, vc and the scales
// ks, vs of the token's block,
//   s_j = scale ks_j (q . kc_j),   o = sum_j e^(s_j) vs_j vc_j / sum_j e^(s_j).
// The cache is read once (2 D bytes per token and head); everything else is
// small, so the kernel is bound by HBM and is built to keep loads in flight.
//
// Where no request can be long, by the width of the table, a workgroup takes all
// of one (request, head).  Otherwise work is counted in units of 128 tokens of one
// (request, head), one more for its beginning and end, and dealt out in equal contiguous shares to a fixed
// number of workgroups, whatever the lengths: a long request is split over many workgroups and short ones are
// taken several to a workgroup.  The shares follow from the lengths, which
// only the device knows, so every workgroup finds its own with a prefix sum.
// A workgroup that covers all of a (request, head) writes the result;
// otherwise it writes its sums, its share's maximum included, and a second
// launch joins them in the order of the tokens.
//
// The query heads that share a key head (up to 16 at a time) are the columns of
// the products: S^T = K Q^T and O^T = V^T P^T, both 16x16x32 in fp16.  The
// accumulator layout of S^T is the operand layout of P^T, so probabilities
// never leave their lane.  Codes are exact in fp16 (int8 through u 2^-10 -
// 128 2^-10, one packed multiply-add for two); q is moved into fp16's range by
// a power of two per head, which is exact down to 2^-28 of its largest entry.
// The running maximum m is that of s_j + log2 vs_j less 15, so that the weights
// p_j = 2^(s_j - m) vs_j that are rounded to fp16 are at most 2^15 whatever the
// blocks' scales: half an ulp, 2^-11 of each that is at least e^-20 of the largest,
// 2^-40 of the largest of those below.  (At most one, they lost a flat tail 17 below
// one high score, whose value may be zero.)  The denominator sums 2^(s_j - m) in
// float32.
//
// 4 x 65521 tokens x 16/4 x 128 take 49 us, 5.4 TB/s, and 5 us to join; 64
// requests of up to 4099 tokens 29 us, 4.0 TB/s, the longest's tiles on one CU; one
// of 777 x 12/4 x 64 6.6 us, the chain of lengths, table, codes and four tiles a
// wave.  More shares than the CUs hold at once, and eight waves to a share, were
// slower.
#include <hip/hip_bf16.h>

#include <algorithm>

#include "../../include/gdn.h"
#include "gdn_attn.hpp"
#include "gdn_launch.hpp"
#include "gdn_pipe.hpp"

namespace gdn {
namespace {

using pipe::make_rsrc;
using pipe::u32x2;
using pipe::u32x4;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

constexpr int kUnit = 128, kTile = 32;  // tokens of a unit, of a wave's tile
// To begin a (request, head) and to end it take about the time of a unit.  Counted
// so, 64 ragged requests x 16/4 x 128 take 28.9 us for 34.3 uncounted, 256 of up
// to 1000 tokens 46.3 for 51.7; 4 x 65521 tokens 61.6 for 60.9.
constexpr int kAhead = 1;
constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;
constexpr float kLowest = -3e38f;  // running maximum before the first token
constexpr float kCodeUp = 1024.f;  // int8 codes enter the products times 2^-10
// The maximum in use lies kUp below the true one, so that the largest weights are
// 2^15 and those down to 2^-29 of it (e^-20) normal numbers of fp16, which ends at
// 65504.  Not where scores pass 2^24: their sums with log2 vs_j are off by more
// than a power of two, and the room is needed for that.
constexpr float kUp = 15.f, kUpBelow = 16777216.f;
// What the denominator sums is 2^(s_j - m), 2^kUp / vs_j where vs_j's token has the
// maximum: for the scales' whole range (2^-126 to 2^121) to fit float32 with 2^31
// tokens, log2 vs_j counts as kLeastLog at least in m (the largest weights of
// smaller scales are below 2^15, still normal), and the sums are taken times 2^-kDown.
constexpr float kLeastLog = -97.f, kDown = 16.f;
constexpr float kDownBy = 1.f / 65536;  // 2^-kDown

// Shares of the work: what the CUs hold at once (three workgroups of the at most
// 168 registers that d = 64 takes, two at d = 128).
constexpr int most_shares(int D) { return 256 * (D == 64 ? 3 : 2); }

struct DecodeSizes {
  int R, Hq, Hkv, G, NG, Gc, bt, width, num_blocks, W, whole;  // whole: waves of a workgroup that takes a whole (request, key head), or 0
};

// Tokens of a request that its table row can hold.
__device__ __forceinline__ int tokens_of(const int* lens, int r, const DecodeSizes& z) {
  const int n = lens[r];
  const long long most = (long long)z.width * z.bt;
  return n <= 0 ? 0 : (n < most ? n : (int)most);
}
__device__ __forceinline__ int units_of(int n) { return (n + kUnit - 1) / kUnit; }
// What a (request, head) counts for where the work is dealt out: kAhead for its
// beginning and end, then its units.
__device__ __forceinline__ int cost_of(int n) { return n ? kAhead + units_of(n) : 0; }

__device__ __forceinline__ int wave_scan(int x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if ((int)(threadIdx.x & 63) >= d) x += y;
  }
  return x;
}

// Two int8 codes (offset by 128), zero-extended to 16 bits, as fp16 times 2^-10.
__device__ __forceinline__ unsigned i8_f16(unsigned w) {
  const f16x2 up{(_Float16)16384.f, (_Float16)16384.f}, off{(_Float16)-0.125f, (_Float16)-0.125f};
  return __builtin_bit_cast(unsigned, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, w), up, off));
}
template <bool HI> __device__ __forceinline__ unsigned e4m3_f16(unsigned w) {
  return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.f, HI));
}

// Eight consecutive codes as an fp16 operand.
template <int FMT> __device__ __forceinline__ f16x8 codes8(unsigned a, unsigned b) {
  u32x4 r;
  if constexpr (FMT == GDN_CACHE_I8) {
    a ^= 0x80808080u;
    b ^= 0x80808080u;
    r[0] = i8_f16(__builtin_amdgcn_perm(0u, a, 0x0c010c00u));
    r[1] = i8_f16(__builtin_amdgcn_perm(0u, a, 0x0c030c02u));
    r[2] = i8_f16(__builtin_amdgcn_perm(0u, b, 0x0c010c00u));
    r[3] = i8_f16(__builtin_amdgcn_perm(0u, b, 0x0c030c02u));
  } else {
    r[0] = e4m3_f16<false>(a);
    r[1] = e4m3_f16<true>(a);
    r[2] = e4m3_f16<false>(b);
    r[3] = e4m3_f16<true>(b);
  }
  return __builtin_bit_cast(f16x8, r);
}

// Four rows of four codes (row j in w[j]) as four columns: out[i] holds code i
// of the four rows as fp16 (two words).
template <int FMT> __device__ __forceinline__ void columns4(const unsigned (&w)[4], u32x2 (&out)[4]) {
  if constexpr (FMT == GDN_CACHE_I8) {
    unsigned x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = w[j] ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned sel = 0x0c000c00u | (unsigned)i | ((unsigned)(4 + i) << 16);
      out[i] = u32x2{i8_f16(__builtin_amdgcn_perm(x[1], x[0], sel)), i8_f16(__builtin_amdgcn_perm(x[3], x[2], sel))};
    }
  } else {
    // bytes (0, 1) and (2, 3) of the row pairs, then the pairs side by side
    const unsigned a01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), a23 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
    const unsigned b01 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), b23 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    out[0] = u32x2{e4m3_f16<false>(a01), e4m3_f16<false>(b01)};
    out[1] = u32x2{e4m3_f16<true>(a01), e4m3_f16<true>(b01)};
    out[2] = u32x2{e4m3_f16<false>(a23), e4m3_f16<false>(b23)};
    out[3] = u32x2{e4m3_f16<true>(a23), e4m3_f16<true>(b23)};
  }
}

// A wave's tile of 32 tokens: two halves of 16, which may lie in two blocks.
// Lane (g, c) holds of half j the codes 16 g .. (D = 64) or 32 g .. (D = 128)
// of token c for K, and NB codes from NB c on of tokens 4 g + i for V.
template <int D> struct Tile {
  static constexpr int KW = D / 16, VW = D / 64, NB = D / 16;  // words
  unsigned k[2][KW];
  unsigned v[2][4][VW];
  float ks[2], vs[2];
  int n[2];  // tokens of the half that count
};

// The blocks that a wave's tile lies in (any where it has no tokens).
struct Blocks {
  int id[2];
};
__device__ __forceinline__ Blocks blocks_of(int tok, int n, const int* row, int bt) {
  const int sh = __builtin_ctz(bt);
  return {{tok < n ? row[tok >> sh] : 0, tok + 16 < n ? row[(tok + 16) >> sh] : 0}};
}

template <int D>
__device__ __forceinline__ void load_tile(Tile<D>& t, const Blocks& b, int tok, int n, int h, const DecodeArgs& a,
                                          const DecodeSizes& z) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int p = tok + 16 * j;
    int left = n - p;
    left = left < 0 ? 0 : (left > 16 ? 16 : left);
    int id = b.id[j];
    if (id < 0 || id >= z.num_blocks) left = 0;
    if (!left) id = 0;
    const size_t tile = (size_t)id * z.Hkv + h;
    const size_t at = (tile * z.bt + (p & (z.bt - 1))) * D;
    const __amdgpu_buffer_rsrc_t rk = make_rsrc(static_cast<const char*>(a.k_cache) + at, left * D);
    const __amdgpu_buffer_rsrc_t rv = make_rsrc(static_cast<const char*>(a.v_cache) + at, left * D);
    t.n[j] = left;
    t.ks[j] = left ? a.k_scale[tile] : 0.f;
    t.vs[j] = left ? a.v_scale[tile] : 1.f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const u32x4 w = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(rk, c * D + (D / 4) * g + 16 * i, 0, 0));
#pragma unroll
      for (int e = 0; e < 4; ++e) t.k[j][4 * i + e] = w[e];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int off = (4 * g + i) * D + (D / 16) * c;
      if constexpr (D == 64) {
        t.v[j][i][0] = __builtin_amdgcn_raw_buffer_load_b32(rv, off, 0, 0);
      } else {
        const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rv, off, 0, 0));
        t.v[j][i][0] = w[0];
        t.v[j][i][1] = w[1];
      }
    }
  }
}

// What a wave carries over the tokens of a (request, head): lane (g, c) has
// column c (a query head), rows NB (4 g + r) + i of O^T in acc[i][r].
template <int D> struct Sums {
  f32x4 acc[D / 16];
  float m, l;  // m is shared by the lanes of a column, l is the lane's own part
};

template <int D, int FMT>
__device__ __forceinline__ void take_tile(Sums<D>& s, const Tile<D>& t, const f16x8 (&q)[D / 32], float qfac) {
  constexpr int NB = D / 16;
  const int g = (threadIdx.x & 63) >> 4;
  float x[2][4], top = kLowest;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    f32x4 y = pipe::zero4();
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks)
      y = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes8<FMT>(t.k[j][2 * ks], t.k[j][2 * ks + 1]), q[ks], y, 0, 0, 0);
    const float f = qfac * t.ks[j];
    const float lv = fmaxf(__builtin_amdgcn_logf(t.vs[j]), kLeastLog);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[j][i] = 4 * g + i < t.n[j] ? y[i] * f : -INFINITY;
      top = fmaxf(top, x[j][i] + lv);
    }
  }
  top = fmaxf(top, __shfl_xor(top, 16));
  top = fmaxf(top, __shfl_xor(top, 32));
  const float m = fmaxf(s.m, fabsf(top) < kUpBelow ? top - kUp : top);
  if (__any(m != s.m)) {
    const float c = __builtin_amdgcn_exp2f(s.m - m);
    s.l *= c;
#pragma unroll
    for (int i = 0; i < NB; ++i) s.acc[i] *= c;
    s.m = m;
  }
  f16x8 p;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = __builtin_amdgcn_exp2f(x[j][i] - m);
      s.l = __builtin_fmaf(e, kDownBy, s.l);
      p[4 * j + i] = (_Float16)(e * t.vs[j]);
    }
  }
#pragma unroll
  for (int w = 0; w < D / 64; ++w) {
    u32x2 col[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned rows[4] = {t.v[j][0][w], t.v[j][1][w], t.v[j][2][w], t.v[j][3][w]};
      columns4<FMT>(rows, col[j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 v{col[0][i][0], col[0][i][1], col[1][i][0], col[1][i][1]};
      s.acc[4 * w + i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, v), p, s.acc[4 * w + i], 0, 0, 0);
    }
  }
}

// The request that unit u = at(U) lies in, of U units over all (request, head)s,
// and its own first unit (both undefined if u is not below U).  By 256 threads;
// scan and found are scratch in LDS.
struct Place {
  long long U, u, base;
  int r;
};
template <class At> __device__ __forceinline__ Place place_of(const DecodeArgs& a, const DecodeSizes& z, int* scan, int* found, At at) {
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), heads = z.Hkv * z.NG;
  const int per = (z.R + 255) / 256, ra = tid * per;
  int mine = 0;
  for (int i = 0; i < per; ++i)
    if (ra + i < z.R) mine += cost_of(tokens_of(a.seq_lens, ra + i, z));
  const int incl = wave_scan(mine);
  if ((tid & 63) == 63) scan[wave] = incl;
  __syncthreads();
  int before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) before += scan[w];
    total += scan[w];
  }
  Place p;
  p.U = (long long)total * heads;
  p.u = at(p.U);
  if (p.u >= (long long)before * heads && p.u < (long long)(before + mine) * heads) {
    int r = ra, first = before;
    for (;; ++r) {
      const int n = cost_of(tokens_of(a.seq_lens, r, z));
      if (p.u < (long long)(first + n) * heads) break;
      first += n;
    }
    found[0] = r;
    found[1] = first;
  }
  __syncthreads();
  p.r = __builtin_amdgcn_readfirstlane(found[0]);
  p.base = (long long)__builtin_amdgcn_readfirstlane(found[1]) * heads;
  return p;
}

// The workspace: two slots to a share, outputs [2 W][Gc][D] and behind them maxima
// and sums [2 W][Gc][2], so that each is aligned to what it is read by (a slot of
// both would begin 8 bytes off for every other odd Gc).
__device__ __forceinline__ float* outputs_at(const DecodeArgs& a, const DecodeSizes& z, int D, size_t slot) {
  return a.ws + slot * z.Gc * D;
}
__device__ __forceinline__ float* sums_at(const DecodeArgs& a, const DecodeSizes& z, int D, size_t slot) {
  return a.ws + (size_t)2 * z.W * z.Gc * D + slot * z.Gc * 2;
}

template <int D, int FMT, int NW, bool WHOLE> __global__ __launch_bounds__(64 * NW, 2) void attn_decode_kernel(DecodeArgs a, DecodeSizes z) {
  constexpr int NB = D / 16, LD = D + 4, kStep = NW * kTile;
  static_assert(WHOLE || kStep == kUnit, "");
  __shared__ alignas(16) float part[NW][16][LD];
  __shared__ float ml[NW][2][16];
  __shared__ int scan[4], found[2];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g = lane >> 4, c = lane & 15;
  const int heads = z.Hkv * z.NG;

  // this workgroup's share [u0, u1) of the units, and the request it starts in
  Place at{};
  long long u0 = 0, u1 = 0;
  if constexpr (!WHOLE) {
    at = place_of(a, z, scan, found, [&](long long U) { return U * blockIdx.x / z.W; });
    u0 = at.u;
    u1 = at.U * (blockIdx.x + 1) / z.W;
    if (u0 >= u1) return;
  }
  // the part of one (request, key head) that a share covers: units [ua, ub)
  struct Part {
    int r, n, nu, cost, h, q0, cols, ua, ub;  // ub <= ua: nothing but of what stands ahead
    long long next;
  };
  int r = WHOLE ? (int)blockIdx.x / heads : at.r;
  long long base = at.base;  // first unit of request r
  auto part_at = [&](long long u) {
    Part p;
    p.r = r;
    p.n = tokens_of(a.seq_lens, r, z);
    p.nu = units_of(p.n);
    p.cost = kAhead + p.nu;
    const int hh = WHOLE ? (int)u : (int)((u - base) / p.cost);
    p.h = hh / z.NG;
    p.q0 = p.h * z.G + (hh - p.h * z.NG) * 16;
    p.cols = min(16, (p.h + 1) * z.G - p.q0);
    if constexpr (WHOLE) {
      p.ua = 0;
      p.ub = p.nu;
      return p;
    }
    const int from = (int)(u - base - (long long)hh * p.cost) - kAhead;
    p.ua = max(from, 0);
    p.ub = (int)min((long long)p.nu, from + (u1 - u));
    p.next = u + (p.ub - from);
    return p;
  };
  Tile<D> t0, t1;
  // of the tile after next: the table is read a tile before the codes that it leads
  // to (64 x 4000 x 16/4 x 64 27.4 us for 30; a third tile on its way costs 3 %)
  Blocks ahead;
  u32x4 qw[D / 32];
  // its queries and first tile, on their way while the part before it is joined
  auto begin = [&](const Part& p) {
    const __hip_bfloat16* src =
        static_cast<const __hip_bfloat16*>(a.q) + (long long)p.r * a.qs + (long long)(p.q0 + min(c, p.cols - 1)) * D;
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks) qw[ks] = *reinterpret_cast<const u32x4*>(src + (D / 4) * g + 8 * ks);
    const int tok = p.ua * kUnit + wave * kTile, end = min(p.n, p.ub * kUnit);
    if (tok < end) {
      const int* row = a.block_table + (size_t)p.r * z.width;
      load_tile<D>(t0, blocks_of(tok, end, row, z.bt), tok, end, p.h, a, z);
      ahead = blocks_of(tok + kStep, end, row, z.bt);
    }
  };

  bool first = true;
  Part cur = part_at(WHOLE ? blockIdx.x - r * heads : u0);
  if (!WHOLE && cur.ub <= cur.ua) return;
  begin(cur);
  for (;;) {
    const int nu = cur.nu, h = cur.h, q0 = cur.q0, cols = cur.cols, ua = cur.ua, ub = cur.ub, rr = cur.r;
    const int* row = a.block_table + (size_t)rr * z.width;

    // query operands, moved into fp16's range
    f16x8 q[D / 32];
    float qfac;
    {
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(pipe::lo_f(qw[ks][e])), fabsf(pipe::hi_f(qw[ks][e]))));
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const int e2 = __builtin_amdgcn_frexp_expf(top);
      const float down = __builtin_amdgcn_ldexpf(1.f, 14 - e2 > 126 ? 126 : 14 - e2);
      qfac = a.scale * kLog2e / down * (FMT == GDN_CACHE_I8 ? kCodeUp : 1.f);
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q[ks][2 * e] = (_Float16)(pipe::lo_f(qw[ks][e]) * down);
          q[ks][2 * e + 1] = (_Float16)(pipe::hi_f(qw[ks][e]) * down);
        }
    }

    Sums<D> s;
    s.m = kLowest;
    s.l = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i) s.acc[i] = pipe::zero4();
    const int end = min(cur.n, ub * kUnit);
    int tok = ua * kUnit + wave * kTile;
    if (tok < end) {
      for (;;) {
        if (tok + kStep < end) load_tile<D>(t1, ahead, tok + kStep, end, h, a, z);
        ahead = blocks_of(tok + 2 * kStep, end, row, z.bt);
        take_tile<D, FMT>(s, t0, q, qfac);
        tok += kStep;
        if (tok >= end) break;
        if (tok + kStep < end) load_tile<D>(t0, ahead, tok + kStep, end, h, a, z);
        ahead = blocks_of(tok + 2 * kStep, end, row, z.bt);
        take_tile<D, FMT>(s, t1, q, qfac);
        tok += kStep;
        if (tok >= end) break;
      }
    }

    const long long u = cur.next;
    bool more = !WHOLE && u < u1;
    if (more) {
      if (u >= base + (long long)cur.cost * heads) {  // the next request that has tokens
        base += (long long)cur.cost * heads;
        for (++r;; r += 64) {
          const unsigned long long some = __ballot(r + lane < z.R && tokens_of(a.seq_lens, min(r + lane, z.R - 1), z) > 0);
          if (some) {
            r += __builtin_ctzll(some);
            break;
          }
        }
        r = __builtin_amdgcn_readfirstlane(r);
      }
      cur = part_at(u);
      more = cur.ub > cur.ua;
      if (more) begin(cur);
    }

    // join the waves
    s.l += __shfl_xor(s.l, 16);
    s.l += __shfl_xor(s.l, 32);
    if (lane < 16) {
      ml[wave][0][c] = s.m;
      ml[wave][1][c] = s.l;
    }
    __syncthreads();
    float M = ml[0][0][c];
#pragma unroll
    for (int w = 1; w < NW; ++w) M = fmaxf(M, ml[w][0][c]);
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) L += ml[w][1][c] * __builtin_amdgcn_exp2f(ml[w][0][c] - M);
    const float mine_w = __builtin_amdgcn_exp2f(s.m - M) * (FMT == GDN_CACHE_I8 ? kCodeUp * kDownBy : kDownBy);
    if (c < cols) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int w = 0; w < NB / 4; ++w)
          *reinterpret_cast<f32x4*>(&part[wave][c][NB * (4 * g + i) + 4 * w]) =
              f32x4{s.acc[4 * w][i] * mine_w, s.acc[4 * w + 1][i] * mine_w, s.acc[4 * w + 2][i] * mine_w,
                    s.acc[4 * w + 3][i] * mine_w};
    }
    const bool whole = ua == 0 && ub == nu;
    const size_t slot = 2 * (size_t)blockIdx.x + (first ? 0 : 1);
    float *o_ws = outputs_at(a, z, D, slot), *m_ws = sums_at(a, z, D, slot);
    if (wave == 0 && lane < cols) {
      if (whole) {
        if (a.lse) a.lse[(size_t)rr * z.Hq + q0 + lane] = L == 0.f ? -INFINITY : (M + (kDown + __builtin_amdgcn_logf(L))) * kLn2;
      } else {
        m_ws[2 * lane] = M;
        m_ws[2 * lane + 1] = L;
      }
    }
    __syncthreads();
    for (int x = tid; x < cols * D / 4; x += 64 * NW) {
      const int col = x / (D / 4), d = 4 * (x % (D / 4));
      f32x4 o = pipe::zero4();
#pragma unroll
      for (int w = 0; w < NW; ++w) o += *reinterpret_cast<const f32x4*>(&part[w][col][d]);
      if (whole) {
        float Mc = ml[0][0][col], Lc = 0.f;
#pragma unroll
        for (int w = 1; w < NW; ++w) Mc = fmaxf(Mc, ml[w][0][col]);
#pragma unroll
        for (int w = 0; w < NW; ++w) Lc += ml[w][1][col] * __builtin_amdgcn_exp2f(ml[w][0][col] - Mc);
        const float inv = Lc == 0.f ? 0.f : 1.f / Lc;
        o *= inv;
        *reinterpret_cast<u32x2*>(static_cast<__bf16*>(a.out) + ((size_t)rr * z.Hq + q0 + col) * D + d) = pipe::cvt4(o);
      } else {
        *reinterpret_cast<f32x4*>(o_ws + col * D + d) = o;
      }
    }
    if (!more) return;
    __syncthreads();
    first = false;
  }
}

// The workgroup that takes unit x of U: the first whose share ends past it.
__device__ __forceinline__ int taker(long long x, long long U, const DecodeSizes& z) {
  return (int)(((x + 1) * z.W + U - 1) / U - 1);
}

// Joins the shares of one (request, query head), in the order of the tokens;
// heads that one workgroup covered are done already.  Requests without tokens
// get their zeros here.  Either a workgroup (DS of them, for D / DS columns
// each) sees to one row of the output, or (CUTS) to a column of the head that
// the end of one share lies in, if no share before it ends there too.
template <int D, int DS, bool CUTS> __global__ __launch_bounds__(128 * (DS == 1 ? 2 : 4)) void attn_decode_join_kernel(DecodeArgs a, DecodeSizes z) {
  constexpr int NT = DS == 1 ? 256 : 512, C = D / DS, NP = NT / (C / 4);  // shares taken side by side
  static_assert(!CUTS || DS == 1, "");
  __shared__ alignas(16) float sum[NT / 64][C], ls[NT / 64], weight[most_shares(D)], part_l[most_shares(D)], red[NT / 64];
  __shared__ int scan[2][NT / 64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, heads = z.Hkv * z.NG;
  int r, hq, col, d0 = 0, i0, i1;
  long long U, P;  // P: the row's first unit
  if constexpr (CUTS) {
    const int cuts = (z.W - 1) * z.Gc;
    if ((int)blockIdx.x >= cuts) {  // zeros, sixteen requests to a workgroup
      const int r0 = (blockIdx.x - cuts) * 16;
      for (int i = r0; i < min(r0 + 16, z.R); ++i) {
        if (tokens_of(a.seq_lens, i, z)) continue;
        for (int x = tid; x < z.Hq * (D / 8); x += NT)
          reinterpret_cast<u32x4*>(static_cast<__bf16*>(a.out) + (size_t)i * z.Hq * D)[x] = u32x4{0u, 0u, 0u, 0u};
        for (int x = tid; a.lse && x < z.Hq; x += NT) a.lse[(size_t)i * z.Hq + x] = -INFINITY;
      }
      return;
    }
    i0 = blockIdx.x / z.Gc;
    col = blockIdx.x - i0 * z.Gc;
    const Place at = place_of(a, z, scan[0], scan[1], [&](long long all) { return all * (i0 + 1) / z.W; });
    if (at.u >= at.U) return;
    U = at.U;
    r = at.r;
    const int cost = cost_of(tokens_of(a.seq_lens, r, z)), hh = (int)((at.u - at.base) / cost), h = hh / z.NG;
    P = at.base + (long long)hh * cost;
    hq = h * z.G + (hh - h * z.NG) * 16 + col;
    if (at.u <= P + kAhead || U * i0 / z.W > P + kAhead || hq >= (h + 1) * z.G) return;
    i1 = taker(P + cost - 1, U, z);
  } else {
    const int x = blockIdx.x / DS;
    d0 = blockIdx.x % DS * C;
    r = x / z.Hq;
    hq = x - r * z.Hq;
    const int h = hq / z.G, in = hq - h * z.G, hh = h * z.NG + in / 16;
    col = in % 16;
    const int n = tokens_of(a.seq_lens, r, z), cost = cost_of(n);
    if (n == 0) {
      if (tid < C / 4)
        *reinterpret_cast<u32x2*>(static_cast<__bf16*>(a.out) + ((size_t)r * z.Hq + hq) * D + d0 + 4 * tid) = u32x2{0u, 0u};
      if (tid == 0 && d0 == 0 && a.lse) a.lse[(size_t)r * z.Hq + hq] = -INFINITY;
      return;
    }
    int all = 0, pre = 0;
    for (int i = tid; i < z.R; i += NT) {
      const int c = cost_of(tokens_of(a.seq_lens, i, z));
      all += c;
      pre += i < r ? c : 0;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      all += __shfl_xor(all, d);
      pre += __shfl_xor(pre, d);
    }
    if (lane == 0) {
      scan[0][wave] = all;
      scan[1][wave] = pre;
    }
    __syncthreads();
    all = pre = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      all += scan[0][w];
      pre += scan[1][w];
    }
    U = (long long)all * heads;
    P = (long long)pre * heads + (long long)hh * cost;
    i0 = taker(P + kAhead, U, z);
    i1 = taker(P + cost - 1, U, z);
    if (i0 == i1) return;
  }
  __bf16* out = static_cast<__bf16*>(a.out) + ((size_t)r * z.Hq + hq) * D + d0;
  const bool writes_lse = tid == 0 && d0 == 0 && a.lse;
  auto at = [&](int i) {
    const bool head_of_share = U * i / z.W >= P;
    return 2 * (size_t)i + (head_of_share ? 0 : 1);
  };
  // maxima and sums of the shares first, as weights; then the outputs, their
  // loads independent of one another
  const int n_parts = i1 - i0 + 1;
  float M = kLowest;
  for (int i = tid; i < n_parts; i += NT) {
    const bool any = U * (i0 + i) / z.W < U * (i0 + i + 1) / z.W;  // a share may be without units
    const float2 x = any ? *reinterpret_cast<const float2*>(sums_at(a, z, D, at(i0 + i)) + 2 * col) : make_float2(kLowest, 0.f);
    weight[i] = x.x;
    part_l[i] = x.y;
    M = fmaxf(M, x.x);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) M = fmaxf(M, __shfl_xor(M, d));
  if (lane == 0) red[wave] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) M = fmaxf(M, red[w]);
  for (int i = tid; i < n_parts; i += NT) weight[i] = part_l[i] == 0.f ? 0.f : __builtin_amdgcn_exp2f(weight[i] - M);
  __syncthreads();
  const int part = tid / (C / 4), d = 4 * (tid % (C / 4));
  f32x4 o = pipe::zero4();
  float L = 0.f;
#pragma unroll 4
  for (int i = part; i < n_parts; i += NP) {
    const float e = weight[i];
    L += e * part_l[i];
    if (e != 0.f) o += *reinterpret_cast<const f32x4*>(outputs_at(a, z, D, at(i0 + i)) + col * D + d0 + d) * e;
  }
#pragma unroll
  for (int x = C / 4; x < 64; x <<= 1) {  // over the shares of a wave
    L += __shfl_xor(L, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], x);
  }
  if (lane < C / 4) *reinterpret_cast<f32x4*>(&sum[wave][d]) = o;
  if (lane == 0) ls[wave] = L;
  __syncthreads();
  if (tid < C / 4) {
    L = 0.f;
    o = pipe::zero4();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      L += ls[w];
      o += *reinterpret_cast<const f32x4*>(&sum[w][4 * tid]);
    }
    o *= L == 0.f ? 0.f : 1.f / L;
    *reinterpret_cast<u32x2*>(out + 4 * tid) = pipe::cvt4(o);
    if (writes_lse) a.lse[(size_t)r * z.Hq + hq] = L == 0.f ? -INFINITY : (M + (kDown + __builtin_amdgcn_logf(L))) * kLn2;
  }
}

DecodeSizes sizes(int R, int Hq, int Hkv, int D, int bt, int width, int num_blocks) {
  DecodeSizes z{};
  z.R = R;
  z.Hq = Hq;
  z.Hkv = Hkv;
  z.G = Hq / Hkv;
  z.NG = (z.G + 15) / 16;
  z.Gc = z.G < 16 ? z.G : 16;
  z.bt = bt;
  z.width = width;
  z.num_blocks = num_blocks;
  // no more shares than there can be units
  const long long units = width ? (((long long)width * bt + kUnit - 1) / kUnit + kAhead) * R * Hkv * z.NG : 0;
  const int most = most_shares(D);
  z.W = units < most ? (int)units : most;
  // one workgroup to a (request, key head), and no join, if none can be long.  Such a
  // call takes as long as the longest of them, the shares what all together and a join
  // take: where each has a CU of its own, the more there are, the longer they may be;
  // beyond that the last ones wait for a CU, and the length that may be grows again as
  // there are more to fill in.  Both ways, us on the GPU, x 16/4 heads, uniformly
  // ragged.  128: 8 of up to 1000 10.9 for 12.5, 32 of 2000 17.8 for 16.5, 56 of 4200 31.5
  // for 32.9, 63 of 5100 37.9 for 38.4, 64 of 4200 32.6 for 34.4, 65 of 4200 36.0 for
  // 36.0, 80 of 2000 27.1 for 28.7, of 4200 46.6 for 43.0, 128 of 4200 62 for 66, 256 of
  // 8000 209 for 220.  64: 8 of 1000 7.9 for 11.4, 48 of 2900 17.4 for 18.6, 64 of 4200
  // 22.5 for 23.3, of 5100 26.5 for 25.4, 65 of 2000 17.6 for 18.3, of 4200 28.8 for
  // 24.3, 128 of 5100 38 for 42, 256 of 8000 118 for 124.
  const long long groups = (long long)R * Hkv * z.NG, cap = ((long long)width * bt + kUnit - 1) / kUnit, cus = 256;
  z.whole = cap <= (groups <= cus ? std::max(8LL, groups / 7) : std::min(64LL, std::max(24LL, groups / 16)));
  // eight waves to each where that leaves none waiting for a CU, and for the long
  // ones: 64 ragged of up to 777 x 16/4 x 128 9.4 for 10.5 with four, 300 of up to
  // 777 36 for 26
  const long long at_once = D == 64 ? 512 : 256;  // of eight waves
  if (z.whole) z.whole = cap > 4 && (groups <= at_once || cap > 16) ? 8 : 4;
  return z;
}

template <int D, int FMT> hipError_t launch(const DecodeArgs& a, const DecodeSizes& z) {
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  if (z.whole) {
    const dim3 grid(z.R * z.Hkv * z.NG);
    if (z.whole == 8) return launch_kernel(attn_decode_kernel<D, FMT, 8, true>, grid, dim3(512), st, a, z);
    return launch_kernel(attn_decode_kernel<D, FMT, 4, true>, grid, dim3(256), st, a, z);
  }
  if (z.W) {
    const hipError_t e = launch_kernel(attn_decode_kernel<D, FMT, 4, false>, dim3(z.W), dim3(256), st, a, z);
    if (e != hipSuccess) return e;
  }
  // few rows: a row's columns over four workgroups, so that a long request's
  // many shares are read by more of them
  const int rows = z.R * z.Hq, cuts = z.W ? (z.W - 1) * z.Gc : 0;
  if (rows < 256) return launch_kernel(attn_decode_join_kernel<D, 4, false>, dim3(rows * 4), dim3(512), st, a, z);
  // by rows or by the ends of shares, whichever is fewer (700 requests of up to
  // 100 tokens x 16/4 x 128: 33.7 us for 43.9 by rows)
  if (rows <= cuts + (z.R + 15) / 16) return launch_kernel(attn_decode_join_kernel<D, 1, false>, dim3(rows), dim3(256), st, a, z);
  return launch_kernel(attn_decode_join_kernel<D, 1, true>, dim3(cuts + (z.R + 15) / 16), dim3(256), st, a, z);
}

}  // namespace

size_t attn_decode_workspace_bytes(int R, int Hq, int Hkv, int D, int bt, int width) {
  const DecodeSizes z = sizes(R, Hq, Hkv, D, bt, width, 0);
  if (z.whole) return 0;
  return ((size_t)2 * z.W * z.Gc * (D + 2) * sizeof(float) + 15) / 16 * 16;
}

hipError_t launch_attn_decode(const DecodeArgs& a) {
  const DecodeSizes z = sizes(a.R, a.Hq, a.Hkv, a.D, a.bt, a.width, a.num_blocks);
  if (a.fmt == GDN_CACHE_I8)
    return a.D == 64 ? launch<64, GDN_CACHE_I8>(a, z) : launch<128, GDN_CACHE_I8>(a, z);
  return a.D == 64 ? launch<64, GDN_CACHE_E4M3>(a, z) : launch<128, GDN_CACHE_E4M3>(a, z);
}

}  // namespace gdn
