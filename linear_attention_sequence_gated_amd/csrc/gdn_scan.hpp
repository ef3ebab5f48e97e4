// gdn_scan.hpp -- parts of the selective state space scan shared by its forward
// and its gradients: steps and decays of a piece of rows, how heads are dealt to
// workgroups, and the walk over the sequences of a segment of rows.
#pragma once

#include <climits>

#include "gdn_block.hpp"
#include "gdn_rows.hpp"

namespace gdn {
namespace scan {

using namespace rows;
using tile::f32x16;

constexpr int Q = 64;             // rows to a piece
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// log(1 + e^z), to a few units of float32's last place also where it is small: the
// series of log(1 + e) for e below 1/16, otherwise the logarithm of u = 1 + e with what
// the sum's rounding lost.  NaN is NaN, here and below.
__device__ __forceinline__ float softplus(float z) {
  const float e = exp2_(fminf(z, 20.f) * kLog2e), u = 1.f + e;
  const float large = __builtin_fmaf(__builtin_amdgcn_logf(u), 0.6931471805599453f, (e - (u - 1.f)) * __builtin_amdgcn_rcpf(u));
  float small = -1.f / 8;
#pragma unroll
  for (int n = 7; n; --n) small = __builtin_fmaf(small, e, n % 2 ? 1.f / n : -1.f / n);
  return !(z <= 20.f) ? z : e < 0.0625f ? small * e : large;
}

// What a row does to the state, as a power of two.  exp2_ gives zero below 2^-126, so that
// a smaller factor, of a row or of a piece, drops a state of any size: an error of up to
// 2^-126 of it.  Exponents below -160 are taken for that, which changes no factor; sums
// over a piece so stay below 2^14, and a difference of two, each of six additions, within
// 13 2^-24 of the piece's sum E: a weight behind strong decays is off by up to 9 E 2^-24 of
// itself.  E is 148 for 64 rows with a d = -1.6, and 10240 at most; results of 24 rows
// behind forty of 2^-160 are 1.65e-3 off in norm, which is their own rounding.
__device__ __forceinline__ float log2_keep(float a, float delta) {
  const float g = a * kLog2e * delta;
  return g < -160.f ? -160.f : g;
}

// Columns of x are taken 64 at a time ("strips"): a head of P = 64 or half of one of
// 128, whose recurrence runs by itself.  Workgroups take NS neighbouring strips of
// one group of heads; a group's last workgroup may have fewer.
struct Strips {
  int per_group;  // strips to a group
  int sets;       // workgroups to a group
};
__host__ __device__ inline Strips strips(int H, int P, int G, int NS) {
  const int per = H / G * (P / 64);
  return {per, (per + NS - 1) / NS};
}

// A workgroup's number among `all`, such that consecutive ones share an XCD and its L2,
// and with it the rows that they all read: the hardware deals workgroups to the eight
// XCDs in turn (8 x 2048 rows x 24 heads of 64: 72 us for the scan, so 69).
__device__ __forceinline__ int neighbours(int id, int all) {
  const int xcd = id & 7;
  return xcd * (all >> 3) + min(xcd, all & 7) + (id >> 3);
}

// Sequences without rows, whose states a call passes through: a padded batch has many of
// them, and few rows with them.  They are dealt to `idle` segments without rows, which
// take the CUs that are left, or, where those are fewer, to all segments.  One sequence
// of 131 rows and 255 without, 24 heads of 64, N = 128: 77 us and 102 for the gradients,
// dealt to the segments with rows alone 971 and 599; the states' copy 74.
struct Idle {
  int first, step;  // of a segment's sequences
};
__device__ __forceinline__ Idle idle_of(int seg, int nseg, int idle) {
  if (idle < nseg) return {seg, nseg + idle};
  return {seg < nseg ? INT_MAX : seg - nseg, idle};
}
inline int idle_segments(int R, int room) { return R < 2 || room < 1 ? 0 : room < R ? room : R; }

// ------------------------------------------------------------------- staging
// Rows of D values to LDS as tile::Stage puts them, one load (of LOADS) at a time.  As
// assembly: a load to LDS that the compiler knows of makes it wait for all such loads
// before whatever it reads from LDS next, of another buffer too, so that no load would
// run beside the products.
struct Source {
  u32x4 rsrc;
};
__device__ __forceinline__ Source source(const void* base, long long stride, long long r0, int n, int D) {
  const unsigned long long at = reinterpret_cast<unsigned long long>(static_cast<const __bf16*>(base) + r0 * stride);
  const unsigned bytes = n > 0 ? (unsigned)((n - 1) * stride + D) * 2u : 0u;
  return {u32x4{(unsigned)__builtin_amdgcn_readfirstlane((int)at), (unsigned)__builtin_amdgcn_readfirstlane((int)(at >> 32)) & 0xffffu,
                (unsigned)__builtin_amdgcn_readfirstlane((int)bytes), (unsigned)pipe::kRsrcWord3}};
}
// 64 pieces of 16 bytes, `ahead` bytes behind src, to consecutive LDS.  The load has no
// result in a register, and takes its addresses as it is issued; that it has arrived is
// waited for by a barrier of its wave (tile::staged_barrier, loads_barrier) and nothing
// reads its part of LDS before.  M0, the address in LDS, is used by nothing else in these
// kernels.  Five waits between a vector instruction that may have written a
// scalar operand and the load are the assembly's own to keep, and one behind M0.  The
// resource's end counts both offsets, `ahead` also where it alone is past the end: rows
// behind a piece read as zero.
__device__ __forceinline__ void load_piece(__bf16* lds, const Source& src, unsigned off, int ahead) {
  const unsigned at = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)(unsigned long long)(tile::lds_void*)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(at), "v"(off), "s"(src.rsrc), "s"(ahead)
               : "memory");
}
template <int D, int N, int NW> struct Stage : tile::Stage<D, N, NW> {
  typedef tile::Stage<D, N, NW> Base;
  __device__ __forceinline__ void load_one(__bf16* lds, const Source& src, int wave, int i) const {
    load_piece(lds + (wave * Base::LOADS + i) * 512, src, Base::off[i], 0);
  }
  __device__ __forceinline__ void load(__bf16* lds, const Source& src, int wave) const {
#pragma unroll
    for (int i = 0; i < Base::LOADS; ++i) load_one(lds, src, wave, i);
  }
};

// The same for one wave that loads R rows by itself: the swizzle repeats after 16
// rows, so that as many offsets as loads of 16 rows serve them all.
template <int D> struct StageWave {
  static constexpr int kRows = 512 / D, kOff = 16 / kRows;  // rows to a load; offsets
  unsigned off[kOff];
  int step;  // bytes between rows 16 apart
  __device__ __forceinline__ void init(long long stride) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kOff; ++i) {
      const int r = kRows * i + lane / (D / 8);
      off[i] = (unsigned)(r * stride * 2) + (pipe::row_off<D>(r, 8 * (lane % (D / 8))) - r * D) * 2;
    }
    step = (int)(stride * 32);
  }
  template <int R> __device__ __forceinline__ void load(__bf16* lds, const Source& src, int ahead) const {
#pragma unroll
    for (int i = 0; i < R / kRows; ++i) load_piece(lds + i * 512, src, off[i % kOff], ahead + i / kOff * step);
  }
};

// A barrier behind which all but this wave's last KEEP loads have arrived.
template <int KEEP> __device__ __forceinline__ void loads_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(KEEP) : "memory");
}

// x, which has arrived when this is reached.  What a load brought has to be asked for
// before the next loads to LDS are issued: the compiler, which does not know of those,
// would wait for them too.
template <class T> __device__ __forceinline__ T arrived(T x) {
  static_assert(sizeof(T) == 4, "");
  asm volatile("" : "+v"(x));
  return x;
}

// ----------------------------------------------------------------- sequences
// cu[i], in LDS where all of them fit.
struct Offsets {
  const int* cu;
  const int* window;  // NULL: not there
  __device__ __forceinline__ int operator()(int i) const {
    return __builtin_amdgcn_readfirstlane(window ? window[i] : cu[i]);
  }
  // How many of the first n offsets are below row.
  __device__ __forceinline__ int below(int n, int row) const {
    int lo = 0;
    while (lo < n) {
      const int mid = lo + (n - lo) / 2;
      if ((*this)(mid) < row) lo = mid + 1;
      else n = mid;
    }
    return lo;
  }
};

// Offsets ready for use by NT threads; ends with a barrier.
template <int NT> __device__ __forceinline__ Offsets offsets(const int* cu, int R, int* window) {
  if (R >= kWindow) return {cu, nullptr};
  for (int i = threadIdx.x; i <= R; i += NT) window[i] = cu[i];
  __syncthreads();
  return {cu, window};
}

// A run of rows of one sequence, at most Q.
struct Piece {
  int row, n, seq;
  bool first, last;  // of its sequence
};

// Whose pieces end at multiples of Q as well: a piece of sequence r with rows of the
// c-th Q then has a number of its own, c + r.
__device__ __forceinline__ int piece_id(const Piece& p) { return p.row / Q + p.seq; }

// The pieces of rows [s0, s1), in order: of the sequence that goes on into them,
// if any, then of those that begin in them.  The rows that it gives ascend, and
// every call ends, whatever cu holds.
template <bool ALIGNED> struct Walk {
  Offsets cu;
  int T, s1, r, rend, beg, pos, end;
  __device__ __forceinline__ void init(const Offsets& c, int R, int T_, int s0, int s1_) {
    cu = c, T = T_, s1 = s1_;
    const int k = cu.below(R, s0);
    rend = cu.below(R, s1);
    r = k - 1;
    beg = pos = end = s0;
    if (k > 0) {
      beg = min(max(cu(k - 1), 0), s0);
      end = min(max(cu(k), s0), T);
    }
  }
  // Whether rows before s0 belong to the first piece's sequence.
  __device__ __forceinline__ bool goes_on() const { return pos < min(end, s1); }
  __device__ __forceinline__ bool next(Piece& p) {
    for (;;) {
      const int e = min(end, s1);
      if (pos < e) {
        p.row = pos, p.n = min(ALIGNED ? Q - pos % Q : Q, e - pos), p.seq = r;
        p.first = pos == beg;
        pos += p.n;
        p.last = pos == end;
        return true;
      }
      if (++r >= rend) return false;
      beg = pos = min(max(cu(r), pos), T);
      end = min(max(cu(r + 1), beg), T);
    }
  }
};

// The same pieces from the last to the first, cut at multiples of Q.
struct WalkBack {
  Offsets cu;
  int T, s0, r, rlow, beg, pos, end;
  __device__ __forceinline__ void take(int top) {  // sequence r, rows below `top`
    beg = min(max(cu(r), 0), top);
    end = min(max(cu(r + 1), beg), T);
    pos = min(end, top);
  }
  __device__ __forceinline__ void init(const Offsets& c, int R, int T_, int s0_, int s1) {
    cu = c, T = T_, s0 = s0_;
    rlow = max(cu.below(R, s0) - 1, 0);
    r = cu.below(R, s1) - 1;
    beg = pos = end = s0;
    if (r >= rlow) take(s1);
  }
  __device__ __forceinline__ bool next(Piece& p) {
    for (;;) {
      const int b = max(beg, s0);
      if (pos > b) {
        const int row = max(b, (pos - 1) / Q * Q);
        p.row = row, p.n = pos - row, p.seq = r;
        p.first = row == beg, p.last = pos == end;
        pos = row;
        return true;
      }
      if (--r < rlow) return false;
      take(pos);
    }
  }
};

// ------------------------------------------------------------ steps of a piece
// Of the piece's rows (a lane each), for one head: in LDS, by one wave.
struct alignas(16) Steps {
  float G[Q];  // sums of the log2 decays up to and including the row
  float u[Q];  // log2(delta) - G
  float v[32];  // delta 2^(G_31 - G) of the first 32
  float w[Q];  // delta 2^(sum of the decays behind the row)
  float total;  // sum of the log2 decays
};

__device__ __forceinline__ float dt_at(const void* dt, bool f32, long long i) { return param(dt, f32, i); }
// The same in two parts, so that nothing waits for the load: its bits, and their number.
__device__ __forceinline__ unsigned dt_bits(const void* dt, bool f32, long long i) {
  return f32 ? static_cast<const unsigned*>(dt)[i] : static_cast<const unsigned short*>(dt)[i];
}
__device__ __forceinline__ float dt_of(unsigned bits, bool f32) { return number(f32 ? bits : bits << 16); }

// Returns the sum over the piece.  No barrier: the wave reads what it wrote.
__device__ __forceinline__ float steps(Steps& s, float z, float a, bool in) {
  const int lane = threadIdx.x & 63;
  const float delta = in ? softplus(z) : 0.f;
  const float g = in ? log2_keep(a, delta) : 0.f;
  const float G = pipe::wave_prefix_sum(g);
  // the sums behind each row, from the last row back: no difference of large numbers
  const float back = pipe::wave_prefix_sum(__shfl(g, 63 - lane));
  const float after = __shfl(back, (62 - lane) & 63);
  const float G31 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, G), 31));
  s.G[lane] = G;
  s.u[lane] = __builtin_amdgcn_logf(delta) - G;
  if (lane < 32) s.v[lane] = delta * exp2_(G31 - G);
  s.w[lane] = delta * exp2_(lane == 63 ? 0.f : after);
  const float total = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, G), 63));
  if (lane == 0) s.total = total;
  pipe::issue_fence();  // read as vectors from here on
  return total;
}

// ------------------------------------------------------------------- products
// The state of a strip's 32 columns, [N][32]: tile t holds rows 32 t ..; a tile's row
// i stands for n = i with bits 2 and 3 exchanged, so that elements 8 b .. 8 b + 7 of
// a lane are the eight n from 16 b + 8 (l / 32) on: an operand of the products with
// rows of C (and B) read eight values at a time.
__device__ __forceinline__ int state_row(int e, int half) { return 16 * (e / 8) + 8 * half + e % 8; }

// Transposed operand whose row l % 32 of the tile is that n.
template <int D> __device__ __forceinline__ int col_base_state(int lane) {
  const int c = lane & 15, m = c & 3;
  return pipe::row_off<D>(4 * (lane >> 5) + (c >> 2), 16 * ((lane >> 4) & 1) + 8 * (m & 1) + 4 * (m >> 1)) * 2;
}

// Transposed operands with eight consecutive k to a lane: column 32 t + l % 32 of a
// staged tile, rows r0 + 8 (l / 32) on (r0 a multiple of 16).
template <int D> __device__ __forceinline__ int col_base8(int lane) {
  const int c = lane & 15;
  return pipe::row_off<D>(8 * (lane >> 5) + (c >> 2), 16 * ((lane >> 4) & 1) + 4 * (c & 3)) * 2;
}
template <int D> __device__ __forceinline__ u32x4 col_frag8(const __bf16* lds, int base, int r0, int t) {
  const char* p = reinterpret_cast<const char*>(lds);
  const u32x2 a = pipe::ld4_tr(reinterpret_cast<const __bf16*>(p + ((base ^ (64 * t)) + r0 * D * 2)));
  const u32x2 b = pipe::ld4_tr(reinterpret_cast<const __bf16*>(p + ((base ^ (64 * t) ^ 16) + (r0 + 4) * D * 2)));
  return pipe::pair(a, b);
}

// Eight bf16 values (of rows k) times eight numbers w, as PARTS bf16 operands that
// add up to the products: to 2^-8, 2^-17 and 2^-25 of them.
template <int PARTS> struct Split {
  u32x4 part[PARTS];
  __device__ __forceinline__ void make(const u32x4& x, const float* w0, const float* w1) {
    const float4 a = *reinterpret_cast<const float4*>(w0), b = *reinterpret_cast<const float4*>(w1);
    float f[8] = {pipe::lo_f(x[0]) * a.x, pipe::hi_f(x[0]) * a.y, pipe::lo_f(x[1]) * a.z, pipe::hi_f(x[1]) * a.w,
                  pipe::lo_f(x[2]) * b.x, pipe::hi_f(x[2]) * b.y, pipe::lo_f(x[3]) * b.z, pipe::hi_f(x[3]) * b.w};
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned c = pipe::cvt2(f[2 * i], f[2 * i + 1]);
        part[p][i] = c;
        f[2 * i] -= pipe::lo_f(c);
        f[2 * i + 1] -= pipe::hi_f(c);
      }
    }
  }
};

// Elements 8 b .. 8 b + 7 of an accumulator tile as two bf16 operands that add up to them,
// to 2^-17.
struct Two {
  u32x4 part[2];
};
__device__ __forceinline__ Two two_parts(const f32x16& x, int b) {
  Two t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = x[8 * b + 2 * i], g = x[8 * b + 2 * i + 1];
    t.part[0][i] = pipe::cvt2(f, g);
    t.part[1][i] = pipe::cvt2(f - pipe::lo_f(t.part[0][i]), g - pipe::hi_f(t.part[0][i]));
  }
  return t;
}

// States in memory, [N][P] float32: the part of a wave's 32 columns.  Addresses are
// computed here, not kept in registers over a loop.
template <int NT> __device__ __forceinline__ void load_state(f32x16 (&S)[NT], const float* src, int P) {
  const int lane = tile::fresh(threadIdx.x & 63), step = tile::fresh(P);
  const float* at = src + (lane >> 5) * 8 * step + (lane & 31);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < 2; ++b, at += 16 * step)
#pragma unroll
      for (int j = 0; j < 8; ++j) S[t][8 * b + j] = at[j * step];
}
template <int NT> __device__ __forceinline__ void store_state(const f32x16 (&S)[NT], float* dst, int P) {
  const int lane = tile::fresh(threadIdx.x & 63), step = tile::fresh(P);
  float* at = dst + (lane >> 5) * 8 * step + (lane & 31);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < 2; ++b, at += 16 * step)
#pragma unroll
      for (int j = 0; j < 8; ++j) at[j * step] = S[t][8 * b + j];
}

// Adds up states of segments along the sequences, [slots][strips][N][64] and behind
// them [slots][strips] of what each segment keeps of the state before it (log2):
// kNone where no sequence crosses the slot's border, kFresh where the one that does
// began (ended) in the segment.  Slot s becomes the state at the border; `back` from
// the last to the first.
constexpr float kNone = 3e38f, kFresh = 2e38f;
template <int N> __device__ __forceinline__ void join(float* ws, int nstrips, int slots, int strip, int i, bool back) {
  const ptrdiff_t step = (ptrdiff_t)nstrips * N * 64;
  const float* kept = ws + slots * step + strip + (back ? (ptrdiff_t)(slots - 1) * nstrips : 0);
  float* at = ws + (ptrdiff_t)strip * N * 64 + i + (back ? (slots - 1) * step : 0);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int U = 8;  // slots whose loads are issued together
  for (int s0 = 0; s0 < slots; s0 += U) {
    float k[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = kNone;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + u < slots) {
        k[u] = kept[u * (back ? -nstrips : nstrips)];
        v[u] = *reinterpret_cast<const float4*>(at + u * (back ? -step : step));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k[u] == kNone) continue;  // what the slot holds is not to be used
      if (k[u] != kFresh) {
        const float f = exp2_(k[u]);
        v[u].x = __builtin_fmaf(f, S.x, v[u].x), v[u].y = __builtin_fmaf(f, S.y, v[u].y);
        v[u].z = __builtin_fmaf(f, S.z, v[u].z), v[u].w = __builtin_fmaf(f, S.w, v[u].w);
        *reinterpret_cast<float4*>(at + u * (back ? -step : step)) = v[u];
      }
      S = v[u];
    }
    at += (back ? -U : U) * step, kept += (back ? -U : U) * nstrips;
  }
}

}  // namespace scan
}  // namespace gdn
