// gdn_rows.hpp -- rows in 16-byte pieces (eight bf16 or four fp32 values), sums
// over lanes, and the sequences that packed rows belong to; for the norm, the
// short convolution and the state space scan.
#pragma once

#include "gdn_tile.hpp"

namespace gdn {
namespace rows {

using pipe::u32x2;
using pipe::u32x4;

// Values of a 16-byte piece.
template <bool F32> constexpr int kPiece = F32 ? 4 : 8;

// A word as a float32 number.  By value: __builtin_bit_cast of a vector's element
// takes the vector's first.
__device__ __forceinline__ float number(unsigned u) { return __builtin_bit_cast(float, u); }

// A piece as float32 numbers.
template <bool F32> __device__ __forceinline__ void unpack(const u32x4& w, float (&f)[kPiece<F32>]) {
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = number(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = pipe::lo_f(w[i]), f[2 * i + 1] = pipe::hi_f(w[i]);
  }
}

// float32 numbers as a piece, rounded to nearest even where it holds bf16.
template <bool F32> __device__ __forceinline__ u32x4 pack(const float (&f)[kPiece<F32>]) {
  u32x4 w;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(unsigned, f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pipe::cvt2(f[2 * i], f[2 * i + 1]);
  }
  return w;
}

// Piece p of a row whose first value has index `at` (p counts kPiece<F32>).
template <bool F32> __device__ __forceinline__ u32x4 piece(const void* base, long long at, int p) {
  return *reinterpret_cast<const u32x4*>(static_cast<const char*>(base) + at * (F32 ? 4 : 2) + (long long)p * 16);
}
template <bool F32> __device__ __forceinline__ void put(void* base, long long at, int p, const u32x4& w) {
  *reinterpret_cast<u32x4*>(static_cast<char*>(base) + at * (F32 ? 4 : 2) + (long long)p * 16) = w;
}

// Pieces of E values, 8 or 16 bytes.
template <bool F32, int E> struct PieceOf {
  static_assert(E == (F32 ? 4 : 8) || (!F32 && E == 4), "");
  typedef std::conditional_t<!F32 && E == 4, u32x2, u32x4> Word;
  static __device__ __forceinline__ Word zero() {
    Word w;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Word) / 4); ++i) w[i] = 0;
    return w;
  }
  static __device__ __forceinline__ Word get(const void* base, long long at, int p) {
    return *reinterpret_cast<const Word*>(static_cast<const char*>(base) + (at + (long long)p * E) * (F32 ? 4 : 2));
  }
  static __device__ __forceinline__ void put(void* base, long long at, int p, const Word& w) {
    *reinterpret_cast<Word*>(static_cast<char*>(base) + (at + (long long)p * E) * (F32 ? 4 : 2)) = w;
  }
  static __device__ __forceinline__ void unpack(const Word& w, float (&f)[E]) {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = number(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) f[2 * i] = pipe::lo_f(w[i]), f[2 * i + 1] = pipe::hi_f(w[i]);
    }
  }
  static __device__ __forceinline__ Word pack(const float (&f)[E]) {
    Word w;
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(unsigned, f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) w[i] = pipe::cvt2(f[2 * i], f[2 * i + 1]);
    }
    return w;
  }
};

// N consecutive parameters from index `at`, bf16 or float32; N a multiple of 4
// and `at` one of N, so that they are whole words of 8 or 16 bytes.
template <int N> __device__ __forceinline__ void params(const void* base, bool f32, long long at, float (&f)[N]) {
  static_assert(N % 4 == 0, "");
  if (f32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 w = p[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[4 * i + e] = number(w[e]);
    }
  } else {
    const u32x2* p = reinterpret_cast<const u32x2*>(static_cast<const unsigned short*>(base) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x2 w = p[i];
      f[4 * i] = pipe::lo_f(w[0]), f[4 * i + 1] = pipe::hi_f(w[0]);
      f[4 * i + 2] = pipe::lo_f(w[1]), f[4 * i + 3] = pipe::hi_f(w[1]);
    }
  }
}

// One parameter, and one written.
__device__ __forceinline__ float param(const void* base, bool f32, long long i) {
  return f32 ? static_cast<const float*>(base)[i] : (float)static_cast<const __bf16*>(base)[i];
}
__device__ __forceinline__ void put_param(void* base, bool f32, long long i, float x) {
  if (f32) static_cast<float*>(base)[i] = x;
  else static_cast<__bf16*>(base)[i] = (__bf16)x;
}

// x times the logistic function of x, and its derivative; e^-x by the hardware's
// 2^x, off by some 2^-22 of the result where it counts.
__device__ __forceinline__ float logistic(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }
__device__ __forceinline__ float silu(float x) { return x * logistic(x); }
__device__ __forceinline__ float silu_slope(float x) {
  const float s = logistic(x);
  return s * (1.f + x * (1.f - s));
}

// Sum over a wave.
__device__ __forceinline__ float wave_sum(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, pipe::wave_prefix_sum(x)), 63));
}

// The largest of non-negative numbers over N consecutive lanes (aligned), NaN
// above all: their bits, compared as whole numbers.
template <int N> __device__ __forceinline__ unsigned lanes_max(unsigned u) {
#pragma unroll
  for (int d = 1; d < N; d *= 2) u = max(u, (unsigned)__shfl_xor((int)u, d));
  return u;
}

// The sequence of each of rows [r0, r0 + N), by NT threads: its number in
// seq[], first row in beg[] and the row behind its last in end[]; rows of no
// sequence get -1 in all.  0 <= beg <= row < end <= T whatever cu holds.  Ends
// with a barrier.  Offsets are looked up in LDS (`window`, kWindow entries): all
// of them where they fit, otherwise those from r0's sequence on, which is found
// NT probes at a time first.
constexpr int kWindow = 512;
template <int N, int NT>
__device__ __forceinline__ void find_seqs(const int* cu, int R, int T, int r0, int* window, int* seq, int* beg, int* end) {
  const int t = threadIdx.x;
  int lo = 0;
  if (R >= kWindow) {
    for (int n = R + 1;;) {
      const int step = (n + NT - 1) / NT, i = t * step;
      const int cnt = __syncthreads_count(i < n && cu[lo + i] <= r0);
      if (cnt > 1) lo += (cnt - 1) * step;
      if (cnt == 0 || step == 1) break;
      n = min(step, R + 1 - lo);
    }
  }
  // cu[lo] is the last offset at or before r0, or lo = 0
  const int last = min(R - lo, kWindow - 1);
  for (int i = t; i <= last; i += NT) window[i] = cu[lo + i];
  __syncthreads();
  for (int i = t; i < N; i += NT) {
    const int row = r0 + i;
    int s = tile::last_at_most([&](int x) { return window[x]; }, 0, last, row) + lo;
    if (s == lo + last && s < R) s = tile::last_at_most([&](int x) { return cu[x]; }, s, R, row);
    int b = -1, e = -1;
    if (s < R && row < T) {
      b = s - lo <= last ? window[s - lo] : cu[s];
      e = min(s + 1 - lo <= last ? window[s + 1 - lo] : cu[s + 1], T);
      if (b > row || e <= row) b = e = -1;
      else b = max(b, 0);
    }
    seq[i] = b < 0 ? -1 : s;
    beg[i] = b;
    end[i] = e;
  }
  __syncthreads();
}

// Rows of sequence s, whatever cu holds.
struct Span {
  int beg, end;
};
__device__ __forceinline__ Span span_of(const int* cu, int T, int s) {
  const int b = min(max(cu[s], 0), T);
  return {b, min(max(cu[s + 1], b), T)};
}

}  // namespace rows
}  // namespace gdn
