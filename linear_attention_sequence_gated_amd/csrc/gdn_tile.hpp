// gdn_tile.hpp -- bf16 32x32x16 matrix-core tiles for the prompt attention
// kernels: rows staged in LDS by direct loads, operands read from there, and
// the rows' sequences.
//
// 32x32 accumulators: lane l holds column l % 32, element e (0..15) is row
// 8 (e / 4) + 4 (l / 32) + e % 4.  An operand of the product holds row (or
// column) l % 32 and eight values of k; the kernels take for k, of a 16-wide
// block, 4 h + j and 8 + 4 h + j (h = l / 32, j = 0..3), where an accumulator
// tile is fed back: its elements 8 b .. 8 b + 7 are then the operand of block b
// as they stand.
#pragma once

#include <hip/hip_bf16.h>

#include "gdn_pipe.hpp"

namespace gdn {
namespace tile {

using pipe::u32x2;
using pipe::u32x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ f32x16 mma(const u32x4& a, const u32x4& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// A lane's value (r[0] or r[1]) and that of lane ^ 32 (the other).  The second
// operand is hidden from the optimiser, which takes the swap of a value with
// itself for that value.
struct Halves {
  float a, b;
};
__device__ __forceinline__ Halves halves(float x) {
  int u = __builtin_bit_cast(int, x), w = u;
  asm("" : "+v"(w));
  const auto r = __builtin_amdgcn_permlane32_swap(u, w, false, false);
  return {__builtin_bit_cast(float, (int)r[0]), __builtin_bit_cast(float, (int)r[1])};
}
__device__ __forceinline__ float max_halves(float x) {
  const Halves h = halves(x);
  return fmaxf(h.a, h.b);
}
__device__ __forceinline__ float sum_halves(float x) {
  const Halves h = halves(x);
  return h.a + h.b;
}

// Elements 8 b .. 8 b + 7 of an accumulator tile as a bf16 operand.
__device__ __forceinline__ u32x4 operand(const f32x16& x, int b) {
  return u32x4{pipe::cvt2(x[8 * b], x[8 * b + 1]), pipe::cvt2(x[8 * b + 2], x[8 * b + 3]),
               pipe::cvt2(x[8 * b + 4], x[8 * b + 5]), pipe::cvt2(x[8 * b + 6], x[8 * b + 7])};
}

// ----------------------------------------------------------- non-finite values
// Non-finite bf16 values have all exponent bits set; the larger of a word's
// halves without their signs, over words.
__device__ __forceinline__ unsigned worst(unsigned m, unsigned w) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  const u16x2 a = __builtin_bit_cast(u16x2, m), b = __builtin_bit_cast(u16x2, w & 0x7fff7fffu);
  return __builtin_bit_cast(unsigned, __builtin_elementwise_max(a, b));
}
__device__ __forceinline__ bool finite(unsigned m) { return (m & 0xffffu) < 0x7f80u && (m >> 16) < 0x7f80u; }

// Words with their non-finite halves set to zero.
__device__ __forceinline__ u32x4 finite_only(u32x4 w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
    if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
  }
  return w;
}

// The score e of a half-tile (of 32 keys, element e) where bit 8 (e / 4) + e % 4
// of `seen` is set, otherwise -infinity (ZERO: zero).
template <bool ZERO> __device__ __forceinline__ float where_seen(float x, unsigned seen, int e) {
  const int bit = 8 * (e / 4) + e % 4, all = (int)(seen << (31 - bit)) >> 31;
  const int other = ZERO ? 0 : (int)0xff800000u;
  return __builtin_bit_cast(float, (all & __builtin_bit_cast(int, x)) | (~all & other));
}
// Bits lo .. hi of a word, those outside it left out.
__device__ __forceinline__ unsigned bits(int lo, int hi) {
  lo = lo < 0 ? 0 : lo;
  hi = hi > 31 ? 31 : hi;
  return lo > hi ? 0u : (0xffffffffu << lo) & (0xffffffffu >> (31 - hi));
}

// Rows [r0, r0 + n) of a [rows, heads, D] array whose rows are `stride`
// elements apart, seen through a buffer resource that ends with them: what lies
// behind reads as zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, long long stride, long long r0, int n, int D) {
  const uint32_t bytes = n > 0 ? (uint32_t)((n - 1) * stride + D) * 2u : 0u;
  return pipe::make_rsrc(static_cast<const __hip_bfloat16*>(base) + r0 * stride, bytes);
}

// 64 pieces of 16 bytes (of 4), straight to consecutive LDS, by one wave.  Not
// templates: the host's pass does not know the 16-byte form.
__device__ __forceinline__ void stage_pieces(__bf16* lds, __amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)lds, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void stage_words(float* lds, __amdgpu_buffer_rsrc_t rsrc) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)lds, 4, (threadIdx.x & 63) * 4, 0, 0, 0);
}

// N rows of D values staged in LDS in the swizzled layout of pipe::row_off, by
// loads that go straight to LDS: a wave's load fills 64 consecutive 16-byte
// pieces, so the swizzle is in which piece of the row each lane asks for.
template <int D, int N, int NW> struct Stage {
  static constexpr int NU = D / 8, LOADS = N * NU / 64 / NW;
  static_assert(N * NU % (64 * NW) == 0, "whole loads");
  uint32_t off[LOADS];  // byte offset of the lane's pieces from the first row
  __device__ __forceinline__ void init(long long stride, int wave) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int p = (wave * LOADS + i) * 64 + lane, r = p / NU, u = p % NU;
      const int piece = (pipe::row_off<D>(r, 8 * u) - r * D) / 8;
      off[i] = (uint32_t)(r * stride * 2) + piece * 16;
    }
  }
  __device__ __forceinline__ void load(__bf16* lds, __amdgpu_buffer_rsrc_t rsrc, int wave) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      stage_pieces(lds + (wave * LOADS + i) * 512, rsrc, off[i]);
  }
  // Sets the values that are not finite, of the part that this wave loaded, to
  // zero; false if there were any.  Its loads have arrived.
  static __device__ __forceinline__ bool scrub(__bf16* lds, int wave) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(lds + (wave * LOADS + i) * 512 + (threadIdx.x & 63) * 8);
      m = worst(worst(worst(worst(m, x[0]), x[1]), x[2]), x[3]);
    }
    if (__all(finite(m))) return true;
#pragma unroll 1
    for (int i = 0; i < LOADS; ++i) {
      u32x4* x = reinterpret_cast<u32x4*>(lds + (wave * LOADS + i) * 512 + (threadIdx.x & 63) * 8);
      *x = finite_only(*x);
    }
    return false;
  }
};

// Whether no wave found anything to scrub.
template <int NW> __device__ __forceinline__ bool all_clean(const int (&bad)[NW]) {
  int x = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) x |= bad[w];
  return __builtin_amdgcn_readfirstlane(x) == 0;
}

// x, which the compiler takes for a new value: what is computed from it is
// computed where it is used, not kept in registers over a loop.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Operand rows: row r0 + l % 32 of a staged tile, its values 16 ks + 8 h .. + 7.
template <int D> __device__ __forceinline__ int row_base(int lane) { return pipe::row_off<D>(lane & 31, 8 * (lane >> 5)) * 2; }
template <int D> __device__ __forceinline__ u32x4 row_frag(const __bf16* lds, int base, int r0, int ks) {
  return *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(lds) + ((base ^ (32 * ks)) + r0 * D * 2));
}

// Transposed operands: column 32 t + l % 32 of a staged tile, rows r0 + 4 h + j
// and r0 + 8 + 4 h + j (r0 a multiple of 16).
template <int D> __device__ __forceinline__ int col_base(int lane) {
  const int c = lane & 15;
  return pipe::row_off<D>(4 * (lane >> 5) + (c >> 2), 16 * ((lane >> 4) & 1) + 4 * (c & 3)) * 2;
}
template <int D> __device__ __forceinline__ u32x4 col_frag(const __bf16* lds, int base, int r0, int t) {
  const char* p = reinterpret_cast<const char*>(lds);
  const u32x2 a = pipe::ld4_tr(reinterpret_cast<const __bf16*>(p + ((base ^ (64 * t)) + r0 * D * 2)));
  const u32x2 b = pipe::ld4_tr(reinterpret_cast<const __bf16*>(p + ((base ^ (64 * t) ^ 32) + (r0 + 8) * D * 2)));
  return pipe::pair(a, b);
}

// Which columns of rows r0 .. r0 + N - 1 of an array hold values of a kind, and
// which of the rows before or behind those, taken together: a tile of rows (keys)
// sees either all of the keys before it (rows behind it) that are of its first
// (last) sequence, or none.  For what was left out of masked tiles: a workgroup
// reads the rows once, whatever they hold, and each lane then a word per row of the
// tile from LDS.  In LDS; look() and clear() by NT threads, with barriers between.
enum class Kind { not_finite, up, down };  // up, down: infinities of that sign, and NaN
template <int D, int N> struct Marks {
  unsigned row[N][D / 32], rest[D / 32];
  static __device__ __forceinline__ unsigned is(unsigned h, Kind kind) {  // of the lower half
    const unsigned size = h & 0x7fffu;
    if (kind == Kind::not_finite) return size >= 0x7f80u;
    return size > 0x7f80u || (h & 0xffffu) == (kind == Kind::up ? 0x7f80u : 0xff80u);
  }
  template <int NT> __device__ __forceinline__ void clear() {
    for (int i = threadIdx.x; i < (N + 1) * (D / 32); i += NT) (&row[0][0])[i] = 0u;
  }
  template <int NT, Kind KIND>
  __device__ __forceinline__ void look(const void* src, long long stride, int lo, int hi, int r0) {
    constexpr int NU = D / 8;  // pieces of eight to a row
    static_assert(NT % NU == 0, "");
    const int u = threadIdx.x % NU, shift = 8 * (u % 4);
    unsigned others = 0;
#pragma unroll 4
    for (int i = lo + (int)threadIdx.x / NU; i < hi; i += NT / NU) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const __hip_bfloat16*>(src) + (long long)i * stride + 8 * u);
      unsigned m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) m |= is(w[e], KIND) << (2 * e) | is(w[e] >> 16, KIND) << (2 * e + 1);
      if (i < r0 || i >= r0 + N) others |= m;
      else if (m) atomicOr(&row[i - r0][u / 4], m << shift);
    }
    if (others) atomicOr(&rest[u / 4], others << shift);
  }
  // Columns 32 w .. of rows lo .. hi - 1 (from r0), and of the others.
  __device__ __forceinline__ unsigned columns(int w, int lo, int hi, bool others) const {
    unsigned m = others ? rest[w] : 0u;
    for (int i = lo; i < hi; ++i) m |= row[i][w];
    return m;
  }
  __device__ __forceinline__ bool any(int lo, int hi, bool others) const {
    unsigned m = 0;
    for (int w = 0; w < D / 32; ++w) m |= columns(w, lo, hi, others);
    return m != 0;
  }
};

// Until this wave's loads into LDS have arrived.
__device__ __forceinline__ void wait_staged() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The same, then for the others' too.
__device__ __forceinline__ void staged_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Until all but the last N of this wave's loads have arrived.
template <int N> __device__ __forceinline__ void wait_all_but() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Until what this wave reads from LDS has arrived.
__device__ __forceinline__ void wait_read() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The keys that 32 rows (a lane's: l % 32) see, [first, last), and the last
// beginning of a sequence among them; last < 0 if none is in a sequence.
struct KeyRange {
  int first, latest, last;
};
__device__ __forceinline__ KeyRange key_range(int beg, int row, int T) {
  int first = beg < 0 ? T : beg, latest = first, last = beg < 0 ? -1 : row + 1;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    first = min(first, __shfl_xor(first, d));
    latest = max(latest, __shfl_xor(latest, d));
    last = max(last, __shfl_xor(last, d));
  }
  return {__builtin_amdgcn_readfirstlane(first), __builtin_amdgcn_readfirstlane(latest), __builtin_amdgcn_readfirstlane(last)};
}

// Sets rows [r0, r0 + n) of one head to zero, by NT threads.
template <int D> __device__ __forceinline__ void zero_rows(__bf16* dst, long long stride, int r0, int n, int NT) {
  for (int i = threadIdx.x; i < n * (D / 8); i += NT)
    *reinterpret_cast<u32x4*>(dst + (long long)(r0 + i / (D / 8)) * stride + i % (D / 8) * 8) = u32x4{0u, 0u, 0u, 0u};
}

// ------------------------------------------------------------------ sequences
// The largest s in [lo, hi] with at(s) <= row, given at(lo) <= row.
template <class At> __device__ __forceinline__ int last_at_most(At at, int lo, int hi, int row) {
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (at(mid) <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Of rows [r0, r0 + N), by NT threads: their sequence's first row in beg[] and
// the row behind its last in end[] (which may be NULL); rows of no sequence get
// beg = end = -1.  0 <= beg <= row < end <= T whatever cu holds.  Ends with a
// barrier.  Offsets are looked up in LDS, in `window` (kWindow entries): all of
// them where they fit, which costs one round trip to memory; otherwise those
// from r0's sequence on, which is found NT probes at a time first.
constexpr int kWindow = 512;
// meanwhile() issues other loads, behind the first of these.
template <int N, int NT, class F>
__device__ __forceinline__ void find_rows(const int* cu, int R, int T, int r0, int* window, int* beg, int* end,
                                          F meanwhile) {
  static_assert(2 * NT >= kWindow, "two loads per thread");
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
  const int one = t <= last ? cu[lo + t] : 0, two = t + NT <= last ? cu[lo + t + NT] : 0;
  meanwhile();
  if (t <= last) window[t] = one;
  if (t + NT <= last) window[t + NT] = two;
  __syncthreads();
  for (int i = t; i < N; i += NT) {
    const int row = r0 + i;
    int s = last_at_most([&](int x) { return window[x]; }, 0, last, row) + lo;
    if (s == lo + last && s < R) s = last_at_most([&](int x) { return cu[x]; }, s, R, row);
    int b = -1, e = -1;
    if (s < R && row < T) {
      b = s - lo <= last ? window[s - lo] : cu[s];
      e = min(s + 1 - lo <= last ? window[s + 1 - lo] : cu[s + 1], T);
      if (b > row || e <= row) b = e = -1;
      else b = max(b, 0);
    }
    beg[i] = b;
    if (end) end[i] = e;
  }
  __syncthreads();
}

// The rank-th longest of the tiles of N rows, by one of NT threads each: as long
// as the keys that its rows see (KEYS: the rows that see its keys), by its first
// (last) row.  Workgroups are started in the order of their numbers, and the
// last ones to end are short ones if they were started by length; with few
// tiles of sequences of many lengths that is worth more than the microsecond
// that the ranking costs every workgroup (13 sequences of up to 1201 rows x 16/4 x
// 128, forward: 73 us for 80; 8 of 2048 x 12/4 x 64: 75 for 84).  Needs tiles <= NT, R < kWindow;
// `window` (kWindow) and `keys` (NT entries) are scratch.  Ends with a barrier.
template <int N, int NT, bool KEYS>
__device__ __forceinline__ int tile_by_length(const int* cu, int R, int T, int tiles, int rank, int* window, int* keys) {
  const int t = threadIdx.x;
  const int one = t <= R ? cu[t] : 0, two = t + NT <= R ? cu[t + NT] : 0;
  if (t <= R) window[t] = one;
  if (t + NT <= R) window[t + NT] = two;
  __syncthreads();
  const int first = t * N, end = min(first + N, T), row = KEYS ? end - 1 : first;
  const int s = last_at_most([&](int x) { return window[x]; }, 0, R, row);
  int len = N;
  if (s < R) len = KEYS ? min(window[s + 1], T) - first : end - max(window[s], 0);
  // unique: longer first, then the later (KEYS: earlier) tile
  const int mine = t < tiles ? (min(max(len, 0), T) / 16) * NT + (KEYS ? NT - 1 - t : t) : -1;
  keys[t] = mine;
  __syncthreads();
  int above = 0;
  for (int i = 0; i < tiles; i += 4) {
    const int4 x = *reinterpret_cast<const int4*>(keys + i);
    above += (x.x > mine) + (x.y > mine) + (x.z > mine) + (x.w > mine);
  }
  __syncthreads();
  if (t < tiles && above == rank) window[0] = t;
  __syncthreads();
  const int found = window[0];
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(found);
}

}  // namespace tile
}  // namespace gdn
