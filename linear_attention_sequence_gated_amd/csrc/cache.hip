// cache.hip -- block tables from request lengths, and the write side of the
// 8-bit paged key / value cache.
#include <hip/hip_bf16.h>

#include "../../include/gdn.h"
#include "gdn_attn.hpp"
#include "gdn_launch.hpp"
#include "gdn_pipe.hpp"

namespace gdn {
namespace {

using pipe::hi_f;
using pipe::lo_f;
using pipe::u32x4;

// ------------------------------------------------------------- block tables
// Request r holds n_r tokens and gets m_r more.  It needs
//   need_r = ceil((n_r + m_r) / bt) - ceil(n_r / bt)
// blocks, taken from the free list at off_r = sum of need over the requests
// before it.  Two prefix sums (tokens and blocks) over the requests are all
// that the outputs depend on.  They are recomputed by every workgroup for the
// kRows requests it serves (R values from the L2, 16 bytes per lane and load)
// rather than handed over by a first launch: the sums cost about a
// microsecond, a launch more.  4096 requests take 8.8 us, 700 the same: bound by
// the chain of lengths, sums, table entry and slot, not by the 0.3 MB.  The last
// workgroup serves no request: it walks
// all of them for the totals and fills the slots behind the last token.
constexpr int kRows = 16, kThreads = 256;

struct Req {
  long long tokens, need;  // what it adds to the two prefix sums
  bool valid;
};

__device__ __forceinline__ Req request(int n, int m, const TablesArgs& a) {
  Req q;
  q.tokens = m > 0 ? m : 0;
  const int sh = __builtin_ctz(a.bt);
  const long long end = (long long)n + m, have = ((long long)n + a.bt - 1) >> sh, all = (end + a.bt - 1) >> sh;
  q.valid = n >= 0 && m >= 0 && all <= a.width && end <= 0x7fffffffLL;
  q.need = q.valid ? all - have : 0;
  return q;
}

__device__ __forceinline__ long long wave_sum64(long long x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// granted: its tokens lie inside the slot map and its blocks on the free list
__device__ __forceinline__ bool granted(const Req& q, long long cu, long long off, const TablesArgs& a) {
  return q.valid && cu + q.tokens <= a.T && (q.need == 0 || off + q.need <= a.n_free);
}

__global__ __launch_bounds__(kThreads) void block_tables_kernel(TablesArgs a) {
  __shared__ long long red[2][kThreads / 64];
  __shared__ int cus[kRows + 1], offs[kRows], held[kRows], have[kRows], ok[kRows];
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const int groups = (a.R + kRows - 1) / kRows;
  if ((int)blockIdx.x < groups) {
    const int r0 = blockIdx.x * kRows;
    long long st = 0, sb = 0;
    for (int i = 4 * t; i < r0; i += 4 * kThreads) {  // r0 is a multiple of 4
      const int4 n = *reinterpret_cast<const int4*>(a.seq_lens + i), m = *reinterpret_cast<const int4*>(a.new_lens + i);
      const Req q0 = request(n.x, m.x, a), q1 = request(n.y, m.y, a), q2 = request(n.z, m.z, a),
                q3 = request(n.w, m.w, a);
      st += (q0.tokens + q1.tokens) + (q2.tokens + q3.tokens);
      sb += (q0.need + q1.need) + (q2.need + q3.need);
    }
    st = wave_sum64(st);
    sb = wave_sum64(sb);
    if (lane == 0) {
      red[0][wave] = st;
      red[1][wave] = sb;
    }
    __syncthreads();
    if (wave == 0) {
      st = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
      sb = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
      const int r = r0 + lane;
      const bool here = lane < kRows && r < a.R;
      const int n = here ? a.seq_lens[r] : 0, m = here ? a.new_lens[r] : 0;
      const Req q = request(n, m, a);
      long long pt = q.tokens, pb = q.need;
#pragma unroll
      for (int d = 1; d < kRows; d <<= 1) {
        const long long x = __shfl_up(pt, d), y = __shfl_up(pb, d);
        if (lane >= d) {
          pt += x;
          pb += y;
        }
      }
      const long long cu = st + pt - q.tokens, off = sb + pb - q.need;
      const bool g = here && granted(q, cu, off, a);
      if (lane < kRows) {
        cus[lane] = cu < a.T ? (int)cu : a.T;
        offs[lane] = (int)off;  // used where granted: below n_free
        held[lane] = n;
        have[lane] = (int)(((long long)n + a.bt - 1) >> __builtin_ctz(a.bt));
        ok[lane] = g;
        if (lane == kRows - 1) cus[kRows] = st + pt < a.T ? (int)(st + pt) : a.T;
      }
      if (here) {
        a.cu_seqlens[r + 1] = (int)(st + pt < a.T ? st + pt : a.T);
        a.lens_after[r] = g ? n + m : n;
        if (r == 0) a.cu_seqlens[0] = 0;
      }
    }
    __syncthreads();
    // fresh entries of the table rows: one wave per request
    for (int i = wave; i < kRows && r0 + i < a.R; i += kThreads / 64) {
      if (!ok[i]) continue;
      const int m = cus[i + 1] - cus[i];
      const int all = (int)(((long long)held[i] + m + a.bt - 1) >> __builtin_ctz(a.bt));
      int* row = a.block_table + (size_t)(r0 + i) * a.width;
      for (int c = have[i] + lane; c < all; c += 64) row[c] = a.free_blocks[offs[i] + c - have[i]];
    }
    // slots of the tokens of these requests: a contiguous stretch of the map
    const int sh = __builtin_ctz(a.bt);
    const int end = cus[kRows];
    for (int base = cus[0]; base < end; base += 4 * kThreads) {
      int slot[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // four at a time, for their reads to overlap
        const int x = base + k * kThreads + t;
        int i = 0;
#pragma unroll
        for (int s = kRows / 2; s; s >>= 1)
          if (cus[i + s] <= x) i += s;
        slot[k] = -1;
        if (x < end && ok[i]) {
          const int pos = held[i] + (x - cus[i]), c = pos >> sh;
          const int id = c < have[i] ? a.block_table[(size_t)(r0 + i) * a.width + c] : a.free_blocks[offs[i] + c - have[i]];
          if (id >= 0 && id < a.num_blocks) slot[k] = (id << sh) + (pos & (a.bt - 1));
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (base + k * kThreads + t < end) a.slot_map[base + k * kThreads + t] = slot[k];
    }
    return;
  }
  // totals: rounds of kPer requests per thread, the running sums carried along
  constexpr int kPer = 16;
  long long ct = 0, cb = 0, used = 0, refused = 0;
  for (int base = 0; base < a.R; base += kThreads * kPer) {
    int n[kPer], m[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const int r = base + t * kPer + i;
      const bool four = r + 3 < a.R;
      const int4 x = four ? *reinterpret_cast<const int4*>(a.seq_lens + r) : make_int4(0, 0, 0, 0);
      const int4 y = four ? *reinterpret_cast<const int4*>(a.new_lens + r) : make_int4(0, 0, 0, 0);
      n[i] = x.x, n[i + 1] = x.y, n[i + 2] = x.z, n[i + 3] = x.w;
      m[i] = y.x, m[i + 1] = y.y, m[i + 2] = y.z, m[i + 3] = y.w;
      if (!four)
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (r + j < a.R) {
            n[i + j] = a.seq_lens[r + j];
            m[i + j] = a.new_lens[r + j];
          }
    }
    long long mt = 0, mb = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const Req q = request(n[i], m[i], a);
      mt += q.tokens;
      mb += q.need;
    }
    long long pt = mt, pb = mb;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const long long x = __shfl_up(pt, d), y = __shfl_up(pb, d);
      if (lane >= d) {
        pt += x;
        pb += y;
      }
    }
    if (lane == 63) {
      red[0][wave] = pt;
      red[1][wave] = pb;
    }
    __syncthreads();
    pt += ct - mt;
    pb += cb - mb;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) {
        pt += red[0][w];
        pb += red[1][w];
      }
      ct += red[0][w];
      cb += red[1][w];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const Req q = request(n[i], m[i], a);
      if (base + t * kPer + i < a.R) {
        if (!granted(q, pt, pb, a)) ++refused;
        else if (q.need) used = pb + q.need;
      }
      pt += q.tokens;
      pb += q.need;
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const long long u = __shfl_xor(used, d);
    used = u > used ? u : used;
    refused += __shfl_xor(refused, d);
  }
  if (lane == 0) {
    red[0][wave] = used;
    red[1][wave] = refused;
  }
  __syncthreads();
  if (t == 0) {
    long long u = 0, f = 0;
    for (int w = 0; w < kThreads / 64; ++w) {
      u = red[0][w] > u ? red[0][w] : u;
      f += red[1][w];
    }
    a.used[0] = (int)u;
    a.used[1] = (int)f;
    if (a.R == 0) a.cu_seqlens[0] = 0;
  }
  for (long long x = (ct < a.T ? ct : a.T) + t; x < a.T; x += kThreads) a.slot_map[x] = -1;
}

// -------------------------------------------------------------- cache append
// Codes of a block's rows for one head share one scale:
//   s = max(s_old, max |x| (1 / M)),  code = rne(x / s),  M = 127 or 448,
// s_old only where the block holds older rows, whose codes are then moved to
// the new scale, code = rne(code s_old / s).  The codes are the rounding of
// 32-bit products (by the reciprocal and by the ratio).
//
// One workgroup per run (the tokens of one call that fall into one block: as they
// follow one another with consecutive slots, a run ends where a slot is not one more
// than that before it, and no other run of the call has the same scale), head and
// tensor: a run's rows fit the registers of its four waves (NL 16-byte
// pieces per lane), so that they are read once and the largest magnitude takes
// one exchange through LDS.  Bound by HBM, 2 bytes read and 1 written per value:
// 9869 tokens x 16 heads of 128, 121 MB, take 22.5 us, 5.4 TB/s; 256 single tokens
// x 4 x 64 5.6 us, the chain of slot, scale and codes.  The rounding to 8 bits is
// the operator itself: half a step of a code, s / 2 (int8) or 2^-4 (e4m3), when a row
// is written, and again whenever its block's scale grows after that (k times: at most
// (k + 1) s / 2; a block filled token by token can grow bt - 1 times).
template <int FMT> constexpr float kMost = FMT == GDN_CACHE_I8 ? 127.f : 448.f;
constexpr float kLeastScale = 7.88860905e-31f;   // 2^-100: a block of zeros keeps a finite reciprocal
constexpr float kMostAbs = 3.38953139e38f;       // infinities count as the largest bf16 value

// Four values as four codes.  NaN becomes zero, infinities the largest code.
template <int FMT> __device__ __forceinline__ unsigned codes4(const float (&y)[4]) {
  float z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[i] = y[i] == y[i] ? y[i] : 0.f;
    z[i] = fminf(fmaxf(z[i], -kMost<FMT>), kMost<FMT>);
  }
  if constexpr (FMT == GDN_CACHE_I8) {
    unsigned b[4];  // adding 1.5 * 2^23 rounds to an integer (nearest even) in the low byte
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __builtin_bit_cast(unsigned, z[i] + 12582912.f) & 0xffu;
    return b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
  } else {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], w, true);
  }
}

template <int FMT> __device__ __forceinline__ void decode4(unsigned w, float (&y)[4]) {
  if constexpr (FMT == GDN_CACHE_I8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (float)(int)(signed char)(w >> (8 * i));
  } else {
    y[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
    y[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
    y[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
    y[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
  }
}

template <int FMT, int D, int NL>
__device__ __forceinline__ void append_run(const __hip_bfloat16* __restrict__ x, long long stride, char* tile,
                                           float* scale, int first, int n, float* red) {
  constexpr int LR = D / 8, RL = 256 / LR;  // lanes per row, rows per load of the workgroup
  const int t = threadIdx.x, row = t / LR, col = t % LR;
  u32x4 w[NL];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    w[i] = u32x4{0u, 0u, 0u, 0u};
    const int r = i * RL + row;
    if (r < n) w[i] = *reinterpret_cast<const u32x4*>(x + (long long)r * stride + 8 * col);
  }
  const float old = first ? *scale : 0.f;
#pragma unroll
  for (int i = 0; i < NL; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(lo_f(w[i][e])), fabsf(hi_f(w[i][e]))));
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  if ((t & 63) == 0) red[t >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float s = fmaxf(fmaxf(old, fminf(top, kMostAbs) * (1.f / kMost<FMT>)), kLeastScale);
  const float inv = 1.f / s;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int r = i * RL + row;
    if (r < n) {
      unsigned c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float y[4] = {lo_f(w[i][2 * h]) * inv, hi_f(w[i][2 * h]) * inv, lo_f(w[i][2 * h + 1]) * inv,
                            hi_f(w[i][2 * h + 1]) * inv};
        c[h] = codes4<FMT>(y);
      }
      *reinterpret_cast<uint2*>(tile + (first + r) * D + 8 * col) = make_uint2(c[0], c[1]);
    }
  }
  if (first && s != old) {
    const float ratio = old / s;
    for (int o = t * 16; o < first * D; o += 256 * 16) {
      u32x4 c = *reinterpret_cast<const u32x4*>(tile + o);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y[4];
        decode4<FMT>(c[e], y);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] *= ratio;
        c[e] = codes4<FMT>(y);
      }
      *reinterpret_cast<u32x4*>(tile + o) = c;
    }
  }
  if (t == 0) *scale = s;
}

// A workgroup looks at `window` consecutive slots (a power of two, at most 64)
// and writes the runs that begin there, for one head of one tensor.
template <int FMT, int D, int NL> __global__ __launch_bounds__(256) void cache_append_kernel(AppendArgs a, int window) {
  __shared__ float red[2][4];
  const int lane = threadIdx.x & 63;
  const int unit = blockIdx.x, which = unit & 1, h = (unit >> 1) % a.H;
  const long long t0 = (long long)((unit >> 1) / a.H) * window;
  const int sh = __builtin_ctz(a.bt), slots = a.num_blocks << sh;
  auto slot_at = [&](long long t) {
    const int s = t >= 0 && t < a.T ? a.slot_map[t] : -1;
    return s >= 0 && s < slots ? s : -1;
  };
  // slots t0 - 1 .. t0 + 126 or so: this lane's, the one before it, and 64 on
  const int mine = slot_at(t0 + lane), far = slot_at(t0 + 64 + lane);
  int before = __shfl_up(mine, 1);
  if (lane == 0) before = slot_at(t0 - 1);
  const bool begins = lane < window && mine >= 0 && (before != mine - 1 || (mine & (a.bt - 1)) == 0);
  unsigned long long todo = __ballot(begins);
  for (int k = 0; todo; k ^= 1) {
    const int i = __builtin_ctzll(todo);
    todo &= todo - 1;
    const int s = __builtin_amdgcn_readlane(mine, i), first = s & (a.bt - 1);
    // its length: the slots that follow one another, up to the block's end; 128
    // at most, of which the last may lie past the slots at hand
    const unsigned long long near_ = __ballot(lane >= i && mine == s + lane - i && first + lane - i < a.bt) >> i;
    const int in_near = 64 - i;
    int n = ~near_ ? __builtin_ctzll(~near_) : 64;
    if (n >= in_near) {
      n = in_near;
      const unsigned long long m = __ballot(far == s + in_near + lane && first + in_near + lane < a.bt);
      const int more = ~m ? __builtin_ctzll(~m) : 64;
      n += more;
      if (more == 64 && first + n < a.bt) {
        const unsigned long long l = __ballot(slot_at(t0 + 128 + lane) == s + n + lane && first + n + lane < a.bt);
        n += ~l ? __builtin_ctzll(~l) : 64;
      }
    }
    const long long tile = (long long)(s >> sh) * a.H + h;
    const __hip_bfloat16* x = static_cast<const __hip_bfloat16*>(which ? a.v : a.k);
    const long long stride = which ? a.vs : a.ks;
    append_run<FMT, D, NL>(x + (t0 + i) * stride + (long long)h * D, stride,
                           static_cast<char*>(which ? a.v_cache : a.k_cache) + tile * a.bt * D,
                           (which ? a.v_scale : a.k_scale) + tile, first, n, red[k]);
  }
}

template <int FMT, int D> hipError_t append_nl(const AppendArgs& a) {
  // A window of one slot spreads single tokens best; a wider one keeps the
  // workgroups that find nothing to begin from being the most of the work.
  int window = 1;
  while (window < 64 && (long long)(a.T + window - 1) / window * a.H * 2 > 8192) window *= 2;
  const dim3 grid((unsigned)((a.T + window - 1) / window * a.H * 2)), block(256);
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  switch (a.bt * D / 2048) {  // loads of 256 lanes x 8 values to a block
    case 0:
    case 1: return launch_kernel(cache_append_kernel<FMT, D, 1>, grid, block, st, a, window);
    case 2: return launch_kernel(cache_append_kernel<FMT, D, 2>, grid, block, st, a, window);
    case 4: return launch_kernel(cache_append_kernel<FMT, D, 4>, grid, block, st, a, window);
    default:
      if constexpr (D == 128) return launch_kernel(cache_append_kernel<FMT, D, 8>, grid, block, st, a, window);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_block_tables(const TablesArgs& a) {
  const int groups = (a.R + kRows - 1) / kRows;
  return launch_kernel(block_tables_kernel, dim3(groups + 1), dim3(kThreads), static_cast<hipStream_t>(a.stream), a);
}

hipError_t launch_cache_append(const AppendArgs& a) {
  if (a.fmt == GDN_CACHE_I8)
    return a.D == 64 ? append_nl<GDN_CACHE_I8, 64>(a) : append_nl<GDN_CACHE_I8, 128>(a);
  return a.D == 64 ? append_nl<GDN_CACHE_E4M3, 64>(a) : append_nl<GDN_CACHE_E4M3, 128>(a);
}

}  // namespace gdn
