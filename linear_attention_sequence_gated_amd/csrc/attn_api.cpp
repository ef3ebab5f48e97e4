// attn_api.cpp -- the C ABI of the attention layer (declared in include/gdn.h):
// validates every argument before anything is enqueued, then launches.
#include <stdint.h>

#include <cmath>
#include <initializer_list>

#include "../../include/gdn.h"
#include "gdn_attn.hpp"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int N> bool all_aligned(const void* const (&ptrs)[N]) {
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return false;
  return true;
}

int status(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

bool known_dtype(int d) { return d == GDN_F32 || d == GDN_BF16 || d == GDN_C64; }

bool block_ok(int bt) { return bt == 16 || bt == 32 || bt == 64 || bt == 128; }

// A scale that is a number: the forward's running maximum would take others for zero.
bool scale_ok(float s) { return std::isfinite(s); }

// A row stride: room for the row, 16-byte aligned rows, no offset past 2^62.
bool stride_ok(long long s, long long row) { return s >= row && s % 8 == 0 && s < (1LL << 40); }

constexpr int kMaxRequests = 1 << 20;
// Slots and tokens are counted in 32 bits by loops that step up to 2048 past the
// last one; their numbers stay below this.
constexpr long long kMostTokens = (1LL << 31) - 4096;

// Sizes of a cache and of the heads that read it.
int cache_shape(int Hkv, int D, int bt, int num_blocks) {
  if (Hkv <= 0 || D <= 0 || bt <= 0 || num_blocks < 0) return GDN_ERR_SHAPE;
  if ((long long)num_blocks * bt >= (1LL << 31) || Hkv >= (1 << 20)) return GDN_ERR_SHAPE;
  if ((D != 64 && D != 128) || !block_ok(bt)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// Heads: whole groups, and few enough for the launches.
int heads_shape(int Hq, int Hkv, int D) {
  if (Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv || Hq >= (1 << 20)) return GDN_ERR_SHAPE;
  return D == 64 || D == 128 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

// A row stride of which 128 rows, the most that a buffer resource covers, stay
// inside 32-bit byte offsets.
bool near_ok(long long s, long long row) { return stride_ok(s, row) && s < (1LL << 24); }

int prompt_shape(int T, int R, int Hq, int Hkv, int D) {
  if (T < 0 || R < 0 || R >= kMaxRequests) return GDN_ERR_SHAPE;
  if (const int s = heads_shape(Hq, Hkv, D)) return s;
  return (long long)T * Hq < (1LL << 28) ? GDN_OK : GDN_ERR_SHAPE;
}

int decode_shape(int R, int Hq, int Hkv, int D, int bt, int width) {
  if (R < 0 || width < 0 || bt <= 0 || R >= kMaxRequests || (long long)width * bt >= kMostTokens) return GDN_ERR_SHAPE;
  if (const int s = heads_shape(Hq, Hkv, D)) return s;
  if ((long long)R * Hq >= (1LL << 23)) return GDN_ERR_SHAPE;  // one workgroup of 512 joins one (request, head)
  // the units of 128 tokens over all requests, and one more for each, stay 32-bit numbers
  if ((((long long)width * bt + 127) / 128 + 1) * R >= (1LL << 31)) return GDN_ERR_SHAPE;
  return block_ok(bt) ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int gdn_block_tables(const int* seq_lens, const int* new_lens, int* block_table, const int* free_blocks,
                     int* slot_map, int* cu_seqlens, int* lens_after, int* used, int R, int width, int n_free,
                     int block_tokens, int num_blocks, int T, void* stream) {
  if (R < 0 || width < 0 || n_free < 0 || num_blocks < 0 || T < 0 || block_tokens <= 0) return GDN_ERR_SHAPE;
  if (R >= kMaxRequests || (long long)num_blocks * block_tokens >= (1LL << 31) || (long long)width * block_tokens >= (1LL << 31))
    return GDN_ERR_SHAPE;
  if (T >= kMostTokens) return GDN_ERR_SHAPE;
  if (!block_ok(block_tokens)) return GDN_ERR_UNSUPPORTED;
  if (!cu_seqlens || !used || (T && !slot_map) || (n_free && !free_blocks)) return GDN_ERR_NULL;
  if (R && (!seq_lens || !new_lens || !lens_after || (width && !block_table))) return GDN_ERR_NULL;
  const void* ptrs[] = {seq_lens, new_lens, block_table, free_blocks, slot_map, cu_seqlens, lens_after, used};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  return status(gdn::launch_block_tables({seq_lens, new_lens, block_table, free_blocks, slot_map, cu_seqlens,
                                          lens_after, used, R, width, n_free, block_tokens, num_blocks, T, stream}));
}

int gdn_cache_append(const void* k, const void* v, const int* slot_map, void* k_cache, void* v_cache, float* k_scale,
                     float* v_scale, long long k_stride, long long v_stride, int T, int Hkv, int D, int block_tokens,
                     int num_blocks, int dtype, int cache_format, void* stream) {
  if (!known_dtype(dtype)) return GDN_ERR_DTYPE;
  if (cache_format != GDN_CACHE_I8 && cache_format != GDN_CACHE_E4M3) return GDN_ERR_DTYPE;
  if (T < 0) return GDN_ERR_SHAPE;
  if (const int s = cache_shape(Hkv, D, block_tokens, num_blocks)) return s;
  if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  const long long row = (long long)Hkv * D;
  if ((long long)T * Hkv >= (1LL << 28) || !stride_ok(k_stride, row) || !stride_ok(v_stride, row)) return GDN_ERR_SHAPE;
  if (T == 0 || num_blocks == 0) return GDN_OK;
  if (!k || !v || !slot_map || !k_cache || !v_cache || !k_scale || !v_scale) return GDN_ERR_NULL;
  const void* ptrs[] = {k, v, slot_map, k_cache, v_cache, k_scale, v_scale};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  return status(gdn::launch_cache_append({k, v, slot_map, k_cache, v_cache, k_scale, v_scale, k_stride, v_stride, T,
                                          Hkv, D, block_tokens, num_blocks, cache_format, stream}));
}

size_t gdn_attn_decode_workspace_bytes(int R, int Hq, int Hkv, int D, int block_tokens, int width) {
  if (decode_shape(R, Hq, Hkv, D, block_tokens, width)) return 0;
  return gdn::attn_decode_workspace_bytes(R, Hq, Hkv, D, block_tokens, width);
}

int gdn_attn_decode(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                    const float* v_scale, const int* block_table, const int* seq_lens, void* out, float* lse,
                    float scale, long long q_stride, int R, int Hq, int Hkv, int D, int block_tokens, int num_blocks,
                    int width, int dtype, int cache_format, void* workspace, size_t workspace_bytes, void* stream) {
  if (!known_dtype(dtype)) return GDN_ERR_DTYPE;
  if (cache_format != GDN_CACHE_I8 && cache_format != GDN_CACHE_E4M3) return GDN_ERR_DTYPE;
  if (const int s = cache_shape(Hkv, D, block_tokens, num_blocks)) return s;
  if (const int s = decode_shape(R, Hq, Hkv, D, block_tokens, width)) return s;
  if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (!stride_ok(q_stride, (long long)Hq * D) || !scale_ok(scale)) return GDN_ERR_SHAPE;
  if (R == 0) return GDN_OK;
  if (!q || !seq_lens || !out || (width && !block_table)) return GDN_ERR_NULL;
  if (num_blocks && (!k_cache || !v_cache || !k_scale || !v_scale)) return GDN_ERR_NULL;
  const void* ptrs[] = {q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, lse, workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  const size_t need = gdn::attn_decode_workspace_bytes(R, Hq, Hkv, D, block_tokens, width);
  if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  return status(gdn::launch_attn_decode({q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, lse,
                                         static_cast<float*>(workspace), scale, q_stride, R, Hq, Hkv, D, block_tokens,
                                         num_blocks, width, cache_format, stream}));
}

int gdn_attn_prompt(const void* q, const void* k, const void* v, const int* cu_seqlens, void* out, float* lse,
                    float scale, long long q_stride, long long k_stride, long long v_stride, int T, int R, int Hq,
                    int Hkv, int D, int dtype, int zero_rest, void* stream) {
  if (!known_dtype(dtype)) return GDN_ERR_DTYPE;
  if (const int s = prompt_shape(T, R, Hq, Hkv, D)) return s;
  if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (!scale_ok(scale)) return GDN_ERR_SHAPE;
  const long long qrow = (long long)Hq * D, krow = (long long)Hkv * D;
  if (!near_ok(q_stride, qrow) || !near_ok(k_stride, krow) || !near_ok(v_stride, krow)) return GDN_ERR_SHAPE;
  if (T == 0) return GDN_OK;
  if (!q || !k || !v || !cu_seqlens || !out || !lse) return GDN_ERR_NULL;
  const void* ptrs[] = {q, k, v, cu_seqlens, out, lse};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  return status(gdn::launch_attn_prompt(
      {q, k, v, cu_seqlens, out, lse, scale, q_stride, k_stride, v_stride, T, R, Hq, Hkv, D,
       zero_rest, stream}));
}

size_t gdn_attn_prompt_bwd_workspace_bytes(int T, int Hq, int Hkv, int D) {
  return prompt_shape(T, 0, Hq, Hkv, D) ? 0 : gdn::attn_prompt_bwd_workspace_bytes(T, Hq, Hkv, D);
}

int gdn_attn_prompt_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse,
                        const void* grad_out, const int* cu_seqlens, void* grad_q, void* grad_k, void* grad_v,
                        float scale, long long q_stride, long long k_stride, long long v_stride,
                        long long grad_out_stride, long long grad_q_stride, long long grad_k_stride,
                        long long grad_v_stride, int T, int R, int Hq, int Hkv, int D, int dtype, int zero_rest,
                        void* workspace, size_t workspace_bytes, void* stream) {
  if (!known_dtype(dtype)) return GDN_ERR_DTYPE;
  if (const int s = prompt_shape(T, R, Hq, Hkv, D)) return s;
  if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (!scale_ok(scale)) return GDN_ERR_SHAPE;
  const long long qrow = (long long)Hq * D, krow = (long long)Hkv * D;
  for (const long long s : {q_stride, grad_out_stride, grad_q_stride})
    if (!near_ok(s, qrow)) return GDN_ERR_SHAPE;
  for (const long long s : {k_stride, v_stride, grad_k_stride, grad_v_stride})
    if (!near_ok(s, krow)) return GDN_ERR_SHAPE;
  if (T == 0) return GDN_OK;
  if (!q || !k || !v || !out || !lse || !grad_out || !cu_seqlens || !grad_q || !grad_k || !grad_v) return GDN_ERR_NULL;
  const void* ptrs[] = {q, k, v, out, lse, grad_out, cu_seqlens, grad_q, grad_k, grad_v, workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_ALIGN;
  if (!workspace || workspace_bytes < gdn::attn_prompt_bwd_workspace_bytes(T, Hq, Hkv, D)) return GDN_ERR_WORKSPACE;
  return status(gdn::launch_attn_prompt_bwd({q, k, v, out, lse, grad_out, cu_seqlens, grad_q, grad_k, grad_v,
                                             static_cast<float*>(workspace), scale, q_stride, k_stride, v_stride,
                                             grad_out_stride, grad_q_stride, grad_k_stride, grad_v_stride, T, R, Hq,
                                             Hkv, D, zero_rest, stream}));
}

}  // extern "C"
