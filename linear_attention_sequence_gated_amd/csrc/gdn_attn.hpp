// gdn_attn.hpp -- internal interface of the attention layer's kernels: block
// tables, the 8-bit paged cache, its single-token read, prompt attention and
// its gradients.  Arguments arrive validated (attn_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

struct TablesArgs {
  const int* seq_lens;
  const int* new_lens;
  int* block_table;
  const int* free_blocks;
  int* slot_map;
  int* cu_seqlens;
  int* lens_after;
  int* used;
  int R, width, n_free, bt, num_blocks, T;
  void* stream;
};
hipError_t launch_block_tables(const TablesArgs& a);

// Strides are distances between tokens, in elements.
struct AppendArgs {
  const void* k;
  const void* v;
  const int* slot_map;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  long long ks, vs;
  int T, H, D, bt, num_blocks, fmt;
  void* stream;
};
hipError_t launch_cache_append(const AppendArgs& a);

struct DecodeArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int* block_table;
  const int* seq_lens;
  void* out;
  float* lse;
  float* ws;
  float scale;
  long long qs;
  int R, Hq, Hkv, D, bt, num_blocks, width, fmt;
  void* stream;
};
size_t attn_decode_workspace_bytes(int R, int Hq, int Hkv, int D, int bt, int width);
hipError_t launch_attn_decode(const DecodeArgs& a);

struct PromptArgs {
  const void* q;
  const void* k;
  const void* v;
  const int* cu;
  void* out;
  float* lse;
  float scale;
  long long qs, ks, vs;
  int T, R, Hq, Hkv, D, zero_rest;
  void* stream;
  bool by_length = false;  // set by the launch: tiles taken by their length
};
// Whether the tiles of 128 rows are ranked by length (tile_by_length): several
// sequences, and more than two workgroups to a CU.  That holds for the kernels of
// which three or four share a CU too, since those that do wait for one another.  Both
// ways, us, forward: 4 sequences of 5480 rows x 12/4 x 64 (516 workgroups) 54.3 for 56.9,
// 13 of 8047 34.0 for 38.7, 8 of 11000 44.6 for 61.0, 13 of 17102 x 16/4 x 128 162 for
// 182; with 400 workgroups 12.5 for 12.1.
inline bool rank_tiles(int T, int R, int per_tile) {
  const int tiles = (T + 127) / 128;
  return R > 1 && R < 512 && tiles <= 256 && (long long)tiles * per_tile > 512;
}
// Whether tiles of 32 rows, their keys split over the waves of a workgroup, are
// faster than tiles of 128 that a workgroup's waves share the keys of: where the
// chain of tiles that the last rows of a sequence go through counts for more than
// the keys' being read four times as often.  With L keys to a sequence (their
// mean), the chain is shorter by something like L, and the work larger by
// something like T Hq (600 + L).  Both ways, us: 1 x 6000 x 12/4 x 64 97 for 117,
// 2 x 4000 90 for 83, 4 x 512 10.3 for 11.7, 8 x 512 18.6 for 15.1; 1 x 3000 x 16/4
// x 128 69 for 100, 1 x 6000 240 for 217, 16 x 64 8.8 for 9.6, 8 x 256 18.8 for 13.5.
inline bool split_keys(int T, int R, int Hq, int D) {
  const long long L = T / (R > 0 ? R : 1);
  return (long long)T * Hq * (600 + L) < (D == 64 ? 82000 : 62000) * L;
}
// The same for tiles of 64 rows with their keys in two halves, D = 128: between
// the two (at D = 64 it gains nothing but for single sequences of about 8000).
inline bool split_halves(int T, int R, int Hq) {
  const long long L = T / (R > 0 ? R : 1);
  return (long long)T * Hq * (600 + L) < 108000 * L;
}
hipError_t launch_attn_prompt(const PromptArgs& a);

struct PromptBwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* out;
  const float* lse;
  const void* grad_out;
  const int* cu;
  void* grad_q;
  void* grad_k;
  void* grad_v;
  float* ws;
  float scale;
  long long qs, ks, vs, gos, gqs, gks, gvs;
  int T, R, Hq, Hkv, D, zero_rest;
  void* stream;
  int shares = 1;  // set by the launch: shares of the query heads of a key head
  bool by_length = false, keys_by_length = false;
};
size_t attn_prompt_bwd_workspace_bytes(int T, int Hq, int Hkv, int D);
hipError_t launch_attn_prompt_bwd(const PromptBwdArgs& a);

}  // namespace gdn
