// Internal interface between the C ABI of the attention side
// (attention_api.cpp) and its kernel launchers.  Not installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "opq_attention.h"

namespace opq {

constexpr int kMaxAxes = 4;

// rotary.hip
hipError_t launch_rotary_table(const double* freq, int64_t pairs, int64_t len, double amplitude,
                               float* table, hipStream_t stream);

struct RotaryArgs {
  const void* x;
  void* out;
  const int32_t* positions;
  const float* table;
  int64_t x_token, x_head, out_token, out_head;  // strides in elements
  int64_t tokens, table_len;
  int heads, dim, rot, axes;
  int end[kMaxAxes];  // first pair past each axis' section
  float turn;         // +1 forward, -1 backward: factor of the sines
};
hipError_t launch_rotary(const RotaryArgs& a, bool bf16, bool interleaved, hipStream_t stream);

// Byte planes of the sixteen bfloat16 levels L_q = bf16(G_q): lo[i] holds the
// low bytes of L_4i..L_4i+3, hi[i] the high bytes.
struct LevelPlanes {
  uint32_t lo[4];
  uint32_t hi[4];
};

// Encoder of OPQ_CACHE_OPQ4 rows: decision points, alpha and the half width of
// the band around half-integers in which the approximate power decides nothing.
struct CacheCodes {
  float t[15];
  float alpha;
  float guard;
};

struct CacheRows {  // one of keys or values
  const void* x;
  int64_t token_stride, head_stride;
  void* codes;
  uint32_t* sign;
  float* scale;
};

// cache.hip
hipError_t launch_cache_write(const CacheRows (&side)[2], const opq_cache& c, bool bf16,
                              int64_t tokens, const int32_t* slots, const CacheCodes& cc,
                              hipStream_t stream);
// x of a side is its output, dense [tokens][heads][dim]
hipError_t launch_cache_read(const CacheRows (&side)[2], const opq_cache& c, bool bf16,
                             int64_t tokens, const int32_t* slots, const LevelPlanes& lp,
                             hipStream_t stream);

constexpr int64_t kMaxMoves = 128;  // rows that opq_cache_move holds of a sequence and head
hipError_t launch_cache_move(const CacheRows (&side)[2], const opq_cache& c, int64_t batch,
                             int64_t count, const int32_t* src, const int32_t* dst,
                             hipStream_t stream);

// attention.hip
struct AttentionPlan {
  int tiles;      // 16-row tiles of query rows in a workgroup
  int group_rows; // query rows of a workgroup
  int groups;     // workgroups that cover a kv head's query rows
  int splits;     // pieces of the keys
  int64_t chunk;  // keys of a piece, a multiple of 128
  size_t workspace;
};
AttentionPlan attention_plan(int64_t batch, int64_t draft, int64_t heads, int64_t kv_heads,
                             int64_t dim, int64_t max_len);

struct AttentionArgs {
  const uint16_t* q;
  int64_t q_batch, q_token, q_head;
  const char* k;
  const uint32_t* k_sign;
  const float* k_scale;
  const char* v;
  const uint32_t* v_sign;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* lens;
  const int32_t* counts;
  const uint32_t* mask;
  int64_t mask_batch, mask_words, max_pages, capacity, chunk;
  uint32_t pages;
  int page_shift, batch, draft, heads, kv_heads, share, rows, splits, groups, group_rows;
  float scale_log2;  // |scale| * log2(e)
  uint32_t q_flip;   // sign bits of two bfloat16: set for a negative scale
  uint16_t* out;
  float* lse;
  float* part_o;   // [splits][batch][kv_heads][rows][dim]
  float* part_ml;  // [splits][batch][kv_heads][rows][2]
  LevelPlanes lp;
};
hipError_t launch_attention(const AttentionArgs& a, int format, int dim, int tiles,
                            hipStream_t stream);

}  // namespace opq
