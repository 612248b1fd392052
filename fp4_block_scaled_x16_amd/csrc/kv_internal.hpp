// Launch interface of the attention operators: norm and rotation of queries
// and keys, the paged key-value cache, attention of one new token per request.
// Arguments have been validated by the caller (kv_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp4.h"

namespace fp4lib {

// Formats of a cache as the kernels' template arguments.
enum KvFmt : int { kKvFp8 = 0, kKvMx8 = 1, kKvMx4 = 2, kKvNv4 = 3, kKvUe4 = 4 };

struct KvCacheArgs {
  uint8_t* codes[2];           // K, V
  uint8_t* scales[2];
  int64_t page, head, token;   // strides of the codes, bytes
  int64_t s_page, s_head, s_block;
  int64_t pages;
  const float* amax;           // [2], two-level formats
  float target;
  int fmt, heads, head_dim;
  int page_shift;              // log2 of the page size
};

struct HeadsArgs {
  uint16_t* x;
  int64_t token, head;         // strides, elements
  int heads;
};

struct NormArgs {
  const void* w[2];            // of q and k; null: no norm
  int w_f32;
  float eps;
  const float* table;          // null: no rotation
  int64_t table_rows;
  int pairs;                   // rotary_dim / 2
  int interleaved;
  const int64_t* positions;
};

// Rows of q and k (x null: left out) normed and rotated, to out[0] and out[1] or,
// where `cache` is given, k's and v's into the cache.
struct QkRowsArgs {
  HeadsArgs in[3];             // q, k, v
  HeadsArgs out[2];
  NormArgs norm;
  KvCacheArgs cache;
  const int64_t* slots;
  int64_t tokens;
  int head_dim, cached;
  int part[4];                 // set by the launcher
};

struct QkGradArgs {
  HeadsArgs x[2], dy[2], dx[2];
  NormArgs norm;
  float* dw[2];                // null: not wanted
  int accumulate;              // added to dw
  float* part;                 // workspace
  int64_t tokens;
  int head_dim;
  int groups[2];               // set by the launcher: workgroups of q and of k
};

struct KvReadArgs {
  KvCacheArgs cache;
  const int64_t* slots;
  int64_t n;
  void* out[2];                // may be null
  int out_f32;
};

struct AttnArgs {
  KvCacheArgs cache;
  HeadsArgs q;
  const int32_t* table;
  int64_t table_stride;
  int table_width;
  const int32_t* lens;
  int requests;
  float scale;
  void* out;                   // [requests, heads, head_dim]
  int out_f32;
  float* lse;                  // null, or [requests, heads]
  float* part;                 // workspace: null with splits == 1
  int64_t part_bytes;
  int splits, min_part;        // set by the launcher: parts of a request at most, tokens of one at least
  int waves;                   // set by the launcher: of a workgroup
  int stream;                  // set by the launcher: codes are read past the caches
  int planned;                 // set by the launcher: the parts go by the lengths (attention_common.hpp)
  int target[2];               // set by the launcher: parts of a key head's requests together (attention.hip)
  int64_t items;               // set by the launcher: a key head's parts at most
  int group, tiles;            // set by the launcher: query heads of a key head, workgroups that share them
  uint32_t by_splits, by_heads;   // set by the launcher: 2^32 / splits and / cache.heads, rounded up
};

hipError_t launch_qk_rows(const QkRowsArgs& a, hipStream_t s);
hipError_t launch_qk_grad(const QkGradArgs& a, hipStream_t s);
int64_t qk_grad_workspace(int head_dim);
hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s);
hipError_t launch_attention(const AttnArgs& a, hipStream_t s);
int64_t attention_workspace(const AttnArgs& a);
void set_attention_splits(int splits);     // fp4_selftest_set_attention_splits

}  // namespace fp4lib
