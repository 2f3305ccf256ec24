// Parameters of the paged 4-bit cache's kernels, shared between the C-ABI host code
// and the kernel translation units.
#pragma once

#include "ra_internal.h"

namespace ra {

// One of the cache's arrays: rows of d / 2 code or d / 16 scale bytes, byte strides.
struct CacheRows {
  uint8_t* data;
  long long s_page, s_head, s_row;
};

struct CacheView {
  CacheRows k, ks, v, vs;
  int n_pages, hk, page_shift;
};

struct CacheSeqs {
  const int* table;
  long long table_stride;
  const int* lens;          // tokens in the cache, the call's own included
  const int* cu;            // prefix sums of the call's new tokens (device)
  int n_seqs, max_tokens;   // max_tokens: max_pages * page
  int total;                // cu[n_seqs]
};

// (rows, heads, d) tensor with element strides; the last dimension is contiguous.
struct Rows3 {
  void* data;
  long long s_row, s_head;
};

struct AppendArgs {
  Rows3 q, k, v, q_out;
  int h, hk, d;             // h = 0: no queries
  const float* cos_t;
  const float* sin_t;
  long long cos_stride, sin_stride;
  int rot, style, max_pos;  // rot = 0: no rotation
  const int* positions;
  CacheView c;
  CacheSeqs s;
  DevCtl ctl;
};
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st);

struct ReadArgs {
  Rows3 k_out, v_out;
  int hk, d;
  CacheView c;
  CacheSeqs s;
  DevCtl ctl;
};
cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t st);

struct CacheAttnArgs {
  Rows3 q, out;
  int out_f32;
  float* lse;
  long long l_sh, l_ss;
  int h, hk, G, d;          // h = hk * G
  int causal, max_new, max_kv;
  float scale_log2;
  void* ws;                 // partial results, cache_attn_ws_bytes
  int whole;                // set by the plan: items are not shared among blocks
  long long items;          // row tiles times key / value heads, cache_attn_items
  int line_shift;           // set by the plan, see LineSeq
  CacheView c;
  CacheSeqs s;
  DevCtl ctl;
};
size_t cache_attn_ws_bytes(long long total, int max_new, int h, int hk, int d, int n_seqs);
long long cache_attn_items(const int* cu_host, int n_seqs, int max_new, int G, int hk);
constexpr long long kMaxCacheItems = 1LL << 28;  // their line's length fits 32 bits
// How a call runs: the kernel that works through the items' pieces, and the one that
// joins them where items may be shared.
struct CacheAttnPlan {
  CacheAttnArgs args;
  int row_tiles;            // of 8 rows in an item: 1, 2 or 4; 0: the tensor-core kernel
  int grid;
  bool big, joins;          // big: the blocks of few rows take a whole SM
};
CacheAttnPlan plan_cache_attn(const CacheAttnArgs& a);
cudaError_t launch_cache_attn(const CacheAttnPlan& p, cudaStream_t st);
cudaError_t launch_cache_join(const CacheAttnPlan& p, cudaStream_t st);
// the variant for many query rows per key / value head
size_t cache_chunk_ws_bytes(int d);
void plan_cache_chunk(CacheAttnPlan& p);
cudaError_t launch_cache_chunk(const CacheAttnPlan& p, cudaStream_t st);
cudaError_t launch_chunk_join(const CacheAttnPlan& p, cudaStream_t st);

}  // namespace ra
