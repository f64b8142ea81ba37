// Shared definitions of the softmax-attention operators that serve beside the KDA layers: per-head
// norm and rotation, the paged key-value cache, and decode attention over it (not public ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"

namespace kda {

constexpr int kAttnMaxDim = 128;             // head sizes: multiples of 16 up to this
constexpr float kE4M3Max = 448.0f;
constexpr float kKvScaleFloor = 5.421010862427522e-20f;  // 2^-64: the smallest scale of a quantised row

// One projection (queries or keys) of norm + rotation: rows [tokens][heads][d], tokens `stride`
// elements apart, heads contiguous.
struct HeadRows {
  const __nv_bfloat16* x;
  int64_t stride;
  int32_t heads;
  const float* w;  // [d] norm weight, null: no norm
};

struct RopeArgs {
  HeadRows q, k, v;           // v only for the cache write (heads 0 otherwise)
  __nv_bfloat16* q_out;       // [tokens][q.heads][d]
  __nv_bfloat16* k_out;       // [tokens][k.heads][d]; null for the cache write
  const float* cos_sin;       // [max_pos][rot]: cos then sin; null: no rotation
  const int32_t* positions;   // [tokens]
  int64_t tokens;
  int32_t d, rot, max_pos, interleaved;
  float eps;
  uint32_t* status;           // may be null
  // cache write
  void* k_cache;
  void* v_cache;
  float* k_scale;             // [pages][heads][page], null: bf16 cache
  float* v_scale;
  const int32_t* slots;       // [tokens], negative: skip the token
  int64_t k_page_stride, v_page_stride;  // elements
  int64_t num_slots;
  int32_t page_shift;
};

struct RopeBwdArgs {
  HeadRows q, k;
  const __nv_bfloat16* dyq;   // [tokens][heads][d]
  const __nv_bfloat16* dyk;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  float* dwq;                 // [d] or null
  float* dwk;
  const float* cos_sin;
  const int32_t* positions;
  int64_t tokens;
  int32_t d, rot, max_pos, interleaved;
  float eps;
  float* partials;            // [CTAs][kAttnMaxDim]
  uint32_t* status;
};

struct KvReadArgs {
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  int64_t k_page_stride, v_page_stride;
  const int32_t* page_table;  // [num_seqs][max_pages]
  const int32_t* cu_seqlens;  // [num_seqs + 1]
  __nv_bfloat16* k_out;       // [total][heads][d]
  __nv_bfloat16* v_out;
  int64_t total;
  int32_t num_seqs, heads, d, page_shift, max_pages, num_pages;
  uint32_t* status;
};

struct AttnDecodeArgs {
  const __nv_bfloat16* q;     // [batch][new_tokens][hq][d]
  const void* k_cache;        // [pages][hkv][page][d]
  const void* v_cache;
  const float* k_scale;       // null: bf16 cache
  const float* v_scale;
  int64_t k_page_stride, v_page_stride;
  const int32_t* page_table;  // [batch][max_pages]
  const int32_t* seq_lens;    // [batch]
  __nv_bfloat16* out;
  float* lse;                 // [batch][new_tokens][hq] or null
  int32_t batch, new_tokens, hq, hkv, d, page_shift, max_pages, num_pages, window;
  float scale, softcap;
  uint8_t* workspace;
};

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream);
cudaError_t launch_qk_norm_rope_bwd(const RopeBwdArgs& a, cudaStream_t stream);
cudaError_t launch_kv_append(const RopeArgs& a, cudaStream_t stream);
cudaError_t launch_kv_read(const KvReadArgs& a, cudaStream_t stream);
cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t stream);
// Pieces of work of a norm + rotation call (their count has to stay below 2^31).
int64_t rope_items(int64_t tokens, int32_t hq, int32_t hk, int32_t hv, int batches = 1);
size_t rope_bwd_workspace_bytes();
size_t attn_decode_workspace_bytes(int32_t rows, int32_t d);

}  // namespace kda
