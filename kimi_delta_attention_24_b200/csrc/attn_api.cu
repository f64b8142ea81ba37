// C ABI of the softmax-attention operators: argument validation and launches.  The declarations and
// the contract live in include/kda.h.
#include <math.h>

#include "attn_common.cuh"
#include "kda_device.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool head_dim_ok(int32_t d) { return d >= 16 && d <= kda::kAttnMaxDim && d % 16 == 0; }
kda_status_t launched(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
cudaStream_t cu(kda_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Rows [tokens][heads][d] of a projection, `stride` elements between tokens.
bool rows_ok(const void* p, int64_t stride, int64_t tokens, int32_t heads, int32_t d) {
  if (heads == 0 || tokens == 0) return true;
  return p && aligned(p, 16) && stride % 8 == 0 && stride >= (int64_t)heads * d && stride <= INT64_MAX / 2 / tokens;
}

// The parts common to the norm + rotation calls: sizes, weights, the rotation's table.
kda_status_t check_rope(const float* q_weight, const float* k_weight, float eps, const float* cos_sin,
                        const int32_t* positions, int64_t tokens, int32_t hq, int32_t hk, int32_t hv, int32_t d,
                        int32_t rot, int32_t max_pos, int32_t interleaved, const void* workspace) {
  if (!head_dim_ok(d)) return KDA_ERR_UNSUPPORTED;
  if (tokens < 0 || tokens > INT32_MAX || hq < 0 || hk < 0 || hq > 65535 || hk > 65535) return KDA_ERR_INVALID_ARGUMENT;
  if (rot < 0 || rot > d || rot % 16 != 0) return KDA_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return KDA_ERR_INVALID_ARGUMENT;
  if ((q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16))) return KDA_ERR_INVALID_ARGUMENT;
  if ((q_weight || k_weight) && !(eps >= 0.f && isfinite(eps))) return KDA_ERR_INVALID_ARGUMENT;
  if (rot > 0 && tokens > 0 && (!cos_sin || !positions || !aligned(cos_sin, 16) || !aligned(positions, 4) || max_pos < 0))
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace && !aligned(workspace, 256)) return KDA_ERR_INVALID_ARGUMENT;
  if (kda::rope_items(tokens, hq, hk, hv) > INT32_MAX / 16) return KDA_ERR_INVALID_ARGUMENT;
  return KDA_OK;
}

// The paged cache: sizes, strides, and whether the scales come as a pair (e4m3) or not at all (bf16).
kda_status_t check_cache(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale, int32_t hkv,
                         int32_t d, int32_t num_pages, int32_t page_size, int64_t k_page_stride, int64_t v_page_stride) {
  if (!head_dim_ok(d)) return KDA_ERR_UNSUPPORTED;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return KDA_ERR_UNSUPPORTED;
  if (hkv <= 0 || hkv > 65535 || num_pages <= 0 || (int64_t)num_pages * page_size > INT32_MAX) return KDA_ERR_INVALID_ARGUMENT;
  if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return KDA_ERR_INVALID_ARGUMENT;
  if ((k_scale == nullptr) != (v_scale == nullptr) || !aligned(k_scale, 4) || !aligned(v_scale, 4)) return KDA_ERR_INVALID_ARGUMENT;
  const int64_t page = (int64_t)hkv * page_size * d, align = k_scale ? 16 : 8;
  // (2^38 elements are beyond any memory: a stride by mistake)
  for (int64_t s : {k_page_stride, v_page_stride})
    if (s < page || s % align != 0 || s >= (int64_t)1 << 38) return KDA_ERR_INVALID_ARGUMENT;
  return KDA_OK;
}

// The factors that scores are multiplied with, in the kernel's units (base 2, with a cap the cap's): normal
// fp32 numbers, or zero for a scale of zero.  (A product that overflows or loses bits would change the scores.)
bool factors_ok(float scale, float softcap) {
  if (!isfinite(scale) || !(softcap >= 0.f) || !isfinite(softcap * kda::kLog2e)) return false;
  const float factor = softcap > 0.f ? scale / softcap : scale * kda::kLog2e;
  return scale == 0.f || isnormal(factor);
}

int log2_of(int32_t n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

kda::HeadRows rows(const void* p, int64_t stride, int32_t heads, const float* w) {
  kda::HeadRows r;
  r.x = static_cast<const __nv_bfloat16*>(p);
  r.stride = stride;
  r.heads = heads;
  r.w = w;
  return r;
}

}  // namespace

extern "C" {

kda_status_t kda_qk_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride, const float* q_weight,
                              const float* k_weight, float eps, const float* cos_sin, const int32_t* positions, void* q_out,
                              void* k_out, int64_t tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                              int32_t rot_dim, int32_t max_positions, int32_t interleaved, void* workspace,
                              kda_stream_t stream) {
  const kda_status_t st = check_rope(q_weight, k_weight, eps, cos_sin, positions, tokens, num_q_heads, num_kv_heads, 0, head_dim,
                                     rot_dim, max_positions, interleaved, workspace);
  if (st != KDA_OK) return st;
  if (!rows_ok(q, q_stride, tokens, num_q_heads, head_dim) || !rows_ok(k, k_stride, tokens, num_kv_heads, head_dim) ||
      !rows_ok(q_out, (int64_t)num_q_heads * head_dim, tokens, num_q_heads, head_dim) ||
      !rows_ok(k_out, (int64_t)num_kv_heads * head_dim, tokens, num_kv_heads, head_dim))
    return KDA_ERR_INVALID_ARGUMENT;
  kda::RopeArgs a = {};
  a.q = rows(q, q_stride, num_q_heads, q_weight);
  a.k = rows(k, k_stride, num_kv_heads, k_weight);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.cos_sin = rot_dim > 0 ? cos_sin : nullptr;
  a.positions = positions;
  a.tokens = tokens;
  a.d = head_dim;
  a.rot = rot_dim;
  a.max_pos = max_positions;
  a.interleaved = interleaved;
  a.eps = eps;
  a.status = static_cast<uint32_t*>(workspace);
  return launched(kda::launch_qk_norm_rope(a, cu(stream)));
}

size_t kda_qk_norm_rope_bwd_workspace_size(void) { return kda::rope_bwd_workspace_bytes(); }

kda_status_t kda_qk_norm_rope_bwd(const void* d_q_out, const void* d_k_out, const void* q, const void* k, int64_t q_stride,
                                  int64_t k_stride, const float* q_weight, const float* k_weight, float eps,
                                  const float* cos_sin, const int32_t* positions, void* dq, void* dk, float* dq_weight,
                                  float* dk_weight, int64_t tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t rot_dim, int32_t max_positions, int32_t interleaved,
                                  void* workspace, size_t workspace_bytes, kda_stream_t stream) {
  const kda_status_t st = check_rope(q_weight, k_weight, eps, cos_sin, positions, tokens, num_q_heads, num_kv_heads, 0, head_dim,
                                     rot_dim, max_positions, interleaved, workspace);
  if (st != KDA_OK) return st;
  const int64_t qs = (int64_t)num_q_heads * head_dim, ks = (int64_t)num_kv_heads * head_dim;
  if (!rows_ok(q, q_stride, tokens, num_q_heads, head_dim) || !rows_ok(k, k_stride, tokens, num_kv_heads, head_dim) ||
      !rows_ok(d_q_out, qs, tokens, num_q_heads, head_dim) || !rows_ok(d_k_out, ks, tokens, num_kv_heads, head_dim) ||
      !rows_ok(dq, qs, tokens, num_q_heads, head_dim) || !rows_ok(dk, ks, tokens, num_kv_heads, head_dim))
    return KDA_ERR_INVALID_ARGUMENT;
  if ((q_weight != nullptr) != (dq_weight != nullptr) || (k_weight != nullptr) != (dk_weight != nullptr) ||
      !aligned(dq_weight, 4) || !aligned(dk_weight, 4))
    return KDA_ERR_INVALID_ARGUMENT;
  if (!workspace) return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < kda_qk_norm_rope_bwd_workspace_size()) return KDA_ERR_WORKSPACE_TOO_SMALL;
  kda::RopeBwdArgs a = {};
  a.q = rows(q, q_stride, num_q_heads, q_weight);
  a.k = rows(k, k_stride, num_kv_heads, k_weight);
  a.dyq = static_cast<const __nv_bfloat16*>(d_q_out);
  a.dyk = static_cast<const __nv_bfloat16*>(d_k_out);
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dwq = dq_weight;
  a.dwk = dk_weight;
  a.cos_sin = rot_dim > 0 ? cos_sin : nullptr;
  a.positions = positions;
  a.tokens = tokens;
  a.d = head_dim;
  a.rot = rot_dim;
  a.max_pos = max_positions;
  a.interleaved = interleaved;
  a.eps = eps;
  a.status = static_cast<uint32_t*>(workspace);
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kda::kWorkspaceHeader);
  return launched(kda::launch_qk_norm_rope_bwd(a, cu(stream)));
}

kda_status_t kda_kv_append(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                           const float* q_weight, const float* k_weight, float eps, const float* cos_sin,
                           const int32_t* positions, void* q_out, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                           const int32_t* slots, int64_t tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                           int32_t rot_dim, int32_t max_positions, int32_t interleaved, int32_t num_pages, int32_t page_size,
                           int64_t k_page_stride, int64_t v_page_stride, void* workspace, kda_stream_t stream) {
  kda_status_t st = check_rope(q_weight, k_weight, eps, cos_sin, positions, tokens, num_q_heads, num_kv_heads, num_kv_heads,
                               head_dim, rot_dim, max_positions, interleaved, workspace);
  if (st != KDA_OK) return st;
  st = check_cache(k_cache, v_cache, k_scale, v_scale, num_kv_heads, head_dim, num_pages, page_size, k_page_stride, v_page_stride);
  if (st != KDA_OK) return st;
  if (!rows_ok(q, q_stride, tokens, num_q_heads, head_dim) || !rows_ok(k, k_stride, tokens, num_kv_heads, head_dim) ||
      !rows_ok(v, v_stride, tokens, num_kv_heads, head_dim) ||
      !rows_ok(q_out, (int64_t)num_q_heads * head_dim, tokens, num_q_heads, head_dim))
    return KDA_ERR_INVALID_ARGUMENT;
  if (tokens > 0 && (!slots || !aligned(slots, 4))) return KDA_ERR_INVALID_ARGUMENT;
  kda::RopeArgs a = {};
  a.q = rows(q, q_stride, num_q_heads, q_weight);
  a.k = rows(k, k_stride, num_kv_heads, k_weight);
  a.v = rows(v, v_stride, num_kv_heads, nullptr);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.cos_sin = rot_dim > 0 ? cos_sin : nullptr;
  a.positions = positions;
  a.tokens = tokens;
  a.d = head_dim;
  a.rot = rot_dim;
  a.max_pos = max_positions;
  a.interleaved = interleaved;
  a.eps = eps;
  a.status = static_cast<uint32_t*>(workspace);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.slots = slots;
  a.k_page_stride = k_page_stride;
  a.v_page_stride = v_page_stride;
  a.num_slots = (int64_t)num_pages * page_size;
  a.page_shift = log2_of(page_size);
  return launched(kda::launch_kv_append(a, cu(stream)));
}

kda_status_t kda_kv_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                         const int32_t* page_table, const int32_t* cu_seqlens, void* k_out, void* v_out, int32_t num_seqs,
                         int64_t total_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t num_pages, int32_t page_size,
                         int32_t max_pages, int64_t k_page_stride, int64_t v_page_stride, void* workspace,
                         kda_stream_t stream) {
  const kda_status_t st = check_cache(k_cache, v_cache, k_scale, v_scale, num_kv_heads, head_dim, num_pages, page_size,
                                      k_page_stride, v_page_stride);
  if (st != KDA_OK) return st;
  if (num_seqs < 0 || total_tokens < 0 || total_tokens > INT32_MAX || max_pages < 0 ||
      (int64_t)max_pages * page_size > INT32_MAX)
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace && !aligned(workspace, 256)) return KDA_ERR_INVALID_ARGUMENT;
  if (kda::rope_items(total_tokens, 2 * num_kv_heads, 0, 0) > INT32_MAX / 16) return KDA_ERR_INVALID_ARGUMENT;
  if (num_seqs > 0 && total_tokens > 0) {
    if (!cu_seqlens || !aligned(cu_seqlens, 4) || !page_table || !aligned(page_table, 4) || !k_out || !v_out ||
        !aligned(k_out, 16) || !aligned(v_out, 16))
      return KDA_ERR_INVALID_ARGUMENT;
  }
  kda::KvReadArgs a = {};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_page_stride = k_page_stride;
  a.v_page_stride = v_page_stride;
  a.page_table = page_table;
  a.cu_seqlens = cu_seqlens;
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.total = total_tokens;
  a.num_seqs = num_seqs;
  a.heads = num_kv_heads;
  a.d = head_dim;
  a.page_shift = log2_of(page_size);
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.status = static_cast<uint32_t*>(workspace);
  return launched(kda::launch_kv_read(a, cu(stream)));
}

size_t kda_attn_decode_workspace_size(int32_t new_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (new_tokens <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 || !head_dim_ok(head_dim))
    return kda::kWorkspaceHeader;
  const int64_t rows = (int64_t)new_tokens * (num_q_heads / num_kv_heads);
  return kda::attn_decode_workspace_bytes(rows > 1 << 20 ? 1 << 20 : (int32_t)rows, head_dim);
}

kda_status_t kda_attn_decode(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                             const int32_t* page_table, const int32_t* seq_lens, float scale, float softcap, int32_t window,
                             void* out, float* lse, int32_t batch, int32_t new_tokens, int32_t num_q_heads,
                             int32_t num_kv_heads, int32_t head_dim, int32_t num_pages, int32_t page_size, int32_t max_pages,
                             int64_t k_page_stride, int64_t v_page_stride, void* workspace, size_t workspace_bytes,
                             kda_stream_t stream) {
  const kda_status_t st = check_cache(k_cache, v_cache, k_scale, v_scale, num_kv_heads, head_dim, num_pages, page_size,
                                      k_page_stride, v_page_stride);
  if (st != KDA_OK) return st;
  if (batch < 0 || new_tokens < 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 || max_pages < 0 ||
      (int64_t)max_pages * page_size > 1 << 30 || window < 0)
    return KDA_ERR_INVALID_ARGUMENT;
  if (!factors_ok(scale, softcap)) return KDA_ERR_INVALID_ARGUMENT;
  const int64_t rows = (int64_t)new_tokens * (num_q_heads / num_kv_heads);
  // (rows, units and the rows' indexes are int32; a unit is a sequence's kv head and 8 or 16 of its rows)
  if (rows > 1 << 20 || (int64_t)batch * num_kv_heads > INT32_MAX / (rows / 16 + 1) ||
      (int64_t)batch * new_tokens > INT32_MAX / num_q_heads)
    return KDA_ERR_INVALID_ARGUMENT;
  if ((int64_t)batch * new_tokens > 0) {
    if (!q || !out || !seq_lens || (max_pages > 0 && !page_table)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(seq_lens, 4) || !aligned(page_table, 4) || q == out)
      return KDA_ERR_INVALID_ARGUMENT;
  }
  if (!workspace || !aligned(workspace, 256)) return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < kda_attn_decode_workspace_size(new_tokens, num_q_heads, num_kv_heads, head_dim))
    return KDA_ERR_WORKSPACE_TOO_SMALL;
  kda::AttnDecodeArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_page_stride = k_page_stride;
  a.v_page_stride = v_page_stride;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.batch = batch;
  a.new_tokens = new_tokens;
  a.hq = num_q_heads;
  a.hkv = num_kv_heads;
  a.d = head_dim;
  a.page_shift = log2_of(page_size);
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.window = window;
  a.scale = scale;
  a.softcap = softcap;
  a.workspace = static_cast<uint8_t*>(workspace);
  return launched(kda::launch_attn_decode(a, cu(stream)));
}

}  // extern "C"
