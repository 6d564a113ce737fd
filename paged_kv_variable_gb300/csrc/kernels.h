// Kernel parameter blocks and launchers (internal).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace pkv {

struct AppendParams {
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  int64_t n_stride_tok, n_stride_head;
  const int32_t* cu_knew;
  const int32_t* cache_seqlens;
  void* k_cache;
  void* v_cache;
  int64_t c_stride_page, c_stride_tok, c_stride_head;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* page_indptr;  // nullable: ragged page list offsets
  int32_t page_size;
  int32_t num_pages;
  int32_t capacity;
  int32_t batch;
  int32_t hkv;
  int32_t total_new;
  const float* k_scale;
  const float* v_scale;
  int* status;
  int status_code_only;  // status is one word (the caller's own); else three: the code and two details
};

// Norm + rotation of query and key rows (pkv_rope_spec), alone or on the way
// into the cache.
struct RopeParams {
  const float* cos_sin;
  int32_t num_positions, rot_dim, interleaved;
  float eps;
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  const __nv_bfloat16* q;  // total_q rows of hq heads
  int64_t q_stride_tok, q_stride_head;
  __nv_bfloat16* q_out;
  int64_t qo_stride_tok, qo_stride_head;
  int32_t total_q, hq;
  const int32_t* cu_q;       // append form: [batch + 1]
  const int32_t* positions;  // plain form: [total_q]
  // the keys (and, append form, values); plain form: k_out and its strides in
  // k_cache, c_stride_tok and c_stride_head
  AppendParams a;
};

// Block scales of a 4-bit cache (e4m3, a byte each) and their strides.
struct Fp4Scales {
  uint8_t* k;
  uint8_t* v;
  int64_t stride_page, stride_tok, stride_head;
};

// A cache's rows as bf16 (pkv_kv_gather).
struct GatherParams {
  __nv_bfloat16* k_out;  // nullable
  __nv_bfloat16* v_out;  // nullable
  int64_t o_stride_tok, o_stride_head;
  const int32_t* cu_rows;
  const int32_t* starts;  // nullable
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* page_indptr;  // nullable
  int32_t page_size, num_pages, capacity, batch, hkv, head_dim, total_rows;
  const void* k_cache;
  const void* v_cache;
  int64_t c_stride_page, c_stride_tok, c_stride_head;
  Fp4Scales sf;
  const float* k_scale;  // nullable: 1
  const float* v_scale;
  const int32_t* lens;   // nullable (copies that an attention reads: k_out bf16, v_out f16, both given): [batch]
                         // rows of a sequence past these are left out, those of a page out of range zeros
  const int32_t* cache_seqlens;  // (with lens) compared with the lengths of the plan
  const int32_t* plan_lc;
  int* status;
};

struct CombineParams {
  const CombineItem* items;
  const int32_t* q_offsets;  // nullable: query row offsets of the sequences (rows placed by the caller)
  const float* partial_o;
  const float* partial_lse;
  __nv_bfloat16* out;
  int64_t o_stride_tok, o_stride_head;
  float* lse;
  int32_t total_q;
  int32_t G;
};

struct AttnParams {
  const __nv_bfloat16* q;
  int64_t q_stride_tok, q_stride_head;
  __nv_bfloat16* out;
  int64_t o_stride_tok, o_stride_head;
  int32_t out_v8;      // every output row starts on 32 bytes: prefill rows are written 32 bytes per store
  float* lse;
  int32_t total_q;     // rows of q / out / lse
  const int32_t* q_offsets;  // nullable: query row offsets of the sequences (rows placed by the caller)
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* page_indptr;  // nullable: ragged page list offsets
  int32_t page_size;   // 0 = contiguous
  int32_t box_rows;    // cache rows per TMA box (divides 128 and the page size)
  int32_t row_gather;  // pages of 1, 2 or 4 tokens: rows gathered with cp.async instead of TMA boxes
  const void* kc;      // caches and their element strides (row gather)
  const void* vc;
  int64_t c_stride_page, c_stride_tok, c_stride_head;
  int32_t num_pages;   // page pool size (contiguous: batch rows of the cache)
  int32_t G;
  int32_t causal;
  float scale_log2;    // softmax_scale * log2(e)
  const float* k_scale;  // (bf16 cache: null, or the cache is copies of a 4-bit one's rows, K as bf16 and V as f16)
  const float* v_scale;
  const float* q_scale;  // nullable (fp8 cache, decode tiles): Q quantised to e4m3 for Q K^T
  const WorkItem* items;
  const int32_t* cta_begin;
  float* partial_o;
  float* partial_lse;
  int* status;
  const int32_t* cache_seqlens;
  const int32_t* plan_lc;  // [2 * batch] largest, then least cache lengths of a call
  int32_t batch;
  int32_t dynamic;     // plan_lc holds bounds; the cache lengths come from cache_seqlens
  int32_t dep_first;   // launched while the call's rotating append drains: wait for it before anything is read
  int32_t dep_late;    // nothing this launch reads comes from the kernel it overlaps
};

// Attention weight of cached keys (pkv_attn_weights).
struct WeightsParams {
  const __nv_bfloat16* q;
  int64_t q_stride_tok, q_stride_head;
  const float* lse;  // rows: cu_q[batch]
  const int32_t* cu_q;
  const int32_t* cu_knew;  // nullable
  const int32_t* cache_seqlens;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* page_indptr;
  int32_t page_size, num_pages, batch, hkv, G;
  const void* k_cache;
  int64_t c_stride_page, c_stride_tok, c_stride_head;
  Fp4Scales sf;
  const float* k_scale;  // nullable: 1
  float* scores;
  const float* scores_in;  // nullable
  int64_t s_stride_seq, s_stride_head;
  int32_t last_queries, max_seqlen_k, max_seqlen_q, max_total_q, causal;
  float scale_log2;
  int* status;
};

// Eviction (pkv_kv_evict).
struct EvictParams {
  const float* scores;
  float* scores_out;  // nullable
  int64_t s_stride_seq, s_stride_head;
  const int32_t* keep;
  const int32_t* cache_seqlens;
  int32_t* new_seqlens;
  int32_t* list;  // [batch, hkv, max_keep] old positions of the kept keys
  int2* info;     // [batch, hkv] kept and old lengths (kept < 0: a sequence that is left alone)
  int32_t fill;   // list is the caller's: entries past the kept ones become -1
  int32_t sinks, recent, max_seqlen_k, max_keep;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* page_indptr;
  int32_t page_size, num_pages, capacity, batch, hkv;
  void* k_cache;
  void* v_cache;
  int64_t c_stride_page, c_stride_tok, c_stride_head;
  Fp4Scales sf;
  int* status;
};

// Start of sequence b's page list, and how many pages it has (-1: unchecked).
__device__ __forceinline__ const int32_t* seq_pages(const int32_t* bt, int32_t stride, const int32_t* indptr, int b,
                                                    int* count) {
  if (indptr != nullptr) {
    const int a = __ldg(indptr + b);
    *count = __ldg(indptr + b + 1) - a;
    return bt + a;
  }
  *count = -1;
  return bt + (int64_t)b * stride;
}

cudaError_t launch_kv_append(const AppendParams& p, int head_dim, bool fp8, cudaStream_t stream);
cudaError_t launch_fp4_append(const AppendParams& p, const Fp4Scales& sf, int head_dim, cudaStream_t stream);
cudaError_t launch_gather(const GatherParams& p, int cache_dtype, cudaStream_t stream);
cudaError_t launch_fp4_attention(const AttnParams& p, const Fp4Scales& sf, int num_items, int max_rows, int capacity,
                                 int head_dim, cudaStream_t stream);
cudaError_t launch_weights(const WeightsParams& p, int head_dim, int cache_dtype, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams& p, int head_dim, int cache_dtype, cudaStream_t stream);
cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, cudaStream_t stream);
cudaError_t launch_rope_kv_append(const RopeParams& p, int head_dim, bool fp8, cudaStream_t stream);
// overlap_prev: launch with programmatic stream serialization, so that the
// kernel's start overlaps the end of the kernel issued just before it on the
// stream (the append kernel for the attention, the attention for the combine);
// the kernel waits for that one before reading what it wrote.
cudaError_t launch_combine(const CombineParams& p, int num_items, int head_dim, bool overlap_prev,
                           cudaStream_t stream);
// the same for plans made for shared prefixes (parts over the prefix and over each sequence's own keys)
cudaError_t launch_combine_shared(const CombineParams& p, int num_items, int max_rows, int max_parts,
                                  int head_dim, bool overlap_prev, cudaStream_t stream);
cudaError_t launch_attention(const AttnParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                             const CUtensorMap& tm_q, int num_ctas, int head_dim, bool fp8, bool has_prefill,
                             bool has_decode, bool overlap_prev, cudaStream_t stream);

}  // namespace pkv
