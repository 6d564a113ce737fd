// C-ABI entry points: argument validation, TMA descriptors, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "fp4.cuh"
#include "kernels.h"

namespace pkv {

namespace {
thread_local char g_err[512] = "";
thread_local cudaEvent_t g_ev_start = nullptr;
thread_local cudaEvent_t g_ev_stop = nullptr;

// Under stream capture the record becomes an event-record node of the graph,
// so that every replay re-records the caller's event around the kernel.
cudaError_t record_profile_event(cudaEvent_t ev, cudaStream_t s) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(s, &cs);
  if (e != cudaSuccess) return e;
  return cs == cudaStreamCaptureStatusActive ? cudaEventRecordWithFlags(ev, s, cudaEventRecordExternal)
                                             : cudaEventRecord(ev, s);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

pkv_status fail(pkv_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

pkv_status validate_problem(const pkv_problem* p);  // plan.cpp

namespace {

pkv_status cuda_fail(cudaError_t e, const char* what) {
  return fail(PKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// 4-D map over a cache (D, Hkv, rows-per-page-or-seq, pages-or-batch); a box
// is cache_box_rows() rows of one 128-byte column chunk with the 128-byte
// swizzle (an fp8 cache at D = 64: its 64-byte rows with the 64-byte swizzle),
// zero fill outside the tensor.
pkv_status make_cache_map(CUtensorMap* map, const pkv_problem& pr, const pkv_fwd_args& a, void* base) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const bool fp8 = pr.cache_dtype == PKV_FP8_E4M3;
  const int es = fp8 ? 1 : 2;
  const cuuint64_t rows = pr.page_size > 0 ? (cuuint64_t)pr.page_size : (cuuint64_t)pr.cache_capacity;
  cuuint64_t dims[4] = {(cuuint64_t)pr.head_dim, (cuuint64_t)pr.num_heads_kv, rows, (cuuint64_t)pr.num_pages};
  cuuint64_t strides[3] = {(cuuint64_t)a.kc_stride_head * es, (cuuint64_t)a.kc_stride_tok * es,
                           (cuuint64_t)a.kc_stride_page * es};
  cuuint32_t box[4] = {(cuuint32_t)(128 / es), 1,
                       (cuuint32_t)cache_box_rows(pr.page_size, pr.cache_capacity, kv_tile_keys(pr.head_dim)), 1};
  const bool narrow = pr.head_dim * es < 128;
  if (narrow) box[0] = (cuuint32_t)pr.head_dim;
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return PKV_OK;
}

// 3-D map over q (D, Hq, total_q): a box of nh heads x 128/nh tokens (nh = G,
// at most 128) is the Q tile of one tensor-core item (row = token * nh + g).
pkv_status make_q_map(CUtensorMap* map, const pkv_problem& pr, const pkv_fwd_args& a, int total_q) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const int nh = tc_group_heads(pr.num_heads_q / pr.num_heads_kv);
  cuuint64_t dims[3] = {(cuuint64_t)pr.head_dim, (cuuint64_t)pr.num_heads_q, (cuuint64_t)(total_q > 0 ? total_q : 1)};
  cuuint64_t strides[2] = {(cuuint64_t)a.q_stride_head * 2, (cuuint64_t)a.q_stride_tok * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)nh, (cuuint32_t)(kPrefillRowsTc / nh)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled (q) failed (%d)", (int)r);
  return PKV_OK;
}

pkv_status validate_cache_args(const pkv_problem& pr, const pkv_fwd_args* a) {
  if (!a) return fail(PKV_ERR_INVALID_ARG, "args is NULL");
  if (!a->k_cache || !a->v_cache) return fail(PKV_ERR_INVALID_ARG, "k_cache / v_cache is NULL");
  if (!aligned16(a->k_cache) || !aligned16(a->v_cache))
    return fail(PKV_ERR_INVALID_ARG, "cache base pointers must be 16-byte aligned");
  if (!a->cache_seqlens) return fail(PKV_ERR_INVALID_ARG, "cache_seqlens is NULL");
  const bool fp4 = pr.cache_dtype == PKV_FP4_E2M1;
  const int es = pr.cache_dtype == PKV_BF16 ? 2 : 1;
  if (a->kc_stride_head <= 0 || a->kc_stride_tok <= 0 || a->kc_stride_page <= 0)
    return fail(PKV_ERR_INVALID_ARG, "cache strides must be positive");
  if ((a->kc_stride_head * es) % 16 || (a->kc_stride_tok * es) % 16 || (a->kc_stride_page * es) % 16)
    return fail(PKV_ERR_INVALID_ARG, "cache strides must be multiples of 16 bytes");
  if (a->kc_stride_head < (fp4 ? pr.head_dim / 2 : pr.head_dim))
    return fail(PKV_ERR_INVALID_ARG, "kc_stride_head < head_dim%s", fp4 ? " / 2" : "");
  if (pr.page_size > 0) {
    if (!a->block_table) return fail(PKV_ERR_INVALID_ARG, "paged cache needs block_table");
    if (!a->page_indptr && a->block_table_stride < pr.cache_capacity / pr.page_size)
      return fail(PKV_ERR_INVALID_ARG, "block_table_stride %d < cache_capacity / page_size", a->block_table_stride);
  }
  if (pr.cache_dtype != PKV_BF16 && (!a->k_scale || !a->v_scale))
    return fail(PKV_ERR_INVALID_ARG, "fp8 and fp4 caches need k_scale and v_scale");
  if (fp4) {
    const int n = pr.head_dim / kFp4Block;  // bytes of a row's scales
    if (!a->k_sf || !a->v_sf) return fail(PKV_ERR_INVALID_ARG, "fp4 cache needs k_sf and v_sf");
    if (reinterpret_cast<uintptr_t>(a->k_sf) % n || reinterpret_cast<uintptr_t>(a->v_sf) % n || a->sf_stride_page <= 0 ||
        a->sf_stride_tok <= 0 || a->sf_stride_head < n || a->sf_stride_page % n || a->sf_stride_tok % n ||
        a->sf_stride_head % n)
      return fail(PKV_ERR_INVALID_ARG, "k_sf / v_sf: base and positive strides must be multiples of %d bytes", n);
  }
  return PKV_OK;
}

Fp4Scales fp4_scales(const pkv_fwd_args* a) {
  return {static_cast<uint8_t*>(a->k_sf), static_cast<uint8_t*>(a->v_sf), a->sf_stride_page, a->sf_stride_tok,
          a->sf_stride_head};
}

cudaError_t run_append(const pkv_problem& pr, const pkv_fwd_args* a, const AppendParams& ap, cudaStream_t s) {
  if (pr.cache_dtype == PKV_FP4_E2M1) return launch_fp4_append(ap, fp4_scales(a), pr.head_dim, s);
  return launch_kv_append(ap, pr.head_dim, pr.cache_dtype == PKV_FP8_E4M3, s);
}

pkv_status validate_new_args(const pkv_problem& pr, const pkv_fwd_args* a) {
  if (!a->k_new || !a->v_new || !a->cu_seqlens_knew)
    return fail(PKV_ERR_INVALID_ARG, "k_new, v_new and cu_seqlens_knew must all be given");
  if (!aligned16(a->k_new) || !aligned16(a->v_new))
    return fail(PKV_ERR_INVALID_ARG, "k_new / v_new must be 16-byte aligned");
  if (a->knew_stride_head < pr.head_dim || a->knew_stride_tok <= 0 || (a->knew_stride_head * 2) % 16 ||
      (a->knew_stride_tok * 2) % 16)
    return fail(PKV_ERR_INVALID_ARG, "k_new strides must be >= head_dim and multiples of 16 bytes");
  return PKV_OK;
}

AppendParams append_params(const pkv_problem& pr, const pkv_fwd_args* a, int32_t total_new, int* status) {
  AppendParams ap{};
  ap.k_new = static_cast<const __nv_bfloat16*>(a->k_new);
  ap.v_new = static_cast<const __nv_bfloat16*>(a->v_new);
  ap.n_stride_tok = a->knew_stride_tok;
  ap.n_stride_head = a->knew_stride_head;
  ap.cu_knew = a->cu_seqlens_knew;
  ap.cache_seqlens = a->cache_seqlens;
  ap.k_cache = a->k_cache;
  ap.v_cache = a->v_cache;
  ap.c_stride_page = a->kc_stride_page;
  ap.c_stride_tok = a->kc_stride_tok;
  ap.c_stride_head = a->kc_stride_head;
  ap.block_table = a->block_table;
  ap.bt_stride = a->block_table_stride;
  ap.page_indptr = a->page_indptr;
  ap.page_size = pr.page_size;
  ap.num_pages = pr.num_pages;
  ap.capacity = pr.cache_capacity;
  ap.batch = pr.batch;
  ap.hkv = pr.num_heads_kv;
  ap.total_new = total_new;
  ap.k_scale = a->k_scale;
  ap.v_scale = a->v_scale;
  ap.status = status;
  return ap;
}

pkv_status validate_rope_spec(const pkv_rope_spec& r, int head_dim) {
  if (r.rot_dim < 0 || r.rot_dim > head_dim || r.rot_dim % 8 != 0)
    return fail(PKV_ERR_INVALID_ARG, "rot_dim %d: a multiple of 8 from 0 to head_dim", r.rot_dim);
  if ((r.rot_dim > 0) != (r.cos_sin != nullptr))
    return fail(PKV_ERR_INVALID_ARG, "cos_sin must be given exactly when rot_dim > 0");
  if (r.rot_dim > 0 && (r.num_positions <= 0 || !aligned16(r.cos_sin)))
    return fail(PKV_ERR_INVALID_ARG, "cos_sin needs num_positions > 0 and a 16-byte aligned base");
  if (r.interleaved != 0 && r.interleaved != 1) return fail(PKV_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if ((r.q_weight && !aligned16(r.q_weight)) || (r.k_weight && !aligned16(r.k_weight)))
    return fail(PKV_ERR_INVALID_ARG, "norm weights must be 16-byte aligned");
  if ((r.q_weight || r.k_weight) && !(std::isfinite(r.eps) && r.eps > 0.f))
    return fail(PKV_ERR_INVALID_ARG, "eps must be finite and positive");
  return PKV_OK;
}

// One bf16 tensor of head rows (tokens, heads, head_dim): base and strides.
pkv_status validate_rows(const char* what, const void* ptr, int64_t stride_tok, int64_t stride_head, int head_dim) {
  if (!ptr) return fail(PKV_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned16(ptr) || stride_head < head_dim || stride_tok <= 0 || stride_head % 8 || stride_tok % 8)
    return fail(PKV_ERR_INVALID_ARG,
                "%s must be 16-byte aligned, with strides that are multiples of 8 elements (heads: >= head_dim)", what);
  return PKV_OK;
}

// An output is its own input (same strides) or, as far as their first elements
// show, another tensor.
pkv_status validate_in_place(const char* what, const void* in, const void* out, int64_t it, int64_t ih, int64_t ot,
                             int64_t oh) {
  if (in == out && (it != ot || ih != oh))
    return fail(PKV_ERR_INVALID_ARG, "%s in place needs the strides of its input", what);
  return PKV_OK;
}

RopeParams rope_params(const pkv_rope_spec& r) {
  RopeParams rp{};
  rp.cos_sin = r.cos_sin;
  rp.num_positions = r.num_positions;
  rp.rot_dim = r.rot_dim;
  rp.interleaved = r.interleaved;
  rp.eps = r.eps;
  rp.q_weight = static_cast<const __nv_bfloat16*>(r.q_weight);
  rp.k_weight = static_cast<const __nv_bfloat16*>(r.k_weight);
  return rp;
}

// Host checks of the rotating append (the problem has passed its own).
pkv_status validate_rope_append(const pkv_problem& pr, const pkv_fwd_args* a, const pkv_rope_append_args* r,
                                int32_t total_q, int32_t total_new) {
  pkv_status st = validate_cache_args(pr, a);
  if (st != PKV_OK) return st;
  if (!r) return fail(PKV_ERR_INVALID_ARG, "rope arguments are NULL");
  if (pr.cache_dtype == PKV_FP4_E2M1)
    return fail(PKV_ERR_UNSUPPORTED, "the rotating forms take bf16 and fp8 caches (pkv_qk_norm_rope first for fp4)");
  st = validate_rope_spec(r->spec, pr.head_dim);
  if (st != PKV_OK) return st;
  if (total_q < 0 || total_new < 0) return fail(PKV_ERR_INVALID_ARG, "total_q or total_new < 0");
  if (pr.batch == 0 && (total_q > 0 || total_new > 0)) return fail(PKV_ERR_INVALID_ARG, "tokens given for batch 0");
  if (total_new > 0) {
    st = validate_new_args(pr, a);
    if (st != PKV_OK) return st;
  }
  if (total_q > 0 && r->q_out) {
    if (!a->cu_seqlens_q) return fail(PKV_ERR_INVALID_ARG, "cu_seqlens_q is NULL");
    if (a->q_rows != 0) return fail(PKV_ERR_UNSUPPORTED, "the rotating append takes packed query rows (q_rows = 0)");
    st = validate_rows("q", a->q, a->q_stride_tok, a->q_stride_head, pr.head_dim);
    if (st != PKV_OK) return st;
    st = validate_rows("q_out", r->q_out, r->qo_stride_tok, r->qo_stride_head, pr.head_dim);
    if (st != PKV_OK) return st;
    st = validate_in_place("q_out", a->q, r->q_out, a->q_stride_tok, a->q_stride_head, r->qo_stride_tok,
                           r->qo_stride_head);
    if (st != PKV_OK) return st;
  }
  return PKV_OK;
}

cudaError_t run_rope_append(const pkv_problem& pr, const pkv_fwd_args* a, const pkv_rope_append_args* r,
                            int32_t total_q, int32_t total_new, int* status, cudaStream_t s) {
  RopeParams rp = rope_params(r->spec);
  rp.a = append_params(pr, a, total_new, status);
  rp.cu_q = a->cu_seqlens_q;
  if (total_q > 0 && r->q_out) {
    rp.q = static_cast<const __nv_bfloat16*>(a->q);
    rp.q_stride_tok = a->q_stride_tok;
    rp.q_stride_head = a->q_stride_head;
    rp.q_out = static_cast<__nv_bfloat16*>(r->q_out);
    rp.qo_stride_tok = r->qo_stride_tok;
    rp.qo_stride_head = r->qo_stride_head;
    rp.total_q = total_q;
    rp.hq = pr.num_heads_q;
  }
  if (total_new == 0) rp.a.hkv = 0;
  return launch_rope_kv_append(rp, pr.head_dim, pr.cache_dtype == PKV_FP8_E4M3, s);
}

bool same_problem(const pkv_problem& x, const pkv_problem& y) {
  return x.batch == y.batch && x.num_heads_q == y.num_heads_q && x.num_heads_kv == y.num_heads_kv &&
         x.head_dim == y.head_dim && x.page_size == y.page_size && x.cache_capacity == y.cache_capacity &&
         x.num_pages == y.num_pages && x.cache_dtype == y.cache_dtype && x.causal == y.causal &&
         x.softmax_scale == y.softmax_scale;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" const char* pkv_last_error(void) { return g_err; }

extern "C" const char* pkv_version(void) { return "pkv 0.1.0 (sm_103a)"; }

extern "C" pkv_status pkv_plan_upload(pkv_plan_t plan, void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan || !workspace) return fail(PKV_ERR_INVALID_ARG, "NULL plan or workspace");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return fail(PKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < plan->layout.total)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu required", workspace_bytes, plan->layout.total);
  cudaError_t e = cudaMemcpyAsync(workspace, plan->image, plan->image_bytes, cudaMemcpyHostToDevice,
                                  static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "plan upload");
  return PKV_OK;
}

extern "C" pkv_status pkv_kv_append(const pkv_problem* problem, const pkv_fwd_args* args, int32_t total_new,
                                    int32_t* device_status, void* stream) {
  pkv_status st = validate_problem(problem);
  if (st != PKV_OK) return st;
  st = validate_cache_args(*problem, args);
  if (st != PKV_OK) return st;
  if (total_new < 0) return fail(PKV_ERR_INVALID_ARG, "total_new < 0");
  if (total_new == 0) return PKV_OK;
  st = validate_new_args(*problem, args);
  if (st != PKV_OK) return st;
  AppendParams ap = append_params(*problem, args, total_new, reinterpret_cast<int*>(device_status));
  ap.status_code_only = 1;
  cudaError_t e = run_append(*problem, args, ap, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
  return PKV_OK;
}

extern "C" pkv_status pkv_qk_norm_rope(const pkv_qk_args* args, const pkv_rope_spec* spec, int32_t* device_status,
                                       void* stream) {
  if (!args || !spec) return fail(PKV_ERR_INVALID_ARG, "args or spec is NULL");
  const pkv_qk_args& a = *args;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", a.head_dim);
  pkv_status st = validate_rope_spec(*spec, a.head_dim);
  if (st != PKV_OK) return st;
  if (a.num_tokens < 0 || a.num_heads_q < 0 || a.num_heads_kv < 0)
    return fail(PKV_ERR_INVALID_ARG, "negative token or head count");
  if (a.num_tokens == 0) return PKV_OK;  // (empty tensors may have no address)
  if ((a.num_heads_q > 0) != (a.q != nullptr) || (a.num_heads_kv > 0) != (a.k != nullptr))
    return fail(PKV_ERR_INVALID_ARG, "heads without a tensor, or a tensor without heads");
  if (a.num_heads_q == 0 && a.num_heads_kv == 0) return PKV_OK;
  if (spec->rot_dim > 0 && !a.positions) return fail(PKV_ERR_INVALID_ARG, "positions is NULL");
  if (a.q) {
    st = validate_rows("q", a.q, a.q_stride_tok, a.q_stride_head, a.head_dim);
    if (st == PKV_OK) st = validate_rows("q_out", a.q_out, a.qo_stride_tok, a.qo_stride_head, a.head_dim);
    if (st == PKV_OK)
      st = validate_in_place("q_out", a.q, a.q_out, a.q_stride_tok, a.q_stride_head, a.qo_stride_tok, a.qo_stride_head);
    if (st != PKV_OK) return st;
  }
  if (a.k) {
    st = validate_rows("k", a.k, a.k_stride_tok, a.k_stride_head, a.head_dim);
    if (st == PKV_OK) st = validate_rows("k_out", a.k_out, a.ko_stride_tok, a.ko_stride_head, a.head_dim);
    if (st == PKV_OK)
      st = validate_in_place("k_out", a.k, a.k_out, a.k_stride_tok, a.k_stride_head, a.ko_stride_tok, a.ko_stride_head);
    if (st != PKV_OK) return st;
  }
  RopeParams rp = rope_params(*spec);
  rp.q = static_cast<const __nv_bfloat16*>(a.q);
  rp.q_stride_tok = a.q_stride_tok;
  rp.q_stride_head = a.q_stride_head;
  rp.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  rp.qo_stride_tok = a.qo_stride_tok;
  rp.qo_stride_head = a.qo_stride_head;
  rp.total_q = a.q ? a.num_tokens : 0;
  rp.hq = a.num_heads_q;
  rp.positions = a.positions;
  rp.a.k_new = static_cast<const __nv_bfloat16*>(a.k);
  rp.a.n_stride_tok = a.k_stride_tok;
  rp.a.n_stride_head = a.k_stride_head;
  rp.a.k_cache = a.k_out;
  rp.a.c_stride_tok = a.ko_stride_tok;
  rp.a.c_stride_head = a.ko_stride_head;
  rp.a.total_new = a.k ? a.num_tokens : 0;
  rp.a.hkv = a.num_heads_kv;
  rp.a.status = reinterpret_cast<int*>(device_status);
  cudaError_t e = launch_qk_norm_rope(rp, a.head_dim, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "qk_norm_rope launch");
  return PKV_OK;
}

extern "C" pkv_status pkv_rope_kv_append(const pkv_problem* problem, const pkv_fwd_args* args,
                                         const pkv_rope_append_args* rope, int32_t total_q, int32_t total_new,
                                         int32_t* device_status, void* stream) {
  pkv_status st = validate_problem(problem);
  if (st != PKV_OK) return st;
  st = validate_rope_append(*problem, args, rope, total_q, total_new);
  if (st != PKV_OK) return st;
  cudaError_t e = run_rope_append(*problem, args, rope, total_q, total_new, reinterpret_cast<int*>(device_status),
                                  static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope_kv_append launch");
  return PKV_OK;
}

namespace pkv {

// Every host-side check of an attention call that does not involve the
// workspace: the problem, the plan it must match, the cache, q / out and the
// new-token arguments.  Nothing is launched or copied before these pass.
pkv_status validate_call(const pkv_problem* problem, const pkv_fwd_args* args, pkv_plan_t plan) {
  pkv_status st = validate_problem(problem);
  if (st != PKV_OK) return st;
  if (!plan) return fail(PKV_ERR_INVALID_ARG, "plan is NULL");
  if (!same_problem(*problem, plan->problem)) return fail(PKV_ERR_INVALID_ARG, "problem differs from the plan's");
  st = validate_cache_args(*problem, args);
  if (st != PKV_OK) return st;
  const pkv_problem& pr = *problem;
  if (plan->total_q > 0) {
    if (!args->q || !args->out || !args->cu_seqlens_q) return fail(PKV_ERR_INVALID_ARG, "q, out or cu_seqlens_q NULL");
    if (args->q_stride_head < pr.head_dim || args->o_stride_head < pr.head_dim || args->q_stride_tok <= 0 ||
        args->o_stride_tok <= 0)
      return fail(PKV_ERR_INVALID_ARG, "q / out strides");
    if (!aligned16(args->q) || !aligned16(args->out) || (args->q_stride_head % 8) || (args->q_stride_tok % 8) ||
        (args->o_stride_head % 8) || (args->o_stride_tok % 8))
      return fail(PKV_ERR_INVALID_ARG, "q / out must be 16-byte aligned with strides multiple of 8 elements");
    if (args->max_seqlen_q < 0) return fail(PKV_ERR_INVALID_ARG, "max_seqlen_q < 0");
    if (args->q_rows != 0 && args->q_rows < plan->total_q)
      return fail(PKV_ERR_INVALID_ARG, "q_rows %d < the plan's %d query rows", args->q_rows, plan->total_q);
  }
  if (args->q_rows < 0) return fail(PKV_ERR_INVALID_ARG, "q_rows < 0");
  if (args->q_rows > 0 && plan->shared)
    return fail(PKV_ERR_UNSUPPORTED, "a plan with shared prefixes takes packed query rows (q_rows = 0)");
  const bool has_new = args->k_new != nullptr || args->v_new != nullptr;
  if (plan->total_new > 0 && !has_new)
    return fail(PKV_ERR_INVALID_ARG, "the plan appends %d tokens but k_new / v_new are NULL", plan->total_new);
  if (plan->total_new == 0 && has_new)
    return fail(PKV_ERR_INVALID_ARG, "k_new given but the plan was made with no new tokens");
  if (plan->total_new > 0) {
    st = validate_new_args(pr, args);
    if (st != PKV_OK) return st;
  }
  if (args->q_scale && pr.cache_dtype != PKV_FP8_E4M3)
    return fail(PKV_ERR_UNSUPPORTED, "q_scale (fp8 Q.K^T) needs an fp8 cache");
  return PKV_OK;
}

}  // namespace pkv

namespace pkv {
namespace {

// The attention of a call, over keys that are all in the cache: the persistent kernel
// and, when a unit was split, the combine.  appended, rotated: the append just launched,
// plain or rotating, that the first launch may overlap.
pkv_status run_attention(const pkv_problem& pr, const pkv_fwd_args* args, const pkv_plan_s* plan, unsigned char* ws,
                         int* status, const float* k_scale, const float* v_scale, bool appended, bool rotated,
                         cudaStream_t s) {
  if (plan->num_items == 0) return PKV_OK;
  pkv_status st = PKV_OK;
  const bool fp4 = pr.cache_dtype == PKV_FP4_E2M1;
  CUtensorMap tk, tv, tq;
  if (!fp4) st = make_cache_map(&tk, pr, *args, args->k_cache);
  if (st != PKV_OK) return st;
  if (!fp4) st = make_cache_map(&tv, pr, *args, args->v_cache);
  if (st != PKV_OK) return st;
  memset(&tq, 0, sizeof(tq));
  if (!fp4 && plan->num_prefill_items > 0) {
    st = make_q_map(&tq, pr, *args, args->q_rows ? args->q_rows : plan->total_q);
    if (st != PKV_OK) return st;
  }

  AttnParams p{};
  p.q = static_cast<const __nv_bfloat16*>(args->q);
  p.q_stride_tok = args->q_stride_tok;
  p.q_stride_head = args->q_stride_head;
  p.out = static_cast<__nv_bfloat16*>(args->out);
  p.o_stride_tok = args->o_stride_tok;
  p.o_stride_head = args->o_stride_head;
  p.out_v8 = (reinterpret_cast<uintptr_t>(args->out) % 32 == 0) && (args->o_stride_tok % 16 == 0) &&
             (args->o_stride_head % 16 == 0);
  p.lse = args->lse;
  p.total_q = args->q_rows ? args->q_rows : plan->total_q;
  // rows placed by the caller (q_rows given): offsets read on the device
  p.q_offsets = args->q_rows ? args->cu_seqlens_q : nullptr;
  p.block_table = args->block_table;
  p.bt_stride = args->block_table_stride;
  p.page_indptr = args->page_indptr;
  p.page_size = pr.page_size;
  p.box_rows = cache_box_rows(pr.page_size, pr.cache_capacity, kv_tile_keys(pr.head_dim));
  p.num_pages = pr.num_pages;
  p.G = pr.num_heads_q / pr.num_heads_kv;
  p.causal = pr.causal;
  p.scale_log2 = pr.softmax_scale * 1.4426950408889634f;
  p.k_scale = k_scale;
  p.q_scale = args->q_scale;
  p.v_scale = v_scale;
  p.items = reinterpret_cast<const WorkItem*>(ws + plan->layout.items);
  p.cta_begin = reinterpret_cast<const int32_t*>(ws + plan->layout.cta_begin);
  p.partial_o = reinterpret_cast<float*>(ws + plan->layout.partial_o);
  p.partial_lse = reinterpret_cast<float*>(ws + plan->layout.partial_lse);
  p.status = status;
  p.cache_seqlens = args->cache_seqlens;
  p.plan_lc = reinterpret_cast<const int32_t*>(ws + plan->layout.plan_lc);
  p.batch = pr.batch;
  p.dynamic = plan->dynamic;
  p.row_gather = pr.page_size > 0 && pr.page_size < kBoxRows;
  p.kc = args->k_cache;
  p.vc = args->v_cache;
  p.c_stride_page = args->kc_stride_page;
  p.c_stride_tok = args->kc_stride_tok;
  p.c_stride_head = args->kc_stride_head;
  cudaError_t e;
  if (g_ev_start && (e = record_profile_event(g_ev_start, s)) != cudaSuccess) return cuda_fail(e, "profile event");
  // Decode-only plans overlap the attention kernel's start with the (small)
  // append kernel and the combine kernel's start with the attention's end.
  // Plans with prefill tiles keep the kernels strictly in order: there the
  // overlap measured slower (large appends, long attention kernels).  Never
  // across a profiling event, which must see the kernels in order.
  const bool overlap = plan->num_prefill_items == 0;
  const bool fp8 = pr.cache_dtype == PKV_FP8_E4M3;
  const bool append_overlaps = appended && !rotated && !g_ev_start;
  // After the rotating append, whose queries it reads from its start, the
  // attention starts while that kernel drains and waits for it before it reads
  // anything (where the first launch is of decode tiles alone).  Without an
  // append it is the call's first kernel, an ordinary launch: a kernel before the
  // call that was itself started early, and does not wait, would hide what came
  // before it.
  const bool first_pf = plan->num_ctas_tc > 0 ? !plan->dec_first : plan->num_prefill_items > 0;
  const bool first = rotated && !g_ev_start && !first_pf;
  p.dep_first = first;
  if (fp4) {
    e = launch_fp4_attention(p, fp4_scales(args), plan->num_items, plan->max_rows, pr.cache_capacity,
                             pr.head_dim, s);
  } else if (plan->num_ctas_tc > 0) {
    // A plan with shared prefixes and both kinds of tiles: the tensor-core tiles
    // on num_ctas_tc SMs and the decode tiles on the others, each in the
    // instance made for them, the second launch overlapping the first and ending
    // only after it.
    AttnParams pd = p;
    pd.cta_begin += plan->num_ctas_tc;
    const int dec_ctas = plan->num_ctas - plan->num_ctas_tc;
    if (plan->dec_first) {
      // the tensor-core tiles are all over prefixes, which no append writes
      e = launch_attention(pd, tk, tv, tq, dec_ctas, pr.head_dim, fp8, false, true, append_overlaps || first, s);
      p.dep_first = 0;
      p.dep_late = 1;
      if (e == cudaSuccess)
        e = launch_attention(p, tk, tv, tq, plan->num_ctas_tc, pr.head_dim, fp8, true, false, true, s);
    } else {
      // the append is complete before the first launch starts
      e = launch_attention(p, tk, tv, tq, plan->num_ctas_tc, pr.head_dim, fp8, true, false, false, s);
      pd.dep_late = 1;
      if (e == cudaSuccess)
        e = launch_attention(pd, tk, tv, tq, dec_ctas, pr.head_dim, fp8, false, true, true, s);
    }
  } else {
    e = launch_attention(p, tk, tv, tq, plan->num_ctas, pr.head_dim, fp8, plan->num_prefill_items > 0,
                         plan->num_decode_items > 0, (overlap && append_overlaps) || first, s);
  }
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  if (g_ev_stop && (e = record_profile_event(g_ev_stop, s)) != cudaSuccess) return cuda_fail(e, "profile event");

  if (plan->num_combine > 0) {
    CombineParams cp{};
    cp.items = reinterpret_cast<const CombineItem*>(ws + plan->layout.combine);
    cp.q_offsets = p.q_offsets;
    cp.partial_o = p.partial_o;
    cp.partial_lse = p.partial_lse;
    cp.out = p.out;
    cp.o_stride_tok = p.o_stride_tok;
    cp.o_stride_head = p.o_stride_head;
    cp.lse = p.lse;
    cp.total_q = p.total_q;
    cp.G = p.G;
    e = plan->row_combine
            ? launch_combine_shared(cp, plan->num_combine, plan->max_combine_rows, plan->max_combine_parts, pr.head_dim,
                                    overlap && !g_ev_stop, s)
            : launch_combine(cp, plan->num_combine, pr.head_dim, overlap && !g_ev_stop, s);
    if (e != cudaSuccess) return cuda_fail(e, "combine launch");
  }
  return PKV_OK;
}

// The sequences of a 4-bit plan whose queries fill tensor-core tiles: their keys as
// bf16, to meet the queries, and their values as f16, to meet P (both exact: code x
// block scale has six significant bits; the tensor scales go into the logits' scale
// and the output), into the workspace, then the attention over those.
pkv_status run_far(const pkv_problem& pr, const pkv_fwd_args* args, pkv_plan_t plan, unsigned char* ws, cudaStream_t s) {
  const FarLayout& F = plan->far_layout;
  const pkv_plan_s* far = plan->far;
  auto ints = [&](size_t at) { return reinterpret_cast<const int32_t*>(ws + at); };
  int* status = reinterpret_cast<int*>(ws + plan->layout.status);
  pkv_fwd_args a = *args;
  a.k_cache = ws + F.k;
  a.v_cache = ws + F.v;
  a.kc_stride_head = pr.head_dim;
  a.kc_stride_tok = (int64_t)pr.num_heads_kv * pr.head_dim;
  a.kc_stride_page = a.kc_stride_tok * kFarPage;
  GatherParams g{};
  g.k_out = static_cast<__nv_bfloat16*>(a.k_cache);
  g.v_out = static_cast<__nv_bfloat16*>(a.v_cache);
  g.o_stride_tok = a.kc_stride_tok;
  g.o_stride_head = a.kc_stride_head;
  g.cu_rows = ints(F.rows);
  g.lens = ints(F.lens);
  g.cache_seqlens = args->cache_seqlens;
  g.plan_lc = ints(plan->layout.plan_lc);
  g.block_table = args->block_table;
  g.bt_stride = args->block_table_stride;
  g.page_indptr = args->page_indptr;
  g.page_size = pr.page_size;
  g.num_pages = pr.num_pages;
  g.capacity = pr.cache_capacity;
  g.batch = pr.batch;
  g.hkv = pr.num_heads_kv;
  g.head_dim = pr.head_dim;
  g.total_rows = F.pages * kFarPage;
  g.k_cache = args->k_cache;
  g.v_cache = args->v_cache;
  g.c_stride_page = args->kc_stride_page;
  g.c_stride_tok = args->kc_stride_tok;
  g.c_stride_head = args->kc_stride_head;
  g.sf = fp4_scales(args);
  g.k_scale = args->k_scale;
  g.status = status;
  // (where no launch before has been timed, the copies are the first that is)
  cudaError_t e;
  if (g_ev_start && (e = record_profile_event(g_ev_start, s)) != cudaSuccess) return cuda_fail(e, "profile event");
  g_ev_start = nullptr;
  e = launch_gather(g, pr.cache_dtype, s);
  if (e != cudaSuccess) return cuda_fail(e, "kv_gather launch");

  // rows where cu_seqlens_q says: the other sequences' lie between these
  a.q_rows = args->q_rows ? args->q_rows : plan->total_q;
  a.cache_seqlens = ints(F.lens);
  a.page_indptr = ints(F.indptr);
  a.block_table = ints(F.table);
  return run_attention(far->problem, &a, far, ws + F.plan, status, args->k_scale, args->v_scale, false, false, s);
}

// The profiling events of a call with two attention launches: no stop after the first, one
// start, before the first that has items (the copies belong to the second); put back at the end.
struct ProfileEvents {
  cudaEvent_t start = g_ev_start, stop = g_ev_stop;
  bool first;
  ProfileEvents(bool has_first, bool two) : first(has_first) {
    if (two) g_ev_stop = nullptr;
  }
  void second() const {
    g_ev_stop = stop;
    if (first) g_ev_start = nullptr;
  }
  ~ProfileEvents() { g_ev_start = start, g_ev_stop = stop; }
};

// The whole call: append (with a rotation, if `rope` is given), attention, combine.
pkv_status run_call(const pkv_problem* problem, const pkv_fwd_args* args, const pkv_rope_append_args* rope,
                    pkv_plan_t plan, void* workspace, size_t workspace_bytes, void* stream) {
  pkv_status st = validate_call(problem, args, plan);
  if (st != PKV_OK) return st;
  pkv_fwd_args rotated;
  if (rope) {
    st = validate_rope_append(*problem, args, rope, plan->total_q, plan->total_new);
    if (st != PKV_OK) return st;
    if (plan->total_q > 0 && !rope->q_out) return fail(PKV_ERR_INVALID_ARG, "q_out is NULL");
  }
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return fail(PKV_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < plan->layout.total)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu required", workspace_bytes, plan->layout.total);
  const pkv_problem& pr = *problem;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  int* status = reinterpret_cast<int*>(ws + plan->layout.status);

  if (rope) {
    cudaError_t e = run_rope_append(pr, args, rope, plan->total_q, plan->total_new, status, s);
    if (e != cudaSuccess) return cuda_fail(e, "rope_kv_append launch");
    // the attention reads the transformed queries
    rotated = *args;
    rotated.q = rope->q_out;
    rotated.q_stride_tok = rope->qo_stride_tok;
    rotated.q_stride_head = rope->qo_stride_head;
    args = &rotated;
  } else if (plan->total_new > 0) {
    AppendParams ap = append_params(pr, args, plan->total_new, status);
    cudaError_t e = run_append(pr, args, ap, s);
    if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
  }
  const bool scaled = pr.cache_dtype != PKV_BF16;
  // (a call with a second attention launch: the profiling events go around both)
  const ProfileEvents events(plan->far && plan->num_items > 0, plan->far != nullptr);
  st = run_attention(pr, args, plan, ws, status, scaled ? args->k_scale : nullptr, scaled ? args->v_scale : nullptr,
                     plan->total_new > 0 && !rope, rope != nullptr, s);
  if (st != PKV_OK || !plan->far) return st;
  events.second();
  return run_far(pr, args, plan, ws, s);
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_attn_varlen_kvcache_fwd(const pkv_problem* problem, const pkv_fwd_args* args,
                                                  pkv_plan_t plan, void* workspace, size_t workspace_bytes,
                                                  void* stream) {
  return run_call(problem, args, nullptr, plan, workspace, workspace_bytes, stream);
}

extern "C" pkv_status pkv_rope_attn_varlen_kvcache_fwd(const pkv_problem* problem, const pkv_fwd_args* args,
                                                       const pkv_rope_append_args* rope, pkv_plan_t plan,
                                                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!rope) return fail(PKV_ERR_INVALID_ARG, "rope arguments are NULL");
  return run_call(problem, args, rope, plan, workspace, workspace_bytes, stream);
}

extern "C" pkv_status pkv_set_profile_events(void* start_event, void* stop_event) {
  if ((start_event == nullptr) != (stop_event == nullptr))
    return fail(PKV_ERR_INVALID_ARG, "give both events or neither");
  g_ev_start = static_cast<cudaEvent_t>(start_event);
  g_ev_stop = static_cast<cudaEvent_t>(stop_event);
  return PKV_OK;
}

extern "C" pkv_status pkv_get_status(void* workspace, void* stream, int32_t* device_status) {
  if (!workspace || !device_status) return fail(PKV_ERR_INVALID_ARG, "NULL workspace or output");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t h[4] = {0, 0, 0, 0};
  cudaError_t e = cudaMemcpyAsync(h, workspace, sizeof(h), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  *device_status = h[0];
  if (h[0] != 0) {
    fail((pkv_status)h[0], "device status %d (info %d, %d)", h[0], h[1], h[2]);
    e = cudaMemsetAsync(workspace, 0, sizeof(h), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "status reset");
  }
  return PKV_OK;
}

extern "C" pkv_status pkv_kv_gather(const pkv_problem* problem, const pkv_fwd_args* args,
                                    const pkv_gather_args* gather, int32_t total_rows, int32_t* device_status,
                                    void* stream) {
  pkv_status st = validate_problem(problem);
  if (st != PKV_OK) return st;
  const pkv_problem& pr = *problem;
  st = validate_cache_args(pr, args);
  if (st != PKV_OK) return st;
  if (!gather) return fail(PKV_ERR_INVALID_ARG, "gather arguments are NULL");
  if (total_rows < 0) return fail(PKV_ERR_INVALID_ARG, "total_rows < 0");
  if (total_rows == 0) return PKV_OK;
  if (pr.batch == 0) return fail(PKV_ERR_INVALID_ARG, "rows given for batch 0");
  if (!gather->cu_rows) return fail(PKV_ERR_INVALID_ARG, "cu_rows is NULL");
  if (!gather->k_out && !gather->v_out) return fail(PKV_ERR_INVALID_ARG, "k_out and v_out are NULL");
  for (const void* o : {gather->k_out, gather->v_out}) {
    if (!o) continue;
    st = validate_rows("k_out / v_out", o, gather->out_stride_tok, gather->out_stride_head, pr.head_dim);
    if (st != PKV_OK) return st;
  }
  GatherParams g{};
  g.k_out = static_cast<__nv_bfloat16*>(gather->k_out);
  g.v_out = static_cast<__nv_bfloat16*>(gather->v_out);
  g.o_stride_tok = gather->out_stride_tok;
  g.o_stride_head = gather->out_stride_head;
  g.cu_rows = gather->cu_rows;
  g.starts = gather->starts;
  g.block_table = args->block_table;
  g.bt_stride = args->block_table_stride;
  g.page_indptr = args->page_indptr;
  g.page_size = pr.page_size;
  g.num_pages = pr.num_pages;
  g.capacity = pr.cache_capacity;
  g.batch = pr.batch;
  g.hkv = pr.num_heads_kv;
  g.head_dim = pr.head_dim;
  g.total_rows = total_rows;
  g.k_cache = args->k_cache;
  g.v_cache = args->v_cache;
  g.c_stride_page = args->kc_stride_page;
  g.c_stride_tok = args->kc_stride_tok;
  g.c_stride_head = args->kc_stride_head;
  g.sf = fp4_scales(args);
  if (pr.cache_dtype != PKV_BF16) {
    g.k_scale = args->k_scale;
    g.v_scale = args->v_scale;
  }
  g.status = reinterpret_cast<int*>(device_status);
  cudaError_t e = launch_gather(g, pr.cache_dtype, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_gather launch");
  return PKV_OK;
}

namespace pkv {
namespace {

// Scores that are written, `keys` of each (sequence, kv head): no two of them may share an address.
pkv_status validate_scores(const pkv_problem& pr, int64_t stride_seq, int64_t stride_head, int32_t keys) {
  const int64_t B = pr.batch, H = pr.num_heads_kv;
  // rows of `n` at `inner`, and such groups at `outer` behind one another
  auto apart = [&](int64_t inner, int64_t n, int64_t outer, int64_t m) {
    return (n <= 1 || inner >= keys) && (m <= 1 || (outer >= keys && (n <= 1 || (outer - keys) / (n - 1) >= inner)));
  };
  if (!apart(stride_head, H, stride_seq, B) && !apart(stride_seq, B, stride_head, H))
    return fail(PKV_ERR_INVALID_ARG, "scores: stride_seq and stride_head: rows of %d keys overlap", keys);
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_attn_weights(const pkv_problem* problem, const pkv_fwd_args* args,
                                       const pkv_weights_args* weights, int32_t* device_status, void* stream) {
  pkv_status st = validate_problem(problem);
  if (st != PKV_OK) return st;
  const pkv_problem& pr = *problem;
  st = validate_cache_args(pr, args);
  if (st != PKV_OK) return st;
  if (!weights) return fail(PKV_ERR_INVALID_ARG, "weights arguments are NULL");
  const pkv_weights_args& w = *weights;
  if (w.max_seqlen_k < 0 || w.max_seqlen_k > pr.cache_capacity)
    return fail(PKV_ERR_INVALID_ARG, "max_seqlen_k %d: 0 to cache_capacity", w.max_seqlen_k);
  const int32_t most = w.max_seqlen_k > 0 ? w.max_seqlen_k : pr.cache_capacity;
  if (most > kMaxSeqlen) return fail(PKV_ERR_UNSUPPORTED, "max_seqlen_k %d > %d", most, kMaxSeqlen);
  if (w.last_queries < 0 || args->max_seqlen_q < 0 || w.max_total_q < 0)
    return fail(PKV_ERR_INVALID_ARG, "last_queries, max_seqlen_q or max_total_q < 0");
  if (args->q_rows != 0) return fail(PKV_ERR_UNSUPPORTED, "attn_weights takes packed query rows (q_rows = 0)");
  if (args->q_scale) return fail(PKV_ERR_UNSUPPORTED, "attn_weights takes no quantised queries (q_scale)");
  if (pr.batch > kMaxGridDim || pr.num_heads_kv > kMaxGridDim)
    return fail(PKV_ERR_UNSUPPORTED, "attn_weights takes at most %d sequences and kv heads", kMaxGridDim);
  if (pr.batch == 0) return PKV_OK;
  if (!w.scores || !args->lse || !args->cu_seqlens_q)
    return fail(PKV_ERR_INVALID_ARG, "scores, lse or cu_seqlens_q is NULL");
  if ((args->k_new != nullptr) && !args->cu_seqlens_knew)
    return fail(PKV_ERR_INVALID_ARG, "k_new is given without cu_seqlens_knew");
  if (w.stride_head < most || w.stride_seq <= 0)
    return fail(PKV_ERR_INVALID_ARG, "scores: stride_head must hold max_seqlen_k (%d) keys", most);
  st = validate_scores(pr, w.stride_seq, w.stride_head, most);
  if (st != PKV_OK) return st;
  st = validate_rows("q", args->q, args->q_stride_tok, args->q_stride_head, pr.head_dim);
  if (st != PKV_OK) return st;
  if (args->max_seqlen_q > INT32_MAX / (pr.num_heads_q / pr.num_heads_kv) - 8)
    return fail(PKV_ERR_UNSUPPORTED, "max_seqlen_q x heads of a group too large");
  WeightsParams p{};
  p.q = static_cast<const __nv_bfloat16*>(args->q);
  p.q_stride_tok = args->q_stride_tok;
  p.q_stride_head = args->q_stride_head;
  p.lse = args->lse;
  p.cu_q = args->cu_seqlens_q;
  p.cu_knew = args->k_new ? args->cu_seqlens_knew : nullptr;
  p.cache_seqlens = args->cache_seqlens;
  p.block_table = args->block_table;
  p.bt_stride = args->block_table_stride;
  p.page_indptr = args->page_indptr;
  p.page_size = pr.page_size;
  p.num_pages = pr.num_pages;
  p.batch = pr.batch;
  p.hkv = pr.num_heads_kv;
  p.G = pr.num_heads_q / pr.num_heads_kv;
  p.k_cache = args->k_cache;
  const int es = pr.cache_dtype == PKV_BF16 ? 2 : 1;
  p.c_stride_page = args->kc_stride_page * es;  // bytes from here on
  p.c_stride_tok = args->kc_stride_tok * es;
  p.c_stride_head = args->kc_stride_head * es;
  p.sf = fp4_scales(args);
  if (pr.cache_dtype != PKV_BF16) p.k_scale = args->k_scale;
  p.scores = w.scores;
  p.scores_in = w.scores_in;
  p.s_stride_seq = w.stride_seq;
  p.s_stride_head = w.stride_head;
  p.last_queries = w.last_queries;
  p.max_seqlen_k = most;
  p.max_seqlen_q = args->max_seqlen_q;
  p.max_total_q = w.max_total_q;
  p.causal = pr.causal;
  p.scale_log2 = pr.softmax_scale * 1.4426950408889634f;
  p.status = reinterpret_cast<int*>(device_status);
  cudaError_t e = launch_weights(p, pr.head_dim, pr.cache_dtype, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "attn_weights launch");
  return PKV_OK;
}

namespace pkv {
namespace {

// Host checks of an eviction's own arguments, and the sections of its workspace.
struct EvictLayout {
  size_t info, list, total;
};

pkv_status evict_layout(const pkv_problem* problem, const pkv_evict_args* e, EvictLayout* L) {
  pkv_status st = validate_problem(problem);
  if (st != PKV_OK) return st;
  const pkv_problem& pr = *problem;
  if (!e) return fail(PKV_ERR_INVALID_ARG, "evict arguments are NULL");
  if (e->max_seqlen_k < 0 || e->max_seqlen_k > pr.cache_capacity || e->max_keep < 0 || e->max_keep > e->max_seqlen_k)
    return fail(PKV_ERR_INVALID_ARG, "max_seqlen_k %d: 0 to cache_capacity; max_keep %d: 0 to max_seqlen_k",
                e->max_seqlen_k, e->max_keep);
  if (e->max_seqlen_k > kMaxSeqlen || e->max_keep > kMaxKeep)
    return fail(PKV_ERR_UNSUPPORTED, "max_seqlen_k %d > %d or max_keep %d > %d", e->max_seqlen_k, kMaxSeqlen,
                e->max_keep, kMaxKeep);
  if (e->sinks < 0 || e->recent < 0) return fail(PKV_ERR_INVALID_ARG, "sinks or recent < 0");
  if (pr.batch > kMaxGridDim || pr.num_heads_kv > kMaxGridDim)
    return fail(PKV_ERR_UNSUPPORTED, "kv_evict takes at most %d sequences and kv heads", kMaxGridDim);
  const size_t heads = (size_t)pr.batch * pr.num_heads_kv;
  L->info = 0;
  L->list = (heads * sizeof(int2) + 255) / 256 * 256;
  L->total = L->list + (e->kept ? 0 : heads * (size_t)e->max_keep * sizeof(int32_t));
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_kv_evict_workspace(const pkv_problem* problem, const pkv_evict_args* evict, size_t* bytes) {
  if (!bytes) return fail(PKV_ERR_INVALID_ARG, "bytes is NULL");
  EvictLayout L{};
  pkv_status st = evict_layout(problem, evict, &L);
  if (st != PKV_OK) return st;
  *bytes = L.total;
  return PKV_OK;
}

extern "C" pkv_status pkv_kv_evict(const pkv_problem* problem, const pkv_fwd_args* args, const pkv_evict_args* evict,
                                   void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream) {
  EvictLayout L{};
  pkv_status st = evict_layout(problem, evict, &L);
  if (st != PKV_OK) return st;
  const pkv_problem& pr = *problem;
  const pkv_evict_args& v = *evict;
  st = validate_cache_args(pr, args);
  if (st != PKV_OK) return st;
  if (pr.batch == 0) return PKV_OK;
  if (!v.scores || !v.keep || !v.new_seqlens) return fail(PKV_ERR_INVALID_ARG, "scores, keep or new_seqlens is NULL");
  if (v.stride_head < v.max_seqlen_k || v.stride_seq < 0)
    return fail(PKV_ERR_INVALID_ARG, "scores: stride_head must hold max_seqlen_k (%d) keys", v.max_seqlen_k);
  if (v.scores_out) {
    st = validate_scores(pr, v.stride_seq, v.stride_head, v.max_seqlen_k);
    if (st != PKV_OK) return st;
  }
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return fail(PKV_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < L.total)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu required", workspace_bytes, L.total);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const int es = pr.cache_dtype == PKV_BF16 ? 2 : 1;
  EvictParams p{};
  p.scores = v.scores;
  p.scores_out = v.scores_out;
  p.s_stride_seq = v.stride_seq;
  p.s_stride_head = v.stride_head;
  p.keep = v.keep;
  p.cache_seqlens = args->cache_seqlens;
  p.new_seqlens = v.new_seqlens;
  p.list = v.kept ? v.kept : reinterpret_cast<int32_t*>(ws + L.list);
  p.info = reinterpret_cast<int2*>(ws + L.info);
  p.fill = v.kept != nullptr;
  p.sinks = v.sinks;
  p.recent = v.recent;
  p.max_seqlen_k = v.max_seqlen_k;
  p.max_keep = v.max_keep;
  p.block_table = args->block_table;
  p.bt_stride = args->block_table_stride;
  p.page_indptr = args->page_indptr;
  p.page_size = pr.page_size;
  p.num_pages = pr.num_pages;
  p.capacity = pr.cache_capacity;
  p.batch = pr.batch;
  p.hkv = pr.num_heads_kv;
  p.k_cache = args->k_cache;
  p.v_cache = args->v_cache;
  p.c_stride_page = args->kc_stride_page * es;  // bytes from here on
  p.c_stride_tok = args->kc_stride_tok * es;
  p.c_stride_head = args->kc_stride_head * es;
  p.sf = fp4_scales(args);
  p.status = reinterpret_cast<int*>(device_status);
  cudaError_t e = launch_evict(p, pr.head_dim, pr.cache_dtype, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_evict launch");
  return PKV_OK;
}
