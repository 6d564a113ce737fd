// KV append scatter and split-KV combine kernels.
//
// Append: flash-attention PR "Add flash_attn_varlen_func_with_kvcache", Usage
// ("kv cache will be updated in-place"; new k/v packed with cu_seqlens_k) and
// Minor Changes (cache lengths kept apart from cu_seqlens_knew);
// TransformerEngine PR "Add KV cache for paged/non-paged attention" (paged and
// non-paged bshd caches, one page table for K and V); vLLM PR "[Kernel][Triton]
// [FP8] ..." (8-bit KV cache).
//
// Combine: merge of the normalised partial outputs of KV chunks of one decode
// unit by their log-sum-exp (the split-KV decode named in the flash-attention
// PR's Limitation and review).
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace pkv {

constexpr int kCombineThreads = 256;

// One warp per (new token, kv head) row; lane l moves elements [l*E, l*E+E).
template <int D, bool FP8>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams p) {
  constexpr int E = D / 32;  // elements per lane: 8 (D=256), 4 (D=128) or 2 (D=64)
  grid_dep_launch();         // the attention kernel may start; it waits before reading appended rows
  const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= (int64_t)p.total_new * p.hkv) return;
  const int t = (int)(row / p.hkv);
  const int h = (int)(row % p.hkv);
  // sequence of token t: the largest b with cu_knew[b] <= t
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_knew + mid) <= t) lo = mid; else hi = mid;
  }
  const int b = lo;
  auto report = [&](int at) {
    if (p.status_code_only) record_code(p.status, PKV_ERR_DEVICE_BOUNDS);
    else record_status(p.status, PKV_ERR_DEVICE_BOUNDS, b, at);
  };
  const int pos = __ldg(p.cache_seqlens + b) + (t - __ldg(p.cu_knew + b));
  if (pos < 0 || pos >= p.capacity) {
    if (lane == 0) report(pos);
    return;
  }
  int64_t dst;
  if (p.page_size > 0) {
    int npages;
    const int32_t* pages = seq_pages(p.block_table, p.bt_stride, p.page_indptr, b, &npages);
    const int pi = pos / p.page_size;
    const int page = (npages >= 0 && pi >= npages) ? -1 : __ldg(pages + pi);
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) report(page);
      return;
    }
    dst = (int64_t)page * p.c_stride_page + (int64_t)(pos % p.page_size) * p.c_stride_tok;
  } else {
    dst = (int64_t)b * p.c_stride_page + (int64_t)pos * p.c_stride_tok;
  }
  dst += (int64_t)h * p.c_stride_head + lane * E;
  const int64_t src = (int64_t)t * p.n_stride_tok + (int64_t)h * p.n_stride_head + lane * E;
  const __nv_bfloat16* kin = p.k_new + src;
  const __nv_bfloat16* vin = p.v_new + src;
  if constexpr (!FP8) {
    __nv_bfloat16* kc = reinterpret_cast<__nv_bfloat16*>(p.k_cache) + dst;
    __nv_bfloat16* vc = reinterpret_cast<__nv_bfloat16*>(p.v_cache) + dst;
    if constexpr (E == 8) {
      *reinterpret_cast<uint4*>(kc) = __ldg(reinterpret_cast<const uint4*>(kin));
      *reinterpret_cast<uint4*>(vc) = __ldg(reinterpret_cast<const uint4*>(vin));
    } else if constexpr (E == 4) {
      *reinterpret_cast<uint2*>(kc) = __ldg(reinterpret_cast<const uint2*>(kin));
      *reinterpret_cast<uint2*>(vc) = __ldg(reinterpret_cast<const uint2*>(vin));
    } else {
      *reinterpret_cast<uint32_t*>(kc) = __ldg(reinterpret_cast<const uint32_t*>(kin));
      *reinterpret_cast<uint32_t*>(vc) = __ldg(reinterpret_cast<const uint32_t*>(vin));
    }
  } else {
    // one IEEE reciprocal per call, then an RN multiply per element (no FMA)
    const float inv_k = __frcp_rn(__ldg(p.k_scale));
    const float inv_v = __frcp_rn(__ldg(p.v_scale));
    auto lo_f = [](uint32_t w) { return __uint_as_float(w << 16); };
    auto hi_f = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
    auto enc2 = [&](uint32_t w, float inv) -> uint32_t {
      return f32x2_to_e4m3x2(__fmul_rn(lo_f(w), inv), __fmul_rn(hi_f(w), inv));
    };
    uint8_t* kc = reinterpret_cast<uint8_t*>(p.k_cache) + dst;
    uint8_t* vc = reinterpret_cast<uint8_t*>(p.v_cache) + dst;
    if constexpr (E == 8) {
      const uint4 kr = __ldg(reinterpret_cast<const uint4*>(kin));
      const uint4 vr = __ldg(reinterpret_cast<const uint4*>(vin));
      *reinterpret_cast<uint2*>(kc) = make_uint2(enc2(kr.x, inv_k) | (enc2(kr.y, inv_k) << 16),
                                                 enc2(kr.z, inv_k) | (enc2(kr.w, inv_k) << 16));
      *reinterpret_cast<uint2*>(vc) = make_uint2(enc2(vr.x, inv_v) | (enc2(vr.y, inv_v) << 16),
                                                 enc2(vr.z, inv_v) | (enc2(vr.w, inv_v) << 16));
    } else if constexpr (E == 4) {
      const uint2 kr = __ldg(reinterpret_cast<const uint2*>(kin));
      const uint2 vr = __ldg(reinterpret_cast<const uint2*>(vin));
      *reinterpret_cast<uint32_t*>(kc) = enc2(kr.x, inv_k) | (enc2(kr.y, inv_k) << 16);
      *reinterpret_cast<uint32_t*>(vc) = enc2(vr.x, inv_v) | (enc2(vr.y, inv_v) << 16);
    } else {
      // D = 64: two elements a lane, one 2-byte store each
      *reinterpret_cast<uint16_t*>(kc) = (uint16_t)enc2(__ldg(reinterpret_cast<const uint32_t*>(kin)), inv_k);
      *reinterpret_cast<uint16_t*>(vc) = (uint16_t)enc2(__ldg(reinterpret_cast<const uint32_t*>(vin)), inv_v);
    }
  }
}

// One block per split unit; a thread owns 8 consecutive columns of a row and
// walks the unit's rows (up to 128: a tensor-core tile of a wide head group).
// Partials are normalised outputs with log2-domain LSEs; chunk s of the unit
// wrote slot0 + s * slot_stride; the merge order over chunks is fixed
// (deterministic).
template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineParams p) {
  const CombineItem ci = p.items[blockIdx.x];
  constexpr int kPerRow = D / 8;
  const int d0 = (threadIdx.x % kPerRow) * 8;
  const int rows = ci.n_q * ci.nh;
  grid_dep_wait();  // the partials come from the attention kernel launched just before
  constexpr float kLn2 = 0.693147180559945309f;
  const int64_t chunk_rows = (int64_t)ci.slot_stride * kDecodeRows;
  for (int row = threadIdx.x / kPerRow; row < rows; row += kCombineThreads / kPerRow) {
    const float* lse = p.partial_lse + (int64_t)ci.slot0 * kDecodeRows + row;
    float m = -INFINITY;
    for (int s = 0; s < ci.nsplit; ++s) m = fmaxf(m, __ldg(lse + s * chunk_rows));
    const float m_use = m == -INFINITY ? 0.f : m;
    float wsum = 0.f;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const float* po = p.partial_o + ((int64_t)ci.slot0 * kDecodeRows + row) * D + d0;
    for (int s = 0; s < ci.nsplit; ++s) {
      const float w = ex2(__ldg(lse + s * chunk_rows) - m_use);
      const float4 a = __ldg(reinterpret_cast<const float4*>(po + s * chunk_rows * D));
      const float4 b = __ldg(reinterpret_cast<const float4*>(po + s * chunk_rows * D + 4));
      wsum += w;
      acc[0] += w * a.x; acc[1] += w * a.y; acc[2] += w * a.z; acc[3] += w * a.w;
      acc[4] += w * b.x; acc[5] += w * b.y; acc[6] += w * b.z; acc[7] += w * b.w;
    }
    const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
    const int tok = (p.q_offsets != nullptr ? __ldg(p.q_offsets + ci.b) + ci.q_i0 : ci.q_row0) + row / ci.nh;
    const int head = ci.hk * p.G + ci.h0 + row % ci.nh;
    uint4 v;
    v.x = pack_bf16(acc[0] * inv, acc[1] * inv);
    v.y = pack_bf16(acc[2] * inv, acc[3] * inv);
    v.z = pack_bf16(acc[4] * inv, acc[5] * inv);
    v.w = pack_bf16(acc[6] * inv, acc[7] * inv);
    *reinterpret_cast<uint4*>(p.out + (int64_t)tok * p.o_stride_tok + (int64_t)head * p.o_stride_head + d0) = v;
    if (p.lse != nullptr && d0 == 0)
      p.lse[(int64_t)head * p.total_q + tok] = wsum > 0.f ? (m_use + __log2f(wsum)) * kLn2 : -INFINITY;
  }
}

// The merge for plans of pkv_plan_shared_prefix: a unit's rows may have parts over
// the chunks of a prefix, in the tiles of the sequences that share it, besides
// the parts over the sequence's own keys.  One warp per row: each lane takes the LSE of
// one part (the common max and the weights come from the warp's lanes), then
// D / 32 columns of every part's row.  Parts are added in a fixed order, the
// prefix's first.  Latency alone bounds it (2048 rows of two parts: 4% of the
// DRAM bandwidth): a warp a row keeps the chain at item, parts, output (a block
// a unit, its rows one after another, took 24 us on 3072 rows of a wide group).
constexpr int kSharedCombineWarps = 4;

// SPLIT: a block takes one row, its warps every fourth part each (rows of many
// parts, which are few; their sums are joined in a fixed order); else a warp a
// row.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(32 * kSharedCombineWarps) combine_shared_kernel(const CombineParams p) {
  constexpr int E = D / 32;  // columns of a lane: 8, 4 or 2
  constexpr int W = SPLIT ? kSharedCombineWarps : 1;
  constexpr float kLn2 = 0.693147180559945309f;
  const CombineItem ci = p.items[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = ci.n_q * ci.nh, parts = ci.p_nsplit + ci.nsplit;
  grid_dep_wait();  // the partials come from the attention kernel launched just before
  const int row = SPLIT ? (int)blockIdx.y : blockIdx.y * kSharedCombineWarps + warp;
  if (row >= rows) return;  // (SPLIT: the whole block)
  const int w0 = SPLIT ? warp : 0;  // this warp's parts: w0, w0 + W, ...
  // partial row of part 0 of each kind, and the rows between its parts
  const int tok = row / ci.nh, g = row - tok * ci.nh;
  const int pt = ci.p_tok0 + tok;
  const int64_t prow = ci.p_nsplit == 0
                           ? 0
                           : ((int64_t)ci.p_slot0 + (int64_t)(pt / ci.p_tq) * ci.p_tile_slots) * kDecodeRows +
                                 (pt % ci.p_tq) * ci.nh + g;
  const int64_t orow = (int64_t)ci.slot0 * kDecodeRows + row;
  auto part_row = [&](int s) {
    return s < ci.p_nsplit ? prow + (int64_t)s * ci.p_chunk_slots * kDecodeRows
                           : orow + (int64_t)(s - ci.p_nsplit) * ci.slot_stride * kDecodeRows;
  };
  auto load = [&](int s, float* v) {
    const float* src = p.partial_o + part_row(s) * D + lane * E;
    if constexpr (E == 2) {
      const float2 x = *reinterpret_cast<const float2*>(src);
      v[0] = x.x, v[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(src + i);
        v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
      }
    }
  };
  // the first parts' rows are in flight while the weights are made
  constexpr int kAhead = 4;
  float ahead[kAhead][E];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (w0 + k * W < parts) load(w0 + k * W, ahead[k]);
  float m = -INFINITY;
  for (int s = lane; s < parts; s += 32) m = fmaxf(m, p.partial_lse[part_row(s)]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float mu = m == -INFINITY ? 0.f : m;
  float wsum = 0.f;
  float acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = 0.f;
  for (int s0 = 0; s0 < parts; s0 += 32) {
    const int n = min(32, parts - s0);
    const float w = lane < n ? ex2(p.partial_lse[part_row(s0 + lane)] - mu) : 0.f;
    wsum += w;
    int s = w0;
    if (s0 == 0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k, s += W) {
        const float ws = __shfl_sync(0xffffffffu, w, s & 31);
        if (s < n) {
#pragma unroll
          for (int i = 0; i < E; ++i) acc[i] = fmaf(ws, ahead[k][i], acc[i]);
        }
      }
    }
#pragma unroll 4
    for (; s < n; s += W) {
      const float ws = __shfl_sync(0xffffffffu, w, s);
      float v[E];
      load(s0 + s, v);
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] = fmaf(ws, v[i], acc[i]);
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
  if constexpr (SPLIT) {
    __shared__ float sums[W][D];
#pragma unroll
    for (int i = 0; i < E; ++i) sums[warp][lane * E + i] = acc[i];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int k = 1; k < W; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] += sums[k][lane * E + i];
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  const int out_row = (p.q_offsets != nullptr ? __ldg(p.q_offsets + ci.b) + ci.q_i0 : ci.q_row0) + tok;
  const int head = ci.hk * p.G + ci.h0 + g;
  __nv_bfloat16* dst = p.out + (int64_t)out_row * p.o_stride_tok + (int64_t)head * p.o_stride_head + lane * E;
  if constexpr (E == 2) {
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
  } else if constexpr (E == 4) {
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
  } else {
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                   pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[(int64_t)head * p.total_q + out_row] = wsum > 0.f ? (mu + __log2f(wsum)) * kLn2 : -INFINITY;
}

cudaError_t launch_kv_append(const AppendParams& p, int head_dim, bool fp8, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.total_new * p.hkv;
  if (rows == 0) return cudaSuccess;
  const int threads = 256;
  const int64_t blocks = (rows * 32 + threads - 1) / threads;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (fp8 && head_dim == 256) {
    kv_append_kernel<256, true><<<(unsigned)blocks, threads, 0, stream>>>(p);
  } else if (fp8 && head_dim == 128) {
    kv_append_kernel<128, true><<<(unsigned)blocks, threads, 0, stream>>>(p);
  } else if (fp8) {
    kv_append_kernel<64, true><<<(unsigned)blocks, threads, 0, stream>>>(p);
  } else if (head_dim == 256) {
    kv_append_kernel<256, false><<<(unsigned)blocks, threads, 0, stream>>>(p);
  } else if (head_dim == 128) {
    kv_append_kernel<128, false><<<(unsigned)blocks, threads, 0, stream>>>(p);
  } else {
    kv_append_kernel<64, false><<<(unsigned)blocks, threads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_combine(const CombineParams& p, int num_items, int head_dim, bool overlap_prev,
                           cudaStream_t stream) {
  if (num_items == 0) return cudaSuccess;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)num_items);
  cfg.blockDim = dim3((unsigned)kCombineThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_prev ? 1 : 0;
  return head_dim == 256   ? cudaLaunchKernelEx(&cfg, combine_kernel<256>, p)
         : head_dim == 128 ? cudaLaunchKernelEx(&cfg, combine_kernel<128>, p)
                           : cudaLaunchKernelEx(&cfg, combine_kernel<64>, p);
}

cudaError_t launch_combine_shared(const CombineParams& p, int num_items, int max_rows, int max_parts, int head_dim,
                                  bool overlap_prev, cudaStream_t stream) {
  if (num_items == 0) return cudaSuccess;
  const bool split = max_parts > 8;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)num_items,
                     (unsigned)(split ? max_rows : (max_rows + kSharedCombineWarps - 1) / kSharedCombineWarps));
  cfg.blockDim = dim3(32u * kSharedCombineWarps);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_prev ? 1 : 0;
  if (split)
    return head_dim == 256   ? cudaLaunchKernelEx(&cfg, combine_shared_kernel<256, true>, p)
           : head_dim == 128 ? cudaLaunchKernelEx(&cfg, combine_shared_kernel<128, true>, p)
                             : cudaLaunchKernelEx(&cfg, combine_shared_kernel<64, true>, p);
  return head_dim == 256   ? cudaLaunchKernelEx(&cfg, combine_shared_kernel<256, false>, p)
         : head_dim == 128 ? cudaLaunchKernelEx(&cfg, combine_shared_kernel<128, false>, p)
                           : cudaLaunchKernelEx(&cfg, combine_shared_kernel<64, false>, p);
}

}  // namespace pkv
