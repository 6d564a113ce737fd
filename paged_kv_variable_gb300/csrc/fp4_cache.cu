// Rows of a cache: the 4-bit append (quantised on the way in) and the gather,
// which reads rows of any cache back as bf16.
//
// Append: y = x * fp32(1/scale), block scale s = e4m3(max |y| / 6), codes
// e2m1(y / s).  A thread owns two blocks of 16 dims of a key row and of the same
// value row, so the maximum needs no other lane; it reads 64 bytes of each and
// writes 16 + 2.  The quotients are rounded as a division is: halfway cases of y / s
// are common (bf16 inputs over a 4-bit significand) and a product with 1/s would
// take some of them off the tie.
//
// A warp's rows are consecutive tokens of a head, which are neighbours in a cache
// whose heads come before its tokens.  Instructions and HBM bound both kernels alike
// on large calls (131072 tokens of 8 heads written and read back 243 us, 5.7 TB/s), the
// launch and the chain sequence, position, page on small ones.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr int kRowThreads = 256;
// A thread has two blocks of a row, `part` and D / 32 + `part` (one block a thread has the
// addresses of a row made twice as often).  Rows of bf16 are read and written in pieces of
// 32 bytes, whole sectors, where they are aligned for it (else 16: 154 in place of 117 us
// for 131072 rows read back).
constexpr int kBlocks = 2;

__device__ __forceinline__ void load16(const __nv_bfloat16* src, int wide, uint32_t* w) {
  if (wide) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(src));
    return;
  }
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(src));
  const uint4 b = __ldg(reinterpret_cast<const uint4*>(src) + 1);
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

__device__ __forceinline__ void store16(__nv_bfloat16* dst, int wide, const uint32_t* w) {
  const uint4 a = make_uint4(w[0], w[1], w[2], w[3]), b = make_uint4(w[4], w[5], w[6], w[7]);
  if (wide) {
    st_global_v8(dst, a, b);
  } else {
    reinterpret_cast<uint4*>(dst)[0] = a;
    reinterpret_cast<uint4*>(dst)[1] = b;
  }
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16 bf16 values -> 8 bytes of codes and the block scale
__device__ __forceinline__ uint2 encode16(const uint32_t* w, float inv, uint32_t& sf) {
  uint64_t y[8];  // the values over the tensor's scale, negated
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = mul_f32x2(f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), f32x2(-inv, -inv));
    float lo, hi;
    f32x2_split(y[i], lo, hi);
    a = fmax3(a, fabsf(lo), fabsf(hi));
  }
  sf = (uint32_t)f32x2_to_e4m3x2(__fdiv_rn(a, 6.f), 0.f) & 0xFFu;
  if (sf == 0) return make_uint2(0u, 0u);
  const float s = f16x2_to_f32(e4m3x2_to_f16x2(sf)).x;
  if (a > 4096.f) {  // (the largest scale, 448: all such values get the largest code)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      f32x2_split(y[i], lo, hi);
      y[i] = f32x2(fminf(fmaxf(lo, -4096.f), 4096.f), fminf(fmaxf(hi, -4096.f), 4096.f));
    }
  }
  // the quotient rounded to nearest: with r = 1/s and q = (-y) r both rounded, q - r (q s + y)
  // is (Markstein, "Computation of elementary functions on the IBM RISC System/6000
  // processor", 1990; q s + y is exact); in this form the sign of a zero stays
  const float r = __frcp_rn(s);
  float q[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t u = mul_f32x2(y[i], f32x2(-r, -r));
    f32x2_split(fma_f32x2(f32x2(-r, -r), fma_f32x2(u, f32x2(s, s), y[i]), u), q[2 * i], q[2 * i + 1]);
  }
  return make_uint2(f32x8_to_e2m1(q), f32x8_to_e2m1(q + 8));
}

// The row of a thread: D / 32 lanes a row, then four consecutive tokens, then heads,
// then the next four tokens.
struct RowOf {
  int part, t, h;
};
__device__ __forceinline__ RowOf row_of(int kb_log2, const FastDiv& heads) {
  const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  const int row = (int)(i >> kb_log2);  // (below 2^31: the launch)
  const int group = quot(row >> 2, heads);
  return {(int)(i & ((1 << kb_log2) - 1)), group * 4 + (row & 3), (row >> 2) - group * heads.d};
}

// Sequence of row t, the largest b with cu[b] <= t, and the row's place in it: 32 probes
// at a time for the warp's first row (the least of its rows' tokens).  SPREAD (few rows a
// sequence): the last 32 candidates come a lane each, with their from, and serve all the warp's
// rows (else a sequence after another from the first row's, up to five dependent loads: an
// append and a gather of a decode batch 7.1 us in a graph in place of 6.7); otherwise most rows are
// of the first one's sequence.
template <bool SPREAD>
struct SeqOf {
  int b, first, from;  // (SPREAD: cu[b] and from[b], null: 0)
  __device__ __forceinline__ int row(const int32_t* cu, int t) const { return t - (SPREAD ? first : __ldg(cu + b)); }
  __device__ __forceinline__ int start(const int32_t* f) const { return SPREAD ? from : f != nullptr ? __ldg(f + b) : 0; }
};
template <bool SPREAD>
__device__ __forceinline__ SeqOf<SPREAD> seq_of(const int32_t* cu, const int32_t* from, int batch, int t) {
  const int lane = threadIdx.x & 31;
  const int least = __reduce_min_sync(0xffffffffu, t);
  constexpr int last = SPREAD ? 32 : 1;
  int lo = 0;
  for (int n = batch; n > last;) {
    const int step = (n + 31) >> 5, at = lo + lane * step;
    const bool below = lane * step < n && (lane == 0 || __ldg(cu + at) <= least);
    const int k = __popc(__ballot_sync(0xffffffffu, below)) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  }
  if constexpr (SPREAD) {
    const bool there = lo + lane < batch;
    const int c = there ? __ldg(cu + lo + lane) : INT32_MAX;
    const int f = there && from != nullptr ? __ldg(from + lo + lane) : 0;
    int k = 0;
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
      if (__shfl_sync(0xffffffffu, c, k + step) <= t) k += step;
    SeqOf<SPREAD> s{lo + k, __shfl_sync(0xffffffffu, c, k), __shfl_sync(0xffffffffu, f, k)};
    if (k < 31) return s;
    while (s.b + 1 < batch && __ldg(cu + s.b + 1) <= t) ++s.b;
    return {s.b, __ldg(cu + s.b), from != nullptr ? __ldg(from + s.b) : 0};
  } else {
    while (lo + 1 < batch && __ldg(cu + lo + 1) <= t) ++lo;
    return {lo, 0, 0};  // (the rest is loaded where it is used, behind the loads of the row)
  }
}

// Few rows a sequence (of `rows`): a warp's are of several.
bool spread_rows(int rows, int batch) { return rows < 16 * (int64_t)batch; }

template <int D, bool SPREAD>
__global__ void __launch_bounds__(kRowThreads) fp4_append_kernel(const AppendParams p, const Fp4Scales sf,
                                                                 const FastDiv heads, const FastDiv pdiv, const int wide) {
  const RowOf r = row_of(D == 64 ? 1 : D == 128 ? 2 : 3, heads);
  const int part = r.part, t = r.t, h = r.h;
  const SeqOf<SPREAD> seq = seq_of<SPREAD>(p.cu_knew, p.cache_seqlens, p.batch, t);
  if (t >= p.total_new) return;
  const int b = seq.b;
  const int64_t src = (int64_t)t * p.n_stride_tok + (int64_t)h * p.n_stride_head + part * 16;
  uint32_t kw[16], vw[16];
#pragma unroll
  for (int k = 0; k < kBlocks; ++k) {
    load16(p.k_new + src + k * (D / 2), wide, kw + 8 * k);
    load16(p.v_new + src + k * (D / 2), wide, vw + 8 * k);
  }
  auto report = [&](int at) {
    if (part != 0) return;
    if (p.status_code_only) record_code(p.status, PKV_ERR_DEVICE_BOUNDS);
    else record_status(p.status, PKV_ERR_DEVICE_BOUNDS, b, at);
  };
  const int pos = seq.start(p.cache_seqlens) + seq.row(p.cu_knew, t);
  if (pos < 0 || pos >= p.capacity) return report(pos);
  int64_t page = b;
  int slot = pos;
  if (p.page_size > 0) {
    int npages;
    const int32_t* pages = seq_pages(p.block_table, p.bt_stride, p.page_indptr, b, &npages);
    const int pi = quot(pos, pdiv);
    const int pg = (npages >= 0 && pi >= npages) ? -1 : __ldg(pages + pi);
    if (pg < 0 || pg >= p.num_pages) return report(pg);
    page = pg;
    slot = pos - pi * p.page_size;
  }
  const int64_t dst = page * p.c_stride_page + (int64_t)slot * p.c_stride_tok + (int64_t)h * p.c_stride_head + part * 8;
  const int64_t sdst = page * sf.stride_page + (int64_t)slot * sf.stride_tok + (int64_t)h * sf.stride_head + part;
  auto put = [&](void* cache, uint8_t* sfs, const uint32_t* w, float inv) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      uint32_t s;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + dst + k * (D / 4)) = encode16(w + 8 * k, inv, s);
      sfs[sdst + k * (D / 32)] = (uint8_t)s;
    }
  };
  put(p.k_cache, sf.k, kw, __frcp_rn(__ldg(p.k_scale)));
  put(p.v_cache, sf.v, vw, __frcp_rn(__ldg(p.v_scale)));
}

// ------------------------------------------------------------------ gather
// A block of 16 dims, key or value: 32, 16 or 8 + 1 bytes in, 32 out (f16: code x block scale
// as f16, without the tensor's scale; of the copies that an attention reads the keys have its
// sign alone).
template <int DT>
__device__ __forceinline__ void read16(const void* cache, const uint8_t* sf, float scale, bool f16, uint32_t* w) {
  uint32_t h[8];
  if constexpr (DT == PKV_FP8_E4M3) {
    const uint4 c = __ldg(static_cast<const uint4*>(cache));
    e4m3x4_to_f16x4(c.x, h[0], h[1]);
    e4m3x4_to_f16x4(c.y, h[2], h[3]);
    e4m3x4_to_f16x4(c.z, h[4], h[5]);
    e4m3x4_to_f16x4(c.w, h[6], h[7]);
  } else {
    const uint2 c = __ldg(static_cast<const uint2*>(cache));
    const uint32_t s = prmt(e4m3x2_to_f16x2(__ldg(sf)), 0u, 0x1010u);
    e2m1x8_to_f16(c.x, h);
    e2m1x8_to_f16(c.y, h + 4);
    // (code * block scale has six significant bits: exact)
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = mul_f16x2(h[i], s);
  }
  if (f16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = h[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 a = f16x2_to_f32(h[i]);
    float lo, hi;
    f32x2_split(mul_f32x2(f32x2(a.x, a.y), f32x2(scale, scale)), lo, hi);
    w[i] = pack_bf16(lo, hi);
  }
}

template <int DT, bool SPREAD>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(const GatherParams p, const FastDiv heads,
                                                             const FastDiv pdiv, const int wide) {
  const RowOf r = row_of(p.head_dim == 64 ? 1 : p.head_dim == 128 ? 2 : 3, heads);
  const int part = r.part, t = r.t, h = r.h;
  if (p.lens != nullptr && blockIdx.x == 0) {
    for (int k = threadIdx.x; k < p.batch; k += kRowThreads)
      if (__ldg(p.cache_seqlens + k) != __ldg(p.plan_lc + k))
        record_status(p.status, PKV_ERR_PLAN_MISMATCH, k, __ldg(p.cache_seqlens + k));
  }
  const SeqOf<SPREAD> seq = seq_of<SPREAD>(p.cu_rows, p.starts, p.batch, t);
  if (t >= p.total_rows) return;
  const int b = seq.b;
  if (p.lens != nullptr && seq.row(p.cu_rows, t) >= __ldg(p.lens + b)) return;
  const int pos = seq.start(p.starts) + seq.row(p.cu_rows, t);
  const int half = p.head_dim / 32;  // blocks between a thread's two
  const int64_t dst = (int64_t)t * p.o_stride_tok + (int64_t)h * p.o_stride_head + part * 16;
  // a position or page out of range: nothing is written or, of copies that an attention reads
  // (a workspace holds rows of the call before), zeros, as the tiles straight over a cache have
  auto report = [&](int at) {
    if (part == 0) record_status(p.status, PKV_ERR_DEVICE_BOUNDS, b, at);
    if (p.lens == nullptr) return;
    const uint32_t none[8] = {};
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      store16(p.k_out + dst + k * half * 16, wide & 2, none);
      store16(p.v_out + dst + k * half * 16, wide & 2, none);
    }
  };
  if (pos < 0 || pos >= p.capacity) return report(pos);
  int64_t page = b;
  int slot = pos;
  if (p.page_size > 0) {
    int npages;
    const int32_t* pages = seq_pages(p.block_table, p.bt_stride, p.page_indptr, b, &npages);
    const int pi = quot(pos, pdiv);
    const int pg = (npages >= 0 && pi >= npages) ? -1 : __ldg(pages + pi);
    if (pg < 0 || pg >= p.num_pages) return report(pg);
    page = pg;
    slot = pos - pi * p.page_size;
  }
  constexpr int kBytes = DT == PKV_BF16 ? 32 : DT == PKV_FP8_E4M3 ? 16 : 8;  // of a block of 16 dims
  const int64_t at = (page * p.c_stride_page + (int64_t)slot * p.c_stride_tok + (int64_t)h * p.c_stride_head) *
                         (DT == PKV_BF16 ? 2 : 1) +
                     part * kBytes;
  const int64_t sat = page * p.sf.stride_page + (int64_t)slot * p.sf.stride_tok + (int64_t)h * p.sf.stride_head + part;
  uint32_t w[2][kBlocks][8];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint8_t* cache = static_cast<const uint8_t*>(x == 0 ? p.k_cache : p.v_cache) + at;
    const uint8_t* sf = (x == 0 ? p.sf.k : p.sf.v) + sat;
    const float* scale = x == 0 ? p.k_scale : p.v_scale;
    if ((x == 0 ? p.k_out : p.v_out) == nullptr) continue;
    float f = scale != nullptr ? __ldg(scale) : 1.f;
    if (p.lens != nullptr) f = f < 0.f ? -1.f : 1.f;
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      if constexpr (DT == PKV_BF16)
        load16(reinterpret_cast<const __nv_bfloat16*>(cache + k * half * kBytes), wide & 1, w[x][k]);
      else
        read16<DT>(cache + k * half * kBytes, sf + k * half, f, x == 1 && p.lens != nullptr, w[x][k]);
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    __nv_bfloat16* out = x == 0 ? p.k_out : p.v_out;
    if (out == nullptr) continue;
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) store16(out + dst + k * half * 16, wide & 2, w[x][k]);
  }
}

auto append_kernel(int head_dim, bool spread) {
  if (head_dim == 256) return spread ? fp4_append_kernel<256, true> : fp4_append_kernel<256, false>;
  if (head_dim == 128) return spread ? fp4_append_kernel<128, true> : fp4_append_kernel<128, false>;
  return spread ? fp4_append_kernel<64, true> : fp4_append_kernel<64, false>;
}

auto rows_kernel(int cache_dtype, bool spread) {
  if (cache_dtype == PKV_FP4_E2M1) return spread ? gather_kernel<PKV_FP4_E2M1, true> : gather_kernel<PKV_FP4_E2M1, false>;
  if (cache_dtype == PKV_FP8_E4M3) return spread ? gather_kernel<PKV_FP8_E4M3, true> : gather_kernel<PKV_FP8_E4M3, false>;
  return spread ? gather_kernel<PKV_BF16, true> : gather_kernel<PKV_BF16, false>;
}

}  // namespace

// Rows of bf16 that start on 32 bytes.
bool wide_rows(const void* a, const void* b, int64_t stride_tok, int64_t stride_head, int64_t stride_page = 0) {
  return (reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) % 32 == 0 && stride_tok % 16 == 0 &&
         stride_head % 16 == 0 && stride_page % 16 == 0;
}

// Blocks of a launch over `rows` tokens (rounded up to four) of `heads` heads; -1: rows, those
// of the last block's idle threads with them, would pass 31 bits.
int64_t row_blocks(int rows, int heads, int head_dim) {
  const int64_t all = ((int64_t)rows + 3) / 4 * 4 * heads;
  if (all > INT32_MAX - kRowThreads) return -1;
  return (all * (head_dim / (16 * kBlocks)) + kRowThreads - 1) / kRowThreads;
}

cudaError_t launch_fp4_append(const AppendParams& p, const Fp4Scales& sf, int head_dim, cudaStream_t stream) {
  if (p.total_new == 0) return cudaSuccess;
  const int64_t blocks = row_blocks(p.total_new, p.hkv, head_dim);
  if (blocks < 0 || blocks > INT32_MAX) return cudaErrorInvalidValue;
  const FastDiv heads = fast_div(p.hkv), pdiv = fast_div(p.page_size > 0 ? p.page_size : 1);
  const int wide = wide_rows(p.k_new, p.v_new, p.n_stride_tok, p.n_stride_head);
  const auto kernel = append_kernel(head_dim, spread_rows(p.total_new, p.batch));
  kernel<<<(unsigned)blocks, kRowThreads, 0, stream>>>(p, sf, heads, pdiv, wide);
  return cudaGetLastError();
}

cudaError_t launch_gather(const GatherParams& p, int cache_dtype, cudaStream_t stream) {
  if (p.total_rows == 0) return cudaSuccess;
  const int64_t blocks = row_blocks(p.total_rows, p.hkv, p.head_dim);
  if (blocks < 0 || blocks > INT32_MAX) return cudaErrorInvalidValue;
  const FastDiv heads = fast_div(p.hkv), pdiv = fast_div(p.page_size > 0 ? p.page_size : 1);
  // bit 0: a bf16 cache's rows, bit 1: the rows written
  const int wide = wide_rows(p.k_cache, p.v_cache, p.c_stride_tok, p.c_stride_head, p.c_stride_page) |
                   wide_rows(p.k_out, p.v_out, p.o_stride_tok, p.o_stride_head) << 1;
  const auto kernel = rows_kernel(cache_dtype, spread_rows(p.total_rows, p.batch));
  kernel<<<(unsigned)blocks, kRowThreads, 0, stream>>>(p, heads, pdiv, wide);
  return cudaGetLastError();
}

}  // namespace pkv
