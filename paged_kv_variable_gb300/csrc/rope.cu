// Per-head RMS norm and rotary position of query and key rows, alone
// (pkv_qk_norm_rope) or on the way into the KV cache (pkv_rope_kv_append).
//
// One warp per (token, run of heads); a block's warps take consecutive tokens,
// consecutive blocks the runs of the same tokens.  A head's D values sit in D / 8 lanes, 8
// a lane, as two 4-value pieces placed so that both members of every rotated
// pair are in the same lane: with pairs (i, i + rot/2) lane l holds
// 4l .. 4l+3 and rot/2 + 4l .. rot/2 + 4l+3, else 8l .. 8l+7.  So the rotation
// exchanges nothing between lanes, each lane needs 4 cosines and 4 sines (not
// 8 of each), and the norm's sum of squares is one shuffle tree of D / 8 lanes.
//
// Everything is fp32 from the bf16 input to the one rounding at the end.
//
// Bound by HBM on large calls (131072 tokens, 32 + 8 heads of 128: norm + rotation
// 391 us = 7.0 TB/s, append to an fp8 cache 413 us = 7.1 TB/s, both at the rate of
// a plain copy), by the launch and a chain of dependent loads (sequence, page, row)
// on a decode batch (64 tokens, inside a graph: 1.9 us norm + rotation, 2.7 us
// append).
#include <cuda_bf16.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr int kRopeWarps = 4;  // (with 8, 4093 tokens took 18.5 us in place of 17.8)
constexpr int kRopeThreads = 32 * kRopeWarps;
constexpr int kRopeBlocks = 10;  // blocks an SM (48 registers a thread)

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack4(uint2 v, float* f) {
  f[0] = bf_lo(v.x);
  f[1] = bf_hi(v.x);
  f[2] = bf_lo(v.y);
  f[3] = bf_hi(v.y);
}

__device__ __forceinline__ uint32_t codes4(const float* f, float inv) {
  return (uint32_t)f32x2_to_e4m3x2(__fmul_rn(f[0], inv), __fmul_rn(f[1], inv)) |
         ((uint32_t)f32x2_to_e4m3x2(__fmul_rn(f[2], inv), __fmul_rn(f[3], inv)) << 16);
}

// Sequence and position of a token.
struct TokenAt {
  int b;
  int pos;
};

// The sequence of token t (the largest b with cu[b] <= t) and its position,
// found by the whole warp: each step probes 32 boundaries at once, and the last
// one brings every candidate's lengths along, so nothing is loaded after the
// search (ragged append of 2000 tokens: 14.3 -> 13.7 us, 131072 into fp8: 449 -> 442).  QUERIES:
// the queries are the last of the positions, cache + new - queries + i.
template <bool QUERIES>
__device__ __forceinline__ TokenAt find_token(const RopeParams& p, int t) {
  const int lane = threadIdx.x & 31;
  const int32_t* cu = QUERIES ? p.cu_q : p.a.cu_knew;
  int lo = 0, n = p.a.batch;
  while (n > 32) {
    const int step = (n + 31) >> 5;
    const bool in = lane * step < n && __ldg(cu + lo + lane * step) <= t;
    const int c = max(1, __popc(__ballot_sync(0xffffffffu, in))) - 1;
    lo += c * step;
    n = min(step, n - c * step);
  }
  const int b = lo + min(lane, n - 1);
  const int start = __ldg(cu + b);
  int first = __ldg(p.a.cache_seqlens + b);  // the sequence's position of its token 0
  if constexpr (QUERIES) {
    first -= __ldg(cu + b + 1) - start;
    if (p.a.total_new > 0) first += __ldg(p.a.cu_knew + b + 1) - __ldg(p.a.cu_knew + b);
  }
  const int c = max(1, __popc(__ballot_sync(0xffffffffu, lane < n && start <= t))) - 1;
  return {lo + c, __shfl_sync(0xffffffffu, first - start, c) + t};
}

// One head's lane share: norm and rotation of the 8 values x (pieces 0..3, 4..7).
// (the operations are spelled out, so that every instance gives the same bits:
// a row rotated alone equals the row rotated into a bf16 cache)
template <int D>
__device__ __forceinline__ void transform(float* x, bool norm, const float* w, float eps, bool rot, bool pairs,
                                          const float* cs, const float* sn) {
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __fmaf_rn(x[i], x[i], ss);
#pragma unroll
    for (int o = D / 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(__fmaf_rn(ss, 1.f / D, eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), w[i]);
  }
  if (rot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = pairs ? 2 * i : i, b = pairs ? 2 * i + 1 : i + 4;
      const float u = x[a], v = x[b];
      x[a] = __fmaf_rn(u, cs[i], -__fmul_rn(v, sn[i]));
      x[b] = __fmaf_rn(v, cs[i], __fmul_rn(u, sn[i]));
    }
  }
}

// APPEND: keys go into the cache (FP8: as e4m3 codes) with the values, positions
// follow from cache_seqlens; else keys go to k_out and positions are given.
// HC: heads of a warp's run, per D / 8 lanes.
template <int D, bool APPEND, bool FP8, bool PAIRS, int HC>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8;          // lanes of a head
  constexpr int kHeads = 32 / kLanes;    // heads side by side in a warp
  constexpr int kRun = kHeads * HC;      // heads of a warp
  // (an ordinary launch, behind everything on the stream; the attention of the
  // same call may start now, and waits for this kernel before it reads anything)
  if constexpr (APPEND) grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int l = lane % kLanes, sub = lane / kLanes;
  const int uq = (p.hq + kRun - 1) / kRun, uk = (p.a.hkv + kRun - 1) / kRun;
  const int units = uq + (APPEND ? 2 : 1) * uk;
  const int tb = blockIdx.x / units, u = blockIdx.x - tb * units;
  const int t = tb * kRopeWarps + (threadIdx.x >> 5);
  // what this warp does: 0 queries, 1 keys, 2 values (of the append)
  const int part = u < uq ? 0 : (u < uq + uk ? 1 : 2);
  if (t >= (part == 0 ? p.total_q : p.a.total_new)) return;
  const int heads = part == 0 ? p.hq : p.a.hkv;
  const int h0 = (part == 0 ? u : part == 1 ? u - uq : u - uq - uk) * kRun + sub;

  // this lane's two pieces, and whether they are rotated
  const int half = p.rot_dim >> 1;
  const bool rot = part < 2 && 8 * l < p.rot_dim;
  const int pa = (!PAIRS && rot) ? 4 * l : 8 * l;
  const int pb = (!PAIRS && rot) ? half + 4 * l : 8 * l + 4;

  // the rows, copied to shared memory while the position is looked up: a warp
  // waiting for its position and table row holds its heads there and not in
  // registers, so more warps fit (131072 tokens, norm + rotation: 480 -> 417 us)
  const __nv_bfloat16* src = part == 0 ? p.q + (int64_t)t * p.q_stride_tok
                                       : (part == 1 ? p.a.k_new : p.a.v_new) + (int64_t)t * p.a.n_stride_tok;
  const int64_t src_head = part == 0 ? p.q_stride_head : p.a.n_stride_head;
  __shared__ __align__(16) uint8_t rows_smem[kRopeWarps][kRun * D * 2];
  uint8_t* mine = rows_smem[threadIdx.x >> 5];
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    const int h = h0 + i * kHeads;
    if (h < heads) cp_async_16(mine + (i * kHeads + sub) * D * 2 + l * 16, src + h * src_head + l * 8, 16);
  }
  cp_async_commit();
  float w[8];
  const __nv_bfloat16* wt = part == 0 ? p.q_weight : p.k_weight;
  const bool norm = part < 2 && wt != nullptr;
  if (norm) {
    unpack4(__ldg(reinterpret_cast<const uint2*>(wt + pa)), w);
    unpack4(__ldg(reinterpret_cast<const uint2*>(wt + pb)), w + 4);
  }

  // position, and (append) the cache row
  int pos = 0, b = 0;
  int64_t dst = 0;
  if constexpr (APPEND) {
    if (part == 0) {
      const TokenAt at = find_token<true>(p, t);
      b = at.b;
      pos = at.pos;
    } else {
      const TokenAt at = find_token<false>(p, t);
      b = at.b;
      pos = at.pos;
      if (pos < 0 || pos >= p.a.capacity) {
        if (lane == 0) record_status(p.a.status, PKV_ERR_DEVICE_BOUNDS, b, pos);
        cp_async_wait_group<0>();  // (no copy in flight when the block ends)
        return;
      }
      if (p.a.page_size > 0) {
        int npages;
        const int32_t* pages = seq_pages(p.a.block_table, p.a.bt_stride, p.a.page_indptr, b, &npages);
        const int pi = pos / p.a.page_size;
        const int page = (npages >= 0 && pi >= npages) ? -1 : __ldg(pages + pi);
        if (page < 0 || page >= p.a.num_pages) {
          if (lane == 0) record_status(p.a.status, PKV_ERR_DEVICE_BOUNDS, b, page);
          cp_async_wait_group<0>();
          return;
        }
        dst = (int64_t)page * p.a.c_stride_page + (int64_t)(pos - pi * p.a.page_size) * p.a.c_stride_tok;
      } else {
        dst = (int64_t)b * p.a.c_stride_page + (int64_t)pos * p.a.c_stride_tok;
      }
    }
  } else {
    pos = p.rot_dim > 0 ? __ldg(p.positions + t) : 0;
    b = t;
  }
  // (a value row is skipped with its key row)
  if (p.rot_dim > 0 && (pos < 0 || pos >= p.num_positions)) {
    if (lane == 0) record_status(p.a.status, PKV_ERR_DEVICE_BOUNDS, b, pos);
    cp_async_wait_group<0>();
    return;
  }
  float cs[4], sn[4];
  if (rot) {
    const float* row = p.cos_sin + (int64_t)pos * p.rot_dim + 4 * l;
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(row));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half));
    cs[0] = c4.x, cs[1] = c4.y, cs[2] = c4.z, cs[3] = c4.w;
    sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
  }

  // (one IEEE reciprocal, as the plain append encodes)
  const float inv = (FP8 && part > 0) ? __frcp_rn(__ldg(part == 1 ? p.a.k_scale : p.a.v_scale)) : 1.f;
  // where the rows go
  uint8_t* out = static_cast<uint8_t*>(part == 2 ? p.a.v_cache : p.a.k_cache);
  int64_t out_head = p.a.c_stride_head * (FP8 ? 1 : 2);
  if constexpr (APPEND) out += dst * (FP8 ? 1 : 2);
  else out += (int64_t)t * p.a.c_stride_tok * 2;
  if (part == 0) {
    out = reinterpret_cast<uint8_t*>(p.q_out + (int64_t)t * p.qo_stride_tok);
    out_head = p.qo_stride_head * 2;
  }
  cp_async_wait_group<0>();
  __syncwarp();
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    const int h = h0 + i * kHeads;
    if (h - sub >= heads) break;  // (warp-uniform)
    const uint8_t* in = mine + (i * kHeads + sub) * D * 2;
    const uint2 ra = *reinterpret_cast<const uint2*>(in + 2 * pa), rb = *reinterpret_cast<const uint2*>(in + 2 * pb);
    float x[8];
    unpack4(ra, x);
    unpack4(rb, x + 4);
    transform<D>(x, norm, w, p.eps, rot, PAIRS, cs, sn);  // (shuffles: every lane of the warp)
    if (h >= heads) break;
    uint8_t* row = out + h * out_head;
    if (FP8 && part > 0) {
      *reinterpret_cast<uint32_t*>(row + pa) = codes4(x, inv);
      *reinterpret_cast<uint32_t*>(row + pb) = codes4(x + 4, inv);
    } else if (part == 2) {  // values: the bits as they came
      *reinterpret_cast<uint2*>(row + 2 * pa) = ra;
      *reinterpret_cast<uint2*>(row + 2 * pb) = rb;
    } else {
      *reinterpret_cast<uint2*>(row + 2 * pa) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
      *reinterpret_cast<uint2*>(row + 2 * pb) = make_uint2(pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
  }
}

template <int D, bool APPEND, bool FP8, bool PAIRS, int HC>
cudaError_t launch_run(const RopeParams& p, cudaStream_t stream) {
  constexpr int kRun = (256 / D) * HC;
  const int64_t uq = (p.hq + kRun - 1) / kRun, uk = (p.a.hkv + kRun - 1) / kRun;
  const int64_t tokens = std::max(p.total_q, p.a.total_new);
  const int64_t blocks = (tokens + kRopeWarps - 1) / kRopeWarps * (uq + (APPEND ? 2 : 1) * uk);
  if (blocks == 0) return cudaSuccess;
  if (blocks > INT32_MAX || tokens > INT32_MAX - kRopeWarps) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)kRopeThreads);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, rope_kernel<D, APPEND, FP8, PAIRS, HC>, p);
}

template <int D, bool APPEND, bool FP8, int HC>
cudaError_t launch_hc(const RopeParams& p, cudaStream_t stream) {
  return p.interleaved ? launch_run<D, APPEND, FP8, true, HC>(p, stream)
                       : launch_run<D, APPEND, FP8, false, HC>(p, stream);
}

// Heads a lane takes one after another: 1 while every warp of that split runs at
// once (152 SMs x 40), where a call is latency; 4 from twice that on, where a
// warp's lookups (sequence, position, table row, weights) are worth spreading over
// more rows; 2 between; 8 for the largest calls without an append whose heads fill
// such runs.  Measured at 32 + 8 heads of 128 (a call inside a captured graph), us
// at 1 / 2 / 4 / 8: norm + rotation of 64 tokens 1.91 / 2.06 / 2.31 / 3.56, of 512
// 5.28 / 4.25 / 4.65 / 6.01, of 4096 26.6 / 18.8 / 17.1 / 18.4, of 131072 - / 507 /
// 417 / 393; append of 64 tokens 2.57 / 2.64 / 2.77 / 2.88, of 4096 28.5 / 19.7 /
// 17.4 / 18.1.
template <int D, bool APPEND, bool FP8>
cudaError_t launch_d(const RopeParams& p, cudaStream_t stream) {
  constexpr int kHeads = 256 / D;
  const int64_t warps = (int64_t)std::max(p.total_q, p.a.total_new) *
                        ((p.hq + kHeads - 1) / kHeads + (APPEND ? 2 : 1) * ((p.a.hkv + kHeads - 1) / kHeads));
  if (warps <= 6080) return launch_hc<D, APPEND, FP8, 1>(p, stream);
  if (warps < 12160) return launch_hc<D, APPEND, FP8, 2>(p, stream);
  if constexpr (!APPEND) {
    if (warps >= 400000 && p.hq >= 8 * kHeads) return launch_hc<D, APPEND, FP8, 8>(p, stream);
  }
  return launch_hc<D, APPEND, FP8, 4>(p, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, cudaStream_t stream) {
  return head_dim == 256   ? launch_d<256, false, false>(p, stream)
         : head_dim == 128 ? launch_d<128, false, false>(p, stream)
                           : launch_d<64, false, false>(p, stream);
}

cudaError_t launch_rope_kv_append(const RopeParams& p, int head_dim, bool fp8, cudaStream_t stream) {
  if (fp8)
    return head_dim == 256   ? launch_d<256, true, true>(p, stream)
           : head_dim == 128 ? launch_d<128, true, true>(p, stream)
                             : launch_d<64, true, true>(p, stream);
  return head_dim == 256   ? launch_d<256, true, false>(p, stream)
         : head_dim == 128 ? launch_d<128, true, false>(p, stream)
                           : launch_d<64, true, false>(p, stream);
}

}  // namespace pkv
