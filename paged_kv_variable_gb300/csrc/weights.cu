// The attention weight that cached keys received (pkv_attn_weights):
//   scores[b, hk, j] = scores_in + sum over rows (i, g) of exp(scale q . k_j - lse)
// The softmax's sums are known (lse), so one pass over K does it, S^T = K Q^T by
// m16n8k16 MMAs with the keys on the 16-row side.  A dot product does not depend on
// the order of the dims, so each lane takes 16 bytes of a key row at a time and the
// queries are laid out to match.  A key's sum is one warp's, in a fixed order:
// there are no atomics.
//
// Few rows (a decode step's, up to 8 or 16): the queries stay in registers and the
// keys stream by, each warp with a ring of its own in shared memory (cp.async), its
// steps every fourth of the block's; HBM bounds it.  (Warps that held 32 keys each
// and ended had their chain length, page, key, query, sum in every wave of blocks: 92
// in place of 51 us on a decode batch.)
//
// Many rows (a window of queries, a prompt): the keys of a step stay in registers and
// the queries pass by from shared memory, where the block puts them in the order of
// the MMA's operand (128 rows at a time).  The warp MMAs (their pipe is in use 53% of the
// time) and the chain MMA, exponential, sum of a tile bound it: 32
// queries a sequence of 8 prompts of 5000 to 16384 fp8 keys, 128 rows a kv head, 76.0 us, of
// which the MMAs at their rate would take 37.  (The same with S^T = K Q^T by tcgen05 MMAs, a key
// a thread, the queries staged as operands (an fp8 one as two e4m3 terms): 88 us, for the
// staging took 5 us of each block and two blocks filled an SM.)
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;

// A cache row by type: bytes, and what a lane's loads of it hold.
template <int D, int DT>
struct Row {
  static constexpr int kBytes = DT == PKV_BF16 ? 2 * D : DT == PKV_FP8_E4M3 ? D : D / 2;
  static constexpr int kPieces = kBytes / 16;
  static constexpr int kSf = DT == PKV_FP4_E2M1 ? D / kFp4Block : 0;
  static constexpr int kWords = D / 8;  // registers of a lane's part of a row, as operand pairs
  // first of the eight dims of registers 4c .. 4c+3 of lane column t
  static __device__ __forceinline__ int dim(int c, int t) {
    if constexpr (DT == PKV_BF16) return 32 * c + 8 * t;
    if constexpr (DT == PKV_FP8_E4M3) return 64 * (c >> 1) + 16 * t + 8 * (c & 1);
    return D == 64 ? 16 * t + 8 * c : 32 * t + 8 * (c & 3) + 128 * (c >> 2);
  }
  // A row's pieces from `get16(piece)` (D = 64 in 4 bits: `get8` of half pieces) and its
  // scales from `sf(byte)` (one, or two as 16 bits), as operand pairs.
  template <class G16, class G8, class S1, class S2>
  static __device__ __forceinline__ void load(int t, uint32_t* w, G16&& get16, G8&& get8, S1&& sf1, S2&& sf2) {
    if constexpr (DT == PKV_BF16) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint4 v = get16(4 * c + t);
        w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
      }
    } else if constexpr (DT == PKV_FP8_E4M3) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint4 v = get16(4 * c + t);
        e4m3x4_to_f16x4(v.x, w[8 * c], w[8 * c + 1]);
        e4m3x4_to_f16x4(v.y, w[8 * c + 2], w[8 * c + 3]);
        e4m3x4_to_f16x4(v.z, w[8 * c + 4], w[8 * c + 5]);
        e4m3x4_to_f16x4(v.w, w[8 * c + 6], w[8 * c + 7]);
      }
    } else if constexpr (D == 64) {
      const uint2 v = get8(t);
      e2m1x8_to_f16(v.x, w);
      e2m1x8_to_f16(v.y, w + 4);
      const uint32_t f = prmt(e4m3x2_to_f16x2(sf1(t)), 0u, 0x1010u);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = mul_f16x2(w[i], f);
    } else {
#pragma unroll
      for (int c = 0; c < D / 128; ++c) {
        const uint4 v = get16(4 * c + t);
        e2m1x8_to_f16(v.x, w + 16 * c);
        e2m1x8_to_f16(v.y, w + 16 * c + 4);
        e2m1x8_to_f16(v.z, w + 16 * c + 8);
        e2m1x8_to_f16(v.w, w + 16 * c + 12);
        const uint32_t f = e4m3x2_to_f16x2(sf2(8 * c + 2 * t));
        const uint32_t f0 = prmt(f, 0u, 0x1010u), f1 = prmt(f, 0u, 0x3232u);
#pragma unroll
        for (int i = 0; i < 16; ++i) w[16 * c + i] = mul_f16x2(w[16 * c + i], i < 8 ? f0 : f1);
      }
    }
  }
};

// Eight dims of a query row (zeros where qr is null).  Over a cache that is not bf16 they
// become f16, times a power of two of the row's (RowScale), which its logits take out again.
__device__ __forceinline__ uint4 query8(const __nv_bfloat16* qr, int d0) {
  return qr ? __ldg(reinterpret_cast<const uint4*>(qr + d0)) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint32_t most8(const uint4& v, uint32_t most) {
  return bf16x2_most(v.x, bf16x2_most(v.y, bf16x2_most(v.z, bf16x2_most(v.w, most))));
}
__device__ __forceinline__ uint4 f16x8(const uint4& v, const RowScale& s) {
  return make_uint4(bf16x2_to_f16x2(s.times(v.x)), bf16x2_to_f16x2(s.times(v.y)), bf16x2_to_f16x2(s.times(v.z)),
                    bf16x2_to_f16x2(s.times(v.w)));
}

template <int DT>
__device__ __forceinline__ void mma(float* s, const uint32_t* a, const uint32_t* b, const uint32_t* q) {
  if constexpr (DT == PKV_BF16) mma_bf16(s, a[0], b[0], a[1], b[1], q[0], q[1]);
  else mma_f16(s, a[0], b[0], a[1], b[1], q[0], q[1]);
}

// A sequence: its query rows and keys, and the query row of row r (token first + r / G).
struct Seq {
  int q0, lq, lk, first, rows, total_q;
  bool ok;
};
__device__ __forceinline__ Seq load_seq(const WeightsParams& p, int b, bool report) {
  Seq s;
  s.q0 = __ldg(p.cu_q + b);
  s.lq = __ldg(p.cu_q + b + 1) - s.q0;
  s.total_q = __ldg(p.cu_q + p.batch);
  s.lk = __ldg(p.cache_seqlens + b);
  if (p.cu_knew != nullptr) s.lk += __ldg(p.cu_knew + b + 1) - __ldg(p.cu_knew + b);
  // (lse is (Hq, total_q): rows outside of it, or of q, are never read)
  s.ok = s.lk >= 0 && s.lk <= p.max_seqlen_k && s.lq >= 0 && s.lq <= p.max_seqlen_q && s.q0 >= 0 &&
         (int64_t)s.q0 + s.lq <= s.total_q && (p.max_total_q == 0 || s.total_q <= p.max_total_q);
  if (!s.ok && report) record_status(p.status, PKV_ERR_PLAN_MISMATCH, b, s.lk);
  s.first = p.last_queries > 0 ? max(0, s.lq - p.last_queries) : 0;
  s.rows = s.ok ? (s.lq - s.first) * p.G : 0;
  return s;
}

// What row r's weights need: its log2-domain LSE and the keys it sees (0: it adds nothing).
__device__ __forceinline__ void row_info(const WeightsParams& p, const Seq& s, int hk, int r, float& l2, int& lim) {
  l2 = 0.f;
  lim = 0;
  if (r >= s.rows) return;
  const int i = s.first + r / p.G;
  const float lse = __ldg(p.lse + (int64_t)(hk * p.G + r % p.G) * s.total_q + s.q0 + i);
  l2 = lse * kLog2e;
  if (lse != -INFINITY) lim = p.causal ? min(s.lk, i + s.lk - s.lq + 1) : s.lk;
}

__device__ __forceinline__ const __nv_bfloat16* query_row(const WeightsParams& p, const Seq& s, int hk, int r) {
  return r < s.rows ? p.q + (int64_t)(s.q0 + s.first + r / p.G) * p.q_stride_tok +
                          (int64_t)(hk * p.G + r % p.G) * p.q_stride_head
                    : nullptr;
}

template <int N>
__device__ __forceinline__ void async_copy(void* dst, const void* src, uint32_t bytes) {
  if constexpr (N == 16)
    cp_async_16(dst, src, bytes);
  else if constexpr (N > 0)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(N), "r"(bytes)
                 : "memory");
}

// ------------------------------------------------------------------ few rows
template <int D, int DT>
struct Stream {
  using R = Row<D, DT>;
  static constexpr int kKeys = R::kBytes <= 256 ? 32 : 16;  // of a step
  static constexpr int kStage = kKeys * (R::kBytes + R::kSf);
  static constexpr int kStages = kStage >= 8192 ? 2 : 4;  // (8 KB: 3 stages leave two blocks an SM, 55 in place of 51 us)
  static constexpr int kBytes = kWarps * kStages * kStage;
  // (rows of 128 bytes and more: those of a row pair that one access reads together on
  // different banks)
  static __device__ __forceinline__ uint32_t off(int r, int c) {
    return (uint32_t)(r * R::kBytes + ((R::kBytes >= 128 ? c ^ ((r & 1) << 2) : c) << 4));
  }
};

// The keys of a block, `chunk` of them from `begin` on, as a warp sees them: every fourth
// step of kKeys keys, through a ring of NS steps of its own in shared memory.
template <int D, int DT, int NS>
struct KeyRing {
  using R = Row<D, DT>;
  using S = Stream<D, DT>;
  const WeightsParams& p;
  const FastDiv& pdiv;
  uint8_t* ring;
  const uint8_t* kc;
  const uint8_t* ks;
  const int32_t* pages = nullptr;
  int npages = -1;
  int b, begin, end, mine, warp, lane;
  int pg;  // page of this lane's key of the next step to copy

  __device__ __forceinline__ KeyRing(const WeightsParams& p_, const FastDiv& d, uint8_t* smem, int b_, int hk, int begin_,
                                     int end_)
      : p(p_), pdiv(d), b(b_), begin(begin_), end(end_), warp(threadIdx.x >> 5), lane(threadIdx.x & 31) {
    const int steps = (end - begin + S::kKeys - 1) / S::kKeys;
    mine = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;
    ring = smem + warp * (NS * S::kStage);
    kc = static_cast<const uint8_t*>(p.k_cache) + (int64_t)hk * p.c_stride_head;
    ks = p.sf.k + (int64_t)hk * p.sf.stride_head;
    if (p.page_size > 0) pages = seq_pages(p.block_table, p.bt_stride, p.page_indptr, b, &npages);
    pg = load_page(0);
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) copy(i);
  }
  __device__ __forceinline__ int key0(int i) const { return begin + (warp + i * kWarps) * S::kKeys; }
  __device__ __forceinline__ int page_of(int j) const {
    const int pi = quot(j, pdiv);
    return (npages >= 0 && pi >= npages) ? -1 : __ldg(pages + pi);
  }
  __device__ __forceinline__ int load_page(int i) const {
    const int j = key0(i) + lane % S::kKeys;
    if (p.page_size == 0) return b;
    return i < mine && j < end ? page_of(j) : 0;
  }
  // starts the copy of step i, the next one (lanes of a warp share a step's keys; rows past
  // the range, or of a bad page, become zeros)
  __device__ __forceinline__ void copy(int i) {
    const int pg_i = pg;
    pg = load_page(i + 1);
    if (i < mine) {
      uint8_t* st = ring + (i % NS) * S::kStage;
      const int kl = lane % S::kKeys, j = key0(i) + kl;
      const int slot = p.page_size > 0 ? j - quot(j, pdiv) * p.page_size : j;
      const bool ok = j < end && (uint32_t)pg_i < (uint32_t)p.num_pages;
      const int64_t off = ok ? (int64_t)pg_i * p.c_stride_page + (int64_t)slot * p.c_stride_tok : -1;
#pragma unroll
      for (int k = 0; k < S::kKeys * R::kPieces / 32; ++k) {
        const int r = (lane + 32 * k) / R::kPieces, c = (lane + 32 * k) % R::kPieces;
        const int64_t o = __shfl_sync(0xffffffffu, off, r);
        async_copy<16>(st + S::off(r, c), kc + (o < 0 ? 0 : o + c * 16), o < 0 ? 0u : 16u);
      }
      if constexpr (R::kSf > 0) {
        const int64_t soff = ok ? (int64_t)pg_i * p.sf.stride_page + (int64_t)slot * p.sf.stride_tok : 0;
        async_copy<R::kSf>(st + S::kKeys * R::kBytes + kl * R::kSf, ks + soff, ok ? R::kSf : 0u);
      }
    }
    cp_async_commit();
  }
  // waits for step i and starts the copy of step i + NS - 1
  __device__ __forceinline__ void next(int i) {
    cp_async_wait_group<NS - 2>();
    __syncwarp();  // every lane's pieces of step i; and every lane has read step i - 1
    copy(i + NS - 1);
  }
  // row 16x + 8h + lane / 4 of step i as operand pairs
  __device__ __forceinline__ void row(int i, int x, int h, uint32_t* w) const {
    const uint32_t st = smem_u32(ring + (i % NS) * S::kStage);
    const int r = 16 * x + 8 * h + (lane >> 2);
    const uint32_t sfa = st + S::kKeys * R::kBytes + r * R::kSf;
    R::load(
        lane & 3, w, [&](int c) { return lds_u128(st + S::off(r, c)); },
        [&](int c) {
          uint2 v;
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(st + r * R::kBytes + c * 8));
          return v;
        },
        [&](int c) {
          uint32_t v;
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(sfa + c));
          return v;
        },
        [&](int c) {
          uint16_t v;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(sfa + c));
          return (uint32_t)v;
        });
  }
};

// The scores of a step: lane (g, t) has key 8t + g of it (16 keys: t < 2).
template <int KEYS>
struct Sums {
  float* out;
  const float* in;
  int ko;
  float was = 0.f, ahead = 0.f;
  __device__ __forceinline__ Sums(const WeightsParams& p, int b, int hk) {
    const int64_t at = (int64_t)b * p.s_stride_seq + (int64_t)hk * p.s_stride_head;
    out = p.scores + at;
    in = p.scores_in != nullptr ? p.scores_in + at : nullptr;
    const int lane = threadIdx.x & 31;
    ko = 8 * (lane & 3) + (lane >> 2);
  }
  template <class K>
  __device__ __forceinline__ void load(const K& k, int i) {  // what step i's sums are added to
    const int j = k.key0(i) + ko;
    ahead = in != nullptr && ko < KEYS && i < k.mine && j < k.end ? in[j] : 0.f;
  }
  // sum[x][h]: this lane's part of key 16x + 8h + g; the four lanes of a key add theirs
  template <class K>
  __device__ __forceinline__ void store(const K& k, int i, const float (*sum)[2]) {
    float mine = 0.f;
#pragma unroll
    for (int x = 0; x < KEYS / 16; ++x)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = sum[x][h];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if ((threadIdx.x & 3) == 2 * x + h) mine = v;
      }
    const int j = k.key0(i) + ko;
    if (ko >= KEYS || j >= k.end) return;
    if (k.p.page_size > 0) {
      const int pg = k.page_of(j);
      if (pg < 0 || pg >= k.p.num_pages) {
        record_status(k.p.status, PKV_ERR_DEVICE_BOUNDS, k.b, pg);
        return;
      }
    }
    out[j] = mine + was;
  }
};

template <int D, int DT, int NQ>
__global__ void __launch_bounds__(kThreads, D == 256 || NQ == 2 ? 2 : 3)
    weights_stream_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ FastDiv pdiv, int chunk) {
  using R = Row<D, DT>;
  using S = Stream<D, DT>;
  constexpr int MT = S::kKeys / 16;
  constexpr int W = R::kWords;
  extern __shared__ __align__(128) uint8_t smem[];
  const int b = blockIdx.z, hk = blockIdx.y;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Seq s = load_seq(p, b, blockIdx.x == 0 && threadIdx.x == 0);
  const int begin = blockIdx.x * chunk, end = min(s.lk, begin + chunk);
  if (!s.ok || begin >= end) return;
  KeyRing<D, DT, S::kStages> keys(p, pdiv, smem, b, hk, begin, end);
  Sums<S::kKeys> sums(p, b, hk);
  sums.load(keys, 0);

  const float sl2 = p.scale_log2 * (p.k_scale != nullptr ? __ldg(p.k_scale) : 1.f);
  uint32_t qw[NQ][W];
  float l2[NQ][2], sl2r[NQ][2];
  int lim[NQ][2];
#pragma unroll
  for (int j = 0; j < NQ; ++j) {
    const __nv_bfloat16* qr = query_row(p, s, hk, 8 * j + g);
    uint4 v[W / 4];
#pragma unroll
    for (int c = 0; c < W / 4; ++c) v[c] = query8(qr, R::dim(c, t));
    sl2r[j][0] = sl2r[j][1] = sl2;
    if constexpr (DT != PKV_BF16) {
      uint32_t most = 0;
#pragma unroll
      for (int c = 0; c < W / 4; ++c) most = most8(v[c], most);
      const RowScale scale(most_of_row(most));
#pragma unroll
      for (int c = 0; c < W / 4; ++c) v[c] = f16x8(v[c], scale);
#pragma unroll
      for (int e = 0; e < 2; ++e) sl2r[j][e] *= __shfl_sync(0xffffffffu, scale.down(), 4 * (2 * t + e));
    }
#pragma unroll
    for (int c = 0; c < W / 4; ++c)
      qw[j][4 * c] = v[c].x, qw[j][4 * c + 1] = v[c].y, qw[j][4 * c + 2] = v[c].z, qw[j][4 * c + 3] = v[c].w;
    row_info(p, s, hk, 8 * j + 2 * t, l2[j][0], lim[j][0]);
    row_info(p, s, hk, 8 * j + 2 * t + 1, l2[j][1], lim[j][1]);
  }

  for (int i = 0; i < keys.mine; ++i) {
    keys.next(i);
    sums.was = sums.ahead;
    sums.load(keys, i + 1);
    const int t0 = keys.key0(i);
    float sum[MT][2];
#pragma unroll
    for (int x = 0; x < MT; ++x) {
      uint32_t kw[2][W];
      keys.row(i, x, 0, kw[0]);
      keys.row(i, x, 1, kw[1]);
      sum[x][0] = sum[x][1] = 0.f;
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < W; k += 2) mma<DT>(c, kw[0] + k, kw[1] + k, qw[j] + k);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w = ex2(fmaf(c[2 * h + e], sl2r[j][e], -l2[j][e]));
            sum[x][h] += t0 + 16 * x + 8 * h + g < lim[j][e] ? w : 0.f;
          }
      }
    }
    sums.store(keys, i, sum);
  }
  cp_async_wait_group<0>();
}

// ------------------------------------------------------------------ many rows
template <int D, int DT>
struct Many {
  static constexpr int kRows = D == 256 ? 64 : 128;  // query rows in shared memory at a time
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kStages = 2;
  static constexpr int kBytes = kQ + kWarps * kStages * Stream<D, DT>::kStage;
};

template <int D, int DT>
__global__ void __launch_bounds__(kThreads, D == 256 ? 2 : 3)
    weights_rows_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ FastDiv pdiv, int chunk) {
  using R = Row<D, DT>;
  using S = Stream<D, DT>;
  using L = Many<D, DT>;
  constexpr int MT = S::kKeys / 16, W = R::kWords;
  extern __shared__ __align__(128) uint8_t smem[];
  // of two rows each: their log2-domain LSEs, and the scales of their logits
  __shared__ __align__(16) float4 s_row[L::kRows / 2];
  __shared__ __align__(8) int s_lim[L::kRows];
  uint4* qs = reinterpret_cast<uint4*>(smem);  // [tile of 8 rows][W / 4][lane]
  const int b = blockIdx.z, hk = blockIdx.y;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Seq s = load_seq(p, b, blockIdx.x == 0 && threadIdx.x == 0);
  const int begin = blockIdx.x * chunk, end = min(s.lk, begin + chunk);
  if (!s.ok || begin >= end) return;
  KeyRing<D, DT, L::kStages> keys(p, pdiv, smem + L::kQ, b, hk, begin, end);
  Sums<S::kKeys> sums(p, b, hk);
  sums.load(keys, 0);
  const float sl2 = p.scale_log2 * (p.k_scale != nullptr ? __ldg(p.k_scale) : 1.f);

  // rows r0 .. r0 + n - 1 into shared memory, in the order of the operand, a warp eight rows at a
  // time; every load of a thread's in flight at once
  auto stage = [&](int r0, int n) {
    constexpr int kEach = L::kRows / 8 / kWarps;  // tiles of eight rows a warp
    const int tile0 = threadIdx.x >> 5;
    uint4 v[kEach][W / 4];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int tile = tile0 + k * kWarps;
      const __nv_bfloat16* qr = 8 * tile < n ? query_row(p, s, hk, r0 + 8 * tile + g) : nullptr;
#pragma unroll
      for (int c = 0; c < W / 4; ++c) v[k][c] = query8(qr, R::dim(c, t));
    }
    for (int i = threadIdx.x; i < L::kRows; i += kThreads) {
      float* row = reinterpret_cast<float*>(&s_row[i >> 1]) + (i & 1);
      row_info(p, s, hk, r0 + i, row[0], s_lim[i]);
      if constexpr (DT == PKV_BF16) row[2] = sl2;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int tile = tile0 + k * kWarps;
      if constexpr (DT != PKV_BF16) {
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < W / 4; ++c) most = most8(v[k][c], most);
        const RowScale scale(most_of_row(most));
#pragma unroll
        for (int c = 0; c < W / 4; ++c) v[k][c] = f16x8(v[k][c], scale);
        if (t == 0) reinterpret_cast<float*>(&s_row[4 * tile + (g >> 1)])[2 + (g & 1)] = sl2 * scale.down();
      }
#pragma unroll
      for (int c = 0; c < W / 4; ++c) qs[(tile * (W / 4) + c) * 32 + lane] = v[k][c];
    }
  };
  const bool once = s.rows <= L::kRows;
  if (once) {
    stage(0, s.rows);
    __syncthreads();
  }
  // every warp takes part in every step (the barriers), with keys or without
  const int steps = (end - begin + kWarps * S::kKeys - 1) / (kWarps * S::kKeys);
  for (int i = 0; i < steps; ++i) {
    keys.next(i);
    sums.was = sums.ahead;
    sums.load(keys, i + 1);
    const int t0 = keys.key0(i);
    uint32_t kw[MT][2][W];
    float sum[MT][2];
    if (i < keys.mine) {
#pragma unroll
      for (int x = 0; x < MT; ++x) {
        keys.row(i, x, 0, kw[x][0]);
        keys.row(i, x, 1, kw[x][1]);
        sum[x][0] = sum[x][1] = 0.f;
      }
    }
    for (int r0 = 0; r0 < s.rows; r0 += L::kRows) {
      const int n = min(L::kRows, s.rows - r0);
      if (!once) {
        // (causal: rows whose last query does not reach this step's keys)
        if (p.causal && s.first + (r0 + n - 1) / p.G + s.lk - s.lq < begin + i * kWarps * S::kKeys) continue;
        __syncthreads();
        stage(r0, n);
        __syncthreads();
      }
      if (i >= keys.mine) continue;
      const int tiles = (n + 7) / 8;
#pragma unroll 2
      for (int j = 0; j < tiles; ++j) {
        uint32_t qw[W];
#pragma unroll
        for (int c = 0; c < W / 4; ++c) {
          const uint4 v = qs[(j * (W / 4) + c) * 32 + lane];
          qw[4 * c] = v.x, qw[4 * c + 1] = v.y, qw[4 * c + 2] = v.z, qw[4 * c + 3] = v.w;
        }
        const float4 row = s_row[4 * j + t];
        const int2 lim = *reinterpret_cast<const int2*>(&s_lim[8 * j + 2 * t]);
        float c[MT][4];
#pragma unroll
        for (int x = 0; x < MT; ++x) c[x][0] = c[x][1] = c[x][2] = c[x][3] = 0.f;
#pragma unroll
        for (int k = 0; k < W; k += 2)
#pragma unroll
          for (int x = 0; x < MT; ++x) mma<DT>(c[x], kw[x][0] + k, kw[x][1] + k, qw + k);
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = t0 + 16 * x + 8 * h + g;
            const float w0 = ex2(fmaf(c[x][2 * h], row.z, -row.x)), w1 = ex2(fmaf(c[x][2 * h + 1], row.w, -row.y));
            sum[x][h] += key < lim.x ? w0 : 0.f;
            sum[x][h] += key < lim.y ? w1 : 0.f;
          }
      }
    }
    if (i < keys.mine) sums.store(keys, i, sum);
  }
  cp_async_wait_group<0>();
}

// Dynamic shared memory of a kernel, set once per device (kept out of the launch path,
// so the call can be captured in a graph).
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (configured.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) configured.fetch_or(bit);
  return e;
}

// Keys of a block: up to `most` steps a warp, fewer while that leaves under four blocks an SM.
// Few rows take eight (four the same, two 57 in place of 51 us on the decode batch), many rows
// four: their blocks are long, and the last wave of them is shorter (the window of 32 queries:
// 82 us with eight, 81 with five, 77.5 with four, 88 with two, whose queries are staged too often).
int block_keys(const WeightsParams& p, int step, int most) {
  int chunk = most * step;
  while (chunk > step && (int64_t)p.batch * p.hkv * ((p.max_seqlen_k + chunk - 1) / chunk) < 4 * 152) chunk /= 2;
  return chunk;
}

template <int D, int DT, int NQ>
cudaError_t launch_stream(const WeightsParams& p, const FastDiv& f, cudaStream_t stream) {
  using S = Stream<D, DT>;
  cudaError_t e = allow_smem<weights_stream_kernel<D, DT, NQ>>(S::kBytes);
  if (e != cudaSuccess) return e;
  const int chunk = block_keys(p, kWarps * S::kKeys, 8);
  const dim3 grid((unsigned)((p.max_seqlen_k + chunk - 1) / chunk), (unsigned)p.hkv, (unsigned)p.batch);
  weights_stream_kernel<D, DT, NQ><<<grid, kThreads, S::kBytes, stream>>>(p, f, chunk);
  return cudaGetLastError();
}

template <int D, int DT>
cudaError_t launch_t(const WeightsParams& p, cudaStream_t stream) {
  const FastDiv f = fast_div(p.page_size > 0 ? p.page_size : 1);
  const int64_t rows = (int64_t)(p.last_queries > 0 ? std::min(p.last_queries, p.max_seqlen_q) : p.max_seqlen_q) * p.G;
  if (rows <= 8) return launch_stream<D, DT, 1>(p, f, stream);
  if constexpr (D <= 128) {
    if (rows <= 16) return launch_stream<D, DT, 2>(p, f, stream);
  }
  using L = Many<D, DT>;
  cudaError_t e = allow_smem<weights_rows_kernel<D, DT>>(L::kBytes);
  if (e != cudaSuccess) return e;
  const int chunk = block_keys(p, kWarps * Stream<D, DT>::kKeys, 4);
  const dim3 grid((unsigned)((p.max_seqlen_k + chunk - 1) / chunk), (unsigned)p.hkv, (unsigned)p.batch);
  weights_rows_kernel<D, DT><<<grid, kThreads, L::kBytes, stream>>>(p, f, chunk);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const WeightsParams& p, int cache_dtype, cudaStream_t stream) {
  if (cache_dtype == PKV_FP4_E2M1) return launch_t<D, PKV_FP4_E2M1>(p, stream);
  if (cache_dtype == PKV_FP8_E4M3) return launch_t<D, PKV_FP8_E4M3>(p, stream);
  return launch_t<D, PKV_BF16>(p, stream);
}

}  // namespace

cudaError_t launch_weights(const WeightsParams& p, int head_dim, int cache_dtype, cudaStream_t stream) {
  if (p.batch == 0 || p.max_seqlen_k == 0) return cudaSuccess;
  return head_dim == 256   ? launch_d<256>(p, cache_dtype, stream)
         : head_dim == 128 ? launch_d<128>(p, cache_dtype, stream)
                           : launch_d<64>(p, cache_dtype, stream);
}

}  // namespace pkv
