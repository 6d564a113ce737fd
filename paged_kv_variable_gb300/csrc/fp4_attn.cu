// Attention over a 4-bit cache: the tiles of a few query rows (8, 16 or 32 at
// head_dim 256, 128 or 64: decode steps, drafted tokens, wide head groups in pieces).
//
// One block of four warps per work item (sequence, kv head, rows, a range of keys);
// the warps take every fourth step of 32 keys, each with a ring of its own in shared
// memory (cp.async, so no warp waits for another and none spins), and merge their sums
// once at the end.  A step is computed transposed, as the other caches' decode tiles
// are: S^T = K Q^T and O^T += V^T P^T with keys and dims on the 16-row side of m16n8k16
// MMAs and the query rows on the 8-column side.
//
// Codes become f16 (e2m1 and e4m3 are subsets, and their product has six
// significant bits: exact) in registers:
//  - K: a dot product does not depend on the order of the dims, so lane (g, t)
//    takes dims 32t .. 32t+31 of key row g in one 16-byte load, each scale once
//    for 16 codes, and the queries are laid out to match.
//  - V: lane (g, t) takes dims (D/8) g .. of four keys; the nibbles of a key pair
//    are interleaved before the conversion, which then gives both keys of a dim
//    in one register, as the MMA wants them.  Rows of O^T are whatever dims fell
//    there; the output is put in order by the merge.
// k_scale goes into the logits' scale, v_scale into the output.  Logits, softmax
// sums and O are fp32; P is rounded to f16 (11 bits), kept above the subnormals
// by a factor 64.
//
// About 635 instructions of a warp for 32 keys at head_dim 128, most of them conversions,
// products with the scales and the interleave.  No unit is near its limit (64 sequences of 512
// to 4096 keys, 8 kv heads, 166 MB: issue slots 57%, ALU 47%, DRAM 53%, FMA 33%, warp MMAs
// 22%): a step is a chain of them, and four warps a scheduler, what the registers allow, wait
// for one another's results (1.6 warps at a fixed latency for each issue).  45 us with the
// combine; two sequences of 131072 keys 64.5 us (4.7 TB/s).
#include <cuda_bf16.h>

#include <atomic>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 32;    // keys of a step
constexpr int kStages = 2;   // steps in a warp's ring
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kPExp = 6.f;  // P = 2^(logit - max + kPExp), so that P <= 2^14 while the max is not moved

template <int D>
struct Fp4Layout {
  static constexpr int kRow = D / 2;            // bytes of a row's codes
  static constexpr int kChunks = kRow / 16;     // 16-byte pieces of it
  static constexpr int kSf = D / kFp4Block;     // bytes of its scales
  static constexpr int kKOff = 0;
  static constexpr int kVOff = kStep * kRow;
  static constexpr int kKsOff = 2 * kStep * kRow;
  static constexpr int kVsOff = kKsOff + kStep * kSf;
  static constexpr int kStage = kVsOff + kStep * kSf;
  static constexpr int kRing = kStages * kStage;  // of a warp
  // the rings, or what the warps merge through them
  static PKV_HOST_DEVICE constexpr int bytes(int nq) {
    return kWarps * kRing > kWarps * nq * D * 32 ? kWarps * kRing : kWarps * nq * D * 32;
  }
  // Keys 0..7 of an MMA's key rows sit at rows 0 4 1 5 2 6 3 7 of the step's eight,
  // so that a key pair of V is rows (t, t + 4).  The pieces of a row are placed so
  // that the lanes that one shared-memory access serves at a time fall on
  // different banks: K reads rows (i, i + 4) together, V rows 0..3 or 4..7.
  static __device__ __forceinline__ uint32_t k_off(int r, int c) {
    if constexpr (D == 64) return (uint32_t)((r ^ (((r >> 2) & 1) << 1)) * 32 + c * 16);
    if constexpr (D == 128) return (uint32_t)((r ^ ((r >> 2) & 1)) * 64 + c * 16);
    return (uint32_t)(r * 128 + ((c ^ (((r >> 2) & 1) << 2)) << 4));
  }
  // what a row r0 on (a multiple of a copy's rows) changes in k_off besides its distance
  static __device__ __forceinline__ constexpr uint32_t k_flip(int r0) { return D == 256 && (r0 & 4) ? 64u : 0u; }
  static __device__ __forceinline__ uint32_t v_off(int r, int c) {
    if constexpr (D == 64) return (uint32_t)(r * 32 + c * 16);
    if constexpr (D == 128) return (uint32_t)(r * 64 + ((c ^ (((r >> 1) & 1) << 1)) << 4));
    return (uint32_t)(r * 128 + ((c ^ ((r & 3) << 1)) << 4));
  }
};

__device__ __forceinline__ int krow(int x) { return ((x & 1) << 2) | (x >> 1); }

template <int N>
__device__ __forceinline__ void cp_async_to(uint32_t dst, const void* src, uint32_t src_bytes) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(src_bytes)
                 : "memory");
}

// A step's 32 rows, and their scales, row by row: rows past the range, or of a bad page,
// become zeros.  key, pg: this lane's.  Out of line: the last step of a range, or pages
// that a copy's rows pass the end of.
template <int D>
__device__ __noinline__ void copy_ragged(const AttnParams& p, int64_t s_page, int64_t s_tok, int key, int pg, int kv_end,
                                         int seq, const uint8_t* k_rows, const uint8_t* v_rows, const uint8_t* ks,
                                         const uint8_t* vs, uint32_t k_dst, uint32_t v_dst, uint32_t s_dst,
                                         const FastDiv& pdiv) {
  using L = Fp4Layout<D>;
  const int lane = threadIdx.x & 31;
  const int slot = p.page_size > 0 ? key - quot(key, pdiv) * p.page_size : key;
  bool ok = key < kv_end;
  if (ok && (uint32_t)pg >= (uint32_t)p.num_pages) {
    record_status(p.status, PKV_ERR_DEVICE_BOUNDS, seq, pg);
    ok = false;
  }
  const int64_t off = ok ? (int64_t)pg * p.c_stride_page + (int64_t)slot * p.c_stride_tok : -1;
#pragma unroll
  for (int k = 0; k < L::kChunks; ++k) {
    const int64_t at = __shfl_sync(0xffffffffu, off, lane / L::kChunks + k * (32 / L::kChunks));
    const uint32_t n = at < 0 ? 0u : 16u;
    cp_async_to<16>((k_dst ^ L::k_flip(k * (32 / L::kChunks))) + k * 512, k_rows + (at < 0 ? 0 : at), n);
    cp_async_to<16>(v_dst + k * 512, v_rows + (at < 0 ? 0 : at), n);
  }
  const int64_t soff = ok ? (int64_t)pg * s_page + (int64_t)slot * s_tok : 0;
  cp_async_to<L::kSf>(s_dst, ks + soff, ok ? L::kSf : 0u);
  cp_async_to<L::kSf>(s_dst + kStep * L::kSf, vs + soff, ok ? L::kSf : 0u);
}

__device__ __forceinline__ uint2 lds_u64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, fp4_blocks(D, 8 * NQ))
    fp4_attn_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ Fp4Scales sf,
                    const __grid_constant__ FastDiv pdiv, const int runs) {
  using L = Fp4Layout<D>;
  constexpr int KS = D / 16;  // k-steps of S^T
  constexpr int DT = D / 16;  // m-tiles of O^T
  constexpr int KW = D / 32;  // 32-bit words of a lane's K codes a row
  constexpr int VW = D / 64;  // and of its V codes a key
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  grid_dep_launch();

  WorkItem w = p.items[blockIdx.x];
  if (p.q_offsets != nullptr) w.q_row0 = __ldg(p.q_offsets + w.b) + w.q_i0;
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.batch; b += kThreads) {
      const int lc = __ldg(p.cache_seqlens + b);
      if (lc > __ldg(p.plan_lc + b) || lc < __ldg(p.plan_lc + p.batch + b))
        record_status(p.status, PKV_ERR_PLAN_MISMATCH, b, lc);
    }
  }
  if (p.dynamic) {
    const int bound = __ldg(p.plan_lc + w.b);
    const int lc = min(max(__ldg(p.cache_seqlens + w.b), 0), bound);
    w.lk = w.lk - bound + lc;
    w.kv_end = min(w.kv_end, w.lk);
    w.kv_begin = min(w.kv_begin, w.kv_end);
  }
  const int R = w.n_q * w.nh;  // rows: token r / nh of the tile, head h0 + r % nh of the group
  const int head0 = w.hk * p.G + w.h0;

  // ------------------------------------------------------------------ this warp's steps
  const int steps = (w.kv_end - w.kv_begin + kStep - 1) / kStep;
  const int mine = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;
  int npages = -1;
  const int32_t* pages = nullptr;
  if (p.page_size > 0) pages = seq_pages(p.block_table, p.bt_stride, p.page_indptr, w.b, &npages);
  // page of this lane's key `key`
  auto load_page = [&](int key) -> int {
    if (p.page_size == 0) return w.b;
    if (key >= w.kv_end) return 0;
    const int pi = quot(key, pdiv);
    return (npages >= 0 && pi >= npages) ? -1 : __ldg(pages + pi);
  };
  // A copy of the warp covers 512 bytes of a step's rows: this lane's piece of the first one,
  // there and here, from which the others are 512 bytes on
  constexpr int kRows = 32 / L::kChunks;  // rows of a copy
  const int prow = lane / L::kChunks, piece = lane % L::kChunks;
  const int64_t lane_src = (int64_t)w.hk * p.c_stride_head + (int64_t)prow * p.c_stride_tok + piece * 16;
  const uint8_t* kl = static_cast<const uint8_t*>(p.kc) + lane_src;
  const uint8_t* vl = static_cast<const uint8_t*>(p.vc) + lane_src;
  const uint8_t* ks = sf.k + (int64_t)w.hk * sf.stride_head;
  const uint8_t* vs = sf.v + (int64_t)w.hk * sf.stride_head;
  const uint32_t ring = smem_u32(smem) + warp * L::kRing;
  const uint32_t k_dst = ring + L::kKOff + L::k_off(prow, piece);
  const uint32_t v_dst = ring + L::kVOff + L::v_off(prow, piece);
  const uint32_t s_dst = ring + L::kKsOff + lane * L::kSf;
  // the copies of the step that starts at this lane's key `key`, on its page pg, into stage `st`
  // (in bytes)
  auto issue = [&](int key, int pg, uint32_t st) {
    const bool whole = runs && __all_sync(0xffffffffu, key < w.kv_end && (uint32_t)pg < (uint32_t)p.num_pages);
    if (whole) {
      // every row is there and the rows of a copy are neighbours in one page: its first row's
      // offset (in 16 bytes) serves the warp
      const int slot = p.page_size > 0 ? key - quot(key, pdiv) * p.page_size : key;
      const uint32_t row = (uint32_t)pg * (uint32_t)(p.c_stride_page >> 4) + (uint32_t)slot * (uint32_t)(p.c_stride_tok >> 4);
      const uint32_t srow =
          (uint32_t)pg * (uint32_t)(sf.stride_page / L::kSf) + (uint32_t)slot * (uint32_t)(sf.stride_tok / L::kSf);
#pragma unroll
      for (int k = 0; k < L::kChunks; ++k) {
        const uint64_t at = (uint64_t)__shfl_sync(0xffffffffu, row, k * kRows) * 16;
        // (the swizzle's bit that the row's third decides)
        const uint32_t flip = L::k_flip(k * kRows);
        cp_async_to<16>((k_dst ^ flip) + k * 512 + st, kl + at, 16u);
        cp_async_to<16>(v_dst + k * 512 + st, vl + at, 16u);
      }
      cp_async_to<L::kSf>(s_dst + st, ks + (uint64_t)srow * L::kSf, L::kSf);
      cp_async_to<L::kSf>(s_dst + kStep * L::kSf + st, vs + (uint64_t)srow * L::kSf, L::kSf);
    } else {
      copy_ragged<D>(p, sf.stride_page, sf.stride_tok, key, pg, w.kv_end, w.b, kl - prow * p.c_stride_tok,
                     vl - prow * p.c_stride_tok, ks, vs, k_dst + st, v_dst + st, s_dst + st, pdiv);
    }
  };
  constexpr int kNext = kWarps * kStep;               // keys between a warp's steps
  const int key0 = w.kv_begin + warp * kStep + lane;  // this lane's key of its first step
  int pg = load_page(key0);
  {
    const int next = load_page(key0 + kNext);
    if (mine > 0) issue(key0, pg, 0);
    cp_async_commit();
    pg = next;
  }

  // ------------------------------------------------------------------ queries
  // Q^T (B operand): row 8j + g, dims as K's lanes have them, in f16
  uint32_t qb[NQ][KS][2];
  bool odd = false;  // some number is not an f16 number (of eight bits: 0, or from 2^-17 below 2^16)
#pragma unroll
  for (int j = 0; j < NQ; ++j) {
    const int r = 8 * j + g;
    const __nv_bfloat16* qr =
        r < R ? p.q + (int64_t)(w.q_row0 + r / w.nh) * p.q_stride_tok + (int64_t)(head0 + r % w.nh) * p.q_stride_head
              : nullptr;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {  // eight dims at a time
      const int d0 = D == 64 ? 16 * t + 8 * c : 32 * t + 8 * (c & 3) + 128 * (c >> 2);
      const uint4 v = qr ? __ldg(reinterpret_cast<const uint4*>(qr + d0)) : make_uint4(0, 0, 0, 0);
      qb[j][2 * c][0] = v.x, qb[j][2 * c][1] = v.y, qb[j][2 * c + 1][0] = v.z, qb[j][2 * c + 1][1] = v.w;
    }
    odd |= !f16_numbers(qb[j][0], 2 * KS);
  }
  // Then each row is taken times a power of two, which its logits take out again.  (In every tile
  // that took 1% more time on long sequences, 4 to 8% with tiles of 16 and 32 rows; of tiles of
  // normally distributed queries less than one in a hundred needs it.)
  __shared__ __align__(8) float downs[kWarps][8 * NQ];
  const bool scaled = __any_sync(0xffffffffu, odd);
  if (scaled) {
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      uint32_t most = 0;
#pragma unroll
      for (int k = 0; k < KS; ++k) most = bf16x2_most(qb[j][k][1], bf16x2_most(qb[j][k][0], most));
      const RowScale scale(most_of_row(most));
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) qb[j][k][e] = scale.times(qb[j][k][e]);
      if (t == 0) downs[warp][8 * j + g] = scale.down();
    }
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) qb[j][k][e] = bf16x2_to_f16x2(qb[j][k][e]);
  // keys that this lane's query rows (columns 2t, 2t + 1 of S^T) see
  int lim[NQ][2];
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * j + 2 * t + e;
      lim[j][e] = w.kv_begin;
      if (r < R) {
        lim[j][e] = w.kv_end;
        if (p.causal) lim[j][e] = min(w.kv_end, w.q_i0 + r / w.nh + w.lk - w.lq + 1);
      }
    }
  // keys that every row (of those that there are) sees
  int all_see = w.kv_end;
  if (p.causal) all_see = min(all_see, w.q_i0 + w.lk - w.lq + 1);
  const float sl2 = p.scale_log2 * __ldg(p.k_scale);
  const float vscale = __ldg(p.v_scale);

  float o[NQ][DT][4];
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[j][dt][0] = o[j][dt][1] = o[j][dt][2] = o[j][dt][3] = 0.f;
  float m[NQ][2], l[NQ][2];
#pragma unroll
  for (int j = 0; j < NQ; ++j) m[j][0] = m[j][1] = -INFINITY, l[j][0] = l[j][1] = 0.f;

  // this lane's place in a step: K rows krow(g) (and 8, 16, 24 on), V rows t and t + 4, and the
  // scales of each
  const uint32_t k_at = ring + L::kKOff + (D == 64 ? L::k_off(krow(g), t >> 1) + (t & 1) * 8 : L::k_off(krow(g), t));
  const uint32_t ks_at = ring + L::kKsOff + krow(g) * L::kSf + (D == 64 ? t : 2 * t);
  const uint32_t v_at = ring + L::kVOff +
                        (D == 64    ? L::v_off(t, g >> 2) + (g & 3) * 4
                         : D == 128 ? L::v_off(t, g >> 1) + (g & 1) * 8
                                    : L::v_off(t, g));
  const uint32_t vs_at = ring + L::kVsOff + t * L::kSf + (D == 64 ? g >> 1 : D == 128 ? g : 2 * g);
  int key = key0;
  uint32_t st = 0;  // the step's ring stage, in bytes
  for (int i = 0; i < mine; ++i, key += kNext, st ^= L::kStage) {
    cp_async_wait_group<0>();
    __syncwarp();  // every lane's pieces of step i; and every lane has read step i - 1
    if (i + 1 < mine) {
      const int next = load_page(key + 2 * kNext);
      issue(key + kNext, pg, st ^ L::kStage);
      pg = next;
    }
    cp_async_commit();
    const int t0 = key - lane;

    // S^T = K Q^T
    float s[NQ][2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int j = 0; j < NQ; ++j) s[j][x][0] = s[j][x][1] = s[j][x][2] = s[j][x][3] = 0.f;
      uint32_t kw[2][KW], ksc[2][KW / 2];  // codes; each word pair's scale, twice a register
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * x + 8 * h;  // (of the rows krow(g) on; eight rows on, the swizzle is the same)
        if constexpr (D == 64) {
          const uint2 v = lds_u64(k_at + st + r * L::kRow);
          kw[h][0] = v.x, kw[h][1] = v.y;
          const uint32_t c = e4m3x2_to_f16x2(lds_u8(ks_at + st + r * L::kSf));
          ksc[h][0] = prmt(c, 0u, 0x1010u);
        } else {
#pragma unroll
          for (int c = 0; c < D / 128; ++c) {
            const uint4 v = lds_u128((c == 0 ? k_at : k_at ^ 64u) + st + r * L::kRow);
            kw[h][4 * c] = v.x, kw[h][4 * c + 1] = v.y, kw[h][4 * c + 2] = v.z, kw[h][4 * c + 3] = v.w;
            const uint32_t f = e4m3x2_to_f16x2(lds_u16(ks_at + st + r * L::kSf + 8 * c));
            ksc[h][2 * c] = prmt(f, 0u, 0x1010u);
            ksc[h][2 * c + 1] = prmt(f, 0u, 0x3232u);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < KW; ++c) {
        uint32_t a[4], b[4];
        e2m1x8_to_f16(kw[0][c], a);
        e2m1x8_to_f16(kw[1][c], b);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = mul_f16x2(a[k], ksc[0][c >> 1]);
          b[k] = mul_f16x2(b[k], ksc[1][c >> 1]);
        }
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
          mma_f16(s[j][x], a[0], b[0], a[1], b[1], qb[j][2 * c][0], qb[j][2 * c][1]);
          mma_f16(s[j][x], a[2], b[2], a[3], b[3], qb[j][2 * c + 1][0], qb[j][2 * c + 1][1]);
        }
      }
    }

    if (scaled) {
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        const float2 d = *reinterpret_cast<const float2*>(&downs[warp][8 * j + 2 * t]);
#pragma unroll
        for (int x = 0; x < 2; ++x) s[j][x][0] *= d.x, s[j][x][1] *= d.y, s[j][x][2] *= d.x, s[j][x][3] *= d.y;
      }
    }

    // mask (select, never add; steps that every row sees whole need none) and online
    // softmax in the log2 domain; the max moves only when it grows by more than 2^8
    const bool mask = t0 + kStep > all_see;
    bool moved = false;
    float al[NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[j][x][c] *= sl2;
      if (mask) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int ka = t0 + 16 * x + krow(g), kb = ka + 8;
          if (ka >= lim[j][0]) s[j][x][0] = -INFINITY;
          if (ka >= lim[j][1]) s[j][x][1] = -INFINITY;
          if (kb >= lim[j][0]) s[j][x][2] = -INFINITY;
          if (kb >= lim[j][1]) s[j][x][3] = -INFINITY;
        }
      }
      float mx[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        mx[e] = fmaxf(fmax3(s[j][0][e], s[j][0][2 + e], s[j][1][e]), s[j][1][2 + e]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 8));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
        const bool bump = mx[e] > m[j][e] + 8.f;
        const float mn = bump ? mx[e] : m[j][e];
        al[j][e] = bump ? ex2(m[j][e] - mn) : 1.f;
        m[j][e] = mn;
        moved |= bump;
        const float mu = mn == -INFINITY ? 0.f : mn - kPExp;
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          s[j][x][e] = ex2(s[j][x][e] - mu);
          s[j][x][2 + e] = ex2(s[j][x][2 + e] - mu);
          sum += s[j][x][e] + s[j][x][2 + e];
        }
        l[j][e] = l[j][e] * al[j][e] + sum;
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          o[j][dt][0] *= al[j][0];
          o[j][dt][1] *= al[j][1];
          o[j][dt][2] *= al[j][0];
          o[j][dt][3] *= al[j][1];
        }
    }

    // O^T += V^T P^T
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t pb[NQ][2];
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        pb[j][0] = movm_t(pack_f16(s[j][x][0], s[j][x][1]));
        pb[j][1] = movm_t(pack_f16(s[j][x][2], s[j][x][3]));
      }
      // keys 2t, 2t + 1 (rows t, t + 4) and those 8 on: codes, and the pair's scales
      uint32_t vw[2][2][VW], vsc[2][(VW + 1) / 2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 16 * x + 8 * h + 4 * e;  // (of the rows t on)
          if constexpr (D == 64) {
            vw[h][e][0] = lds_u32(v_at + st + r * L::kRow);
            f[e] = lds_u8(vs_at + st + r * L::kSf);
          } else if constexpr (D == 128) {
            const uint2 v = lds_u64(v_at + st + r * L::kRow);
            vw[h][e][0] = v.x, vw[h][e][1] = v.y;
            f[e] = lds_u8(vs_at + st + r * L::kSf);
          } else {
            const uint4 v = lds_u128(v_at + st + r * L::kRow);
            vw[h][e][0] = v.x, vw[h][e][1] = v.y, vw[h][e][2] = v.z, vw[h][e][3] = v.w;
            f[e] = lds_u16(vs_at + st + r * L::kSf);
          }
        }
        vsc[h][0] = e4m3x2_to_f16x2(prmt(f[0], f[1], 0x7740u));
        if constexpr (VW == 4) vsc[h][1] = e4m3x2_to_f16x2(prmt(f[0], f[1], 0x7751u));
      }
#pragma unroll
      for (int c = 0; c < VW; ++c) {
        uint32_t a[2][4], b[2][4];  // even and odd dims of the word
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u = vw[h][0][c], v = vw[h][1][c];
          e2m1x8_to_f16((u & 0x0F0F0F0Fu) | ((v << 4) & 0xF0F0F0F0u), a[h]);
          e2m1x8_to_f16(((u >> 4) & 0x0F0F0F0Fu) | (v & 0xF0F0F0F0u), b[h]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            a[h][k] = mul_f16x2(a[h][k], vsc[h][c >> 1]);
            b[h][k] = mul_f16x2(b[h][k], vsc[h][c >> 1]);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < NQ; ++j)
            mma_f16(o[j][4 * c + k], a[0][k], b[0][k], a[1][k], b[1][k], pb[j][0], pb[j][1]);
      }
    }
  }
  cp_async_wait_group<0>();

  // ------------------------------------------------------------------ merge of the warps
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], 4);
      l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], 8);
      l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], 16);
    }
  __shared__ float ml[kWarps][8 * NQ][2];
  if (g == 0) {
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ml[warp][8 * j + 2 * t + e][0] = m[j][e];
        ml[warp][8 * j + 2 * t + e][1] = l[j][e];
      }
  }
  __syncthreads();  // the rings are no longer read
  constexpr int kFrag = NQ * DT * 32;  // float4 of a warp's O^T
  static_assert(kWarps * kFrag * 16 <= L::bytes(NQ), "the warps' sums fit");
  float4* buf = reinterpret_cast<float4*>(smem);
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
      buf[warp * kFrag + (j * DT + dt) * 32 + lane] = make_float4(o[j][dt][0], o[j][dt][1], o[j][dt][2], o[j][dt][3]);
  __syncthreads();
  // a thread: eight dims of a row.  Dim d of row 8j + 2t + e is in m-tile (d % (D/8)) / 2,
  // lane 4 (d / (D/8)) + t, component e + 2 (d % 2)
  for (int idx = threadIdx.x; idx < R * (D / 8); idx += kThreads) {
    const int row = idx / (D / 8), d0 = (idx % (D / 8)) * 8;
    float M = -INFINITY;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) M = fmaxf(M, ml[x][row][0]);
    const float mu = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const float f = ex2(ml[x][row][0] - mu);
      sum += f * ml[x][row][1];
      const float* src = reinterpret_cast<const float*>(
          buf + x * kFrag + ((row >> 3) * DT + (d0 % (D / 8)) / 2) * 32 + 4 * (d0 / (D / 8)) + ((row & 7) >> 1));
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += f * src[(k >> 1) * 128 + (row & 1) + 2 * (k & 1)];
    }
    const float inv = sum > 0.f ? vscale / sum : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= inv;
    const float lse2 = sum > 0.f ? mu - kPExp + __log2f(sum) : -INFINITY;
    if (w.partial >= 0) {
      float* dst = p.partial_o + ((int64_t)w.partial * kDecodeRows + row) * D + d0;
      *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
      if (d0 == 0) p.partial_lse[(int64_t)w.partial * kDecodeRows + row] = lse2;
    } else {
      const int tok = w.q_row0 + row / w.nh, head = head0 + row % w.nh;
      *reinterpret_cast<uint4*>(p.out + (int64_t)tok * p.o_stride_tok + (int64_t)head * p.o_stride_head + d0) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      if (d0 == 0 && p.lse != nullptr) p.lse[(int64_t)head * p.total_q + tok] = lse2 * kLn2;
    }
  }
}

template <int D, int NQ>
cudaError_t launch_t(const AttnParams& p, const Fp4Scales& sf, int num_items, int capacity, cudaStream_t s) {
  using L = Fp4Layout<D>;
  // once per device (kept out of the launch path, so the call can be captured in a graph)
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(fp4_attn_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes(NQ));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  // rows of a copy (16, 8 or 4 of them) lie in one page, and offsets in 16 bytes (in a
  // row's scales) fit 32 bits
  const auto fits = [&](int64_t page, int64_t tok, int64_t unit) {
    return (p.num_pages * page + (p.page_size > 0 ? p.page_size : capacity) * tok) / unit <= UINT32_MAX;
  };
  const int runs = (p.page_size == 0 || p.page_size % (32 / L::kChunks) == 0) && fits(p.c_stride_page, p.c_stride_tok, 16) &&
                   fits(sf.stride_page, sf.stride_tok, L::kSf);
  fp4_attn_kernel<D, NQ><<<(unsigned)num_items, kThreads, L::bytes(NQ), s>>>(
      p, sf, fast_div(p.page_size > 0 ? p.page_size : 1), runs);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_attention(const AttnParams& p, const Fp4Scales& sf, int num_items, int max_rows, int capacity,
                                 int head_dim, cudaStream_t stream) {
  if (num_items == 0) return cudaSuccess;
  if (head_dim == 256) return launch_t<256, 1>(p, sf, num_items, capacity, stream);
  if (head_dim == 128)
    return max_rows <= 8 ? launch_t<128, 1>(p, sf, num_items, capacity, stream)
                         : launch_t<128, 2>(p, sf, num_items, capacity, stream);
  return max_rows <= 8    ? launch_t<64, 1>(p, sf, num_items, capacity, stream)
         : max_rows <= 16 ? launch_t<64, 2>(p, sf, num_items, capacity, stream)
                          : launch_t<64, 4>(p, sf, num_items, capacity, stream);
}

}  // namespace pkv
