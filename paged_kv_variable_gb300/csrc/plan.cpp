// Host scheduling step: validation, prefill/decode classification, split-KV
// chunking and longest-processing-time assignment of tiles to persistent CTAs.
//
// flashinfer PR "[Refactor] Uniform PoDAttention API with Horizontal Fusion SMs
// Schedule": one persistent launch serves prefill and decode requests, the
// partition of SMs follows the KV-cache load (Key Changes 2), requests are
// classified by query length (Limitations: "qo_len > threshold"), and a zero
// KV length must not be rejected (the review's failing test).  flash-attention
// PR "Add flash_attn_varlen_func_with_kvcache", Limitation: a fixed
// num_splits = 1 hurts decode, so decode units are cut into KV chunks here.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <exception>
#include <functional>
#include <new>
#include <vector>

#include "internal.h"

namespace pkv {

namespace {

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct Tile {
  WorkItem item;
  double cost;
  bool prefix = false;  // over a shared prefix
};

// Groups of consecutive sequences whose first prefix_lens[g] tokens are the same.
struct SharedPrefixes {
  int32_t num_groups;
  const int32_t* starts;  // [num_groups + 1]
  const int32_t* prefix_lens;
  bool always;  // shared whether or not the time model says that it pays
};

// Consecutive sequences whose queries attend the same `keys` first keys in
// common tiles.
struct PrefixRun {
  int b0;         // first sequence (its pages are the ones read)
  int tokens;     // query tokens of all its sequences
  int64_t q_row;  // the first one's packed row
  int keys;       // shared keys, a whole number of pages
  bool dec;       // all rows in one warp-MMA tile
  int tq, tiles;  // query tokens a tile, tiles
  int per_item;   // tiles an item holds (two where an item's query tiles share its K/V tiles)
  int nchunks, chunk;
  int tile_slots;             // partial slots of a tile
  std::vector<int32_t> slot0;  // first partial slot of each kv head
};

// Per-key model costs (relative units): a decode key streams 2*D*esize bytes
// from HBM for one kv head; a prefill key costs one 128-row MMA step.  (The
// weight of a prefill key against a decode key was measured on the mixed
// prefill + decode batch: 0.418 ms at this weight, 0.440 at 0.7 of it, 0.426
// at 1.2 times and 0.442 at twice it; prefill-only batches do not move.)
double decode_cost(int keys, int d, int esize) { return 64.0 + keys * (2.0 * d * esize) / 512.0; }
double prefill_cost(int keys, int rows, int d) { return 256.0 + keys * (rows * d * 4.0) / 65536.0; }

// Time model (us) of the launches of a plan with shared prefixes, from
// measurements on a GB300: what the choice of SMs and chunks below balances.
struct TimeModel {
  double tile1, tile2;  // a tensor-core K/V tile of 128 keys, one and two query tiles
  // a decode CTA: bytes a us, us an item besides, least us an item; the GPU's bytes a us
  double rate, item, least, hbm;
  int cps;  // decode CTAs an SM
  int d;
  double key_bytes;
  TimeModel(int head_dim, bool fp8) : d(head_dim) {
    if (fp8) {
      tile1 = d == 64 ? 2.0 : d == 128 ? 3.0 : 4.0;
      tile2 = d == 64 ? 2.6 : 3.8;
      rate = d == 64 ? 19e3 : d == 128 ? 28e3 : 43e3;
      item = d == 64 ? 1.4 : 3.0;
      least = d == 64 ? 2.3 : 3.7;
      hbm = d == 64 ? 4.6e6 : 5.4e6;
    } else {
      tile1 = tile2 = d == 64 ? 1.0 : d == 128 ? 1.1 : 2.2;
      rate = d == 64 ? 26e3 : d == 128 ? 57e3 : 49e3;
      item = d == 64 ? 1.0 : d == 128 ? 1.2 : 0.6;
      least = d == 64 ? 2.4 : d == 128 ? 2.8 : 3.5;
      hbm = 6.3e6;
    }
    cps = (fp8 ? d <= 128 : d == 64) ? 2 : 1;
    key_bytes = 2.0 * d * (fp8 ? 1 : 2);
  }
  static constexpr double kItemTc = 4.5;    // start and end of a tensor-core chunk

  // `keys` of decode work in `units` units, the longest of `longest` keys
  double decode(int64_t keys, int64_t units, int64_t longest, int sms) const {
    if (units == 0) return 0.0;
    if (sms <= 0) return HUGE_VAL;
    const double ctas = (double)sms * cps;
    const double chunk = std::max(512.0, (double)keys / (2.0 * sms));
    const double items = std::max((double)units, (double)keys / chunk);
    const double bytes = keys * key_bytes;
    const double each = std::max(least, item + bytes / items / rate);
    const double one = std::max(least, item + std::min((double)longest, chunk) * key_bytes / rate);
    return std::max({bytes / hbm, items * each / ctas, std::min(items, std::ceil(items / ctas)) * each * 0.9, one});
  }

  // the combine kernel: `rows` part rows of all units, `parts` of the unit with most
  double combine(double rows, int64_t parts) const {
    return 3.5 + (parts > 8 ? 0.03 : 0.1) * parts + rows * 2.0 * d * sizeof(float) / 5e6;
  }
};

// The decode work of a batch (with each sequence's first shared[b] keys taken out).
struct DecodeWork {
  int64_t keys = 0, units = 0, longest = 0;
  void add(int64_t n, int64_t count) {
    keys += n * count;
    units += count;
    longest = std::max(longest, n);
  }
};

// What a plan with shared prefixes takes by the model: SMs of the tensor-core
// tiles, keys a chunk of theirs, and the time.
struct SplitChoice {
  int sms_tc;
  int64_t chunk;
  double time;
};

SplitChoice choose_split(const pkv_problem& p, const std::vector<PrefixRun>& runs, const int32_t* q_lens,
                         const int32_t* cache_lens, const int32_t* new_lens, const int32_t* shared, int num_sms,
                         int n_sub, int tq, int dec_rows) {
  const int G = p.num_heads_q / p.num_heads_kv, D = p.head_dim;
  const TimeModel tm(D, p.cache_dtype == PKV_FP8_E4M3);
  DecodeWork dec;
  int64_t longest = 0;  // of the units that tensor-core tiles may cut
  double fixed = 0;     // tensor-core tiles that are not cut
  int64_t fixed_items = 0;
  std::vector<int64_t> cut;  // keys of each sequence whose tensor-core tiles may be cut
  double own_rows = 0;  // rows of the units in parts over their own keys
  for (const PrefixRun& r : runs) {
    if (r.dec)
      dec.add(r.keys, p.num_heads_kv);
    else
      longest = std::max<int64_t>(longest, r.keys);
  }
  for (int b = 0; b < p.batch; ++b) {
    const int lq = q_lens[b];
    if (lq == 0) continue;
    const int64_t keys = (int64_t)cache_lens[b] + (new_lens ? new_lens[b] : 0) - shared[b];
    if ((int64_t)lq * G <= dec_rows) {
      dec.add(keys, p.num_heads_kv);
    } else if (lq <= tq) {
      longest = std::max(longest, keys);
      cut.push_back(keys);
    } else {
      const int64_t n = (int64_t)p.num_heads_kv * n_sub * ((lq + tq - 1) / tq);
      fixed += n * (tm.kItemTc + keys / 128.0 * tm.tile1);
      fixed_items += n;
    }
    if (shared[b] > 0) own_rows += (double)lq * p.num_heads_q;
  }
  SplitChoice best{num_sms, 1 << 30, HUGE_VAL};
  for (int64_t k = 2;; k += std::max<int64_t>(1, k / 4)) {
    const int64_t ch = k * kKvTile;
    double sum = fixed, most = 0, rows = own_rows;
    int64_t items = fixed_items;
    auto add = [&](int64_t keys, int64_t n, double tile) {
      if (keys <= 0 || n <= 0) return;
      const int64_t c = (keys + ch - 1) / ch, each = ((keys + c - 1) / c + kKvTile - 1) / kKvTile;
      const double t = tm.kItemTc + each * tile;
      items += c * n;
      sum += c * n * t;
      most = std::max(most, t);
    };
    for (const PrefixRun& r : runs) {
      rows += (double)r.tokens * p.num_heads_q * (r.dec ? 1 : (r.keys + ch - 1) / ch);
      if (r.dec) continue;
      add(r.keys, (int64_t)p.num_heads_kv * (r.tiles / r.per_item), r.per_item == 2 ? tm.tile2 : tm.tile1);
      add(r.keys, (int64_t)p.num_heads_kv * (r.tiles % r.per_item), tm.tile1);
    }
    for (int64_t keys : cut) add(keys, (int64_t)p.num_heads_kv * n_sub, tm.tile1);
    auto consider = [&](int sms) {
      const double tc = items == 0 ? 0.0
                                   : std::max({most, sum / sms, (double)((items + sms - 1) / sms) * sum / items});
      const double t = std::max(tc, tm.decode(dec.keys, dec.units, dec.longest, items ? num_sms - sms : num_sms)) +
                       tm.combine(rows, (longest + ch - 1) / ch + 1);
      if (t < best.time) best = {sms, ch, t};
    };
    if (dec.units == 0 || items == 0 || num_sms < 2) {
      consider(num_sms);
    } else {
      for (int sms = std::max(1, num_sms / 38); sms < num_sms; sms += std::max(1, num_sms / 38)) consider(sms);
      if (items < num_sms) consider((int)items);
    }
    if (ch >= longest) break;
  }
  return best;
}

// The time of the batch planned without sharing, by the same model: one launch
// in which both kinds of tiles share every SM, units cut as make_plan cuts them.
double plain_time(const pkv_problem& p, const int32_t* q_lens, const int32_t* cache_lens, const int32_t* new_lens,
                  int num_sms, int n_sub, int tq, int dec_rows) {
  const int G = p.num_heads_q / p.num_heads_kv;
  const TimeModel tm(p.head_dim, p.cache_dtype == PKV_FP8_E4M3);
  DecodeWork dec;
  double split_keys = 0;
  bool any_tc = false;
  for (int b = 0; b < p.batch; ++b) {
    if (q_lens[b] == 0) continue;
    const int64_t keys = (int64_t)cache_lens[b] + (new_lens ? new_lens[b] : 0);
    const bool d = (int64_t)q_lens[b] * G <= dec_rows;
    if (d) dec.add(keys, p.num_heads_kv);
    any_tc |= !d;
    if (d || q_lens[b] <= tq) split_keys += (double)keys * p.num_heads_kv * (d ? 1 : n_sub);
  }
  const double chunk = std::max(512.0, split_keys / ((any_tc ? 4.0 : 2.0) * num_sms));
  double sum = 0, most = 0, part_rows = 0, most_parts = 1;
  int64_t items = 0;
  for (int b = 0; b < p.batch; ++b) {
    const int lq = q_lens[b];
    if (lq == 0) continue;
    const int64_t keys = (int64_t)cache_lens[b] + (new_lens ? new_lens[b] : 0);
    const double parts = std::max(1.0, std::ceil(keys / chunk));
    const bool d = (int64_t)lq * G <= dec_rows;
    if (!d) {
      const bool whole = lq > tq;
      const int64_t n = (int64_t)p.num_heads_kv * n_sub * (whole ? (lq + tq - 1) / tq : (int64_t)parts);
      const double t = tm.kItemTc + (whole ? keys : std::min((double)keys, chunk)) / 128.0 * tm.tile1;
      items += n;
      sum += n * t;
      most = std::max(most, t);
    }
    if ((d || lq <= tq) && parts > 1) {
      part_rows += parts * lq * p.num_heads_q;
      most_parts = std::max(most_parts, parts);
    }
  }
  const double tc =
      items ? std::max({most, sum / num_sms, (double)((items + num_sms - 1) / num_sms) * sum / items}) : 0.0;
  return tc + tm.decode(dec.keys, dec.units, dec.longest, num_sms) +
         (most_parts > 1 ? tm.combine(part_rows, (int64_t)most_parts) : 0.0);
}

}  // namespace

pkv_status validate_problem(const pkv_problem* p) {
  if (!p) return fail(PKV_ERR_INVALID_ARG, "problem is NULL");
  if (p->batch < 0) return fail(PKV_ERR_INVALID_ARG, "batch < 0");
  if (p->num_heads_q <= 0 || p->num_heads_kv <= 0)
    return fail(PKV_ERR_INVALID_ARG, "head counts must be positive");
  if (p->num_heads_q % p->num_heads_kv != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_heads_q (%d) %% num_heads_kv (%d) != 0", p->num_heads_q,
                p->num_heads_kv);
  // any group size: groups of more than 128 heads are cut into head sub-groups
  if (p->cache_dtype != PKV_BF16 && p->cache_dtype != PKV_FP8_E4M3)
    return fail(PKV_ERR_INVALID_ARG, "cache_dtype %d unknown", p->cache_dtype);
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", p->head_dim);
  if (p->page_size < 0 || p->page_size > 256 ||
      (p->page_size >= kBoxRows && p->page_size % kBoxRows != 0) ||
      (p->page_size > 0 && p->page_size < kBoxRows && (p->page_size & (p->page_size - 1)) != 0))
    return fail(PKV_ERR_UNSUPPORTED, "page_size %d: 0, 1, 2, 4 or a multiple of %d up to 256", p->page_size,
                kBoxRows);
  if (p->cache_capacity <= 0) return fail(PKV_ERR_INVALID_ARG, "cache_capacity must be positive");
  if (p->page_size > 0 && p->cache_capacity % p->page_size != 0)
    return fail(PKV_ERR_INVALID_ARG, "cache_capacity must be a multiple of page_size");
  if (p->num_pages <= 0) return fail(PKV_ERR_INVALID_ARG, "num_pages must be positive");
  if (p->page_size == 0 && p->num_pages < p->batch)
    return fail(PKV_ERR_INVALID_ARG, "contiguous cache: batch_size_cache (num_pages) < batch");
  if (!std::isfinite(p->softmax_scale) || !(p->softmax_scale > 0.0f))
    return fail(PKV_ERR_INVALID_ARG, "softmax_scale must be finite and positive");
  return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

namespace {

pkv_status make_plan(const pkv_problem* problem, const int32_t* h_q_lens, const int32_t* h_cache_lens,
                     const int32_t* h_new_lens, int32_t num_sms, bool dynamic, const SharedPrefixes* groups,
                     pkv_plan_t* out_plan, size_t* out_workspace_bytes) {
  if (!out_plan || !out_workspace_bytes) return fail(PKV_ERR_INVALID_ARG, "output pointers are NULL");
  *out_plan = nullptr;
  *out_workspace_bytes = 0;
  pkv_status st = validate_problem(problem);
  if (st != PKV_OK) return st;
  const pkv_problem& p = *problem;
  const int B = p.batch;
  if (B > 0 && (!h_q_lens || !h_cache_lens)) return fail(PKV_ERR_INVALID_ARG, "length arrays are NULL");
  if (num_sms <= 0) return fail(PKV_ERR_INVALID_ARG, "num_sms must be positive");

  const int G = p.num_heads_q / p.num_heads_kv;
  const int D = p.head_dim;
  const int esize = p.cache_dtype == PKV_BF16 ? 2 : 1;
  const int prefill_rows = kPrefillRowsTc;
  // tensor-core tiles: nh_tc heads of a group x tq query tokens (128 rows at
  // most); a group of more than 128 heads takes n_sub head sub-groups
  const int nh_tc = tc_group_heads(G);
  const int n_sub = (G + nh_tc - 1) / nh_tc;
  const int tq_prefill = prefill_rows / nh_tc;  // query tokens per tensor-core tile
  // A unit (sequence, kv head[, head sub-group]) is a decode unit (warp-MMA
  // tile) if its rows fit 16, else tensor-core tiles; units whose queries fit
  // one tile (decode steps of wide groups, short query runs) can be split
  // along the keys like decode units.
  const int dec_rows = decode_rows(D);  // rows of a warp-MMA decode tile (8 at D = 256)
  auto is_decode = [&](int lq) { return (int64_t)lq * G <= dec_rows; };
  auto splittable = [&](int lq) { return is_decode(lq) || lq <= tq_prefill; };
  // an item of a long query run holds up to two consecutive tiles (fp8 cache,
  // head dims up to 128; plans without decode tiles), which share its K/V tiles
  bool any_decode = false, any_prefill = false;
  for (int b = 0; b < B; ++b) {
    any_decode |= h_q_lens[b] > 0 && is_decode(h_q_lens[b]);
    any_prefill |= h_q_lens[b] > 0 && !is_decode(h_q_lens[b]);
  }

  // Shared prefixes: shared[b] keys of sequence b are attended by its run's
  // common tiles, the rest by its own.  A prefix is shared in whole pages (the
  // tokens of its last, partly filled page are each sequence's own).
  std::vector<int32_t> shared(B, 0), least(B, 0), run_of(B, -1), run_tok(B, 0);
  std::vector<PrefixRun> runs;
  if (groups != nullptr) {
    if (groups->num_groups < 0 || (groups->num_groups > 0 && (!groups->starts || !groups->prefix_lens)))
      return fail(PKV_ERR_INVALID_ARG, "group arrays are NULL or their count is negative");
    const int ng = groups->num_groups;
    for (int g = 0; g < ng; ++g) {
      const int b0 = groups->starts[g], b1 = groups->starts[g + 1], len = groups->prefix_lens[g];
      if (b0 < 0 || b1 < b0 || b1 > B || (g > 0 && b0 < groups->starts[g - 1]))
        return fail(PKV_ERR_INVALID_ARG, "group_starts must rise from 0 to at most the batch (group %d)", g);
      if (len < 0) return fail(PKV_ERR_INVALID_ARG, "negative prefix length of group %d", g);
      if (len == 0) continue;
      if (p.cache_capacity >= kPrefixLk / 2)
        return fail(PKV_ERR_UNSUPPORTED, "shared prefixes: cache_capacity %d is too large", p.cache_capacity);
      if (p.page_size == 0)
        return fail(PKV_ERR_UNSUPPORTED,
                    "shared prefixes need a paged cache (a contiguous one stores a copy a sequence)");
      const int keys = len / p.page_size * p.page_size;
      PrefixRun run{};
      int members = 0;
      // A run is kept if its common tiles are fewer than its sequences, each
      // of which would read the prefix for itself (never with head groups of
      // more than 64, whose tiles hold one token).
      auto close_run = [&]() {
        run.dec = is_decode(run.tokens);
        run.tq = run.dec ? run.tokens : tq_prefill;
        run.tiles = run.tokens > 0 ? (run.tokens + run.tq - 1) / run.tq : 0;
        if (run.tiles < members && keys > 0) {
          run.keys = keys;
          run.tile_slots = run.dec ? 1 : kPrefillRowsTc / kDecodeRows;
          run.per_item = run.dec ? 1 : prefill_q_tiles(D, p.cache_dtype == PKV_FP8_E4M3);
          for (int b = run.b0, n = members; n > 0; ++b) {
            if (h_q_lens[b] == 0) continue;
            shared[b] = keys;
            run_of[b] = (int)runs.size();
            --n;
          }
          runs.push_back(run);
        }
        members = 0;
        run = PrefixRun{};
      };
      for (int b = b0; b < b1; ++b) {
        const int lq = h_q_lens[b], lc = h_cache_lens[b], ln = h_new_lens ? h_new_lens[b] : 0;
        if (lq < 0 || lc < 0 || ln < 0) return fail(PKV_ERR_INVALID_ARG, "negative length at sequence %d", b);
        if (lc < len)
          return fail(PKV_ERR_INVALID_ARG, "sequence %d: cache length %d < the prefix of its group (%d)", b, lc, len);
        least[b] = len;
        if (lq == 0) continue;
        // every query must see the whole prefix (causal: the first one does),
        // and the queries fit one tile (long runs fill tiles of their own)
        const int64_t lk = (int64_t)(dynamic ? len : lc) + ln;
        if (!splittable(lq) || (p.causal && lk - lq + 1 < keys)) {
          close_run();
          continue;
        }
        if (members == 0) run.b0 = b;
        run_tok[b] = run.tokens;
        run.tokens += lq;
        ++members;
      }
      close_run();
    }
  }
  // Sharing pays once the keys it saves outweigh the parts' combine kernel (four
  // sequences on 512 keys: 11.5 us a call shared, 10.4 not; 64 on 2048: 42 and 98).
  if (!runs.empty() && !groups->always) {
    const double with = choose_split(p, runs, h_q_lens, h_cache_lens, h_new_lens, shared.data(), num_sms, n_sub,
                                     tq_prefill, dec_rows).time;
    const double without =
        plain_time(p, h_q_lens, h_cache_lens, h_new_lens, num_sms, n_sub, tq_prefill, dec_rows);
    if (with >= 0.9 * without) {
      runs.clear();
      shared.assign(B, 0);
    }
  }
  // (plans with shared prefixes launch their decode tiles apart)
  const bool sp = !runs.empty();
  const int tq_item = tq_prefill * (any_decode && !sp ? 1 : prefill_q_tiles(D, p.cache_dtype == PKV_FP8_E4M3));
  for (const PrefixRun& r : runs) {
    any_decode |= r.dec;
    any_prefill |= !r.dec;
  }
  // decode-only plans over an fp8 cache at head dims up to 128, or a bf16 one
  // at head dim 64 (rows of 128 bytes), run two CTAs an SM
  const bool two_ctas = (p.cache_dtype == PKV_FP8_E4M3 ? D <= 128 : D == 64) && (!any_prefill || sp);
  const int cps = two_ctas ? 2 : 1;

  int64_t total_q = 0, total_new = 0, total_split_keys = 0, total_dec_keys = 0;
  for (int b = 0; b < B; ++b) {
    int lq = h_q_lens[b], lc = h_cache_lens[b], ln = h_new_lens ? h_new_lens[b] : 0;
    if (lq < 0 || lc < 0 || ln < 0) return fail(PKV_ERR_INVALID_ARG, "negative length at sequence %d", b);
    if ((int64_t)lc + ln > p.cache_capacity)
      return fail(PKV_ERR_INVALID_ARG, "sequence %d: cache_len %d + new_len %d > capacity %d", b, lc, ln,
                  p.cache_capacity);
    total_q += lq;
    total_new += ln;
    if (dynamic && lq > 0 && !splittable(lq))
      return fail(PKV_ERR_UNSUPPORTED,
                  "dynamic plans take requests whose queries fit one tile (sequence %d: %d query tokens > %d)", b, lq,
                  std::max(tq_prefill, dec_rows / G));
    if (lq > 0 && splittable(lq))
      total_split_keys += (int64_t)(lc + ln - shared[b]) * p.num_heads_kv * (is_decode(lq) ? 1 : n_sub);
    if (is_decode(lq) && lq > 0) total_dec_keys += (int64_t)(lc + ln - shared[b]) * p.num_heads_kv;
  }
  for (const PrefixRun& r : runs)
    if (r.dec) total_dec_keys += (int64_t)r.keys * p.num_heads_kv;
  if (total_q > INT32_MAX / 2 || total_new > INT32_MAX / 2)
    return fail(PKV_ERR_UNSUPPORTED, "total tokens too large");

  // split-KV chunk: at least 2 splittable items per SM in decode-only plans, 4
  // when prefill tiles share the launch (their gaps want finer decode items),
  // chunks >= 512 keys.  Measured: the fp8 decode batch (two CTAs an SM) 59.1
  // against 60.9 us at 4, one of random lengths 61.7 against 64.9; the bf16
  // decode batch the same attention kernel and 100.4 against 101.8 us a call
  // (fewer partials to combine); the mixed batch 0.417 against 0.430 ms at 4.
  auto chunk_for = [&](int64_t items_per_sm, int64_t keys, int sms) {
    const int64_t target = items_per_sm * sms;
    const int64_t c = (keys + target - 1) / target;
    return std::max<int64_t>(512, (c + kKvTile - 1) / kKvTile * kKvTile);
  };
  // Plans with shared prefixes: the SMs that the tensor-core tiles get (the
  // decode tiles run on the others at the same time), and the chunks.
  int sms_tc = num_sms;
  int64_t chunk_tc = 1 << 30;
  if (sp) {
    const SplitChoice c = choose_split(p, runs, h_q_lens, h_cache_lens, h_new_lens, shared.data(), num_sms, n_sub,
                                       tq_prefill, dec_rows);
    sms_tc = c.sms_tc;
    chunk_tc = c.chunk;
  }
  const int sms_dec = sp && any_prefill ? std::max(1, num_sms - sms_tc) : num_sms;
  const int64_t dec_keys = sp ? total_dec_keys : total_split_keys;
  int64_t chunk = 1 << 30;
  if (dec_keys > 0) chunk = chunk_for(any_prefill && !sp ? 4 : 2, dec_keys, sms_dec);
  // A decode-only plan whose units are placed as evenly whole (one item an SM
  // as the target) as in chunks of the half is not split at all: no partials
  // and no combine kernel (the bf16 decode batch: 98.1 against 100.3 us a
  // call, the same attention kernel).  Judged on the model costs of a
  // longest-first placement; batches with a few long sequences stay split.
  if ((!any_prefill || sp) && dec_keys > 0) {
    const int ctas = sms_dec * cps;
    std::vector<double> c, load;
    c.reserve((size_t)B * 4);
    load.reserve((size_t)ctas);
    auto busiest = [&](int64_t ch) {  // the longest-first placement's largest CTA cost
      c.clear();
      for (int b = 0; b < B; ++b) {  // one cost per chunk; every kv head has the same
        if (h_q_lens[b] == 0 || (sp && !is_decode(h_q_lens[b]))) continue;
        const int lk = h_cache_lens[b] + (h_new_lens ? h_new_lens[b] : 0) - shared[b];
        const int n = lk <= ch ? 1 : (int)((lk + ch - 1) / ch);
        for (int k = 0; k < n; ++k)
          c.push_back(decode_cost((int)(std::min<int64_t>((int64_t)(k + 1) * ch, lk) - (int64_t)k * ch), D, esize));
      }
      for (const PrefixRun& r : runs) {
        if (!r.dec) continue;
        for (int64_t k = 0; k < r.keys; k += ch)
          c.push_back(decode_cost((int)std::min<int64_t>(ch, r.keys - k), D, esize));
      }
      std::sort(c.begin(), c.end(), std::greater<double>());
      load.assign((size_t)ctas, 0.0);  // a min-heap over the CTA loads
      for (double x : c)
        for (int hk = 0; hk < p.num_heads_kv; ++hk) {
          std::pop_heap(load.begin(), load.end(), std::greater<double>());
          load.back() += x;
          std::push_heap(load.begin(), load.end(), std::greater<double>());
        }
      return *std::max_element(load.begin(), load.end());
    };
    const int64_t whole = chunk_for(1, dec_keys, sms_dec);
    if (whole != chunk && busiest(whole) <= 1.02 * busiest(chunk)) chunk = whole;
  }
  // (plans with shared prefixes: the tensor-core units have chunks of their own)
  auto chunk_of = [&](bool dec) { return dec || !sp ? chunk : chunk_tc; };
  auto nchunks_of = [&](int lk, bool dec) {
    const int64_t ch = chunk_of(dec);
    return lk <= ch ? 1 : (int)((lk + ch - 1) / ch);
  };
  for (PrefixRun& r : runs) {
    // chunks of nearly the same size
    const int n = nchunks_of(r.keys, r.dec);
    r.chunk = ((r.keys + n - 1) / n + kKvTile - 1) / kKvTile * kKvTile;
    r.nchunks = (r.keys + r.chunk - 1) / r.chunk;
  }

  int64_t num_tiles_est = 0;
  for (int b = 0; b < B; ++b) {
    const int lq = h_q_lens[b], lk = h_cache_lens[b] + (h_new_lens ? h_new_lens[b] : 0);
    if (lq == 0) continue;
    num_tiles_est += (int64_t)p.num_heads_kv * (is_decode(lq) ? nchunks_of(lk, true)
                                                : (int64_t)n_sub * (splittable(lq) ? nchunks_of(lk, false)
                                                                                   : (lq + tq_item - 1) / tq_item));
  }
  std::vector<Tile> tiles;
  tiles.reserve((size_t)num_tiles_est);
  std::vector<CombineItem> combines;
  int64_t num_slots = 0;
  int32_t n_dec = 0, n_pre = 0;
  int64_t q_row = 0;
  for (int b = 0, r = 0; b < B; ++b) {
    if (r < (int)runs.size() && runs[r].b0 == b) runs[r++].q_row = q_row;
    q_row += h_q_lens[b];
  }
  // the tiles over the shared prefixes: every tile of a run's query tokens
  // against every chunk of the prefix, each into its own partial slots
  for (PrefixRun& r : runs) {
    for (int hk = 0; hk < p.num_heads_kv; ++hk) {
      r.slot0.push_back((int32_t)num_slots);
      for (int c = 0; c < r.nchunks; ++c) {
        for (int t = 0; t < r.tiles; t += r.per_item) {
          const int nt = std::min(r.per_item, r.tiles - t);  // query tiles of the item
          Tile x{};
          x.item.b = r.b0;
          x.item.hk = hk;
          x.item.q_row0 = (int32_t)(r.q_row + (int64_t)t * r.tq);
          x.item.q_i0 = t * r.tq;
          x.item.n_q = std::min(nt * r.tq, r.tokens - t * r.tq);
          // (each query as the one query of its row: it sees every key of the prefix)
          x.item.lq = 1;
          x.item.lk = kPrefixLk;
          x.item.kv_begin = c * r.chunk;
          x.item.kv_end = std::min(r.keys, (c + 1) * r.chunk);
          x.item.kind = r.dec ? kDecode : kPrefill;
          x.item.partial = (int32_t)num_slots;
          x.item.nh = G;  // (h0 = 0: groups of up to 64 heads)
          x.prefix = true;
          const int keys = x.item.kv_end - x.item.kv_begin;
          x.cost = r.dec ? decode_cost(keys, D, esize)
                         : std::max(decode_cost(keys, D, esize), prefill_cost(keys, nt * prefill_rows, D));
          tiles.push_back(x);
          num_slots += nt * r.tile_slots;
          if (r.dec) ++n_dec; else ++n_pre;
        }
      }
    }
  }
  q_row = 0;
  for (int b = 0; b < B; ++b) {
    int lq = h_q_lens[b], lc = h_cache_lens[b], ln = h_new_lens ? h_new_lens[b] : 0;
    int lk = lc + ln;
    if (lq == 0) continue;
    for (int hk = 0; hk < p.num_heads_kv; ++hk) {
      const bool dec = is_decode(lq);
      for (int sg = 0; sg < (dec ? 1 : n_sub); ++sg) {
        const int h0 = dec ? 0 : sg * nh_tc;
        const int nh = dec ? G : std::min(nh_tc, G - h0);
        if (splittable(lq)) {
          // one query tile (all lq tokens), possibly cut into KV chunks; with a
          // shared prefix the keys past it, always into partials
          const int first = shared[b];
          const bool part = first > 0;
          const int nchunks = lk > first || !part ? nchunks_of(lk - first, dec) : 0;
          const int64_t chunk_u = chunk_of(dec);
          const int rows = lq * nh;
          const int stride = (rows + kDecodeRows - 1) / kDecodeRows;  // 16-row partial slots per chunk
          const int64_t slot0 = nchunks > 1 || part ? num_slots : -1;
          for (int c = 0; c < nchunks; ++c) {
            Tile t{};
            t.item.b = b;
            t.item.hk = hk;
            t.item.q_row0 = (int32_t)q_row;
            t.item.q_i0 = 0;
            t.item.n_q = lq;
            t.item.lq = lq;
            t.item.lk = lk;
            t.item.kv_begin = (int32_t)std::min<int64_t>(first + (int64_t)c * chunk_u, lk);
            t.item.kv_end = (int32_t)std::min<int64_t>(first + (int64_t)(c + 1) * chunk_u, lk);
            t.item.kind = dec ? kDecode : kPrefill;
            t.item.partial = nchunks > 1 || part ? (int32_t)(num_slots + (int64_t)c * stride) : -1;
            t.item.h0 = h0;
            t.item.nh = nh;
            const int keys = t.item.kv_end - t.item.kv_begin;
            t.cost = dec ? decode_cost(keys, D, esize)
                         : std::max(decode_cost(keys, D, esize), prefill_cost(keys, prefill_rows, D));
            tiles.push_back(t);
            if (dec) ++n_dec; else ++n_pre;
          }
          if (nchunks > 1 || part) {
            CombineItem ci{};
            ci.b = b;
            ci.q_row0 = (int32_t)q_row;
            ci.n_q = lq;
            ci.hk = hk;
            ci.nsplit = nchunks;
            ci.slot0 = (int32_t)slot0;
            ci.slot_stride = stride;
            ci.h0 = h0;
            ci.nh = nh;
            if (part) {
              const PrefixRun& r = runs[run_of[b]];
              ci.p_nsplit = r.nchunks;
              ci.p_slot0 = r.slot0[hk];
              ci.p_chunk_slots = r.tiles * r.tile_slots;
              ci.p_tq = r.tq;
              ci.p_tile_slots = r.tile_slots;
              ci.p_tok0 = run_tok[b];
            }
            combines.push_back(ci);
            num_slots += (int64_t)nchunks * stride;
          }
        } else {
          for (int i0 = 0; i0 < lq; i0 += tq_item) {
            int n = std::min(tq_item, lq - i0);
            int kv_end = lk;  // the keys of the item's last query token
            if (p.causal) kv_end = std::max(0, std::min(lk, i0 + n + lk - lq));
            Tile t{};
            t.item.b = b;
            t.item.hk = hk;
            t.item.q_row0 = (int32_t)(q_row + i0);
            t.item.q_i0 = i0;
            t.item.n_q = n;
            t.item.lq = lq;
            t.item.lk = lk;
            t.item.kv_begin = 0;
            t.item.kv_end = kv_end;
            t.item.kind = kPrefill;
            t.item.partial = -1;
            t.item.h0 = h0;
            t.item.nh = nh;
            // each query tile of the item attends the keys of its own last token
            t.cost = 0.0;
            for (int s = i0; s < i0 + n; s += tq_prefill) {
              const int ns = std::min(tq_prefill, i0 + n - s);
              const int ke = p.causal ? std::max(0, std::min(lk, s + ns + lk - lq)) : lk;
              t.cost += prefill_cost(ke, prefill_rows, D);
            }
            tiles.push_back(t);
            ++n_pre;
          }
        }
      }
    }
    q_row += lq;
  }
  if (num_slots > INT32_MAX / (kDecodeRows * 256))
    return fail(PKV_ERR_UNSUPPORTED, "too many split-KV partial slots");

  // longest processing time first onto the least-loaded CTA (ties: the lowest
  // CTA index), found with a tournament tree over the CTAs' (load, index)
  // pairs; each CTA keeps its items in the order they were assigned
  // (plans with shared prefixes: tensor-core tiles and decode tiles apart, on
  // sms_tc and sms_dec SMs, the tensor-core CTAs first)
  const int num_items = (int)tiles.size();
  std::vector<double> costs(num_items);
  for (int i = 0; i < num_items; ++i) costs[i] = tiles[i].cost;
  std::vector<int> order(num_items);
  for (int i = 0; i < num_items; ++i) order[i] = i;
  std::stable_sort(order.begin(), order.end(), [&](int a, int c) { return costs[a] > costs[c]; });
  const bool apart = sp && n_dec > 0 && n_pre > 0;
  const int num_tc = apart ? std::min(sms_tc, (int)n_pre) : 0;
  const int num_ctas = apart ? num_tc + std::min(sms_dec * cps, (int)n_dec)
                             : std::max(1, std::min(num_sms * (any_prefill ? 1 : cps), num_items));
  std::vector<int> cta_of(num_items), cta_count(num_ctas, 0);
  using Load = std::pair<double, int>;
  std::vector<Load> loads;
  auto assign = [&](int first, int ctas, auto&& takes) {
    int leaves = 1;
    while (leaves < ctas) leaves *= 2;
    const Load none{HUGE_VAL, INT32_MAX};
    std::vector<Load> tree(2 * (size_t)leaves, none);  // node i: the lesser of nodes 2i and 2i+1
    for (int c = 0; c < ctas; ++c) tree[leaves + c] = {0.0, c};
    for (int i = leaves - 1; i >= 1; --i) tree[i] = std::min(tree[2 * i], tree[2 * i + 1]);
    for (int idx : order) {
      if (!takes(idx)) continue;
      const int c = tree[1].second;
      cta_of[idx] = first + c;
      ++cta_count[first + c];
      int i = leaves + c;
      tree[i].first += costs[idx];
      for (i >>= 1; i >= 1; i >>= 1) tree[i] = std::min(tree[2 * i], tree[2 * i + 1]);
    }
    loads.insert(loads.end(), tree.begin() + leaves, tree.begin() + leaves + ctas);
  };
  if (apart) {
    assign(0, num_tc, [&](int i) { return tiles[i].item.kind == kPrefill; });
    assign(num_tc, num_ctas - num_tc, [&](int i) { return tiles[i].item.kind == kDecode; });
  } else {
    assign(0, num_ctas, [](int) { return true; });
  }
  double max_cost = 0, sum_cost = 0;
  int max_items = 0;
  std::sort(loads.begin(), loads.end());  // summed lightest first
  for (const Load& l : loads) {
    max_cost = std::max(max_cost, l.first);
    sum_cost += l.first;
  }
  for (int c = 0; c < num_ctas; ++c) max_items = std::max(max_items, cta_count[c]);

  // workspace layout
  WorkspaceLayout L{};
  size_t off = 0;
  L.status = off;
  off = align_up(off + 16, 256);
  L.items = off;
  off = align_up(off + sizeof(WorkItem) * (size_t)std::max(1, num_items), 256);
  L.cta_begin = off;
  off = align_up(off + sizeof(int32_t) * (size_t)(num_ctas + 1), 256);
  L.combine = off;
  off = align_up(off + sizeof(CombineItem) * (size_t)std::max<size_t>(1, combines.size()), 256);
  L.plan_lc = off;
  off = align_up(off + 2 * sizeof(int32_t) * (size_t)std::max(1, B), 256);
  size_t image_bytes = off;
  L.partial_o = off;
  off = align_up(off + sizeof(float) * (size_t)num_slots * kDecodeRows * D, 256);
  L.partial_lse = off;
  off = align_up(off + sizeof(float) * (size_t)num_slots * kDecodeRows, 256);
  L.total = off;

  pkv_plan_s* plan = new (std::nothrow) pkv_plan_s();
  if (!plan) return fail(PKV_ERR_INVALID_ARG, "out of host memory");
  plan->image = (unsigned char*)calloc(1, image_bytes);
  plan->item_cost = (double*)calloc((size_t)std::max(1, num_items), sizeof(double));
  if (!plan->image || !plan->item_cost) {
    free(plan->image);
    free(plan->item_cost);
    delete plan;
    return fail(PKV_ERR_INVALID_ARG, "out of host memory");
  }
  plan->problem = p;
  plan->num_ctas = num_items > 0 ? num_ctas : 0;
  plan->num_ctas_tc = num_tc;
  // The decode tiles usually take longest, so their launch comes first; but two
  // of their CTAs an SM would spread over every SM and leave the tensor-core
  // CTAs none, and tensor-core tiles over appended keys would wait for them.
  bool tc_prefix_only = true;
  for (const Tile& t : tiles) tc_prefix_only &= t.item.kind == kDecode || t.prefix;
  plan->dec_first = apart && cps == 1 && tc_prefix_only;
  plan->max_combine_rows = plan->max_combine_parts = 0;
  for (const CombineItem& c : combines) {
    plan->max_combine_rows = std::max(plan->max_combine_rows, c.n_q * c.nh);
    plan->max_combine_parts = std::max(plan->max_combine_parts, c.nsplit + c.p_nsplit);
  }
  plan->num_slots = (int32_t)num_slots;
  plan->total_q = (int32_t)total_q;
  plan->total_new = (int32_t)total_new;
  plan->max_items_per_cta = max_items;
  plan->num_decode_items = n_dec;
  plan->num_prefill_items = n_pre;
  plan->num_split_units = (int32_t)combines.size();
  plan->max_cta_cost = max_cost;
  plan->mean_cta_cost = num_ctas ? sum_cost / num_ctas : 0.0;
  plan->layout = L;
  plan->image_bytes = image_bytes;
  plan->num_items = num_items;
  plan->num_combine = (int32_t)combines.size();
  plan->dynamic = dynamic ? 1 : 0;
  plan->shared = runs.empty() ? 0 : 1;
  plan->row_combine = groups != nullptr;

  WorkItem* items = (WorkItem*)(plan->image + L.items);
  int32_t* cta_begin = (int32_t*)(plan->image + L.cta_begin);
  cta_begin[0] = 0;
  for (int c = 0; c < num_ctas; ++c) cta_begin[c + 1] = cta_begin[c] + cta_count[c];
  std::vector<int32_t> fill(cta_begin, cta_begin + num_ctas);
  for (int idx : order) {
    const int k = fill[cta_of[idx]]++;
    items[k] = tiles[idx].item;
    plan->item_cost[k] = costs[idx];
  }
  if (!combines.empty()) memcpy(plan->image + L.combine, combines.data(), combines.size() * sizeof(CombineItem));
  int32_t* lc = (int32_t*)(plan->image + L.plan_lc);
  for (int b = 0; b < B; ++b) {
    lc[b] = h_cache_lens[b];
    lc[B + b] = dynamic ? least[b] : h_cache_lens[b];  // (dynamic: 0, or the prefix of the sequence's group)
  }

  *out_plan = plan;
  *out_workspace_bytes = L.total;
  return PKV_OK;
}

}  // namespace

namespace {

// make_plan for the C entries: what the containers throw becomes a status.
template <class... Args>
pkv_status make_plan_noexcept(Args... args) noexcept {
  try {
    return make_plan(args...);
  } catch (const std::exception&) {
    return fail(PKV_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // namespace

extern "C" pkv_status pkv_plan(const pkv_problem* problem, const int32_t* h_q_lens,
                               const int32_t* h_cache_lens, const int32_t* h_new_lens,
                               int32_t num_sms, pkv_plan_t* out_plan, size_t* out_workspace_bytes) {
  return make_plan_noexcept(problem, h_q_lens, h_cache_lens, h_new_lens, num_sms, false, nullptr, out_plan,
                            out_workspace_bytes);
}

extern "C" pkv_status pkv_plan_decode_dynamic(const pkv_problem* problem, const int32_t* h_q_lens,
                                              const int32_t* h_max_cache_lens, const int32_t* h_new_lens,
                                              int32_t num_sms, pkv_plan_t* out_plan, size_t* out_workspace_bytes) {
  return make_plan_noexcept(problem, h_q_lens, h_max_cache_lens, h_new_lens, num_sms, true, nullptr, out_plan,
                   out_workspace_bytes);
}

extern "C" pkv_status pkv_plan_shared_prefix(const pkv_problem* problem, const int32_t* h_q_lens,
                                             const int32_t* h_cache_lens, const int32_t* h_new_lens,
                                             int32_t num_groups, const int32_t* h_group_starts,
                                             const int32_t* h_prefix_lens, int32_t always, int32_t dynamic,
                                             int32_t num_sms, pkv_plan_t* out_plan, size_t* out_workspace_bytes) {
  const SharedPrefixes groups{num_groups, h_group_starts, h_prefix_lens, always != 0};
  return make_plan_noexcept(problem, h_q_lens, h_cache_lens, h_new_lens, num_sms, dynamic != 0, &groups, out_plan,
                   out_workspace_bytes);
}

extern "C" pkv_status pkv_plan_get_stats(pkv_plan_t plan, pkv_plan_stats* s) {
  if (!plan || !s) return fail(PKV_ERR_INVALID_ARG, "NULL plan or stats");
  s->num_items = plan->num_items;
  s->num_decode_items = plan->num_decode_items;
  s->num_prefill_items = plan->num_prefill_items;
  s->num_split_units = plan->num_split_units;
  s->num_ctas = plan->num_ctas;
  s->total_q = plan->total_q;
  s->total_new = plan->total_new;
  s->max_items_per_cta = plan->max_items_per_cta;
  s->max_cta_cost = plan->max_cta_cost;
  s->mean_cta_cost = plan->mean_cta_cost;
  s->upload_bytes = (int64_t)plan->image_bytes;
  s->workspace_bytes = (int64_t)plan->layout.total;
  return PKV_OK;
}

extern "C" pkv_status pkv_plan_get_items(pkv_plan_t plan, pkv_work_item* h_items, int32_t capacity,
                                         int32_t* count) {
  if (!plan || !count) return fail(PKV_ERR_INVALID_ARG, "NULL plan or count");
  *count = plan->num_items;
  if (!h_items || capacity <= 0) return PKV_OK;
  const WorkItem* items = (const WorkItem*)(plan->image + plan->layout.items);
  const int32_t* cta_begin = (const int32_t*)(plan->image + plan->layout.cta_begin);
  int n = 0;
  for (int c = 0; c < plan->num_ctas && n < capacity; ++c) {
    for (int k = cta_begin[c]; k < cta_begin[c + 1] && n < capacity; ++k, ++n) {
      const WorkItem& w = items[k];
      pkv_work_item& o = h_items[n];
      o.seq = w.b;
      o.kv_head = w.hk;
      o.q_row0 = w.q_row0;
      o.q_index0 = w.q_i0;
      o.n_q = w.n_q;
      o.q_len = w.lq;
      o.kv_len = w.lk == kPrefixLk ? w.kv_end : w.lk;
      o.kv_begin = w.kv_begin;
      o.kv_end = w.kv_end;
      o.kind = w.kind;
      o.partial_slot = w.partial;
      o.cta = c;
      o.head0 = w.h0;
      o.num_heads = w.nh;
      o.cost = plan->item_cost[k];
    }
  }
  return PKV_OK;
}

extern "C" void pkv_plan_destroy(pkv_plan_t plan) {
  if (!plan) return;
  free(plan->image);
  free(plan->item_cost);
  delete plan;
}
