"""Attention of a batch whose sequences share prefixes (plans of
``plan_shared_prefix``), against 64-bit attention of every sequence by itself.

Tolerances (derived, per element).  With weights w_j and A = sum_j w_j |v_j|:
the probabilities are rounded once for P V (half a step: 2^-8 relative in bf16,
2^-11 in f16 over an fp8 cache), so at most that times A; the output is rounded
once (2^-8 |out|); fp32 sums, exp2 and the merge of the parts stay below 2^-14 A.
The log-sum-exp uses the unrounded probabilities: the logits' fp32 dot products
(D terms, 2^-24 each of scale sum |q k|) stay below 1.2e-4 for the values here,
exp2 and log2 below 2^-18; 2^-12 is used.
"""
import numpy as np
import pytest

import oracle
from tests import harness as H
from tests.test_rope import AppendCase, _Fake, bf16, close_bf16, np64, rows64, table64

LSE_TOL = 2.0 ** -12


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_variable_gb300 as m
    from paged_kv_variable_gb300 import build as b
    b.build()
    m.lib()
    return m


def problem(pkv, **kw):
    base = dict(batch=4, num_heads_q=8, num_heads_kv=2, head_dim=128, page_size=16, cache_capacity=4096,
                num_pages=1000, cache_dtype="bf16", causal=True, softmax_scale=128 ** -0.5)
    base.update(kw)
    return pkv.make_problem(**base)


# ------------------------------------------------------------------ the plan (host)
def test_refusals(pkv):
    def call(starts=(0, 4), prefix=(64,), q=(1,) * 4, cache=(100,) * 4, new=(1,) * 4, status=1, dynamic=False, **kw):
        with pytest.raises(pkv.PkvError) as e:
            pkv.plan_shared_prefix(problem(pkv, **kw), q, cache, new, group_starts=starts, prefix_lens=prefix,
                                   dynamic=dynamic, num_sms=4)
        assert e.value.status == status and pkv.last_error()

    call(starts=(0, 5))                              # past the batch
    call(starts=(-1, 4))
    call(starts=(2, 1))
    call(starts=(0, 3, 2, 4), prefix=(16, 16, 16))
    call(prefix=(-1,))
    call(prefix=(101,))                              # longer than a sequence's cache
    call(prefix=(64,), cache=(100, 63, 100, 100))
    call(page_size=0, num_pages=4, status=2)         # contiguous
    call(cache=(100, 100, 100, -5))
    call(cache=(4096, 100, 100, 100))                # past the capacity
    call(head_dim=96, status=2)
    call(q=(200,) * 4, dynamic=True, status=2)       # (as for a plain dynamic plan)
    for bad in (dict(group_starts=(0, 4), prefix_lens=(1, 2)), dict(group_starts=(), prefix_lens=())):
        with pytest.raises(ValueError):
            pkv.plan_shared_prefix(problem(pkv), (1,) * 4, (100,) * 4, None, num_sms=4, **bad)
    with pytest.raises(ValueError):
        pkv.plan_shared_prefix(problem(pkv), (1,) * 3, (100,) * 4, None, group_starts=(0, 4), prefix_lens=(16,),
                               num_sms=4)
    L = pkv.lib()
    import ctypes
    h, n = ctypes.c_void_p(), ctypes.c_size_t()
    lens = np.full(4, 100, np.int32)
    assert L.pkv_plan_shared_prefix(problem(pkv), lens.ctypes.data, lens.ctypes.data, None, 1, None, None, 0, 0, 4,
                                    h, n) == 1
    assert L.pkv_plan_shared_prefix(problem(pkv), lens.ctypes.data, lens.ctypes.data, None, -1, None, None, 0, 0, 4,
                                    h, n) == 1


def test_placed_rows_refused(pkv):
    """q_rows > 0 (rows placed by the caller) is refused before anything is launched."""
    pl = pkv.plan_shared_prefix(problem(pkv), (1,) * 4, (2000,) * 4, None, group_starts=(0, 4), prefix_lens=(1600,),
                                always=True, num_sms=4)
    q, c = _Fake((4, 8, 128)), _Fake((1000, 16, 2, 128), ptr=1 << 24)
    i32, bt = _Fake((5,), "int32"), _Fake((4, 256), "int32")
    ws = _Fake((pl.workspace_bytes,), "uint8", ptr=1 << 28)
    ws.numel, ws.element_size = (lambda: ws.shape[0]), (lambda: 1)
    args = pkv.make_args(q=q, out=q, cu_seqlens_q=i32, max_seqlen_q=1, k_cache=c, v_cache=c, cache_seqlens=i32,
                         block_table=bt, q_rows=8)
    with pytest.raises(pkv.PkvError) as e:
        pkv.attn_varlen_kvcache_fwd(problem(pkv), args, pl, ws, stream=0)
    assert e.value.status == 2


PLANS = [
    # hq, hkv, d, dtype, page, causal, q, cache, new, starts, prefix
    (8, 2, 128, "bf16", 16, True, [1] * 40, [1500 + 7 * b for b in range(40)], [1] * 40, [0, 40], [1300]),
    (8, 2, 128, "fp8", 16, True, [1] * 40, [1500 + 7 * b for b in range(40)], None, [0, 10, 11, 40], [1300, 1500, 700]),
    (12, 2, 64, "bf16", 24, True, [4, 0, 2, 1, 5], [600, 700, 640, 655, 800], [4, 1, 2, 1, 5], [0, 5], [599]),
    (41, 1, 128, "bf16", 16, False, [1, 1, 1], [600, 700, 512], None, [0, 3], [512]),       # one sequence: prefix only
    (71, 1, 128, "bf16", 16, False, [1, 1, 1], [600, 700, 512], None, [0, 3], [512]),       # a tile a token: not shared
    (400, 2, 64, "bf16", 8, True, [1, 1, 1], [600, 700, 540], [2, 1, 1], [0, 3], [512]),    # the same
    (8, 2, 128, "bf16", 16, True, [30, 30, 31], [900] * 3, [30, 30, 31], [0, 3], [800]),    # a tile a sequence: the same
    (4, 1, 256, "bf16", 16, True, [1, 1, 1], [6000, 7000, 5400], [1, 1, 1], [0, 3], [5000]),
    (8, 2, 128, "bf16", 16, True, [1, 300, 1, 1, 2], [900] * 5, [1, 300, 1, 1, 2], [0, 5], [800]),  # a long run inside
    (8, 2, 128, "bf16", 16, True, [1, 40, 1, 1, 2], [900] * 5, [0, 0, 0, 0, 0], [0, 5], [880]),     # one sees less
]


@pytest.mark.parametrize("dynamic", [False, True])
@pytest.mark.parametrize("i", range(len(PLANS)))
def test_plan_covers_every_key_once(pkv, i, dynamic):
    hq, hkv, d, dtype, page, causal, q, cache, new, starts, prefix = PLANS[i]
    if dynamic and max(q) * (hq // hkv) > 128:
        pytest.skip("not a dynamic batch")
    B, G = len(q), hq // hkv
    cap = 8192 // page * page
    prob = problem(pkv, batch=B, num_heads_q=hq, num_heads_kv=hkv, head_dim=d, page_size=page, cache_dtype=dtype,
                   causal=causal, cache_capacity=cap)
    pl = pkv.plan_shared_prefix(prob, q, cache, new, group_starts=starts, prefix_lens=prefix, dynamic=dynamic,
                                always=True, num_sms=8)
    row_of = np.concatenate([[0], np.cumsum(q)])
    seq_of = np.repeat(np.arange(B), q)
    lk = np.array(cache) + (np.array(new) if new is not None else 0)
    cover, slots, used_shared = {}, {}, 0
    for it in pl.items():
        rows = range(it["q_row0"], it["q_row0"] + it["n_q"])
        several = len({seq_of[r] for r in rows}) > 1 or it["q_len"] == 1 != q[it["seq"]]
        used_shared += several
        if it["kind"] == 0:
            assert it["n_q"] * it["num_heads"] <= (8 if d == 256 else 16) and it["num_heads"] == G
        else:
            assert it["n_q"] * it["num_heads"] <= 128 * (2 if dtype == "fp8" and d <= 128 else 1)
        assert it["kv_begin"] % min(page, 8) == 0
        for r in rows:
            for h in range(it["head0"], it["head0"] + it["num_heads"]):
                cover.setdefault((r, it["kv_head"] * G + h), []).append((it["kv_begin"], it["kv_end"]))
        if it["partial_slot"] >= 0:
            n = -(-it["n_q"] * it["num_heads"] // 16)
            for s in range(it["partial_slot"], it["partial_slot"] + n):
                assert s not in slots, "a partial slot written twice"
                slots[s] = it
    for b in range(B):
        for r in range(row_of[b], row_of[b + 1]):
            horizon = min(lk[b], r - row_of[b] + lk[b] - q[b] + 1) if causal else lk[b]
            for h in range(hq):
                at = 0
                for lo, hi in sorted(cover.pop((r, h))):
                    assert lo == at
                    at = hi
                assert horizon <= at <= lk[b]
    assert not cover
    not_shared = G > 64 or min(q) == 30
    assert (used_shared > 0) != not_shared
    if not_shared:
        return
    # the same batch without sharing reads every prefix once a sequence
    def keys(plan):
        return sum(it["kv_end"] - it["kv_begin"] for it in plan.items())
    if max(q) * G <= 128 and len(q) < 30:
        assert keys(pl) < keys(pkv.plan(prob, q, cache, new, num_sms=8))


def test_shared_where_it_pays(pkv):
    """A few sequences on a short prefix are planned as without it; many, or a long one, are not."""
    def plans(B, prefix, sms=152, **kw):
        prob = problem(pkv, batch=B, num_heads_q=32, num_heads_kv=8, cache_capacity=1 << 16, **kw)
        args = (prob, [1] * B, [prefix + 40 + b for b in range(B)], None)
        shared = pkv.plan_shared_prefix(*args, group_starts=[0, B], prefix_lens=[prefix], num_sms=sms)
        return shared.items() != pkv.plan(*args, num_sms=sms).items()

    for dtype in ("bf16", "fp8"):
        assert not plans(4, 512, cache_dtype=dtype)
        assert not plans(2, 128, cache_dtype=dtype)
        assert plans(64, 2048, cache_dtype=dtype)
        assert plans(4, 32768, cache_dtype=dtype)


def test_nothing_to_share_equals_the_plain_plan(pkv):
    prob = problem(pkv)
    args = ((1, 2, 0, 300), (3000, 2000, 10, 400), (1, 2, 1, 300))
    plain = pkv.plan(prob, *args, num_sms=8)
    for starts, prefix in (([0], []), ([0, 4], [0]), ([0, 4], [9]), ([0, 1, 2, 4], [2000, 1000, 10]),
                           ([0, 1, 4], [0, 10])):
        pl = pkv.plan_shared_prefix(prob, *args, group_starts=starts, prefix_lens=prefix, always=True, num_sms=8)
        assert pl.items() == plain.items()


# ------------------------------------------------------------------ parity
class Shared:
    """A batch of groups over a paged pool; the prefix pages stand in every
    table of their group.  Slots that no token holds are NaN (bf16)."""

    def __init__(self, pkv, torch, seed, *, starts, prefix, own, q, new=None, hq=8, hkv=2, d=128, page=16, fp8=False,
                 causal=True, q_scale=None, ragged=False, num_sms=None, dynamic=False, bound=0, shares=True):
        rng = np.random.default_rng(seed)
        self.pkv, self.torch, self.fp8, self.causal, self.page, self.d, self.hq = pkv, torch, fp8, causal, page, d, hq
        B = len(q)
        self.q_lens = np.asarray(q, np.int32)
        self.new = None if new is None else np.asarray(new, np.int32)
        group = np.full(B, -1)
        for g in range(len(prefix)):
            group[starts[g]:starts[g + 1]] = g
        pre = np.array([prefix[g] if g >= 0 else 0 for g in group])
        self.cache = (pre + np.asarray(own)).astype(np.int32)          # before the call's append
        self.lk = self.cache + (0 if new is None else self.new)
        cap = int(-(-(self.lk.max() + bound) // page) * page)
        width = cap // page
        full = [p // page for p in prefix]
        need = sum(full) + int(sum(width - (full[g] if g >= 0 else 0) for g in group)) + 1
        perm = iter(rng.permutation(need))
        self.pages = np.zeros((B, width), np.int32)
        for g in range(len(prefix)):
            self.pages[starts[g]:starts[g + 1], :full[g]] = [next(perm) for _ in range(full[g])]
        for b in range(B):
            n0 = full[group[b]] if group[b] >= 0 else 0
            self.pages[b, n0:] = [next(perm) for _ in range(width - n0)]
        shape = (need, page, hkv, d)
        held = np.zeros((need, page), bool)
        for b in range(B):
            pos = np.arange(self.cache[b])
            held[self.pages[b, pos // page], pos % page] = True
        if fp8:
            self.kc, self.vc = (torch.from_numpy(rng.integers(0, 256, shape).astype(np.uint8)).cuda() for _ in "kv")
            for c in (self.kc, self.vc):       # codes of magnitude up to 1.75 x scale, NaN where nothing is held
                c.copy_(torch.where(torch.from_numpy(held).cuda()[:, :, None, None], (c & 0x80) | (c % 0x3f), 0x7f))
            self.ks, self.vs = (torch.tensor([s], dtype=torch.float32, device="cuda") for s in (0.9, 1.1))
        else:
            self.kc, self.vc = bf16(torch, rng, *shape), bf16(torch, rng, *shape)
            for c in (self.kc, self.vc):
                c[torch.from_numpy(~held).cuda()] = float("nan")
            self.ks = self.vs = None
        tq = int(self.q_lens.sum())
        self.q = bf16(torch, rng, tq, hq, d, scale=2.0)
        self.q_scale = None if q_scale is None else torch.tensor([q_scale], dtype=torch.float32, device="cuda")
        self.knew = self.vnew = self.cu_new = None
        if new is not None:
            tn = int(self.new.sum())
            self.knew, self.vnew = bf16(torch, rng, max(tn, 1), hkv, d), bf16(torch, rng, max(tn, 1), hkv, d)
            self.cu_new = H.i32(np.concatenate([[0], np.cumsum(self.new)]))
        self.out = torch.full((tq, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((hq, tq), float("nan"), dtype=torch.float32, device="cuda")
        self.cu_q, self.lens = H.i32(np.concatenate([[0], np.cumsum(self.q_lens)])), H.i32(self.cache)
        self.extra = dict(block_table=H.i32(self.pages))
        if ragged:
            counts = -(-self.lk // page)
            self.extra = dict(block_table=H.i32(np.concatenate([self.pages[b, :n] for b, n in enumerate(counts)])),
                              page_indptr=H.i32(np.concatenate([[0], np.cumsum(counts)])))
        self.problem = pkv.make_problem(batch=B, num_heads_q=hq, num_heads_kv=hkv, head_dim=d, page_size=page,
                                        cache_capacity=cap, num_pages=need, cache_dtype="fp8" if fp8 else "bf16",
                                        causal=causal, softmax_scale=d ** -0.5)
        self.plan = pkv.plan_shared_prefix(self.problem, self.q_lens, self.cache + bound, self.new,
                                           group_starts=starts, prefix_lens=prefix, always=True, dynamic=dynamic,
                                           num_sms=num_sms)
        # shared: some tile holds rows of several sequences
        first = np.repeat(np.arange(B), self.q_lens)
        assert shares == any(first[it["q_row0"]] != first[it["q_row0"] + it["n_q"] - 1] for it in self.plan.items())
        self.ws = pkv.workspace_tensor(self.plan.workspace_bytes)
        self.plan.upload(self.ws)

    def args(self, **over):
        kw = dict(q=self.q, out=self.out, lse=self.lse, cu_seqlens_q=self.cu_q,
                  max_seqlen_q=int(self.q_lens.max()), k_cache=self.kc, v_cache=self.vc, cache_seqlens=self.lens,
                  k_new=self.knew, v_new=self.vnew, cu_seqlens_knew=self.cu_new, k_scale=self.ks, v_scale=self.vs,
                  q_scale=self.q_scale, **self.extra)
        if self.new is not None and self.new.sum() == 0:
            kw.update(k_new=None, v_new=None, cu_seqlens_knew=None)
        kw.update(over)
        return self.pkv.make_args(**kw)

    def run(self, stream=None):
        self.pkv.attn_varlen_kvcache_fwd(self.problem, self.args(), self.plan, self.ws, stream=stream)
        return self.pkv.get_status(self.ws, stream=stream)

    def check(self):
        """The output against each sequence's attention over its own table, in 64 bits."""
        kd, vd = ((oracle.e4m3_decode(H.to_numpy_bits(x)) * float(s) if self.fp8 else np64(x))
                  for x, s in ((self.kc, self.ks), (self.vc, self.vs)))
        q = np64(self.q)
        if self.q_scale is not None:
            qs = float(self.q_scale)
            q = oracle.e4m3_decode(oracle.fp8_quantize(H.to_numpy_bits(self.q), qs)) * qs
        out, lse = H.bf16_to_f64(self.out), self.lse.double().cpu().numpy()
        half_p = 2.0 ** -11 if self.fp8 else 2.0 ** -8
        r0 = 0
        for b, (lq, lk) in enumerate(zip(self.q_lens, self.lk)):
            pos = np.arange(lk)
            K, V = (c[self.pages[b, pos // self.page], pos % self.page] for c in (kd, vd))
            want, want_lse = oracle.attend(q[r0:r0 + lq], K, V, self.causal, self.d ** -0.5)
            mean_abs, _ = oracle.attend(q[r0:r0 + lq], K, np.abs(V), self.causal, self.d ** -0.5)
            tol = (half_p + 2.0 ** -14) * mean_abs * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
            err = np.abs(out[r0:r0 + lq] - want)
            assert np.all(err <= tol), (b, float((err - tol).max()), float(err.max()))
            z = lse[:, r0:r0 + lq]
            assert np.array_equal(np.isfinite(z), np.isfinite(want_lse))
            fin = np.isfinite(want_lse)
            assert np.all(np.abs(z[fin] - want_lse[fin]) <= LSE_TOL), b
            r0 += lq


@pytest.fixture
def gpu(pkv):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


rnd = np.random.default_rng(77)
CASES = dict(
    few_rows=dict(starts=[0, 4], prefix=[512], own=[3, 60, 1, 30], q=[1] * 4),                     # one warp-MMA tile
    one_tile=dict(starts=[0, 20], prefix=[1000], own=rnd.integers(1, 200, 20), q=[1] * 20),        # prefix % page != 0
    two_tiles=dict(starts=[0, 50], prefix=[1536], own=rnd.integers(1, 900, 50), q=[1] * 50),
    odd_tiles=dict(starts=[0, 45], prefix=[2001], own=rnd.integers(5, 300, 45), q=rnd.integers(1, 6, 45), hq=6, hkv=2),
    groups=dict(starts=[0, 9, 10, 30], prefix=[640, 300, 1300], own=rnd.integers(6, 100, 33),
                q=list(rnd.integers(0, 6, 30)) + [1, 2, 90]),
    new_tokens=dict(starts=[0, 12], prefix=[700], own=rnd.integers(0, 100, 12), q=rnd.integers(1, 5, 12),
                    new=rnd.integers(4, 8, 12)),
    long_run_inside=dict(starts=[0, 8], prefix=[500], own=[20] * 8, q=[1, 1, 300, 1, 1, 33, 1, 2],
                         new=[1, 1, 300, 1, 1, 33, 1, 2]),
    prefix_only=dict(starts=[0, 5], prefix=[512], own=[0, 40, 0, 16, 3], q=[1] * 5),
    not_all_see_it=dict(starts=[0, 5], prefix=[512], own=[0, 4, 3, 16, 9], q=[4, 4, 8, 4, 4]),
    non_causal=dict(starts=[0, 12], prefix=[900], own=rnd.integers(0, 50, 12), q=rnd.integers(1, 9, 12), causal=False),
    d64=dict(starts=[0, 33], prefix=[1100], own=rnd.integers(1, 300, 33), q=[2] * 33, d=64, hq=12, hkv=2, new=[2] * 33),
    d256=dict(starts=[0, 20], prefix=[1100], own=rnd.integers(1, 300, 20), q=[1] * 20, d=256, hq=8, hkv=2),
    d256_few=dict(starts=[0, 2], prefix=[1100], own=[20, 30], q=[1] * 2, d=256, hq=8, hkv=2),
    mqa=dict(starts=[0, 10], prefix=[1100], own=rnd.integers(1, 900, 10), q=[1] * 10, hq=32, hkv=1),
    wide=dict(starts=[0, 3], prefix=[600], own=[5, 600, 77], q=[1] * 3, hq=60, hkv=1),
    not_shared=dict(starts=[0, 3], prefix=[600], own=[5, 600, 77], q=[1] * 3, hq=200, hkv=1, shares=False),  # head sub-groups
    mha=dict(starts=[0, 40], prefix=[600], own=rnd.integers(1, 90, 40), q=[1] * 40, hq=3, hkv=3),
    page1=dict(starts=[0, 20], prefix=[333], own=rnd.integers(1, 90, 20), q=[1] * 20, page=1),
    page4=dict(starts=[0, 20], prefix=[335], own=rnd.integers(1, 90, 20), q=[1] * 20, page=4),
    page4_few=dict(starts=[0, 3], prefix=[335], own=[20, 30, 8], q=[1] * 3, page=4),
    page2=dict(starts=[0, 20], prefix=[334], own=rnd.integers(1, 90, 20), q=[1] * 20, page=2),
    outside_split=dict(starts=[0, 10], prefix=[900], own=list(rnd.integers(1, 90, 10)) + [9000, 3, 12000], q=[1] * 13),
    page24=dict(starts=[0, 20], prefix=[480], own=rnd.integers(1, 90, 20), q=[1] * 20, page=24),
    page256=dict(starts=[0, 20], prefix=[800], own=rnd.integers(1, 900, 20), q=[1] * 20, page=256),
    ragged=dict(starts=[0, 20], prefix=[480], own=rnd.integers(1, 90, 20), q=[1] * 20, ragged=True),
    many_chunks=dict(starts=[0, 20], prefix=[20000], own=rnd.integers(1, 5000, 20), q=[1] * 20, hq=4, hkv=1),
    many_chunks_d64=dict(starts=[0, 20], prefix=[20000], own=rnd.integers(1, 50, 20), q=[1] * 20, hq=4, hkv=1, d=64),
    many_chunks_d256=dict(starts=[0, 20], prefix=[20000], own=rnd.integers(1, 50, 20), q=[1] * 20, hq=4, hkv=1, d=256),
    full=dict(starts=[0, 64], prefix=[6000], own=rnd.integers(1, 1500, 64), q=[1] * 64, hq=32, hkv=8),
    one_sm=dict(starts=[0, 20], prefix=[900], own=rnd.integers(1, 400, 20), q=[1] * 20, num_sms=1),
    few_sms=dict(starts=[0, 20], prefix=[1900], own=rnd.integers(1, 400, 20), q=[1] * 20, num_sms=7),
)
FP8 = ("few_rows", "one_tile", "two_tiles", "odd_tiles", "groups", "new_tokens", "long_run_inside", "prefix_only", "d64",
       "d256", "d256_few", "page2", "mqa", "wide", "page1", "page4", "page24", "outside_split", "many_chunks", "full", "one_sm", "few_sms")


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_against_64_bits(pkv, gpu, name):
    c = Shared(pkv, gpu, 1, **CASES[name])
    assert c.run() == 0, pkv.last_error()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("name", FP8)
def test_fp8_against_64_bits(pkv, gpu, name):
    c = Shared(pkv, gpu, 2, fp8=True, **CASES[name])
    assert c.run() == 0, pkv.last_error()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["one_tile", "few_rows", "d64"])
def test_fp8_quantised_queries(pkv, gpu, name):
    c = Shared(pkv, gpu, 3, fp8=True, q_scale=0.02, **CASES[name])
    assert c.run() == 0, pkv.last_error()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["groups", "two_tiles"])
def test_same_bits_every_run_and_near_the_plain_plan(pkv, gpu, name):
    torch = gpu
    c = Shared(pkv, torch, 4, **CASES[name])
    assert c.run() == 0
    first, lse = c.out.clone(), c.lse.clone()
    c.out.fill_(float("nan"))
    assert c.run() == 0
    assert torch.equal(first, c.out) and torch.equal(lse, c.lse)
    plain = pkv.plan(c.problem, c.q_lens, c.cache, c.new)
    ws = pkv.workspace_tensor(plain.workspace_bytes)
    plain.upload(ws)
    pkv.attn_varlen_kvcache_fwd(c.problem, c.args(), plain, ws)
    assert pkv.get_status(ws) == 0
    c.check()
    # without a workspace of the caller's
    c.out.fill_(float("nan"))
    pkv.attn_varlen_kvcache_fwd_noalloc(c.problem, c.args(), c.plan)
    assert pkv.get_status_noalloc() == 0
    assert torch.equal(first, c.out)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 4, 16])
def test_long_query_runs_of_one_cta_at_head_dim_256(pkv, gpu, page):
    """Items one after another on one SM, whose last V tile has rows past the sequence to zero: the zeros go into
    that tile's stage, not into the one before it that still waits for its copies (slow over small pages)."""
    c = Shared(pkv, gpu, 7, starts=[0, 8], prefix=[0], own=[1255] * 8, q=[33] * 8, hq=24, hkv=3, d=256, page=page,
               num_sms=1, shares=False)
    for _ in range(3):
        c.out.fill_(float("nan"))
        assert c.run() == 0
        c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["two_tiles", "few_rows", "d64", "d256"])
def test_strided_queries_and_outputs(pkv, gpu, name):
    """Queries out of a packed projection, outputs into wider rows, no lse; nothing around them is written."""
    torch = gpu
    c = Shared(pkv, torch, 13, **CASES[name])
    tq, hq, d = c.q.shape
    packed = torch.full((tq + 2, hq + 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    packed[:tq, 1:hq + 1] = c.q
    c.q = packed[:tq, 1:hq + 1]
    wide = torch.full((tq + 2, hq, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    c.out = wide[1:tq + 1, :, :d]
    assert c.run() == 0
    c.check()
    first = c.out.clone()
    assert torch.all(wide[0] == 7.0) and torch.all(wide[tq + 1] == 7.0) and torch.all(wide[:, :, d:] == 7.0)
    c.out.fill_(0.0)
    pkv.attn_varlen_kvcache_fwd(c.problem, c.args(lse=None), c.plan, c.ws)
    assert pkv.get_status(c.ws) == 0
    assert torch.equal(first, c.out)


@pytest.mark.gpu
@pytest.mark.parametrize("name,fp8", [("two_tiles", False), ("two_tiles", True), ("few_rows", False), ("d64", False),
                                      ("mqa", True), ("not_shared", False), ("d256", False)])
def test_calls_between_kernels_that_write_and_read(pkv, gpu, name, fp8):
    """A call may start while the kernel before it drains: it attends the queries which that kernel wrote, and what
    follows reads its output, call after call, from the host and in a graph."""
    torch = gpu
    c = Shared(pkv, torch, 17, fp8=fp8, **CASES[name])
    queries = [c.q.clone(), (c.q.float() * 0.5 + 0.1).bfloat16(), c.q.flip(0).contiguous()]
    want = []
    for q in queries:
        c.q.copy_(q)
        torch.cuda.synchronize()
        assert c.run() == 0
        torch.cuda.synchronize()
        want.append(c.out.clone())
    busy = torch.randn(1 << 24, device="cuda")
    args = c.args()

    def chain(got):
        for i in range(12):
            busy.mul_(1.0001)                     # something that takes a while
            c.q.copy_(queries[i % 3])
            pkv.attn_varlen_kvcache_fwd(c.problem, args, c.plan, c.ws)
            got[i].copy_(c.out)

    got = [torch.empty_like(c.out) for _ in range(12)]
    chain(got)
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))
    for g in got:
        g.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(got)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))
    assert pkv.get_status(c.ws) == 0


@pytest.mark.gpu
def test_placed_rows_where_nothing_is_shared(pkv, gpu):
    """A plan that ends up sharing nothing takes query rows placed by the caller, split units among them."""
    torch = gpu
    c = Shared(pkv, torch, 19, starts=[0, 3], prefix=[600], own=[5, 9000, 7700], q=[1] * 3, hq=200, hkv=1, shares=False)
    assert c.run() == 0 and c.plan.stats()["num_split_units"] > 0
    want, want_lse = c.out.clone(), c.lse.clone()
    at = [7, 2, 4]                                # rows of the three sequences among nine
    q = torch.zeros(9, *c.q.shape[1:], dtype=torch.bfloat16, device="cuda")
    q[at] = c.q
    out = torch.full_like(q, 7.0)
    lse = torch.full((c.hq, 9), 7.0, dtype=torch.float32, device="cuda")
    cu = H.i32(at + [9])
    pkv.attn_varlen_kvcache_fwd(c.problem, c.args(q=q, out=out, lse=lse, cu_seqlens_q=cu, q_rows=9), c.plan, c.ws)
    assert pkv.get_status(c.ws) == 0
    assert torch.equal(out[at], want) and torch.equal(lse[:, at], want_lse)
    out[at], lse[:, at] = 7.0, 7.0
    assert torch.all(out == 7.0) and torch.all(lse == 7.0)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["two_tiles", "few_rows"])
def test_queries_from_another_stream(pkv, gpu, name):
    """The queries come from a side stream, joined by an event right before the call."""
    torch = gpu
    c = Shared(pkv, torch, 18, **CASES[name])
    assert c.run() == 0
    want, q = c.out.clone(), c.q.clone()
    busy, side, args = torch.randn(1 << 25, device="cuda"), torch.cuda.Stream(), c.args()
    main = torch.cuda.current_stream()
    for _ in range(5):
        c.q.fill_(0.0)
        c.out.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            busy.mul_(1.0001)
            c.q.copy_(q)
        c.lens.add_(0)                            # a kernel of the call's own stream, done at once
        main.wait_stream(side)
        pkv.attn_varlen_kvcache_fwd(c.problem, args, c.plan, c.ws)
        torch.cuda.synchronize()
        assert torch.equal(want, c.out)
    assert pkv.get_status(c.ws) == 0


@pytest.mark.gpu
def test_two_calls_at_once(pkv, gpu):
    """Calls on two streams, each with its plan and workspace."""
    torch = gpu
    cases = [Shared(pkv, torch, 14, **CASES["full"]), Shared(pkv, torch, 15, fp8=True, **CASES["two_tiles"]),
             Shared(pkv, torch, 16, **CASES["new_tokens"])]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [c.args() for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, a, st in zip(cases, args, streams):
            pkv.attn_varlen_kvcache_fwd(c.problem, a, c.plan, c.ws, stream=st)
    torch.cuda.synchronize()
    for c in cases:
        assert pkv.get_status(c.ws) == 0
        c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_one_sequence_of_nan_stays_alone(pkv, gpu, fp8):
    """NaN among the own keys of the sequence whose table the prefix is read through touches no other."""
    torch = gpu
    c = Shared(pkv, torch, 5, fp8=fp8, **CASES["one_tile"])
    n0 = 1000 // 16
    pos = np.arange(n0 * 16, int(c.lk[0]))
    at = tuple(torch.from_numpy(x.astype(np.int64)).cuda() for x in (c.pages[0, pos // 16], pos % 16))
    for cache in (c.kc, c.vc):
        cache[at] = 0x7f if fp8 else float("nan")
    assert c.run() == 0
    assert torch.isnan(c.out[0]).all()
    c.out[0], c.lse[:, 0] = 0.0, 0.0
    c.q_lens, c.lk, c.pages = c.q_lens[1:], c.lk[1:], c.pages[1:]
    c.q, c.out, c.lse = c.q[1:], c.out[1:], c.lse[:, 1:]
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8,few", [(False, False), (True, False), (False, True)])
def test_dynamic_decode_loop_in_a_graph(pkv, gpu, fp8, few):
    """One dynamic plan and one captured graph over growing lengths; bounds are checked on the device."""
    torch = gpu
    steps, B = 4, 3 if few else 24
    own = np.random.default_rng(6).integers(0, 700, B)
    c = Shared(pkv, torch, 7, fp8=fp8, starts=[0, B], prefix=[1040], own=own, q=[1] * B, new=[1] * B, dynamic=True,
               bound=steps)
    base = c.cache.copy()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    args = c.args()
    pkv.attn_varlen_kvcache_fwd(c.problem, args, c.plan, c.ws, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pkv.attn_varlen_kvcache_fwd(c.problem, args, c.plan, c.ws, stream=stream)
    rng = np.random.default_rng(8)
    for s in range(steps):
        for t in (c.q, c.knew, c.vnew):
            t.copy_(bf16(torch, rng, *t.shape))
        c.lens.copy_(H.i32(base + s))
        c.lk = base + s + 1
        c.out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert pkv.get_status(c.ws) == 0
        c.check()
    for bad in (base + steps + 1, np.where(np.arange(B) == B - 1, 1039, base)):   # past the bound, below the prefix
        c.lens.copy_(H.i32(bad))
        graph.replay()
        torch.cuda.synchronize()
        assert pkv.get_status(c.ws) == 7


@pytest.mark.gpu
def test_static_length_mismatch_and_bad_page_are_reported(pkv, gpu):
    c = Shared(pkv, gpu, 9, **CASES["one_tile"])
    c.lens.copy_(H.i32(c.cache + 1))
    assert c.run() == 7
    c.lens.copy_(H.i32(c.cache))
    assert c.run() == 0
    table = c.pages.copy()
    table[0, 3] = 1 << 20                       # a page of the prefix, as the first sequence lists it
    c.extra = dict(block_table=H.i32(table))
    assert c.run() == 6


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_rotated_append_and_shared_attention_together(pkv, gpu, fp8):
    """A decode step as a model runs it: per-head norm and rotation, append, attention over a shared prefix, one call."""
    torch = gpu
    B, pre = 20, 512
    own = np.random.default_rng(10).integers(1, 90, B)
    c = Shared(pkv, torch, 11, fp8=fp8, starts=[0, B], prefix=[pre], own=own, q=[2] * B, new=[2] * B)
    rng = np.random.default_rng(12)
    table = table64(1024, 128)
    table_t = torch.from_numpy(table).cuda()
    qw, kw = (1 + 0.2 * bf16(torch, rng, c.d)).bfloat16(), (1 + 0.2 * bf16(torch, rng, c.d)).bfloat16()
    raw = c.q.clone()
    rope = pkv.make_rope_append_args(spec=pkv.make_rope_spec(cos_sin=table_t, q_weight=qw, k_weight=kw), q_out=c.q)
    q_in = raw.clone()
    pkv.rope_attn_varlen_kvcache_fwd(c.problem, c.args(q=q_in), rope, c.plan, c.ws)
    assert pkv.get_status(c.ws) == 0
    pos = np.concatenate([n + np.arange(2) for n in c.cache])
    want_q, mag = rows64(np64(raw), np64(qw), pos, table, False, 1e-6)
    close_bf16(c.q, want_q, mag)
    if not fp8:
        want_k, mag = rows64(np64(c.knew), np64(kw), pos, table, False, 1e-6)
        seq = np.repeat(np.arange(B), 2)
        got = c.kc[torch.from_numpy(c.pages[seq, pos // 16].astype(np.int64)).cuda(), torch.from_numpy(pos % 16).cuda()]
        close_bf16(got, want_k, mag)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
def test_lengths_below_the_prefix_are_reported_where_nothing_is_shared(pkv, gpu, wide):
    """A dynamic plan checks its prefixes whether or not they pay: sharing declined by the time model, or never
    possible (head groups of more than 64)."""
    torch = gpu
    B = 3
    kw = dict(hq=200, hkv=1) if wide else dict(hq=8, hkv=2)
    c = Shared(pkv, torch, 31, starts=[0, B], prefix=[256], own=[5, 40, 17], q=[1] * B, new=[1] * B, dynamic=True,
               bound=3, shares=not wide, **kw)
    c.plan = pkv.plan_shared_prefix(c.problem, c.q_lens, c.cache + 3, c.new, group_starts=[0, B], prefix_lens=[256],
                                    dynamic=True)
    plain = pkv.plan_decode_dynamic(c.problem, c.q_lens, c.cache + 3, c.new)
    assert c.plan.items() == plain.items() and c.plan.stats()["num_split_units"] == 0
    c.ws = pkv.workspace_tensor(c.plan.workspace_bytes)
    c.plan.upload(c.ws)
    assert c.run() == 0
    c.check()
    # (-1: the append, which comes first, reports the position)
    for at, lc, status in ((1, 255, 7), (1, 256, 0), (2, -1, 6), (0, int(c.cache[0]) + 4, 7), (0, int(c.cache[0]), 0)):
        lens = c.cache.copy()
        lens[at] = lc
        c.lens.copy_(H.i32(lens))
        assert c.run() == status
