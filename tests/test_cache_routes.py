"""Attention over a 4-bit cache by either route, tiles straight over its rows and tensor-core tiles over copies of them:
the same answers, the same precision, over the whole range of its inputs."""
import numpy as np
import pytest
import torch

from tests import long_cache as LC
from tests.test_fp4 import attend


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_variable_gb300 as m
    from paged_kv_variable_gb300 import build as b
    b.build()
    m.lib()
    return m


# ------------------------------------------------------------------ pages out of range
@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(64, 32, 8), (128, 16, 4), (256, 8, 2)])
@pytest.mark.parametrize("bad", ["past the pool", "negative", "past the list"])
def test_rows_of_a_bad_page_are_zeros_by_either_route(pkv, d, hq, hkv, bad):
    """Whatever the workspace held before: a page out of range is recorded and its rows count as zeros, bit for bit as a
    page of zeros in its place does."""
    lens, lq = [300, 900], [1, 700]
    cache = LC.Cache(81, dtype="fp4", lens=lens, hkv=hkv, d=d, page=16)
    q, out, lse, plan, ws, args, prob = attend(pkv, cache, hq, lq, [0, 0])
    assert {(it["seq"], it["kind"]) for it in plan.items()} == {(0, 0), (1, 1)}
    spare = (set(range(cache.pages)) - set(cache.table_np.ravel().tolist())).pop()
    for held in cache.kv:
        for t in held:
            t[spare] = 0
    n = [-(-x // 16) for x in lens]
    flat = LC.i32(np.concatenate([cache.table_np[b, :k] for b, k in enumerate(n)]))
    indptr = LC.i32(np.cumsum([0] + n))
    args = cache.args(pkv, q=q, out=out, lse=lse, cu_seqlens_q=LC.i32([0, 1, 701]), max_seqlen_q=700,
                      block_table=flat, page_indptr=indptr)
    at = [2, n[0] + 3] if bad != "past the list" else [n[0] + n[1] - 1]
    flat[at] = spare
    pkv.attn_varlen_kvcache_fwd(prob, args, plan, ws)
    assert pkv.get_status(ws) == 0
    want = out.clone(), lse.clone()
    if bad == "past the list":
        indptr[2] -= 1
    else:
        flat[at] = cache.pages if bad == "past the pool" else -1
    for fill in (None, 0xFF):  # what the call before left there, and NaN
        if fill is not None:
            ws.fill_(fill)
        plan.upload(ws)
        pkv.attn_varlen_kvcache_fwd(prob, args, plan, ws)
        assert pkv.get_status(ws) == 6
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16])
def test_rows_that_no_copy_writes_are_not_seen(pkv, page):
    """The copies' last pages end behind the sequences: what the workspace held there shows nowhere."""
    cache = LC.Cache(82, dtype="fp4", lens=[900, 513, 129], hkv=4, d=128, page=page)
    q, out, lse, plan, ws, args, prob = attend(pkv, cache, 16, [700, 300, 129], [0] * 3)
    assert {it["kind"] for it in plan.items()} == {1}
    want = out.clone(), lse.clone()
    ws.fill_(0xFF)
    plan.upload(ws)
    pkv.attn_varlen_kvcache_fwd(prob, args, plan, ws)
    assert pkv.get_status(ws) == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
