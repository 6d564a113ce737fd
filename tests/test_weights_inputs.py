"""What attn_weights and kv_gather read by offsets on the device: tensors with too few values are refused before a launch,
rows outside of them by the kernel."""
import numpy as np
import pytest
import torch

from tests import long_cache as LC
from tests.test_fp4 import make as make_fp4
from tests.test_rope import _Fake
from tests.test_weights import S, make


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_variable_gb300 as m
    from paged_kv_variable_gb300 import build as b
    b.build()
    m.lib()
    return m


@pytest.mark.parametrize("over,word", [
    (dict(lse=_Fake((1, 1), "float32")), "lse"), (dict(lse=_Fake((4, 4), "bfloat16")), "lse"),
    (dict(lse=_Fake((4, 4), "float64")), "lse"), (dict(lse=_Fake((0,), "float32")), "lse"),
    (dict(cu_seqlens_q=_Fake((1,), "int32")), "cu_seqlens_q"), (dict(cu_seqlens_q=_Fake((2,), "int32")), "cu_seqlens_q"),
    (dict(cu_seqlens_q=_Fake((3,), "int64")), "cu_seqlens_q"),
    (dict(k_new=_Fake((4, 2, 64)), v_new=_Fake((4, 2, 64)), cu_seqlens_knew=_Fake((2,), "int32")), "cu_seqlens_knew"),
    (dict(k_new=_Fake((4, 2, 64)), v_new=_Fake((4, 2, 64)), cu_seqlens_knew=_Fake((3,), "int64")), "cu_seqlens_knew"),
    (dict(q=_Fake((4, 4, 64), "float16")), "q "), (dict(cache_seqlens=_Fake((1,), "int32")), "cache_seqlens"),
])
def test_weights_of_short_tensors_are_refused(pkv, over, word):
    prob, args = make(pkv, **over)
    with pytest.raises(pkv.PkvError, match=word) as e:
        pkv.attn_weights(prob, args, pkv.make_weights_args(scores=S), stream=0)
    assert e.value.status == 1


@pytest.mark.parametrize("q,lse,rows", [(4, (4, 4), 4), (9, (4, 4), 4), (4, (4, 9), 4), (4, (19,), 4), (3, (4, 2), 2)])
def test_rows_that_the_tensors_hold(pkv, q, lse, rows):
    """The bound that goes with the call: the rows of the shorter one of q and lse.  (The call ends at a later check.)"""
    prob, args = make(pkv, q=_Fake((q, 4, 64), ptr=(1 << 20) + 8), lse=_Fake(lse, "float32"))
    w = pkv.make_weights_args(scores=S)
    with pytest.raises(pkv.PkvError, match="aligned"):
        pkv.attn_weights(prob, args, w, stream=0)
    assert w.max_total_q == rows
    # addresses put in by hand: nothing is known of them
    args.q, args.lse = (1 << 20) + 24, 1 << 22
    with pytest.raises(pkv.PkvError, match="aligned"):
        pkv.attn_weights(prob, args, w, stream=0)
    assert w.max_total_q == 0


@pytest.mark.parametrize("starts", [0, 1])
def test_gathers_with_short_starts_are_refused(pkv, starts):
    prob, args = make_fp4(pkv)
    g = pkv.make_gather_args(cu_rows=_Fake((3,), "int32"), k_out=_Fake((4, 2, 64)), starts=_Fake((starts,), "int32"))
    with pytest.raises(pkv.PkvError, match="starts"):
        pkv.kv_gather(prob, args, g, 4, stream=0)


@pytest.mark.gpu
@pytest.mark.parametrize("lq", [1, 40])
@pytest.mark.parametrize("what", ["total", "beyond", "negative"])
def test_rows_outside_of_the_tensors_are_not_read(pkv, lq, what):
    """Offsets beyond q and lse, or that leave their own total: recorded, those sequences' scores as they were."""
    cache = LC.Cache(91, dtype="bf16", lens=[100, 70, 64], hkv=2, d=64, page=16)
    q = torch.randn(3 * lq, 4, 64, device="cuda").bfloat16()
    lse = torch.zeros(4, 3 * lq, device="cuda")
    good = [0, lq, 2 * lq, 3 * lq]
    cu = {"total": [0, lq, 2 * lq, 3 * lq + 1], "beyond": [0, 3 * lq, 2 * lq, 2 * lq], "negative": [-lq, 0, lq, 2 * lq]}[what]
    left = {"total": [0, 1, 2], "beyond": [0, 1], "negative": [0]}[what]
    prob, found = cache.problem(pkv, 4), []
    for c in (good, cu):
        status = torch.zeros(3, dtype=torch.int32, device="cuda")
        scores = torch.full((3, 2, 100), 3.0, device="cuda")
        args = cache.args(pkv, q=q, lse=lse, cu_seqlens_q=LC.i32(c), max_seqlen_q=3 * lq)
        pkv.attn_weights(prob, args, pkv.make_weights_args(scores=scores, max_seqlen_k=100), status)
        found.append((status.tolist(), scores))
    assert found[0][0] == [0, 0, 0] and found[1][0][0] == 7
    for b, n in enumerate(cache.lens):
        assert not bool((found[0][1][b, :, :n] == 3).any())
        assert bool((found[1][1][b] == 3).all()) == (b in left)
