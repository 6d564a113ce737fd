"""What the Python binding refuses before anything is launched: tensors that hold
fewer rows than the call reads or writes, or other heads, and pairs that do not
share their strides.  (The library sees addresses alone.)"""
import numpy as np
import pytest

from tests.test_rope import _Fake


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_variable_gb300 as m
    from paged_kv_variable_gb300 import build as b
    b.build()
    m.lib()
    return m


def make(pkv, **over):
    """Two sequences, 3 + 1 queries and new tokens, 4 and 2 heads of 64."""
    prob = pkv.make_problem(batch=2, num_heads_q=4, num_heads_kv=2, head_dim=64, page_size=16, cache_capacity=64,
                            num_pages=8, cache_dtype="bf16", causal=True, softmax_scale=0.125)
    c = _Fake((8, 16, 2, 64), ptr=1 << 24)
    kw = dict(q=_Fake((4, 4, 64)), out=_Fake((4, 4, 64)), lse=_Fake((4, 4), "float32"), cu_seqlens_q=_Fake((3,), "int32"),
              max_seqlen_q=3, k_cache=c, v_cache=c, cache_seqlens=_Fake((2,), "int32"), k_new=_Fake((4, 2, 64)),
              v_new=_Fake((4, 2, 64)), cu_seqlens_knew=_Fake((3,), "int32"), block_table=_Fake((2, 4), "int32"))
    kw.update(over)
    return prob, pkv.make_args(**kw), pkv.plan(prob, [3, 1], [37, 5], [3, 1], num_sms=4)


def workspace():
    """One that the library refuses (its address), after the binding's own checks."""
    ws = _Fake((1 << 20,), "uint8", ptr=(1 << 28) + 16)
    ws.numel, ws.element_size = (lambda: 1 << 20), (lambda: 1)
    return ws


def calls(pkv, prob, args, pl, q_out=None):
    """The calls that read every tensor of args, each as a function."""
    rope = pkv.make_rope_append_args(spec=pkv.make_rope_spec(cos_sin=_Fake((64, 64), "float32")),
                                     q_out=q_out or _Fake((4, 4, 64)))
    ws = workspace()
    return [lambda: pkv.attn_varlen_kvcache_fwd(prob, args, pl, ws, stream=0),
            lambda: pkv.rope_attn_varlen_kvcache_fwd(prob, args, rope, pl, ws, stream=0)]


def test_enough_rows_reach_the_library(pkv):
    for over in ({}, dict(q=_Fake((9, 4, 64)), k_new=_Fake((5, 2, 64)), v_new=_Fake((5, 2, 64))),
                 dict(lse=_Fake((4, 9), "float32")), dict(lse=None)):
        for call in calls(pkv, *make(pkv, **over)):
            with pytest.raises(pkv.PkvError) as e:
                call()
            assert e.value.status == 1 and "workspace" in pkv.last_error()


@pytest.mark.parametrize("over", [
    dict(q=_Fake((3, 4, 64))), dict(q=_Fake((4, 2, 64))), dict(q=_Fake((4, 4, 32))),
    dict(out=_Fake((3, 4, 64))), dict(out=_Fake((4, 3, 64))), dict(lse=_Fake((4, 3), "float32")),
    dict(k_new=_Fake((3, 2, 64)), v_new=_Fake((3, 2, 64))), dict(k_new=_Fake((4, 1, 64)), v_new=_Fake((4, 1, 64))),
    dict(k_new=_Fake((4, 2, 32)), v_new=_Fake((4, 2, 32)))])
def test_too_few_rows_or_other_heads(pkv, over):
    for call in calls(pkv, *make(pkv, **over)):
        with pytest.raises(ValueError) as e:
            call()
        assert isinstance(e.value, pkv.PkvError) and e.value.status == 1


def test_rows_placed_by_the_caller(pkv):
    """q_rows is the row count of q, out and lse, of a plan for shared prefixes that shares nothing too."""
    for rows, fits in ((9, True), (8, False)):
        q = _Fake((rows, 4, 64))
        prob, args, pl = make(pkv, q=q, out=q, lse=None, q_rows=9)
        none = pkv.plan_shared_prefix(prob, [3, 1], [37, 5], [3, 1], group_starts=[0], prefix_lens=[], num_sms=4)
        for p in (pl, none):
            with pytest.raises(pkv.PkvError) as e:
                calls(pkv, prob, args, p)[0]()
            assert fits != isinstance(e.value, ValueError)


def test_appends(pkv):
    few = dict(k_new=_Fake((3, 2, 64)), v_new=_Fake((3, 2, 64)))
    prob, args, _ = make(pkv, **few)
    rope = pkv.make_rope_append_args(spec=pkv.make_rope_spec(cos_sin=_Fake((64, 64), "float32")))
    with pytest.raises(ValueError):
        pkv.kv_append(prob, args, 4, stream=0)
    with pytest.raises(ValueError):
        pkv.rope_kv_append(prob, args, rope, 0, 4, stream=0)
    prob, args, _ = make(pkv, q=_Fake((3, 4, 64)))
    with_q = pkv.make_rope_append_args(spec=pkv.make_rope_spec(cos_sin=_Fake((64, 64), "float32")),
                                       q_out=_Fake((4, 4, 64)))
    with pytest.raises(ValueError):
        pkv.rope_kv_append(prob, args, with_q, 4, 4, stream=0)
    # the rotating forms take bf16 rows alone
    for over in (dict(q=_Fake((4, 4, 64), "float16")), dict(k_new=_Fake((4, 2, 64), "uint8"), v_new=_Fake((4, 2, 64)))):
        prob, args, _ = make(pkv, **over)
        with pytest.raises(ValueError):
            pkv.rope_kv_append(prob, args, with_q, 4, 4, stream=0)


def test_pairs_share_shape_and_strides(pkv):
    packed = [4 * 64, 64, 1]
    for over in (dict(v_new=_Fake((4, 2, 64), strides=packed)), dict(v_new=_Fake((3, 2, 64))),
                 dict(v_cache=_Fake((8, 16, 2, 64), strides=[4096, 256, 64, 1])),
                 dict(v_cache=_Fake((7, 16, 2, 64)))):
        with pytest.raises(ValueError):
            make(pkv, **over)
    make(pkv, k_new=_Fake((4, 2, 64), strides=packed), v_new=_Fake((4, 2, 64), strides=packed))
    # (the stride of a dim of one element is not used)
    make(pkv, k_new=_Fake((1, 2, 64)), v_new=_Fake((1, 2, 64), strides=[7, 64, 1]))


@pytest.mark.parametrize("over", [
    dict(cu_seqlens_q=_Fake((2,), "int32")), dict(cache_seqlens=_Fake((1,), "int32")),
    dict(cu_seqlens_knew=_Fake((2,), "int32")), dict(block_table=_Fake((1, 4), "int32")),
    dict(block_table=_Fake((8,), "int32"), page_indptr=_Fake((2,), "int32")),
    *(dict(k_cache=_Fake(s), v_cache=_Fake(s)) for s in ((7, 16, 2, 64), (8, 8, 2, 64), (8, 16, 1, 64), (8, 16, 2, 32)))])
def test_offsets_tables_and_caches_too_small(pkv, over):
    prob, args, pl = make(pkv, **over)
    for call in calls(pkv, prob, args, pl):
        with pytest.raises(ValueError):
            call()


def test_a_ragged_page_list_reaches_the_library(pkv):
    for call in calls(pkv, *make(pkv, block_table=_Fake((5,), "int32"), page_indptr=_Fake((3,), "int32"))):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert "workspace" in pkv.last_error() and not isinstance(e.value, ValueError)


def test_an_address_put_in_later_is_taken_as_it_is(pkv):
    prob, args, pl = make(pkv, q=_Fake((3, 4, 64)))
    args.q = 1 << 21
    with pytest.raises(pkv.PkvError):
        calls(pkv, prob, args, pl)[0]()


def test_short_length_lists(pkv):
    prob, _, _ = make(pkv)
    for lens in (([3], [37, 5], [3, 1]), ([3, 1], [37], [3, 1]), ([3, 1], [37, 5], [3])):
        with pytest.raises(ValueError):
            pkv.plan(prob, *lens, num_sms=4)
        with pytest.raises(ValueError):
            pkv.plan_decode_dynamic(prob, *lens, num_sms=4)
    assert pkv.plan(prob, [3, 1, 9], [37, 5, 9], [3, 1, 9], num_sms=4).total_new == 4


def test_status_words(pkv):
    one = _Fake((1,), "int32")
    one.numel, one.element_size = (lambda: 1), (lambda: 4)
    prob, args, _ = make(pkv)
    spec = pkv.make_rope_spec(cos_sin=_Fake((64, 64), "float32"))
    with pytest.raises(ValueError):
        pkv.rope_kv_append(prob, args, pkv.make_rope_append_args(spec=spec), 0, 4, device_status=one, stream=0)
    with pytest.raises(ValueError):
        pkv.qk_norm_rope(pkv.make_qk_args(q=_Fake((4, 4, 64)), positions=_Fake((4,), "int32")), spec,
                         device_status=one, stream=0)


def test_structs_keep_their_tensors(pkv):
    """A table, weight or scale made in the call lives as long as the struct that holds its address."""
    import gc
    import weakref
    alive = {}

    def new(what, *shape, dtype="bfloat16"):
        t = _Fake(shape, dtype)
        alive[what] = weakref.ref(t)
        return t

    spec = pkv.make_rope_spec(cos_sin=new("table", 64, 64, dtype="float32"), q_weight=new("q_weight", 64),
                              k_weight=new("k_weight", 64))
    rope = pkv.make_rope_append_args(spec=spec, q_out=new("q_out", 4, 4, 64))
    del spec
    qk = pkv.make_qk_args(q=new("q", 4, 4, 64), k=new("k", 4, 2, 64), positions=new("pos", 4, dtype="int32"),
                          q_out=new("qo", 4, 4, 64), k_out=new("ko", 4, 2, 64))
    args = pkv.make_args(q=new("aq", 4, 4, 64), out=new("out", 4, 4, 64), lse=new("lse", 4, 4, dtype="float32"),
                         cu_seqlens_q=new("cu", 3, dtype="int32"), max_seqlen_q=3,
                         k_cache=new("kc", 8, 16, 2, 64), v_cache=new("vc", 8, 16, 2, 64),
                         cache_seqlens=new("lens", 2, dtype="int32"), k_new=new("kn", 4, 2, 64),
                         v_new=new("vn", 4, 2, 64), cu_seqlens_knew=new("cun", 3, dtype="int32"),
                         block_table=new("bt", 2, 4, dtype="int32"), k_scale=new("ks", 1, dtype="float32"),
                         v_scale=new("vs", 1, dtype="float32"), page_indptr=new("pi", 3, dtype="int32"),
                         q_scale=new("qs", 1, dtype="float32"))
    gc.collect()
    assert [w for w, r in alive.items() if r() is None] == []
    del rope, qk, args
    gc.collect()
    assert [w for w, r in alive.items() if r() is not None] == []


def test_current_stream_with_and_without_the_raw_query(pkv, monkeypatch):
    import types
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    assert pkv._stream_handle(None) == 103
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert pkv._stream_handle(None) == 77
    assert pkv._stream_handle(5) == 5 and pkv._stream_handle(types.SimpleNamespace(cuda_stream=9)) == 9
