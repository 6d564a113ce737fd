"""A call follows everything that was put on its stream before it.

A kernel that starts while its predecessor drains waits for that predecessor
alone, which need not itself have waited for what came before.  So only a call's
own kernels start early, behind one another.  The calls are captured and the
edges of the graph read: the one from the kernel before the call is an ordinary
one (the kernel starts once that has completed, and with it all before it).
"""
import ctypes

import numpy as np
import pytest

from tests import harness as H
from tests.test_rope import AppendCase, bf16
from tests.test_shared_prefix import Shared

pytestmark = pytest.mark.gpu

PROGRAMMATIC = 1  # CU_GRAPH_DEPENDENCY_TYPE_PROGRAMMATIC


@pytest.fixture(scope="module")
def pkv():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_variable_gb300 as m
    from paged_kv_variable_gb300 import build as b
    b.build()
    return m


class _EdgeData(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_uint8), ("to_port", ctypes.c_uint8), ("type", ctypes.c_uint8),
                ("reserved", ctypes.c_uint8 * 5)]


def edges_of(call):
    """Captures a kernel of torch's and then the call.  Returns the kinds of the
    edges out of that kernel, and of the others."""
    import torch
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    x = torch.zeros(1 << 16, device="cuda")
    call(stream)                                # once outside capture
    torch.cuda.synchronize()
    graph, n = ctypes.c_void_p(), ctypes.c_size_t()
    handle = ctypes.c_void_p(stream.cuda_stream)
    with torch.cuda.stream(stream):
        assert cu.cuStreamBeginCapture_v2(handle, 2) == 0    # (relaxed)
        x.add_(1.0)
        call(stream)
        assert cu.cuStreamEndCapture(handle, ctypes.byref(graph)) == 0
    assert cu.cuGraphGetRootNodes(graph, None, ctypes.byref(n)) == 0 and n.value == 1
    root = (ctypes.c_void_p * 1)()
    assert cu.cuGraphGetRootNodes(graph, root, ctypes.byref(n)) == 0
    assert cu.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(n)) == 0
    a, b, data = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (_EdgeData * n.value)()
    assert cu.cuGraphGetEdges_v2(graph, a, b, data, ctypes.byref(n)) == 0
    assert cu.cuGraphDestroy(graph) == 0
    first = [d.type for f, d in zip(a, data) if f == root[0]]
    return first, [d.type for f, d in zip(a, data) if f != root[0]]


def test_norm_and_rotation(pkv):
    import torch
    c = AppendCase(pkv, torch, 1, d=128, page=16, fp8=False, new=[1] * 5, cached=[9] * 5)
    pos = H.i32(np.arange(5))
    args = pkv.make_qk_args(q=c.q, k=c.k, positions=pos, q_out=c.q_out, k_out=torch.empty_like(c.k))
    assert edges_of(lambda s: pkv.qk_norm_rope(args, c.spec, stream=s)) == ([0], [])


@pytest.mark.parametrize("fp8", [False, True])
def test_appends(pkv, fp8):
    import torch
    c = AppendCase(pkv, torch, 2, d=128, page=16, fp8=fp8, new=[1] * 5, cached=[9] * 5)
    a = c.args()
    assert edges_of(lambda s: c.run(stream=s)) == ([0], [])
    assert edges_of(lambda s: pkv.kv_append(c.problem, a, c.tn, stream=s)) == ([0], [])


def attention(pkv, c, rope=False, new=True, num_sms=8, cache=None):
    import torch
    out = torch.empty_like(c.q_out)
    cached = c.cached if cache is None else cache
    plan = pkv.plan(c.problem, c.q_lens, cached, c.new if new else None, num_sms=num_sms)
    ws = pkv.workspace_tensor(plan.workspace_bytes)
    plan.upload(ws)
    lens = H.i32(cached)
    over = {} if new else dict(k_new=None, v_new=None, cu_seqlens_knew=None)
    args = c.args(out=out, cache_seqlens=lens, **over)

    def call(s):
        if rope:
            pkv.rope_attn_varlen_kvcache_fwd(c.problem, args, c.rope, plan, ws, stream=s)
        else:
            pkv.attn_varlen_kvcache_fwd(c.problem, args, plan, ws, stream=s)

    call.keep = (out, lens, args)
    return call, plan


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q", [1, 200])
def test_attention_over_the_cache_alone(pkv, d, fp8, q):
    import torch
    c = AppendCase(pkv, torch, 3, d=d, page=16, fp8=fp8, new=[q] * 3, cached=[4000, 900, 30])
    call, plan = attention(pkv, c, new=False, cache=c.cached + c.new)
    first, rest = edges_of(call)
    assert first == [0] and len(rest) == (plan.stats()["num_split_units"] > 0)


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_the_calls_own_kernels_overlap(pkv, fp8, rope):
    """Append, attention and combine of a decode call: each starts behind the one before it."""
    import torch
    c = AppendCase(pkv, torch, 4, d=128, page=16, fp8=fp8, new=[1] * 3, cached=[6000, 900, 30])
    call, plan = attention(pkv, c, rope=rope)
    assert plan.stats()["num_split_units"] > 0
    first, rest = edges_of(call)
    assert first == [0] and rest == [PROGRAMMATIC, PROGRAMMATIC]


@pytest.mark.parametrize("kw", [
    dict(starts=[0, 20], prefix=[900], own=[90] * 20, q=[1] * 20),
    dict(starts=[0, 20], prefix=[900], own=[90] * 20, q=[1] * 20, fp8=True),
    dict(starts=[0, 3], prefix=[900], own=[90] * 3, q=[1] * 3),
    dict(starts=[0, 20], prefix=[900], own=[90] * 20, q=[1] * 20, new=[1] * 20),
    dict(starts=[0, 20], prefix=[900], own=[90] * 20, q=[1] * 20, new=[1] * 20, fp8=True),
])
def test_shared_prefixes(pkv, kw):
    import torch
    c = Shared(pkv, torch, 5, **kw)
    args = c.args()
    first, rest = edges_of(lambda s: pkv.attn_varlen_kvcache_fwd(c.problem, args, c.plan, c.ws, stream=s))
    assert first == [0] and rest


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens", [2, 700])
@pytest.mark.parametrize("form", ["rotating", "plain", "call"])
def test_keys_and_values_written_just_before_and_read_just_after(pkv, form, tokens, fp8):
    """The append reads the queries, keys, values and lengths that the kernel before it
    wrote, and the kernel after it the cache: eager and in a graph, step after step."""
    import torch
    c = AppendCase(pkv, torch, 11, d=128, page=16, fp8=fp8, new=[tokens, 1, tokens // 2], cached=[20, 0, 33], far=900)
    rng = np.random.default_rng(12)
    inputs = [[bf16(torch, rng, *t.shape) for t in (c.q, c.k, c.v)] + [H.i32(np.array(lens, np.int32))]
              for lens in ([20, 0, 33], [7, 30, 2], [16, 1, 0])]
    empty = [c.kc.clone(), c.vc.clone()]
    out = torch.zeros_like(c.q_out)
    args = c.args(out=out)
    plans = []
    for lens in ([20, 0, 33], [7, 30, 2], [16, 1, 0]):
        plan = pkv.plan(c.problem, c.q_lens, lens, c.new)
        plans.append((plan, pkv.workspace_tensor(plan.workspace_bytes)))
        plan.upload(plans[-1][1])
    busy = torch.randn(1 << 24, device="cuda")

    def step(i, got):
        busy.mul_(1.0001)
        for cache, e in zip((c.kc, c.vc), empty):
            cache.copy_(e)
        for t, x in zip((c.q, c.k, c.v, c.lens), inputs[i % 3]):
            t.copy_(x)
        if form == "plain":
            pkv.kv_append(c.problem, args, c.tn)
        elif form == "rotating":
            pkv.rope_kv_append(c.problem, args, c.rope, c.tq, c.tn)
        else:
            plan, ws = plans[i % 3]
            pkv.rope_attn_varlen_kvcache_fwd(c.problem, args, c.rope, plan, ws)
        for g, x in zip(got, (c.kc, c.vc, c.q_out, out)):
            g.copy_(x)

    def buffers():
        return [torch.zeros_like(x) for x in (c.kc, c.vc, c.q_out, out)]

    def same(a, b):
        return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))

    c.q_out.zero_()
    want = []
    for i in range(3):
        want.append(buffers())
        step(i, want[-1])
        torch.cuda.synchronize()
        if form != "plain":                     # (against 64 bits)
            c.cached = inputs[i][3].cpu().numpy()
            c.check(*(H.to_numpy_bits(e).copy() for e in empty))
    assert not any(same(want[i], want[j]) for i, j in ((0, 1), (1, 2), (0, 2)))
    got = [buffers() for _ in range(9)]
    for i, g in enumerate(got):
        step(i, g)
    torch.cuda.synchronize()
    assert all(same(g, want[i % 3]) for i, g in enumerate(got))
    for g in got:
        for x in g:
            x.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, g in enumerate(got):
            step(i, g)
    graph.replay()
    torch.cuda.synchronize()
    assert all(same(g, want[i % 3]) for i, g in enumerate(got))
