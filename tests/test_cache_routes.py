"""Attention over a 4-bit cache by either route, tiles straight over its rows and tensor-core tiles over copies of them:
the same answers, the same precision, over the whole range of its inputs."""
import ctypes

import numpy as np
import pytest
import torch

from tests import long_cache as LC
from tests.test_fp4 import attend, check
from tests.test_stream_order import _EdgeData
from tests.test_weights import run_evict, run_weights


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


# ------------------------------------------------------------------ precision
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_scale", [1.5, 4.0])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_are_as_precise_as_decode_steps(pkv, d, q_scale, causal):
    """The bound of the tiles straight over the cache (P rounded to 11 bits, kept above the subnormals) holds for prompts
    over copies too: with sharp logits few keys take the weight, and the roundings of P do not average out."""
    lens, lq = [900, 1537, 65], [700, 300, 65]
    cache = LC.Cache(83, dtype="fp4", lens=lens, hkv=4, d=d, page=16)
    q, out, lse, plan, ws, args, prob = attend(pkv, cache, 16, lq, [0] * 3, causal=causal, q_scale=q_scale)
    assert {it["kind"] for it in plan.items()} == {1}
    check(cache, out, lse, q, lq, lens, causal)


@pytest.mark.gpu
def test_prompts_with_few_keys_of_weight(pkv):
    """Values of 0 under all keys but those with the smallest weights: a weight far below the largest one counts."""
    lens, lq, hkv, d = [640], [512], 2, 128
    x = np.random.default_rng(5).standard_normal((2, 640, hkv, d))
    x[1, :320] = 0                       # (causal: the first rows see zeros alone)
    x[0, :320] *= 3
    cache = LC.Cache(84, dtype="fp4", lens=lens, hkv=hkv, d=d, page=16, values=x)
    q, out, lse, plan, ws, args, prob = attend(pkv, cache, 32, lq, [0], causal=False, q_scale=4.0)
    assert {it["kind"] for it in plan.items()} == {1}
    check(cache, out, lse, q, lq, lens, False)


# ------------------------------------------------------------------ the range of the queries
def scaled(pkv, cache, q, lq, power, hq, causal=True, softmax_scale=None, routes=None):
    """Outputs for q 2^power and the softmax's scale 2^-power: the same numbers, but for what a narrower type loses."""
    rows = sum(lq)
    out = torch.full((rows, hq, cache.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, rows), float("nan"), dtype=torch.float32, device="cuda")
    prob = cache.problem(pkv, hq, causal, (softmax_scale or cache.d ** -0.5) * 2.0 ** -power)
    plan = pkv.plan(prob, lq, cache.lens)
    ws = pkv.workspace_tensor(plan.workspace_bytes)
    plan.upload(ws)
    q = (q.double() * 2.0 ** power).bfloat16()
    args = cache.args(pkv, q=q, out=out, lse=lse, cu_seqlens_q=LC.i32(np.cumsum([0] + lq)), max_seqlen_q=max(lq))
    pkv.attn_varlen_kvcache_fwd(prob, args, plan, ws)
    assert pkv.get_status(ws) == 0
    if routes is not None:
        assert {it["kind"] for it in plan.items()} == routes
    return out, lse, args, prob


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(64, 32, 4), (64, 32, 1), (128, 16, 4), (256, 8, 2)])
@pytest.mark.parametrize("power", [-100, -20, 20, 100])
def test_queries_of_any_magnitude(pkv, d, hq, hkv, power):
    """Queries near both ends of bf16's range, decode steps, drafts and prompts: the bits of the ordinary ones."""
    lens, lq = [700, 300, 129, 33, 900], [1, 1, 3, 1, 700]
    cache = LC.Cache(85, dtype="fp4", lens=lens, hkv=hkv, d=d, page=16)
    g = torch.Generator().manual_seed(6)
    q = (1.5 * torch.randn(sum(lq), hq, d, generator=g)).bfloat16().cuda()
    want = scaled(pkv, cache, q, lq, 0, hq, routes={0, 1})
    check(cache, want[0], want[1], q, lq, lens, True)
    got = scaled(pkv, cache, q, lq, power, hq)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq", [(64, 16), (64, 32), (128, 16), (256, 8)])
def test_rows_of_different_magnitudes_in_one_tile(pkv, d, hq):
    """Heads of a group from 2^-40 to 2^40 of one another, one of zeros, one with an infinity, which shows in no other."""
    lens, lq = [300, 40], [1, 1]
    cache = LC.Cache(86, dtype="fp4", lens=lens, hkv=1, d=d, page=16)
    g = torch.Generator().manual_seed(7)
    q = torch.randn(2, hq, d, generator=g).double().cuda()
    q = (q * torch.tensor([2.0 ** (20 * (h % 5 - 2)) for h in range(hq)], device="cuda").double()[None, :, None]).bfloat16()
    q[:, 3] = 0
    clean, q[:, 5, 7] = q.clone(), float("inf")
    want = scaled(pkv, cache, clean, lq, 0, hq)
    got = scaled(pkv, cache, q, lq, 0, hq)
    others = [h for h in range(hq) if h != 5]
    assert torch.equal(got[0][:, others], want[0][:, others]) and torch.equal(got[1][others], want[1][others])
    for h in range(hq):  # each head's row alone
        one = scaled(pkv, cache, clean[:, h:h + 1].contiguous(), lq, 0, 1)
        check(cache, one[0], one[1], clean[:, h:h + 1], lq, lens, True)
    check(cache, want[0], want[1], clean, lq, lens, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("d,hq,lq", [(64, 8, 1), (128, 16, 1), (256, 8, 1), (64, 16, 40), (128, 8, 300), (256, 4, 40)])
@pytest.mark.parametrize("power", [-100, -20, 20, 100])
def test_weights_of_queries_of_any_magnitude(pkv, dtype, d, hq, lq, power):
    lens = [400, 65]
    cache = LC.Cache(87, dtype=dtype, lens=lens, hkv=1, d=d, page=16)
    g = torch.Generator().manual_seed(8)
    q = (1.5 * torch.randn(2 * lq, hq, d, generator=g)).bfloat16().cuda()
    lse = torch.cat([f[1] for f in LC.attention(cache, q, [lq] * 2, lens, True)], 1).float().contiguous()
    status, found = torch.zeros(3, dtype=torch.int32, device="cuda"), []
    for x in (0, power):
        prob = cache.problem(pkv, hq, True, d ** -0.5 * 2.0 ** -x)
        qx = (q.double() * 2.0 ** x).bfloat16()
        scores = torch.zeros(2, 1, 400, device="cuda")
        args = cache.args(pkv, q=qx, lse=lse, cu_seqlens_q=LC.i32([0, lq, 2 * lq]), max_seqlen_q=lq)
        pkv.attn_weights(prob, args, pkv.make_weights_args(scores=scores, max_seqlen_k=400), status)
        found.append(scores)
    assert status.tolist() == [0, 0, 0] and torch.equal(*found)


# ------------------------------------------------------------------ the bytes of the copies
def kinds_of(pkv, lq, lens, hq, hkv, d):
    prob = pkv.make_problem(batch=len(lq), num_heads_q=hq, num_heads_kv=hkv, head_dim=d, page_size=64,
                            cache_capacity=-(-max(lens) // 64) * 64, num_pages=1 << 18, cache_dtype="fp4", causal=True,
                            softmax_scale=0.1)
    plan = pkv.plan(prob, lq, lens, None, num_sms=152)
    kinds = {}
    for it in plan.items():
        kinds.setdefault(it["seq"], set()).add(it["kind"])
    return [kinds[b] for b in range(len(lq))], plan.workspace_bytes


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (32, 8, 64), (16, 4, 256)])
def test_copies_up_to_their_bound(pkv, hq, hkv, d):
    """Prompts that fill the 4 GiB of copies keep them when more come; those that do not fit go without."""
    token = 4 * d * hkv
    keys = 16384 * 4096 // token
    full = (4 << 30) // (token * keys)
    for more in (0, 1, 7):
        kinds, size = kinds_of(pkv, [512] * (full + more), [keys] * (full + more), hq, hkv, d)
        assert [k == {1} for k in kinds].count(True) == full and [k == {0} for k in kinds].count(True) == more
        assert (4 << 30) < size < (4 << 30) + (64 << 20)
    # a long one that does not fit beside the others does not keep them out, nor a short one behind it
    kinds, _ = kinds_of(pkv, [512] * (full - 1) + [1024, 512], [keys] * (full - 1) + [2 * keys, keys // 2], hq, hkv, d)
    assert kinds == [{1}] * (full - 1) + [{0}, {1}]
    kinds, _ = kinds_of(pkv, [256] * (full // 2) + [64], [2 * keys] * (full // 2) + [2048], hq, hkv, d)
    assert kinds.count({1}) >= full // 2 and len(kinds) == full // 2 + 1


@pytest.mark.gpu
def test_prompts_without_a_workspace(pkv):
    """A prompt whose copies would not fit the fixed scratch is attended straight over the cache; what was planned stays."""
    lens, lq, hq = [8200, 40], [300, 1], 16
    cache = LC.Cache(88, dtype="fp4", lens=lens, hkv=8, d=128, page=16)
    q, out, lse, plan, ws, args, prob = attend(pkv, cache, hq, lq, [3, 1])
    assert {(it["seq"], it["kind"]) for it in plan.items()} == {(0, 1), (1, 0)} and plan.workspace_bytes > 32 << 20
    for _ in range(2):
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        pkv.attn_varlen_kvcache_fwd_noalloc(prob, args, plan)
        assert pkv.get_status_noalloc() == 0
        check(cache, out, lse, q, lq, lens, True)
    assert {(it["seq"], it["kind"]) for it in plan.items()} == {(0, 1), (1, 0)}
    args.keep[5][0] -= 1  # lengths other than the plan's
    pkv.attn_varlen_kvcache_fwd_noalloc(prob, args, plan)
    assert pkv.get_status_noalloc() == 7


# ------------------------------------------------------------------ profiling events
def nodes_of(call):
    """Captures a call: its nodes in order, each "kernel" or "event" (they form a chain)."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    graph, n = ctypes.c_void_p(), ctypes.c_size_t()
    handle = ctypes.c_void_p(stream.cuda_stream)
    with torch.cuda.stream(stream):
        assert cu.cuStreamBeginCapture_v2(handle, 2) == 0  # (relaxed)
        call(stream)
        assert cu.cuStreamEndCapture(handle, ctypes.byref(graph)) == 0
    root = (ctypes.c_void_p * 1)()
    assert cu.cuGraphGetRootNodes(graph, None, ctypes.byref(n)) == 0 and n.value == 1
    assert cu.cuGraphGetRootNodes(graph, root, ctypes.byref(n)) == 0
    assert cu.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(n)) == 0
    a, b, data = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (_EdgeData * n.value)()
    assert cu.cuGraphGetEdges_v2(graph, a, b, data, ctypes.byref(n)) == 0
    after, at, found = dict(zip(a, b)), root[0], []
    assert len(after) == n.value
    while at is not None:
        kind = ctypes.c_int()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(at), ctypes.byref(kind)) == 0
        found.append({0: "kernel", 7: "event"}[kind.value])
        at = after.get(at)
    assert cu.cuGraphDestroy(graph) == 0
    return found


@pytest.mark.gpu
@pytest.mark.parametrize("lens,lq,new,kinds", [
    ([900, 513], [700, 300], [0, 0], {1}), ([900, 513], [700, 300], [700, 0], {1}), ([900, 50], [700, 1], [0, 1], {0, 1}),
    ([900, 50], [1, 1], [1, 1], {0}),
])
def test_profiling_events_go_around_the_copies(pkv, lens, lq, new, kinds):
    """The start event stands behind the append and before everything else, the copies of prompts among it, whether or not
    tiles straight over the cache come first; the stop event behind the last attention launch."""
    cache = LC.Cache(89, dtype="fp4", lens=lens, hkv=4, d=128, page=16)
    q, out, lse, plan, ws, args, prob = attend(pkv, cache, 16, lq, new)
    assert {it["kind"] for it in plan.items()} == kinds
    call = lambda s: pkv.attn_varlen_kvcache_fwd(prob, args, plan, ws, stream=s)
    plain = nodes_of(call)
    assert set(plain) == {"kernel"}
    a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    a.record(), b.record()
    torch.cuda.synchronize()
    pkv.set_profile_events(a, b)
    try:
        found = nodes_of(call)
    finally:
        pkv.set_profile_events(None, None)
    assert found.count("event") == 2 and [k for k in found if k == "kernel"] == plain
    start = found.index("event")
    assert start == (1 if sum(new) else 0)                    # behind the append
    behind = found[found.index("event", start + 1) + 1:]
    assert len(behind) <= 1                                   # a combine at most
    assert plain == nodes_of(call)


# ------------------------------------------------------------------ rows placed by the caller
def placed(pkv, cache, hq, lq, starts, rows, *, dynamic=False, causal=True):
    """The same call with packed rows and with rows at `starts` of `rows`, the others NaN."""
    g = torch.Generator().manual_seed(9)
    q = (1.5 * torch.randn(sum(lq), hq, cache.d, generator=g)).bfloat16().cuda()
    at = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, lq)])
    q2 = torch.full((rows, hq, cache.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    q2[at] = q
    prob, found = cache.problem(pkv, hq, causal), []
    plan = (pkv.plan_decode_dynamic if dynamic else pkv.plan)(prob, lq, cache.lens)
    ws = pkv.workspace_tensor(plan.workspace_bytes)
    for x, cu, kw in ((q, np.cumsum([0] + lq), {}), (q2, starts + [rows], dict(q_rows=rows))):
        out = torch.full_like(x, 7.0)
        lse = torch.full((hq, x.shape[0]), 7.0, device="cuda")
        plan.upload(ws)
        args = cache.args(pkv, q=x, out=out, lse=lse, cu_seqlens_q=LC.i32(cu), max_seqlen_q=max(lq), **kw)
        pkv.attn_varlen_kvcache_fwd(prob, args, plan, ws)
        assert pkv.get_status(ws) == 0
        found.append((out, lse))
    (out, lse), (out2, lse2) = found
    check(cache, out, lse, q, lq, cache.lens, causal)
    assert torch.equal(out2[at], out) and torch.equal(lse2[:, at], lse)
    left = np.setdiff1d(np.arange(rows), at)
    assert bool((out2[left] == 7).all()) and bool((lse2[:, left] == 7).all())
    return plan


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(64, 64, 4), (128, 32, 4), (256, 16, 4)])
@pytest.mark.parametrize("dynamic", [False, True])
def test_placed_rows_of_split_runs(pkv, d, hq, hkv, dynamic):
    """Runs of more than one tile whose keys are split: the parts of a later tile are joined into its own rows."""
    cache = LC.Cache(71, dtype="fp4", lens=[9011, 5000, 30], hkv=hkv, d=d, page=16)
    plan = placed(pkv, cache, hq, [5, 4, 3], [11, 2, 20], 24, dynamic=dynamic)
    split = {it["q_index0"] for it in plan.items() if it["partial_slot"] >= 0}
    assert len(split) > 1


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 4), (256, 8, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_placed_rows_of_prompts(pkv, d, hq, hkv, causal):
    cache = LC.Cache(72, dtype="fp4", lens=[900, 50, 1537], hkv=hkv, d=d, page=16)
    plan = placed(pkv, cache, hq, [700, 1, 300], [350, 3, 20], 1100, causal=causal)
    assert {it["kind"] for it in plan.items()} == {0, 1}


# ------------------------------------------------------------------ long sequences
@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,lq", [(64, 6, 3), (128, 4, 1), (128, 16, 40)])
def test_long_documents(pkv, d, hq, lq):
    """131072 keys and a few more, by tiles of few rows and of 128: attention, the keys' weights, an eviction."""
    lens = [131072 + 77]
    cache = LC.Cache(73, dtype="fp4", lens=lens, hkv=1, d=d, page=64, head_major=True)
    attend(pkv, cache, hq, [lq], [min(lq, 2)])
    run_weights(pkv, cache, hq, [lq])
    scores = torch.rand(1, 1, lens[0], generator=torch.Generator().manual_seed(d)).cuda()
    run_evict(pkv, cache, scores, [8200], 4, 1000)


# ------------------------------------------------------------------ scales of any sign
@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(64, 32, 4), (128, 16, 4), (256, 8, 2)])
@pytest.mark.parametrize("k_scale", [-0.07, -2.0, 0.0])
def test_key_scales_below_zero_and_of_zero(pkv, d, hq, hkv, k_scale):
    """Both routes order the logits, not the sums of products: a tensor scale below 0, and of 0 (all keys alike)."""
    lens, lq = [700, 900, 300], [1, 700, 4]
    cache = LC.Cache(74, dtype="fp4", lens=lens, hkv=hkv, d=d, page=16)
    cache.k_scale = k_scale
    cache.scales[0].fill_(k_scale)
    plan = attend(pkv, cache, hq, lq, [0] * 3)[3]
    assert {it["kind"] for it in plan.items()} == {0, 1}
