"""Norm and rotation of queries and keys, alone and on the way into the cache.

The expected rows are computed here in 64 bits from the definition.  Tolerances
(derived, per element):

* fp32 arithmetic: the sum of squares of a lane's 8 values and the shuffle tree
  round at most 13 times (halved by the root), rsqrt is within 2 ulp, the two
  products of the norm and the two roundings of the rotation's FMA form add 5 more:
  below 16 roundings of 2^-24, i.e. 2^-20 of the pair's magnitude |a| + |b|;
  2^-19 is used.
* the result's one rounding: half a step, 2^-8 relative for bf16, 2^-4 relative
  (2^-10 absolute among the subnormals) for e4m3 codes.
"""
import numpy as np
import pytest

import oracle
import synth
from tests import harness as H

ARITH = 2.0 ** -19


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_variable_gb300 as m
    from paged_kv_variable_gb300 import build as b
    b.build()
    m.lib()
    return m


# ------------------------------------------------------------------ refusals (host)
class _Fake:
    """Pointer, shape and strides of a tensor that is never read."""

    def __init__(self, shape, dtype="bfloat16", ptr=1 << 20, strides=None):
        self.shape, self.dtype, self._ptr = tuple(shape), dtype, ptr
        if strides is None:
            strides, acc = [], 1
            for n in reversed(shape):
                strides.insert(0, acc)
                acc *= n
        self._strides = strides

    def data_ptr(self):
        return self._ptr

    def stride(self, i):
        return self._strides[i]

    def dim(self):
        return len(self.shape)


def _status(pkv, fn):
    with pytest.raises(pkv.PkvError) as e:
        fn()
    assert pkv.last_error()
    return e.value.status


def test_qk_norm_rope_refusals(pkv):
    table, pos = _Fake((100, 64), "float32"), _Fake((5,), "int32")
    q, k = _Fake((5, 4, 64)), _Fake((5, 2, 64), ptr=1 << 24)

    def call(spec=None, **over):
        kw = dict(q=q, k=k, positions=pos)
        kw.update(over)
        return _status(pkv, lambda: pkv.qk_norm_rope(pkv.make_qk_args(**kw), spec or pkv.make_rope_spec(cos_sin=table),
                                                     stream=0))

    assert call(q=_Fake((5, 4, 96)), k=None) == 2                                   # head_dim
    assert call(spec=pkv.make_rope_spec(cos_sin=_Fake((100, 12), "float32"))) == 1  # rot_dim % 8
    assert call(spec=pkv.make_rope_spec(cos_sin=_Fake((100, 128), "float32"))) == 1  # rot_dim > head_dim
    assert call(spec=pkv.make_rope_spec(cos_sin=_Fake((0, 64), "float32"))) == 1    # an empty table
    assert call(spec=pkv.make_rope_spec(cos_sin=_Fake((100, 64), "float32", ptr=(1 << 20) + 8))) == 1
    assert call(spec=pkv.make_rope_spec(cos_sin=table, q_weight=_Fake((64,)), eps=0.0)) == 1
    assert call(spec=pkv.make_rope_spec(cos_sin=table, q_weight=_Fake((64,)), eps=float("nan"))) == 1
    assert call(spec=pkv.make_rope_spec(cos_sin=table, k_weight=_Fake((64,), ptr=(1 << 20) + 2))) == 1
    assert call(positions=None) == 1
    assert call(q=_Fake((5, 4, 64), ptr=(1 << 20) + 8)) == 1                         # misaligned
    assert call(q=_Fake((5, 4, 64), strides=[4 * 68, 68, 1])) == 1                  # head stride not 16 bytes
    assert call(q_out=_Fake((5, 4, 64), strides=[512, 64, 1])) == 1                 # in place, other strides
    bad = pkv.make_rope_spec(cos_sin=table)
    bad.interleaved = 2
    assert call(spec=bad) == 1
    args = pkv.make_qk_args(q=q, positions=pos)
    args.num_heads_kv = 3                                                           # heads without a tensor
    assert _status(pkv, lambda: pkv.qk_norm_rope(args, pkv.make_rope_spec(cos_sin=table), stream=0)) == 1
    args = pkv.make_qk_args(q=q, positions=pos)
    args.num_tokens = -1
    assert _status(pkv, lambda: pkv.qk_norm_rope(args, pkv.make_rope_spec(cos_sin=table), stream=0)) == 1
    # nothing to do: no launch (empty tensors have no address)
    for ptr in (0, 1 << 20):
        args = pkv.make_qk_args(q=_Fake((0, 4, 64), ptr=ptr), k=_Fake((0, 2, 64), ptr=ptr),
                                positions=_Fake((0,), "int32", ptr=ptr))
        pkv.qk_norm_rope(args, pkv.make_rope_spec(cos_sin=table), stream=0)


def test_binding_refuses_wrong_tensors(pkv):
    with pytest.raises(ValueError):
        pkv.make_qk_args()
    with pytest.raises(ValueError):
        pkv.make_qk_args(q=_Fake((5, 4, 64), "float16"))
    with pytest.raises(ValueError):
        pkv.make_qk_args(q=_Fake((5, 4, 64), strides=[512, 1, 4]))
    with pytest.raises(ValueError):
        pkv.make_qk_args(q=_Fake((5, 4, 64)), k=_Fake((6, 4, 64)))
    with pytest.raises(ValueError):
        pkv.make_qk_args(q=_Fake((5, 4, 64)), positions=_Fake((4,), "int32"))
    with pytest.raises(ValueError):
        pkv.make_qk_args(q=_Fake((5, 4, 64)), positions=_Fake((5,), "int64"))
    with pytest.raises(ValueError):
        pkv.make_qk_args(q=_Fake((5, 4, 64)), k_out=_Fake((5, 4, 64)))
    with pytest.raises(ValueError):
        pkv.make_rope_spec(cos_sin=_Fake((10, 64), "bfloat16"))
    with pytest.raises(ValueError):
        pkv.make_rope_spec(cos_sin=_Fake((10, 64), "float32", strides=[128, 1]))
    with pytest.raises(ValueError):
        pkv.make_rope_spec(q_weight=_Fake((64,), "float32"))


def test_binding_checks_the_transform_against_the_problem(pkv):
    """Weights of another head_dim, an output too small for the queries: refused before anything is launched."""
    with pytest.raises(ValueError):
        pkv.make_rope_spec(q_weight=_Fake((64,)), k_weight=_Fake((128,)))
    short = pkv.make_rope_spec(q_weight=_Fake((32,)))
    with pytest.raises(ValueError):
        pkv.qk_norm_rope(pkv.make_qk_args(q=_Fake((5, 4, 64))), short, stream=0)
    prob, args, _, _ = _append_call(pkv)
    pl = pkv.plan(prob, [3, 1], [37, 5], [3, 1], num_sms=4)
    table = pkv.make_rope_spec(cos_sin=_Fake((64, 64), "float32"))
    for spec, q_out in ((short, _Fake((4, 4, 64))), (table, _Fake((3, 4, 64))), (table, _Fake((4, 2, 64))),
                        (table, _Fake((4, 4, 128)))):
        rope = pkv.make_rope_append_args(spec=spec, q_out=q_out)
        with pytest.raises(ValueError):
            pkv.rope_kv_append(prob, args, rope, 4, 4, stream=0)
        with pytest.raises(ValueError):
            pkv.rope_attn_varlen_kvcache_fwd(prob, args, rope, pl, None, stream=0)


def _append_call(pkv, **over):
    """Good arguments of the rotating append over fake tensors, with changes."""
    q, k = _Fake((4, 4, 64)), _Fake((4, 2, 64), ptr=1 << 22)
    cache = _Fake((8, 16, 2, 64), ptr=1 << 24)
    i32 = _Fake((3,), "int32", ptr=1 << 16)
    kw = dict(q=q, out=q, cu_seqlens_q=i32, max_seqlen_q=3, k_cache=cache, v_cache=cache, cache_seqlens=i32, k_new=k,
              v_new=k, cu_seqlens_knew=i32, block_table=_Fake((2, 4), "int32", ptr=1 << 17))
    rest = dict(spec=pkv.make_rope_spec(cos_sin=_Fake((64, 64), "float32")), q_out=q, total_q=4, total_new=4,
                causal=True)
    for name, v in over.items():
        (rest if name in rest else kw)[name] = v
    prob = pkv.make_problem(batch=2, num_heads_q=4, num_heads_kv=2, head_dim=64, page_size=16, cache_capacity=64,
                            num_pages=8, cache_dtype="bf16", causal=rest["causal"], softmax_scale=0.125)
    return prob, pkv.make_args(**kw), pkv.make_rope_append_args(spec=rest["spec"], q_out=rest["q_out"]), rest


def test_rope_kv_append_refusals(pkv):
    def call(**over):
        prob, args, rope, rest = _append_call(pkv, **over)
        return _status(pkv, lambda: pkv.rope_kv_append(prob, args, rope, rest["total_q"], rest["total_new"], stream=0))

    assert call(total_new=-1) == 1
    assert call(total_q=-1) == 1
    assert call(k_new=None, v_new=None, cu_seqlens_knew=None) == 1
    assert call(cu_seqlens_q=None) == 1
    assert call(q=_Fake((4, 4, 64), ptr=(1 << 20) + 4)) == 1
    assert call(q_out=_Fake((4, 4, 64), ptr=(1 << 21) + 4)) == 1
    assert call(q_out=_Fake((4, 4, 64), strides=[512, 64, 1])) == 1    # in place, other strides
    assert call(block_table=None) == 1
    assert call(q_rows=9) == 2                                         # placed query rows
    assert call(spec=pkv.make_rope_spec(cos_sin=_Fake((64, 20), "float32"))) == 1
    assert call(spec=pkv.make_rope_spec(cos_sin=_Fake((64, 64), "float32"), q_weight=_Fake((64,)), eps=-1.0)) == 1
    prob, args, rope, _ = _append_call(pkv)
    assert pkv.lib().pkv_rope_kv_append(prob, args, None, 4, 4, None, None) == 1
    assert pkv.lib().pkv_qk_norm_rope(None, None, None, None) == 1
    # nothing to do: no launch
    pkv.rope_kv_append(prob, args, rope, 0, 0, stream=0)


def test_rope_attention_refusals(pkv):
    def call(ws_bytes=None, plan_new=(3, 1), **over):
        prob, args, rope, _ = _append_call(pkv, **over)
        pl = pkv.plan(prob, [3, 1], [37, 5], list(plan_new) if plan_new else None, num_sms=4)
        ws = _Fake((pl.workspace_bytes if ws_bytes is None else ws_bytes,), "uint8", ptr=1 << 28)
        ws.numel, ws.element_size = (lambda: ws.shape[0]), (lambda: 1)
        return _status(pkv, lambda: pkv.rope_attn_varlen_kvcache_fwd(prob, args, rope, pl, ws, stream=0))

    assert call(q_out=None) == 1
    assert call(q_rows=9) == 2
    assert call(ws_bytes=256) == 3
    assert call(plan_new=None) == 1                                    # the plan appends nothing, k_new is given
    assert call(spec=pkv.make_rope_spec(cos_sin=_Fake((64, 128), "float32"))) == 1
    prob, args, rope, _ = _append_call(pkv)
    pl = pkv.plan(prob, [3, 1], [37, 5], [3, 1], num_sms=4)
    assert pkv.lib().pkv_rope_attn_varlen_kvcache_fwd(prob, args, None, pl.handle, 1 << 28, 1 << 20, None) == 1


# ------------------------------------------------------------------ expected rows (64 bits)
def table64(n, rot, base=10000.0, start=0):
    """fp32 table of n positions, angles taken in 64 bits."""
    ang = (start + np.arange(n, dtype=np.float64))[:, None] * base ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def rows64(x, w, pos, table, interleaved, eps):
    """x (T, H, D) -> the transformed rows and each element's pair magnitude |a| + |b|."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * np.asarray(w, np.float64)
    rot = 0 if table is None else table.shape[1]
    y, mag = x.copy(), np.abs(x)
    if rot:
        c = table[pos, :rot // 2].astype(np.float64)[:, None, :]
        s = table[pos, rot // 2:].astype(np.float64)[:, None, :]
        ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
        ib = ia + (1 if interleaved else rot // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def close_bf16(got_t, want, mag):
    got = H.bf16_to_f64(got_t)
    d = ARITH * mag
    tol = 2.0 ** -8 * (np.abs(want) + d) + d
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))


def close_codes(codes, want, mag, scale):
    """e4m3 codes (uint8) of want / scale."""
    got = oracle.e4m3_decode(codes)
    z = np.clip(want / scale, -448, 448)
    d = ARITH * mag / scale + 2.0 ** -23 * np.abs(z)
    tol = np.maximum(2.0 ** -4 * (np.abs(z) + d), 2.0 ** -10) + d
    assert np.all(np.abs(got - z) <= tol), float(np.max(np.abs(got - z) - tol))


@pytest.fixture
def gpu(pkv):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def bf16(torch, rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda().bfloat16()


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def _weights(torch, rng, which, d):
    w = {k: (1 + 0.3 * bf16(torch, rng, d)).bfloat16() for k in ("q", "k")}
    return w["q"] if "q" in which else None, w["k"] if "k" in which else None


# ------------------------------------------------------------------ norm and rotation alone
@pytest.mark.gpu
@pytest.mark.parametrize("d,rot,interleaved,norm", [
    (64, 64, False, "qk"), (64, 32, True, ""), (64, 8, False, "k"), (128, 128, False, ""), (128, 128, True, "qk"),
    (128, 64, False, "q"), (128, 72, False, "qk"), (128, 40, True, "qk"), (128, 0, False, "qk"),
    (256, 256, False, "qk"), (256, 96, True, "k"), (256, 24, False, "q")])
@pytest.mark.parametrize("tokens,hq,hkv", [(1, 32, 8), (37, 7, 1), (129, 3, 5)])
def test_qk_norm_rope(pkv, gpu, d, rot, interleaved, norm, tokens, hq, hkv):
    torch = gpu
    rng = np.random.default_rng(d + rot + tokens)
    eps, far = 1e-5, 1000
    x = bf16(torch, rng, tokens, hq + 2 * hkv, d, scale=3.0)
    q, k = x[:, :hq], x[:, hq:hq + hkv]                    # views of a packed projection
    qw, kw = _weights(torch, rng, norm, d)
    table = table64(far, rot, start=100000) if rot else None
    pos = rng.integers(0, far, tokens).astype(np.int32)
    spec = pkv.make_rope_spec(cos_sin=None if table is None else torch.from_numpy(table).cuda(),
                              interleaved=interleaved, eps=eps, q_weight=qw, k_weight=kw)
    q_out = torch.full((tokens, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((tokens + 3, hkv, 2 * d), float("nan"), dtype=torch.bfloat16, device="cuda")[:tokens, :, :d]
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    positions = H.i32(pos)
    keep = [spec, table]
    table_t = None if table is None else torch.from_numpy(table).cuda()
    if table_t is not None:
        spec.cos_sin = table_t.data_ptr()
    before = x.clone()
    pkv.qk_norm_rope(pkv.make_qk_args(q=q, k=k, positions=positions, q_out=q_out, k_out=k_out), spec,
                     device_status=status)
    assert int(status[0]) == 0 and keep
    for got, src, w in ((q_out, q, qw), (k_out, k, kw)):
        want, mag = rows64(np64(src), np64(w), pos, table, interleaved, eps)
        close_bf16(got, want, mag)
    assert torch.equal(x, before)
    # in place: the same bits, and the values of the packed row untouched
    want_q, want_k = q_out.clone(), k_out.clone()
    pkv.qk_norm_rope(pkv.make_qk_args(q=q, k=k, positions=positions), spec)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(x[:, hq + hkv:], before[:, hq + hkv:])


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [401, 701])       # two, four heads a lane
@pytest.mark.parametrize("d,hq,hkv,interleaved", [(64, 66, 22, False), (128, 33, 11, True), (256, 15, 5, False)])
def test_many_rows(pkv, gpu, tokens, d, hq, hkv, interleaved):
    """The splits of heads that larger calls take, at head counts that do not fill them; alone and into the cache."""
    torch = gpu
    c = AppendCase(pkv, torch, tokens + d, d=d, page=16, fp8=d == 128, new=[tokens - 150, 0, 150], cached=[0, 3, 37],
                   hq=hq, hkv=hkv, rot=d // 2, interleaved=interleaved, norm="qk")
    k0, v0 = H.to_numpy_bits(c.kc).copy(), H.to_numpy_bits(c.vc).copy()
    c.run()
    assert int(c.status[0]) == 0
    c.check(k0, v0)
    pq, _, _ = c.positions()
    q, k, positions = torch.empty_like(c.q_out), torch.empty(c.k.shape, dtype=c.k.dtype, device="cuda"), H.i32(pq)
    pkv.qk_norm_rope(pkv.make_qk_args(q=c.q, k=c.k, positions=positions, q_out=q, k_out=k), c.spec)
    assert torch.equal(q, c.q_out)
    close_bf16(k, *rows64(np64(c.k), np64(c.kw), pq, c.table, interleaved, c.eps))


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv,tokens", [(64, 39, 5, 35011), (128, 21, 3, 31013), (256, 11, 1, 34001)])
def test_a_large_call_equals_its_pieces(pkv, gpu, d, hq, hkv, tokens):
    """The widest split of heads (eight a lane) gives the bits of the others, which smaller calls take."""
    torch = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    x = torch.randn(tokens, hq + hkv, d, device="cuda", generator=g, dtype=torch.bfloat16)
    pos = torch.randint(0, 500, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    table = torch.from_numpy(table64(500, d)).cuda()
    w = (1 + 0.3 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    spec = pkv.make_rope_spec(cos_sin=table, q_weight=w, k_weight=w)
    outs = [torch.zeros_like(x) for _ in range(2)]

    def call(out, a, b):
        pkv.qk_norm_rope(pkv.make_qk_args(q=x[a:b, :hq], k=x[a:b, hq:], positions=pos[a:b], q_out=out[a:b, :hq],
                                          k_out=out[a:b, hq:]), spec)

    call(outs[0], 0, tokens)
    for a in range(0, tokens, 5000):
        call(outs[1], a, min(tokens, a + 5000))
    assert torch.equal(*outs)
    n = 64
    want, mag = rows64(np64(x[-n:]), np64(w), pos[-n:].cpu().numpy(), table.cpu().numpy(), False, 1e-6)
    close_bf16(outs[0][-n:], want, mag)


@pytest.mark.gpu
def test_qk_norm_rope_one_side_and_strides(pkv, gpu):
    """q alone, k alone, heads outermost, another stream."""
    torch = gpu
    rng = np.random.default_rng(5)
    tokens, h, d = 50, 6, 128
    table = table64(64, d)
    table_t = torch.from_numpy(table).cuda()
    pos = rng.integers(0, 64, tokens).astype(np.int32)
    positions = H.i32(pos)
    src = bf16(torch, rng, h, tokens, d).transpose(0, 1)          # (tokens, h, d), head stride > token stride
    spec = pkv.make_rope_spec(cos_sin=table_t)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for side in ("q", "k"):
        dst = torch.empty(tokens, h, d, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        pkv.qk_norm_rope(pkv.make_qk_args(**{side: src, side + "_out": dst}, positions=positions), spec, stream=stream)
        stream.synchronize()
        close_bf16(dst, *rows64(np64(src), None, pos, table, False, 1.0))


@pytest.mark.gpu
def test_qk_norm_rope_bad_positions_and_values(pkv, gpu):
    """A bad position skips its token alone and is reported; NaN and infinity stay in their head."""
    torch = gpu
    rng = np.random.default_rng(6)
    tokens, h, d, far = 9, 5, 64, 16
    table = table64(far, d)
    table_t = torch.from_numpy(table).cuda()
    pos = rng.integers(0, far, tokens).astype(np.int32)
    pos[2], pos[7] = far, -1
    x = bf16(torch, rng, tokens, h, d)
    x[4, 1, 3], x[4, 2, 5], x[5, 0] = float("nan"), float("inf"), 0.0
    w = _weights(torch, rng, "q", d)[0]
    out = torch.full_like(x, 7.0)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    positions = H.i32(pos)
    pkv.qk_norm_rope(pkv.make_qk_args(q=x, positions=positions, q_out=out),
                     pkv.make_rope_spec(cos_sin=table_t, q_weight=w), device_status=status)
    assert int(status[0]) == 6 and int(status[1]) in (2, 7) and int(status[2]) in (far, -1)
    good = np.ones((tokens, h), bool)
    good[[2, 7]] = False
    assert torch.all(out[[2, 7]] == 7.0)
    assert torch.isnan(out[4, 1]).any()
    good[4, 1] = good[4, 2] = False
    want, mag = rows64(np.where(good[..., None], np64(x), 0.0), np64(w), np.clip(pos, 0, far - 1), table, False, 1e-6)
    got = out.clone()
    got[torch.from_numpy(~good).cuda()] = 0.0
    close_bf16(got, want, mag)
    assert torch.all(out[5, 0] == 0.0)


# ------------------------------------------------------------------ rotation on the way into the cache
class AppendCase:
    def __init__(self, pkv, torch, seed, *, d, page, fp8, new, cached, q_lens=None, hq=6, hkv=2, rot=None,
                 interleaved=False, norm="", ragged=False, far=None, spare_pages=3):
        rng = np.random.default_rng(seed)
        self.pkv, self.torch, self.d, self.page, self.fp8, self.interleaved = pkv, torch, d, page, fp8, interleaved
        self.new, self.cached = np.asarray(new, np.int32), np.asarray(cached, np.int32)
        self.q_lens = self.new if q_lens is None else np.asarray(q_lens, np.int32)
        B = len(new)
        self.tq, self.tn = int(self.q_lens.sum()), int(self.new.sum())
        cap = int(max(1, (self.new + self.cached).max()))
        self.eps = 1e-6
        rot = d if rot is None else rot
        self.table = table64(far or cap + 1, rot) if rot else None
        self.qw, self.kw = _weights(torch, rng, norm, d)
        x = bf16(torch, rng, max(self.tq, self.tn, 1), hq + 2 * hkv, d)
        self.q, self.k, self.v = x[:self.tq, :hq], x[:self.tn, hq:hq + hkv], x[:self.tn, hq + hkv:]
        if page:
            width = -(-cap // page)
            cap, n_pages = width * page, B * width + spare_pages
            self.pages = rng.permutation(n_pages)[:B * width].reshape(B, width).astype(np.int32)
            shape = (n_pages, page, hkv, d)
        else:
            self.pages, n_pages, shape = None, B + 1, (B + 1, cap, hkv, d)
        if fp8:
            self.kc, self.vc = (torch.from_numpy(rng.integers(0, 127, shape).astype(np.uint8)).cuda() for _ in "kv")
        else:
            self.kc, self.vc = bf16(torch, rng, *shape), bf16(torch, rng, *shape)
        self.ks, self.vs = (torch.tensor([s], dtype=torch.float32, device="cuda") for s in (0.011, 0.017))
        self.problem = pkv.make_problem(batch=B, num_heads_q=hq, num_heads_kv=hkv, head_dim=d, page_size=page,
                                        cache_capacity=cap, num_pages=n_pages, cache_dtype="fp8" if fp8 else "bf16",
                                        causal=True, softmax_scale=d ** -0.5)
        self.q_out = torch.full((self.tq, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.table_t = None if self.table is None else torch.from_numpy(self.table).cuda()
        self.spec = pkv.make_rope_spec(cos_sin=self.table_t, interleaved=interleaved, eps=self.eps, q_weight=self.qw,
                                       k_weight=self.kw)
        self.rope = pkv.make_rope_append_args(spec=self.spec, q_out=self.q_out)
        self.cu_n = H.i32(np.concatenate([[0], np.cumsum(self.new)]))
        self.cu_q = H.i32(np.concatenate([[0], np.cumsum(self.q_lens)]))
        self.lens = H.i32(self.cached)
        self.bt = None if self.pages is None else H.i32(self.pages)
        self.extra = dict(block_table=self.bt)
        if ragged:
            counts = np.array([-(-int(n + c) // page) for n, c in zip(self.new, self.cached)])
            self.flat = H.i32(np.concatenate([self.pages[b, :n] for b, n in enumerate(counts)]))
            self.indptr = H.i32(np.concatenate([[0], np.cumsum(counts)]))
            self.extra = dict(block_table=self.flat, page_indptr=self.indptr)
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")

    def args(self, **over):
        kw = dict(q=self.q, out=None, cu_seqlens_q=self.cu_q, max_seqlen_q=int(self.q_lens.max()), k_cache=self.kc,
                  v_cache=self.vc, cache_seqlens=self.lens, k_new=self.k if self.tn else None,
                  v_new=self.v if self.tn else None, cu_seqlens_knew=self.cu_n, k_scale=self.ks if self.fp8 else None,
                  v_scale=self.vs if self.fp8 else None, **self.extra)
        kw.update(over)
        return self.pkv.make_args(**kw)

    def run(self, stream=None):
        self.pkv.rope_kv_append(self.problem, self.args(), self.rope, self.tq, self.tn, device_status=self.status,
                                stream=stream)

    def positions(self):
        """Of each query and each new token, and the cache slot of each new token."""
        pq = np.concatenate([c + n - lq + np.arange(lq) for lq, n, c in zip(self.q_lens, self.new, self.cached)])
        pk = np.concatenate([c + np.arange(n) for n, c in zip(self.new, self.cached)])
        seq = np.repeat(np.arange(len(self.new)), self.new)
        at = (self.pages[seq, pk // self.page], pk % self.page) if self.page else (seq, pk)
        return pq.astype(np.int64), pk.astype(np.int64), at

    def check(self, k0, v0):
        """Against the 64-bit rows; k0, v0: the caches (numpy) before the call."""
        pq, pk, at = self.positions()
        if self.tq:
            close_bf16(self.q_out, *rows64(np64(self.q), np64(self.qw), pq, self.table, self.interleaved, self.eps))
        kc, vc = H.to_numpy_bits(self.kc), H.to_numpy_bits(self.vc)
        if self.tn:
            want, mag = rows64(np64(self.k), np64(self.kw), pk, self.table, self.interleaved, self.eps)
            if self.fp8:
                close_codes(kc[at], want, mag, float(self.ks))
                v_want = oracle.fp8_quantize(H.to_numpy_bits(self.v.contiguous()), float(self.vs))
            else:
                rows = self.torch.from_numpy(kc[at].view(np.int16)).view(self.torch.bfloat16)
                close_bf16(rows, want, mag)
                v_want = H.to_numpy_bits(self.v.contiguous())
            assert np.array_equal(vc[at], v_want)          # values as the plain append writes them
            kc[at], vc[at] = k0[at], v0[at]
        assert np.array_equal(kc, k0) and np.array_equal(vc, v0)   # nothing else is written


APPENDS = [
    dict(d=128, page=16, fp8=False, new=[1] * 7, cached=[0, 5, 15, 16, 17, 200, 31]),
    dict(d=128, page=16, fp8=True, new=[1] * 7, cached=[0, 5, 15, 16, 17, 200, 31], norm="qk"),
    dict(d=64, page=0, fp8=False, new=[3, 0, 40, 1], cached=[0, 9, 17, 100], norm="k", interleaved=True),
    dict(d=64, page=24, fp8=True, new=[3, 0, 40, 1], cached=[0, 9, 17, 100], rot=32),
    dict(d=256, page=1, fp8=False, new=[2, 30], cached=[7, 0], rot=64, norm="qk"),
    dict(d=256, page=64, fp8=True, new=[70, 1, 64], cached=[0, 63, 64], interleaved=True, norm="q"),
    dict(d=128, page=4, fp8=True, new=[0, 0, 5, 0], cached=[1, 2, 3, 0], rot=0, norm="k"),
    # fewer or more queries than new tokens, none, and queries without new tokens
    dict(d=128, page=16, fp8=False, new=[4, 4, 0, 9], cached=[10, 20, 30, 0], q_lens=[1, 6, 5, 0]),
    dict(d=128, page=16, fp8=False, new=[0, 0], cached=[10, 20], q_lens=[3, 20], norm="q"),
    dict(d=64, page=8, fp8=False, new=[5, 6], cached=[10, 20], q_lens=[0, 0], hq=4, hkv=4),
    dict(d=128, page=16, fp8=False, new=[17, 3], cached=[30, 0], ragged=True),
    dict(d=64, page=2, fp8=True, new=[17, 3], cached=[30, 0], ragged=True, hq=15, hkv=3),
]


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_rope_kv_append(pkv, gpu, i):
    c = AppendCase(pkv, gpu, i, **APPENDS[i])
    k0, v0 = H.to_numpy_bits(c.kc).copy(), H.to_numpy_bits(c.vc).copy()
    c.run()
    assert int(c.status[0]) == 0
    c.check(k0, v0)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [31, 32, 33, 65, 1025, 2100])
def test_rope_kv_append_many_sequences(pkv, gpu, batch):
    """The sequence of a token is found among few and many, some of them without tokens."""
    rng = np.random.default_rng(batch)
    new = rng.integers(0, 3, batch)
    new[-1] = 1
    c = AppendCase(pkv, gpu, batch, d=64, page=8, fp8=False, new=new, cached=rng.integers(0, 20, batch), hq=1, hkv=1)
    k0, v0 = H.to_numpy_bits(c.kc).copy(), H.to_numpy_bits(c.vc).copy()
    c.run()
    assert int(c.status[0]) == 0
    c.check(k0, v0)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rope_kv_append_equals_the_steps_apart(pkv, gpu, d):
    """bf16: bit for bit what the transform followed by the plain append writes."""
    torch = gpu
    c = AppendCase(pkv, torch, d, d=d, page=16, fp8=False, new=[5, 1, 30], cached=[11, 0, 40], norm="qk", rot=d // 2)
    kc, vc = c.kc.clone(), c.vc.clone()
    c.run()
    pq, pk, _ = c.positions()
    q, k = torch.empty_like(c.q_out), torch.empty_like(c.k, memory_format=torch.contiguous_format)
    positions = H.i32(pq)
    pkv.qk_norm_rope(pkv.make_qk_args(q=c.q, k=c.k, positions=positions, q_out=q, k_out=k), c.spec)
    v = c.v.contiguous()
    pkv.kv_append(c.problem, c.args(k_cache=kc, v_cache=vc, k_new=k, v_new=v), c.tn)
    assert torch.equal(q, c.q_out) and torch.equal(kc, c.kc) and torch.equal(vc, c.vc)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [3, 900])
def test_calls_between_kernels_that_write_and_read(pkv, gpu, tokens):
    """A call may start while the kernel before it drains: it reads what that kernel wrote (queries, keys, lengths),
    and what follows reads its results, from the host and in a graph."""
    torch = gpu
    c = AppendCase(pkv, torch, 30, d=128, page=16, fp8=False, new=[tokens, 1, tokens], cached=[3, 40, 9], norm="qk",
                   far=tokens + 64)
    inputs = [(bf16(torch, np.random.default_rng(i), *c.q.shape), H.i32(c.cached - i)) for i in range(3)]
    pos = H.i32(c.positions()[0])
    qk = pkv.make_qk_args(q=c.q_out, positions=pos)
    args, total = c.args(), torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    busy = torch.randn(1 << 24, device="cuda")

    def step(i, got):
        busy.mul_(1.0001)
        c.q.copy_(inputs[i % 3][0])
        c.lens.copy_(inputs[i % 3][1])
        pkv.rope_kv_append(c.problem, args, c.rope, c.tq, c.tn)
        pkv.qk_norm_rope(qk, c.spec)               # once more over its own queries, in place
        got.copy_(c.q_out)

    want = []
    for i in range(3):
        step(i, total)
        torch.cuda.synchronize()
        want.append((total.clone(), c.kc.clone()))
    got = [torch.empty_like(total) for _ in range(12)]
    for i, g in enumerate(got):
        step(i, g)
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3][0]) for i, g in enumerate(got))
    for g in got:
        g.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, g in enumerate(got):
            step(i, g)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3][0]) for i, g in enumerate(got))


@pytest.mark.gpu
def test_rope_kv_append_in_place_and_twice(pkv, gpu):
    """Queries rotated in place; two calls of one batch write the same."""
    torch = gpu
    c = AppendCase(pkv, torch, 3, d=128, page=16, fp8=False, new=[5, 1, 30], cached=[11, 0, 40])
    c.run()
    k1, q1 = c.kc.clone(), c.q_out.clone()
    c.run()
    assert torch.equal(k1, c.kc) and torch.equal(q1, c.q_out)
    pkv.rope_kv_append(c.problem, c.args(), pkv.make_rope_append_args(spec=c.spec, q_out=c.q), c.tq, c.tn)
    assert torch.equal(c.q, q1) and torch.equal(k1, c.kc)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["page", "capacity", "table", "negative"])
def test_rope_kv_append_reports_bad_rows(pkv, gpu, what):
    """A row out of range is skipped, key and value, and reported; the rest is written."""
    torch = gpu
    c = AppendCase(pkv, torch, 8, d=64, page=8, fp8=False, new=[2, 3], cached=[6, 10],
                   far=12 if what == "table" else None)
    k0, v0 = H.to_numpy_bits(c.kc).copy(), H.to_numpy_bits(c.vc).copy()
    bad = np.zeros(5, bool)
    if what == "page":                       # sequence 1, positions 10..12: entry 1
        table = c.pages.copy()
        table[1, 1] = 1000
        c.extra = dict(block_table=H.i32(table))
        bad[2:] = True
    elif what == "capacity":
        c.lens = H.i32([6, 1 << 30])
        bad[2:] = True
    elif what == "negative":
        c.lens = H.i32([-1, 10])
        bad[0] = True
        c.cached = np.array([-1, 10], np.int32)
    else:
        bad[4] = True                        # position 12 of a table of 12
    c.run()
    assert int(c.status[0]) == 6
    pq, pk, at = c.positions()
    kc, vc = H.to_numpy_bits(c.kc), H.to_numpy_bits(c.vc)
    fine = tuple(x[~bad] for x in at)
    assert np.array_equal(vc[fine], H.to_numpy_bits(c.v.contiguous())[~bad])
    want, mag = rows64(np64(c.k), None, np.clip(pk, 0, len(c.table) - 1), c.table, False, c.eps)
    close_bf16(torch.from_numpy(kc[fine].view(np.int16)).view(torch.bfloat16), want[~bad], mag[~bad])
    kc[fine], vc[fine] = k0[fine], v0[fine]
    assert np.array_equal(kc, k0) and np.array_equal(vc, v0)


@pytest.mark.gpu
def test_rope_kv_append_far_into_a_large_cache(pkv, gpu):
    """Element offsets past 32 bits."""
    torch = gpu
    d, page, hkv = 128, 16, 1
    pages = (1 << 32) // (page * hkv * d) + 8
    kc = torch.empty(pages, page, hkv, d, dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    c = AppendCase(pkv, torch, 4, d=d, page=page, fp8=True, new=[3, 2], cached=[14, 0], hq=2, hkv=hkv)
    table = np.array([[pages - 1, pages - 2], [pages - 5, 0]], np.int32)
    c.kc, c.vc, c.pages = kc, vc, table
    c.extra = dict(block_table=H.i32(table))
    c.problem.num_pages = pages
    c.run()
    assert int(c.status[0]) == 0
    _, pk, at = c.positions()
    got_k = np.stack([kc[int(p), int(s)].cpu().numpy() for p, s in zip(*at)])
    got_v = np.stack([vc[int(p), int(s)].cpu().numpy() for p, s in zip(*at)])
    close_codes(got_k, *rows64(np64(c.k), None, pk, c.table, False, c.eps), float(c.ks))
    assert np.array_equal(got_v, oracle.fp8_quantize(H.to_numpy_bits(c.v.contiguous()), float(c.vs)))


# ------------------------------------------------------------------ rotation, append and attention in one call
def _attention64(c, q, kc, vc, lens):
    """Causal attention of bf16 queries q over the caches as they stand, in 64 bits."""
    out, lse, r0 = [], [], 0
    kd, vd = ((oracle.e4m3_decode(H.to_numpy_bits(x)) * float(s) if c.fp8 else np64(x))
              for x, s in ((kc, c.ks), (vc, c.vs)))
    for b, (lq, lk) in enumerate(zip(c.q_lens, lens)):
        pos = np.arange(lk)
        at = (c.pages[b, pos // c.page], pos % c.page) if c.page else (np.full(lk, b), pos)
        o, z = oracle.attend(np64(q[r0:r0 + lq]), kd[at], vd[at], True, c.d ** -0.5)
        out.append(o)
        lse.append(z)
        r0 += lq
    return np.concatenate(out), np.concatenate(lse, axis=1)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(d=128, page=16, fp8=False, new=[1] * 6, cached=[900, 5, 15, 2000, 17, 200], hq=8, hkv=2),
    dict(d=128, page=16, fp8=True, new=[1] * 6, cached=[900, 5, 15, 2000, 17, 200], hq=8, hkv=2, norm="qk"),
    dict(d=64, page=0, fp8=False, new=[200, 1, 33], cached=[100, 700, 0], hq=8, hkv=2, norm="qk", interleaved=True),
    dict(d=256, page=16, fp8=False, new=[2, 90], cached=[300, 0], hq=4, hkv=1, rot=128),
    dict(d=128, page=8, fp8=False, new=[0, 0], cached=[300, 77], q_lens=[2, 1], hq=8, hkv=8),
])
def test_rope_attention_call(pkv, gpu, kw):
    """Rotating append + attention, against 64 bits and against the two calls apart."""
    torch = gpu
    c = AppendCase(pkv, torch, 21, **kw)
    out, lse = torch.empty_like(c.q_out), torch.empty(kw["hq"], c.tq, dtype=torch.float32, device="cuda")
    k0, v0 = c.kc.clone(), c.vc.clone()
    plan = pkv.plan(c.problem, c.q_lens, c.cached, c.new if c.tn else None)
    ws = pkv.workspace_tensor(plan.workspace_bytes)
    plan.upload(ws)
    pkv.rope_attn_varlen_kvcache_fwd(c.problem, c.args(out=out, lse=lse), c.rope, plan, ws)
    assert pkv.get_status(ws) == 0
    q1, k1, v1 = c.q_out.clone(), c.kc.clone(), c.vc.clone()
    c.check(H.to_numpy_bits(k0).copy(), H.to_numpy_bits(v0).copy())
    want, want_lse = _attention64(c, c.q_out, c.kc, c.vc, c.cached + c.new)
    H.compare_out(out, want, H.FP8_TOL if c.fp8 else H.BF16_TOL)
    H.compare_lse(lse, want_lse)
    # apart: the rotating append, then attention over what it wrote
    c.kc.copy_(k0)
    c.vc.copy_(v0)
    c.run()
    assert torch.equal(q1, c.q_out) and torch.equal(k1, c.kc) and torch.equal(v1, c.vc)
    lens = c.cached + c.new
    plan2 = pkv.plan(c.problem, c.q_lens, lens, None)
    ws2 = pkv.workspace_tensor(plan2.workspace_bytes)
    plan2.upload(ws2)
    out2, lens_t = torch.empty_like(out), H.i32(lens)
    pkv.attn_varlen_kvcache_fwd(c.problem, c.args(q=c.q_out, out=out2, cache_seqlens=lens_t, k_new=None, v_new=None,
                                                  cu_seqlens_knew=None), plan2, ws2)
    assert pkv.get_status(ws2) == 0
    assert torch.equal(out, out2)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_rope_attention_decode_loop_in_a_graph(pkv, gpu, fp8):
    """One captured call serves decode steps whose lengths grow on the device."""
    torch = gpu
    base, steps = np.array([70, 900, 0, 333], np.int32), 4
    c = AppendCase(pkv, torch, 9, d=128, page=16, fp8=fp8, new=[1] * 4, cached=base + steps, hq=8, hkv=2, norm="qk")
    rng = np.random.default_rng(10)
    plan = pkv.plan_decode_dynamic(c.problem, c.q_lens, base + steps, c.new)
    ws = pkv.workspace_tensor(plan.workspace_bytes)
    plan.upload(ws)
    out = torch.empty_like(c.q_out)
    args = c.args(out=out)
    c.lens.copy_(H.i32(base))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    pkv.rope_attn_varlen_kvcache_fwd(c.problem, args, c.rope, plan, ws, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pkv.rope_attn_varlen_kvcache_fwd(c.problem, args, c.rope, plan, ws, stream=stream)
    for s in range(steps):
        for t in (c.q, c.k, c.v):
            t.copy_(bf16(torch, rng, *t.shape))
        c.lens.copy_(H.i32(base + s))
        out.fill_(float("nan"))
        c.cached = base + s
        k0, v0 = H.to_numpy_bits(c.kc).copy(), H.to_numpy_bits(c.vc).copy()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert pkv.get_status(ws) == 0
        c.check(k0, v0)
        want, _ = _attention64(c, c.q_out, c.kc, c.vc, c.cached + 1)
        H.compare_out(out, want, H.FP8_TOL if fp8 else H.BF16_TOL)
