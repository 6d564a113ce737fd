"""The serving operators around the paged KV cache, as measured calls.

Three operators of one decode or prefill step of a transformer layer, in the
order in which a model runs them:

* ``qk_norm_rope``   per-head RMS norm of queries and keys and the position
  rotation in the same pass, out of a packed qkv projection;
* ``rope_kv_append`` the same transform on the way into the (paged or
  contiguous, bf16 or fp8) cache: rotated queries out, rotated keys and plain
  values appended;
* ``shared_prefix``  attention of a batch whose sequences share a long prefix
  of cache pages, which is computed once for all of them.

``run`` computes the plain form in elementary fp32 torch operations, or (``own``)
makes the library's calls.  Lengths come from the case alone, values from the
seed.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
PAGE = 16


# ------------------------------------------------------------------ cases
def listed():
    c = []
    # --- per-head norm and rotation
    # one sequence decoding one token: launch latency
    c.append(dict(name="norm-rope 1 token", op="qk_norm_rope", tokens=1, hq=32, hkv=8, d=128, rot=128, pairs=False,
                  norm=True, far=131072))
    # a prefill batch of an odd token count, rotation over half of each head in
    # neighbouring pairs, no norm
    c.append(dict(name="norm-rope 4093 tokens pairs", op="qk_norm_rope", tokens=4093, hq=32, hkv=8, d=128, rot=64,
                  pairs=True, norm=False, far=8192))
    # 64 prompts of 2048 tokens
    c.append(dict(name="norm-rope 131072 tokens", op="qk_norm_rope", tokens=131072, hq=32, hkv=8, d=128, rot=128,
                  pairs=False, norm=True, far=131072))
    # --- rotation and append
    # a decode batch over a bf16 paged cache: one token a sequence
    c.append(dict(name="rope-append decode 64", op="rope_kv_append", batch=64, new=1, ragged=False, cached=255, hq=32,
                  hkv=8, d=128, rot=128, pairs=False, norm=False, page=PAGE, fp8=False, lens=1))
    # the same over an e4m3 cache, with the per-head norm
    c.append(dict(name="rope-append decode 64 fp8", op="rope_kv_append", batch=64, new=1, ragged=False, cached=255,
                  hq=32, hkv=8, d=128, rot=128, pairs=False, norm=True, page=PAGE, fp8=True, lens=2))
    # ragged prompts on a cached prefix, contiguous cache
    c.append(dict(name="rope-append prefill ragged", op="rope_kv_append", batch=8, new=512, ragged=True, cached=1536,
                  hq=32, hkv=8, d=128, rot=128, pairs=False, norm=True, page=0, fp8=False, lens=3))
    # 64 prompts of 2048 tokens into an empty e4m3 cache
    c.append(dict(name="rope-append prefill fp8", op="rope_kv_append", batch=64, new=2048, ragged=False, cached=0,
                  hq=32, hkv=8, d=128, rot=128, pairs=False, norm=False, page=PAGE, fp8=True, lens=4))
    # --- attention over a shared prefix
    # four samples of one short prompt: latency
    c.append(dict(name="shared-prefix 4 x 512", op="shared_prefix", groups=1, seqs=4, prefix=512, own_max=64, lq=1,
                  hq=32, hkv=8, d=128, page=PAGE, fp8=False, lens=5))
    # a decode batch under one system prompt
    c.append(dict(name="shared-prefix 64 x 2048", op="shared_prefix", groups=1, seqs=64, prefix=2048, own_max=1024,
                  lq=1, hq=32, hkv=8, d=128, page=PAGE, fp8=False, lens=6))
    # four prompts of different lengths, 16 samples each, four drafted tokens
    # a sequence (causal among them), head dim 64, six heads a group
    c.append(dict(name="shared-prefix 4 groups drafts", op="shared_prefix", groups=4, seqs=16, prefix=6000,
                  own_max=700, lq=4, hq=12, hkv=2, d=64, page=PAGE, fp8=False, lens=7))
    # e4m3 cache
    c.append(dict(name="shared-prefix 64 x 8192 fp8", op="shared_prefix", groups=1, seqs=64, prefix=8192, own_max=1024,
                  lq=1, hq=32, hkv=8, d=128, page=PAGE, fp8=True, lens=8))
    # a long document under 64 questions
    c.append(dict(name="shared-prefix 64 x 32768", op="shared_prefix", groups=1, seqs=64, prefix=32768, own_max=4096,
                  lq=1, hq=32, hkv=8, d=128, page=PAGE, fp8=False, lens=9))
    return c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "rope_kv_append", "shared_prefix"])
    d = rng.choice([64, 128, 256])
    hq, hkv = rng.choice([(32, 8) if d > 64 else (32, 4), (16, 2), (6, 6), (14, 2), (20, 1)])
    if op == "shared_prefix":
        # (no more queries x keys, nor own keys, than the largest listed case)
        while True:
            groups, seqs = _log(rng, 1, 8), _log(rng, 1, 64)
            lq, prefix, own_max = rng.choice([1, 1, 2, 5]), _log(rng, 64, 32768), _log(rng, 5, 4096)
            pairs = groups * seqs * lq * hq * d * prefix
            keys = groups * seqs * hkv * d * own_max
            if pairs <= 64 * 32 * 128 * 32768 and keys <= 64 * 8 * 128 * 4096 and groups * prefix <= 65536:
                break
        return dict(op=op, groups=groups, seqs=seqs, prefix=prefix, own_max=own_max, lq=lq, hq=hq, hkv=hkv, d=d,
                    page=rng.choice([8, 16, 16, 64, 256]), fp8=rng.random() < 0.4, lens=rng.randrange(1 << 20))
    rot = rng.choice([d, d, d // 2])
    pairs, norm = rng.random() < 0.3, rng.random() < 0.5
    if op == "qk_norm_rope":
        most = 131072 * 40 * 128 // ((hq + hkv) * d)
        return dict(op=op, tokens=_log(rng, 1, min(131072, most)), hq=hq, hkv=hkv, d=d, rot=rot, pairs=pairs,
                    norm=norm, far=_log(rng, 512, 131072))
    while True:
        batch, new, cached = _log(rng, 1, 256), _log(rng, 1, 2048), _log(rng, 1, 2048)
        if (batch * new * (hq + 2 * hkv) * d <= 131072 * 48 * 128
                and batch * (new + cached) * hkv * d <= 64 * 2064 * 8 * 128):
            break
    return dict(op=op, batch=batch, new=new, ragged=rng.random() < 0.6, cached=cached, hq=hq, hkv=hkv, d=d, rot=rot,
                pairs=pairs, norm=norm, page=rng.choice([0, 1, 8, 16, 16, 64]), fp8=rng.random() < 0.4,
                lens=rng.randrange(1 << 20))


# ------------------------------------------------------------------ lengths (of the case alone)
def _append_lens(c):
    r = random.Random(c["lens"])
    new = [r.randint(1, c["new"]) if c["ragged"] else c["new"] for _ in range(c["batch"])]
    cached = [r.randint(0, c["cached"]) for _ in range(c["batch"])]
    return cached, new


def _prefix_lens(c):
    """Prefix length of each group (whole pages, as a prefix cache shares them)
    and keys of each sequence past its prefix."""
    r = random.Random(c["lens"])
    groups, page = c["groups"], c["page"]
    prefix = [max(page, r.randint(c["prefix"] // 2, c["prefix"]) // page * page) for _ in range(groups - 1)]
    prefix.append(max(page, c["prefix"] // page * page))
    mine = [r.randint(max(c["lq"], c["own_max"] // 8), c["own_max"]) for _ in range(groups * c["seqs"])]
    return prefix, mine


# ------------------------------------------------------------------ inputs
def _table(far, rot, device):
    """Rotation angles in 64 bits, cosines then sines in 32."""
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(far, dtype=torch.float64, device=device)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()


def _weights(c, g):
    if not c["norm"]:
        return None, None
    return tuple((1 + 0.2 * torch.randn(c["d"], device="cuda", generator=g)).bfloat16() for _ in range(2))


def _qkv(c, tokens, g):
    """Views of a packed qkv projection's output, as a model has them."""
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    x = torch.randn(tokens, hq + 2 * hkv, d, device="cuda", generator=g, dtype=torch.bfloat16)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(shape, fp8, g):
    """A cache and (fp8) the scale of its codes."""
    x = torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16)
    if not fp8:
        return x
    return (x.float() / 0.01).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"c": c}
    if c["op"] == "qk_norm_rope":
        s["q"], s["k"], _ = _qkv(c, c["tokens"], g)
        s["pos"] = torch.randint(0, c["far"], (c["tokens"],), device="cuda", generator=g, dtype=torch.int32)
        s["table"] = _table(c["far"], c["rot"], "cuda")
        s["qw"], s["kw"] = _weights(c, g)
        if own:
            # output buffers and the call's argument structs, as a serving program keeps them
            import paged_kv_variable_gb300 as pkv
            s["pkv"] = pkv
            s["q_out"], s["k_out"] = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (s["q"], s["k"]))
            s["spec"] = pkv.make_rope_spec(cos_sin=s["table"], interleaved=c["pairs"], q_weight=s["qw"],
                                           k_weight=s["kw"], eps=EPS)
            s["args"] = pkv.make_qk_args(q=s["q"], k=s["k"], positions=s["pos"], q_out=s["q_out"], k_out=s["k_out"])
        return s

    fp8, page, hkv, d = c["fp8"], c["page"], c["hkv"], c["d"]
    s["scale"] = torch.tensor([0.01], dtype=torch.float32, device="cuda")
    if c["op"] == "rope_kv_append":
        cached, new = _append_lens(c)
        batch, cap = c["batch"], max(a + b for a, b in zip(cached, new))
        s["cu"] = _i32([0] + list(np.cumsum(new)))
        s["cached"] = _i32(cached)
        s["q"], s["k"], s["v"] = _qkv(c, sum(new), g)
        s["table"] = _table(cap, c["rot"], "cuda")
        s["qw"], s["kw"] = _weights(c, g)
        s["pages"] = None
        if page:
            width = -(-cap // page)
            s["pages"] = torch.randperm(batch * width, device="cuda", generator=g).int().view(batch, width)
            shape, cap = (batch * width, page, hkv, d), width * page
        else:
            shape = (batch, cap, hkv, d)
        s["kc"], s["vc"] = _pool(shape, fp8, g), _pool(shape, fp8, g)
        if own:
            import paged_kv_variable_gb300 as pkv
            s["pkv"], s["total"] = pkv, sum(new)
            s["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
            s["problem"] = pkv.make_problem(batch=batch, num_heads_q=c["hq"], num_heads_kv=hkv, head_dim=d,
                                            page_size=page, cache_capacity=cap, num_pages=shape[0],
                                            cache_dtype="fp8" if fp8 else "bf16", causal=True,
                                            softmax_scale=d ** -0.5)
            s["rope"] = pkv.make_rope_append_args(
                spec=pkv.make_rope_spec(cos_sin=s["table"], interleaved=c["pairs"], q_weight=s["qw"],
                                        k_weight=s["kw"], eps=EPS), q_out=s["q_out"])
            s["args"] = pkv.make_args(q=s["q"], out=None, cu_seqlens_q=s["cu"], max_seqlen_q=max(new),
                                      k_cache=s["kc"], v_cache=s["vc"], cache_seqlens=s["cached"], k_new=s["k"],
                                      v_new=s["v"], cu_seqlens_knew=s["cu"], block_table=s["pages"],
                                      k_scale=s["scale"] if fp8 else None, v_scale=s["scale"] if fp8 else None)
        return s

    # shared prefix: the pages of a group's prefix stand in every one of its
    # sequences' block tables, followed by the sequence's own pages
    prefix, mine = _prefix_lens(c)
    groups, seqs = c["groups"], c["seqs"]
    pre_pages = [p // page for p in prefix]
    own_pages = [-(-m // page) for m in mine]
    total = sum(pre_pages) + sum(own_pages)
    perm = np.random.RandomState(int(seed) % (1 << 32)).permutation(total)
    width = max(pre_pages[i // seqs] + n for i, n in enumerate(own_pages))
    table = np.zeros((groups * seqs, width), np.int32)
    at = 0
    for i in range(groups):
        got = perm[at:at + pre_pages[i]]
        at += pre_pages[i]
        table[i * seqs:(i + 1) * seqs, :pre_pages[i]] = got[None, :]
    for b, n in enumerate(own_pages):
        p = pre_pages[b // seqs]
        table[b, p:p + n] = perm[at:at + n]
        at += n
    s["pages"] = torch.from_numpy(table).cuda()
    lens = [prefix[b // seqs] + m for b, m in enumerate(mine)]
    s["prefix"], s["lens"] = _i32(prefix), _i32(lens)
    s["own_most"], s["prefix_most"] = max(mine), max(prefix)
    shape = (total, page, hkv, d)
    s["kc"], s["vc"] = _pool(shape, fp8, g), _pool(shape, fp8, g)
    rows = groups * seqs * c["lq"]
    # (logits of standard deviation 2: some keys matter more than others)
    s["q"] = (2 * torch.randn(rows, c["hq"], d, device="cuda", generator=g)).bfloat16()
    if own:
        import paged_kv_variable_gb300 as pkv
        s["pkv"] = pkv
        batch = groups * seqs
        s["problem"] = pkv.make_problem(batch=batch, num_heads_q=c["hq"], num_heads_kv=hkv, head_dim=d, page_size=page,
                                        cache_capacity=width * page, num_pages=total,
                                        cache_dtype="fp8" if fp8 else "bf16", causal=True, softmax_scale=d ** -0.5)
        s["plan"] = pkv.plan_shared_prefix(s["problem"], [c["lq"]] * batch, lens, None,
                                           group_starts=[i * seqs for i in range(groups + 1)], prefix_lens=prefix)
        s["ws"] = pkv.workspace_tensor(s["plan"].workspace_bytes)
        s["plan"].upload(s["ws"])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(c["hq"], rows, dtype=torch.float32, device="cuda")
        s["cu"] = _i32([c["lq"] * b for b in range(batch + 1)])
        s["args"] = pkv.make_args(q=s["q"], out=s["out"], lse=s["lse"], cu_seqlens_q=s["cu"], max_seqlen_q=c["lq"],
                                  k_cache=s["kc"], v_cache=s["vc"], cache_seqlens=s["lens"], block_table=s["pages"],
                                  k_scale=s["scale"] if fp8 else None, v_scale=s["scale"] if fp8 else None)
    return s


# ------------------------------------------------------------------ the operators
def _transform(x, w, pos, table, pairs):
    """x (T, H, D): RMS norm over D (w given), then the rotation of the first
    rot dims by the angles of row `pos` of the table; fp32."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    rot = table.shape[1]
    half = rot // 2
    row = table[pos.long()]
    cos, sin = row[:, None, :half], row[:, None, half:]
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _codes(x, scale):
    return (x.float() * (1.0 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _as_values(cache):
    """A cache as the numbers it holds (e4m3 codes: their values, times no scale)."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def run(state):
    s = state
    c = s["c"]
    if c["op"] == "qk_norm_rope":
        if own:
            s["pkv"].qk_norm_rope(s["args"], s["spec"])
            return s["q_out"], s["k_out"]
        return tuple(_transform(x, w, s["pos"], s["table"], c["pairs"]).bfloat16()
                     for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    if c["op"] == "rope_kv_append":
        if own:
            s["pkv"].rope_kv_append(s["problem"], s["args"], s["rope"], s["total"], s["total"])
            return s["q_out"], _as_values(s["kc"]), _as_values(s["vc"])
        t = torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32)
        seq = torch.searchsorted(s["cu"][1:], t, right=True)
        pos = (s["cached"][seq] + t - s["cu"][seq]).long()
        q, k = (_transform(x, w, pos, s["table"], c["pairs"]) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
        at = (s["pages"][seq, pos // c["page"]].long(), pos % c["page"]) if c["page"] else (seq, pos)
        s["kc"][at] = _codes(k, s["scale"]) if c["fp8"] else k.bfloat16()
        s["vc"][at] = _codes(s["v"], s["scale"]) if c["fp8"] else s["v"]
        return q.bfloat16(), _as_values(s["kc"]), _as_values(s["vc"])

    if own:
        s["pkv"].attn_varlen_kvcache_fwd(s["problem"], s["args"], s["plan"], s["ws"])
        return s["out"], s["lse"]
    groups, seqs, lq, hkv, d, page = (c[x] for x in ("groups", "seqs", "lq", "hkv", "d", "page"))
    per = c["hq"] // hkv

    def rows(cache, pages):  # (n, m) pages -> (n, hkv, m * page, d) keys or values
        x = cache[pages.long()]
        x = x.view(torch.float8_e4m3fn).float() * s["scale"] if c["fp8"] else x.float()
        return x.flatten(1, 2).transpose(1, 2)

    q = s["q"].float().view(groups, seqs, lq, hkv, per, d) * d ** -0.5
    # the prefix keys, once for all the queries of a group: (groups, hkv, queries x heads, keys)
    first = s["pages"][::seqs, :s["prefix_most"] // page]
    kp, vp = rows(s["kc"], first), rows(s["vc"], first)
    sp = q.permute(0, 3, 1, 2, 4, 5).reshape(groups, hkv, seqs * lq * per, d) @ kp.transpose(2, 3)
    j = torch.arange(sp.shape[-1], device="cuda")
    sp = sp.masked_fill((j >= s["prefix"][:, None])[:, None, None, :], -math.inf)
    # each sequence's own keys: (groups x seqs, hkv, queries x heads, keys)
    batch = groups * seqs
    skip = s["prefix"].repeat_interleave(seqs)
    n = -(-s["own_most"] // page)
    cols = (skip // page)[:, None] + torch.arange(n, device="cuda")
    mine = s["pages"].gather(1, cols.clamp(max=s["pages"].shape[1] - 1).long())
    ko, vo = rows(s["kc"], mine), rows(s["vc"], mine)
    so = q.reshape(batch, lq, hkv, per, d).transpose(1, 2).reshape(batch, hkv, lq * per, d) @ ko.transpose(2, 3)
    j = torch.arange(so.shape[-1], device="cuda")
    sees = (s["lens"] - skip - lq)[:, None] + 1 + torch.arange(lq, device="cuda")  # own keys query i sees
    hidden = (j[None, None, :] >= sees[:, :, None]).repeat_interleave(per, dim=1)
    so = so.masked_fill(hidden[:, None], -math.inf)
    # one softmax over both
    sp = sp.view(groups, hkv, seqs, lq * per, -1).transpose(1, 2).reshape(batch, hkv, lq * per, -1)
    most = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    sp, so = torch.exp(sp - most), torch.exp(so - most)
    total = sp.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
    op = (sp.view(groups, seqs, hkv, lq * per, -1).transpose(1, 2).reshape(groups, hkv, seqs * lq * per, -1) @ vp)
    op = op.view(groups, hkv, seqs, lq * per, d).transpose(1, 2).reshape(batch, hkv, lq * per, d)
    out = (op + so @ vo.masked_fill((j >= (s["lens"] - skip)[:, None])[:, None, :, None], 0.0)) / total
    lse = (most + torch.log(total)).view(batch, hkv, lq, per)
    out = out.view(batch, hkv, lq, per, d).transpose(1, 2).reshape(batch * lq, c["hq"], d)
    return out.bfloat16(), lse.permute(1, 3, 0, 2).reshape(c["hq"], batch * lq)


# ------------------------------------------------------------------ work of one pass
def work(case):
    c = case
    hq, d = c["hq"], c["d"]
    if c["op"] == "qk_norm_rope":
        n = c["tokens"] * (hq + c["hkv"]) * d
        spots = min(c["tokens"], c["far"])
        return {"bytes": 4 * n + 4 * c["tokens"] + 4 * c["rot"] * spots, "flops": n * (3 + 4 * c["norm"])}
    if c["op"] == "rope_kv_append":
        cached, new = _append_lens(c)
        t, es = sum(new), 1 if c["fp8"] else 2
        spots = len({p for a, b in {(a, a + b) for a, b in zip(cached, new)} for p in range(a, b)})
        pages = sum(-(-(a + b) // c["page"]) - a // c["page"] for a, b in zip(cached, new)) if c["page"] else 0
        n = t * (hq + c["hkv"]) * d
        return {"bytes": 4 * t * hq * d + 2 * t * c["hkv"] * d * (2 + es) + 4 * c["rot"] * spots + 8 * c["batch"]
                + 4 * pages, "flops": n * (3 + 4 * c["norm"])}
    prefix, mine = _prefix_lens(c)
    seqs, lq, es = c["seqs"], c["lq"], 1 if c["fp8"] else 2
    keys = sum(prefix) + sum(mine)
    pairs = sum(lq * (prefix[b // seqs] + m) - lq * (lq - 1) // 2 for b, m in enumerate(mine))
    rows = len(mine) * lq
    return {"bytes": 2 * keys * c["hkv"] * d * es + 4 * rows * hq * d + 4 * rows * hq
            + 4 * (sum(prefix) + sum(mine)) // c["page"], "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_rows(x, w, ang, pairs, rot):
    """The transform in 64 bits, the rotation as a product of complex numbers
    (ang: the table's cos + i sin of each token)."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    z = (torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) if pairs else
         torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()))
    z = z * ang[:, None, :]
    y = x.clone()
    if pairs:
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] != "shared_prefix":
        rot, t = c["rot"], s["table"].double()
        ang = torch.complex(t[:, :rot // 2].contiguous(), t[:, rot // 2:].contiguous())
    if c["op"] == "qk_norm_rope":
        a = ang[s["pos"].long()]
        return tuple(_exact_rows(x, w, a, c["pairs"], rot) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    if c["op"] == "rope_kv_append":
        cached, new = _append_lens(c)
        inv = 1.0 / s["scale"].double() if c["fp8"] else None
        held = [_as_values(x).double() for x in (s["kc"], s["vc"])]
        q, t0 = [], 0
        for b, (lc, n) in enumerate(zip(cached, new)):
            a = ang[lc:lc + n]
            q.append(_exact_rows(s["q"][t0:t0 + n], s["qw"], a, c["pairs"], rot))
            k = _exact_rows(s["k"][t0:t0 + n], s["kw"], a, c["pairs"], rot)
            v = s["v"][t0:t0 + n].double()
            if c["fp8"]:
                k, v = ((x * inv).clamp(-448, 448) for x in (k, v))
            pos = torch.arange(lc, lc + n, device="cuda")
            for cache, x in zip(held, (k, v)):
                if c["page"]:
                    cache[s["pages"][b, pos // c["page"]].long(), pos % c["page"]] = x
                else:
                    cache[b, pos] = x
            t0 += n
        return torch.cat(q), held[0], held[1]
    # one sequence at a time over all its keys, as if nothing were shared
    prefix, mine = _prefix_lens(c)
    lq, hkv, d, per = c["lq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(c["hq"], s["q"].shape[0], dtype=torch.float64, device="cuda")
    for b, m in enumerate(mine):
        n = prefix[b // c["seqs"]] + m
        pages = s["pages"][b, :-(-n // c["page"])].long()
        k, v = (_as_values(x[pages]).double().flatten(0, 1)[:n] for x in (s["kc"], s["vc"]))
        if c["fp8"]:
            k, v = k * s["scale"].double(), v * s["scale"].double()
        q = s["q"][b * lq:(b + 1) * lq].double().view(lq, hkv, per, d)
        x = torch.einsum("ihgd,jhd->hgij", q, k) / math.sqrt(d)
        seen = torch.arange(n, device="cuda")[None, :] <= torch.arange(lq, device="cuda")[:, None] + n - lq
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        z = torch.logsumexp(x, dim=-1)
        out[b * lq:(b + 1) * lq] = torch.einsum("hgij,jhd->ihgd", torch.exp(x - z[..., None]), v).reshape(
            lq, c["hq"], d)
        lse[:, b * lq:(b + 1) * lq] = z.reshape(c["hq"], lq)
    return out, lse
