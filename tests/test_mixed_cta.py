"""Prefill and decode tiles on one CTA: tiles of one kind after tiles of the
other take over the K/V stages that those used.  Every plan here is for a single
CTA, so that the order of its items (the costliest first) is the order in which
they run; each call is repeated, over keys and values that the caches have lost
and over ones that they hold, and compared with the oracle and with itself.
"""
import numpy as np
import pytest

import oracle
import synth
from tests import harness as H

pytestmark = pytest.mark.gpu

DECODE, PREFILL = 0, 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_variable_gb300 import build
    build.build()


def mixed_case(d, dtype, P, causal, q_lens, cache_lens, q8=False, sentinel="nan", hq=4, hkv=2):
    import dataclasses
    q_lens, cache_lens = np.array(q_lens, np.int32), np.array(cache_lens, np.int32)
    cap = int(((q_lens + cache_lens).max() + 15) // 16 * 16 + 16)
    spec = synth.Spec(batch=len(q_lens), hq=hq, hkv=hkv, d=d, page_size=P, causal=causal,
                      softmax_scale=float(np.float32(1.0 / np.sqrt(d))), cache_dtype=dtype, q_lens=q_lens,
                      cache_lens=cache_lens, new_lens=q_lens.copy(), capacity=cap, name="mixed-cta")
    case = synth.make_case(spec, np.random.default_rng(9000 + d + P + int(causal)), sentinel=sentinel)
    if q8:
        amax = float(np.abs(synth.bf16_bits_to_f32(case.q)).max())
        case = dataclasses.replace(case, q_scale=float(np.float32(amax / 448.0)))
    return case


def run_on_one_cta(case, repeats=16):
    """The kinds of the CTA's items, in order."""
    import torch
    g = H.GpuCase(case, num_sms=1)
    kinds = [it["kind"] for it in g.plan.items()]
    g.write_prefix()
    ref = oracle.forward(case)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")  # (larger than the L2)
    first = None
    for i in range(repeats):
        g.out.fill_(float("nan"))
        g.lse.fill_(float("nan"))
        if i % 2:
            flush.fill_(i)
            g.q.copy_(g.q.clone())  # (the queries are in the L2, the cache is not)
        g.run()
        torch.cuda.synchronize()
        assert g.status() == 0, g.pkv.last_error()
        bits = H.to_numpy_bits(g.out)
        if first is None:
            first = bits
            H.compare_out(g.out, ref["out"], H.FP8_TOL if case.spec.cache_dtype == "fp8" else H.BF16_TOL)
            H.compare_lse(g.lse, ref["lse"])
        assert np.array_equal(first, bits), f"run {i} differs from the first"
    return kinds


FORMS = [(256, "bf16", False), (128, "bf16", False), (64, "bf16", False), (128, "fp8", False), (256, "fp8", False),
         (128, "fp8", True)]


@pytest.mark.parametrize("P", [1, 4, 16])
@pytest.mark.parametrize("lk", ["whole tiles", "ragged"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,dtype,q8", FORMS)
def test_decode_after_prefill(d, dtype, q8, causal, lk, P):
    """Prompts of several tiles, then decode units of one to four: a decode tile's
    V stage last held a V tile of the prompt's last P V's."""
    if lk == "whole tiles":
        case = mixed_case(d, dtype, P, causal, [128, 1, 64, 1, 2], [640, 255, 704, 127, 382], q8)
    else:
        case = mixed_case(d, dtype, P, causal, [131, 1, 77, 1, 2], [571, 300, 610, 20, 397], q8, sentinel="finite")
    kinds = run_on_one_cta(case)
    turn = kinds.index(DECODE)
    assert turn > 0 and set(kinds[:turn]) == {PREFILL} and set(kinds[turn:]) == {DECODE}


def _decode_keys(d, dtype, cost):
    """Keys of a decode unit that the plan rates at about `cost` (model units)."""
    return int((cost - 64) * 512 / (2 * d * (1 if dtype == "fp8" else 2)))


@pytest.mark.parametrize("P", [1, 4, 16])
@pytest.mark.parametrize("extra", [0, 65, 130, 254])
@pytest.mark.parametrize("d,dtype,q8", FORMS)
def test_prefill_after_decode(d, dtype, q8, extra, P):
    """Decode units, then short prompts: the warps that take no part in decode tiles
    (the S issuer, the converters) reach the prompt's first tiles while the decode
    tiles that fill the same stages may still be on their way."""
    n = _decode_keys(d, dtype, 420 + 130 * d // 128) + extra
    case = mixed_case(d, dtype, P, True, [1, 130, 1, 70, 2, 129], [n, 0, n + 67, 0, n + 128, 0], q8)
    kinds = run_on_one_cta(case)
    turn = kinds.index(PREFILL)
    assert turn > 0 and set(kinds[:turn]) == {DECODE} and set(kinds[turn:]) == {PREFILL}


@pytest.mark.parametrize("P", [1, 16])
@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("d,dtype,q8", FORMS)
def test_kinds_in_turn(d, dtype, q8, seed, P):
    """Decode units and prompts alternating, some of a single tile."""
    rng = np.random.default_rng(seed)
    q_lens, cache_lens = [], []
    for cost in rng.permutation(np.arange(330, 330 + 8 * 40, 40)):
        keys = _decode_keys(d, dtype, cost) + int(rng.integers(0, 8))
        if dtype == "bf16" or keys > 20:
            q_lens.append(1)
            cache_lens.append(keys)
        q_lens.append(int(rng.integers(65, 75)))
        cache_lens.append(max(0, int((cost - 256) * 128 / d) - 40 + int(rng.integers(0, 5))))
    case = mixed_case(d, dtype, P, bool(seed % 2), q_lens, cache_lens, q8)
    kinds = run_on_one_cta(case)
    assert sum(a != b for a, b in zip(kinds, kinds[1:])) >= 6
