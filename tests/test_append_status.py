"""The status of the plain append is one word of the caller's."""
import pytest

from tests import harness as H
from tests.test_rope import AppendCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [8, 0])
def test_append_writes_one_status_word(page):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_variable_gb300 as pkv
    from paged_kv_variable_gb300 import build as b
    b.build()
    c = AppendCase(pkv, torch, 8, d=64, page=page, fp8=False, new=[2, 3], cached=[6, 10])
    c.lens = H.i32([6, 1 << 30])                  # sequence 1: past the capacity
    words = torch.tensor([0, 77, 78, 79], dtype=torch.int32, device="cuda")
    pkv.kv_append(c.problem, c.args(), c.tn, device_status=words[:1])
    assert words.tolist() == [6, 77, 78, 79]
    # the first code stays
    words[0] = 5
    pkv.kv_append(c.problem, c.args(), c.tn, device_status=words[:1])
    assert words.tolist() == [5, 77, 78, 79]
    # and the rotating append's is three
    words[0] = 0
    pkv.rope_kv_append(c.problem, c.args(), c.rope, c.tq, c.tn, device_status=words)
    assert words.tolist()[0] == 6 and words.tolist()[1] == 1 and words.tolist()[3] == 79
