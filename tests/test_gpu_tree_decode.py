"""The decoding example: rounds of append, attention, tree verification and
commit leave exactly the committed tokens' entries in the cache."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("tree_decode", os.path.join(ROOT, "examples", "tree_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# bf16: one rounding (2^-8); e4m3: half of an eighth of the largest entry's power of two (2^-4 of it), in rows
# whose own largest is at most that
@pytest.mark.gpu
@pytest.mark.parametrize("fmt,bound", [("bf16", 2.0 ** -7), ("e4m3", 2.0 ** -4 * 1.01)])
def test_rounds_leave_the_committed_entries(fmt, bound):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    m = _example()
    state = m.run(rounds=7, B=5, fmt=fmt, seed=3)
    assert sum(len(h) for h in state[3]) > 7 * 5       # some drafts were kept
    assert m.check(*state) <= bound
