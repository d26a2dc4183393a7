"""The example's rounds: selection, write, tree attention, weights, commit and eviction together."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_verify_rounds():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kv4_verify.py")
    spec = importlib.util.spec_from_file_location("kv4_verify", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main(rounds=30, say=lambda *_: None)
    # outputs are rounded to bf16 (half a step, 2^-8 of a value, is the most) after probabilities in fp16 (2^-11)
    assert r["worst"] < 2.0 ** -8 + 2.0 ** -10
    assert r["evictions"] >= 1 and r["committed"] >= 3 * 30
    assert all(n <= 256 for n in r["lengths"])
    # beyond the lengths nothing is left in the account
    for s, n in enumerate(r["lengths"]):
        assert not bool(r["mass"][s, :, n:].any())
