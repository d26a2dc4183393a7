"""Refusals of outputs that share memory with inputs or with each other (CPU: every check comes before any CUDA call)."""
import ctypes as C

import pytest

from test_prompt_abi import FAKE, attend, down, gate_up, layer, lib, prompt, rot, rotate  # noqa: F401  (lib: fixture)
from serving_router_softmax_gb300 import _lib as L

torch = pytest.importorskip("torch")

# (The addresses are made up: a call that was not refused would run on them.)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="refusals are tested where no kernel can run")


def test_rotate(lib):  # noqa: F811
    """4 and 2 heads of 64 in bf16, 3 tokens: q 512 bytes a token, k 256."""
    packed = dict(q_token_stride=384, k_token_stride=384, oq_token_stride=384, ok_token_stride=384)
    a, b, c = FAKE, 2 * FAKE, 3 * FAKE
    good = [dict(q=a, k=b, oq=a, ok=b), dict(q=a, k=b, oq=c, ok=4 * FAKE), dict(q=a, k=a, oq=b, ok=c), dict(q=a, k=b, oq=a, ok=c),
            dict(q=a, k=b, oq=a + 3 * 512, ok=b - 3 * 256)]
    for at in good:  # no device here: as far as the launch
        assert rotate(lib, rot(), **at) == L.MOE_ERR_CUDA, at
    assert rotate(lib, rot(**packed), q=a, k=a + 512, oq=a, ok=a + 512) == L.MOE_ERR_CUDA  # in place in one buffer
    assert rotate(lib, rot(n_k_heads=0), q=a, k=a, oq=b, ok=b) == L.MOE_ERR_CUDA          # (k is not looked at)
    bad = [dict(q=a, k=b, oq=b, ok=a),              # each on the other's input
           dict(q=a, k=b, oq=c, ok=c), dict(q=a, k=b, oq=c, ok=c + 3 * 512 - 16),
           dict(q=a, k=a, oq=a, ok=b),              # in place, and still to be read as k
           dict(q=a, k=b, oq=a + 16, ok=c), dict(q=a, k=b, oq=a + 512, ok=c), dict(q=a, k=b, oq=b + 3 * 256 - 16, ok=c),
           dict(q=a, k=b, oq=c, ok=b + 128)]
    for at in bad:
        assert rotate(lib, rot(), **at) == L.MOE_ERR_ARG, at
    assert rotate(lib, rot(**packed), q=a, k=a + 512, oq=a, ok=a + 496) == L.MOE_ERR_ARG
    assert rotate(lib, rot(**packed), q=a, k=a + 512, oq=a + 512, ok=b) == L.MOE_ERR_ARG
    assert rotate(lib, rot(**packed), q=a, k=a + 512, oq=a + 768, ok=b) == L.MOE_ERR_ARG


def test_prompt_attend(lib):  # noqa: F811
    """9 tokens, 8 heads on 2 of 64: out 9,216 bytes, lse 288; q 1,024 bytes a token, k and v 256."""
    q, k, v, out, lse = (i * FAKE for i in (2, 3, 4, 5, 6))
    assert attend(lib, prompt(), q=q, k=k, v=v, out=out, lse=lse) == L.MOE_ERR_CUDA
    assert attend(lib, prompt(), q=q, k=q, v=q, out=out, lse=None) == L.MOE_ERR_CUDA
    assert attend(lib, prompt(), q=q, k=k, v=v, out=q + 9216, lse=out) == L.MOE_ERR_CUDA
    for at in (dict(out=q), dict(out=k), dict(out=v), dict(out=q + 9216 - 16), dict(out=k - 9216 + 16), dict(lse=q), dict(lse=k + 256), dict(lse=v - 284),
               dict(lse=out), dict(lse=out + 9216 - 4), dict(lse=out - 284)):
        assert attend(lib, prompt(), **{**dict(q=q, k=k, v=v, out=out, lse=lse), **at}) == L.MOE_ERR_ARG, at


def test_group_products(lib):  # noqa: F811
    """300 tokens of 2 experts, H 128, I 192: x and y 76,800 bytes, h 230,400."""
    a, b, c = FAKE, 2 * FAKE, 3 * FAKE
    need = lib.moe_group_down_workspace(C.byref(layer()), 300, 2)
    assert gate_up(lib, layer(), x=a, h=b) == L.MOE_ERR_CUDA and gate_up(lib, layer(), x=a, h=a + 76800) == L.MOE_ERR_CUDA
    for h in (a, a + 76800 - 16, a - 230400 + 16):
        assert gate_up(lib, layer(), x=a, h=h) == L.MOE_ERR_ARG, h
    assert gate_up(lib, layer(H=128, I=128), T=40, k=1, x=a, h=a) == L.MOE_ERR_ARG  # of one shape
    assert down(lib, layer(), h=a, y=b, ws=c, size=need) == L.MOE_ERR_CUDA
    for at in (dict(y=a), dict(y=a + 230400 - 16), dict(y=a - 76800 + 16), dict(ws=a), dict(ws=b), dict(ws=a + 229376), dict(ws=b - need + 256), dict(y=c + need - 16)):
        assert down(lib, layer(), **{**dict(h=a, y=b, ws=c, size=need), **at}) == L.MOE_ERR_ARG, at
