"""Failure paths of a prompt's calls without any GPU fault: with the test hooks MOE_TEST_STALL_GROUP and MOE_TEST_STALL_PROMPT copies are
left out, so the waits for them run out after their budget (2 s).  The call must report MOE_DEV_TIMEOUT and leave the context
usable: the next one gives the same result as before."""
import time

import pytest

from test_gpu_prompt import gen, make_ids, make_layer, mv, randn  # noqa: F401  (mv: fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def stalled(mv, hook, call):  # noqa: F811
    err = mv.new_dev_err()
    want = call(err)
    torch.cuda.synchronize()
    assert err.item() == 0
    lib = mv._lib.load()
    assert lib.moe_test_set_stall(hook) == mv._lib.MOE_OK
    try:
        t0 = time.time()
        call(err)
        torch.cuda.synchronize()
        waited = time.time() - t0
    finally:
        lib.moe_test_set_stall(0)
    assert err.item() == mv._lib.DEV_TIMEOUT
    assert 1.5 < waited < 30.0, waited
    err.zero_()
    got = call(err)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("T", [3, 900])
def test_group_products(mv, T):  # noqa: F811
    g = gen(61)
    H, I, E, k = 512, 320, 5, 2
    _, layer = make_layer(mv, g, H, I, E, True)
    x, ids = randn(g, T, H), make_ids(g, T, E, k, 0.3)
    u = mv.union_permute(ids, E)
    p = torch.rand((T, k), generator=g, device="cuda")
    h = mv.group_gate_up(x, layer, u, k)
    stalled(mv, mv._lib.TEST_STALL_GROUP, lambda err: mv.group_gate_up(x, layer, u, k, dev_err=err))
    stalled(mv, mv._lib.TEST_STALL_GROUP, lambda err: mv.group_down(h, layer, u, p, dev_err=err))


@pytest.mark.parametrize("D,lengths", [(64, [5, 0, 700]), (128, [300, 1]), (128, [2000])])
def test_prompt_attend(mv, D, lengths):  # noqa: F811
    g = gen(62)
    T = sum(lengths)
    q, k, v = randn(g, T, 8, D), randn(g, T, 2, D), randn(g, T, 2, D)
    start = [0]
    for n in lengths:
        start.append(start[-1] + n)
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    stalled(mv, mv._lib.TEST_STALL_PROMPT, lambda err: mv.prompt_attend(q, k, v, st, dev_err=err)[0])
