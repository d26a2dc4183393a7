"""Failure paths of kv4_attend and kv4_weigh without any GPU fault: with the test hooks MOE_TEST_STALL_KV4_ATTEND and MOE_TEST_STALL_KV4_FIRST
the last tile of each CTA's share is not copied, or the first one not taken as copied, so the wait for it runs out after its budget (2 s): long after
everything else of the CTA has been started, or with the pipeline full behind it.  MOE_TEST_STALL_KV4_WEIGH does so with the first keys
of a CTA.  The call must report MOE_DEV_TIMEOUT and leave the context usable: the next one gives the same result as before."""
import time

import numpy as np
import pytest

from test_gpu_kv4 import MANY, bf16, dev, make_cache, mv  # noqa: F401  (mv: fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hook", ["TEST_STALL_KV4_ATTEND", "TEST_STALL_KV4_FIRST"])
@pytest.mark.parametrize("max_q", [2, MANY])
@pytest.mark.parametrize("D,base", [(64, [3000, 40]), (128, [20000, 7])])
def test_a_wait_that_runs_out_is_reported(mv, hook, max_q, D, base):  # noqa: F811
    rng = np.random.default_rng(91)
    new = [2, 1]
    _, cache = make_cache(mv, rng, [b + n for b, n in zip(base, new)], 2, D, 64)
    q = bf16(rng.standard_normal((3, 8, D))).cuda()
    args = (cache, q, dev(np.array([0, 2, 3], np.int32)), dev(np.array(base, np.int32)), max_q)
    err = mv.new_dev_err()
    want = mv.kv4_attend(*args, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    lib = mv._lib.load()
    assert lib.moe_test_set_stall(getattr(mv._lib, hook)) == mv._lib.MOE_OK
    try:
        t0 = time.time()
        mv.kv4_attend(*args, dev_err=err)
        torch.cuda.synchronize()
        waited = time.time() - t0
    finally:
        lib.moe_test_set_stall(0)
    assert err.item() == mv._lib.DEV_TIMEOUT
    assert 1.5 < waited < 30.0, waited
    err.zero_()
    got = mv.kv4_attend(*args, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("max_q", [2, 40, MANY])
@pytest.mark.parametrize("Hq,D,base", [(8, 64, [3000, 40]), (8, 128, [20000, 7]), (128, 128, [300, 1000])])
def test_a_wait_for_keys_that_runs_out_is_reported(mv, max_q, Hq, D, base):  # noqa: F811
    """One CTA an item, and clusters that share its rows."""
    rng = np.random.default_rng(92)
    new = [2, 1]
    _, cache = make_cache(mv, rng, [b + n for b, n in zip(base, new)], 2, D, 64)
    q = bf16(rng.standard_normal((3, Hq, D))).cuda()
    args = (q, dev(np.array([0, 2, 3], np.int32)), dev(np.array(base, np.int32)), max_q)
    _, lse = mv.kv4_attend(cache, *args)
    err = mv.new_dev_err()
    want = mv.kv4_weigh(cache, *args, lse, cache.new_mass(), dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    lib = mv._lib.load()
    assert lib.moe_test_set_stall(mv._lib.TEST_STALL_KV4_WEIGH) == mv._lib.MOE_OK
    try:
        t0 = time.time()
        mv.kv4_weigh(cache, *args, lse, cache.new_mass(), dev_err=err)
        torch.cuda.synchronize()
        waited = time.time() - t0
    finally:
        lib.moe_test_set_stall(0)
    assert err.item() == mv._lib.DEV_TIMEOUT
    assert 1.5 < waited < 30.0, waited
    err.zero_()
    got = mv.kv4_weigh(cache, *args, lse, cache.new_mass(), dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(got, want)
