"""A prompt's calls at their edges, against plain implementations in 64 bits (tolerances as in test_gpu_prompt)."""
import pytest

from test_gpu_prompt import down_exact, gate_up_exact, gen, make_ids, make_layer, mv, randn, within  # noqa: F401  (mv: fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [64, 320, 384, 448, 768, 832])
@pytest.mark.parametrize("T,E", [(1, 1), (40, 3), (1500, 4)])
def test_group_products_end_with_nothing_in_flight(mv, T, E, K):  # noqa: F811
    """Fewer, as many and more steps than the ring of copies has places, one tile and many: the last waits of a launch are for what
    has come, and launches follow one another without a pause."""
    g = gen(T + K)
    (wg, wd), layer = make_layer(mv, g, K, K, E, K % 128 == 0)
    x, ids = randn(g, T, K), make_ids(g, T, E, 1, 0.2)
    p = torch.rand((T, 1), generator=g, device="cuda")
    err = mv.new_dev_err()
    u = mv.union_permute(ids, E, dev_err=err)
    h = mv.group_gate_up(x, layer, u, 1, dev_err=err)
    y = mv.group_down(h, layer, u, p, dev_err=err)
    want, tol = gate_up_exact(x, wg, ids, u["inv"])
    within(h, want, tol, "gate_up")
    want, tol = down_exact(h, wd, ids, u["inv"], p)
    within(y, want, tol, "down")
    torch.cuda.synchronize()
    again = []
    for _ in range(30):
        again.append((mv.group_gate_up(x, layer, u, 1, dev_err=err), mv.group_down(h, layer, u, p, dev_err=err)))
    assert all(torch.equal(a, h) and torch.equal(b, y) for a, b in again)
    assert err.item() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths", [[1], [128], [129, 0, 1], [600], [1100, 40, 7]])
def test_prompt_attend_ends_with_nothing_in_flight(mv, D, lengths):  # noqa: F811
    """Fewer and more steps than the ring of copies has places, an item a CTA at most: launches follow one another without a pause."""
    g = gen(D + sum(lengths))
    T = sum(lengths)
    q, k, v = randn(g, T, 8, D), randn(g, T, 4, D), randn(g, T, 4, D)
    start = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    err = mv.new_dev_err()
    want = mv.prompt_attend(q, k, v, start, dev_err=err)
    torch.cuda.synchronize()
    again = [mv.prompt_attend(q, k, v, start, dev_err=err) for _ in range(30)]
    assert all(torch.equal(a, b) for got in again for a, b in zip(got, want))
    assert err.item() == 0
