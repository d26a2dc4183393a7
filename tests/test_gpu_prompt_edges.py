"""A prompt's calls at their edges, against plain implementations in 64 bits (tolerances as in test_gpu_prompt)."""
import numpy as np
import pytest

from test_gpu_prompt import (BF, F32, Prompt, attend_check, attend_exact, down_exact, gate_up_exact, gen, make_ids, make_layer,  # noqa: F401
                             mv, randn, within)  # (mv: fixture)

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


# ------------------------------------------------------------------ scores far from zero
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_attend_scores_far_above_zero(mv, D):  # noqa: F811
    """A row with a score past 2^31 (times log2 e) is NaN, up to the scores that fp32 does not hold; the rows before it are as
    without it, and a score short of it is as good as any."""
    g = gen(81 + D)
    T = 300
    q, k, v = torch.zeros((T, 2, D), device="cuda"), torch.zeros((T, 1, D), device="cuda"), randn(g, T, 1, D)
    q[..., 0] = 1.0
    k[:100, 0, 0] = torch.randn(100, generator=g, device="cuda")
    st = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    want, z, ot, lt = attend_exact(q[:100].bfloat16(), k[:100].bfloat16(), v[:100], [0, 100], 1.0)
    for low, high in ((31, 40), (60, 90), (127, 128)):
        # powers of two between, with all the digits that bf16 has: products with the scale are rounded up and down
        k[100:, 0, 0] = torch.exp2(torch.linspace(low, high - 0.01, T - 100, device="cuda"))
        out, lse = mv.prompt_attend(q.bfloat16(), k.bfloat16(), v, st, scale=1.0)
        assert out[100:].isnan().all() and lse[100:].isnan().all(), (low, high)
        within(out[:100], want, ot)
        within(lse[:100], z, lt)
    # one key that all the rows behind it are sure of
    k[100:, 0, 0] = torch.randn(T - 100, generator=g, device="cuda")
    for far in (2.0 ** 20, 255 * 2.0 ** 20, 185 * 2.0 ** 22, 2.0 ** 30):
        k[120, 0, 0] = far
        out, lse = mv.prompt_attend(q.bfloat16(), k.bfloat16(), v, st, scale=1.0)
        # its probability is 2^r for the r that the reference was rounded by: rounded to bf16, not to 1, and the result once more
        alone = v[120:121].double().expand(T - 120, 2, D)
        within(out[120:], alone, alone.abs() * (2 * BF + BF * BF + 2.0 ** -18), far)
        assert ((lse[120:].double() - far).abs() <= far * 4 * F32).all(), far


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_attend_scores_far_below_zero(mv, D):  # noqa: F811
    """Keys with scores past -2^31 (times log2 e) have no part in a row that sees others; a row with no other is NaN."""
    g = gen(82 + D)
    T, far = 420, 200
    q, k, v = torch.zeros((T, 2, D), device="cuda"), torch.zeros((T, 1, D), device="cuda"), randn(g, T, 1, D)
    q[..., 0] = 1.0
    k[far:, 0, 0] = torch.randn(T - far, generator=g, device="cuda")
    st = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    want, z, ot, lt = attend_exact(q[far:].bfloat16(), k[far:].bfloat16(), v[far:], [0, T - far], 1.0)
    for low, high in ((31, 40), (60, 90), (127, 128)):
        k[:far, 0, 0] = -torch.exp2(torch.linspace(low, high - 0.01, far, device="cuda"))
        out, lse = mv.prompt_attend(q.bfloat16(), k.bfloat16(), v, st, scale=1.0)
        assert out[:far].isnan().all() and lse[:far].isnan().all(), (low, high)
        within(out[far:], want, ot, (low, high))
        within(lse[far:], z, lt, (low, high))


# ------------------------------------------------------------------ outputs and inputs in one memory
def test_outputs_on_inputs_are_refused(mv):  # noqa: F811
    g = gen(91)
    T = 40
    rot, pos, st = mv.Rotary.standard(64), torch.arange(T, dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    q, k = randn(g, T, 4, 64), randn(g, T, 4, 64)
    _, layer = make_layer(mv, g, 128, 128, 2, False)
    x, u = randn(g, T, 128), mv.union_permute(make_ids(g, T, 2, 1, 0.0), 2)
    w, more = torch.ones((T, 1), device="cuda"), torch.empty(T * 4 * 64 * 2 + T * 4 * 4, dtype=torch.uint8, device="cuda")
    both = more[:T * 4 * 64 * 2].view(torch.bfloat16).view(T, 4, 64)
    before = [t.clone() for t in (q, k, x)]
    for call in (lambda: mv.rotate(rot, q, k, pos, out_q=k, out_k=q), lambda: mv.rotate(rot, q, k, pos, out_q=both, out_k=both),
                 lambda: mv.rotate(rot, q, q, pos, out_q=q), lambda: mv.rotate(rot, q[1:], None, pos[1:], out_q=q[:-1]),
                 lambda: mv.prompt_attend(q, k, k, st, out=q), lambda: mv.prompt_attend(q, k, k, st, out=k),
                 lambda: mv.prompt_attend(q, k, k, st, out=both, lse=more[:T * 16].view(torch.float32).view(T, 4)),
                 lambda: mv.group_gate_up(x, layer, u, 1, out=x), lambda: mv.group_down(x, layer, u, w, y=x),
                 lambda: mv.group_down(x, layer, u, w, workspace=x.view(torch.uint8).view(-1).repeat(4), y=x)):
        with pytest.raises(mv.MoEError):
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((q, k, x), before))


def test_rotate_in_place_in_one_buffer(mv):  # noqa: F811
    """Queries, keys and values as slices of one buffer, tokens or heads outermost, parts behind one another or head by head."""
    g = gen(92)
    T, H, D = 33, 6, 64
    rot, pos = mv.Rotary.standard(D), torch.arange(T, dtype=torch.int32, device="cuda")
    for shape, order in (((T, 3, H, D), (0, 2, 1, 3)), ((T, H, 3, D), (0, 1, 2, 3)), ((3, H, T, D), (2, 1, 0, 3)), ((H, 3, T, D), (2, 0, 1, 3))):
        x = randn(g, *shape)
        parts = x.permute(*order)  # [T, H, 3, D]
        q, k, v = (parts[:, :, i] for i in range(3))
        want, held = mv.rotate(rot, q, k, pos), v.clone()
        got = mv.rotate(rot, q, k, pos, out_q=q, out_k=k)
        assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, held)


# ------------------------------------------------------------------ sums whose terms cancel
@pytest.mark.parametrize("tiled", [False, True])
def test_group_down_terms_that_cancel(mv, tiled):  # noqa: F811
    """Two experts that are nearly alike, with weights of 1 and -1: an output is off by 2^-8 of its terms' sizes and of itself."""
    g = gen(101)
    T, H, I, E, k = 400, 256, 320, 4, 2
    wg, wd = randn(g, E, 2 * I, H, std=H ** -0.5), randn(g, E, H, I, std=I ** -0.5)
    wg[1::2], wd[1::2] = wg[::2], (wd[::2].float() * (1 + 2.0 ** -6)).to(torch.bfloat16)
    layer = mv.ExpertLayer(wg, wd, "bf16")
    if tiled:
        layer = mv.pack_tiled(layer)
    pair = 2 * torch.randint(0, E // 2, (T, 1), generator=g, device="cuda")
    ids = torch.cat([pair, pair + 1], 1).to(torch.int32)
    w = torch.tensor([[1.0, -1.0]], device="cuda").repeat(T, 1)
    err = mv.new_dev_err()
    u = mv.union_permute(ids, E, dev_err=err)
    h = mv.group_gate_up(randn(g, T, H), layer, u, k, dev_err=err)
    y = mv.group_down(h, layer, u, w, dev_err=err)
    assert err.item() == 0
    want, size, sums = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(3))
    place = u["inv"].long().view(T, k)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        hd, wt = h[place[t, j]].double(), wd[e].double()
        want[t] += w[t, j].double()[:, None] * (hd @ wt.t())
        size[t] += (hd @ wt.t()).abs()
        sums[t] += hd.abs() @ wt.abs().t()
    assert want.abs().sum() < 0.05 * size.sum()
    # products of I terms in fp32; each rounded to bf16; their sum of k in fp32; the result rounded
    within(y, want, (1 + BF) * ((BF + k * F32) * size + (1 + BF) * I * F32 * sums) + BF * want.abs(), "y")
