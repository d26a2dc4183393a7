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


# ------------------------------------------------------------------ beside the cache's attention and the verify step
def test_prompt_attend_and_the_cache_give_the_same(mv):  # noqa: F811
    """A prompt through both attentions: outputs and log-sums are as near each other as each one's roundings, and the exact
    difference that rounding the held values to bf16 makes, allow."""
    from oracle import kv_cache as okv
    g = gen(111)
    T, Hq, Hkv, D, page = 300, 8, 2, 128, 64
    q, k, v = randn(g, T, Hq, D), randn(g, T, Hkv, D), randn(g, T, Hkv, D)
    cache = mv.Kv4Cache.new(8, Hkv, page, D, 1, 6)
    cache.table[0] = torch.tensor([5, 0, 7, 2, 1, 3], dtype=torch.int32, device="cuda")
    i = torch.arange(T, dtype=torch.int32, device="cuda")
    mv.kv4_append(cache, k, v, torch.zeros_like(i), i)
    kh, vh = mv.kv4_read(cache, torch.zeros_like(i), i)
    st = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out, lse = mv.prompt_attend(q, kh, vh, st)
    o4, l4 = mv.kv4_attend(cache, q, st, torch.zeros(1, dtype=torch.int32, device="cuda"), T)
    mine = attend_exact(q, kh, vh, [0, T], D ** -0.5)
    pages = okv.Pages(cache.pages.cpu().numpy(), cache.table.cpu().numpy(), page, D)
    theirs = okv.attend(pages, q.float().cpu().numpy(), [0, T], [0], D ** -0.5)
    want, z, ot, lt = (torch.from_numpy(theirs[n]).cuda() for n in (0, 1, 3, 4))
    within(out, mine[0], mine[2], "prompt_attend")
    within(o4, want, ot, "kv4_attend")
    within(out, o4.double(), mine[2] + ot + (mine[0] - want).abs(), "out")
    within(lse, l4.double(), mine[3] + lt + (mine[1] - z).abs(), "lse")
    # the bounds tell a key more or less: they are far below what the last key of a row is worth
    assert (mine[3] + lt + (mine[1] - z).abs()).max() < 2.0 ** -6 and (lse - l4).abs().max() < 2.0 ** -6


def test_the_step_after_a_prompts_pass(mv):  # noqa: F811
    """The keys and values that a pass has written are in their slots, and the next step's tokens attend over them."""
    from oracle import kv_cache as okv
    lengths, Hq, Hkv, D = [150, 1, 64, 333], 8, 2, 64
    pr = Prompt(mv, 32, lengths)
    k = pr.run()[1]
    v = pr.qkv[:, Hq + Hkv:]
    # the same rows in a cache of other pages
    other = mv.Kv4Cache.new(4 * 12, Hkv, 32, D, 4, 12)
    other.table.copy_(torch.arange(48, dtype=torch.int32).flip(0).view(4, 12))
    held = mv.kv4_append(other, k, v, pr.seq, pr.slot, held=True)
    assert all(torch.equal(a, b) for a, b in zip(mv.kv4_read(pr.cache, pr.seq, pr.slot), held))
    g = gen(112)
    qkv, four = randn(g, 4, Hq + 2 * Hkv, D), torch.arange(5, dtype=torch.int32, device="cuda")
    base = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    pos = torch.stack([base, base + 7, base + 9]).contiguous()
    q, k = mv.rotate(pr.rot, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], pos)
    mv.kv4_append(pr.cache, k, qkv[:, Hq + Hkv:], four[:4], base)
    out, lse = mv.kv4_attend(pr.cache, q, four, base, 1)
    pages = okv.Pages(pr.cache.pages.cpu().numpy(), pr.cache.table.cpu().numpy(), 32, D)
    want, z, _, ot, lt, _ = okv.attend(pages, q.float().cpu().numpy(), range(5), lengths, D ** -0.5)
    assert np.all(np.abs(out.float().cpu().numpy() - want) <= ot) and np.all(np.abs(lse.cpu().numpy() - z) <= lt)


# ------------------------------------------------------------------ the largest sizes
@pytest.mark.parametrize("Hq,Hkv,D,lengths", [
    (1, 1, 64, [9001]), (2, 1, 128, [6007, 3]), (3, 1, 64, [4097]),                       # long sequences
    (2, 1, 64, [(i * 29) % 11 for i in range(2048)]), (4, 4, 128, [(i * 5) % 3 for i in range(2048)]),  # as many as are taken
    (1024, 8, 64, [3, 70]), (1024, 1024, 128, [40, 91]), (1024, 512, 64, [129]),          # query heads
])
def test_prompt_attend_largest(mv, Hq, Hkv, D, lengths):  # noqa: F811
    g = gen(sum(lengths) + Hq)
    T = sum(lengths) + 3
    attend_check(mv, randn(g, T, Hq, D), randn(g, T, Hkv, D), randn(g, T, Hkv, D), lengths, D ** -0.5, first=1)


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("T,H,I,E,k", [(300, 3264, 192, 3, 2), (130, 192, 3264, 2, 1), (40, 3264, 3264, 2, 1)])
def test_group_products_of_odd_row_tiles(mv, T, H, I, E, k, tiled):  # noqa: F811
    """Matrices of an odd number of row tiles, the last one part of a tile."""
    g = gen(T + H)
    (wg, wd), layer = make_layer(mv, g, H, I, E, tiled)
    x, ids = randn(g, T, H), make_ids(g, T, E, k, 0.3)
    err = mv.new_dev_err()
    u = mv.union_permute(ids, E, dev_err=err)
    h = mv.group_gate_up(x, layer, u, k, dev_err=err)
    want, tol = gate_up_exact(x, wg, ids, u["inv"])
    within(h, want, tol, "gate_up")
    p = torch.rand((T, k), generator=g, device="cuda") - 0.3
    y = mv.group_down(h, layer, u, p, dev_err=err)
    want, tol = down_exact(h, wd, ids, u["inv"], p)
    within(y, want, tol, "down")
    assert err.item() == 0


@pytest.mark.parametrize("T,E,k", [(8192, 128, 8), (4096, 256, 16), (32768, 8, 2)])
def test_the_largest_union(mv, T, E, k):  # noqa: F811
    """Routing, union and products of as many tokens as union_permute takes; a token more is refused, and goes in a second part."""
    g = gen(E)
    H, I = 64, 64
    (wg, wd), layer = make_layer(mv, g, H, I, E, True)
    x, gate = randn(g, T + 1, H), randn(g, E, H, std=0.1)
    err = mv.new_dev_err()

    def experts(x):
        ids, w = mv.route(mv.router_logits(x, gate), k, dev_err=err)
        u = mv.union_permute(ids, E, dev_err=err)
        h = mv.group_gate_up(x, layer, u, k, dev_err=err)
        return ids, w, u, h, mv.group_down(h, layer, u, w, dev_err=err)

    ids, w, u, h, y = experts(x[:T])
    assert err.item() == 0
    order = torch.argsort(ids.view(-1).long(), stable=True)
    assert torch.equal(u["perm_token"].long(), order // k) and torch.equal(u["perm_slot"].long(), order % k)
    want, tol = gate_up_exact(x[:T], wg, ids, u["inv"])
    within(h, want, tol, "gate_up")
    want, tol = down_exact(h, wd, ids, u["inv"], w)
    within(y, want, tol, "down")
    with pytest.raises(mv.MoEError):
        experts(x)
    half = T // 2
    for part in (x[:half], x[half:]):
        ids, w, u, h, y = experts(part)
        want, tol = down_exact(h, wd, ids, u["inv"], w)
        within(y, want, tol, "a part")
    assert err.item() == 0


@pytest.mark.parametrize("T,H,I,E,k,tiled", [(500, 64, 128, 1024, 16, True), (90, 128, 64, 1000, 8, False), (3, 1 << 18, 64, 2, 1, False),
                                             (2, 64, 1 << 18, 2, 2, True)])
def test_group_products_of_many_experts_and_long_rows(mv, T, H, I, E, k, tiled):  # noqa: F811
    g = gen(T + E)
    (wg, wd), layer = make_layer(mv, g, H, I, E, tiled)
    x, ids = randn(g, T, H), make_ids(g, T, E, k, 0.0)
    err = mv.new_dev_err()
    u = mv.union_permute(ids, E, dev_err=err)
    h = mv.group_gate_up(x, layer, u, k, dev_err=err)
    want, tol = gate_up_exact(x, wg, ids, u["inv"])
    within(h, want, tol, "gate_up")
    p = torch.rand((T, k), generator=g, device="cuda") - 0.3
    y = mv.group_down(h, layer, u, p, dev_err=err)
    want, tol = down_exact(h, wd, ids, u["inv"], p)
    within(y, want, tol, "down")
    assert err.item() == 0


def test_rotate_largest(mv):  # noqa: F811
    """As many tokens, and as many heads, as are taken: rows far behind the first turn as they do alone."""
    g = gen(121)
    for T, Hq, Hk, D in ((1 << 24, 1, 0, 16), (1 << 24, 1, 1, 64), (40, 4000, 96, 64), (70001, 300, 20, 128)):
        rot = mv.Rotary.standard(D)
        x = randn(g, T, Hq + Hk, D)
        pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3
        q, k = mv.rotate(rot, x[:, :Hq], x[:, Hq:] if Hk else None, pos)
        for part in (slice(0, 30), slice(T // 2, T // 2 + 20), slice(T - 33, T)):
            a, b = mv.rotate(rot, x[part, :Hq], x[part, Hq:] if Hk else None, pos[part])
            assert torch.equal(q[part], a) and (b is None or torch.equal(k[part], b)), (T, part)


@pytest.mark.parametrize("T,Hq,Hkv,D,n", [(1 << 24, 1, 1, 64, 8192), (40000, 1024, 8, 128, 100)])
def test_prompt_attend_most_rows(mv, T, Hq, Hkv, D, n):  # noqa: F811
    """As many tokens as are taken, and outputs of more than 2^31 values."""
    g = gen(122)
    q, k, v = randn(g, T, Hq, D), randn(g, T, Hkv, D), randn(g, T, Hkv, D)
    start = list(range(0, T + 1, n))
    err = mv.new_dev_err()
    out, lse = mv.prompt_attend(q, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), dev_err=err)
    assert err.item() == 0
    for s in (0, len(start) // 2, len(start) - 2):
        at = slice(start[s], start[s + 1])
        want, z, ot, lt = attend_exact(q[at], k[at], v[at], [0, n], D ** -0.5)
        within(lse[at], z, lt, s)
        within(out[at], want, ot, s)
