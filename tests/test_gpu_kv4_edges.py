"""The 4-bit KV cache calls at the edges of their ranges: value scales far apart, values that are not finite, several threads and
streams at once, rows left out of the weights, strides that nothing is reached by.
Helpers and tolerances as in test_gpu_kv4."""
import numpy as np
import pytest

from oracle import kv_cache as K
from test_gpu_kv4 import MANY, bf16, dev, make_cache, make_tree, mv  # noqa: F401  (mv: fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def attend(mv, cache, q, new, base, max_q, scale, visible=None):  # noqa: F811
    q_start = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    out, lse = mv.kv4_attend(cache, bf16(q).cuda(), q_start, dev(np.asarray(base, np.int32)), max_q, scale=scale,
                             visible=None if visible is None else dev(visible))
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), lse


def small_products(pg, q, new, base, scale, visible=None):
    """What fp16's smallest step adds to the oracle's bound of a row's outputs: half a step (2^-25) of the row's largest
    probability times value scale, for each code that it sees."""
    D, G = pg.D, q.shape[1] // pg.raw.shape[1]
    add = np.zeros(q.shape[:2])
    qh = bf16(q).double().numpy()
    at = 0
    for s, (n, b) in enumerate(zip(new, base)):
        m = K.seen(b, n, None if visible is None else visible[at:at + n].astype(np.uint64)) & pg.valid(s, b + n)[None]
        for h in range(pg.raw.shape[1]):
            kc, ks, kz = pg.entries(s, h, b + n, 0)
            vc, vs, _ = pg.entries(s, h, b + n, 1)
            for i in range(n):
                for g in range(h * G, (h + 1) * G):
                    S = scale * ((kz[:, None] + ks[:, None] * kc)[m[i]] @ qh[at + i, g])
                    p = np.exp(S - S.max())
                    add[at + i, g] = 2.0 ** -25 * np.max(p / p.sum() * vs[m[i]]) * vc[m[i]].sum(0).max()
        at += n
    return add[..., None]


# ------------------------------------------------------------------ value scales far apart
@pytest.mark.parametrize("max_q", [1, MANY])
@pytest.mark.parametrize("D,page,base", [(64, 64, 3000), (128, 32, 32767)])
@pytest.mark.parametrize("ratio", [0.02, 1e-4])
def test_a_dominant_slot_of_small_values(mv, max_q, D, page, base, ratio):  # noqa: F811
    """Nearly all weight lies on one slot whose values are far smaller than the others' (an attention sink).  Many sequences on
    the same pages, so that one CTA takes a long run of slots with it."""
    rng = np.random.default_rng(D + base)
    pg, _ = make_cache(mv, rng, [base + 1], 1, D, page)
    q = bf16(rng.standard_normal((1, 1, D))).double().numpy()
    scale, S = D ** -0.5, 320
    want = np.log(999.0 * base) + 1.0  # its score, the others' being of variance 1 or so
    pg.write(0, 5, 0, q[0] * (want / scale / np.sum(q * q)))
    pg.write(0, 5, 1, rng.standard_normal((1, D)) * ratio)
    cache = mv.Kv4Cache(dev(pg.raw), dev(np.repeat(pg.table, S, 0)), page, D)
    got, lse = attend(mv, cache, np.repeat(q, S, 0), [1] * S, [base] * S, max_q, scale)
    o, l, _, ot, lt, _ = K.attend(pg, q, [0, 1], [base], scale)
    assert np.all(np.abs(lse.cpu().numpy() - l) <= lt)
    off = np.abs(got - o) / (ot + small_products(pg, q, [1], [base], scale))
    assert off.max() <= 1, off.max((1, 2)).round(2).tolist()


@pytest.mark.parametrize("max_q", [5, MANY])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("small", [1e-3, 0.05])
def test_a_hidden_slot_of_large_values(mv, max_q, D, page, small):  # noqa: F811
    """New tokens whose values are in the tens of thousands, beside a context of small ones: rows that see none of
    them are as exact as without them."""
    rng = np.random.default_rng(D)
    base, new = [150], [5]
    pg, cache = make_cache(mv, rng, [155], 2, D, page, spread=small)
    q = rng.standard_normal((5, 8, D))
    for j in (151, 153):
        pg.write(0, j, 1, rng.uniform(-30000, 30000, (2, D)))
    cache.pages.copy_(torch.from_numpy(pg.raw))
    visible = np.array([1, 2, 0b101, 0b1000, 0b10101], dtype=np.int64)  # tokens 1 and 3 see themselves
    got, lse = attend(mv, cache, q, new, base, max_q, 1.0, visible)
    o, l, _, ot, lt, _ = K.attend(pg, bf16(q).double().numpy(), [0, 5], base, 1.0, visible.astype(np.uint64))
    assert np.all(np.abs(lse.cpu().numpy() - l) <= lt)
    off = np.abs(got - o) / (ot + small_products(pg, q, new, base, 1.0, visible))
    assert off.max() <= 1, off.max((1, 2))


# ------------------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("max_q", [4, 64, MANY])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_a_value_row_that_is_not_finite_spoils_outputs_alone(mv, max_q, D, page):  # noqa: F811
    """A context slot and a tree token whose values were beyond fp16 (held as scale 0 and zero NaN): outputs of the rows that
    see one are NaN; lse and weights go by the keys."""
    rng = np.random.default_rng(51 + D)
    base, new = [90, 70], [3, 4]
    pg, cache = make_cache(mv, rng, [93, 74], 2, D, page)
    bad = np.zeros((2, D))
    bad[:, 3] = 1e6
    pg.write(0, 20, 1, bad)      # seen by all of sequence 0
    pg.write(1, 71, 1, bad)      # new token 1 of sequence 1
    cache.pages.copy_(torch.from_numpy(pg.raw))
    visible = np.array([1, 3, 5, 1, 3, 5, 0b1011], dtype=np.int64)
    q = rng.standard_normal((7, 8, D))
    qh = bf16(q).double().numpy()
    got, lse = attend(mv, cache, q, new, base, max_q, 0.1, visible)
    got_lse = lse.cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        o, l, mass, ot, lt, mt = K.attend(pg, qh, [0, 3, 7], base, 0.1, visible.astype(np.uint64), lse_in=got_lse)
    nan = np.isnan(o).all((1, 2))
    assert nan.tolist() == [True, True, True, False, True, False, True]
    assert np.isnan(got[nan]).all()
    assert np.all(np.abs(got[~nan] - o[~nan]) <= ot[~nan])
    assert np.all(np.abs(got_lse - l) <= lt)
    m = cache.new_mass()
    mv.kv4_weigh(cache, bf16(q).cuda(), dev(np.array([0, 3, 7], np.int32)), dev(np.array(base, np.int32)), max_q, lse, m,
                 visible=dev(visible), scale=0.1)
    m = m.cpu().numpy().astype(np.float64)
    for (s, h), w in mass.items():
        assert np.all(np.abs(m[s, h, :len(w)] - w) <= mt[s, h] + 2.0 ** -23 * w)


# ------------------------------------------------------------------ the binding's workspaces
def cut_calls(mv, rng):  # noqa: F811
    """Calls of different shapes whose items are cut between CTAs: (cache, arguments of kv4_attend)."""
    calls = []
    for Hkv, D, base, new, max_q in ((2, 128, 5000, 1, 1), (1, 64, 9000, 3, MANY), (4, 64, 3000, 2, 2), (1, 128, 4000, 4, MANY)):
        _, cache = make_cache(mv, rng, [base + new], Hkv, D, 64)
        q = bf16(rng.standard_normal((new, 8, D))).cuda()
        calls.append((cache, (q, dev(np.array([0, new], np.int32)), dev(np.array([base], np.int32)), max_q)))
    return calls


def test_two_threads_on_one_stream(mv):  # noqa: F811
    import threading
    calls = cut_calls(mv, np.random.default_rng(81))
    want = [mv.kv4_attend(c, *a) for c, a in calls]
    torch.cuda.synchronize()
    off, start = [], threading.Barrier(2)

    def work(first):
        start.wait()
        got = []
        for i in range(400):
            n = (first + i) % len(calls)
            got.append((n, mv.kv4_attend(calls[n][0], *calls[n][1])))
        torch.cuda.synchronize()
        off.extend(n for n, (o, l) in got if not (torch.equal(o, want[n][0]) and torch.equal(l, want[n][1])))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not off


def test_two_streams_at_once(mv):  # noqa: F811
    calls = cut_calls(mv, np.random.default_rng(82))
    want = [mv.kv4_attend(c, *a) for c, a in calls]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(200):
        n = i % len(calls)
        got.append((n, mv.kv4_attend(calls[n][0], *calls[n][1], stream=streams[i % 3])))
    torch.cuda.synchronize()
    for n, (o, l) in got:
        assert torch.equal(o, want[n][0]) and torch.equal(l, want[n][1])


def test_a_graph_has_workspaces_of_its_own(mv):  # noqa: F811
    """Captured calls with the binding's workspace: replays beside other calls on the stream that they were captured from."""
    calls = cut_calls(mv, np.random.default_rng(83))
    want = [mv.kv4_attend(c, *a) for c, a in calls]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [mv.kv4_attend(c, *a) for c, a in calls]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(side):
            g.replay()
        beside = [mv.kv4_attend(c, *a) for c, a in calls]
    torch.cuda.synchronize()
    for x in (got, beside):
        for (o, l), w in zip(x, want):
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])


# ------------------------------------------------------------------ rows left out of the weights
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("Hq,D,page,new,max_q", [(8, 64, 16, 5, 5), (8, 128, 64, 5, 5), (32, 128, 64, 5, 5), (16, 64, 32, 60, 60), (8, 128, 16, 5, MANY)])
def test_rows_without_a_sum_add_no_weight(mv, tree, Hq, D, page, new, max_q):  # noqa: F811
    """Rows whose lse is -inf add nothing whatever they hold, NaN and infinities in q, and whatever the slots hold."""
    rng = np.random.default_rng(61 + Hq + D)
    base, none = 200, [1, new - 1]
    pg, cache = make_cache(mv, rng, [base + new], 2, D, page)
    q = rng.standard_normal((new, Hq, D))
    visible = make_tree(rng, new) if tree else None
    _, lse = attend(mv, cache, q, [new], [base], max_q, 0.1, visible)
    lse[none] = float("-inf")
    clean = q.copy()
    clean[none] = 0.0
    q[1, :, 7], q[new - 1, :, 9] = np.nan, np.inf
    q_start, b = dev(np.array([0, new], np.int32)), dev(np.array([base], np.int32))
    vis = None if visible is None else dev(visible)
    got, want = cache.new_mass(), cache.new_mass()
    mv.kv4_weigh(cache, bf16(q).cuda(), q_start, b, max_q, lse, got, visible=vis, scale=0.1)
    mv.kv4_weigh(cache, bf16(clean).cuda(), q_start, b, max_q, lse, want, visible=vis, scale=0.1)
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())
    assert np.allclose(got.sum(2).cpu().numpy(), Hq // 2 * (new - 2), rtol=1e-3)  # a row's weights add up to 1
    # No row has a sum: keys that are not finite, of the context and of new tokens, reach nothing either.
    for j in (3, base, base + new - 1):
        pg.par[pg.table[0][j // page], :, j % page, :2] = np.float16("nan")
    cache.pages.copy_(torch.from_numpy(pg.raw))
    held = torch.rand_like(got)
    got = held.clone()
    mv.kv4_weigh(cache, bf16(q).cuda(), q_start, b, max_q, torch.full_like(lse, float("-inf")), got, visible=vis, scale=0.1)
    assert torch.equal(got, held)


# ------------------------------------------------------------------ infinities in q
@pytest.mark.parametrize("max_q", [1, 64, MANY])
def test_an_infinity_in_q_gives_nan_or_an_empty_row(mv, max_q):  # noqa: F811
    """Scores that are -inf for every slot make a row of zeros with lse -inf; a score of +inf or NaN among them makes the row NaN."""
    rng = np.random.default_rng(65)
    pg, cache = make_cache(mv, rng, [40], 1, 64, 16)
    for j in range(40):
        k = rng.uniform(1.0, 2.0, (1, 64))
        k[0, 5], k[0, 6] = 3.0, 1.0  # the largest code, the smallest
        pg.write(0, j, 0, k)
    cache.pages.copy_(torch.from_numpy(pg.raw))
    q = rng.standard_normal((1, 4, 64))
    q[0, 0, 5], q[0, 1, 5], q[0, 2, 6] = -np.inf, np.inf, -np.inf  # -inf; +inf; infinity times code 0
    got, lse = attend(mv, cache, q, [1], [39], max_q, 0.125)
    lse = lse.cpu().numpy()
    assert not got[0, 0].any() and np.isneginf(lse[0, 0])
    assert np.isnan(got[0, 1:3]).all() and np.isnan(lse[0, 1:3]).all()
    o, l, _, ot, lt, _ = K.attend(pg, bf16(np.nan_to_num(q, posinf=0, neginf=0)).double().numpy(), [0, 1], [39], 0.125)
    assert np.all(np.abs(got[0, 3] - o[0, 3]) <= ot[0, 3]) and abs(lse[0, 3] - l[0, 3]) <= lt[0, 3]


# ------------------------------------------------------------------ strides that no element is reached by
def test_strides_of_a_lone_token_and_a_lone_head_are_free(mv):  # noqa: F811
    rng = np.random.default_rng(71)
    D, page = 64, 16
    pg, cache = make_cache(mv, rng, [20], 1, D, page)
    lone = lambda x, strides: torch.as_strided(x, (1, 1, D), strides)  # noqa: E731
    k = torch.from_numpy(rng.standard_normal((1, 1, D)).astype(np.float32)).cuda()
    i32 = lambda *a: dev(np.array(a, np.int32))  # noqa: E731
    for t in (k, k.to(torch.bfloat16)):
        want = mv.kv4_append(cache, t, t, i32(0), i32(7), held=True)
        got = mv.kv4_append(cache, lone(t, (67, 1, 1)), lone(t, (1, 3, 1)), i32(0), i32(7), held=True)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    three = torch.from_numpy(rng.standard_normal((3, 1, D)).astype(np.float32)).cuda()
    got = mv.kv4_append(cache, torch.as_strided(three, (3, 1, D), (D, 5, 1)), three, i32(0, 0, 0), i32(1, 2, 3), held=True)
    assert torch.equal(got[0], got[1])
    q = bf16(rng.standard_normal((1, 1, D))).cuda()
    want = mv.kv4_attend(cache, q, i32(0, 1), i32(19), 1)
    got = mv.kv4_attend(cache, lone(q, (3, 7, 1)), i32(0, 1), i32(19), 1)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    a, b = cache.new_mass(), cache.new_mass()
    mv.kv4_weigh(cache, q, i32(0, 1), i32(19), 1, want[1], a)
    mv.kv4_weigh(cache, lone(q, (3, 7, 1)), i32(0, 1), i32(19), 1, want[1], b)
    assert torch.equal(a, b) and float(a.sum()) > 0.99
    with pytest.raises(mv.MoEError):  # two heads: their stride counts
        mv.kv4_attend(cache, torch.as_strided(bf16(rng.standard_normal((1, 3, D))).cuda(), (1, 2, D), (2 * D, 67, 1)), i32(0, 1), i32(19), 1)


# ------------------------------------------------------------------ nothing in the cache
def test_a_cache_without_sequences(mv):  # noqa: F811
    cache = mv.Kv4Cache.new(0, 2, 16, 64, 0, 4)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    new_len, origin, mass = mv.kv4_evict(cache, cache.new_mass(), i32(), 4, 1)
    assert new_len.shape == (0,) and origin.shape == (0, 2, 4) and mass.shape == (0, 2, 64)
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = mv.kv4_attend(cache, q, i32(0), i32(), 1)
    assert out.shape == (0, 4, 64) and mv.kv4_weigh(cache, q, i32(0), i32(), 1, lse, mass) is mass
    err = mv.new_dev_err()
    x = torch.ones((2, 2, 64), device="cuda")
    k, v = mv.kv4_append(cache, x, x, i32(0, 0), i32(-1, 0), held=True, dev_err=err)  # there is no sequence 0
    torch.cuda.synchronize()
    assert err.item() == mv._lib.DEV_BAD_ID and not bool(k.any()) and not bool(v.any())
