"""The 4-bit KV cache calls against the 64-bit oracle: codes and eviction bit-exact, attention and weights within the
error bounds that the oracle derives from the kernels' roundings."""
import numpy as np
import pytest

from oracle import kv_cache as K

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import serving_router_softmax_gb300 as m
    return m


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def make_cache(mv, rng, totals, Hkv, D, page, spread=1.0, spare=3, at_least=0):
    """A cache whose sequence s holds totals[s] slots of quantised normal rows; every other slot and page holds NaN parameters."""
    need = [-(-t // page) for t in totals]
    n = max(sum(need) + spare, at_least)
    raw = rng.integers(0, 256, (n, Hkv, page * (D + 8)), dtype=np.uint8)
    table = np.full((len(totals), max(1, max(need, default=1))), -1, dtype=np.int32)
    perm = rng.permutation(n)
    pg = K.Pages(raw, table, page, D)
    pg.par[:] = np.float16("nan")
    at = 0
    for s, t in enumerate(totals):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
        if not t:
            continue
        for part in range(2):
            x = rng.standard_normal((t, Hkv, D)) * spread * np.exp(0.5 * rng.standard_normal((t, Hkv, 1)))
            code, scale, zero = K.quantise(x)
            j = np.arange(t)
            p = table[s][j // page]
            pg.codes[part][p, :, j % page] = code[..., 0::2] | (code[..., 1::2] << 4)
            pg.par[p, :, j % page, 2 * part], pg.par[p, :, j % page, 2 * part + 1] = scale, zero
    return pg, mv.Kv4Cache(dev(raw), dev(table), page, D)


def make_tree(rng, n, full=False):
    bits = []
    for i in range(n):
        bits.append((bits[int(rng.integers(max(0, i - 3), i))] if i else 0) | (1 << i))
    return np.array(bits, dtype=np.uint64).astype(np.int64) if n else np.zeros(0, np.int64)


def check_attention(mv, pg, cache, q, new, base, scale, visible, err_want=0, weigh=True, max_q=None):
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    err = mv.new_dev_err()
    dq = q if isinstance(q, torch.Tensor) else bf16(q).cuda()
    vis = None if visible is None else dev(visible)
    mq = max_q or max(1, max(new))
    out, lse = mv.kv4_attend(cache, dq, dev(q_start), dev(np.asarray(base, np.int32)), mq, visible=vis, scale=scale, dev_err=err)
    again, _ = mv.kv4_attend(cache, dq, dev(q_start), dev(np.asarray(base, np.int32)), mq, visible=vis, scale=scale)
    torch.cuda.synchronize()
    assert err.item() == err_want
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "two runs differ"
    qh = dq.float().cpu().numpy()
    got_lse = lse.cpu().numpy().astype(np.float64)
    o, l, mass, ot, lt, mt = K.attend(pg, qh, q_start, base, scale, None if visible is None else visible.astype(np.uint64), lse_in=got_lse if weigh else None)
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isneginf(got_lse) == np.isneginf(l))
    fin = np.isfinite(l)
    assert np.all(np.abs(got_lse[fin] - l[fin]) <= lt[fin]), np.max(np.abs(got_lse[fin] - l[fin]) / lt[fin])
    bad = np.abs(got - o) > ot
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(got - o)[bad])), np.argwhere(bad)[:5].tolist())
    if weigh:
        m0 = np.random.default_rng(5).random((cache.n_seq, cache.n_kv_heads, cache.max_slots)).astype(np.float32)
        m = dev(m0)
        err.zero_()
        mv.kv4_weigh(cache, dq, dev(q_start), dev(np.asarray(base, np.int32)), mq, lse, m, visible=vis, scale=scale, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == err_want
        gm = m.cpu().numpy().astype(np.float64)
        for (s, h), w in mass.items():
            n = len(w)
            assert np.array_equal(gm[s, h, n:], m0[s, h, n:])
            want = m0[s, h, :n] + w
            assert np.all(np.abs(gm[s, h, :n] - want) <= mt[s, h] + 2.0 ** -23 * want), (s, h)
    return out, lse


MANY = 1 << 20  # a number of new tokens (at most) that makes the kernel for many rows the better one for any cache


ATTEND = [  # (Hq, Hkv, D, page, base lengths, new tokens, tree)
    (8, 8, 128, 16, [1], [1], False), (8, 1, 64, 32, [0], [1], False), (4, 4, 64, 64, [15, 16, 17], [1, 1, 1], False),
    (32, 4, 128, 64, [63, 64, 65, 0, 200], [1, 1, 1, 1, 1], False), (16, 2, 128, 128, [1000, 3], [7, 5], True),
    (64, 4, 128, 64, [300, 129, 0], [7, 1, 4], True), (21, 3, 64, 16, [100, 47], [3, 2], True),
    (6, 2, 128, 256, [255, 256, 257], [2, 0, 3], False), (16, 16, 64, 32, [77], [28], True),
    (24, 1, 128, 32, [500], [6], True), (4, 2, 64, 64, [70], [64], True), (8, 2, 128, 16, [33, 0], [100, 70], False),
    (8, 1, 64, 64, [190], [150], False), (2, 1, 128, 64, [5000], [1], False), (32, 8, 64, 64, [3000, 1, 700], [1, 1, 1], False),
    (40, 8, 128, 64, [0, 0, 0, 0], [1, 2, 3, 4], True), (64, 2, 128, 64, [9000, 4000], [5, 3], True),
    (32, 1, 64, 16, [2500], [17], False), (16, 2, 128, 256, [0], [300], False), (64, 1, 64, 128, [700, 65], [2, 3], True)]


@pytest.mark.parametrize("Hq,Hkv,D,page,base,new,tree", ATTEND)
def test_attention_and_weights(mv, Hq, Hkv, D, page, base, new, tree):
    rng = np.random.default_rng(Hq * 7 + D + sum(base))
    pg, cache = make_cache(mv, rng, [b + n for b, n in zip(base, new)], Hkv, D, page)
    q = rng.standard_normal((sum(new), Hq, D)) * 1.5
    vis = np.concatenate([make_tree(rng, n) for n in new]) if tree else None
    check_attention(mv, pg, cache, q, new, base, D ** -0.5, vis)


@pytest.mark.parametrize("Hq,Hkv,D,page,base,new,tree", ATTEND)
def test_attention_of_the_kernel_for_many_rows(mv, Hq, Hkv, D, page, base, new, tree):
    rng = np.random.default_rng(Hq * 7 + D + sum(base) + 1)
    pg, cache = make_cache(mv, rng, [b + n for b, n in zip(base, new)], Hkv, D, page)
    q = rng.standard_normal((sum(new), Hq, D)) * 1.5
    vis = np.concatenate([make_tree(rng, n) for n in new]) if tree else None
    check_attention(mv, pg, cache, q, new, base, D ** -0.5, vis, max_q=MANY)


@pytest.mark.parametrize("max_q", [1, 2, 5, 40, MANY])
def test_max_q_chooses_the_kernel_only(mv, max_q):
    rng = np.random.default_rng(2)
    base, new = [150, 20], [6, 3]
    pg, cache = make_cache(mv, rng, [156, 23], 2, 64, 32)
    q = rng.standard_normal((9, 8, 64))
    check_attention(mv, pg, cache, q, new, base, 0.2, np.concatenate([make_tree(rng, n) for n in new]), max_q=max_q)


@pytest.mark.parametrize("max_q", [None, 64, MANY])
@pytest.mark.parametrize("spread,scale", [(1e-5, 3e3), (1e-3, 100.0), (200.0, 1e-4), (1.0, 4.0), (1.0, 0.0), (1.0, -0.3)])
def test_ranges_of_values_and_scores(mv, spread, scale, max_q):
    """Tiny and large values (scales across fp16), one-sided softmaxes, a zero and a negative factor."""
    rng = np.random.default_rng(9)
    base, new = [400], [2]
    pg, cache = make_cache(mv, rng, [402], 2, 128, 64, spread=spread)
    check_attention(mv, pg, cache, rng.standard_normal((2, 8, 128)), new, base, scale, None, max_q=max_q)


@pytest.mark.parametrize("max_q", [None, 64, MANY])
def test_query_magnitudes(mv, max_q):
    """Rows of q from 2^-100 to 2^60 beside each other: each is scaled by its own power of two."""
    rng = np.random.default_rng(10)
    pg, cache = make_cache(mv, rng, [130], 1, 128, 64, spread=0.01)
    q = rng.standard_normal((1, 8, 128)) * np.array([2.0 ** e for e in (-100, -40, -10, 0, 4, 6, 8, 10)])[None, :, None]
    check_attention(mv, pg, cache, q, [1], [129], 0.05, None, max_q=max_q)


@pytest.mark.parametrize("max_q", [None, 64, MANY])
def test_constant_rows_have_zero_scale(mv, max_q):
    rng = np.random.default_rng(11)
    pg, cache = make_cache(mv, rng, [40], 1, 64, 16)
    for j in (3, 17, 39):
        pg.write(0, j, 1, np.full((1, 64), 0.75))
        pg.write(0, j, 0, np.full((1, 64), -0.5))
    cache.pages.copy_(torch.from_numpy(pg.raw))
    check_attention(mv, pg, cache, rng.standard_normal((1, 8, 64)) * 2, [1], [39], 0.125, None, max_q=max_q)


@pytest.mark.parametrize("max_q", [None, 64, MANY])
def test_all_rows_constant(mv, max_q):
    """Every value row constant: the output is the softmax mean of the zeros."""
    rng = np.random.default_rng(12)
    pg, cache = make_cache(mv, rng, [70], 2, 64, 32)
    for j in range(70):
        pg.write(0, j, 1, np.repeat(rng.standard_normal((2, 1)) * 1e-3, 64, 1))
    cache.pages.copy_(torch.from_numpy(pg.raw))
    check_attention(mv, pg, cache, rng.standard_normal((3, 8, 64)), [3], [67], 0.125, None, max_q=max_q)


@pytest.mark.parametrize("max_q", [5, 64, MANY])
def test_empty_rows_and_nan_in_masked_slots(mv, max_q):
    """A tree token whose key and value are NaN is seen by itself alone; a padding token sees nothing."""
    rng = np.random.default_rng(13)
    base, new = [30, 0], [5, 4]
    pg, cache = make_cache(mv, rng, [35, 4], 2, 64, 16)
    vis = np.array([1, 3, 4, 9, 0b11001, 1, 0, 0b101, 0], dtype=np.int64)
    for part in range(2):
        pg.par[pg.table[0][32 // 16], :, 32 % 16, 2 * part:2 * part + 2] = np.float16("nan")   # new token 2 of sequence 0
        pg.par[pg.table[1][0], :, 1, 2 * part:2 * part + 2] = np.float16("inf")                # new token 1 of sequence 1
    cache.pages.copy_(torch.from_numpy(pg.raw))
    q = rng.standard_normal((9, 8, 64))
    q_start = dev(np.array([0, 5, 9], np.int32))
    out, lse = mv.kv4_attend(cache, bf16(q).cuda(), q_start, dev(np.array(base, np.int32)), max_q, visible=dev(vis), scale=0.2)
    mass = cache.new_mass()
    clean = lse.clone()
    clean[2] = float("-inf")
    mv.kv4_weigh(cache, bf16(q).cuda(), q_start, dev(np.array(base, np.int32)), max_q, clean, mass, visible=dev(vis), scale=0.2)
    torch.cuda.synchronize()
    o, l = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(o[2]).all() and np.isnan(l[2]).all()
    for i in (6, 8):
        assert not o[i].any() and np.isneginf(l[i]).all()
    assert np.isfinite(np.delete(o, 2, 0)).all()
    m = mass.cpu().numpy()
    assert np.isfinite(m).all() and m[1, :, 3].max() == 0
    # sum of a row's weights is 1: four rows of sequence 0, two of sequence 1, 4 query heads per kv head
    assert np.allclose(m.sum(2), [[16, 16], [8, 8]], atol=1e-3)
    vis2 = vis.copy()
    vis2[2] = 0
    ref = K.attend(pg, bf16(q).float().numpy(), [0, 5, 9], base, 0.2, vis2.astype(np.uint64))
    keep = [i for i in range(9) if i != 2]
    assert np.all(np.abs(o[keep] - ref[0][keep]) <= ref[3][keep])


@pytest.mark.parametrize("max_q", [2, 64, MANY])
def test_nan_query_rows_stay_alone(mv, max_q):
    rng = np.random.default_rng(14)
    pg, cache = make_cache(mv, rng, [50], 1, 128, 16)
    q = rng.standard_normal((2, 4, 128))
    q[0, 1, 5], q[1, 2, 9] = np.nan, np.inf
    out, lse = mv.kv4_attend(cache, bf16(q).cuda(), dev(np.array([0, 2], np.int32)), dev(np.array([48], np.int32)), max_q)
    o = out.float().cpu().numpy()
    assert np.isnan(o[0, 1]).all() and np.isnan(o[1, 2]).all()
    o[0, 1] = o[1, 2] = 0
    assert np.isfinite(o).all()


@pytest.mark.parametrize("max_q", [None, 64, MANY])
def test_bad_pages_and_lengths_are_flagged_and_left_out(mv, max_q):
    rng = np.random.default_rng(15)
    base, new = [100, 40], [2, 2]
    pg, cache = make_cache(mv, rng, [102, 42], 2, 64, 16)
    pg.table[0, 2], pg.table[1, 0] = 10 ** 6, -5
    cache.table.copy_(torch.from_numpy(pg.table))
    check_attention(mv, pg, cache, rng.standard_normal((4, 4, 64)), new, base, 0.2, None, err_want=mv._lib.DEV_BAD_ID, max_q=max_q)
    err = mv.new_dev_err()
    out = torch.full((4, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    mv.kv4_attend(cache, bf16(rng.standard_normal((4, 4, 64))).cuda(), dev(np.array([0, 2, 4], np.int32)),
                  dev(np.array([100, cache.max_slots - 1], np.int32)), max_q or 2, out=out, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() & mv._lib.DEV_CAPACITY and bool((out[2:] == 7).all()) and not bool((out[:2] == 7).any())
    err.zero_()
    mv.kv4_attend(cache, out, dev(np.array([0, 3, 2], np.int32)), dev(np.array([-1, 5], np.int32)), max_q or 2, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() & mv._lib.DEV_CAPACITY


def test_strided_queries_and_another_stream(mv):
    rng = np.random.default_rng(16)
    base, new = [90], [6]
    pg, cache = make_cache(mv, rng, [96], 2, 128, 32)
    fused = bf16(rng.standard_normal((6, 12, 128))).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check_attention(mv, pg, cache, fused[:, 2:10], new, base, 0.1, None)
    side.synchronize()
    heads_first = bf16(rng.standard_normal((8, 6, 128))).cuda().transpose(0, 1)
    check_attention(mv, pg, cache, heads_first, new, base, 0.1, None)


def test_pages_beyond_32_bit_offsets(mv):
    """Pages at byte offsets past 2^32."""
    rng = np.random.default_rng(17)
    D, page, Hkv = 128, 64, 8
    n = (1 << 32) // (Hkv * page * (D + 8)) + 40
    small, _ = make_cache(mv, rng, [200], Hkv, D, page)
    raw = torch.zeros((n, Hkv, page * (D + 8)), dtype=torch.uint8, device="cuda")
    table = np.array([[n - 1, n - 9, 1, n - 20]], dtype=np.int32)
    for i in range(4):
        raw[int(table[0, i])] = dev(small.raw[small.table[0, i]])
    cache = mv.Kv4Cache(raw, dev(table), page, D)
    q = rng.standard_normal((1, 16, D))
    check_attention(mv, small, cache, q, [1], [199], 0.1, None)
    x = bf16(rng.standard_normal((1, Hkv, D))).cuda()
    k, v = mv.kv4_append(cache, x, -x, dev(np.array([0], np.int32)), dev(np.array([120], np.int32)), held=True)
    k2, v2 = mv.kv4_read(cache, dev(np.array([0], np.int32)), dev(np.array([120], np.int32)))
    assert torch.equal(k, k2) and torch.equal(v, v2) and float((k - x).abs().max()) < 0.5


@pytest.mark.parametrize("max_q", [2, 64, MANY])
def test_attend_in_a_graph(mv, max_q):
    rng = np.random.default_rng(18)
    pg, cache = make_cache(mv, rng, [300, 40], 2, 64, 16)
    q = bf16(rng.standard_normal((4, 8, 64))).cuda()
    qs, base = dev(np.array([0, 2, 4], np.int32)), dev(np.array([298, 38], np.int32))
    out = torch.empty((4, 8, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, 8), device="cuda")
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    want, _ = mv.kv4_attend(cache, q, qs, base, max_q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mv.kv4_attend(cache, q, qs, base, max_q, out=out, lse=lse, workspace=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    base -= 20  # the lengths are read at replay time
    g.replay()
    again, _ = mv.kv4_attend(cache, q, qs, base, max_q)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and not torch.equal(out, want)


# ------------------------------------------------------------------ write and read
@pytest.mark.parametrize("T,Hkv,D,page,f32", [(1, 1, 64, 16, False), (7, 4, 128, 64, False), (130, 3, 128, 32, True),
                                              (333, 8, 64, 256, False), (50, 1, 128, 128, True)])
def test_append_and_read_match_the_oracle(mv, T, Hkv, D, page, f32):
    rng = np.random.default_rng(T + D)
    S, slots = 3, 200
    pg, cache = make_cache(mv, rng, [slots] * S, Hkv, D, page)
    x = rng.standard_normal((T, 2 * Hkv, D)).astype(np.float32) * 3
    x[:, :, 7] += 12.0
    if T > 20:
        x[3] = 1.25           # constant rows
        x[5] = np.round(x[5] * 4) / 4
        x[6, 0] = np.arange(D) % 31 * 0.5 - 1   # quotients on halves
        x[8] *= 1e-6          # scales at the bottom of fp16
        x[9] *= 5000.0
    t = torch.from_numpy(x) if f32 else bf16(x)
    x = t.float().numpy()
    place = rng.permutation(S * slots)[:T]
    seq, slot = (place // slots).astype(np.int32), (place % slots).astype(np.int32)
    if T > 20:
        slot[11] = -1
    g = t.cuda()
    err = mv.new_dev_err()
    k, v = mv.kv4_append(cache, g[:, :Hkv], g[:, Hkv:], dev(seq), dev(slot), held=True, dev_err=err)
    for i in range(T):
        if slot[i] >= 0:
            pg.write(int(seq[i]), int(slot[i]), 0, x[i, :Hkv])
            pg.write(int(seq[i]), int(slot[i]), 1, x[i, Hkv:])
    torch.cuda.synchronize()
    # rows beyond fp16 (some of those scaled by 5000) are held as NaN and flagged
    assert err.item() == (mv._lib.DEV_BAD_KV if np.abs(x[slot >= 0]).max() > 65504 else 0)
    assert np.array_equal(cache.pages.cpu().numpy(), pg.raw), "pages differ"
    err.zero_()
    rk, rv = mv.kv4_read(cache, dev(seq), dev(slot), torch.float32 if f32 else torch.bfloat16, dev_err=err)
    assert err.item() == 0
    for a, b in ((rk, k), (rv, v)):
        assert np.array_equal(a.float().cpu().numpy(), b.float().cpu().numpy(), equal_nan=True)
    for i in range(T):
        for part, got in ((0, k), (1, v)):
            if slot[i] < 0:
                assert not bool(got[i].any())
                continue
            c, s, z = K.quantise(x[i, :Hkv] if part == 0 else x[i, Hkv:])
            want = z[:, None] + s[:, None] * c
            half = 2.0 ** -24 if f32 else 2.0 ** -8 + 2.0 ** -23
            g64 = got[i].double().cpu().numpy()
            assert np.array_equal(np.isnan(g64), np.isnan(want))
            assert np.all(np.abs(g64 - want)[~np.isnan(want)] <= half * np.abs(want[~np.isnan(want)]))
    # without the held values the cache gets the same bytes
    pg2, cache2 = make_cache(mv, np.random.default_rng(T + D), [slots] * S, Hkv, D, page)
    assert mv.kv4_append(cache2, g[:, :Hkv], g[:, Hkv:], dev(seq), dev(slot)) is None
    assert torch.equal(cache2.pages, cache.pages)


def test_append_flags_bad_values_and_places(mv):
    rng = np.random.default_rng(21)
    pg, cache = make_cache(mv, rng, [40, 40], 2, 64, 16)
    before = cache.pages.clone()
    x = rng.standard_normal((6, 2, 64)).astype(np.float32)
    x[1, 0, 3], x[2, 1, 5], x[3, 0, 1] = np.nan, np.inf, 1e5
    g = torch.from_numpy(x).cuda()
    ok = torch.from_numpy(rng.standard_normal((6, 2, 64)).astype(np.float32)).cuda()
    err = mv.new_dev_err()
    i32 = lambda *a: dev(np.array(a, np.int32))  # noqa: E731
    k, v = mv.kv4_append(cache, g, ok, i32(0, 0, 0, 0, 0, 0), i32(0, 1, 2, 3, 4, 5), held=True, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == mv._lib.DEV_BAD_KV
    kn = torch.isnan(k).all(-1).cpu().numpy()
    assert kn.tolist() == [[False, False], [True, False], [False, True], [True, False], [False, False], [False, False]]
    assert bool(torch.isfinite(v).all())
    cache.pages.copy_(before)
    for seq, slot in ((-1, 0), (2, 0), (0, -2), (0, 10 ** 6), (1, cache.max_slots)):
        err.zero_()
        k, v = mv.kv4_append(cache, ok, ok, i32(*[seq] * 6), i32(*[slot] * 6), held=True, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == mv._lib.DEV_BAD_ID and not bool(k.any())
        err.zero_()
        k, v = mv.kv4_read(cache, i32(seq), i32(slot), dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == mv._lib.DEV_BAD_ID and not bool(k.any()) and not bool(v.any())
    assert torch.equal(cache.pages, before)


# ------------------------------------------------------------------ eviction
def check_evict(mv, pg, cache, mass, lens, keep, recent, in_place, err_want=0):
    err = mv.new_dev_err()
    m = dev(mass)
    out = m if in_place else torch.full_like(m, 3.0)
    new_len, origin, got = mv.kv4_evict(cache, m, dev(np.asarray(lens, np.int32)), keep, recent, mass_out=None if in_place else out, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == err_want
    raw0 = pg.raw.copy()
    old = K.Pages(raw0, pg.table, pg.page, pg.D)
    want_mass = (mass if in_place else np.full_like(mass, 3.0)).copy()
    og = origin.cpu().numpy()
    for s, n in enumerate(lens):
        assert new_len[s].item() == min(n, keep)
        for h in range(cache.n_kv_heads):
            pick = K.evict(mass[s, h], n, keep, recent)
            assert og[s, h, :len(pick)].tolist() == pick.tolist(), (s, h)
            assert (og[s, h, len(pick):] == -1).all()
            want_mass[s, h, :len(pick)] = mass[s, h, pick]
            want_mass[s, h, len(pick):n] = 0
            i = np.arange(len(pick))
            p, r, ps, rs = pg.table[s][i // pg.page], i % pg.page, pg.table[s][pick // pg.page], pick % pg.page
            for part in range(2):
                pg.codes[part][p, h, r] = old.codes[part][ps, h, rs]
            pg.par[p, h, r] = old.par[ps, h, rs]
    assert np.array_equal(cache.pages.cpu().numpy(), pg.raw), "entries differ"
    assert np.array_equal(got.cpu().numpy(), want_mass, equal_nan=True)


@pytest.mark.parametrize("Hkv,D,page,lens,keep,recent", [
    (1, 64, 16, [10], 4, 1), (2, 128, 64, [300, 100, 0, 101], 100, 20), (3, 64, 32, [1025, 64], 64, 64),
    (1, 128, 16, [5000], 1000, 0), (2, 64, 256, [257], 256, 3), (1, 128, 128, [2500, 2501], 2499, 128),
    (4, 128, 64, [1], 1, 0), (1, 64, 64, [70, 3], 1, 0), (2, 128, 32, [9000, 20], 700, 33), (1, 64, 16, [33000], 8000, 100)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_matches_the_oracle(mv, Hkv, D, page, lens, keep, recent, in_place):
    rng = np.random.default_rng(keep + sum(lens))
    pg, cache = make_cache(mv, rng, lens, Hkv, D, page)
    mass = np.exp(2 * rng.standard_normal((len(lens), Hkv, cache.max_slots))).astype(np.float32)
    mass[rng.random(mass.shape) < 0.3] = 0.0      # many ties
    mass[rng.random(mass.shape) < 0.1] = 1.0
    check_evict(mv, pg, cache, mass, lens, keep, recent, in_place)


def test_evict_with_equal_signed_and_nan_masses(mv):
    rng = np.random.default_rng(30)
    lens = [600, 601, 602, 603]
    pg, cache = make_cache(mv, rng, lens, 1, 64, 16)
    mass = np.zeros((4, 1, cache.max_slots), dtype=np.float32)
    mass[0] = 2.0
    mass[1] = rng.standard_normal(cache.max_slots)
    mass[2, 0, ::2] = -0.0
    mass[3] = rng.random(cache.max_slots)
    mass[3, 0, 5:400:3] = np.nan
    mass[3, 0, 7] = np.inf
    mass[3, 0, 9] = -np.inf
    check_evict(mv, pg, cache, mass, lens, 500, 10, False, err_want=mv._lib.DEV_BAD_PROB)


def test_evict_flags_lengths_and_pages(mv):
    rng = np.random.default_rng(31)
    pg, cache = make_cache(mv, rng, [64, 64], 1, 64, 16)
    before = cache.pages.clone()
    m = torch.rand((2, 1, cache.max_slots), device="cuda")
    err = mv.new_dev_err()
    new_len, origin, _ = mv.kv4_evict(cache, m, dev(np.array([-1, cache.max_slots + 1], np.int32)), 8, 2, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == mv._lib.DEV_CAPACITY and new_len.tolist() == [0, 0] and bool((origin == -1).all())
    assert torch.equal(cache.pages, before)
    cache.table[0, 3] = 10 ** 6
    err.zero_()
    m[:, :, :48] = 0
    mv.kv4_evict(cache, m, dev(np.array([64, 0], np.int32)), 8, 2, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == mv._lib.DEV_BAD_ID and torch.equal(cache.pages, before)


def test_python_refusals(mv):
    rng = np.random.default_rng(40)
    pg, cache = make_cache(mv, rng, [20], 2, 64, 16)
    i32 = lambda *a: dev(np.array(a, np.int32))  # noqa: E731
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    bad = [lambda: mv.Kv4Cache(cache.pages, cache.table, 32, 64), lambda: mv.Kv4Cache(cache.pages, cache.table.long(), 16, 64),
           lambda: mv.kv4_attend(cache, q.float(), i32(0, 1), i32(19), 1), lambda: mv.kv4_attend(cache, q[:, :3], i32(0, 1), i32(19), 1),
           lambda: mv.kv4_attend(cache, q, i32(0), i32(19), 1), lambda: mv.kv4_attend(cache, q, i32(0, 1), i32(19).long(), 1),
           lambda: mv.kv4_attend(cache, q, i32(0, 1), i32(19), 0), lambda: mv.kv4_attend(cache, q, i32(0, 1), i32(19), 1, visible=i32(1)),
           lambda: mv.kv4_attend(cache, q, i32(0, 1), i32(19), 1, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: mv.kv4_attend(cache, q.cpu(), i32(0, 1), i32(19), 1),
           lambda: mv.kv4_append(cache, q[:, :2], q[:, :2].float(), i32(0), i32(0)), lambda: mv.kv4_append(cache, q, q, i32(0), i32(0)),
           lambda: mv.kv4_append(cache, q[:, :2].half(), q[:, :2].half(), i32(0), i32(0)),
           lambda: mv.kv4_read(cache, i32(0, 1), i32(0)), lambda: mv.kv4_read(cache, i32(0), i32(0), torch.float16),
           lambda: mv.kv4_evict(cache, cache.new_mass(), i32(20), 4, 5), lambda: mv.kv4_evict(cache, cache.new_mass()[:, :, :4], i32(20), 4, 1),
           lambda: mv.kv4_weigh(cache, q, i32(0, 1), i32(19), 1, torch.zeros(4, device="cuda"), cache.new_mass())]
    for f in bad:
        with pytest.raises(mv.MoEError):
            f()
    empty = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert mv.kv4_append(cache, empty, empty, none, none) is None
    out, lse = mv.kv4_attend(cache, torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"), i32(0, 0), i32(20), 1)
    assert out.shape == (0, 4, 64)


def test_workspace_refusals(mv):
    rng = np.random.default_rng(41)
    pg, cache = make_cache(mv, rng, [20], 2, 64, 16)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    q_start, base = dev(np.array([0, 1], np.int32)), dev(np.array([19], np.int32))
    need = mv.kv4_attend_workspace_bytes(cache, q, 1)
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(need, dtype=torch.float32, device="cuda"),
               torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2], torch.empty(need - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 256, dtype=torch.uint8, device="cuda")[1:]):
        with pytest.raises(mv.MoEError):
            mv.kv4_attend(cache, q, q_start, base, 1, workspace=ws)
    mv.kv4_attend(cache, q, q_start, base, 1, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
