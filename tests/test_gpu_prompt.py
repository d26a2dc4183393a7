"""A prompt's pass through a layer (rotary positions, causal attention of packed prompts, products grouped by expert) against
plain implementations in 64 bits.

Tolerances count roundings: one to bf16 is off by at most 2^-8 of the value, one to fp32 by 2^-24; a sum of n products in
fp32, in whatever order and with products or partial sums cut off instead of rounded, by n * 2^-23 of the sum of the terms'
absolute values."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -23  # a rounding to bf16; a step of an fp32 sum


@pytest.fixture(scope="module")
def mv():
    import __graft_entry__ as g
    g.build()
    import serving_router_softmax_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def within(got, want, tol, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol) & ~(got.isnan() & want.isnan()) & ~(got == want)
    assert not bad.any(), (what, int(bad.sum()), ((got - want).abs() / tol).nan_to_num(0).max().item())


# ------------------------------------------------------------------ rotary positions
def rotate_exact(x, pos, freqs, axes, interleaved, inverse):
    """(rotated, |a| + |b| of each value's pair) in 64 bits; the angle in whole turns is taken off exactly."""
    n = len(freqs)
    y = x.double().clone()
    mag = y.abs()
    from fractions import Fraction
    whole = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)  # 2 pi
    for i, (f, ax) in enumerate(zip(freqs, axes)):
        turn = Fraction(float(f)) / whole
        part = [float((turn * int(p)) % 1) for p in pos[ax].tolist()]
        ang = 2 * math.pi * torch.tensor(part, dtype=torch.float64, device=x.device)[:, None] * (-1 if inverse else 1)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        xa, xb = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = xa * ang.cos() - xb * ang.sin(), xa * ang.sin() + xb * ang.cos()
        mag[..., a] = mag[..., b] = xa.abs() + xb.abs()
    return y, mag


def rotate_tol(want, mag, dtype):
    # cosine and sine within 2^-22, a product and a sum rounded, the result rounded to its type
    return mag * (2.0 ** -22 + 3 * 2.0 ** -24) + (BF if dtype is torch.bfloat16 else 2.0 ** -24) * want.abs()


ROTATE = [(1, 1, 0, 64, 64, 1), (28, 64, 4, 128, 128, 1), (333, 5, 1, 128, 112, 3), (7, 3, 2, 64, 32, 4), (1025, 14, 2, 256, 256, 2),
          (3, 1, 1, 24, 16, 1), (2, 130, 7, 512, 512, 3)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R,A", ROTATE)
def test_rotate(mv, T, Hq, Hk, D, R, A, interleaved, dtype):
    g = gen(T + D)
    x = randn(g, T, Hq + Hk + 1, D, dtype=dtype)  # slices of one projection's output
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk] if Hk else None
    freqs = [10000.0 ** (-i / (R // 2)) for i in range(R // 2)]
    axes = [(i * 7) % A for i in range(R // 2)]
    axes[0] = A - 1
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (A, T), generator=g, device="cuda").to(torch.int32)
    pos[0, : T // 2] %= 1000
    rot = mv.Rotary(freqs, D, axes, interleaved)
    for inverse in (False, True):
        err = mv.new_dev_err()
        before = x.clone()
        oq, ok = mv.rotate(rot, q, k, pos, inverse=inverse, dev_err=err)
        assert err.item() == 0 and torch.equal(x, before) and (ok is None) == (Hk == 0)
        for got, a in ((oq, q), (ok, k)):
            if a is not None:
                want, mag = rotate_exact(a, pos, freqs, axes, interleaved, inverse)
                within(got, want, rotate_tol(want, mag, dtype))
                assert torch.equal(got[..., R:], a[..., R:])
    # in place, one axis of positions as [T], the same result
    y = x.clone()
    mv.rotate(rot, y[:, :Hq], y[:, Hq:Hq + Hk] if Hk else None, pos if A > 1 else pos[0], inverse=True, out_q=y[:, :Hq],
              out_k=y[:, Hq:Hq + Hk] if Hk else None)
    assert torch.equal(y[:, :Hq], oq) and torch.equal(y[:, Hq + Hk:], x[:, Hq + Hk:])


def test_rotate_back_is_the_gradient(mv):
    """The inverse of the rotation undoes it, and is the gradient: (R u) . w = u . (R^-1 w), against differences too."""
    g = gen(3)
    rot = mv.Rotary.standard(64, sections=[8, 12, 12])
    u, w = randn(g, 17, 6, 64, dtype=torch.float32), randn(g, 17, 6, 64, dtype=torch.float32)
    pos = torch.randint(0, 5000, (3, 17), generator=g, device="cuda").to(torch.int32)
    ru, back = mv.rotate(rot, u, None, pos)[0], mv.rotate(rot, w, None, pos, inverse=True)[0]
    within(mv.rotate(rot, ru, None, pos, inverse=True)[0], u.double(), 2.0 ** -19 * (1 + u.double().abs().amax()))
    # each side carries at most 2^-21 (|a| + |b|) a value
    assert abs((ru.double() * w).sum() - (u.double() * back).sum()).item() < 2.0 ** -19 * (u.abs().sum() * w.abs().amax()).item()
    d = torch.zeros_like(u)
    d[5, 2, 11] = 1.0  # linear: a difference of any size is the derivative
    diff = (mv.rotate(rot, u + d, None, pos)[0].double() - ru.double()).mul(w).sum()
    assert abs(diff.item() - back[5, 2, 11].item()) < 2.0 ** -18 * w.abs().amax().item() * u.abs().amax().item()


def test_rotate_far_positions_repeat(mv):
    """A frequency of a whole part of a turn: positions a period apart turn alike, to the last bit, 2^31 positions on."""
    rot = mv.Rotary([2 * math.pi / 64] * 8, 16)
    x = randn(gen(5), 4, 2, 16, dtype=torch.float32)
    pos = torch.tensor([5, 5 + 64, 5 + (1 << 20), (1 << 31) - 64 + 5], dtype=torch.int32, device="cuda")
    x[:] = x[:1]
    y = mv.rotate(rot, x, None, pos)[0]
    # 2 pi as a double is 2^-53 of it off: 2^31 positions make that 2^-28 of a turn
    within(y, y[:1].double().expand_as(y), 2.0 ** -21 * (x.abs().amax().double() * 4))


def test_rotate_bad_axis_is_reported(mv):
    rot = mv.Rotary.standard(32, sections=[8, 8])
    rot._axis[3] = 9
    x = randn(gen(6), 5, 2, 32)
    pos = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    err = mv.new_dev_err()
    y = mv.rotate(rot, x, None, pos, dev_err=err)[0]
    assert err.item() == mv._lib.DEV_BAD_ID
    assert torch.equal(y[..., 3], x[..., 3]) and torch.equal(y[..., 19], x[..., 19])


def test_rotate_nothing(mv):
    rot = mv.Rotary.standard(64)
    x = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert mv.rotate(rot, x, None, torch.empty(0, dtype=torch.int32, device="cuda"))[0].shape == (0, 4, 64)


# ------------------------------------------------------------------ attention of packed prompts
def attend_exact(q, k, v, start, scale):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits; rows of no sequence are left out of all (zero)."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda"), torch.zeros((T, Hq), dtype=torch.float64, device="cuda")
    ot, lt = torch.zeros_like(out), torch.zeros_like(lse)
    qd, kd, vd = q.double(), k.double(), v.double()
    for b, e in zip(start, start[1:]):
        for i0 in range(b, e, 512):
            i1 = min(i0 + 512, e)
            for h in range(Hq):
                kk, vv, qq = kd[b:i1, h // G], vd[b:i1, h // G], qd[i0:i1, h]
                later = torch.arange(b, i1, device="cuda") > torch.arange(i0, i1, device="cuda")[:, None]
                s = (qq @ kk.t() * scale).masked_fill(later, -math.inf)
                z = torch.logsumexp(s, 1)
                p = (s - z[:, None]).exp()
                # a score: D products summed, times the scale, minus the reference, in an exponential good to 2^-21
                ds = ((qq.abs() @ kk.abs().t()) * abs(scale) * D * F32 + (s.abs() + z.abs()[:, None]) * 4 * F32).masked_fill(later, 0).amax(1)
                n = i1 - b
                o = p @ torch.where(vv.isfinite(), vv, 0.0)
                mag = p @ vv.abs().nan_to_num(0, 0)
                out[i0:i1, h], lse[i0:i1, h] = o, z
                lt[i0:i1, h] = ds + n * F32 + z.abs() * 2 * F32 + 2.0 ** -20
                # probabilities rounded to bf16, sums over the keys, the quotient, the result rounded
                ot[i0:i1, h] = mag * (BF + n * F32 + 2 * ds + n * F32 + 2.0 ** -19)[:, None] + BF * o.abs()
    return out, lse, ot, lt


def attend_check(mv, q, k, v, lengths, scale, first=0):
    start = [first]
    for n in lengths:
        start.append(start[-1] + n)
    err = mv.new_dev_err()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    mv.prompt_attend(q, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), scale=scale, out=out, lse=lse, dev_err=err)
    assert err.item() == 0
    want, z, ot, lt = attend_exact(q, k, v, start, scale)
    a, b = start[0], start[-1]
    assert (out[:a] == 7).all() and (out[b:] == 7).all() and (lse[:a] == 7).all() and (lse[b:] == 7).all()
    within(lse[a:b], z[a:b], lt[a:b], "lse")
    within(out[a:b], want[a:b], ot[a:b], "out")
    return out, lse


ATTEND = [
    (4, 2, 64, [1]), (1, 1, 128, [1]), (8, 8, 128, [2, 1, 0, 3]), (32, 8, 128, [77]), (14, 2, 64, [129, 128, 127, 1, 0, 300]),
    (16, 1, 128, [16, 17, 513]), (3, 1, 64, [1000]), (5, 1, 128, [200, 41, 42, 43]), (128, 1, 64, [9]), (100, 1, 128, [5, 130]),
    (1, 1, 64, [1537]), (6, 2, 128, [255, 256, 257, 511]), (64, 4, 128, [70, 600]), (2, 1, 128, [2500]),
]


@pytest.mark.parametrize("Hq,Hkv,D,lengths", ATTEND)
def test_prompt_attend(mv, Hq, Hkv, D, lengths):
    g = gen(Hq * 1000 + sum(lengths))
    T = sum(lengths) + 5
    qkv = randn(g, T, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    attend_check(mv, q, k, v, lengths, D ** -0.5, first=2)
    # a scale of 0 (every key alike), then other strides: heads outermost, and a scale of the other sign
    attend_check(mv, q, k, v, lengths, 0.0)
    ho = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    attend_check(mv, *ho, lengths, -0.3 * D ** -0.5)


def test_prompt_attend_many_sequences(mv):
    g = gen(8)
    lengths = [(i * 37) % 41 for i in range(700)]
    T = sum(lengths)
    attend_check(mv, randn(g, T, 4, 64), randn(g, T, 2, 64), randn(g, T, 2, 64), lengths, 0.125)


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_attend_growing_scores(mv, D):
    """Scores that grow along the keys, by far more than one reference of the exponentials covers, and fall again."""
    g = gen(9)
    T = 900
    q, k, v = randn(g, T, 4, D), randn(g, T, 1, D), randn(g, T, 1, D)
    q[..., 0] = 8.0
    k[..., 0] = (torch.arange(T, device="cuda") % 500 * 0.25 * (D / 64) ** 0.5).to(torch.bfloat16)[:, None]
    attend_check(mv, q, k, v, [T], D ** -0.5)
    attend_check(mv, -q, k, v, [T], D ** -0.5)


def test_prompt_attend_not_finite(mv):
    """What a row does not see (later tokens, other sequences, rows of no sequence) has no effect, whatever it holds."""
    g = gen(10)
    T, D = 700, 128
    for Hq, Hkv in ((8, 1), (2, 2)):
        q, k, v = randn(g, T, Hq, D), randn(g, T, Hkv, D), randn(g, T, Hkv, D)
        lengths, start = [300, 250], [20, 320, 570]
        st = torch.tensor(start, dtype=torch.int32, device="cuda")
        want, wl = mv.prompt_attend(q, k, v, st)
        bad = [float("nan"), float("inf"), -float("inf")]
        k2, v2, q2 = k.clone(), v.clone(), q.clone()
        for x in (q2, k2, v2):
            x[:20], x[570:] = float("nan"), float("inf")
        at = {60: 0, 170: 1, 299 + 20: 2, 330: 0, 560: 1}  # rows of sequences whose values or keys are not finite
        for t, b in at.items():
            v2[t, 0, 5] = bad[b]
        o, l = mv.prompt_attend(q2, k2, v2, st)
        assert torch.equal(l[20:570], wl[20:570])
        first = torch.full((T,), T, device="cuda")
        first[20:320], first[320:570] = 60, 330
        sees = (torch.arange(T, device="cuda") >= first)
        G = Hq // Hkv
        hit = torch.zeros((T, Hq, D), dtype=torch.bool, device="cuda")
        hit[:, :G, 5] = sees[:, None]
        inside = torch.zeros(T, dtype=torch.bool, device="cuda")
        inside[20:570] = True
        assert torch.equal(o[inside][~hit[inside]], want[inside][~hit[inside]])
        assert not o[inside][hit[inside]].isfinite().any()
        k3 = k2.clone()
        k3[400, 0, 3] = float("nan")
        o, l = mv.prompt_attend(q2, k3, v, st)
        rows = (torch.arange(T, device="cuda") >= 400) & (torch.arange(T, device="cuda") < 570)
        assert l[rows][:, :G].isnan().all() and o[rows][:, :G].isnan().all()
        assert torch.equal(l[20:400], wl[20:400]) and torch.equal(o[20:400], want[20:400])
        q2[100, 0, 0] = float("nan")
        o, l = mv.prompt_attend(q2, k, v, st)
        assert l[100, 0].isnan() and o[100, 0].isnan().all()
        l[100, 0], o[100, 0] = wl[100, 0], want[100, 0]
        assert torch.equal(l[20:570], wl[20:570]) and torch.equal(o[20:570], want[20:570])


def test_prompt_attend_scores_of_minus_infinity(mv):
    """Keys that score -inf count as not seen; a row without any other gives zeros and -inf."""
    g = gen(11)
    T, D = 300, 64
    q, k, v = randn(g, T, 2, D).abs(), randn(g, T, 1, D), randn(g, T, 1, D)
    q[..., 1:] = 0.0
    q[..., 0] = 1.0
    k[:200, 0, 0] = -float("inf")
    k[:200, 0, 1:] = 0.0
    out, lse = mv.prompt_attend(q, k, v, torch.tensor([0, T], dtype=torch.int32, device="cuda"), scale=1.0)
    # 0 * 0 and -inf * 1 only: the products of the rest are not NaN
    assert (out[:200] == 0).all() and (lse[:200] == -math.inf).all()
    want, z, ot, lt = attend_exact(q[200:], k[200:], v[200:], [0, 100], 1.0)
    within(lse[200:], z, lt)
    within(out[200:], want, ot)


def test_prompt_attend_bad_starts(mv):
    g = gen(12)
    T = 400
    q, k, v = randn(g, T, 4, 64), randn(g, T, 2, 64), randn(g, T, 2, 64)
    st = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
    mv.prompt_attend(q, k, v, st)
    for bad in ([0, 100, 90, 300], [0, 100, 100, 401], [-1, 100, 100, 300], [0, 100, 2000000000, 300]):
        err = mv.new_dev_err()
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        mv.prompt_attend(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out, dev_err=err)
        assert err.item() == mv._lib.DEV_CAPACITY, bad
        assert (out == 7).all()


def test_prompt_attend_nothing(mv):
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = mv.prompt_attend(e, e, e, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    x = randn(gen(1), 5, 4, 64)
    out = torch.full_like(x, 7.0)
    mv.prompt_attend(x, x, x, torch.zeros(1, dtype=torch.int32, device="cuda"), out=out)
    mv.prompt_attend(x, x, x, torch.tensor([2, 2, 2], dtype=torch.int32, device="cuda"), out=out)
    assert (out == 7).all()


def test_prompt_attend_agrees_with_the_cache(mv):
    """The same prompt through the 4-bit cache, from the values the cache holds."""
    g = gen(13)
    T, Hq, Hkv, D = 500, 8, 2, 128
    q, k, v = randn(g, T, Hq, D), randn(g, T, Hkv, D), randn(g, T, Hkv, D)
    cache = mv.Kv4Cache.new(10, Hkv, 64, D, 1, 8)
    cache.table[0] = torch.arange(8, dtype=torch.int32, device="cuda")
    i = torch.arange(T, dtype=torch.int32, device="cuda")
    kh, vh = mv.kv4_append(cache, k, v, torch.zeros_like(i), i, held=True)
    st = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out, lse = mv.prompt_attend(q, kh, vh, st)
    want, z, ot, lt = attend_exact(q, kh, vh, [0, T], D ** -0.5)
    within(lse, z, lt)
    within(out, want, ot)
    o4, l4 = mv.kv4_attend(cache, q, st, torch.zeros(1, dtype=torch.int32, device="cuda"), T)
    # the held values are rounded to bf16 for the one and not for the other: 2^-8 of each key and value
    ds = 2 * BF * (q.double().abs().amax(2) * kh.double().abs().sum(2).amax() * D ** -0.5)
    assert ((l4.double() - z).abs() <= lt + ds).all()


# ------------------------------------------------------------------ products grouped by expert
def make_layer(mv, g, H, I, E, tiled):
    w = randn(g, E, 2 * I, H, std=H ** -0.5), randn(g, E, H, I, std=I ** -0.5)
    layer = mv.ExpertLayer(w[0], w[1], "bf16")
    return w, (mv.pack_tiled(layer) if tiled else layer)


def make_ids(g, T, E, k, skew, empty=()):
    score = torch.randn((T, E), generator=g, device="cuda") - skew * torch.arange(E, device="cuda")
    score[:, list(empty)] = -1e9
    return score.topk(k, 1)[1].to(torch.int32)


def gate_up_exact(x, w, ids, inv):
    T, k = ids.shape
    I = w.shape[1] // 2
    h, tol = (torch.zeros((T * k, I), dtype=torch.float64, device="cuda") for _ in range(2))
    place = inv.long().view(T, k)
    H = x.shape[1]
    for e in range(w.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        xd, wd = x[t].double(), w[e].double()
        z, m = xd @ wd.t(), (xd.abs() @ wd.abs().t()) * H * F32
        a, u, da, du = z[:, :I], z[:, I:], m[:, :I], m[:, I:]
        s = a * torch.sigmoid(a)
        h[place[t, j]] = s * u
        # silu's slope is at most 1.1; exponential and quotient within 2^-19
        tol[place[t, j]] = 1.1 * da * (u.abs() + du) + s.abs() * du + (BF + 2.0 ** -19) * (s * u).abs()
    return h, tol


def down_exact(h, w, ids, inv, p):
    T, k = ids.shape
    y, tol = (torch.zeros((T, w.shape[1]), dtype=torch.float64, device="cuda") for _ in range(2))
    place = inv.long().view(T, k)
    I = h.shape[1]
    for e in range(w.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        hd, wd, f = h[place[t, j]].double(), w[e].double(), p[t, j].double()[:, None]
        o, m = hd @ wd.t(), (hd.abs() @ wd.abs().t()) * I * F32
        y[t] += f * o
        # the product rounded to bf16, k terms summed
        tol[t] += f.abs() * (m + (o.abs() + m) * (BF + k * F32))
    return y, tol + BF * (y.abs() + tol)


GROUP = [  # T, H, I, E, k, skew, experts without tokens
    (1, 64, 64, 1, 1, 0.0, ()), (5, 256, 512, 16, 2, 0.0, (0, 15)), (37, 128, 192, 8, 2, 0.5, (3,)), (300, 320, 448, 12, 3, 1.0, ()),
    (700, 128, 64, 4, 4, 0.0, ()), (513, 64, 320, 3, 1, 3.0, ()), (64, 2880, 192, 5, 2, 0.0, ()), (260, 192, 2880, 2, 1, 0.0, ()),
    (33, 1024, 1536, 40, 6, 0.1, (7, 8)), (1100, 512, 128, 6, 2, 0.2, (2,)),
]


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("T,H,I,E,k,skew,empty", GROUP)
def test_group_products(mv, T, H, I, E, k, skew, empty, tiled):
    g = gen(T + H + I)
    (wg, wd), layer = make_layer(mv, g, H, I, E, tiled)
    x, ids = randn(g, T, H), make_ids(g, T, E, k, skew, empty)
    err = mv.new_dev_err()
    u = mv.union_permute(ids, E, dev_err=err)
    h = torch.full((T * k, I), 7.0, dtype=torch.bfloat16, device="cuda")
    mv.group_gate_up(x, layer, u, k, out=h, dev_err=err)
    assert err.item() == 0
    want, tol = gate_up_exact(x, wg, ids, u["inv"])
    within(h, want, tol, "gate_up")
    p = torch.rand((T, k), generator=g, device="cuda") - 0.2
    y = mv.group_down(h, layer, u, p, dev_err=err)
    assert err.item() == 0
    want, tol = down_exact(h, wd, ids, u["inv"], p)
    within(y, want, tol, "down")


def test_group_products_agree_with_the_verify_call(mv):
    g = gen(21)
    T, H, I, E, k = 29, 256, 384, 16, 4
    _, layer = make_layer(mv, g, H, I, E, True)
    x, ids = randn(g, T, H), make_ids(g, T, E, k, 0.1)
    p = torch.rand((T, k), generator=g, device="cuda")
    u = mv.union_permute(ids, E)
    want = mv.verify_ffn(x, k, layer, u, p).double()
    got = mv.group_down(mv.group_gate_up(x, layer, u, k), layer, u, p).double()
    # both round h to bf16; the products and their sum are rounded here only: three times 2^-8 of a row's largest value
    assert ((got - want).abs().amax(1) <= 3 * BF * k * want.abs().amax(1)).all()


def test_group_products_of_a_pool(mv):
    """Experts in pool slots, in another order than their ids."""
    g = gen(22)
    T, H, I, E, k = 90, 128, 192, 6, 2
    for tiled in (False, True):
        _, layer = make_layer(mv, g, H, I, E, tiled)
        host = mv.HostExperts([layer])
        pool = mv.ExpertPool(host, [[1, 4]], n_stage=6)
        x, ids = randn(g, T, H), make_ids(g, T, E, k, 0.0)
        p = torch.rand((T, k), generator=g, device="cuda")
        u = mv.union_permute(ids, E)
        mv.stage_experts(pool.layers[0], u)
        err = mv.new_dev_err()
        h = mv.group_gate_up(x, pool.layers[0], u, k, dev_err=err)
        assert torch.equal(h, mv.group_gate_up(x, layer, u, k))
        assert torch.equal(mv.group_down(h, pool.layers[0], u, p, dev_err=err), mv.group_down(h, layer, u, p))
        assert err.item() == 0


def test_group_products_not_finite(mv):
    """A token or an expert that is not finite touches its own rows alone."""
    g = gen(23)
    T, H, I, E, k = 400, 128, 128, 3, 1
    (wg, wd), layer = make_layer(mv, g, H, I, E, False)
    x, ids = randn(g, T, H), make_ids(g, T, E, k, 0.0)
    p = torch.ones((T, k), device="cuda")
    u = mv.union_permute(ids, E)
    want = mv.group_gate_up(x, layer, u, k)
    wy = mv.group_down(want, layer, u, p)
    x2 = x.clone()
    x2[77], x2[130, 5] = float("nan"), float("inf")
    h = mv.group_gate_up(x2, layer, u, k)
    rows = u["inv"][[77, 130]].long()
    keep = torch.ones(T * k, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(h[keep], want[keep]) and h[rows[0]].isnan().all() and not h[rows[1]].isfinite().all()
    y = mv.group_down(torch.where(keep[:, None], want, float("nan")), layer, u, p)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[77, 130]] = False
    assert torch.equal(y[keep], wy[keep]) and y[[77, 130]].isnan().all()
    wg[1] = float("nan")
    h = mv.group_gate_up(x, layer, u, k)
    mine = (ids[u["perm_token"].long(), 0] == 1)
    assert h[mine].isnan().all() and torch.equal(h[~mine], want[~mine])


def test_group_products_bad_unions(mv):
    g = gen(24)
    T, H, I, E, k = 50, 64, 128, 8, 2
    _, layer = make_layer(mv, g, H, I, E, False)
    x, ids = randn(g, T, H), make_ids(g, T, E, k, 0.0)
    p = torch.rand((T, k), generator=g, device="cuda")
    good = mv.union_permute(ids, E)
    want = mv.group_gate_up(x, layer, good, k)
    wy = mv.group_down(want, layer, good, p)

    def change(name, at, value):
        u = {n: t.clone() for n, t in good.items()}
        u[name][at] = value
        return u

    off = good["offsets"].tolist()
    for u, bit, group in ((change("n_unique", 0, E + 1), mv._lib.DEV_CAPACITY, None), (change("n_unique", 0, -3), mv._lib.DEV_CAPACITY, None),
                          (change("unique", 2, E), mv._lib.DEV_BAD_ID, 2), (change("unique", 2, -1), mv._lib.DEV_BAD_ID, 2),
                          (change("offsets", E, T * k + 1), mv._lib.DEV_BAD_ID, E - 1), (change("offsets", 0, -5), mv._lib.DEV_BAD_ID, 0),
                          (change("offsets", 1, 1 << 30), mv._lib.DEV_BAD_ID, 0)):
        err = mv.new_dev_err()
        h = torch.full_like(want, 7.0)
        mv.group_gate_up(x, layer, u, k, out=h, dev_err=err)
        assert err.item() == bit
        if group is None:
            assert (h == 7).all()
            err.zero_()
            assert (mv.group_down(want, layer, u, p, dev_err=err) == 0).all() and err.item() == bit
        else:
            a, b = off[group], off[group + 1]
            assert (h[a:b] == 7).all()
            if u["offsets"].tolist() == off:
                assert torch.equal(h[:a], want[:a]) and torch.equal(h[b:], want[b:])
    err = mv.new_dev_err()
    u = change("perm_token", 7, T)
    h = mv.group_gate_up(x, layer, u, k, dev_err=err)
    assert err.item() == mv._lib.DEV_BAD_ID and torch.equal(h[:7], want[:7]) and torch.equal(h[8:], want[8:])
    err.zero_()
    u = change("inv", 2 * 11 + 1, T * k)
    y = mv.group_down(want, layer, u, p, dev_err=err)
    keep = torch.arange(T, device="cuda") != 11
    assert err.item() == mv._lib.DEV_BAD_ID and torch.equal(y[keep], wy[keep])
    # none of the experts: zeros
    err.zero_()
    assert (mv.group_down(want, layer, change("n_unique", 0, 0), p, dev_err=err) == 0).all() and err.item() == 0


def test_group_nothing(mv):
    _, layer = make_layer(mv, gen(25), 64, 64, 2, False)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    u = mv.union_permute(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 2)
    h = mv.group_gate_up(x, layer, u, 2)
    assert h.shape == (0, 64)
    assert mv.group_down(h, layer, u, torch.empty((0, 2), device="cuda")).shape == (0, 64)


# ------------------------------------------------------------------ together, as they are used
class Prompt:
    """A layer's pass over packed prompts: rotation, attention, the cache, routing, experts."""

    def __init__(self, mv, seed, lengths, Hq=8, Hkv=2, D=64, H=256, I=192, E=8, k=2):
        g = gen(seed)
        self.mv, self.k, self.E = mv, k, E
        T = sum(lengths)
        self.rot = mv.Rotary.standard(D, sections=[8, 12, 12])
        self.x, self.qkv = randn(g, T, H), randn(g, T, Hq + 2 * Hkv, D)
        self.Hq, self.Hkv = Hq, Hkv
        self.pos = torch.randint(0, 4000, (3, T), generator=g, device="cuda").to(torch.int32)
        self.seq = torch.cat([torch.full((n,), s, dtype=torch.int32) for s, n in enumerate(lengths)]).cuda()
        self.slot = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths]).cuda()
        start = [0]
        for n in lengths:
            start.append(start[-1] + n)
        self.start = torch.tensor(start, dtype=torch.int32, device="cuda")
        width = max(-(-n // 32) for n in lengths) + 1
        self.cache = mv.Kv4Cache.new(len(lengths) * width, Hkv, 32, D, len(lengths), width)
        self.cache.table.copy_(torch.arange(len(lengths) * width, dtype=torch.int32).view(len(lengths), width))
        self.weights, self.layer = make_layer(mv, g, H, I, E, True)
        self.gate = randn(g, E, H, std=0.1)

    def run(self):
        mv, Hq, Hkv = self.mv, self.Hq, self.Hkv
        q, k = mv.rotate(self.rot, self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.pos)
        v = self.qkv[:, Hq + Hkv:]
        out, lse = mv.prompt_attend(q, k, v, self.start)
        mv.kv4_append(self.cache, k, v, self.seq, self.slot)
        ids, w = mv.route(mv.router_logits(self.x, self.gate), self.k)
        u = mv.union_permute(ids, self.E)
        y = mv.group_down(mv.group_gate_up(self.x, self.layer, u, self.k), self.layer, u, w)
        return q, k, out, lse, ids, w, y


def test_a_prompts_pass(mv):
    lengths = [150, 1, 64, 333]
    pr = Prompt(mv, 31, lengths)
    q, k, out, lse, ids, w, y = pr.run()
    for got, x in ((q, pr.qkv[:, :8]), (k, pr.qkv[:, 8:10])):
        want, mag = rotate_exact(x, pr.pos, [10000.0 ** (-i / 32) for i in range(32)], [0] * 8 + [1] * 12 + [2] * 12, False, False)
        within(got, want, rotate_tol(want, mag, torch.bfloat16))
    o, z, ot, lt = attend_exact(q, k, pr.qkv[:, 10:], pr.start.tolist(), 64 ** -0.5)
    within(out, o, ot)
    within(lse, z, lt)
    u = mv.union_permute(ids, 8)
    h, ht = gate_up_exact(pr.x, pr.weights[0], ids, u["inv"])
    got = mv.group_gate_up(pr.x, pr.layer, u, 2)
    within(got, h, ht)
    want, tol = down_exact(got, pr.weights[1], ids, u["inv"], w)
    within(y, want, tol)
    # the next verify step attends over what was written
    base = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    qn, kn = mv.rotate(pr.rot, q[:4], k[:4], pr.pos[:, :4].contiguous())
    mv.kv4_append(pr.cache, kn, pr.qkv[:4, 10:], torch.arange(4, dtype=torch.int32, device="cuda"), base)
    o2, l2 = mv.kv4_attend(pr.cache, qn, torch.arange(5, dtype=torch.int32, device="cuda"), base, 1)
    assert o2.isfinite().all() and l2.isfinite().all()


def test_captured_and_replayed(mv):
    """Two graphs of the pass, replayed beside each other on two streams and beside eager calls: the same results."""
    prs = [Prompt(mv, 41, [200, 40]), Prompt(mv, 42, [33, 300, 1])]
    wants = [pr.run() for pr in prs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in prs]
    for pr in prs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(pr.run())
        graphs.append(gr)
    for _ in range(3):
        for t in [t for o in outs for t in o]:
            t.zero_()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        eager = prs[0].run()
        torch.cuda.synchronize()
        for got, want in list(zip(outs, wants)) + [(eager, wants[0])]:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    # new inputs in the same memory
    prs[0].qkv.mul_(0.5)
    prs[0].x.neg_()
    want = prs[0].run()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want))


def test_other_streams_and_repeats(mv):
    """A call's `stream` argument, and the same bits from every repeat."""
    pr = Prompt(mv, 51, [700, 130, 9], Hq=14, Hkv=2, D=128 // 2)
    want = pr.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q, k = mv.rotate(pr.rot, pr.qkv[:, :14], pr.qkv[:, 14:16], pr.pos, stream=s)
    out, lse = mv.prompt_attend(q, k, pr.qkv[:, 16:], pr.start, stream=s)
    u = mv.union_permute(want[4], pr.E, stream=s)
    y = mv.group_down(mv.group_gate_up(pr.x, pr.layer, u, 2, stream=s), pr.layer, u, want[5], stream=s)
    s.synchronize()
    for a, b in zip((q, k, out, lse, y), want[:4] + want[6:]):
        assert torch.equal(a, b)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(pr.run(), want))


@pytest.mark.parametrize("Hq,Hkv,D", [(64, 4, 128), (14, 2, 64), (8, 8, 128)])
def test_prompt_attend_many_items(mv, Hq, Hkv, D):
    """More blocks than CTAs, of one step and of several, again and again: no wait runs out, the same bits every time."""
    g = gen(14)
    lengths = [300, 20, 1, 700, 16, 16, 129, 0, 60] * 14
    T = sum(lengths)
    q, k, v = randn(g, T, Hq, D), randn(g, T, Hkv, D), randn(g, T, Hkv, D)
    start = [0]
    for n in lengths:
        start.append(start[-1] + n)
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    err = mv.new_dev_err()
    out, lse = mv.prompt_attend(q, k, v, st, dev_err=err)
    want, z, ot, lt = attend_exact(q[:2484], k[:2484], v[:2484], start[:19], D ** -0.5)
    within(lse[:2484], z, lt)
    within(out[:2484], want, ot)
    for _ in range(40):
        o, l = mv.prompt_attend(q, k, v, st, dev_err=err)
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert err.item() == 0


def test_two_threads_at_once(mv):
    """Calls of several host threads, each on its own stream, beside each other."""
    import threading
    prs = [Prompt(mv, 60 + i, lengths) for i, lengths in enumerate(([400, 3], [64, 64, 250], [1, 1, 900]))]
    wants = [pr.run() for pr in prs]
    torch.cuda.synchronize()
    bad = []

    def work(pr, want):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(12):
                    got = pr.run()
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(prs, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


# ------------------------------------------------------------------ offsets past 32 bits
def test_far_apart_rows(mv):
    """Token strides that put rows billions of values apart."""
    g = gen(71)
    T, far = 4, (1 << 30) + 64
    near = randn(g, T, 4, 64)
    store = torch.empty(far * (T - 1) + 4 * 64, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((T, 4, 64), (far, 64, 1))
    x.copy_(near)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rot = mv.Rotary.standard(64)
    want = mv.rotate(rot, near[:, :2], near[:, 2:], pos)
    got = mv.rotate(rot, x[:, :2], x[:, 2:], pos, out_q=x[:, :2], out_k=x[:, 2:])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x.copy_(near)
    st = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    want = mv.prompt_attend(near[:, :2], near[:, 2:3], near[:, 3:], st)
    got = mv.prompt_attend(x[:, :2], x[:, 2:3], x[:, 3:], st)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_group_products_of_many_rows(mv):
    """As many rows as are taken: outputs of more than 2^31 values."""
    g = gen(72)
    T, H, I, E = 1 << 22, 64, 576, 3
    (wg, wd), layer = make_layer(mv, g, H, I, E, False)
    x = randn(g, T, H)
    ids = torch.randint(0, E, (T,), generator=g, device="cuda")
    order = torch.argsort(ids, stable=True).to(torch.int32)
    inv = torch.empty_like(order)
    inv[order.long()] = torch.arange(T, dtype=torch.int32, device="cuda")
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.bincount(ids, minlength=E).cumsum(0)]).to(torch.int32)
    u = {"n_unique": torch.tensor([E], dtype=torch.int32, device="cuda"), "unique": torch.arange(E, dtype=torch.int32, device="cuda"),
         "offsets": off, "perm_token": order, "inv": inv}
    err = mv.new_dev_err()
    h = mv.group_gate_up(x, layer, u, 1, dev_err=err)
    y = mv.group_down(h, layer, u, torch.ones((T, 1), device="cuda"), dev_err=err)
    assert err.item() == 0
    pick = torch.cat([torch.arange(500), torch.arange(T // 2, T // 2 + 500), torch.arange(T - 500, T)]).cuda()
    want, tol = gate_up_exact(x[pick], wg, ids[pick][:, None], torch.arange(len(pick), device="cuda"))
    within(h[inv[pick].long()], want, tol)
    want, tol = down_exact(h[inv[pick].long()], wd, ids[pick][:, None], torch.arange(len(pick), device="cuda"), torch.ones((len(pick), 1), device="cuda"))
    within(y[pick], want, tol)


def test_the_first_calls_of_a_process_are_captured(mv):
    """Nothing is looked up or raised by a first call that a capture does not allow."""
    import subprocess
    import sys
    code = """
import torch, serving_router_softmax_gb300 as mv
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
q, k, x = r(300, 8, 128), r(300, 2, 128), r(300, 128)
layer = mv.ExpertLayer(r(4, 256, 128), r(4, 128, 128), "bf16")
rot, pos = mv.Rotary.standard(128), torch.arange(300, dtype=torch.int32, device="cuda")
st = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
ids = torch.randint(0, 4, (300, 1), generator=g, device="cuda").to(torch.int32)
w = torch.ones((300, 1), device="cuda")
def run():
    a, b = mv.rotate(rot, q, k, pos)
    o, z = mv.prompt_attend(a, b, k, st)
    u = mv.union_permute(ids, 4)
    return o, z, mv.group_down(mv.group_gate_up(x, layer, u, 1), layer, u, w)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
want = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
"""
    import os
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]
