"""Pins of the 4-bit KV cache oracle (CPU): hand-worked entries, byte layout, masks, attention and eviction."""
import numpy as np
import pytest

from oracle import kv_cache as K


def test_quantise_by_hand():
    x = np.array([[0.0, 1.0, 15.0, 7.4, 7.6, 3.5, 4.5, 14.9]])
    code, scale, zero = K.quantise(x)
    assert scale.tolist() == [1.0] and zero.tolist() == [0.0]
    assert code.tolist() == [[0, 1, 15, 7, 8, 4, 4, 15]]  # halves go to the even code
    code, scale, zero = K.quantise(np.full((1, 8), 2.5))
    assert scale[0] == 0 and zero[0] == 2.5 and not code.any()
    code, scale, zero = K.quantise(np.array([[np.nan] + [1.0] * 7, [np.inf] + [1.0] * 7, [70000.0] + [1.0] * 7]))
    assert not scale.any() and np.isnan(zero).all() and not code.any()


def test_quantise_is_within_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 64)).astype(np.float32)
    code, scale, zero = K.quantise(x)
    got = zero[:, None] + scale[:, None] * code
    # half a step, the zero's and the scale's own rounding (fp16, half a unit: 2^-11)
    assert np.all(np.abs(got - x) <= scale[:, None] * (0.5 + 15 * 2.0 ** -11) + np.abs(zero[:, None]) * 2.0 ** -11)


def test_page_layout_by_hand():
    page, D = 16, 64
    raw = np.zeros((2, 1, page * (D + 8)), dtype=np.uint8)
    pg = K.Pages(raw, np.array([[1, 0]]), page, D)
    pg.write(0, 3, 0, np.arange(64, dtype=np.float64)[None] / 63 * 15)
    pg.write(0, 18, 1, -np.arange(64, dtype=np.float64)[None])
    codes = np.rint(np.arange(64) / 63 * 15).astype(int)
    row = raw[1, 0, 3 * 32:4 * 32]
    assert (row & 15).tolist() == codes[0::2].tolist() and (row >> 4).tolist() == codes[1::2].tolist()
    assert raw[1, 0, 16 * 64 + 3 * 8:][:4].view(np.float16).tolist() == [1.0, 0.0]
    assert raw[0, 0, 16 * 64 + 2 * 8 + 4:][:4].view(np.float16).tolist() == [np.float16(4.2), -63.0]
    code, s, z = pg.entries(0, 0, 19, 1)
    assert code[18, 0] == 15 and code[18, 63] == 0 and z[18] == -63


def test_masks():
    assert K.seen(2, 3).tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    assert K.seen(1, 2, np.array([1, 2])).tolist() == [[1, 1, 0], [1, 0, 1]]
    assert not K.seen(0, 1, np.array([0])).any()


def test_attend_by_hand():
    page, D = 16, 64
    raw = np.zeros((1, 1, page * (D + 8)), dtype=np.uint8)
    pg = K.Pages(raw, np.array([[0]]), page, D)
    k = np.zeros((2, D))
    k[1, 0] = 1.0
    v = np.stack([np.zeros(D), np.full(D, 3.0)])
    for j in range(2):
        pg.write(0, j, 0, k[j:j + 1])
        pg.write(0, j, 1, v[j:j + 1])
    q = np.zeros((1, 2, D))
    q[0, 0, 0] = np.log(3.0)
    s1 = float(np.float16(1 / 15)) * 15  # the held value of 1
    out, lse, mass, ot, lt, mt = K.attend(pg, q, [0, 1], [1], 1.0, lse_in=np.array([[np.log(1 + 3 ** s1), np.log(2.0)]]))
    assert out[0, 0, 5] == pytest.approx(3 * 3 ** s1 / (1 + 3 ** s1), rel=1e-12)
    assert out[0, 1, 5] == pytest.approx(1.5) and lse[0, 1] == pytest.approx(np.log(2.0))
    assert mass[0, 0].tolist() == pytest.approx([1 / (1 + 3 ** s1) + 0.5, 3 ** s1 / (1 + 3 ** s1) + 0.5])
    assert np.all(ot > 0) and np.all(lt > 0)


def test_evict_by_hand():
    m = np.array([5.0, 1.0, 1.0, 9.0, np.nan, 1.0, 0.0, 0.0], dtype=np.float32)
    assert K.evict(m, 8, 8, 2).tolist() == list(range(8))
    assert K.evict(m, 8, 5, 2).tolist() == [0, 1, 3, 6, 7]       # the tie of ones goes to the lower slot
    assert K.evict(m, 8, 2, 2).tolist() == [6, 7]
    assert K.evict(m, 8, 7, 0).tolist() == [0, 1, 2, 3, 5, 6, 7]  # the NaN goes first
    assert K.evict(-m, 4, 1, 0).tolist() == [1]
