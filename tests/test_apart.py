"""Whether strided rows share memory, as the calls' checks work it out, against sets of addresses (CPU)."""
import ctypes as C
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def apart(tmp_path_factory):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("apart")
    (d / "apart.cpp").write_text('#include "apart.cuh"\nextern "C" int rows_apart(const moe::Rows* a, const moe::Rows* b) '
                                 "{ return moe::rows_apart(*a, *b); }\n")
    subprocess.run([cc, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "serving_router_softmax_gb300", "csrc"),
                    "-o", str(d / "apart.so"), str(d / "apart.cpp")], check=True)
    fn = C.CDLL(str(d / "apart.so")).rows_apart

    def call(a, b):
        ra, rb = (C.c_longlong * 6)(*a), (C.c_longlong * 6)(*b)
        return bool(fn(ra, rb))
    return call


def addresses(at, T, token, H, head, width):
    return {at + t * token + h * head + x for t in range(T) for h in range(H) for x in range(width)}


def reach(at, T, token, H, head, width):
    return at, at + max(T - 1, 0) * token + max(H - 1, 0) * head + width


def test_random_rows(apart):
    r = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(60000):
        token = r.choice([0, 1, 2, 3, 6, 8, 12, 20, 24, 40])
        a = (r.randrange(100, 160), r.choice([1, 1, 2, 3, 5]), token, r.choice([1, 2, 3]), r.choice([0, 1, 2, 3, 4, 6, 8, 30, 60]), r.randrange(1, 6))
        b = (r.randrange(100, 160), r.choice([1, 1, 2, 3, 5]), token, r.choice([1, 2, 4]), r.choice([0, 1, 2, 3, 4, 6, 8, 30, 60]), r.randrange(1, 6))
        want = not (addresses(*a) & addresses(*b))
        assert apart(a, b) == apart(b, a) == want, (a, b)
        seen[want] += 1
    assert min(seen.values()) > 5000


def test_other_token_strides_need_other_ranges(apart):
    r = random.Random(2)
    for _ in range(20000):
        a = (r.randrange(100, 200), r.randrange(2, 5), r.randrange(1, 30), r.choice([1, 2]), r.randrange(1, 9), r.randrange(1, 6))
        b = (r.randrange(100, 200), r.randrange(2, 5), a[2] + r.randrange(1, 9), r.choice([1, 2]), r.randrange(1, 9), r.randrange(1, 6))
        (a0, a1), (b0, b1) = reach(*a), reach(*b)
        assert apart(a, b) == (a1 <= b0 or b1 <= a0)
        assert not (addresses(*a) & addresses(*b)) or not apart(a, b)


def test_layouts_of_a_projection(apart):
    """Queries, keys and values as slices of one buffer, in every order of tokens, heads and parts."""
    T, Hq, Hk, D = 1000, 48, 6, 256
    base, N = 1 << 30, Hq + 2 * Hk
    tokens_first = [(base + h * D, T, N * D, n, D, D) for h, n in ((0, Hq), (Hq, Hk), (Hq + Hk, Hk))]
    heads_first = [(base + h * T * D, T, D, n, T * D, D) for h, n in ((0, Hq), (Hq, Hk), (Hq + Hk, Hk))]
    by_head = [(base + i * D, T, 3 * Hq * D, Hq, 3 * D, D) for i in range(3)]
    heads_then_parts = [(base + i * T * D, T, D, Hq, 3 * T * D, D) for i in range(3)]
    for layout in (tokens_first, heads_first, by_head, heads_then_parts):
        for i, a in enumerate(layout):
            for j, b in enumerate(layout):
                assert apart(a, b) == (i != j)
            moved = (a[0] + 2, *a[1:])
            assert not apart(a, moved)
    # rows that interleave within one span and end before they would meet
    assert apart((base, 2, 1 << 40, 1, 0, 512), (base + 512, 2, 1 << 40, 1, 0, 512))
    assert not apart((base, 2, 1 << 40, 1, 0, 513), (base + 512, 2, 1 << 40, 1, 0, 512))
    assert apart((base, 0, 512, 4, 512, 512), (base, 9, 512, 4, 512, 512))
    # the largest sizes: past 32 bits
    T, wide = 1 << 24, 128 * 1024 * 2
    assert not apart((base, T, wide, 1, 0, wide), (base + (T - 1) * wide, 1, 0, 1, 0, 1))
    assert apart((base, T, wide, 1, 0, wide), (base + T * wide, 1, 0, 1, 0, 1))
