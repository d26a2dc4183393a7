"""Refusals and struct layouts of the kv4_* calls (CPU: every check comes before any CUDA call)."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

from serving_router_softmax_gb300 import _lib as L

FAKE = 1 << 20  # an aligned non-NULL placeholder: refused calls use no pointer
HDR = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_verify.h")


@pytest.fixture(scope="module")
def lib():
    return L.load()


def cache(**kw):
    f = dict(n_pages=8, page_size=64, n_kv_heads=2, head_dim=128, n_seq=2, max_pages=4, pages=FAKE, table=FAKE)
    f.update(kw)
    return L.Kv4CacheStruct(**f)


def rows(**kw):
    f = dict(T=3, dtype=L.DTYPE_BF16, k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128)
    f.update(kw)
    return L.Kv4RowsCfg(**f)


def attn(**kw):
    f = dict(T=3, n_q_heads=8, max_q=2, scale=0.1, q_token_stride=1024, q_head_stride=128)
    f.update(kw)
    return L.Kv4AttnCfg(**f)


BAD_CACHE = [(dict(n_pages=-1), L.MOE_ERR_ARG), (dict(n_seq=-1), L.MOE_ERR_ARG), (dict(max_pages=0), L.MOE_ERR_ARG),
             (dict(n_kv_heads=0), L.MOE_ERR_ARG), (dict(pages=None), L.MOE_ERR_ARG), (dict(table=None), L.MOE_ERR_ARG),
             (dict(pages=FAKE + 8), L.MOE_ERR_ARG), (dict(table=FAKE + 2), L.MOE_ERR_ARG),
             (dict(head_dim=96), L.MOE_ERR_UNSUPPORTED), (dict(head_dim=256), L.MOE_ERR_UNSUPPORTED),
             (dict(page_size=8), L.MOE_ERR_UNSUPPORTED), (dict(page_size=48), L.MOE_ERR_UNSUPPORTED),
             (dict(page_size=512), L.MOE_ERR_UNSUPPORTED), (dict(n_kv_heads=1025), L.MOE_ERR_UNSUPPORTED),
             (dict(n_seq=4097), L.MOE_ERR_UNSUPPORTED), (dict(max_pages=1 << 25), L.MOE_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_bad_caches_are_refused_by_every_call(lib, kw, want):
    c = C.byref(cache(**kw))
    r, a, e = C.byref(rows()), C.byref(attn()), C.byref(L.Kv4EvictCfg(4, 2))
    assert lib.kv4_append(c, FAKE, FAKE, r, FAKE, FAKE, None, None, None, None) == want
    assert lib.kv4_read(c, FAKE, FAKE, r, FAKE, FAKE, None, None) == want
    assert lib.kv4_attend_workspace(c, a) == 0
    assert lib.kv4_attend(c, FAKE, FAKE, FAKE, None, a, FAKE, FAKE, FAKE, 1 << 40, None, None) == want
    assert lib.kv4_weigh(c, FAKE, FAKE, FAKE, None, FAKE, a, FAKE, None, None) == want
    assert lib.kv4_evict(c, FAKE, FAKE, e, FAKE, FAKE, FAKE, None, None) == want


def test_null_structs(lib):
    c = C.byref(cache())
    assert lib.kv4_append(None, FAKE, FAKE, C.byref(rows()), FAKE, FAKE, None, None, None, None) == L.MOE_ERR_ARG
    assert lib.kv4_append(c, FAKE, FAKE, None, FAKE, FAKE, None, None, None, None) == L.MOE_ERR_ARG
    assert lib.kv4_attend(c, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, 1 << 40, None, None) == L.MOE_ERR_ARG
    assert lib.kv4_evict(c, FAKE, FAKE, None, FAKE, FAKE, FAKE, None, None) == L.MOE_ERR_ARG


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), L.MOE_ERR_ARG), (dict(dtype=L.DTYPE_E4M3_B128), L.MOE_ERR_UNSUPPORTED),
    (dict(T=1 << 30), L.MOE_ERR_UNSUPPORTED), (dict(k_token_stride=257), L.MOE_ERR_UNSUPPORTED),
    (dict(v_head_stride=4), L.MOE_ERR_UNSUPPORTED), (dict(k_head_stride=-128), L.MOE_ERR_UNSUPPORTED)])
def test_append_refuses_bad_rows(lib, kw, want):
    assert lib.kv4_append(C.byref(cache()), FAKE, FAKE, C.byref(rows(**kw)), FAKE, FAKE, None, None, None, None) == want


def test_append_and_read_refuse_bad_pointers(lib):
    c, r = C.byref(cache()), C.byref(rows())
    for bad in (None, FAKE + 2):
        assert lib.kv4_append(c, bad, FAKE, r, FAKE, FAKE, None, None, None, None) == L.MOE_ERR_ARG
        assert lib.kv4_append(c, FAKE, bad, r, FAKE, FAKE, None, None, None, None) == L.MOE_ERR_ARG
        assert lib.kv4_append(c, FAKE, FAKE, r, bad, FAKE, None, None, None, None) == L.MOE_ERR_ARG
        assert lib.kv4_append(c, FAKE, FAKE, r, FAKE, bad, None, None, None, None) == L.MOE_ERR_ARG
        assert lib.kv4_read(c, FAKE, FAKE, r, bad, FAKE, None, None) == L.MOE_ERR_ARG
        assert lib.kv4_read(c, bad, FAKE, r, FAKE, FAKE, None, None) == L.MOE_ERR_ARG
    assert lib.kv4_append(c, FAKE, FAKE, r, FAKE, FAKE, FAKE, None, None, None) == L.MOE_ERR_ARG  # one held output only
    assert lib.kv4_append(c, FAKE, FAKE, r, FAKE, FAKE, FAKE + 2, FAKE, None, None) == L.MOE_ERR_ARG
    z = C.byref(rows(T=0))  # nothing to do needs no pointers
    assert lib.kv4_append(c, None, None, z, None, None, None, None, None, None) == L.MOE_OK
    assert lib.kv4_read(c, None, None, z, None, None, None, None) == L.MOE_OK


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), L.MOE_ERR_ARG), (dict(n_q_heads=0), L.MOE_ERR_ARG), (dict(n_q_heads=7), L.MOE_ERR_ARG),
    (dict(max_q=0), L.MOE_ERR_ARG), (dict(scale=float("nan")), L.MOE_ERR_ARG), (dict(scale=float("inf")), L.MOE_ERR_ARG),
    (dict(n_q_heads=4098), L.MOE_ERR_UNSUPPORTED), (dict(q_token_stride=1020), L.MOE_ERR_UNSUPPORTED),
    (dict(q_head_stride=-128), L.MOE_ERR_UNSUPPORTED), (dict(T=1 << 28), L.MOE_ERR_UNSUPPORTED)])
def test_attention_refuses_bad_shapes(lib, kw, want):
    c, a = C.byref(cache()), C.byref(attn(**kw))
    assert lib.kv4_attend_workspace(c, a) == 0
    assert lib.kv4_attend(c, FAKE, FAKE, FAKE, None, a, FAKE, FAKE, FAKE, 1 << 40, None, None) == want
    assert lib.kv4_weigh(c, FAKE, FAKE, FAKE, None, FAKE, a, FAKE, None, None) == want


def test_strides_of_a_lone_token_or_head_are_not_looked_at(lib):
    c = C.byref(cache(n_kv_heads=1))
    assert lib.kv4_attend_workspace(c, C.byref(attn(T=1, q_token_stride=-3))) > 0
    assert lib.kv4_attend_workspace(c, C.byref(attn(n_q_heads=1, q_head_stride=7))) > 0
    assert lib.kv4_attend_workspace(c, C.byref(attn(T=2, q_token_stride=7))) == 0
    assert lib.kv4_attend_workspace(c, C.byref(attn(n_q_heads=2, q_head_stride=7))) == 0


def test_attention_refuses_bad_pointers_and_workspaces(lib):
    c, a = C.byref(cache()), C.byref(attn())
    need = lib.kv4_attend_workspace(c, a)
    assert need > 0
    ok = [FAKE, FAKE, FAKE, None, a, FAKE, FAKE, FAKE, need, None, None]
    for at, bad in ((0, None), (0, FAKE + 2), (1, None), (2, None), (2, FAKE + 2), (3, FAKE + 4), (5, None), (5, FAKE + 2), (6, FAKE + 2)):
        args = list(ok)
        args[at] = bad
        assert lib.kv4_attend(c, *args) == L.MOE_ERR_ARG, (at, bad)
    for ws, n in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        args = list(ok)
        args[7], args[8] = ws, n
        assert lib.kv4_attend(c, *args) == L.MOE_ERR_WORKSPACE
    ok = [FAKE, FAKE, FAKE, None, FAKE, a, FAKE, None, None]
    for at, bad in ((0, None), (0, FAKE + 2), (1, None), (2, None), (3, FAKE + 4), (4, None), (6, None), (6, FAKE + 2)):
        args = list(ok)
        args[at] = bad
        assert lib.kv4_weigh(c, *args) == L.MOE_ERR_ARG, (at, bad)
    z = C.byref(attn(T=0))
    assert lib.kv4_attend(c, None, None, None, None, z, None, None, None, 0, None, None) == L.MOE_OK
    assert lib.kv4_weigh(c, None, None, None, None, None, z, None, None, None) == L.MOE_OK


def test_a_cache_without_sequences_needs_no_table(lib):
    c = C.byref(cache(n_seq=0, table=None, n_pages=0, pages=None))
    assert lib.kv4_evict(c, None, None, C.byref(L.Kv4EvictCfg(4, 2)), None, None, None, None, None) == L.MOE_OK
    a = C.byref(attn(T=0))
    assert lib.kv4_attend_workspace(c, a) > 0
    assert lib.kv4_attend(c, None, None, None, None, a, None, None, None, 0, None, None) == L.MOE_OK
    assert lib.kv4_weigh(c, None, None, None, None, None, a, None, None, None) == L.MOE_OK
    assert lib.kv4_append(c, None, None, C.byref(rows(T=0)), None, None, None, None, None, None) == L.MOE_OK
    assert lib.kv4_read(c, None, None, C.byref(rows(T=0)), None, None, None, None) == L.MOE_OK


def test_evict_refusals(lib):
    c = C.byref(cache())
    for keep, recent in ((0, 0), (4, -1), (4, 5), (-1, 0)):
        assert lib.kv4_evict(c, FAKE, FAKE, C.byref(L.Kv4EvictCfg(keep, recent)), FAKE, FAKE, FAKE, None, None) == L.MOE_ERR_ARG
    e = C.byref(L.Kv4EvictCfg(4, 2))
    for at in (0, 1, 3, 4, 5):
        args = [FAKE, FAKE, e, FAKE, FAKE, FAKE, None, None]
        for bad in (None, FAKE + 2):
            args[at] = bad
            assert lib.kv4_evict(c, *args) == L.MOE_ERR_ARG, at
    assert lib.kv4_evict(C.byref(cache(n_seq=0)), None, None, e, None, None, None, None, None) == L.MOE_OK


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    pairs = {"kv4_cache": L.Kv4CacheStruct, "kv4_rows_cfg": L.Kv4RowsCfg, "kv4_attn_cfg": L.Kv4AttnCfg,
             "kv4_evict_cfg": L.Kv4EvictCfg}
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HDR}"', "int main(void) {"]
    for name, py in pairs.items():
        lines.append(f'  printf("{name} sizeof %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-o", str(exe), str(src)], check=True)
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in
           subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()}
    for name, py in pairs.items():
        assert got[name, "sizeof"] == C.sizeof(py)
        for f, _ in py._fields_:
            assert got[name, f] == getattr(py, f).offset, (name, f)
