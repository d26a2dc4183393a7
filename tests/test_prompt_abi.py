"""Refusals and struct layouts of the calls of a prompt's pass (CPU: every check comes before any CUDA call)."""
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


# ------------------------------------------------------------------ moe_rotate
def rot(**kw):
    f = dict(T=3, n_q_heads=4, n_k_heads=2, head_dim=64, rotary_dim=64, n_axes=1, interleaved=0, inverse=0, dtype=L.DTYPE_BF16,
             q_token_stride=256, q_head_stride=64, k_token_stride=128, k_head_stride=64,
             oq_token_stride=256, oq_head_stride=64, ok_token_stride=128, ok_head_stride=64)
    f.update(kw)
    return L.RotateCfg(**f)


def rotate(lib, cfg, q=FAKE, k=FAKE, pos=FAKE, turns=FAKE, axis=FAKE, oq=2 * FAKE, ok=2 * FAKE, err=None):
    return lib.moe_rotate(q, k, pos, turns, axis, None if cfg is None else C.byref(cfg), oq, ok, err, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), L.MOE_ERR_ARG), (dict(n_q_heads=0), L.MOE_ERR_ARG), (dict(n_k_heads=-1), L.MOE_ERR_ARG), (dict(n_axes=0), L.MOE_ERR_ARG),
    (dict(interleaved=2), L.MOE_ERR_ARG), (dict(inverse=-1), L.MOE_ERR_ARG), (dict(T=(1 << 24) + 1), L.MOE_ERR_UNSUPPORTED),
    (dict(n_axes=5), L.MOE_ERR_UNSUPPORTED), (dict(n_q_heads=4095), L.MOE_ERR_UNSUPPORTED), (dict(dtype=L.DTYPE_E4M3_B128), L.MOE_ERR_UNSUPPORTED),
    (dict(head_dim=60), L.MOE_ERR_UNSUPPORTED), (dict(head_dim=520, rotary_dim=512), L.MOE_ERR_UNSUPPORTED),
    (dict(rotary_dim=24), L.MOE_ERR_UNSUPPORTED), (dict(rotary_dim=0), L.MOE_ERR_UNSUPPORTED), (dict(rotary_dim=80), L.MOE_ERR_UNSUPPORTED),
    (dict(q_token_stride=252), L.MOE_ERR_UNSUPPORTED), (dict(k_head_stride=-64), L.MOE_ERR_UNSUPPORTED),
    (dict(oq_token_stride=128), L.MOE_ERR_UNSUPPORTED),   # rows of an output that share values
    (dict(ok_head_stride=32), L.MOE_ERR_UNSUPPORTED), (dict(oq_token_stride=0), L.MOE_ERR_UNSUPPORTED)])
def test_rotate_refusals(lib, kw, want):
    assert rotate(lib, rot(**kw)) == want


def test_rotate_pointers(lib):
    assert rotate(lib, None) == L.MOE_ERR_ARG
    for name in ("q", "k", "pos", "turns", "axis", "oq", "ok"):
        assert rotate(lib, rot(), **{name: None}) == L.MOE_ERR_ARG, name
        assert rotate(lib, rot(), **{name: FAKE + 2}) == L.MOE_ERR_ARG, name
    assert rotate(lib, rot(), err=FAKE + 1) == L.MOE_ERR_ARG
    assert rotate(lib, rot(T=0), q=None, k=None, pos=None) == L.MOE_OK
    # in place with other strides than the input's
    assert rotate(lib, rot(oq_token_stride=512), oq=FAKE) == L.MOE_ERR_ARG
    assert rotate(lib, rot(k_head_stride=128, k_token_stride=256), ok=FAKE) == L.MOE_ERR_ARG


# ------------------------------------------------------------------ moe_prompt_attend
def prompt(**kw):
    f = dict(T=9, n_seq=2, n_q_heads=8, n_kv_heads=2, head_dim=64, scale=0.125, q_token_stride=512, q_head_stride=64,
             k_token_stride=128, k_head_stride=64, v_token_stride=128, v_head_stride=64)
    f.update(kw)
    return L.PromptCfg(**f)


def attend(lib, cfg, q=FAKE, k=FAKE, v=FAKE, start=FAKE, out=FAKE, lse=FAKE, err=None):
    return lib.moe_prompt_attend(q, k, v, start, None if cfg is None else C.byref(cfg), out, lse, err, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), L.MOE_ERR_ARG), (dict(n_seq=-1), L.MOE_ERR_ARG), (dict(n_kv_heads=0), L.MOE_ERR_ARG), (dict(n_q_heads=0), L.MOE_ERR_ARG),
    (dict(n_q_heads=7), L.MOE_ERR_ARG), (dict(scale=float("nan")), L.MOE_ERR_ARG), (dict(scale=float("inf")), L.MOE_ERR_ARG),
    (dict(scale=3e38), L.MOE_ERR_ARG), (dict(scale=-3e38), L.MOE_ERR_ARG),
    (dict(head_dim=96), L.MOE_ERR_UNSUPPORTED), (dict(head_dim=256), L.MOE_ERR_UNSUPPORTED), (dict(T=(1 << 24) + 1), L.MOE_ERR_UNSUPPORTED),
    (dict(n_seq=2049), L.MOE_ERR_UNSUPPORTED), (dict(n_q_heads=258), L.MOE_ERR_UNSUPPORTED), (dict(n_q_heads=1026), L.MOE_ERR_UNSUPPORTED),
    (dict(q_token_stride=508), L.MOE_ERR_UNSUPPORTED), (dict(k_head_stride=-64), L.MOE_ERR_UNSUPPORTED), (dict(v_token_stride=1), L.MOE_ERR_UNSUPPORTED), (dict(k_head_stride=0), L.MOE_ERR_UNSUPPORTED)])
def test_prompt_refusals(lib, kw, want):
    assert attend(lib, prompt(**kw)) == want


def test_prompt_pointers(lib):
    assert attend(lib, None) == L.MOE_ERR_ARG
    for name in ("q", "k", "v", "start", "out"):
        assert attend(lib, prompt(), **{name: None}) == L.MOE_ERR_ARG, name
    for name in ("q", "k", "v", "out"):
        assert attend(lib, prompt(), **{name: FAKE + 8}) == L.MOE_ERR_ARG, name
    for name in ("start", "lse", "err"):
        assert attend(lib, prompt(), **{name: FAKE + 2}) == L.MOE_ERR_ARG, name
    assert attend(lib, prompt(T=0), q=None, k=None, v=None, out=None) == L.MOE_OK
    assert attend(lib, prompt(n_seq=0), q=None) == L.MOE_OK


# ------------------------------------------------------------------ moe_group_*
def layer(pool=None, **kw):
    f = dict(H=128, I=192, E=8, dtype=L.DTYPE_BF16, layout=L.LAYOUT_ROWMAJOR, w_gate_up=FAKE, w_down=FAKE)
    f.update(kw)
    return L.LayerWeights(pool=None if pool is None else C.pointer(pool), **f)


def gate_up(lib, lw, T=300, k=2, x=FAKE, n=FAKE, u=FAKE, o=FAKE, p=FAKE, h=FAKE, err=None):
    return lib.moe_group_gate_up(x, T, k, None if lw is None else C.byref(lw), n, u, o, p, h, err, None)


def down(lib, lw, T=300, k=2, h=FAKE, n=FAKE, u=FAKE, o=FAKE, p=FAKE, w=FAKE, y=FAKE, ws=FAKE, size=1 << 40, err=None):
    return lib.moe_group_down(h, T, k, None if lw is None else C.byref(lw), n, u, o, p, w, y, ws, size, err, None)


@pytest.mark.parametrize("kw,T,k,want", [
    ({}, -1, 2, L.MOE_ERR_ARG), ({}, 300, 0, L.MOE_ERR_ARG), ({}, 300, 17, L.MOE_ERR_UNSUPPORTED), ({}, 1 << 22, 2, L.MOE_ERR_UNSUPPORTED),
    ({}, (1 << 22) + 1, 1, L.MOE_ERR_UNSUPPORTED), (dict(H=100), 300, 2, L.MOE_ERR_UNSUPPORTED), (dict(I=96), 300, 2, L.MOE_ERR_UNSUPPORTED),
    (dict(E=0), 300, 2, L.MOE_ERR_UNSUPPORTED), (dict(E=1025), 300, 2, L.MOE_ERR_UNSUPPORTED), (dict(dtype=L.DTYPE_F32), 300, 2, L.MOE_ERR_UNSUPPORTED),
    (dict(dtype=L.DTYPE_E4M3_B128), 300, 2, L.MOE_ERR_UNSUPPORTED), (dict(layout=2), 300, 2, L.MOE_ERR_ARG),
    (dict(w_gate_up=None, w_down=None), 300, 2, L.MOE_ERR_ARG), (dict(w_gate_up=FAKE + 8, w_down=FAKE + 8), 300, 2, L.MOE_ERR_ARG),
    (dict(pool=L.ExpertPool(0, 0, 0, FAKE, FAKE, FAKE, FAKE)), 300, 2, L.MOE_ERR_ARG),
    (dict(pool=L.ExpertPool(4, 2, 2, FAKE, FAKE, FAKE, None)), 300, 2, L.MOE_ERR_ARG),
    (dict(E=1024, H=1 << 16, I=1 << 16, layout=L.LAYOUT_TILED), 300, 2, L.MOE_ERR_UNSUPPORTED)])
def test_group_refusals(lib, kw, T, k, want):
    assert gate_up(lib, layer(**kw), T, k) == want
    assert down(lib, layer(**kw), T, k) == want
    assert lib.moe_group_down_workspace(C.byref(layer(**kw)), T, k) == 0


def test_group_pointers(lib):
    assert gate_up(lib, None) == L.MOE_ERR_ARG and down(lib, None) == L.MOE_ERR_ARG
    assert lib.moe_group_down_workspace(None, 4, 2) == 0
    for call, names, wide in ((gate_up, "xnuoph", "xh"), (down, "hnuopwy", "hy")):
        for name in names:
            assert call(lib, layer(), **{name: None}) == L.MOE_ERR_ARG, name
            assert call(lib, layer(), **{name: FAKE + (8 if name in wide else 2)}) == L.MOE_ERR_ARG, name
        assert call(lib, layer(), err=FAKE + 1) == L.MOE_ERR_ARG
    need = lib.moe_group_down_workspace(C.byref(layer()), 300, 2)
    assert need >= 300 * 2 * 128 * 2
    assert down(lib, layer(), size=need - 1) == L.MOE_ERR_WORKSPACE
    assert down(lib, layer(), ws=None) == L.MOE_ERR_WORKSPACE
    assert down(lib, layer(), ws=FAKE + 128) == L.MOE_ERR_ARG
    assert gate_up(lib, layer(), T=0, x=None) == L.MOE_OK and down(lib, layer(), T=0, h=None, ws=None) == L.MOE_OK


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    pairs = {"moe_rotate_cfg": L.RotateCfg, "moe_prompt_cfg": L.PromptCfg}
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HDR}"', "int main(void) {",
             '  printf("classes n %d\\n", MOE_PROF_CLASSES);']
    for name, py in pairs.items():
        lines.append(f'  printf("{name} sizeof %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-o", str(tmp_path / "layout"), str(src)], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split("\n")
    got = {(a, b): int(c) for a, b, c in (line.split() for line in out if line)}
    assert got["classes", "n"] == len(L.PROF_CLASSES)
    for name, py in pairs.items():
        assert got[name, "sizeof"] == C.sizeof(py)
        for f, _ in py._fields_:
            assert got[name, f] == getattr(py, f).offset, (name, f)


# ------------------------------------------------------------------ the binding
def test_rotary_angles():
    """The part of a turn, times 2^64, of each frequency; pi by Machin's formula."""
    pytest.importorskip("torch")
    from fractions import Fraction

    from serving_router_softmax_gb300.prompt import Rotary

    def atan_inverse(n):
        return sum(Fraction((-1) ** i, (2 * i + 1) * n ** (2 * i + 1)) for i in range(60))

    turn = 8 * (4 * atan_inverse(5) - atan_inverse(239))
    freqs = [1.0, 0.1, 1e-4, 3.0, 7.0, -0.5, 2.0 ** -60, 0.0]
    r = Rotary(freqs, 32, [0, 1, 2, 0, 1, 2, 0, 3], device="cpu")
    assert [t % 2 ** 64 for t in r._turns.tolist()] == [round(Fraction(f) / turn * 2 ** 64) % 2 ** 64 for f in freqs]
    assert (r.rotary_dim, r.head_dim, r.n_axes) == (16, 32, 4)


def test_rotary_refusals():
    pytest.importorskip("torch")
    from serving_router_softmax_gb300.api import MoEError
    from serving_router_softmax_gb300.prompt import Rotary
    for args in (([1.0] * 7, 64), ([], 64), ([1.0] * 8, 8), ([1.0] * 8, 20), ([1.0] * 8, 520), ([1.0] * 8, 64, [0] * 7),
                 ([1.0] * 8, 64, [4] * 8), ([1.0] * 8, 64, [-1] * 8), ([float("nan")] * 8, 64), ([float("inf")] * 8, 64)):
        with pytest.raises(MoEError):
            Rotary(*args, device="cpu")
    with pytest.raises(MoEError):
        Rotary.standard(64, sections=[8, 8], device="cpu")
    assert Rotary.standard(64, sections=[8, 12, 12], device="cpu")._axis.tolist() == [0] * 8 + [1] * 12 + [2] * 12


def test_host_tensors_are_refused():
    torch = pytest.importorskip("torch")
    import serving_router_softmax_gb300 as mv
    x, i = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    lay = mv.ExpertLayer(torch.zeros((2, 128, 64), dtype=torch.bfloat16), torch.zeros((2, 64, 64), dtype=torch.bfloat16), "bf16")
    for call in (lambda: mv.rotate(mv.Rotary.standard(64, device="cpu"), x, None, i), lambda: mv.prompt_attend(x, x, x, i),
                 lambda: mv.group_gate_up(x[:, 0], lay, {}, 1), lambda: mv.group_down(x[:, 0], lay, {}, torch.zeros((4, 1)))):
        with pytest.raises(mv.MoEError):
            call()
