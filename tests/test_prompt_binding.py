"""Host side of the binding of a prompt's pass without a GPU: tensors and library are stand-ins that record what a call would
enqueue (as in test_kv4_binding)."""
import pytest

from test_kv4_binding import Library, Machine, Stream, Tensor, f32, i32

torch = pytest.importorskip("torch")

from serving_router_softmax_gb300 import prompt  # noqa: E402
from serving_router_softmax_gb300.api import ExpertLayer, MoEError  # noqa: E402


class PromptLibrary(Library):
    def moe_group_down_workspace(self, lw, T, k):
        return 4096

    def __getattr__(self, name):
        if not name.startswith("moe_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append((name, self.machine.current(), args))
            return 0
        return call


@pytest.fixture
def machine(monkeypatch):
    m = Machine(monkeypatch)
    m.lib = PromptLibrary(m)
    monkeypatch.setattr(prompt, "_raw_stream", lambda index: 16 * index)
    monkeypatch.setattr(prompt, "_current_device", m.current)
    prompt._plans.clear()
    yield m
    prompt._plans.clear()


class Rot:
    """A Rotary of device `index`."""
    def __init__(self, index, axes=2):
        self.head_dim, self.rotary_dim, self.n_axes, self.interleaved = 64, 32, axes, False
        self._turns, self._axis = Tensor((16,), torch.int64, index), Tensor((16,), torch.int32, index)
        self.device = self._turns.device


def bf(shape, index):
    return Tensor(shape, torch.bfloat16, index)


def calls(index, at=None, other=None, **kw):
    """Every call with tensors of device `index`; those named in `at` on device `other` instead."""
    d = lambda name: other if at == name else index  # noqa: E731
    err = i32(1, d("dev_err"))
    layer = ExpertLayer(bf((4, 256, 64), d("gate_up")), bf((4, 64, 128), d("down")), "bf16")
    union = {"n_unique": i32(1, d("n_unique")), "unique": i32(4, d("unique")), "offsets": i32(5, d("offsets")),
             "perm_token": i32(6, d("perm_token")), "inv": i32(6, d("inv"))}
    return {
        "moe_rotate": lambda: prompt.rotate(Rot(d("rot")), bf((3, 4, 64), d("q")), bf((3, 2, 64), d("k")), Tensor((2, 3), torch.int32, d("pos")),
                                            out_q=bf((3, 4, 64), d("out_q")), out_k=bf((3, 2, 64), d("out_k")), dev_err=err, **kw),
        "moe_prompt_attend": lambda: prompt.prompt_attend(bf((3, 4, 64), d("q")), bf((3, 2, 64), d("k")), bf((3, 2, 64), d("v")), i32(2, d("start")),
                                                          out=bf((3, 4, 64), d("out")), lse=f32((3, 4), d("lse")), dev_err=err, **kw),
        "moe_group_gate_up": lambda: prompt.group_gate_up(bf((3, 64), d("x")), layer, union, 2, out=bf((6, 128), d("out")), dev_err=err, **kw),
        "moe_group_down": lambda: prompt.group_down(bf((6, 128), d("h")), layer, union, f32((3, 2), d("w")), y=bf((3, 64), d("y")),
                                                    workspace=Tensor((4096,), torch.uint8, d("workspace")), dev_err=err, **kw),
    }


NAMED = {"moe_rotate": ["rot", "q", "k", "pos", "out_q", "out_k", "dev_err"],
         "moe_prompt_attend": ["q", "k", "v", "start", "out", "lse", "dev_err"],
         "moe_group_gate_up": ["x", "gate_up", "down", "n_unique", "unique", "offsets", "perm_token", "out", "dev_err"],
         "moe_group_down": ["h", "gate_up", "down", "n_unique", "unique", "offsets", "inv", "w", "y", "workspace", "dev_err"]}


@pytest.mark.parametrize("name", sorted(NAMED))
def test_calls_run_on_the_device_of_their_tensors(machine, name):
    for index, current, kw in ((0, 0, {}), (1, 0, {}), (0, 1, {}), (1, 0, dict(stream=Stream(1))), (1, 1, dict(stream=Stream(1)))):
        with machine.on(current):
            calls(index, **kw)[name]()
            assert machine.current() == current
        got, on, args = machine.lib.calls[-1]
        assert (got, on, args[-1]) == (name, index, 16 * index)


@pytest.mark.parametrize("name,at", [(n, a) for n in sorted(NAMED) for a in NAMED[n]])
def test_tensors_of_another_device_are_refused(machine, name, at):
    calls(1)[name]()  # a call of this shape has been made before
    n = len(machine.lib.calls)
    for other in (0, -1):
        with pytest.raises(MoEError):
            calls(1, at, other)[name]()
    assert len(machine.lib.calls) == n


@pytest.mark.parametrize("name", sorted(NAMED))
def test_streams_of_another_device_are_refused(machine, name):
    with pytest.raises(MoEError):
        calls(1, stream=Stream(0))[name]()
    assert not machine.lib.calls


def test_shapes_and_types_are_checked_once_known_too(machine):
    """A call of a good shape leaves nothing behind that lets a bad one through."""
    rot, q, k = Rot(0), bf((3, 4, 64), 0), bf((3, 2, 64), 0)
    pos, lay = Tensor((2, 3), torch.int32, 0), ExpertLayer(bf((4, 256, 64), 0), bf((4, 64, 128), 0), "bf16")
    u = {"n_unique": i32(1, 0), "unique": i32(4, 0), "offsets": i32(5, 0), "perm_token": i32(6, 0), "inv": i32(6, 0)}
    x, h, w, st = bf((3, 64), 0), bf((6, 128), 0), f32((3, 2), 0), i32(2, 0)
    good = [lambda: prompt.rotate(rot, q, k, pos), lambda: prompt.rotate(rot, q, None, pos), lambda: prompt.prompt_attend(q, k, k, st),
            lambda: prompt.group_gate_up(x, lay, u, 2), lambda: prompt.group_down(h, lay, u, w)]
    for _ in range(2):
        for call in good:
            call()
    n = len(machine.lib.calls)
    half = Tensor((3, 4, 64), torch.float16, 0)
    bad = [
        lambda: prompt.rotate(rot, half, None, pos), lambda: prompt.rotate(rot, q, f32((3, 2, 64), 0), pos),
        lambda: prompt.rotate(rot, q, bf((2, 2, 64), 0), pos), lambda: prompt.rotate(rot, bf((3, 4, 32), 0), None, pos),
        lambda: prompt.rotate(rot, q, k, i32(3, 0)), lambda: prompt.rotate(rot, q, k, Tensor((3, 3), torch.int32, 0)),
        lambda: prompt.rotate(rot, q, k, Tensor((2, 3), torch.int64, 0)), lambda: prompt.rotate(rot, q, k, pos, out_q=k),
        lambda: prompt.rotate(rot, q, k, pos, out_k=bf((3, 2, 32), 0)), lambda: prompt.rotate(rot, x, None, pos),
        lambda: prompt.prompt_attend(half, k, k, st), lambda: prompt.prompt_attend(q, k, bf((3, 1, 64), 0), st),
        lambda: prompt.prompt_attend(q, bf((2, 2, 64), 0), bf((2, 2, 64), 0), st), lambda: prompt.prompt_attend(q, k, k, Tensor((2,), torch.int64, 0)),
        lambda: prompt.prompt_attend(q, k, k, i32(0, 0)), lambda: prompt.prompt_attend(q, k, k, Tensor((1, 2), torch.int32, 0)),
        lambda: prompt.prompt_attend(q, k, k, st, out=bf((3, 4, 32), 0)), lambda: prompt.prompt_attend(q, k, k, st, lse=f32((4, 3), 0)),
        lambda: prompt.group_gate_up(x, lay, u, 3), lambda: prompt.group_gate_up(x, lay, u, 0), lambda: prompt.group_gate_up(bf((3, 128), 0), lay, u, 2),
        lambda: prompt.group_gate_up(f32((3, 64), 0), lay, u, 2), lambda: prompt.group_gate_up(x, lay, dict(u, offsets=i32(4, 0)), 2),
        lambda: prompt.group_gate_up(x, ExpertLayer(bf((4, 256, 64), 0), bf((4, 64, 128), 0), "e4m3"), u, 2),
        lambda: prompt.group_down(bf((5, 128), 0), lay, u, w), lambda: prompt.group_down(h, lay, u, f32((6,), 0)),
        lambda: prompt.group_down(h, lay, u, bf((3, 2), 0)), lambda: prompt.group_down(h, lay, u, w, y=f32((3, 64), 0)),
        lambda: prompt.group_down(h, lay, u, w, workspace=f32((4096,), 0)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(MoEError):
            call()
            raise AssertionError(i)
    assert len(machine.lib.calls) == n


def test_layers_smaller_than_they_say_are_refused(machine):
    u = {"n_unique": i32(1, 0), "unique": i32(4, 0), "offsets": i32(5, 0), "perm_token": i32(6, 0), "inv": i32(6, 0)}
    x, h, w = bf((3, 64), 0), bf((6, 128), 0), f32((3, 2), 0)
    both = [lambda lay: prompt.group_gate_up(x, lay, u, 2), lambda lay: prompt.group_down(h, lay, u, w)]
    # H 64, I 128, 4 experts: 4 x 256 x 64 and 4 x 64 x 128 values; tiled, 64 rows of down are 128.
    good = [ExpertLayer(bf((4, 256, 64), 0), bf((4, 64, 128), 0), "bf16"),
            ExpertLayer(bf((4 * 256 * 64,), 0), bf((4 * 128 * 128,), 0), "bf16", layout="tiled", dims=(64, 128, 4))]
    for _ in range(2):
        for lay in good:
            for call in both:
                call(lay)
                at = machine.lib.calls[-1][2][3]._obj
                assert (at.w_gate_up, at.w_down) == (lay.gate_up.at, lay.down.at)  # this layer's, not one's of its shape
        good.append(ExpertLayer(bf((4, 256, 64), 0), bf((4, 64, 128), 0), "bf16"))
    n = len(machine.lib.calls)
    bad = [ExpertLayer(bf((4, 256, 64), 0), bf((3, 64, 128), 0), "bf16"), ExpertLayer(bf((4, 256, 64), 0), bf((4, 64, 127), 0), "bf16"),
           ExpertLayer(bf((4 * 256 * 64 - 1,), 0), bf((4 * 128 * 128,), 0), "bf16", layout="tiled", dims=(64, 128, 4)),
           ExpertLayer(bf((4 * 256 * 64,), 0), bf((4 * 64 * 128,), 0), "bf16", layout="tiled", dims=(64, 128, 4)),
           ExpertLayer(bf((4 * 256 * 64,), 0), bf((4 * 128 * 128,), 0), "bf16", layout="tiled", dims=(64, 128, 5)),
           ExpertLayer(bf((4 * 256 * 64,), 0), bf((4 * 128 * 128,), 0), "bf16", layout="tiled", dims=(64, 192, 4))]
    apart = ExpertLayer(bf((4, 256, 64), 0), bf((4, 64, 128), 0), "bf16")
    apart.down.is_contiguous = lambda: False
    for lay in [*bad, apart]:
        for call in both:
            with pytest.raises(MoEError):
                call(lay)
    assert len(machine.lib.calls) == n
