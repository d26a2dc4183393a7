"""Host side of the kv4_* binding without a GPU: tensors and library are stand-ins that record what a call would enqueue."""
import contextlib
import ctypes as C
import itertools
import threading

import pytest

torch = pytest.importorskip("torch")

from serving_router_softmax_gb300 import kv4  # noqa: E402
from serving_router_softmax_gb300.api import MoEError  # noqa: E402


class Tensor:
    """What the binding asks of a contiguous tensor of device `index` (-1: the host)."""
    _at = itertools.count(1 << 20, 1 << 24)

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.is_cuda = index >= 0
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")
        self.at = next(self._at)

    def data_ptr(self):
        return self.at

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def stride(self, d=None):
        st = [self.shape[i + 1:].numel() for i in range(len(self.shape))]
        return tuple(st) if d is None else st[d]


class Library:
    """Records each call with the device that is current; `inside` runs in the middle of one."""
    def __init__(self, machine):
        self.machine, self.calls, self.inside = machine, [], lambda: None

    def kv4_attend_workspace(self, cache, cfg):
        return 4096

    def moe_status_str(self, status):
        return b"?"

    def __getattr__(self, name):
        if not name.startswith("kv4_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append((name, self.machine.current(), args))
            self.inside()
            return 0
        return call


class Machine:
    def __init__(self, monkeypatch):
        self._current = threading.local()
        self.lib = Library(self)
        monkeypatch.setattr(kv4.L, "load", lambda: self.lib)
        monkeypatch.setattr(kv4, "_raw_stream", lambda index: 16 * index)
        monkeypatch.setattr(kv4, "_current_device", self.current, raising=False)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        monkeypatch.setattr(torch.cuda, "device", self.on)
        monkeypatch.setattr(torch.cuda, "stream", lambda stream: self.on(stream.device_index))
        monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Tensor(shape if isinstance(shape, (tuple, list)) else (shape,), dtype, device.index))

    def current(self):
        return getattr(self._current, "index", 0)

    @contextlib.contextmanager
    def on(self, index):
        before = self.current()
        self._current.index = index
        try:
            yield
        finally:
            self._current.index = before


@pytest.fixture
def machine(monkeypatch):
    return Machine(monkeypatch)


def cache_on(index):
    return kv4.Kv4Cache(Tensor((8, 2, 64 * 136), torch.uint8, index), Tensor((2, 4), torch.int32, index), 64, 128)


def queries(index):
    """q, q_start, base of two sequences with three tokens in all."""
    return Tensor((3, 8, 128), torch.bfloat16, index), Tensor((3,), torch.int32, index), Tensor((2,), torch.int32, index)


def test_calls_of_two_threads_on_one_stream_do_not_share_a_workspace(machine):
    """kv4_attend is two launches; the interpreter lock is free between them, so another thread's may come in between."""
    both = threading.Barrier(2, timeout=30)
    machine.lib.inside = both.wait
    caches, errors = [cache_on(0), cache_on(0)], []

    def work(c):
        try:
            for _ in range(3):
                kv4.kv4_attend(c, *queries(0), 2)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
            both.abort()

    threads = [threading.Thread(target=work, args=(c,)) for c in caches]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    used = {}
    for _, _, args in machine.lib.calls:
        used.setdefault(C.addressof(args[0]._obj), set()).add(args[8])
    a, b = used.values()
    assert len(a) == 1 and len(b) == 1 and a != b  # kept from call to call, each thread's its own


def test_workspaces_are_kept_for_a_few_streams_only(machine, monkeypatch):
    c, seen = cache_on(0), []
    for stream in list(range(100)) + [99, 99]:
        monkeypatch.setattr(kv4, "_raw_stream", lambda index, s=stream: s)
        kv4.kv4_attend(c, *queries(0), 2)
        seen.append(machine.lib.calls[-1][2][8])
    assert seen[-1] == seen[-2] == seen[-3] and len(set(seen)) == 100
    assert len(kv4._workspaces.held) <= 16


# ------------------------------------------------------------------ devices
def rows(index, heads=2):
    return Tensor((3, heads, 128), torch.bfloat16, index)


def i32(n, index):
    return Tensor((n,), torch.int32, index)


def f32(shape, index):
    return Tensor(shape, torch.float32, index)


def calls(c, index, at=None, other=None, **kw):
    """Every call on cache c with tensors of device `index`; those named in `at` on device `other` instead."""
    d = lambda name: other if at == name else index  # noqa: E731
    q = lambda: (Tensor((3, 8, 128), torch.bfloat16, d("q")), i32(3, d("q_start")), i32(2, d("base")), 2)  # noqa: E731
    vis = lambda: Tensor((3,), torch.int64, d("visible"))  # noqa: E731
    err, mass = i32(1, d("dev_err")), f32((2, 2, 256), d("mass"))
    return {
        "kv4_append": lambda: kv4.kv4_append(c, rows(d("k")), rows(d("v")), i32(3, d("seq")), i32(3, d("slot")), held=True, dev_err=err, **kw),
        "kv4_read": lambda: kv4.kv4_read(c, i32(3, d("seq")), i32(3, d("slot")), dev_err=err, **kw),
        "kv4_attend": lambda: kv4.kv4_attend(c, *q(), visible=vis(), out=Tensor((3, 8, 128), torch.bfloat16, d("out")),
                                             lse=f32((3, 8), d("lse")), workspace=Tensor((4096,), torch.uint8, d("workspace")), dev_err=err, **kw),
        "kv4_weigh": lambda: kv4.kv4_weigh(c, *q(), f32((3, 8), d("lse")), mass, visible=vis(), dev_err=err, **kw),
        "kv4_evict": lambda: kv4.kv4_evict(c, mass, i32(2, d("lens")), 4, 1, mass_out=f32((2, 2, 256), d("mass_out")), dev_err=err, **kw),
    }


NAMED = {"kv4_append": ["k", "v", "seq", "slot", "dev_err"], "kv4_read": ["seq", "slot", "dev_err"],
         "kv4_attend": ["q", "q_start", "base", "visible", "out", "lse", "workspace", "dev_err"],
         "kv4_weigh": ["q", "q_start", "base", "visible", "lse", "mass", "dev_err"], "kv4_evict": ["mass", "lens", "mass_out", "dev_err"]}


class Stream:
    def __init__(self, index):
        self.device_index, self.device = index, torch.device("cuda", index)


@pytest.mark.parametrize("name", sorted(NAMED))
def test_calls_run_on_the_device_of_the_cache(machine, name):
    for index, current, kw in ((0, 0, {}), (1, 0, {}), (0, 1, {}), (1, 0, dict(stream=Stream(1))), (1, 1, dict(stream=Stream(1)))):
        with machine.on(current):
            calls(cache_on(index), index, **kw)[name]()
            assert machine.current() == current
        got, on, args = machine.lib.calls[-1]
        assert (got, on, args[-1]) == (name, index, 16 * index)
    c = cache_on(1)
    need = []
    machine.lib.kv4_attend_workspace = lambda *a: need.append(machine.current()) or 4096
    kv4.kv4_attend_workspace_bytes(c, Tensor((3, 8, 128), torch.bfloat16, 1), 2)
    assert need == [1]


@pytest.mark.parametrize("name,at", [(n, a) for n in sorted(NAMED) for a in NAMED[n]])
def test_tensors_of_another_device_are_refused(machine, name, at):
    c = cache_on(1)
    calls(c, 1)[name]()  # a call of this shape has been made before
    n = len(machine.lib.calls)
    for other in (0, -1):
        with pytest.raises(MoEError):
            calls(c, 1, at, other)[name]()
    assert len(machine.lib.calls) == n


@pytest.mark.parametrize("name", sorted(NAMED))
def test_streams_of_another_device_are_refused(machine, name):
    with pytest.raises(MoEError):
        calls(cache_on(1), 1, stream=Stream(0))[name]()
    assert not machine.lib.calls
