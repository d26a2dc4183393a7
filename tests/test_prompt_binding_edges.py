"""Host side of a prompt's calls where their arguments are out of the ordinary: stand-ins as in test_prompt_binding."""
import pytest

from test_prompt_binding import Rot, bf, machine  # noqa: F401  (machine: fixture)
from test_kv4_binding import Tensor, cache_on, i32, queries

torch = pytest.importorskip("torch")

from serving_router_softmax_gb300 import kv4, prompt  # noqa: E402
from serving_router_softmax_gb300.api import MoEError  # noqa: E402


def test_numbers_are_taken_as_they_are_now(machine):  # noqa: F811
    """A scale or a flag that comes as a tensor is read at each call, whatever an earlier call with the same tensor has seen."""
    q, k, st = bf((3, 4, 64), 0), bf((3, 2, 64), 0), i32(2, 0)
    scale, back = torch.tensor(0.5), torch.tensor(False)
    cache, (cq, start, base) = cache_on(0), queries(0)
    pos = Tensor((2, 3), torch.int32, 0)
    for value in (0.5, 0.25, -1.0):
        scale.fill_(value)
        prompt.prompt_attend(q, k, k, st, scale=scale)
        assert machine.lib.calls[-1][2][4]._obj.scale == value
        prompt.prompt_attend(q, k, k, st, scale=value)
        assert machine.lib.calls[-1][2][4]._obj.scale == value
    assert len([key for key in prompt._plans if key[0] == "attend"]) == 3
    for value in (0.5, 0.25):
        scale.fill_(value)
        assert kv4._attn_plan(cache, cq, 2, scale)[0]._obj.scale == value
    for value in (False, True):
        back.fill_(value)
        prompt.rotate(Rot(0), q, k, pos, inverse=back)
        assert machine.lib.calls[-1][2][5]._obj.inverse == value


def test_an_odd_number_of_turned_dimensions_is_refused():
    """(Not rounded down to the pairs that fit: their frequencies would be another embedding's.)"""
    for odd in (33, 49, 17):
        with pytest.raises(MoEError):
            prompt.Rotary.standard(64, rotary_dim=odd, device="cpu")
    assert prompt.Rotary.standard(64, rotary_dim=48, device="cpu").rotary_dim == 48
