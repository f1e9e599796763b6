"""A call of the layers on a stream that the caller names, with stand-ins for the streams and
the tensors (no GPU needed)."""

import contextlib
import types

import pytest
import torch


@pytest.fixture
def mods(monkeypatch):
    from recurrent_associative_memory_gb300 import tensors
    made, entered = [], []

    def external(handle, device=None):
        made.append((handle, device))
        return types.SimpleNamespace(cuda_stream=handle, device=device)

    @contextlib.contextmanager
    def current(stream):
        entered.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "stream", current)

    @tensors.on_stream
    def op(x, y=None, *, stream=None):
        return x, y, stream, len(entered)

    return op, made, entered


def on(index):
    return types.SimpleNamespace(device=torch.device("cuda", index))


@pytest.mark.parametrize("by_name", [False, True])
def test_a_raw_handle_belongs_to_the_tensors_device(mods, by_name):
    op, made, entered = mods
    x = on(1)
    got = op(x=x, y=3, stream=77) if by_name else op(x, 3, stream=77)
    assert made == [(77, torch.device("cuda", 1))] and len(entered) == 1
    assert got == (x, 3, None, 1)   # ran with that stream current, and took no other


def test_a_stream_of_another_device_is_refused(mods):
    op, _, entered = mods
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        op(on(1), stream=types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 0)))
    assert not entered
    same = types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 1))
    op(on(1), stream=same)
    assert entered == [same]


def test_without_a_stream_nothing_is_switched(mods):
    op, made, entered = mods
    assert op(on(1))[3] == 0 and not made and not entered


def test_what_is_not_on_a_gpu_reaches_the_checks(mods):
    op, made, entered = mods
    assert op(torch.zeros(2), stream=77)[3] == 0 and not made and not entered
