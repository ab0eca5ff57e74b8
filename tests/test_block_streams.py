"""Which stream a call's memory belongs to and in which order a layer checks and
launches, followed on the host with stand-ins for streams and launches.  No GPU
needed."""
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def xm():
    import padding_free_expert_amd as m
    return m


class Like:
    """A tensor of a device that the allocator's stand-in knows."""
    is_cuda, device = True, torch.device("cpu")

    def get_device(self):
        return 0


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def allocations(xm, monkeypatch):
    """The handle of the stream that is current at each torch.empty; 5 is current
    outside any context."""
    at, seen = [5], []

    @contextlib.contextmanager
    def enter(s):
        at.append(s.cuda_stream)
        yield
        at.pop()

    empty = torch.empty

    def spy(*a, **kw):
        seen.append(at[-1])
        return empty(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: Stream(h))
    monkeypatch.setattr(xm, "_raw_stream", lambda dev: at[-1])
    monkeypatch.setattr(torch, "empty", spy)
    return seen


@pytest.mark.parametrize("stream,owner", [(None, 5), (Stream(9), 9), (11, 11), (Stream(5), 5), (0, 0)])
def test_a_workspace_belongs_to_the_calls_stream(xm, allocations, stream, owner):
    """Memory that another stream still writes goes out again on that stream only: a
    workspace taken on the current stream for a call on a second one would be
    written by both."""
    ws, n = xm._workspace(None, 1000, Like(), stream)
    assert n >= 1000 and allocations == [owner]


def test_a_callers_workspace_is_used_as_it_is(xm, allocations):
    mine = torch.zeros(64, dtype=torch.uint8)
    ws, n = xm._workspace(mine, 1000, Like(), Stream(9))
    assert ws is mine and n == 64 and allocations == []


def test_the_gates_workspace_belongs_to_the_calls_stream(xm, allocations, monkeypatch):
    T, d, E, k = 6, 64, 8, 2
    x = torch.zeros((T, d), dtype=torch.bfloat16)
    wg, ids = torch.zeros((d, E), dtype=torch.bfloat16), torch.zeros((T, k), dtype=torch.int32)
    w, logits = torch.zeros((T, k)), torch.zeros((T, E))
    inner = xm._workspace
    monkeypatch.setattr(xm, "_workspace", lambda ws, need, like, stream=None: inner(ws, need, Like(), stream))
    monkeypatch.setattr(xm, "xmoe_route_workspace_size", lambda *a: 1000)
    with pytest.raises(ValueError, match="device tensors"):   # what follows the workspace: the pointers
        xm.xmoe_route(x, wg, k, ids, w, logits, stream=Stream(9))
    assert allocations == [9]
