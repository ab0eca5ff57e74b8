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


class Device:
    """Stand-ins for what a layer launches and for the streams it launches on: every
    write and read of its weights must be ordered, by the stream or by an event."""

    def __init__(self, monkeypatch, names):
        from padding_free_expert_amd import layer
        self.log, self.current, dev = [], self.stream(1), self
        self.capturing = set()

        class Event:
            def record(self, stream):
                dev.log.append(("record", self, stream.cuda_stream))

        @contextlib.contextmanager
        def enter(s):
            was, dev.current = dev.current, s
            yield
            dev.current = was

        for n in names:
            monkeypatch.setattr(layer, n, lambda *a, stream=None, name=n, **kw: dev.log.append(
                (name, a, (stream or dev.current).cuda_stream)))
        monkeypatch.setattr(torch.cuda, "Event", Event)
        monkeypatch.setattr(torch.cuda, "Stream", lambda device=None: dev.stream(77))
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: dev.stream(h))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: dev.current)
        monkeypatch.setattr(torch.cuda, "stream", enter)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: dev.current.cuda_stream in dev.capturing)

    def stream(self, handle):
        dev = self

        class S(Stream):
            def wait_event(self, e):
                dev.log.append(("wait", e, self.cuda_stream))

            def wait_stream(self, other):
                dev.log.append(("join", other.cuda_stream, self.cuda_stream))
        return S(handle)

    def ordered(self, writes, read):
        """The last call of `writes` is followed by its stream's event, and that is
        waited for before every later call of `read` on another stream."""
        event = home = None
        seen = set()
        for name, what, at in self.log:
            if name == writes:
                event, home, seen = None, at, {at}
            elif name == "record" and at == home:
                event = what
            elif name == "wait" and what is event:
                seen.add(at)
            elif name == "join" and what in seen:
                seen.add(at)
            elif name == read and at not in seen:
                return False
        return home is not None


BLOCK8 = ["xmoe_mx8_quantize_weights", "xmoe_add_rmsnorm", "xmoe_route", "xmoe_build_pft", "xmoe_expert_ffn_up_mx8",
          "xmoe_expert_ffn_down_mx8", "xmoe_combine"]


def _weights(dt=torch.bfloat16, shared=True, T=4, d=64, E=4, h=32):
    z = torch.zeros
    w = dict(wg=z((d, E), dtype=dt), w1=z((E, d, h), dtype=dt), w3=z((E, d, h), dtype=dt), w2=z((E, h, d), dtype=dt),
             norm=z(d, dtype=dt))
    if shared:
        w.update(s1=z((d, h), dtype=dt), s3=z((d, h), dtype=dt), s2=z((h, d), dtype=dt))
    return w, z((T, d), dtype=dt)


@pytest.mark.parametrize("shared", [False, True])
def test_8_bit_weights_are_read_behind_their_quantization(xm, monkeypatch, shared):
    """Whatever stream quantizes them and whatever stream the forward is on."""
    from padding_free_expert_amd.layer import MoEBlock8
    dev = Device(monkeypatch, BLOCK8)
    w, x = _weights(shared=shared)
    order = lambda: dev.ordered("xmoe_mx8_quantize_weights", "xmoe_expert_ffn_up_mx8")
    block = MoEBlock8(w, 4, 2)                 # on stream 1
    block.forward(x)
    assert order() and not any(n == "wait" for n, _, _ in dev.log)
    block.forward(x, stream=dev.stream(2))
    assert order()
    n = len(dev.log)
    block.forward(x, stream=dev.stream(2))     # one wait a stream is enough
    assert order() and not any(e[0] == "wait" for e in dev.log[n:])
    block.refresh_weights(stream=dev.stream(3))
    for s in (None, dev.stream(2), dev.stream(3)):
        block.forward(x, stream=s)
        assert order()


def test_a_captured_quantization_or_forward_waits_for_no_event_outside(xm, monkeypatch):
    """An event of one side of a capture cannot be waited for on the other."""
    from padding_free_expert_amd.layer import MoEBlock8
    dev = Device(monkeypatch, BLOCK8)
    w, x = _weights()
    block = MoEBlock8(w, 4, 2)
    dev.capturing.add(2)
    n = len(dev.log)
    block.forward(x, stream=dev.stream(2))
    block.refresh_weights(stream=dev.stream(2))
    assert not any(e[0] in ("wait", "record") for e in dev.log[n:])
    dev.capturing.clear()
    block.forward(x, stream=dev.stream(2))
    assert any(e[0] == "wait" for e in dev.log[n:])


LAYER = ["xmoe_add_rmsnorm", "xmoe_route", "xmoe_build_pft", "xmoe_build_pft_shared", "xmoe_expert_ffn_up",
         "xmoe_expert_ffn_up_gather", "xmoe_expert_ffn_down", "xmoe_combine", "xmoe_balance_loss", "xmoe_combine_bwd",
         "xmoe_expert_ffn_bwd", "xmoe_route_bwd", "xmoe_route_bwd_balance", "xmoe_expert_ffn_bwd_dact_gather",
         "xmoe_expert_ffn_bwd_dw2", "xmoe_expert_ffn_bwd_dw13_gather", "xmoe_expert_ffn_bwd_dx", "xmoe_dispatch_bwd",
         "xmoe_add_rmsnorm_bwd"]


def test_merged_weights_are_read_behind_their_copies(xm, monkeypatch):
    from padding_free_expert_amd.layer import PaddingFreeMoE
    dev = Device(monkeypatch, LAYER)
    w, x = _weights()
    m = PaddingFreeMoE(w, 4, 2, merge_shared=True)     # on stream 1
    for s in (None, dev.stream(2)):
        n = len(dev.log)
        m.forward(x, stream=s)
        m.backward(x, stream=s)
        waits = [i for i, e in enumerate(dev.log[n:]) if e[0] == "wait"]
        assert waits == ([] if s is None else [0])
    m.refresh_weights(stream=dev.stream(3))
    what, event, at = dev.log[-1]
    assert (what, at) == ("record", 3)
    n = len(dev.log)
    m.backward(x, stream=dev.stream(2))
    assert dev.log[n] == ("wait", event, 2)


@pytest.mark.parametrize("kw,err", [
    (dict(), "seq_offsets"), (dict(seq_offsets=torch.zeros(2, dtype=torch.int32)), "seq_offsets"),
    (dict(seq_offsets=torch.zeros(3)), "seq_offsets"), (dict(seq_offsets=torch.zeros(6, dtype=torch.int32)[::2]), "seq_offsets"),
    (dict(token_mask=torch.zeros(5, dtype=torch.bool)), "token_mask"), (dict(token_mask=torch.zeros(4)), "token_mask"),
    (dict(token_mask=torch.zeros(4, dtype=torch.bool, device="meta")), "token_mask"),
    (dict(x=torch.zeros((3, 64), dtype=torch.bfloat16)), "x"), (dict(x=torch.zeros((4, 64))), "x")])
def test_a_refused_forward_launches_nothing(xm, monkeypatch, kw, err):
    from padding_free_expert_amd.layer import PaddingFreeMoE
    dev = Device(monkeypatch, LAYER)
    w, x = _weights()
    m = PaddingFreeMoE(w, 4, 2, balance_alpha=0.1, n_seq=2)
    good = dict(x=x, seq_offsets=torch.zeros(3, dtype=torch.int32))
    bad = {**({"x": x} if not kw else good), **kw}
    del dev.log[:]
    with pytest.raises((ValueError, TypeError), match=err):
        m.forward(**bad)
    assert dev.log == []
    m.forward(**good)
    assert dev.log


@pytest.mark.parametrize("kw,err", [(dict(dloss=torch.zeros(())), "dloss"), (dict(dloss=torch.zeros(1, dtype=torch.bfloat16)), "dloss"),
                                    (dict(dy=torch.zeros((4, 32), dtype=torch.bfloat16)), "dy")])
def test_a_refused_backward_launches_nothing(xm, monkeypatch, kw, err):
    from padding_free_expert_amd.layer import PaddingFreeMoE
    dev = Device(monkeypatch, LAYER)
    w, x = _weights()
    m = PaddingFreeMoE(w, 4, 2, balance_alpha=0.1)
    m.forward(x)
    del dev.log[:]
    with pytest.raises((ValueError, TypeError), match=err):
        m.backward(**{**dict(dy=x), **kw})
    assert dev.log == []
    m.backward(x, dloss=torch.zeros(1))
    assert dev.log


def test_the_layer_without_the_loss_ignores_its_arguments(xm, monkeypatch):
    from padding_free_expert_amd.layer import PaddingFreeMoE
    Device(monkeypatch, LAYER)
    w, x = _weights()
    m = PaddingFreeMoE(w, 4, 2)
    m.forward(x, token_mask=torch.zeros(9))
    m.backward(x, dloss=torch.zeros(9))


def test_the_serving_block_refuses_what_its_forward_could_not_take(xm, monkeypatch):
    """Its rows are bf16, so the gate and the norm are; the experts' weights are
    quantized from either type."""
    from padding_free_expert_amd.layer import MoEBlock8
    dev = Device(monkeypatch, BLOCK8)
    w, x = _weights()
    for bad in (_weights(torch.float32)[0], {**w, "wg": w["wg"].float()}, {**w, "norm": w["norm"].float()}):
        with pytest.raises(TypeError, match="wg|norm"):
            MoEBlock8(bad, 4, 2)
    assert dev.log == []
    MoEBlock8({**w, "w1": w["w1"].float(), "w3": w["w3"].float(), "w2": w["w2"].float()}, 4, 2).forward(x)


def test_a_layers_passes_run_on_its_device(xm, monkeypatch):
    """Every launch of a pass with the weights' device as the current one."""
    from padding_free_expert_amd import layer
    at = [0]

    @contextlib.contextmanager
    def enter(like):
        assert like.shape == (64, 4)    # the gate's weights
        at.append(1)
        yield
        at.pop()

    Device(monkeypatch, LAYER + BLOCK8)
    launches = []
    for n in set(LAYER + BLOCK8) - {"xmoe_add_rmsnorm", "xmoe_add_rmsnorm_bwd"}:    # these see to it themselves
        monkeypatch.setattr(layer, n, lambda *a, **kw: launches.append(at[-1]))
    monkeypatch.setattr(layer, "_on_device", enter)
    w, x = _weights()
    block = layer.MoEBlock(w, 4, 2, balance_alpha=0.1)
    block.forward(x)
    block.backward(x)
    layer.MoEBlock8(w, 4, 2).forward(x)
    m = layer.PaddingFreeMoE(w, 4, 2, merge_shared=True)
    m.forward(x)
    m.backward(x)
    assert launches and set(launches) == {1} and at == [0]
