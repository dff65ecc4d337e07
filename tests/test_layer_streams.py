"""Results that the layer operators' tensor calls allocate belong to the stream
that the call launches on.

On the CPU the allocations record the stream they were made under (no library
call).  On a GPU torch's current stream is kept busy with work that still reads a
freed block, or that a fill would have to wait for, while a call runs elsewhere.
"""
import contextlib

import pytest

torch = pytest.importorskip("torch")

BF16 = torch.bfloat16
CURRENT, LAUNCH, OTHER = 7, 9, 11


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class OnGpu:
    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture
def world(monkeypatch):
    """torch_api over recorders; .made lists (stream, readers) of each allocation."""
    import __graft_entry__

    __graft_entry__.build()
    from collective_datapath_atom_gb300 import torch_api

    class World:
        T = torch_api
        made, calls, stream = [], [], CURRENT

        @staticmethod
        def handle(stream):
            h = type("Handle", (), {})()
            h.R, h.stream_handle = 1, stream
            return h

    w = World()

    def allocate(make):
        def f(*shape, **kw):
            t = OnGpu(make(*shape, dtype=kw.get("dtype")))
            readers = []
            t.record_stream = lambda s: readers.append(s.cuda_stream)
            w.made.append((w.stream, readers))
            return t
        return f

    @contextlib.contextmanager
    def under(s):
        before, w.stream = w.stream, s.cuda_stream
        yield
        w.stream = before

    def set_stream(handle, stream):
        handle.stream_handle = stream if isinstance(stream, int) else stream.cuda_stream

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(w.stream))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch, "empty", allocate(torch.empty))
    monkeypatch.setattr(torch, "zeros", allocate(torch.zeros))
    monkeypatch.setattr(torch_api, "purlin_set_stream", set_stream)
    for name in ("purlin_rms_norm", "purlin_rms_norm_backward", "purlin_grouped_matmul",
                 "purlin_grouped_matmul_weight_grad"):
        monkeypatch.setattr(torch_api, name, lambda *a, **kw: w.calls.append(a[0].stream_handle))
    return w


def mat(*shape, dtype=BF16):
    return OnGpu(torch.ones(*shape, dtype=dtype))


def every_call(T, handle, stream=None):
    x, v, i = mat(4, 64), mat(64), mat(2, dtype=torch.int64)
    T.rms_norm(x, v, handle, stream=stream)
    T.rms_norm(x, v, handle, quantize=True, stream=stream)
    T.rms_norm_backward(x, x, v, handle, stream=stream)
    T.grouped_matmul(x, mat(2, 32, 64), i, i, handle, stream=stream)
    T.grouped_matmul_weight_grad(mat(4, 32), x, i, i, handle, stream=stream)


@pytest.mark.parametrize("handle,stream,launch", [
    (CURRENT, None, CURRENT), (LAUNCH, None, LAUNCH), (CURRENT, LAUNCH, LAUNCH),
    (OTHER, LAUNCH, LAUNCH), (LAUNCH, CURRENT, CURRENT), (0, None, 0)])
def test_results_belong_to_the_launch_stream(world, handle, stream, launch):
    every_call(world.T, world.handle(handle), stream)
    assert world.calls == [launch] * 5
    assert len(world.made) == 7
    for made_on, readers in world.made:
        assert made_on == launch
        assert readers == ([] if launch == CURRENT else [CURRENT])


def test_a_stream_set_through_the_binding_is_the_handle_s(monkeypatch):
    import __graft_entry__

    __graft_entry__.build()
    import collective_datapath_atom_gb300 as P

    monkeypatch.setattr(P, "_ok", lambda status, what: None)
    ctx = P.Context(0, 1, 5)
    assert ctx.stream_handle == 5
    P.purlin_set_stream(ctx, Stream(6))      # the library refuses the null context; recorded all the same
    assert ctx.stream_handle == 6


@pytest.mark.gpu
def test_calls_beside_a_busy_current_stream():
    import __graft_entry__

    __graft_entry__.build()
    from collective_datapath_atom_gb300 import torch_api as T

    rows, k, n = 512, 256, 128
    x = torch.randint(-3, 4, (rows, k), device="cuda").bfloat16()
    w = torch.randint(-3, 4, (1, n, k), device="cuda").bfloat16()
    v = torch.ones(k, device="cuda", dtype=BF16)
    begin, count = torch.zeros(1, device="cuda").long(), torch.full((1,), rows, device="cuda")
    want = (x.double() @ w[0].double().t()).float().bfloat16()
    s = torch.cuda.Stream()
    h = T.initialize(1, stream=s)
    try:
        unit = T.rms_norm(x, v, h)
        T.check(h)
        torch.cuda.synchronize()
        # a fill that went to the current stream would wait behind the sleep
        torch.cuda._sleep(100_000_000)
        y = T.grouped_matmul(x, w, begin, count, h)
        T.check(h)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        # a freed block that the current stream still has to read
        held = torch.full((rows, k), 3.0, device="cuda", dtype=BF16)
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        read = held.clone()
        del held
        z = T.rms_norm(x, v, h)
        T.check(h)
        torch.cuda.synchronize()
        assert bool((read == 3.0).all()) and torch.equal(z, unit)
        # the call's own stream argument
        y = T.grouped_matmul(x, w, begin, count, h, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    finally:
        T.finalize(h)
