"""The expert layer's use of streams, checked without a GPU: streams are
modelled by vector clocks and memory by the stream it was allocated on.

Every tensor that a library call or a torch operation touches has to be
ordered after its last use on another stream, and to belong to the stream that
uses it or to be recorded there: memory that is dropped goes back to the stream
that allocated it."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode
from torch.utils._pytree import tree_leaves


class Model:
    def __init__(self):
        self.current, self.faults = None, []
        self.home, self.recorded, self.last, self.alive = {}, {}, {}, []

    def stream(self, name):
        m = self

        class Stream:
            def __init__(self):
                self.name, self.cuda_stream, self.clock, self.seen = name, hash(name) & 0xFFFF, 0, {}

            def wait_stream(self, other):
                for s, c in list(other.seen.items()) + [(other, other.clock)]:
                    self.seen[s] = max(self.seen.get(s, 0), c)

        s = Stream()
        if m.current is None:
            m.current = s
        return s

    @staticmethod
    def key(t):
        return t.untyped_storage()._cdata

    def owned(self, t):
        """A tensor new to the model: allocated on the current stream."""
        if self.key(t) not in self.home:
            self.home[self.key(t)] = self.current
            self.alive.append(t.untyped_storage())  # (no address comes back)

    def touch(self, where, stream, t):
        k = self.key(t)
        self.owned(t)
        if self.home[k] is not stream and stream not in self.recorded.get(k, ()):
            self.faults.append(f"{where}: memory of {self.home[k].name} used on {stream.name}")
        s, c = self.last.get(k, (stream, 0))
        if s is not stream and stream.seen.get(s, 0) < c:
            self.faults.append(f"{where}: used on {stream.name} without waiting for {s.name}")
        stream.clock += 1
        self.last[k] = (stream, stream.clock)


def tensors(o):
    if isinstance(o, torch.Tensor):
        return [o]
    return [t for t in vars(o).values() if isinstance(t, torch.Tensor)] if hasattr(o, "__dict__") else []


@pytest.fixture
def model(monkeypatch):
    from fp4_quantization_amd import moe
    m = Model()

    class Operations(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            for t in tree_leaves((args, kwargs or {}, out)):
                if isinstance(t, torch.Tensor):
                    m.touch(str(func), m.current, t) if "empty" not in str(func) else m.owned(t)
            return out

    def call(name):
        def run(*args, stream=None, **kwargs):
            args = list(args) + list(kwargs.values())
            for a in [a for a in args if hasattr(a, "cuda_stream")]:
                stream = a
            for t in [t for a in args for t in tensors(a)]:
                m.touch(name, stream or m.current, t)
        return run

    class Workspace:
        def __init__(self, rows, cols, groups=1, device="cpu", stream=None):
            self.buf = torch.empty(64, dtype=torch.uint8)
            m.touch("Workspace", stream or m.current, self.buf)

    @contextlib.contextmanager
    def stream(s):
        before, m.current = m.current, s or m.current
        yield
        m.current = before

    host = ("ufp4_recipe_config", "ufp4_expert_rows")
    for name in [n for n in vars(moe) if n.startswith("ufp4_") and n not in host]:
        monkeypatch.setattr(moe, name, call(name))
    monkeypatch.setattr(moe, "Workspace", Workspace)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: m.current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: m.recorded.setdefault(m.key(t), set()).add(s))
    m.stream("main")
    with Operations():
        yield m, moe.ExpertLayer


def inputs(T=6, k=2, E=3, W=32, H=32):
    g = torch.Generator().manual_seed(1)
    return (torch.randn(E, 2 * H, W, generator=g).bfloat16(), torch.randn(E, W, H, generator=g).bfloat16(),
            torch.randn(T, W, generator=g).bfloat16(), torch.randint(0, E, (T, k), generator=g, dtype=torch.int32),
            torch.rand(T, k, generator=g), torch.randn(T, W, generator=g).bfloat16())


def test_the_model_sees_mistakes(model):
    m, _ = model
    main, side = m.current, m.stream("side")
    t = torch.zeros(4)
    m.touch("read", side, t)
    assert len(m.faults) == 2  # not ordered, and the memory is main's
    side.wait_stream(main)
    t.record_stream(side)
    m.faults.clear()
    m.touch("read", side, t)
    assert not m.faults
    u = torch.ones(4)
    u.record_stream(side)
    m.touch("read", side, u)
    assert len(m.faults) == 1  # made after the wait


def test_current_stream(model):
    m, Layer = model
    w_in, w_out, x, ids, w, dy = inputs()
    layer = Layer(w_in, w_out)
    y, saved = layer.forward(x, ids, w)
    layer.backward(saved, dy)
    assert not m.faults, m.faults


@pytest.mark.parametrize("transposed", [False, True])
def test_another_stream(model, transposed):
    m, Layer = model
    w_in, w_out, x, ids, w, dy = inputs()
    if transposed:  # load has to copy it
        w_in = w_in.transpose(1, 2).contiguous().transpose(1, 2)
    main, side = m.current, m.stream("side")
    layer = Layer(w_in, w_out)
    layer.load(w_in, w_out, stream=side)
    main.wait_stream(side)
    y, saved = layer.forward(x, ids, w, stream=side)
    grads = layer.backward(saved, dy, stream=side)
    assert not m.faults, m.faults
    # what comes back is the side stream's
    assert m.current is main
    for t in (y, *grads):
        assert m.home[m.key(t)] is side


def test_a_stream_for_each_call(model):
    """Weights loaded, a forward and a backward pass on three streams, each
    ordered by the caller's."""
    m, Layer = model
    w_in, w_out, x, ids, w, dy = inputs()
    main = m.current
    layer = Layer(w_in, w_out)
    for i in range(2):
        a, b, c = (m.stream(n + str(i)) for n in "abc")
        layer.load(w_in, w_out, stream=a)
        main.wait_stream(a)
        y, saved = layer.forward(x, ids, w, stream=b)
        main.wait_stream(b)
        layer.backward(saved, dy, stream=c)
        main.wait_stream(c)
        layer.forward(x, ids, w, train=False)
        assert not m.faults, m.faults


def test_current_stream_changed_between_calls(model):
    m, Layer = model
    w_in, w_out, x, ids, w, dy = inputs()
    main, side = m.current, m.stream("side")
    layer = Layer(w_in, w_out)
    y, saved = layer.forward(x, ids, w)
    side.wait_stream(main)
    with torch.cuda.stream(side):
        for t in (x, ids, w, dy):  # the caller's tensors are the caller's to record
            t.record_stream(side)
        layer.backward(saved, dy)
        layer.forward(x, ids, w)
    assert not m.faults, m.faults
