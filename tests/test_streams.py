"""Calls on a stream that is not the current one: what they allocate belongs to
that stream, so no buffer is in use on both without an order.

On the CPU the streams are stand-ins and the library's calls are recorded; a
dispatch mode sees every allocation."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import mixture_experts_ffn_layer_b200 as moe
from mixture_experts_ffn_layer_b200 import block

BF16 = torch.bfloat16
ALLOCATING = {"aten.empty", "aten.empty_like", "aten.new_empty", "aten.empty_strided", "aten.zeros", "aten.full"}


class _Stream:
    device = torch.device("cpu")
    cuda_stream = 0


class _Seen(TorchDispatchMode):
    """The current stream at every allocation."""

    def __init__(self, current):
        super().__init__()
        self.current, self.at = current, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if str(func).rsplit(".", 1)[0] in ALLOCATING:
            self.at.append(self.current[-1])
        return func(*args, **(kwargs or {}))


@pytest.fixture
def streams(monkeypatch):
    """current: the stack of current streams; launched: (entry point, its stream)
    of every call of the library; kept: streams that a result was marked used on."""
    current, launched, kept = [_Stream()], [], []

    @contextlib.contextmanager
    def switch(stream):
        current.append(stream)
        try:
            yield
        finally:
            current.pop()

    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: kept.append(s), raising=False)

    def recorder(name):
        def call(*args, **kw):
            given = [a for a in (*args, kw.get("stream")) if isinstance(a, _Stream)]
            launched.append((name, given[0] if given else current[-1]))
        return call

    here = lambda t, call, *args, **kw: call(*args, **kw)
    for module in (moe, block):
        monkeypatch.setattr(module, "_on", here)
    for name in ("moe_rmsnorm", "moe_fp8_matmul", "moe_forward_few", "moe_forward"):
        monkeypatch.setattr(block.B, name, recorder(name))
        monkeypatch.setattr(moe, name, recorder(name))
    return current, launched, kept


def _layer(E=4, D=64, I=64):
    z = lambda *s: torch.zeros(s, dtype=BF16)
    return moe.MoELayer(z(E, D), z(E), z(E, 2 * I, D), z(E, 2 * I), z(E, D, I), z(E, D), 2)


def _calls():
    x, gamma = torch.zeros((3, 64), dtype=BF16), torch.ones(64, dtype=BF16)
    many = torch.zeros((40, 64), dtype=BF16)
    f8 = torch.float8_e4m3fn
    fp8 = (torch.zeros((3, 64)).to(f8), torch.zeros((3, 1)), torch.zeros((1, 64, 64)).to(f8), torch.zeros((1, 1, 1)),
           torch.zeros(256, dtype=torch.uint8))
    layer = _layer()
    return {"rmsnorm": lambda s: moe.rmsnorm(x, gamma, residual=x, stream=s),
            "rmsnorm_fp8": lambda s: moe.rmsnorm_fp8(x, gamma, residual=x, stream=s),
            "fp8_matmul": lambda s: moe.fp8_matmul(*fp8, stream=s),
            "forward_few": lambda s: layer.forward_few(x, stream=s),
            "forward": lambda s: layer.forward(many, stream=s),
            "block, few": lambda s: moe.MoEBlock(layer, gamma)(x, x, stream=s),
            "block, many": lambda s: moe.MoEBlock(layer, gamma)(many, many, stream=s)}


@pytest.mark.parametrize("what", sorted(_calls()))
def test_buffers_belong_to_the_given_stream(what, streams):
    current, launched, kept = streams
    call = _calls()[what]
    other = _Stream()
    with _Seen(current) as seen:
        got = call(other)
    assert seen.at and all(s is other for s in seen.at)
    assert launched and all(s is other for _, s in launched)
    # what is handed back is the caller's stream's to use as well
    results = [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    assert len(kept) >= len(results) and all(s is current[0] for s in kept)


def test_a_stream_of_another_device_is_refused(streams):
    class Elsewhere(_Stream):
        device = torch.device("meta")

    for call in _calls().values():
        with pytest.raises(ValueError):
            call(Elsewhere())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
def test_block_on_another_stream(T):
    # the block runs behind a pause on its stream; meanwhile the current stream
    # takes and fills tensors of the sizes that the block has let go
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)
    E, D, I = 8, 320, 192
    layer = moe.MoELayer(rand(E, D), rand(E), rand(E, 2 * I, D), rand(E, 2 * I), rand(E, D, I), rand(E, D), 2)
    run = moe.MoEBlock(layer, 1 + rand(D))
    x, residual = rand(T, D), rand(T, D)
    want_y, want_s = run(x, residual)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        y, s = run(x, residual, stream=side)
        others = [torch.full((T, D), float(i), dtype=BF16, device="cuda") for i in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(s, want_s)
        for i, t in enumerate(others):
            assert bool((t == i).all())
    assert layer.device_status() == 0


@pytest.mark.gpu
def test_norm_and_product_on_another_stream():
    # buffers of the current stream that were let go while work there still reads
    # them are not written early by the other stream
    T, D, N = 64, 1024, 512
    x = torch.randn((T, D), device="cuda").to(BF16)
    gamma = torch.ones(D, dtype=BF16, device="cuda")
    w = torch.randn((1, N, D), device="cuda").to(torch.float8_e4m3fn)
    w_scale = torch.ones((1, N // 128, D // 128), device="cuda")
    ws = moe.alloc_fp8_workspace(moe.fp8_dims(T, 1, N, D))
    want = moe.fp8_matmul(*moe.rmsnorm_fp8(x, gamma)[:2], w, w_scale, ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        old = [torch.full((T, D), 1.0, dtype=BF16, device="cuda") for _ in range(4)]
        torch.cuda._sleep(2_000_000)
        sums = [t.float().sum() for t in old]
        del old
        q, scale, _ = moe.rmsnorm_fp8(x, gamma, stream=side)
        out = moe.fp8_matmul(q, scale, w, w_scale, ws, stream=side)
        y, _ = moe.rmsnorm(x, gamma, stream=side)
        torch.cuda.synchronize()
        assert all(float(v) == T * D for v in sums)
        assert torch.equal(out, want) and torch.equal(y, moe.rmsnorm(x, gamma)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
def test_block_on_a_forked_stream_of_a_capture(T):
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)
    E, D, I = 8, 320, 192
    layer = moe.MoELayer(rand(E, D), rand(E), rand(E, 2 * I, D), rand(E, 2 * I), rand(E, D, I), rand(E, D), 2)
    run = moe.MoEBlock(layer, 1 + rand(D))
    x, residual = rand(T, D), rand(T, D)
    want_y, want_s = run(x, residual)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        y, s = run(x, residual, stream=side)
        here.wait_stream(side)
        y2, s2 = run(y, s)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(s, want_s)
        again = run(want_y, want_s)
        assert torch.equal(y2, again[0]) and torch.equal(s2, again[1])
    assert layer.device_status() == 0
