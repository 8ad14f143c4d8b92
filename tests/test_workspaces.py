"""The workspaces that MoELayer keeps: what a call on another stream, a captured
one, or one for more tokens leaves to the others."""
import ctypes
import gc
import weakref

import pytest
import torch

import mixture_experts_ffn_layer_b200 as moe
from mixture_experts_ffn_layer_b200 import _binding
from test_abi import _Arena

BF16 = torch.bfloat16


def _layer(E=4, D=64, I=64, k=2, device="cpu", seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: (0.1 * torch.randn(s, generator=g, device=device)).to(BF16)
    return moe.MoELayer(r(E, D), r(E), r(E, 2 * I, D), r(E, 2 * I), r(E, D, I), r(E, D), k)


@pytest.fixture
def used(monkeypatch):
    """The workspace of every call of the library, which is not made."""
    calls = []
    monkeypatch.setattr(moe, "_on", lambda t, call, *args, **kw: call(*args, **kw))
    monkeypatch.setattr(moe, "moe_forward_few", lambda *a, **kw: calls.append(a[9]))
    monkeypatch.setattr(moe, "moe_forward", lambda *a, **kw: calls.append(a[9]))
    return calls


def test_few_token_workspace_is_there_before_any_call_and_stays(used):
    layer = _layer()
    mine = layer._few_ws
    assert mine is not None and not bool(mine.any())
    few, many = torch.zeros((2, 64), dtype=BF16), torch.zeros((200, 64), dtype=BF16)
    for x, call in ((few, layer.forward_few), (many, layer.forward), (few, layer.forward_few),
                    (torch.zeros((16, 64), dtype=BF16), layer.forward_few), (few, layer.forward)):
        call(x)
    assert [ws is mine for ws in used] == [True, False, True, True, False]
    # enough for every number of tokens that it takes
    for T in range(1, layer.few_max_tokens + 1):
        assert moe.workspace_bytes(moe.dims(T, 64, 4, 2, 64)) <= mine.numel()


def test_few_token_workspace_of_mxfp4_is_the_bf16_layers():
    lib, ar = moe.load(), _Arena(64 << 20)
    d, dq = moe.dims(4, 64, 4, 2, 64), moe.dims(4, 64, 4, 2, 64, wfmt=moe.MOE_W_MXFP4)
    n = moe.workspace_bytes(d)
    assert n < moe.workspace_bytes(dq)
    ptr = [ctypes.c_void_p(ar.take()) for _ in range(6)]
    ws, W = ctypes.c_void_p(ar.take(n)), lambda: _binding.Weight(ar.take(), ar.take())
    w1, w2 = W(), W()
    x, wr, br, b1, b2, y = ptr
    assert lib.moe_forward_few(dq, x, wr, br, w1, b1, w2, b2, y, ws, n - 1, None) == 3
    # (enough bytes: the next thing that is refused is T, looked at first)
    assert lib.moe_forward_few(moe.dims(17, 64, 4, 2, 64, wfmt=moe.MOE_W_MXFP4), x, wr, br, w1, b1, w2, b2, y, ws, n,
                               None) == 2


def test_layer_without_a_one_launch_form():
    # sizes that no entry point takes: made as ever, refused by the calls
    layer = _layer(D=96)
    assert layer._few_ws is None
    with pytest.raises(moe.MoeError):
        layer.forward_few(torch.zeros((2, 96), dtype=BF16))


@pytest.mark.parametrize("captured", [False, True])
def test_larger_batch_keeps_a_captured_workspace(captured, used, monkeypatch):
    # what a graph writes to when it is replayed is not given back; what none
    # holds is
    layer, capturing = _layer(), [captured]
    monkeypatch.setattr(moe, "_capturing", lambda t: capturing[0])
    layer.forward(torch.zeros((40, 64), dtype=BF16))
    capturing[0] = False
    before = weakref.ref(used[0])
    used.clear()
    layer.forward(torch.zeros((500, 64), dtype=BF16))
    gc.collect()
    assert (before() is not None) == captured
    assert before() is None or before() is not used[0]


def test_workspace_recorded_into_a_graph_is_zeroed_for_other_calls(used, monkeypatch):
    # its zero-fill was recorded, not run
    layer, capturing = _layer(), [True]
    monkeypatch.setattr(moe, "_capturing", lambda t: capturing[0])
    x = torch.zeros((40, 64), dtype=BF16)
    layer.forward(x)
    used[0].fill_(7)
    capturing[0] = False
    layer.forward(x)
    assert used[1] is used[0] and not bool(used[1][:256].any())
    used[1][0] = 5  # an error that a kernel recorded
    layer.forward(x)
    assert int(used[2][0]) == 5


def test_workspace_is_marked_used_on_other_streams(used, monkeypatch):
    layer, at, marked = _layer(), [11], []
    monkeypatch.setattr(moe, "_stream_id", lambda t: at[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: at[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: marked.append(s), raising=False)
    x = torch.zeros((40, 64), dtype=BF16)
    layer.forward(x)
    assert marked == []
    at[0] = 12
    layer.forward(x)
    assert marked == [12]


def test_calls_run_with_the_layers_device_current(monkeypatch):
    where = []
    monkeypatch.setattr(moe, "_on", lambda t, call, *args, **kw: where.append((t.device, call)) or 0)
    layer, x = _layer(), torch.zeros((3, 64), dtype=BF16)
    layer.forward(x)
    layer.forward_few(x)
    layer.device_status()
    assert [call for _, call in where] == [moe.moe_forward, moe.moe_forward_few] + 2 * [moe.moe_read_device_status]
    assert all(device == x.device for device, _ in where)


def test_workspace_for_more_tokens_that_is_smaller(used):
    # beyond 18 tiles of 128 tokens the router keeps no partial sums
    more, fewer = 18 * 128 + 1, 18 * 128
    need = [moe.workspace_bytes(moe.dims(T, 512, 64, 1, 64)) for T in (more, fewer)]
    assert need[0] < need[1]
    layer = _layer(E=64, D=512, k=1)
    for T in (more, fewer):
        layer.forward(torch.zeros((T, 512), dtype=BF16))
    assert [ws.numel() for ws in used] == need


@pytest.mark.gpu
def test_captured_batch_outlives_a_larger_one():
    layer = _layer(E=8, D=320, I=192, device="cuda")
    x, big = (torch.randn((T, 320), device="cuda").to(BF16) for T in (40, 4000))
    want, y = layer(x), torch.zeros_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, out=y)
    n = layer._ws.numel()
    big_y = layer(big)
    others = [torch.full((n,), i + 1, dtype=torch.uint8, device="cuda") for i in range(8)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(layer(big), big_y)
    for i, t in enumerate(others):
        assert bool((t == i + 1).all())
    assert layer.device_status() == 0


@pytest.mark.gpu
def test_first_batch_in_a_graph():
    layer = _layer(E=8, D=320, I=192, device="cuda")
    x = torch.randn((40, 320), device="cuda").to(BF16)
    want, y = _layer(E=8, D=320, I=192, device="cuda")(x), torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, out=y)
    assert torch.equal(layer(x), want) and layer.device_status() == 0
    graph.replay()
    assert torch.equal(y, want) and layer.device_status() == 0


@pytest.mark.gpu
def test_status_of_another_stream():
    layer = _layer(E=8, D=320, I=192, device="cuda")
    x = torch.randn((40, 320), device="cuda").to(BF16)
    want = layer(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
    y2 = layer(x, stream=side)
    # an error on that stream, seen by reading the status there
    moe.moe_selftest_wait_timeout(layer._ws, 1000, stream=side)
    assert layer.device_status(side) == 5
    assert torch.equal(y2, want) and layer.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("first", ["captured", "other stream"])
def test_first_call_elsewhere(first):
    layer, x = _layer(E=16, D=512, I=256, device="cuda"), torch.randn((5, 512), device="cuda").to(BF16)
    want = _layer(E=16, D=512, I=256, device="cuda").forward_few(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if first == "captured":
        graph, y = torch.cuda.CUDAGraph(), torch.zeros_like(x)
        with torch.cuda.graph(graph):
            layer.forward_few(x, out=y)
        assert torch.equal(layer.forward_few(x), want)  # before any replay
        for _ in range(3):
            graph.replay()
            assert torch.equal(y, want)
    else:
        y = layer.forward_few(x, stream=side)
        side.synchronize()
        assert torch.equal(y, want)
    assert torch.equal(layer.forward_few(x), want)
    assert layer.device_status() == 0


@pytest.mark.gpu
def test_captured_block_outlives_a_larger_batch():
    # a decode step in a graph, then a long batch, whose workspace is another one,
    # and tensors that take what memory there is
    layer = _layer(E=8, D=320, I=192, device="cuda")
    run = moe.MoEBlock(layer, torch.ones(320, dtype=BF16, device="cuda"))
    x, r = (torch.randn((4, 320), device="cuda").to(BF16) for _ in range(2))
    want_y, want_s = run(x, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = run(x, r)
    big = torch.randn((3000, 320), device="cuda").to(BF16)
    big_y, _ = run(big, big)
    sizes = [4096, 65536, 1 << 20, layer._few_ws.numel()]
    others = [torch.full((n,), i + 1, dtype=torch.uint8, device="cuda") for i, n in enumerate(sizes * 8)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(s, want_s)
    for i, t in enumerate(others):
        assert bool((t == i + 1).all())
    assert torch.equal(run(big, big)[0], big_y)
    assert layer.device_status() == 0
