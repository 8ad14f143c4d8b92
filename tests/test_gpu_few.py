"""The one-launch layer for a few tokens (moe_forward_few) against the oracle.

Tolerance: y_ref is the oracle's output before its final bf16 rounding, in
fp64 with h rounded to bf16. The kernel's sums are fp32 (errors near 1e-6 of
the sums' rms), so an h element lies on the other side of a rounding border
only now and then; one such element, at four times the rms of h and three
times that of W2, moves an output by 12 / sqrt(I) * 2^-8 of its rms, 6e-3 for
the smallest I = 64; the gate weights are off by under 1e-5. So
|y - y_ref| <= 2^-8 |y_ref| (y's own rounding) + 8e-3 rms(y_ref)."""
import dataclasses

import pytest
import torch

import mixture_experts_ffn_layer_b200 as moe
import oracle
import synthetic
from helpers import SWIGLU, dims_of

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
GPTOSS = (moe.MOE_ACT_GPTOSS, 1.702, 7.0)


def _few(inp, act=SWIGLU, ws=None, y=None, stream=None):
    s = inp.shape
    d = dims_of(inp, act)
    ws = moe.alloc_workspace(d) if ws is None else ws
    y = torch.full((s.T, s.D), float("nan"), dtype=BF16, device="cuda") if y is None else y
    moe.moe_forward_few(d, inp.x, inp.Wr, inp.br, inp.W1, inp.b1, inp.W2, inp.b2, y, ws, W1_scales=inp.W1_scales,
                        W2_scales=inp.W2_scales, stream=stream)
    return y, ws


def _ref(inp, act=SWIGLU):
    _, idx, w = oracle.route(inp.x, inp.Wr, inp.br, inp.shape.k)
    return oracle.ffn_tokens(inp.x, idx, w, inp.W1, inp.b1, inp.W2, inp.b2, W1_scales=inp.W1_scales,
                             W2_scales=inp.W2_scales, return_exact=True, act=act)[1]


def _close(y, ref):
    y, ref = y.double().cpu(), ref.double().cpu()
    bound = 2.0 ** -8 * ref.abs() + 8e-3 * ref.pow(2).mean().sqrt()
    assert bool(((y - ref).abs() <= bound).all()), float(((y - ref).abs() / bound).max())


def _make(T, D, E, k, I, wfmt, seed=0):
    return synthetic.make_custom(T, D, E, k, I, seed=seed + T + 3 * E, device="cuda", wfmt=wfmt,
                                 reject=oracle.gap_reject())


@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,D,E,k,I,act", [
    (1, 64, 1, 1, 64, SWIGLU),          # one expert, fewer granules than SMs, two units of 32
    (1, 256, 8, 2, 128, GPTOSS),
    (2, 192, 4, 4, 320, SWIGLU),        # k = E
    (16, 64, 2, 2, 64, GPTOSS),         # every token on both experts: 16 rows each
    (8, 1088, 16, 3, 704, SWIGLU),      # the last size of one column group
    (9, 704, 16, 3, 1088, SWIGLU),      # the first of two
    (16, 192, 256, 8, 320, SWIGLU),     # largest E and k: up to 128 active experts
    (5, 2880, 32, 4, 2880, GPTOSS),
    (16, 4096, 4, 2, 128, SWIGLU),      # the most resident activations: 16 x 4096
    (4, 16384, 2, 1, 64, SWIGLU),       # the longest reductions, several stages per granule
    (3, 64, 3, 2, 16384, GPTOSS),
    (7, 2880, 8, 2, 512, SWIGLU),       # MXFP4: W1's rows copied as they lie, W2's one by one
    (13, 512, 8, 2, 704, GPTOSS),       # and the other way round
])
def test_shapes(T, D, E, k, I, act, wfmt):
    inp = _make(T, D, E, k, I, wfmt)
    y, ws = _few(inp, act)
    assert moe.moe_read_device_status(ws) == 0
    _close(y, _ref(inp, act))


@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
def test_every_token_count(wfmt):
    full = _make(16, 320, 8, 2, 192, wfmt)
    ref = _ref(full)
    for T in range(1, 17):
        inp = dataclasses.replace(full, shape=dataclasses.replace(full.shape, T=T), x=full.x[:T].contiguous())
        y, ws = _few(inp)
        _close(y, ref[:T])


@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
def test_experts_with_few_and_with_many_tokens(wfmt):
    # one expert takes every token (two groups of 8), the others a few (one)
    inp = _make(16, 448, 24, 3, 320, wfmt)
    br = torch.zeros(24)
    br[11] = 30.0
    inp = dataclasses.replace(inp, br=br.to(BF16).cuda())
    if bool(oracle.gap_reject()(inp.x, inp.Wr, inp.br, 3).any()):
        pytest.skip("a token's routing is not unique under reassociation")
    y, _ = _few(inp)
    _close(y, _ref(inp))


@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
def test_all_tokens_on_the_same_experts(wfmt):
    inp = _make(16, 2880, 32, 4, 256, wfmt)
    br = torch.zeros(32)
    br[[3, 17, 30, 31]] = torch.tensor([40.0, 50.0, 60.0, 70.0])
    inp = dataclasses.replace(inp, br=br.to(BF16).cuda())
    y, _ = _few(inp)
    _close(y, _ref(inp))


@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("D,I", [(64, 64), (192, 320), (2880, 704), (1024, 2880)])
def test_every_number_of_rows_per_expert(D, I, wfmt):
    # every token on every expert: 1 to 16 rows each, over reductions of 2 to 90
    # units of 32 that do not divide evenly among the warps
    full = _make(16, D, 3, 3, I, wfmt)
    ref = _ref(full)
    for T in (1, 2, 3, 4, 5, 8, 9, 15, 16):
        inp = dataclasses.replace(full, shape=dataclasses.replace(full.shape, T=T), x=full.x[:T].contiguous())
        y, ws = _few(inp)
        assert moe.moe_read_device_status(ws) == 0
        _close(y, ref[:T])


@pytest.mark.parametrize("T", [2, 4, 7])
def test_nonfinite_token_among_those_of_its_experts(T):
    # the tokens share an MMA's columns with several units of the reduction
    inp = _make(T, 320, 2, 2, 192, "mxfp4")
    ref = _ref(inp)
    inp.x[1, 5] = float("nan")
    inp.x[1, 300] = float("inf")
    y, _ = _few(inp)
    keep = [t for t in range(T) if t != 1]
    _close(y[keep], ref[keep])
    assert bool(torch.isnan(y[1]).all())


def test_ties_go_to_the_lower_expert():
    inp = _make(6, 128, 40, 3, 64, "bf16")
    inp.Wr.zero_()
    inp.br.zero_()
    inp.br[[7, 33]] = 1.0  # then 7, 33 and the lowest of the others, 0
    y, _ = _few(inp)
    idx = torch.tensor([[7, 33, 0]] * 6, dtype=torch.int32)
    w = torch.softmax(torch.tensor([[1.0, 1.0, 0.0]] * 6), 1)
    _close(y, oracle.ffn_tokens(inp.x, idx, w, inp.W1, inp.b1, inp.W2, inp.b2, return_exact=True)[1])


@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
def test_nonfinite_token_reaches_only_itself(wfmt):
    inp = _make(12, 256, 8, 2, 128, wfmt)
    ref = _ref(inp)
    inp.x[4, 17] = float("nan")
    inp.x[9, 200] = float("inf")
    y, ws = _few(inp)
    assert moe.moe_read_device_status(ws) == 0
    keep = [t for t in range(12) if t not in (4, 9)]
    _close(y[keep], ref[keep])
    assert bool(torch.isnan(y[4]).all())
    assert not bool(torch.isfinite(y[9]).any())


@pytest.mark.parametrize("e", [-100, -60, 12])
def test_mxfp4_rows_of_any_magnitude(e):
    # activations far from f16's range: a row's power-of-two scale carries them
    # (an identity-like activation so that h has the same range: act_limit inf)
    inp = _make(5, 192, 4, 2, 128, "mxfp4")
    inp.Wr.zero_()
    inp.br.copy_(torch.tensor([3.0, 2.0, 1.0, 0.0]))
    inp.b1.zero_()
    inp.b1[:, :128] = 1.0  # a gate near 1 keeps h linear in the up half for tiny rows
    inp.b2.zero_()
    inp.x[0] *= 2.0 ** 20
    inp.x[1:] *= 2.0 ** e
    inp.x[4, 100:] *= 2.0 ** -30  # a wide range inside one row
    y, _ = _few(inp)
    ref = _ref(inp)
    for t in range(5):
        _close(y[t:t + 1], ref[t:t + 1])


def test_mxfp4_scales_of_any_size():
    # scale bytes from 2^-127 up; the outputs' own scale is set by the largest
    inp = _make(3, 256, 4, 2, 128, "mxfp4")
    g = torch.Generator(device="cuda").manual_seed(1)
    inp.W1_scales.copy_(torch.randint(0, 128, inp.W1_scales.shape, generator=g, device="cuda"))
    inp.W2_scales.copy_(torch.randint(0, 140, inp.W2_scales.shape, generator=g, device="cuda"))
    y, _ = _few(inp)
    _close(y, _ref(inp))


@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
def test_repeatable_on_a_shared_workspace(wfmt):
    # call after call, with other sizes and the batched layer on the same
    # workspace between them: the same bits
    inp = _make(16, 704, 16, 4, 320, wfmt)
    small = dataclasses.replace(inp, shape=dataclasses.replace(inp.shape, T=3), x=inp.x[:3].contiguous())
    y, ws = _few(inp)
    ys, _ = _few(small)
    d = dims_of(inp)
    for _ in range(3):
        assert torch.equal(_few(small, ws=ws)[0], ys)
        z = torch.empty_like(y)
        moe.moe_forward(d, inp.x, inp.Wr, inp.br, inp.W1, inp.b1, inp.W2, inp.b2, z, ws, W1_scales=inp.W1_scales,
                        W2_scales=inp.W2_scales)
        assert torch.equal(_few(inp, ws=ws)[0], y)
    assert moe.moe_read_device_status(ws) == 0


def test_two_streams_and_graphs():
    # two workspaces on two streams at once; two captured graphs that share one
    a, b = _make(4, 512, 16, 4, 512, "bf16"), _make(11, 512, 16, 4, 512, "mxfp4")
    ya, ws_a = _few(a)
    yb, ws_b = _few(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        outs.append((_few(a, ws=ws_a, stream=s1)[0], _few(b, ws=ws_b, stream=s2)[0]))
    torch.cuda.synchronize()
    # (the NaN fill of y ran on the default stream: compare a second pass with outputs made before)
    za, zb = torch.empty_like(ya), torch.empty_like(yb)
    torch.cuda.synchronize()
    for _ in range(20):
        _few(a, ws=ws_a, y=za, stream=s1)
        _few(b, ws=ws_b, y=zb, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(za, ya) and torch.equal(zb, yb)
    d = dims_of(b)
    ws = moe.alloc_workspace(d)
    ws = torch.zeros(max(ws.numel(), ws_a.numel()), dtype=torch.uint8, device="cuda")
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    za.zero_()
    zb.zero_()
    with torch.cuda.graph(g1):
        _few(a, ws=ws, y=za)
    with torch.cuda.graph(g2):
        _few(b, ws=ws, y=zb)
    for _ in range(4):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(za, ya) and torch.equal(zb, yb)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [2, 40])
def test_block_of_norm_and_layer(T, wfmt):
    # residual addition, norm and layer as a transformer block runs them, few
    # and many tokens, against the oracle on the norm's own output
    inp = _make(T, 320, 8, 2, 192, wfmt)
    scales = {} if wfmt == "bf16" else dict(W1_scales=inp.W1_scales, W2_scales=inp.W2_scales)
    layer = moe.MoELayer(inp.Wr, inp.br, inp.W1, inp.b1, inp.W2, inp.b2, k=2, **scales)
    g = torch.Generator(device="cuda").manual_seed(T)
    gamma = (1 + 0.1 * torch.randn(320, generator=g, device="cuda")).to(BF16)
    residual = torch.randn((T, 320), generator=g, device="cuda").to(BF16)
    y, s = moe.MoEBlock(layer, gamma)(inp.x, residual)
    assert layer.device_status() == 0
    assert torch.equal(s, (inp.x.float() + residual.float()).to(BF16))
    n, _ = moe.rmsnorm(s, gamma)
    _, idx, w = oracle.route(n, inp.Wr, inp.br, 2)
    if bool(oracle.gap_reject()(n, inp.Wr, inp.br, 2).any()):
        pytest.skip("a token's routing is not unique under reassociation")
    ref = oracle.ffn_tokens(n, idx, w, inp.W1, inp.b1, inp.W2, inp.b2, return_exact=True, **scales)[1]
    if T == 2:
        _close(y, ref)
    else:
        y, ref = y.double().cpu(), ref.double()
        assert float((y - ref).abs().max()) <= (2e-2 if wfmt == "bf16" else 6e-2) * float(ref.pow(2).mean().sqrt())
    want = layer.forward_few(n) if T == 2 else layer(n)
    assert torch.equal(y if T == 2 else y.to(BF16).cuda(), want)


def test_two_host_threads():
    # calls of different sizes from two threads at once, each with its own
    # stream and workspace
    import threading
    cases = [_make(1, 512, 16, 4, 512, "mxfp4"), _make(7, 1024, 16, 4, 2048, "mxfp4")]
    want = [_few(c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def run(inp, y, ws):
        try:
            stream = torch.cuda.Stream()
            out = torch.empty_like(y)
            for _ in range(50):
                _few(inp, ws=ws, y=out, stream=stream)
            stream.synchronize()
            if not torch.equal(out, y):
                bad.append("differs")
        except Exception as err:
            bad.append(repr(err))

    threads = [threading.Thread(target=run, args=(c, y, ws)) for c, (y, ws) in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []
    for _, ws in want:
        assert moe.moe_read_device_status(ws) == 0


def test_two_graphs_at_once():
    # captured calls with a workspace each, replayed on two streams at once
    cases = [_make(2, 512, 16, 4, 512, "mxfp4"), _make(9, 448, 8, 2, 704, "bf16")]
    want = [_few(c) for c in cases]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, (y, ws) in zip(cases, want):
        out, graph = torch.zeros_like(y), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                _few(c, ws=ws, y=out)
        graphs.append(graph)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for out, (y, ws) in zip(outs, want):
        assert moe.moe_read_device_status(ws) == 0
        assert torch.equal(out, y)


@pytest.mark.parametrize("T", [5, 12, 40, 300])
@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("half", ["gate", "up"])
def test_nan_of_an_expert_passes_the_clamps(half, wfmt, T):
    # a NaN in one expert's bias reaches every token of that expert and no other,
    # through the GPT-OSS activation too, few tokens or many
    inp = _make(T, 256, 8, 2, 128, wfmt)
    _, idx, w = oracle.route(inp.x, inp.Wr, inp.br, 2)
    expert = int(idx[0, 0])
    inp.b1[expert, 7 if half == "gate" else 128 + 7] = float("nan")
    hit = (idx == expert).any(1)
    assert not bool(hit.all())
    d = dims_of(inp, GPTOSS)
    if T <= 16:
        y, ws = _few(inp, GPTOSS)
    else:
        y, ws = torch.empty_like(inp.x), moe.alloc_workspace(d)
        moe.moe_forward(d, inp.x, inp.Wr, inp.br, inp.W1, inp.b1, inp.W2, inp.b2, y, ws, W1_scales=inp.W1_scales,
                        W2_scales=inp.W2_scales)
    assert moe.moe_read_device_status(ws) == 0
    assert torch.equal(torch.isnan(y).all(1).cpu(), hit) and not bool(torch.isnan(y.cpu()[~hit]).any())
    if T <= 16:
        ref = _ref(dataclasses.replace(inp, b1=torch.nan_to_num(inp.b1)), GPTOSS)
        _close(y.cpu()[~hit], ref[~hit])


@pytest.mark.parametrize("wfmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 6, 16])
def test_infinite_hidden_unit_beside_large_finite_ones(T, wfmt):
    # h from the biases alone: one unit overflows to infinity, another is -1e30;
    # outputs that weigh both with 1 or -1 are infinite, not NaN
    D, I = 128, 64
    inp = _make(T, D, 1, 1, I, wfmt)
    inp.b1.zero_()
    inp.b1[0, 0], inp.b1[0, I] = 1e30, 1e30
    inp.b1[0, 1], inp.b1[0, I + 1] = 1e20, -1e10
    inp.b2.zero_()
    inp.W1.zero_()
    if wfmt == "mxfp4":
        inp.W1_scales.fill_(127)
        inp.W2_scales.fill_(127)
        inp.W2.zero_()
        inp.W2[0, ::2, 0] = 0x22   # codes of 1 for units 0 and 1
        inp.W2[0, 1::2, 0] = 0xAA  # of -1
    else:
        inp.W2.zero_()
        inp.W2[0, ::2, :2], inp.W2[0, 1::2, :2] = 1.0, -1.0
    y, ws = _few(inp)
    assert moe.moe_read_device_status(ws) == 0
    want = torch.full((T, D), float("inf"), dtype=BF16, device="cuda")
    want[:, 1::2] *= -1
    assert torch.equal(y, want)


def _every_pass(cases, passes, run):
    """run(workspaces, outputs) fills `passes` outputs of each case, every one of
    which is compared with that of a single call."""
    want = [_few(c) for c in cases]
    outs = [[torch.zeros_like(y) for _ in range(passes)] for y, _ in want]
    torch.cuda.synchronize()
    run([ws for _, ws in want], outs)
    torch.cuda.synchronize()
    for (y, ws), got in zip(want, outs):
        assert moe.moe_read_device_status(ws) == 0
        assert all(torch.equal(out, y) for out in got)


def test_two_streams_every_pass():
    cases = [_make(4, 512, 16, 4, 512, "bf16"), _make(11, 512, 16, 4, 512, "mxfp4")]
    streams = [torch.cuda.Stream() for _ in cases]

    def run(spaces, outs):
        for i in range(200):
            for c, ws, out, stream in zip(cases, spaces, outs, streams):
                _few(c, ws=ws, y=out[i], stream=stream)

    _every_pass(cases, 200, run)


def test_two_graphs_on_one_workspace_every_pass():
    cases = [_make(4, 512, 16, 4, 512, "bf16"), _make(11, 512, 16, 4, 512, "mxfp4")]
    shared = torch.zeros(max(moe.workspace_bytes(dims_of(c)) for c in cases), dtype=torch.uint8, device="cuda")

    def run(_, outs):
        graphs, into = [], [torch.zeros_like(out[0]) for out in outs]
        for c, y in zip(cases, into):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                _few(c, ws=shared, y=y)
        for i in range(100):
            for graph, y, out in zip(graphs, into, outs):
                graph.replay()
                out[i].copy_(y)

    _every_pass(cases, 100, run)
    assert moe.moe_read_device_status(shared) == 0


def test_two_graphs_at_once_every_pass():
    cases = [_make(2, 512, 16, 4, 512, "mxfp4"), _make(9, 448, 8, 2, 704, "bf16")]
    streams = [torch.cuda.Stream() for _ in cases]

    def run(spaces, outs):
        graphs = []
        for c, ws, out in zip(cases, spaces, outs):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                for y in out:
                    _few(c, ws=ws, y=y)
        torch.cuda.synchronize()
        for _ in range(5):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()

    _every_pass(cases, 20, run)


def test_two_host_threads_every_pass():
    import threading
    cases = [_make(1, 512, 16, 4, 512, "mxfp4"), _make(7, 1024, 16, 4, 2048, "mxfp4")]
    failed = []

    def run(spaces, outs):
        def calls(inp, ws, out):
            try:
                stream = torch.cuda.Stream()
                for y in out:
                    _few(inp, ws=ws, y=y, stream=stream)
                stream.synchronize()
            except Exception as err:
                failed.append(repr(err))

        threads = [threading.Thread(target=calls, args=a) for a in zip(cases, spaces, outs)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()

    _every_pass(cases, 100, run)
    assert failed == []
