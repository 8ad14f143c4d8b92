"""RMSNorm with the residual's addition (moe_rmsnorm) against a plain
implementation in 64 bits.

Tolerances. s is one fp32 addition rounded to the stream's type: equal to the
rounded 64-bit sum except where the fp32 addition itself rounds, so at most one
step of the type. y: the fp32 sum of D squares is off by less than D * 2^-24
relative (in fact far less), rsqrt by 2 ulp and two products by one rounding
each, under 2^-18 together for D <= 16384; bf16 output adds half a step, 2^-8.
q: half a step of E4M3 (2^-4 of the value, or 2^-10 absolute below the smallest
normal 2^-6) of y / c, whose own error is again under 2^-17."""
import pytest
import torch

import mixture_experts_ffn_layer_b200 as moe

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _inputs(T, D, ldx, res, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, ldx), generator=g, device="cuda").to(BF16)[:, :D]
    gamma = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(BF16)
    residual = None if res is None else (3 * torch.randn((T, D), generator=g, device="cuda")).to(res)
    return x, gamma, residual


def _stream(x, residual):
    return x.double() if residual is None else (x.double() + residual.double()).to(residual.dtype)


def _norm(s, gamma, eps):
    s = s.double()
    return s / torch.sqrt(s.pow(2).mean(1, keepdim=True) + eps) * gamma.double()


def _check_res(res, x, residual):
    if residual is None:
        assert res is None
        return
    exact = x.double() + residual.double()
    assert res.dtype == residual.dtype
    assert bool(((res.double() - exact).abs() <= torch.finfo(res.dtype).eps * exact.abs()).all())


SHAPES = [(1, 16, 16), (1, 2880, 2880), (3, 64, 80), (257, 2880, 2880), (5, 4112, 6208), (2, 8192, 8192),
          (2, 8208, 8208), (3, 16384, 16400), (130, 208, 224), (1000, 144, 144)]


@pytest.mark.parametrize("res", [None, BF16, F32])
@pytest.mark.parametrize("T,D,ldx", SHAPES)
def test_bf16_output(T, D, ldx, res):
    x, gamma, residual = _inputs(T, D, ldx, res, T + D)
    y, s = moe.rmsnorm(x, gamma, 1e-5, residual=residual)
    _check_res(s, x, residual)
    ref = _norm(x if s is None else s, gamma, 1e-5)
    assert bool(((y.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -17) * ref.abs()).all())


@pytest.mark.parametrize("res", [None, BF16, F32])
@pytest.mark.parametrize("T,D,ldx", SHAPES)
def test_e4m3_output(T, D, ldx, res):
    x, gamma, residual = _inputs(T, D, ldx, res, 7 * T + D)
    q, scale, s = moe.rmsnorm_fp8(x, gamma, 1e-5, residual=residual)
    _check_res(s, x, residual)
    ref = _norm(x if s is None else s, gamma, 1e-5)
    nb = -(-D // 128)
    blocks = torch.nn.functional.pad(ref, (0, nb * 128 - D)).view(T, nb, 128)
    c = blocks.abs().amax(-1).clamp_min(2.0 ** -100) / 448
    assert scale.shape == (T, nb)
    assert bool(((scale.double() - c).abs() <= 2.0 ** -17 * c).all())
    want = ref / c.repeat_interleave(128, 1)[:, :D]
    got = q.to(F32).double()
    assert bool(((got - want).abs() <= (2.0 ** -4 + 2.0 ** -16) * want.abs().clamp_min(2.0 ** -6)).all())


def test_both_outputs_and_in_place_residual():
    # y and q of one call are those of two calls, bit for bit; the residual may
    # be updated in place; row and column neighbours of the outputs stay
    T, D = 33, 2880
    x, gamma, residual = _inputs(T, D, D, BF16, 5)
    y1, s1 = moe.rmsnorm(x, gamma, 1e-6, residual=residual)
    q1, c1, _ = moe.rmsnorm_fp8(x, gamma, 1e-6, residual=residual)
    ybuf = torch.full((T + 2, D), 7.0, dtype=BF16, device="cuda")
    qbuf = torch.full((T + 2, D), 3, dtype=torch.uint8, device="cuda")
    cbuf = torch.full((T * 23 + 16,), -1.0, device="cuda")
    r = residual.clone()
    n = moe.NormDims(T, D, D, 1e-6, moe.MOE_T_BF16)
    moe.moe_rmsnorm(n, x, r, gamma, r, ybuf[1:T + 1], qbuf[1:T + 1].view(E4M3), cbuf)
    assert torch.equal(r, s1) and torch.equal(ybuf[1:T + 1], y1)
    assert torch.equal(qbuf[1:T + 1], q1.view(torch.uint8)) and torch.equal(cbuf[:T * 23].view(T, 23), c1)
    assert bool((ybuf[0] == 7).all() and (ybuf[-1] == 7).all() and (qbuf[0] == 3).all() and (qbuf[-1] == 3).all())
    assert bool((cbuf[T * 23:] == -1).all())


def test_no_stream_written_without_res_out():
    T, D = 4, 256
    x, gamma, residual = _inputs(T, D, D, F32, 9)
    before = residual.clone()
    y = torch.empty((T, D), dtype=BF16, device="cuda")
    moe.moe_rmsnorm(moe.NormDims(T, D, D, 1e-5, moe.MOE_T_F32), x, residual, gamma, None, y, None, None)
    assert torch.equal(residual, before)
    assert torch.equal(y, moe.rmsnorm(x, gamma, 1e-5, residual=residual)[0])


def test_zeros_tiny_huge_and_nan_rows():
    D = 384
    x = torch.zeros((6, D), dtype=BF16, device="cuda")
    x[1] = 2.0 ** -120  # squares vanish in fp32: eps alone sets the norm
    x[2, 5] = 2.0 ** 60
    x[3] = 1.0
    x[3, 200] = float("nan")
    x[4, 0] = float("inf")
    x[5, 128:256] = 1.0  # a quantisation block beside two of zeros
    gamma = torch.ones(D, dtype=BF16, device="cuda")
    y, _ = moe.rmsnorm(x, gamma, 1e-5)
    q, scale, _ = moe.rmsnorm_fp8(x, gamma, 1e-5)
    assert bool((y[0] == 0).all()) and bool((q[0].float() == 0).all())
    assert bool((scale[0].double() - 2.0 ** -100 / 448).abs().max() <= 2.0 ** -120)
    ref = _norm(x[[1, 2, 5]], gamma, 1e-5)
    assert bool(((y[[1, 2, 5]].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -17) * ref.abs()).all())
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(q[3].float()).all())
    assert bool(torch.isnan(y[4, 0])) and bool(torch.isnan(q[4, 0].float()))
    assert bool((q[5].float()[128:256] == 448).all()) and bool((q[5].float()[256:] == 0).all())


def test_no_rows():
    x, gamma, residual = _inputs(0, 128, 128, BF16, 1)
    y, s = moe.rmsnorm(x, gamma, residual=residual)
    assert y.shape == (0, 128) and s.shape == (0, 128)


def test_other_stream_and_graph():
    T, D = 19, 2880
    x, gamma, residual = _inputs(T, D, D, BF16, 3)
    want_y, want_s = moe.rmsnorm(x, gamma, residual=residual)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, s = moe.rmsnorm(x, gamma, residual=residual, stream=side)
    side.synchronize()
    assert torch.equal(y, want_y) and torch.equal(s, want_s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = moe.rmsnorm(x, gamma, residual=residual)
    x2 = torch.randn((T, D), device="cuda").to(BF16)
    x.copy_(x2)
    graph.replay()
    want_y, want_s = moe.rmsnorm(x2, gamma, residual=residual)
    assert torch.equal(y, want_y) and torch.equal(s, want_s)


def test_quotients_next_to_a_border():
    # rows of +-1 leave y = +-gamma exactly, and c = 49 / 448 is a number of few
    # bits: gamma = 7/64 * m has the quotient m exactly, half-way between two
    # neighbours of E4M3 for these m, and goes to the even one. (y * (448 / 49) in
    # fp32 lies above half-way for m = 23 and up.)
    D = 256
    m = torch.arange(17, 33, 2, device="cuda", dtype=F32)
    gamma = torch.full((D,), 7 / 64, device="cuda")
    for block in (0, 128):
        gamma[block] = 49.0
        gamma[block + 1:block + 9] = 7 / 64 * m
        gamma[block + 9:block + 17] = 7 / 64 * m / 8
    assert torch.equal(gamma.to(BF16).float(), gamma)
    x = torch.ones((3, D), dtype=BF16, device="cuda")
    x[1] = -1.0
    x[2, ::2] = -1.0
    q, scale, _ = moe.rmsnorm_fp8(x, gamma.to(BF16), 0.0)
    assert bool((scale == 49 / 448).all())
    even = torch.tensor([16, 20, 20, 24, 24, 28, 28, 32], device="cuda", dtype=F32)  # of 17, 19, ... 31
    for row in range(3):
        for block in (0, 128):
            sign = x[row, block + 1:block + 9].float()
            assert torch.equal(q[row, block + 1:block + 9].float(), sign * even)
            sign = x[row, block + 9:block + 17].float()
            assert torch.equal(q[row, block + 9:block + 17].float(), sign * even / 8)


def test_nonfinite_values_reach_the_scale():
    # c = max|y| / 448 of a block with a NaN is NaN, and so are its codes
    D = 384
    x = torch.ones((4, D), dtype=BF16, device="cuda")
    x[0, 200] = float("nan")
    x[1, 130] = float("inf")
    x[2, 383] = float("-inf")
    gamma = torch.ones(D, dtype=BF16, device="cuda")
    y, _ = moe.rmsnorm(x, gamma)
    q, scale, _ = moe.rmsnorm_fp8(x, gamma)
    assert bool(torch.isnan(y[0]).all()) and bool(torch.isnan(q[0].float()).all())
    assert bool(torch.isnan(scale[0]).all())
    for row, col in ((1, 130), (2, 383)):
        bad = torch.arange(D, device="cuda") // 128 == col // 128
        assert bool(torch.isnan(y[row, col])) and int(torch.isnan(y[row]).sum()) == 1
        assert torch.equal(torch.isnan(scale[row]), bad[::128])
        assert torch.equal(torch.isnan(q[row].float()), bad)
        assert bool((q[row].float()[~bad] == 0).all())
        assert bool((scale[row][~bad[::128]].double() - 2.0 ** -100 / 448).abs().max() <= 2.0 ** -120)
    # y beyond fp32: an infinite scale, beside which finite y are zero
    gamma[5] = 3e38
    x[3, 5] = 8.0
    q, scale, _ = moe.rmsnorm_fp8(x[3:], gamma)
    assert bool(torch.isinf(scale[0, 0])) and bool(torch.isnan(q[0, 5].float()))
    keep = [c for c in range(128) if c != 5]
    assert bool((q[0].float()[keep] == 0).all())
    assert bool(torch.isfinite(scale[0, 1:]).all()) and bool((q[0].float()[128:] == 448).all())
