"""The block-scaled FP8 product (moe_fp8_matmul) against its definition in 64
bits.

Tolerance: the products of E4M3 values are exact and a block's 128 of them are
summed in fp32, as are the ceil(K/128) blocks with their scales; each addition
rounds by at most 2^-24 of a partial sum, which is at most the sum of the
terms' magnitudes, S. With the two roundings of the scale product that is under
(128 + K/128 + 4) * 2^-24 * S, taken twice for tensor-core additions that cut
rather than round. A bf16 output adds half a step, 2^-8 of the value."""
import pytest
import torch

import mixture_experts_ffn_layer_b200 as moe

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _make(R, E, N, K, seed, bias=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    a = (40 * torch.randn((R, K), generator=g, device="cuda")).to(E4M3)
    w = (40 * torch.randn((E, N, K), generator=g, device="cuda")).to(E4M3)
    a_scale = torch.exp(torch.randn((R, kb), generator=g, device="cuda")) * 1e-2
    w_scale = torch.exp(torch.randn((E, nb, kb), generator=g, device="cuda")) * 1e-3
    b = torch.randn((E, N), generator=g, device="cuda").to(BF16) if bias else None
    return a, a_scale, w, w_scale, b


def _ref(a, a_scale, w, w_scale, b, offsets):
    """out and the sum of its terms' magnitudes, fp64; rows outside every segment are NaN."""
    R, K = a.shape
    E, N, _ = w.shape
    out = torch.full((R, N), float("nan"), dtype=torch.float64, device="cuda")
    mag = out.clone()
    A = a.double() * a_scale.double().repeat_interleave(128, 1)[:, :K]
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        W = w[e].double() * w_scale[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        out[lo:hi] = A[lo:hi] @ W.t()
        mag[lo:hi] = A[lo:hi].abs() @ W.abs().t()
        if b is not None:
            out[lo:hi] += b[e].double()
            mag[lo:hi] += b[e].double().abs()
    return out, mag


def _check(got, ref, mag, K, lo=0, hi=None):
    tol = 2 * (128 + K / 128 + 4) * 2.0 ** -24 * mag
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * ref.abs()
    bad = ~((got.double() - ref).abs() <= tol)[lo:hi]
    assert not bool(bad.any()), int(bad.sum())


def _run(R, E, N, K, offsets, dtype, bias=True, seed=0):
    a, a_scale, w, w_scale, b = _make(R, E, N, K, seed + R + E, bias)
    ref, mag = _ref(a, a_scale, w, w_scale, b, offsets)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ws = moe.alloc_fp8_workspace(moe.fp8_dims(R, E, N, K, dtype))
    out = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
    moe.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, bias=b, out=out)
    assert moe.moe_read_device_status(ws) == 0
    _check(out, ref, mag, K, 0, offsets[-1])
    assert bool((out[offsets[-1]:] == 7).all())  # rows behind the last segment
    return out


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,N,K", [(1, 16, 16), (1, 2880, 2880), (17, 272, 144), (32, 128, 128), (33, 64, 256),
                                   (128, 256, 128), (129, 400, 1040), (300, 2880, 2880), (1000, 528, 528),
                                   (513, 1040, 4096), (2100, 5760, 272)])  # (the last: 256-column tiles)
def test_dense(R, N, K, dtype):
    out = _run(R, 1, N, K, [0, R], dtype, bias=R != 128)
    a, a_scale, w, w_scale, b = _make(R, 1, N, K, R + 1, R != 128)
    ws = moe.alloc_fp8_workspace(moe.fp8_dims(R, 1, N, K, dtype))
    plain = moe.fp8_matmul(a, a_scale, w, w_scale, ws, bias=b, out_dtype=dtype)  # without offsets: all rows
    assert torch.equal(plain, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,N,K,extra", [
    ([3, 0, 5], 144, 272, 0),
    ([0, 0, 40, 1, 0], 272, 144, 3),              # empty first and last experts, rows behind the last segment
    ([32, 33, 31, 128, 129, 127, 1, 0], 528, 400, 0),
    ([700, 0, 257, 1], 272, 656, 5),              # wide tiles
    ([0, 0, 0], 64, 64, 4),                       # no rows at all in any segment
    ([2] * 256, 64, 128, 0),                      # the most experts
    ([400, 390, 0, 1, 600, 129, 128, 500], 2880, 144, 7),  # 256 columns
    ([1500, 0, 701], 4112, 400, 3),               # ragged in rows and columns
    ([0, 1793, 257, 1], 5120, 160, 0),
])
def test_grouped(counts, N, K, extra, dtype):
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    _run(offsets[-1] + extra, len(counts), N, K, offsets, dtype)


def test_experts_do_not_leak():
    # NaN weights of one expert and NaN rows of another reach only their own outputs
    counts, N, K = [5, 9, 4], 80, 208
    offsets = [0, 5, 14, 18]
    a, a_scale, w, w_scale, b = _make(18, 3, N, K, 3)
    ref, mag = _ref(a, a_scale, w, w_scale, b, offsets)
    w.view(torch.uint8)[1] = 0x7F
    a.view(torch.uint8)[16] = 0x7F
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ws = moe.alloc_fp8_workspace(moe.fp8_dims(18, 3, N, K))
    out = moe.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, bias=b, out_dtype=F32)
    keep = [0, 1, 2, 3, 4, 14, 15, 17]
    _check(out[keep], ref[keep], mag[keep], K)
    assert bool(torch.isnan(out[5:14]).all()) and bool(torch.isnan(out[16]).all())


@pytest.mark.parametrize("offsets", [[0, 9, 4, 12], [0, 4, 9, 13], [1, 4, 9, 12], [0, -1, 4, 12]])
def test_bad_offsets_write_nothing(offsets):
    a, a_scale, w, w_scale, b = _make(12, 3, 64, 64, 1)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ws = moe.alloc_fp8_workspace(moe.fp8_dims(12, 3, 64, 64))
    out = torch.full((12, 64), 5.0, dtype=BF16, device="cuda")
    moe.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, bias=b, out=out)
    assert moe.moe_read_device_status(ws) == 6
    assert bool((out == 5).all())


def test_no_rows_stream_and_graph():
    a, a_scale, w, w_scale, b = _make(70, 2, 272, 400, 11)
    off = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    ws = moe.alloc_fp8_workspace(moe.fp8_dims(70, 2, 272, 400))
    assert moe.fp8_matmul(a[:0], a_scale[:0], w, w_scale, ws, offsets=off, bias=b).shape == (0, 272)
    want = moe.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, bias=b)
    side = torch.cuda.Stream()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    moe.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, bias=b, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, bias=b, out=out)
    off.copy_(torch.tensor([0, 55, 70], dtype=torch.int32))  # other segments, same graph
    graph.replay()
    assert torch.equal(out, moe.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, bias=b))


def test_norm_feeds_the_product():
    # residual addition, norm, quantisation and a projection, as a block runs
    # them, against the projection of the dequantised operands
    T, D, N = 37, 2880, 1024
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((T, D), generator=g, device="cuda").to(BF16)
    residual = torch.randn((T, D), generator=g, device="cuda")
    gamma = torch.ones(D, dtype=BF16, device="cuda")
    q, scale, s = moe.rmsnorm_fp8(x, gamma, 1e-5, residual=residual)
    _, _, w, w_scale, b = _make(T, 1, N, D, 4)
    ws = moe.alloc_fp8_workspace(moe.fp8_dims(T, 1, N, D))
    out = moe.fp8_matmul(q, scale, w, w_scale, ws, bias=b, out_dtype=F32)
    ref, mag = _ref(q, scale, w, w_scale, b, [0, T])
    _check(out, ref, mag, D)
    # and the quantised rows are the norm's within E4M3: 2^-4 of each value, 2^-10 of a block's scale
    y = (s.double() / torch.sqrt(s.double().pow(2).mean(1, keepdim=True) + 1e-5))
    c = scale.double().repeat_interleave(128, 1)[:, :D]
    assert bool(((q.to(F32).double() * c - y).abs() <= (2.0 ** -4 + 2.0 ** -16) * y.abs().maximum(2.0 ** -6 * c)).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,N,K", [
    ([200], 5760, 272),                     # dense, tiles of 192 columns: one round, where 64 would take two
    ([700], 4112, 144),                     # 192, ragged rows and columns
    ([0, 11, 7] * 10 + [33, 129], 2880, 400),  # grouped, 192
    ([8, 0, 40, 31, 33, 1, 9, 7], 4096, 272),  # few rows, 256
    ([130, 0, 257, 90], 4096, 272),         # more, 256
    ([3, 1], 272, 1040),                    # 64
])
def test_tiles_on_both_sides_of_the_rule(counts, N, K, dtype):
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    _run(offsets[-1], len(counts), N, K, offsets, dtype, seed=5)
