"""Refusals and sizes of the operators around the layer, checked on the host
(nothing is enqueued)."""
import ctypes

import pytest
import torch

import mixture_experts_ffn_layer_b200 as moe
from mixture_experts_ffn_layer_b200 import _binding
from test_abi import _Arena

vp = ctypes.c_void_p


def test_rmsnorm_arguments():
    lib = moe.load()
    ar = _Arena()
    x, r, g, y, q, c = (vp(ar.take()) for _ in range(6))
    off = vp(ar.take() + 16)

    def call(T=4, D=64, ldx=64, eps=1e-5, rt=0, x=x, r=r, g=g, ro=None, y=y, q=None, c=None):
        return lib.moe_rmsnorm(_binding.NormDims(T, D, ldx, eps, rt), x, r, g, ro, y, q, c, None)

    assert call(T=0) == 0  # no rows: nothing is enqueued, pointers are not looked at
    assert call(T=0, x=None, r=None, g=None, y=None) == 0
    assert call(T=-1) == 1
    assert call(D=0) == 1
    assert call(ldx=48) == 1
    assert call(eps=-1e-5) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(rt=2) == 1
    assert call(D=72, ldx=80) == 2 and call(ldx=72) == 2 and call(D=16400, ldx=16400) == 2
    assert call(x=None) == 1 and call(g=None) == 1 and call(y=None) == 1
    assert call(q=q) == 1 and call(c=c) == 1  # codes and scales come together
    assert call(r=None, ro=r) == 1  # a stream without a residual
    for name in ("x", "r", "g", "y"):
        assert call(**{name: off}) == 1
    assert call(ro=off) == 1 and call(q=off, c=c) == 1 and call(q=q, c=off) == 1


def test_rmsnorm_tensor_checks():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    g = torch.ones(64, dtype=torch.bfloat16)
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(x=x.t()), dict(gamma=g[:32]), dict(gamma=g.float()),
                dict(residual=x[:2]), dict(residual=x.half()), dict(res_out=x), dict(out=x[:2]), dict(out=x.float()),
                dict(residual=x, res_out=x.float()), dict(residual=torch.zeros((4, 128), dtype=torch.bfloat16)[:, :64])):
        with pytest.raises(ValueError):
            moe.rmsnorm(**{"x": x, "gamma": g, **bad})


def test_few_max_tokens():
    assert moe.few_max_tokens(moe.dims(1, 2880, 32, 4, 2880)) == 16
    assert moe.few_max_tokens(moe.dims(9999, 4096, 32, 4, 64)) == 16  # T is not read
    assert moe.few_max_tokens(moe.dims(1, 4160, 32, 4, 64)) == 15
    assert moe.few_max_tokens(moe.dims(1, 64, 4, 2, 16384, wfmt=moe.MOE_W_MXFP4)) == 4
    assert moe.few_max_tokens(moe.dims(1, 96, 4, 2, 64)) == 0  # not a supported layer


def test_forward_few_arguments():
    lib = moe.load()
    ar = _Arena(64 << 20)
    d, dq = moe.dims(4, 64, 4, 2, 64), moe.dims(4, 64, 4, 2, 64, wfmt=moe.MOE_W_MXFP4)
    n, nq = moe.workspace_bytes(d), moe.workspace_bytes(dq)
    ws = vp(ar.take(max(n, nq)))
    x, wr, br, b1, b2, y = (vp(ar.take()) for _ in range(6))
    w1, w2, s1, s2 = (ar.take() for _ in range(4))
    off = vp(ar.take() + 16)
    W = _binding.Weight

    def call(d=d, x=x, wr=wr, br=br, w1=W(w1), b1=b1, w2=W(w2), b2=b2, y=y, ws=ws, n=n):
        return lib.moe_forward_few(d, x, wr, br, w1, b1, w2, b2, y, ws, n, None)

    assert call(d=moe.dims(17, 64, 4, 2, 64)) == 2
    assert call(d=moe.dims(5, 64, 4, 2, 16384)) == 2  # 5 x 16384 activations
    assert call(d=moe.dims(0, 64, 4, 2, 64)) == 1
    assert call(n=n - 1) == 3 and call(ws=None) == 1 and call(ws=vp(ar.take() + 8)) == 1
    for name in ("x", "wr", "br", "b1", "b2", "y"):
        assert call(**{name: None}) == 1 and call(**{name: off}) == 1, name
    assert call(w1=W(None)) == 1 and call(w2=W(w2 + 16)) == 1
    # MXFP4: read as stored, a prepared form alone is not enough
    q = dict(d=dq, n=nq)
    assert call(**q) == 1  # no scales
    assert call(**q, w1=W(w1, s1), w2=W(w2)) == 1
    assert call(**q, w1=W(None, None, w1), w2=W(w2, s2)) == 1
    assert call(**q, w1=W(w1, None, s1), w2=W(w2, s2)) == 1


def test_workspace_for_more_tokens_is_enough_for_fewer():
    # around the one-launch layer's limit, where its logits could weigh more
    # than another token's rows
    for wfmt in (moe.MOE_W_BF16, moe.MOE_W_MXFP4):
        n = [moe.workspace_bytes(moe.dims(T, 64, 256, 1, 64, wfmt=wfmt)) for T in range(1, 40)]
        assert n == sorted(n), wfmt


def test_forward_few_tensor_checks():
    E, D, I = 4, 64, 64
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    layer = moe.MoELayer(z(E, D), z(E), z(E, 2 * I, D), z(E, 2 * I), z(E, D, I), z(E, D), 2)
    x = z(3, D)
    for bad in (z(3, D + 8), z(3, 2 * D)[:, ::2], x.float(), z(D), x.to("meta")):
        with pytest.raises(ValueError):
            layer.forward_few(bad)
    for bad in (z(2, D), z(3, 2 * D)[:, :D], x.float(), x.to("meta")):
        with pytest.raises(ValueError):
            layer.forward_few(x, out=bad)


def test_fp8_sizes_and_arguments():
    lib = moe.load()
    D = moe.fp8_dims
    assert moe.fp8_workspace_bytes(D(5, 3, 64, 64)) >= 4
    for bad, code in ((D(-1, 1, 64, 64), 1), (D(4, 0, 64, 64), 1), (D(4, 1, 0, 64), 1), (D(4, 1, 64, -16), 1),
                      (_binding.Fp8Dims(4, 1, 64, 64, 2), 1), (D(4, 257, 64, 64), 2), (D(4, 1, 72, 64), 2),
                      (D(4, 1, 64, 72), 2), (D(4, 1, 65552, 64), 2), (D(4, 1, 64, 65552), 2),
                      (D((1 << 30) + 1, 1, 64, 64), 2), (D(1 << 30, 1, 65536, 16), 2)):
        assert lib.moe_check_fp8(bad) == code
        with pytest.raises(moe.MoeError):
            moe.fp8_workspace_bytes(bad)
    ar = _Arena()
    a, sa, off, w, sw, b, out, ws = (vp(ar.take()) for _ in range(8))
    mis = vp(ar.take() + 16)

    def call(d=D(4, 3, 64, 64), a=a, sa=sa, off=off, w=w, sw=sw, b=b, out=out, ws=ws, n=256):
        return lib.moe_fp8_matmul(d, a, sa, off, w, sw, b, out, ws, n, None)

    assert call(d=D(0, 3, 64, 64), a=None, out=None) == 0  # no rows: nothing is enqueued
    assert call(off=None) == 1  # several experts without segments
    assert call(n=0) == 3
    for name in ("a", "sa", "w", "sw", "out", "ws"):
        assert call(**{name: None}) == 1 and call(**{name: mis}) == 1, name
    assert call(off=mis) == 1 and call(b=mis) == 1


def test_fp8_tensor_checks():
    f8, f32 = torch.float8_e4m3fn, torch.float32
    ok = dict(a=torch.zeros((4, 144)).to(f8), a_scale=torch.zeros((4, 2)), w=torch.zeros((2, 160, 144)).to(f8),
              w_scale=torch.zeros((2, 2, 2)), ws=torch.zeros(256, dtype=torch.uint8),
              offsets=torch.zeros(3, dtype=torch.int32), bias=torch.zeros((2, 160), dtype=torch.bfloat16))
    for bad in (dict(a=torch.zeros((4, 144))), dict(a=torch.zeros((4, 160)).to(f8)), dict(a_scale=torch.zeros((4, 1))),
                dict(w_scale=torch.zeros((2, 1, 2))), dict(offsets=None), dict(offsets=torch.zeros(3)),
                dict(offsets=torch.zeros(2, dtype=torch.int32)), dict(bias=torch.zeros((2, 160))),
                dict(out=torch.zeros((4, 144), dtype=f32)), dict(out=torch.zeros((4, 160), dtype=torch.float16)),
                dict(out_dtype=torch.float16), dict(a_scale=torch.zeros((2, 4)).t())):
        with pytest.raises(ValueError):
            moe.fp8_matmul(**{**ok, **bad})


def test_layer_weights_are_dense_and_on_one_device():
    # the kernels read them by their addresses alone
    E, D, I = 4, 64, 64
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    ok = dict(Wr=z(E, D), br=z(E), W1=z(E, 2 * I, D), b1=z(E, 2 * I), W2=z(E, D, I), b2=z(E, D))
    moe.MoELayer(**ok, k=2)
    for name, t in ok.items():
        wide = z(*t.shape[:-1], 2 * t.shape[-1])[..., ::2]
        for bad in (t.to("meta"), wide):
            with pytest.raises(ValueError):
                moe.MoELayer(**{**ok, name: bad}, k=2)
    with pytest.raises(ValueError):
        moe.MoELayer(**ok, k=2, W1_scales=torch.zeros((E, 2 * I, 2), dtype=torch.uint8, device="meta"),
                     W2_scales=torch.zeros((E, D, 2), dtype=torch.uint8))
