"""MoEBlock's way through its parts, with stand-ins for the kernels (the
numbers are compared on the GPU, with the layer's)."""
import pytest
import torch

from mixture_experts_ffn_layer_b200 import block

BF16 = torch.bfloat16


@pytest.fixture
def plain(monkeypatch):
    def rmsnorm(x, gamma, eps=1e-5, residual=None, **kw):
        s = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
        v = s.float()
        y = (v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + eps) * gamma.float()).to(BF16)
        return y, None if residual is None else s

    monkeypatch.setattr(block, "rmsnorm", rmsnorm)
    monkeypatch.setattr(block, "_on", lambda t, call, *args: call(*args))


class _Layer:
    few_max_tokens = 4

    def __init__(self):
        self.calls = []

    def forward(self, n):
        self.calls.append(("forward", n.shape[0]))
        return 2 * n

    def forward_few(self, n):
        self.calls.append(("few", n.shape[0]))
        return 2 * n


class _Sharded:
    """As ExpertParallelMoE: every rank's call takes part, tokens or not."""

    def __init__(self):
        self.calls = []

    def forward(self, n):
        self.calls.append(n.shape[0])
        return 2 * n

    __call__ = forward


def _rows(T, seed=0):
    return torch.randn((T, 64), generator=torch.Generator().manual_seed(seed)).to(BF16)


def test_first_block_of_a_model(plain):
    # without a residual the stream begins with x
    layer, gamma = _Layer(), torch.ones(64, dtype=BF16)
    x = _rows(3)
    y, s = block.MoEBlock(layer, gamma)(x, None)
    assert torch.equal(s, x) and s.is_contiguous()
    assert torch.equal(y, 2 * block.rmsnorm(x, gamma)[0])
    wide = _rows(3, 1).repeat(1, 2)[:, :64]  # rows of a wider projection
    y2, s2 = block.MoEBlock(layer, gamma)(wide, None)
    assert torch.equal(s2, wide) and s2.is_contiguous()
    y3, s3 = block.MoEBlock(layer, gamma)(y, s)  # and the next block adds to it
    assert torch.equal(s3, (y.float() + x.float()).to(BF16))


def test_few_and_many_tokens(plain):
    layer, gamma = _Layer(), torch.ones(64, dtype=BF16)
    for T in (1, 4, 5, 0):
        y, s = block.MoEBlock(layer, gamma)(_rows(T), _rows(T, 1))
        assert y.shape == s.shape == (T, 64)
    assert layer.calls == [("few", 1), ("few", 4), ("forward", 5)]


def test_expert_parallel_layer(plain):
    layer, gamma = _Sharded(), torch.ones(64, dtype=BF16)
    for T in (0, 1, 5):
        x, r = _rows(T), _rows(T, 1)
        y, s = block.MoEBlock(layer, gamma)(x, r)
        assert torch.equal(y, 2 * block.rmsnorm(x, gamma, residual=r)[0])
    assert layer.calls == [0, 1, 5]
