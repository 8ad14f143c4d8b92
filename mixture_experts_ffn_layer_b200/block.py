"""What stands around the MoE layer in a transformer block: the residual's
addition and RMSNorm in front of it (write-up, "model flow"), with outputs in
bf16 or block-scaled E4M3, and ``MoEBlock``, which runs the norm and the layer
together."""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _binding as B

BF16 = torch.bfloat16


def _require(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


def _norm_dims(x: torch.Tensor, gamma: torch.Tensor, eps: float, residual: Optional[torch.Tensor]) -> B.NormDims:
    _require(x.dim() == 2 and x.dtype == BF16 and x.stride(1) == 1, "x must be a (T, D) bf16 tensor of dense rows")
    T, D = x.shape
    _require(gamma.shape == (D,) and gamma.dtype == BF16 and gamma.is_contiguous(), "gamma must be a (D,) bf16 tensor")
    _require(gamma.device == x.device, "gamma and x must be on one device")
    if residual is not None:
        _require(residual.shape == x.shape and residual.dtype in (BF16, torch.float32) and residual.is_contiguous(),
                 "residual must be a contiguous (T, D) bf16 or fp32 tensor")
        _require(residual.device == x.device, "residual and x must be on one device")
    f32 = residual is not None and residual.dtype == torch.float32
    return B.NormDims(T, D, x.stride(0) if T > 1 else max(D, 1), eps, B.MOE_T_F32 if f32 else B.MOE_T_BF16)


def rmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, res_out: Optional[torch.Tensor] = None,
            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(y, s): s = x + residual in the residual's type (None without one) and
    y = RMSNorm(s) * gamma in bf16. Rows of x may be strided. ``res_out`` may
    be the residual itself."""
    n = _norm_dims(x, gamma, eps, residual)
    y = out if out is not None else torch.empty(x.shape, dtype=BF16, device=x.device)
    res = res_out if res_out is not None or residual is None else torch.empty_like(residual)
    with torch.cuda.device(x.device):
        B.moe_rmsnorm(n, x, residual, gamma, res, y, None, None, stream)
    return y, res


def rmsnorm_fp8(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5, residual: Optional[torch.Tensor] = None,
                res_out: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(q, q_scale, s): as rmsnorm with y quantised to E4M3, one fp32 scale
    per row and 128 columns."""
    n = _norm_dims(x, gamma, eps, residual)
    T, D = x.shape
    q = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty((T, -(-D // 128)), dtype=torch.float32, device=x.device)
    res = res_out if res_out is not None or residual is None else torch.empty_like(residual)
    with torch.cuda.device(x.device):
        B.moe_rmsnorm(n, x, residual, gamma, res, None, q, scale, stream)
    return q, scale, res


class MoEBlock:
    """The feed-forward half of a transformer block: residual addition,
    RMSNorm and the MoE layer. ``forward(x, residual)`` returns (y, s) with
    s = x + residual, the residual stream, and y = layer(RMSNorm(s) * gamma),
    which the next block adds to s. Batches of at most ``layer.few_max_tokens``
    tokens take the one-launch layer."""

    def __init__(self, layer, gamma: torch.Tensor, eps: float = 1e-5):
        self.layer, self.gamma, self.eps = layer, gamma, eps

    def forward(self, x: torch.Tensor, residual: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        n, s = rmsnorm(x, self.gamma, self.eps, residual=residual, stream=stream)
        T = x.shape[0]
        if T == 0:
            return n, s
        few = T <= self.layer.few_max_tokens
        return (self.layer.forward_few if few else self.layer.forward)(n, stream=stream), s

    __call__ = forward
