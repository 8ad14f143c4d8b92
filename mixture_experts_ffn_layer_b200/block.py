"""What stands around the MoE layer in a transformer block: the residual's
addition and RMSNorm in front of it (write-up, "model flow"), with outputs in
bf16 or block-scaled E4M3, and ``MoEBlock``, which runs the norm and the layer
together.

A call with ``stream`` runs on that stream and takes its buffers from it; the
inputs must be ready there (``stream.wait_stream``) and stay until it is done, as
for any use of a tensor on a second stream."""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _binding as B

BF16 = torch.bfloat16


def _require(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


def _on(t: torch.Tensor, call, *args):
    """call(*args) with t's device current."""
    if t.is_cuda and t.get_device() == torch._C._cuda_getDevice():  # (a device tensor: CUDA is initialised)
        return call(*args)
    with torch.cuda.device(t.device):
        return call(*args)


def _under(stream, at: torch.Tensor, call, *args, **kw):
    """call(*args, **kw) with `stream` current, so that what the call allocates
    is that stream's; what it returns is marked as used on the caller's too."""
    _require(stream.device == at.device, "stream must be one of the tensors' device")
    caller = torch.cuda.current_stream(stream.device)
    if caller == stream:
        return call(*args, **kw)
    with torch.cuda.stream(stream):
        got = call(*args, **kw)
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None:
            t.record_stream(caller)
    return got


def _norm_dims(x: torch.Tensor, gamma: torch.Tensor, eps: float, residual: Optional[torch.Tensor]) -> B.NormDims:
    _require(x.dim() == 2 and x.dtype == BF16 and x.stride(1) == 1, "x must be a (T, D) bf16 tensor of dense rows")
    T, D = x.shape
    at = x.get_device()
    _require(gamma.dtype == BF16 and gamma.shape == (D,) and gamma.is_contiguous() and gamma.get_device() == at,
             "gamma must be a (D,) bf16 tensor on x's device")
    f32 = False
    if residual is not None:
        f32 = residual.dtype == torch.float32
        _require((f32 or residual.dtype == BF16) and residual.shape == (T, D) and residual.is_contiguous() and
                 residual.get_device() == at, "residual must be a contiguous (T, D) bf16 or fp32 tensor on x's device")
    return B.NormDims(T, D, x.stride(0) if T > 1 else max(D, 1), eps, B.MOE_T_F32 if f32 else B.MOE_T_BF16)


def _like(out: Optional[torch.Tensor], of: Optional[torch.Tensor], what: str) -> Optional[torch.Tensor]:
    """`out` checked against `of`'s shape, type and device, or a new tensor; None without `of`."""
    if out is None:
        return None if of is None else torch.empty_like(of)
    _require(of is not None, f"{what} without a residual")
    _require(out.shape == of.shape and out.dtype == of.dtype and out.is_contiguous() and out.device == of.device,
             f"{what} must be a contiguous (T, D) tensor of its input's type, on its device")
    return out


def rmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, res_out: Optional[torch.Tensor] = None,
            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(y, s): s = x + residual in the residual's type (None without one) and
    y = RMSNorm(s) * gamma in bf16. Rows of x may be strided. ``res_out`` may
    be the residual itself."""
    if stream is not None:
        return _under(stream, x, rmsnorm, x, gamma, eps, residual, out, res_out)
    n = _norm_dims(x, gamma, eps, residual)
    y = _like(out, x, "out")
    res = _like(res_out, residual, "res_out")
    _on(x, B.moe_rmsnorm, n, x, residual, gamma, res, y, None, None)
    return y, res


def rmsnorm_fp8(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5, residual: Optional[torch.Tensor] = None,
                res_out: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(q, q_scale, s): as rmsnorm with y quantised to E4M3, one fp32 scale
    per row and 128 columns."""
    if stream is not None:
        return _under(stream, x, rmsnorm_fp8, x, gamma, eps, residual, res_out)
    n = _norm_dims(x, gamma, eps, residual)
    T, D = x.shape
    q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    scale = x.new_empty(T, -(-D // 128), dtype=torch.float32)
    res = _like(res_out, residual, "res_out")
    _on(x, B.moe_rmsnorm, n, x, residual, gamma, res, None, q, scale)
    return q, scale, res


def fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, ws: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, out_dtype=BF16, stream=None) -> torch.Tensor:
    """The block-scaled FP8 product (moe_fp8_matmul): a (R, K) and w (E, N, K)
    E4M3, a_scale (R, ceil(K/128)) and w_scale (E, ceil(N/128), ceil(K/128))
    fp32, as rmsnorm_fp8 gives the left operand. With ``offsets`` (E+1) int32
    the rows of [offsets[e], offsets[e+1]) are multiplied with w[e]; without,
    E = 1 and all rows are. ``bias`` (E, N) bf16. Returns (R, N)."""
    if stream is not None:
        return _under(stream, a, fp8_matmul, a, a_scale, w, w_scale, ws, offsets, bias, out, out_dtype)
    of_a, of_w = a.shape, w.shape
    _require(len(of_a) == 2 and len(of_w) == 3 and of_a[1] == of_w[2], "a must be (R, K) and w (E, N, K)")
    R, K = of_a
    E, N, _ = of_w
    kb, nb = -(-K // 128), -(-N // 128)
    _require(a.dtype == torch.float8_e4m3fn and w.dtype == torch.float8_e4m3fn, "a and w must be float8_e4m3fn")
    _require(a_scale.dtype == torch.float32 and w_scale.dtype == torch.float32 and a_scale.shape == (R, kb) and
             w_scale.shape == (E, nb, kb), "a_scale must be (R, K/128) and w_scale (E, N/128, K/128) fp32")
    _require(E == 1 if offsets is None else offsets.shape == (E + 1,) and offsets.dtype == torch.int32,
             "offsets must be (E+1,) int32, or None with E = 1")
    _require(bias is None or (bias.shape == (E, N) and bias.dtype == BF16), "bias must be (E, N) bf16")
    if out is None:
        _require(out_dtype in (BF16, torch.float32), "out_dtype must be bf16 or fp32")
        out = a.new_empty(R, N, dtype=out_dtype)
    else:
        _require(out.shape == (R, N) and out.dtype in (BF16, torch.float32), "out must be (R, N) bf16 or fp32")
    at = a.get_device()
    for t in (a, a_scale, w, w_scale, ws, offsets, bias, out):
        if t is not None and (t.get_device() != at or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on one device")
    _on(a, B.moe_fp8_matmul, B.fp8_dims(R, E, N, K, out.dtype), a, a_scale, offsets, w, w_scale, bias, out, ws)
    return out


class MoEBlock:
    """The feed-forward half of a transformer block: residual addition,
    RMSNorm and the MoE layer. ``forward(x, residual)`` returns (y, s) with
    s = x + residual, the residual stream, and y = layer(RMSNorm(s) * gamma),
    which the next block adds to s. The first block of a model has no residual
    (None): s is x, in the same buffer where its rows are dense.

    ``layer`` is a MoELayer or an ExpertParallelMoE; the latter is called with no
    tokens too, since every rank takes part in it. A MoELayer's batches of at
    most ``few_max_tokens`` tokens take the one-launch layer: MXFP4 weights then
    meet activations that are more exact than the batched layer's pairs of E4M3,
    so a row's result can depend on the batch's size by more than the sums'
    order."""

    def __init__(self, layer, gamma: torch.Tensor, eps: float = 1e-5):
        self.layer, self.gamma, self.eps = layer, gamma, eps

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor],
                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        if stream is not None:  # (the normed rows between the two are the stream's own)
            return _under(stream, x, self.forward, x, residual)
        n, s = rmsnorm(x, self.gamma, self.eps, residual=residual)
        if residual is None:
            s = x.contiguous()
        most = getattr(self.layer, "few_max_tokens", None)
        if most is None:  # an expert-parallel layer
            return _on(x, self.layer.forward, n), s
        T = x.shape[0]
        if T == 0:
            return n, s
        return _on(x, self.layer.forward_few if T <= most else self.layer.forward, n), s

    __call__ = forward
