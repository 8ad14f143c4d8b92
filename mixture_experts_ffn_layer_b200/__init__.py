"""B200 (sm_100a) GPT-OSS-style MoE feed-forward layer.

The compute lives in libmoe.so (C ABI in include/moe.h); this package is its
thin binding plus a convenience ``MoELayer`` that owns the workspace. The
library is loaded on first use; a missing library is an error, never a
fallback.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._binding import (  # noqa: F401
    MOE_W_BF16, MOE_W_MXFP4, MOE_ACT_SWIGLU, MOE_ACT_GPTOSS, EXPORTS, MoeError, Dims, dims, load, workspace_bytes,
    alloc_workspace, check_dims,
    moe_route, moe_permute, moe_gather, moe_mlp1, moe_mlp2, moe_ffn_grouped, moe_combine, moe_forward,
    moe_read_device_status, status_str, moe_permute_noalloc, moe_selftest_wait_timeout, mxfp4_prepared_bytes,
    moe_mxfp4_prepare, mxfp4_prepare, MOE_T_BF16, MOE_T_F32, NormDims, moe_forward_few, few_max_tokens, moe_rmsnorm,
    Fp8Dims, fp8_dims, fp8_workspace_bytes, alloc_fp8_workspace, moe_fp8_matmul,
)
from .ep import CudaLocalOps, ExpertParallelMoE, ep_forward  # noqa: F401,E402
from .block import _on, _under, MoEBlock, fp8_matmul, rmsnorm, rmsnorm_fp8  # noqa: F401,E402


def _capturing(t: torch.Tensor) -> bool:
    return t.is_cuda and torch.cuda.is_current_stream_capturing()


def _stream_id(t: torch.Tensor) -> int:
    """The current stream of t's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if t.is_cuda else 0


class MoELayer:
    """One MoE FFN layer's weights on the device plus its workspace.

    ``forward(x)`` enqueues the whole layer (moe_forward) on the current
    stream, or on ``stream`` with buffers of that stream, and returns y (T, D)
    bf16. Weights: Wr (E,D), br (E), W1 (E,2I,D),
    b1 (E,2I), W2 (E,D,I), b2 (E,D) bf16 -- or W1/W2 as MXFP4 codes with
    ``W1_scales``/``W2_scales``. ``act`` is MOE_ACT_SWIGLU or MOE_ACT_GPTOSS
    (with the caller's ``act_alpha`` and ``act_limit``). All of them dense and on
    one device. One layer serves one stream at a time."""

    def __init__(self, Wr, br, W1, b1, W2, b2, k: int, W1_scales=None, W2_scales=None, act=MOE_ACT_SWIGLU,
                 act_alpha: float = 1.0, act_limit: float = float("inf")):
        for t in (Wr, br, W1, b1, W2, b2, W1_scales, W2_scales):
            if t is not None and (t.device != Wr.device or not t.is_contiguous()):
                raise ValueError("weights must be contiguous and on one device")
        self.Wr, self.br, self.W1, self.b1, self.W2, self.b2 = Wr, br, W1, b1, W2, b2
        self.W1_scales, self.W2_scales = W1_scales, W2_scales
        self.k = k
        self.E, self.D = Wr.shape
        self.I = b1.shape[1] // 2
        self.wfmt = MOE_W_BF16 if W1_scales is None else MOE_W_MXFP4
        self.act, self.act_alpha, self.act_limit = act, act_alpha, act_limit
        self._ws: Optional[torch.Tensor] = None
        self._ws_T: Optional[int] = None  # tokens of the last call
        self._ws_home = 0          # the stream it was allocated on
        self._ws_captured = False  # a graph holds it
        self._ws_recorded = False  # its zero-fill was recorded into a graph, not run
        self._kept = []            # workspaces that graphs hold
        # forward_few's workspace holds the counters of its grid barriers. It is made
        # and zeroed here and never replaced: a first call on another stream or
        # inside a capture finds it zeroed, and a captured call finds it in place
        # after forward has taken a larger one. (A bf16 layer's is enough.)
        self._few_ws: Optional[torch.Tensor] = None
        most = self.few_max_tokens
        if most:
            self._few_ws = alloc_workspace(dims(most, self.D, self.E, k, self.I), device=Wr.device)
        # MXFP4 weights: their prepare-once form (scale layout of the
        # block-scaled MMAs), made here so that no call repeats it
        self.W1_prepared = self.W2_prepared = None
        if self.wfmt == MOE_W_MXFP4:
            d1 = self.dims(1)
            self.W1_prepared = mxfp4_prepare(d1, 1, W1, W1_scales)
            self.W2_prepared = mxfp4_prepare(d1, 2, W2, W2_scales)
        if Wr.is_cuda and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(Wr.device).synchronize()

    def dims(self, T: int) -> Dims:
        return dims(T, self.D, self.E, self.k, self.I, self.wfmt, self.act, self.act_alpha, self.act_limit)

    def workspace(self, T: int) -> torch.Tensor:
        """forward's workspace for T tokens, to be used on the current stream."""
        capturing = _capturing(self.Wr)
        if T != self._ws_T and (self._ws is None or self._ws.numel() < workspace_bytes(self.dims(T))):
            if self._ws_captured:
                self._kept.append(self._ws)
            self._ws = alloc_workspace(self.dims(T), device=self.Wr.device)
            self._ws_home, self._ws_captured, self._ws_recorded = _stream_id(self.Wr), False, capturing
        self._ws_T = T
        if capturing:
            self._ws_captured = True
            return self._ws
        if self._ws_recorded:
            self._ws[:256].zero_()  # the status word's part
            self._ws_recorded = False
        if self._ws_home != _stream_id(self.Wr):
            self._ws.record_stream(torch.cuda.current_stream(self.Wr.device))
        return self._ws

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        if stream is not None:
            return _under(stream, x, self.forward, x, out)
        T = x.shape[0]
        y = out if out is not None else torch.empty((T, self.D), dtype=torch.bfloat16, device=x.device)
        _on(x, moe_forward, self.dims(T), x, self.Wr, self.br, self.W1, self.b1, self.W2, self.b2, y,
            self.workspace(T), self.W1_scales, self.W2_scales, None, self.W1_prepared, self.W2_prepared)
        return y

    __call__ = forward

    @property
    def few_max_tokens(self) -> int:
        """The most tokens forward_few takes."""
        return few_max_tokens(self.dims(1))

    def forward_few(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """forward for at most few_max_tokens tokens in one launch
        (moe_forward_few): the latency path of a decode step. MXFP4 weights
        are read as stored, so the layer keeps their codes and scales."""
        if stream is not None:
            return _under(stream, x, self.forward_few, x, out)
        if x.dim() != 2 or x.shape[1] != self.D or x.dtype != torch.bfloat16 or not x.is_contiguous():
            raise ValueError("x must be a contiguous (T, D) bf16 tensor")
        if x.device != self.Wr.device:
            raise ValueError("x must be on the layer's device")
        if out is not None and (out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous() or
                                out.device != x.device):
            raise ValueError("out must be a contiguous tensor of x's shape and type, on its device")
        T = x.shape[0]
        y = out if out is not None else torch.empty_like(x)
        ws = self._few_ws if self._few_ws is not None else self.workspace(T)  # (which refuses what has none)
        _on(x, moe_forward_few, self.dims(T), x, self.Wr, self.br, self.W1, self.b1, self.W2, self.b2, y,
            ws, self.W1_scales, self.W2_scales)
        return y

    def device_status(self, stream=None) -> int:
        """Wait for the current stream, or ``stream``, then read and clear the
        status words of the layer's workspaces: an error recorded since the last
        call, 0 if none. (After a first call inside a capture: not before the
        graph has run.)"""
        status = [_on(ws, moe_read_device_status, ws, stream) for ws in (self._few_ws, self._ws, *self._kept)
                  if ws is not None]
        return next((st for st in status if st), 0)
