"""Binding of the operators around the expert forward: the RMS norm with MXFP8
output, the fused MXFP8 product and the router's load-balance loss.

Like ``api``: argument marshalling only, every step runs in the library's
kernels.  An MXFP8 activation is a pair ``(q, s)``: e4m3 payload uint8 [.., K]
and its scales in the tensor-core layout, an opaque uint8 array
[ceil(M/128) * 128, ceil(K/128) * 4].  Payload rows of many are a multiple of 128
bytes apart (``q`` is then a view of a wider array): rows that straddle cache
lines slow the product's loads by a fifth.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .api import _u8, mx_quantize_3d, mx_scales_to_mma_layout

ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


_BF16, _F32, _U8, _I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int64
_empty = torch.empty
# The current stream's handle by device index: torch.cuda.current_stream without the
# Stream object, which takes longer than a launch.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _bad(t, name, dtypes):
    """What is wrong with a tensor that is not on CUDA, contiguous and of one of dtypes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name, dtypes):
    """A CUDA tensor of one of ``dtypes``, contiguous."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes
            and t.is_contiguous()):
        _bad(t, name, dtypes)


_HALF_OR_FLOAT = (_BF16, _F32)
# More rows than this get payload rows a multiple of 128 bytes apart (below it
# the product is bound by the weights' rows, and the view costs host time).
_PAD_ROWS = 256


def _payload(shape, M, dev):
    """An e4m3 payload to write and the distance of its rows."""
    K = shape[-1]
    if M <= _PAD_ROWS or K % 128 == 0 or len(shape) != 2:
        return _empty(shape, dtype=_U8, device=dev), K
    ld = -(-K // 128) * 128
    return _empty((M, ld), dtype=_U8, device=dev)[:, :K], ld


def _payload_rows(t, name):
    """The distance of a payload's rows: contiguous, or 2D with rows further apart."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is _U8:
        if t.is_contiguous():
            return t.shape[-1] if t.dim() else 0
        if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
            return t.stride(0)
    _bad(t, name, (_U8,))


def _mma_scale_shape(M: int, K: int):
    return (-(-M // 128) * 128, -(-K // 128) * 4)


def mx_add_rmsnorm_quant(x, weight, residual=None, eps: float = 1e-6, bf16_out: bool = False,
                         mma_scales: bool = False, residual_out=None) -> dict:
    """h = x + residual; y = bf16(h * weight / sqrt(mean(h^2) + eps)); MXFP8 of y.

    x bf16 [.., H] (contiguous, or 2D with rows further apart), weight bf16 or
    fp32 [H], residual bf16 or fp32 [.., H].  Returns ``q`` (e4m3 codes uint8
    [.., H]), ``s`` (e8m0 uint8 [.., ceil(H/32)], or the tensor-core layout
    with ``mma_scales``: what ``mxfp8_linear_fused`` reads), ``y`` (bf16,
    with ``bf16_out``: what the router reads) and ``residual`` (h in the
    residual's type; pass ``residual_out=residual`` to update it in place)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x must be a torch.Tensor of at least one dimension")
    shape = x.shape
    H = ldx = shape[-1]
    if x.is_cuda and x.dtype is _BF16 and len(shape) == 2 and x.stride(1) == 1:
        if shape[0] > 1:
            ldx = x.stride(0)
            if ldx < H:
                raise ValueError("x: overlapping rows")
    else:
        _rows(x, "x", (_BF16,))
    _rows(weight, "weight", _HALF_OR_FLOAT)
    if weight.shape != (H,):
        raise ValueError(f"weight is {tuple(weight.shape)}, x has H = {H}")
    dev = x.device
    M = x.numel() // H if H else 0
    res_ptr = res_out_ptr = y_ptr = None
    res32 = 0
    if residual is not None:
        _rows(residual, "residual", _HALF_OR_FLOAT)
        if residual.shape != shape:
            raise ValueError(f"residual is {tuple(residual.shape)}, x is {tuple(shape)}")
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        else:
            _rows(residual_out, "residual_out", (residual.dtype,))
            if residual_out.shape != shape:
                raise ValueError(f"residual_out is {tuple(residual_out.shape)}, x is {tuple(shape)}")
        res32 = residual.dtype is _F32
        res_ptr, res_out_ptr = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if mma_scales:
        q, ldq = _payload(shape, M, dev)
        s = _empty(_mma_scale_shape(M, H), dtype=_U8, device=dev)
    else:
        q, ldq = _empty(shape, dtype=_U8, device=dev), H
        s = _empty((*shape[:-1], -(-H // 32)), dtype=_U8, device=dev)
    out = {"q": q, "s": s}
    if residual is not None:
        out["residual"] = residual_out
    if bf16_out:
        out["y"] = y = _empty(shape, dtype=_BF16, device=dev)
        y_ptr = y.data_ptr()
    rc = _lib.load().mx_add_rmsnorm_quant(
        x.data_ptr(), ldx, res_ptr, res32, res_out_ptr, weight.data_ptr(), weight.dtype is _F32,
        eps, M, H, y_ptr, q.data_ptr(), ldq, s.data_ptr(), mma_scales, _raw_stream(dev.index))
    if rc:
        _lib.check("mx_add_rmsnorm_quant", rc)
    return out


def mxfp8_linear_fused_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib.load().mxfp8_linear_fused_workspace_size(M, N, K))


def mxfp8_linear_fused(x, wq, ws_mma, bias=None, act=None, residual=None, mx_out: bool = False,
                       out=None, workspace=None):
    """act(x . wq^T + bias) + residual with an MXFP8 product.

    x: bf16 [.., K] (MX-quantized per token on the device) or an MXFP8 pair
    (q, s) with tensor-core scales; wq e4m3 [N, K] (its rows may be further
    apart), ws_mma its scales in the tensor-core layout; bias bf16 or fp32 [N]; act one of "none", "relu",
    "gelu", "gelu_tanh", "silu"; residual bf16 [.., N].  Returns bf16 [.., N],
    or with ``mx_out`` the MXFP8 pair of act(..) (no residual)."""
    wq = _u8(wq)
    _check_weight(wq, ws_mma, bias, act)
    return _fused(x, wq, ws_mma, bias, ACTIVATIONS[act], residual, mx_out, out, workspace)


def _check_weight(wq, ws_mma, bias, act):
    _payload_rows(wq, "wq")
    if wq.dim() != 2:
        raise ValueError(f"wq: expected 2 dims, got {tuple(wq.shape)}")
    N, K = wq.shape
    _rows(ws_mma, "ws_mma", (_U8,))
    rows, cols = _mma_scale_shape(N, K)
    if ws_mma.numel() != rows * cols:
        raise ValueError("ws_mma is not in the tensor-core layout of wq's scales")
    if act not in ACTIVATIONS:
        raise ValueError(f"act: expected one of {sorted(k for k in ACTIVATIONS if k)}, got {act!r}")
    if bias is not None:
        _rows(bias, "bias", _HALF_OR_FLOAT)
        if bias.shape != (N,):
            raise ValueError(f"bias is {tuple(bias.shape)}, wq has N = {N}")


def _fused(x, wq, ws_mma, bias, act, residual, mx_out, out, workspace):
    """mxfp8_linear_fused on a checked weight.  workspace: a tensor, None, or a
    function of (M, device) that gives one (or None) for bf16 input."""
    N, K = wq.shape
    x_ptr = xq_ptr = xs_ptr = ws_ptr = res_ptr = out_ptr = oq_ptr = os_ptr = None
    ws_bytes = ldx = ldo = 0
    lib = _lib.load()
    if type(x) is tuple:
        xin, xs = x
        xin = _u8(xin)
        ldx = _payload_rows(xin, "x[0]")
        _rows(xs, "x[1]", (_U8,))
    else:
        xin, xs = x, None
        _rows(x, "x", (_BF16,))
    shape = xin.shape
    if not shape or shape[-1] != K:
        raise ValueError(f"wq is {tuple(wq.shape)}, x is {tuple(shape)}")
    M = xin.numel() // K if K else 0
    dev = xin.device
    if xs is not None:
        rows, cols = _mma_scale_shape(M, K)
        if xs.numel() != rows * cols:
            raise ValueError("x's scales are not in the tensor-core layout")
        xq_ptr, xs_ptr = xin.data_ptr(), xs.data_ptr()
    else:
        x_ptr = x.data_ptr()
        if workspace is None:
            need = lib.mxfp8_linear_fused_workspace_size(M, N, K)
            workspace = _empty(need, dtype=_U8, device=dev) if need else None
        elif callable(workspace):
            workspace = workspace(M, dev)
        if workspace is not None:
            ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    shape = (M, N) if len(shape) == 2 else (*shape[:-1], N)
    if residual is not None:
        if mx_out:
            raise ValueError("an MXFP8 result takes no residual")
        _rows(residual, "residual", (_BF16,))
        if residual.shape != shape:
            raise ValueError(f"residual is {tuple(residual.shape)}, the result {shape}")
        res_ptr = residual.data_ptr()
    if mx_out:
        if out is not None:
            raise ValueError("out holds a bf16 result")
        oq, ldo = _payload(shape, M, dev)
        out = (oq, _empty(_mma_scale_shape(M, N), dtype=_U8, device=dev))
        oq_ptr, os_ptr = out[0].data_ptr(), out[1].data_ptr()
    else:
        if out is None:
            out = _empty(shape, dtype=_BF16, device=dev)
        else:
            _rows(out, "out", (_BF16,))
            if out.shape != shape:
                raise ValueError(f"out is {tuple(out.shape)}, the result {shape}")
        out_ptr = out.data_ptr()
    bias_ptr, bias32 = (None, 0) if bias is None else (bias.data_ptr(), bias.dtype is _F32)
    rc = lib.mxfp8_linear_fused(
        x_ptr, xq_ptr, ldx, xs_ptr, wq.data_ptr(), wq.stride(0), ws_mma.data_ptr(), M, N, K,
        bias_ptr, bias32, act, res_ptr, out_ptr, oq_ptr, ldo, os_ptr, ws_ptr, ws_bytes,
        _raw_stream(dev.index))
    if rc:
        _lib.check("mxfp8_linear_fused", rc)
    return out


class MXFP8FusedLinear:
    """An MXFP8 linear with bias and activation, and the residual's addition.

    Weights as ``MXFP8Linear``: ``from_bf16`` quantizes at load, the
    constructor takes an offline checkpoint's payload and [N, ceil(K/32)]
    scales, which are re-laid once (a payload of K % 128 != 0 as well, its rows
    to a multiple of 128 bytes apart).  Calls take bf16 rows or an MXFP8 pair."""

    def __init__(self, wq, ws, bias=None, act=None):
        self.wq = _u8(wq)
        self.N, self.K = self.wq.shape
        self.ws_mma = mx_scales_to_mma_layout(ws, self.K)
        self.bias, self.act = bias, act
        _check_weight(self.wq, self.ws_mma, bias, act)
        if self.K % 128:
            wide = _empty((self.N, -(-self.K // 128) * 128), dtype=_U8, device=self.wq.device)
            self.wq = wide[:, :self.K].copy_(self.wq)
        self._ws = None
        self._need = {}  # rows -> workspace bytes

    @classmethod
    def from_bf16(cls, w, bias=None, act=None):
        return cls(*mx_quantize_3d(w), bias=bias, act=act)

    def workspace(self, M: int, device):
        need = self._need.get(M)
        if need is None:
            need = self._need[M] = mxfp8_linear_fused_workspace_size(M, self.N, self.K)
        if not need:
            return None
        if self._ws is None or self._ws.numel() < need:
            self._ws = _empty(need, dtype=_U8, device=device)
        return self._ws

    def __call__(self, x, residual=None, mx_out: bool = False, out=None):
        return _fused(x, self.wq, self.ws_mma, self.bias, ACTIVATIONS[self.act], residual, mx_out,
                      out, self.workspace)


def moe_balance_loss_workspace_size(T: int, E: int) -> int:
    return int(_lib.load().moe_balance_loss_workspace_size(T, E))


# up to this many tokens the loss is one kernel without a workspace
_BALANCE_ONE_KERNEL = 1024


def _balance(logits, topk_ids, mask, counts, coef, grad):
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor (the library has no CPU path)")
    shape = logits.shape
    if logits.dtype is not _F32 or len(shape) != 2:
        raise TypeError("logits: expected fp32 [T, E]")
    T, E = shape
    if E > 1 and logits.stride(1) != 1:
        raise ValueError("logits: a row must be contiguous")
    ldl = logits.stride(0) if T > 1 else E
    if ldl < E:
        raise ValueError("logits: overlapping rows")
    _rows(topk_ids, "topk_ids", (torch.int32,))
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError("logits and topk_ids disagree on T")
    mask_ptr = counts_ptr = grad_ptr = None
    if mask is not None:
        _rows(mask, "mask", (torch.bool, torch.uint8))
        if mask.shape != (T,):
            raise ValueError(f"mask is {tuple(mask.shape)}, logits have T = {T}")
        mask_ptr = mask.data_ptr()
    if counts is not None:
        _rows(counts, "counts", (_I64,))
        if counts.shape != (E,):
            raise ValueError(f"counts is {tuple(counts.shape)}, logits have E = {E}")
        counts_ptr = counts.data_ptr()
    dev = logits.device
    lib = _lib.load()
    ws_ptr, need = None, 0
    if T > _BALANCE_ONE_KERNEL:
        need = lib.moe_balance_loss_workspace_size(T, E)
        ws = _empty(need, dtype=_U8, device=dev)
        ws_ptr = ws.data_ptr()
    loss = _empty((), dtype=_F32, device=dev)
    own_counts = _empty(E, dtype=_I64, device=dev)
    out = {"loss": loss, "counts": own_counts}
    if grad:
        out["dlogits"] = d = _empty(shape, dtype=_F32, device=dev)
        grad_ptr = d.data_ptr()
    rc = lib.moe_balance_loss(
        logits.data_ptr(), ldl, topk_ids.data_ptr(), mask_ptr, counts_ptr, T, E,
        topk_ids.shape[1], coef, loss.data_ptr(), own_counts.data_ptr(), grad_ptr, ws_ptr, need,
        _raw_stream(dev.index))
    if rc:
        _lib.check("moe_balance_loss", rc)
    return out


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk_ids, mask, counts, coef):
        r = _balance(logits, topk_ids, mask, counts, coef, True)
        ctx.save_for_backward(r["dlogits"])
        ctx.mark_non_differentiable(r["counts"])
        return r["loss"], r["counts"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        return ctx.saved_tensors[0] * dloss, None, None, None, None


def moe_balance_loss(logits, topk_ids, mask=None, counts=None, coef: float = 1.0,
                     grad: bool = False) -> dict:
    """The router's load-balance loss coef * E * sum_e f_e mean_t p_te.

    logits fp32 [T, E] (rows may be further apart), topk_ids int32 [T, k] (of
    ``moe_router_gate_topk``), mask bool or uint8 [T] (True: the token counts),
    counts int64 [E] to take f from instead of this call's own (e.g. summed
    over micro-batches or ranks).  Returns ``loss`` (fp32 scalar) and ``counts``
    (int64 [E], this call's).  The loss and its gradient come from one pass:
    with ``grad`` the result holds ``dlogits`` fp32 [T, E]; without it, and
    with logits that require a gradient, ``loss`` is differentiable by
    autograd (once)."""
    if not grad and isinstance(logits, torch.Tensor) and logits.requires_grad \
            and torch.is_grad_enabled():
        loss, own = _BalanceLoss.apply(logits, topk_ids, mask, counts, float(coef))
        return {"loss": loss, "counts": own}
    return _balance(logits, topk_ids, mask, counts, float(coef), grad)
