"""The operators around the expert forward in a transformer block (CPU oracle,
float64).

TEST INFRASTRUCTURE ONLY -- see the package docstring.

* the residual's addition and the RMS norm whose rows are MX-quantized;
* the dense MXFP8 product with bias, activation and residual;
* the router's load-balance loss, its counts and the logits' gradient.
"""

from __future__ import annotations

import math

import numpy as np

from . import mx


def add_rmsnorm(x, w, eps: float, residual=None, residual_dtype: str = "bf16"):
    """(h, y): h = x + residual rounded to the residual's type (h = x without
    one), y = h * w / sqrt(mean(h^2) + eps), not rounded."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
        if residual_dtype == "bf16":
            h = mx.bf16_bits_to_f64(mx.f64_to_bf16_bits(h))
        else:
            h = h.astype(np.float32).astype(np.float64)
    ms = np.mean(h * h, axis=-1, keepdims=True)
    return h, h / np.sqrt(ms + eps) * np.asarray(w, np.float64)


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activation(name, z):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore"):
        if name == "relu":
            return np.maximum(z, 0.0)
        if name == "gelu":
            return 0.5 * z * _erfc(-z / math.sqrt(2.0))
        if name == "gelu_tanh":
            return z / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
        if name == "silu":
            return z / (1.0 + np.exp(-z))
    return z


def linear_fused(xv, wv, bias=None, act=None):
    """act(xv . wv^T + bias), the operands given by the values they stand for."""
    z = np.asarray(xv, np.float64) @ np.asarray(wv, np.float64).T
    return activation(act, z if bias is None else z + np.asarray(bias, np.float64))


def balance_loss(logits, topk_ids, mask=None, counts=None, coef: float = 1.0):
    """(loss, this call's counts, dlogits)."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    live = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    own = np.bincount(np.asarray(topk_ids)[live].reshape(-1), minlength=E).astype(np.int64)
    c = own if counts is None else np.asarray(counts, np.int64)
    n, total = int(live.sum()), int(c.sum())
    grad = np.zeros((T, E))
    if n == 0 or total == 0:
        return 0.0, own, grad
    f = c / total
    p = np.zeros((T, E))
    zl = z[live]
    top = zl.max(axis=1, keepdims=True)
    e = np.exp(zl - np.where(np.isneginf(top), 0.0, top))
    den = e.sum(axis=1, keepdims=True)
    p[live] = np.divide(e, den, out=np.zeros_like(e), where=den != 0)
    s = p @ f
    loss = coef * E * s.sum() / n
    grad = coef * E / n * p * (f[None, :] - s[:, None])
    return float(loss), own, grad
