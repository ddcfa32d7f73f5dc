"""The oracle of the operators around the expert forward against closed forms
and differences, and the refusals of their entry points (no GPU needed)."""

import ctypes as C
import math

import numpy as np
import pytest

from oracle import block


@pytest.fixture(scope="module")
def lib():
    from mxfp8_block_scaled_moe_gb300 import _lib, build
    build.build()
    return _lib.load()


def test_rmsnorm_of_a_constant_row_is_the_weight():
    h, y = block.add_rmsnorm(np.full((2, 32), 3.0), np.arange(32.0), 0.0, np.full((2, 32), -1.0))
    assert np.array_equal(h, np.full((2, 32), 2.0))
    assert np.allclose(y, np.arange(32.0)[None, :], rtol=1e-15)
    assert np.array_equal(block.add_rmsnorm(np.zeros((1, 16)), np.ones(16), 1e-6)[1],
                          np.zeros((1, 16)))


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations(act):
    z = np.array([-60.0, -3.0, -0.5, 0.0, 0.5, 3.0, 60.0])
    v = block.activation(act, z)
    assert v[3] == 0.0 and abs(v[0]) < 1e-20 and v[6] == 60.0
    # each is z * g(z) with g(z) + g(-z) = 1, so v(z) - v(-z) = z
    assert np.allclose(v[[4, 5, 6]] - v[[2, 1, 0]], z[4:], rtol=1e-14)
    if act == "gelu":
        assert v[4] == pytest.approx(0.25 * (1 + math.erf(0.5 / math.sqrt(2))), rel=1e-14)
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (0.5 + 0.044715 * 0.125)
        assert v[4] == pytest.approx(0.25 * (1 + math.tanh(u)), rel=1e-14)


def test_balance_loss_of_uniform_routing_is_one():
    T, E, k = 12, 6, 2
    ids = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    loss, counts, grad = block.balance_loss(np.zeros((T, E)), ids)
    assert loss == pytest.approx(1.0, rel=1e-15)
    assert np.array_equal(counts, np.full(E, T * k // E))
    assert np.abs(grad).max() < 1e-17


@pytest.mark.parametrize("given", [False, True])
def test_balance_gradient_against_differences(given):
    rng = np.random.default_rng(5)
    T, E, k = 9, 7, 3
    z = rng.standard_normal((T, E))
    ids = np.argsort(-z, axis=1)[:, :k]
    mask = np.array([1, 1, 0, 1, 1, 1, 0, 1, 1])
    counts = rng.integers(0, 50, E) if given else None
    args = dict(mask=mask, counts=counts, coef=0.3)
    grad = block.balance_loss(z, ids, **args)[2]
    h = 1e-5
    for t in range(T):
        for e in range(E):
            d = np.zeros((T, E))
            d[t, e] = h
            num = (block.balance_loss(z + d, ids, **args)[0]
                   - block.balance_loss(z - d, ids, **args)[0]) / (2 * h)
            assert num == pytest.approx(grad[t, e], abs=1e-9)


def test_balance_loss_of_nothing():
    ids = np.zeros((3, 1), int)
    z = np.full((3, 4), np.nan)
    loss, counts, grad = block.balance_loss(z, ids, mask=np.zeros(3))
    assert loss == 0 and not counts.any() and not grad.any()
    assert block.balance_loss(np.zeros((0, 4)), np.zeros((0, 1), int))[0] == 0
    # a row of -inf has probability 0 everywhere
    loss, _, grad = block.balance_loss(np.full((3, 4), -np.inf), ids)
    assert loss == 0 and not grad.any()


# ---------------------------------------------------------------- refusals

P, ODD, NUL = C.c_void_p(4096), C.c_void_p(4097), C.c_void_p(0)
P16 = C.c_void_p(4096 + 16)


def _norm(lib, **kw):
    a = dict(x=P, ldx=64, residual=P, residual_fp32=0, residual_out=P, weight=P, weight_fp32=0,
             eps=1e-6, M=4, H=64, y=P, q=P, ldq=64, scale=P, mma=0, stream=NUL)
    a.update(kw)
    return lib.mx_add_rmsnorm_quant(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(H=72), 3), (dict(H=0), 3), (dict(M=-1), 3), (dict(ldx=48), 3), (dict(M=1 << 31), 3),
    (dict(eps=-1.0), 3), (dict(eps=float("nan")), 3), (dict(H=32784, ldx=32784, ldq=32784), 4),
    (dict(ldq=48), 3), (dict(ldq=72), 2),
    (dict(x=NUL), 1), (dict(weight=NUL), 1), (dict(q=NUL), 1), (dict(scale=NUL), 1),
    (dict(residual=NUL), 1), (dict(residual_out=NUL), 1), (dict(x=ODD), 2), (dict(ldx=68), 2),
    (dict(weight=P16), 2), (dict(residual=P16), 2), (dict(residual_out=P16), 2), (dict(y=P16), 2),
    (dict(M=0, x=NUL, q=NUL), 0)])
def test_norm_refusals(lib, kw, code):
    assert _norm(lib, **kw) == code


def _linear(lib, **kw):
    a = dict(x=P, xq=NUL, ldx=64, xs=NUL, wq=P, ldw=64, ws=P, M=4, N=64, K=64, bias=P, bias32=0,
             act=1, residual=P, out=P, oq=NUL, ldo=64, os=NUL, ws_=P, ws_bytes=1 << 30, stream=NUL)
    a.update(kw)
    return lib.mxfp8_linear_fused(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(K=40), 3), (dict(N=40), 3), (dict(M=-1), 3), (dict(M=1 << 24), 3), (dict(act=5), 3),
    (dict(act=-1), 3), (dict(oq=P, os=P), 4), (dict(out=NUL, oq=P, os=P), 4),
    (dict(xq=P, xs=P), 4), (dict(wq=NUL), 1), (dict(ws=NUL), 1), (dict(x=NUL), 1),
    (dict(x=NUL, xq=P), 1), (dict(out=NUL, residual=NUL), 1),
    (dict(out=NUL, residual=NUL, oq=P), 1), (dict(x=ODD), 2), (dict(wq=ODD), 2),
    (dict(bias=ODD), 2), (dict(residual=ODD), 2), (dict(out=ODD), 2), (dict(M=33, ws_=NUL), 5),
    (dict(ldw=48), 3), (dict(ldw=72), 2),
    (dict(x=NUL, xq=P, xs=P, ldx=48), 3), (dict(x=NUL, xq=P, xs=P, ldx=72), 2),
    (dict(out=NUL, residual=NUL, oq=P, os=P, ldo=48), 3),
    (dict(out=NUL, residual=NUL, oq=P, os=P, ldo=72), 2), (dict(M=33, ws_bytes=256), 5), (dict(M=33, ws_=P16), 2), (dict(M=0, x=NUL, wq=NUL, ws_=NUL), 0)])
def test_linear_refusals(lib, kw, code):
    assert _linear(lib, **kw) == code


def _bal(lib, **kw):
    a = dict(logits=P, ldl=8, ids=P, mask=P, counts_in=P, T=4, E=8, k=2, coef=1.0, loss=P,
             counts=P, dlogits=P, ws=P, ws_bytes=1 << 20, stream=NUL)
    a.update(kw)
    return lib.moe_balance_loss(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 3), (dict(E=0), 3), (dict(k=0), 3), (dict(k=9), 3), (dict(ldl=7), 3),
    (dict(T=1 << 30), 3), (dict(E=1025, ldl=1025), 4), (dict(E=64, ldl=64, k=33), 4),
    (dict(logits=NUL), 1), (dict(ids=NUL), 1), (dict(loss=NUL), 1), (dict(counts=NUL), 1),
    (dict(logits=ODD), 2), (dict(counts=ODD), 2), (dict(ws=ODD), 2), (dict(T=4096, ws=NUL), 5),
    (dict(T=4096, ws_bytes=8), 5)])
def test_balance_refusals(lib, kw, code):
    assert _bal(lib, **kw) == code


def test_workspace_sizes(lib):
    assert lib.mxfp8_linear_fused_workspace_size(200, 64, 336) >= 200 * 336 + 2 * 3 * 512
    assert lib.mxfp8_linear_fused_workspace_size(100, 64, 40) == 0
    # few rows and a K range that fits are quantized in the product's kernel
    assert lib.mxfp8_linear_fused_workspace_size(8, 64, 64) == 0
    assert lib.mxfp8_linear_fused_workspace_size(33, 64, 64) > 0
    assert lib.mxfp8_linear_fused_workspace_size(-1, 64, 64) == 0
    assert lib.moe_balance_loss_workspace_size(16384, 128) >= 128 * 4
    assert lib.moe_balance_loss_workspace_size(4, 2000) == 0
    # one kernel without a workspace up to 1024 tokens
    assert lib.moe_balance_loss_workspace_size(1024, 128) == 0
    assert lib.moe_balance_loss_workspace_size(1025, 128) > 0


def test_bindings_refuse():
    import torch

    import mxfp8_block_scaled_moe_gb300 as mm
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    u = torch.zeros(64, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        mm.mx_add_rmsnorm_quant(x, torch.ones(64))
    with pytest.raises(ValueError, match="CUDA"):
        mm.mxfp8_linear_fused(x, u, u)
    with pytest.raises(ValueError, match="CUDA"):
        mm.moe_balance_loss(torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32))
