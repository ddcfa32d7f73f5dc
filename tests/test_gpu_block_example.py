"""The block example: its parts meet as they are used together.

Its dense expert is checked against the 64-bit oracle on the block's own MXFP8
input, with the routed experts' result as the block computed it.  Tolerance:
the product rounds once to bf16, 2^-8 of the result.  The MXFP8 rows between the
two products may differ from the oracle's requantisation in 0.1% of their
elements by one step (2^-3 of the element at most): 2^-3 of the magnitude of
that many terms, taken as 2^-3 of the largest 0.2% of each result's terms."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import block as ob, mx

from _util import bits16, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples",
                        "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return mx.bf16_bits_to_f64(bits16(t))


@pytest.mark.parametrize("T", [1, 70, 600])
def test_block(ex, T):
    E, H, I, S, k = 8, 256, 128, 400, 2
    b = ex.random_block(E=E, H=H, I=I, S=S, k=k)
    torch.manual_seed(T)
    x, res = (torch.randn(T, H, device="cuda").bfloat16() for _ in range(2))
    out, stream = b(x, res)
    torch.cuda.synchronize()
    h, y = ob.add_rmsnorm(f64(x), np.ones(H), 1e-6, f64(res))
    assert np.array_equal(f64(stream), h)
    n = b.normed(x, res)
    assert np.all(np.abs(f64(n["y"]) - y) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(y))
    routed = f64(b.experts(n["y"], b.route(n["y"])["logits"]))

    def weight(lin):
        q, s = u8(lin.wq), u8(lin.ws_mma)
        KT = s.shape[-1] // 4
        s = s.reshape(-1, KT, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(-1, KT * 4)
        return mx.mx_dequantize(q, s[:q.shape[0], :-(-q.shape[1] // 32)])

    a = ob.linear_fused(mx.mx_dequantize(*mx.mx_quantize(f64(n["y"]))), weight(b.up), None, "silu")
    pad = np.pad(a, ((0, 0), (0, -S % 32)))
    av = mx.mx_dequantize(*mx.mx_quantize(pad))[:, :S]
    wd = weight(b.down)
    want = av @ wd.T + routed
    terms = np.sort(np.abs(av)[:, None, :] * np.abs(wd)[None], axis=-1)
    slack = 2.0 ** -3 * terms[..., -max(1, S // 500):].sum(-1)
    got = f64(out)
    assert np.all(np.abs(got - want) <= slack + 2.0 ** -8 * (np.abs(want) + slack) + 2.0 ** -20)
    # the same bits again
    assert torch.equal(out, b(x, res)[0])


def test_balance_training_evens_the_load(ex):
    b = ex.random_block(E=16, H=256, I=128, S=256, k=2)
    torch.manual_seed(3)
    x = (torch.randn(2000, 256, device="cuda") + torch.randn(256, device="cuda")).bfloat16()
    res = torch.randn(2000, 256, device="cuda").bfloat16()
    mask = torch.arange(2000, device="cuda") % 4 != 0
    first, counts = b.balance_step(x, res, mask)
    assert int(counts.sum()) == 2 * int(mask.sum())
    for _ in range(30):
        last, after = b.balance_step(x, res, mask)
    assert float(last) < float(first) and int(after.max()) < int(counts.max())
