"""GPU parity of the operators around the expert forward with the 64-bit oracle.

Tolerances (half a step of a type is eps / 2: bf16 2^-8, fp32 2^-24):

* residual stream, MXFP8 codes and scales of the norm (against the oracle's
  quantizer on the device's own bf16 rows), counts, exactness pins of the
  product: bit for bit;
* normed rows: the bf16 rounding, 2^-8, and the fp32 statistics and products,
  fewer than 2^7 roundings of 2^-24 (half of them under a square root);
* product: the bf16 rounding of the result, and the fp32 accumulation,
  K * 2^-24 * sum |x w| carried through an activation of slope < 1.2, and the
  activation itself, 2^-16 relative (a few roundings of an exponent's argument
  of up to 2^5);
* MXFP8 result of the product: at most 0.1% of the elements off, by one step;
* loss and gradient: softmax terms e^-a with a < 2^6 carry a 2^-24 rounding of
  a, the sums up to E / 32 + 5 roundings: 2^-16 relative to the terms' sizes.
"""

import math

import numpy as np
import pytest
import torch

from oracle import block, mx

from _util import bits16, requant_mismatch, to_bf16_tensor, u8

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()
    import mxfp8_block_scaled_moe_gb300 as m
    return m


def f64(t):
    if t.dtype == torch.bfloat16:
        return mx.bf16_bits_to_f64(bits16(t))
    return t.cpu().numpy().astype(np.float64)


def untile(s, rows, K):
    """[rows, ceil(K/32)] of the tensor-core layout, and its padding slots of those rows."""
    KT = -(-K // 128)
    s = u8(s).reshape(-1, KT, 32, 4, 4)            # row block, slice, r % 32, r / 32, kb
    s = s.transpose(0, 3, 2, 1, 4).reshape(-1, KT * 4)[:rows]
    nb = -(-K // 32)
    return s[:, :nb], s[:, nb:]


def randn(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * scale


# ---------------------------------------------------------------- norm

def check_norm(mm, x, w, res, eps=1e-6, **kw):
    r = mm.mx_add_rmsnorm_quant(x, w, residual=res, eps=eps, bf16_out=True, **kw)
    torch.cuda.synchronize()
    H = x.shape[-1]
    rd = "fp32" if res is not None and res.dtype == torch.float32 else "bf16"
    h, y = block.add_rmsnorm(f64(x), f64(w), eps, None if res is None else f64(res), rd)
    if res is not None:
        assert np.array_equal(f64(r["residual"]), h)
    yd = f64(r["y"])
    assert np.all(np.abs(yd - y) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(y) + 2.0 ** -133)
    q, s = mx.mx_quantize(yd.reshape(-1, H))
    assert np.array_equal(u8(r["q"]).reshape(-1, H), q)
    if kw.get("mma_scales"):
        got, pad = untile(r["s"], q.shape[0], H)
        assert np.array_equal(got, s) and np.all(pad == 127)
    else:
        assert np.array_equal(u8(r["s"]).reshape(s.shape), s)
    return r


@pytest.mark.parametrize("M,H", [(1, 16), (3, 48), (1, 2048), (130, 336), (5, 1152), (257, 4304),
                                 (2, 12288), (3, 16400), (2, 32768), (1000, 2048), (7, 4096)])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
def test_norm(mm, M, H, res):
    x = randn(M + H, M, H).bfloat16()
    x[:, ::37] *= 20
    w = 1 + 0.1 * randn(H, H)
    for wt, mma in ((torch.bfloat16, False), (torch.float32, True)):
        check_norm(mm, x, w.to(wt), None if res is None else randn(7, M, H).to(res),
                   mma_scales=mma)


def test_norm_special_rows(mm):
    H = 272
    x = randn(3, 6, H).bfloat16()
    x[0] = 0                                       # a zero row
    x[1] = 1e-20                                   # below eps
    x[2, :32] = 0                                  # a zero block
    x[3] *= 1e15
    x[4, 5] = 3e4                                  # one element carries the row
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    w[40] = 0
    r = check_norm(mm, x, w, None)
    assert not u8(r["q"])[0].any() and not u8(r["s"])[0].any()
    check_norm(mm, x, w, -x)                       # the sum cancels: zero rows
    check_norm(mm, x[3:5], w, None, eps=0.0)


def test_norm_views_in_place_and_leading_dimensions(mm):
    x = randn(1, 9, 400).bfloat16()
    w = torch.ones(336, device=DEV)
    # rows of a wider tensor, aligned to 32 and to 16 bytes only
    a = check_norm(mm, x[:, :336], w, None)
    for off in (0, 16, 8, 56):
        v = x[:, off:off + 336]
        b = check_norm(mm, v, w, None)
        c = mm.mx_add_rmsnorm_quant(v.contiguous(), w)
        assert torch.equal(b["q"], c["q"]) and torch.equal(b["s"], c["s"])
    with pytest.raises(mm.api._lib.MXMoEError) as e:
        mm.mx_add_rmsnorm_quant(x[:, 4:340], w)
    assert e.value.code == 2
    # a residual stream updated in place
    for dt in (torch.bfloat16, torch.float32):
        res = randn(2, 9, 336).to(dt)
        want = mm.mx_add_rmsnorm_quant(x[:, :336], w, residual=res)
        got = mm.mx_add_rmsnorm_quant(x[:, :336], w, residual=res, residual_out=res)
        assert got["residual"] is res and torch.equal(res, want["residual"])
        assert torch.equal(got["q"], want["q"])
    # [.., H] and no rows
    x3 = randn(4, 2, 3, 336).bfloat16()
    r = mm.mx_add_rmsnorm_quant(x3, w, bf16_out=True)
    flat = mm.mx_add_rmsnorm_quant(x3.view(6, 336), w)
    assert r["q"].shape == (2, 3, 336) and r["s"].shape == (2, 3, 11)
    assert torch.equal(r["q"].view(6, 336), flat["q"])
    assert mm.mx_add_rmsnorm_quant(x[:0, :336], w)["q"].shape == (0, 336)
    assert a["y"].shape == (9, 336)


def test_norm_bytes_are_those_of_the_separate_quantizer(mm):
    x, w = randn(5, 300, 2048).bfloat16(), randn(6, 2048).bfloat16()
    r = mm.mx_add_rmsnorm_quant(x, w, bf16_out=True)
    q, s = mm.mx_quantize_3d(r["y"])
    assert torch.equal(r["q"], q) and torch.equal(r["s"], s)
    t = mm.mx_add_rmsnorm_quant(x, w, mma_scales=True)
    ref, _ = untile(mm.mx_scales_to_mma_layout(s, 2048), 300, 2048)
    assert np.array_equal(untile(t["s"], 300, 2048)[0], ref)


def test_norm_refusals(mm):
    x, w = randn(1, 4, 64).bfloat16(), torch.ones(64, device=DEV)
    for bad in (lambda: mm.mx_add_rmsnorm_quant(x, w[:32]),
                lambda: mm.mx_add_rmsnorm_quant(x, w, residual=x[:2]),
                lambda: mm.mx_add_rmsnorm_quant(x, w, residual_out=x),
                lambda: mm.mx_add_rmsnorm_quant(x, w, residual=x, residual_out=x[:2].clone()),
                lambda: mm.mx_add_rmsnorm_quant(x[:1].expand(4, 64), w),
                lambda: mm.mx_add_rmsnorm_quant(x.view(2, 2, 64).transpose(0, 1), w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mm.mx_add_rmsnorm_quant(x.float(), w),
                lambda: mm.mx_add_rmsnorm_quant(x, w.half()),
                lambda: mm.mx_add_rmsnorm_quant(x, w, residual=x.half())):
        with pytest.raises(TypeError):
            bad()


# ---------------------------------------------------------------- fused product

def lossless(rng, rows, K):
    """Integer values an MXFP8 row holds exactly, with block scales around 1."""
    v = rng.integers(-8, 9, (rows, K)).astype(np.float64)
    v[:, ::32] = 8.0                               # the block maximum fixes its scale
    v[:, -1] = 8.0
    return v


SHAPES = [(1, 16, 16), (1, 128, 4096), (5, 400, 336), (32, 4096, 1024), (33, 144, 272),
          (64, 256, 2048), (100, 4304, 160), (128, 512, 512), (129, 1152, 4304), (200, 400, 336),
          (257, 272, 1040), (600, 2048, 768), (1500, 4096, 256), (4096, 1040, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_exactness_pins(mm, M, N, K):
    """Every partial sum exact in fp32, so the bf16 result is the oracle's, bit for bit."""
    rng = np.random.default_rng(M + N + K)
    xv, wv = lossless(rng, M, K), lossless(rng, N, K)
    bias = rng.integers(-20, 21, N).astype(np.float64)
    res = rng.integers(-30, 31, (M, N)).astype(np.float64)
    x = to_bf16_tensor(mx.f64_to_bf16_bits(xv), DEV)
    w = to_bf16_tensor(mx.f64_to_bf16_bits(wv), DEV)
    bt = to_bf16_tensor(mx.f64_to_bf16_bits(bias), DEV)
    rt = to_bf16_tensor(mx.f64_to_bf16_bits(res), DEV)
    z = xv @ wv.T
    for b, act, r in ((None, None, None), (bt, "relu", rt), (bt.float(), "none", None)):
        want = block.activation(act, z + (0 if b is None else bias)) + (0 if r is None else res)
        got = mm.MXFP8FusedLinear.from_bf16(w, bias=b, act=act)(x, residual=r)
        torch.cuda.synchronize()
        assert mm.device_status() == 0
        assert np.array_equal(bits16(got), mx.f64_to_bf16_bits(want)), (b is None, act)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 400, 336), (32, 1040, 12288),
                                   (100, 144, 4304), (300, 1152, 1168), (2100, 4304, 256)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_values(mm, M, N, K, act):
    x = randn(M + K, M, K).bfloat16()
    x[:, ::101] *= 20
    lin = mm.MXFP8FusedLinear.from_bf16(randn(N, N, K, scale=0.02).bfloat16(), act=act,
                                        bias=randn(3, N).to((torch.bfloat16, torch.float32)[M % 2]))
    wq, ws = mm.mx_quantize_3d(randn(N, N, K, scale=0.02).bfloat16())
    res = randn(9, M, N, scale=2).bfloat16()
    pick = np.unique(np.r_[0, M - 1, np.random.default_rng(0).integers(0, M, 40)])
    xv = mx.mx_dequantize(*mx.mx_quantize(f64(x[torch.from_numpy(pick).to(DEV)])))
    wv = mx.mx_dequantize(u8(wq), u8(ws))
    v = block.linear_fused(xv, wv, f64(lin.bias), act)
    acc = 1.2 * K * 2.0 ** -24 * (np.abs(xv) @ np.abs(wv).T + np.abs(f64(lin.bias)))
    err = acc + 2.0 ** -16 * np.abs(v) + 2.0 ** -100
    for r in (None, res):
        got = f64(lin(x, residual=r))[pick]
        want = v if r is None else v + f64(r)[pick]
        assert np.all(np.abs(got - want) <= err + 2.0 ** -8 * (np.abs(want) + err))
    q, s = lin(x, mx_out=True)
    torch.cuda.synchronize()
    assert mm.device_status() == 0
    got_s, pad = untile(s, M, N)
    assert np.all(pad == 127)
    wide = lambda a: np.pad(a, ((0, 0), (0, -N % 32)))  # noqa: E731  whole blocks
    qv, sv = mx.mx_quantize(v)
    frac, step = requant_mismatch(wide(u8(q)[pick]), got_s[pick], wide(qv), sv)
    assert frac <= 1e-3 and step <= 1.0, (frac, step)


def test_linear_input_forms_agree(mm):
    """bf16 rows, the norm's MXFP8 rows and a product's MXFP8 rows."""
    for M in (1, 40, 300, 1100):
        x, w = randn(M, M, 1152).bfloat16(), randn(1, 1152)
        lin = mm.MXFP8FusedLinear.from_bf16(randn(2, 4304, 1152, scale=0.02).bfloat16())
        r = mm.mx_add_rmsnorm_quant(x, w, mma_scales=True, bf16_out=True)
        assert torch.equal(lin((r["q"], r["s"])), lin(r["y"]))
        # a relu of lossless integers in MXFP8 is read back as it is
    rng = np.random.default_rng(1)
    v = lossless(rng, 70, 336)
    eye = to_bf16_tensor(mx.f64_to_bf16_bits(np.eye(336)), DEV)
    one = mm.MXFP8FusedLinear.from_bf16(eye, act="relu")
    x = to_bf16_tensor(mx.f64_to_bf16_bits(v), DEV)
    pair = one(x, mx_out=True)
    assert np.array_equal(f64(one(pair)), np.maximum(v, 0))
    assert np.array_equal(f64(one(x)), np.maximum(v, 0))


def test_linear_plain_equals_the_existing_linear(mm):
    for M, N, K in ((200, 400, 336), (1024, 1024, 2048)):
        x, w = randn(1, M, K).bfloat16(), randn(2, N, K, scale=0.02).bfloat16()
        a, b = mm.MXFP8FusedLinear.from_bf16(w)(x), mm.MXFP8Linear.from_bf16(w)(x)
        err = (f64(a) - f64(b))
        # both round the same sum, accumulated in another order
        assert np.all(np.abs(err) <= 2.0 ** -7 * np.abs(f64(b)) + K * 2.0 ** -24 * 400)


def test_linear_in_place_strided_and_repeated(mm):
    M, N, K = 150, 336, 512
    lin = mm.MXFP8FusedLinear.from_bf16(randn(2, N, K, scale=0.02).bfloat16(), act="silu")
    x, res = randn(1, M, K).bfloat16(), randn(3, M, N).bfloat16()
    want = lin(x, residual=res)
    for _ in range(3):
        assert torch.equal(lin(x, residual=res), want)
    acc = res.clone()
    assert lin(x, residual=acc, out=acc) is acc and torch.equal(acc, want)
    assert torch.equal(lin(x.view(10, 15, K), residual=res.view(10, 15, N)).view(M, N), want)
    assert lin(x[:0]).shape == (0, N)
    big = torch.empty(M * N + 8, dtype=torch.bfloat16, device=DEV)   # 16-byte aligned only
    out = big[8:].view(M, N)
    assert torch.equal(lin(x, residual=res, out=out), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = lin(x, residual=res)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)


def test_linear_payload_rows_further_apart(mm):
    """Pairs and weights whose rows are 16 bytes or more apart from packed ones."""
    for M in (7, 300):
        for N, K in ((400, 336), (272, 512)):
            x = randn(M, M, K).bfloat16()
            lin = mm.MXFP8FusedLinear.from_bf16(randn(2, N, K, scale=0.02).bfloat16(), act="silu")
            r = mm.mx_add_rmsnorm_quant(x, torch.ones(K, device=DEV), mma_scales=True)
            q, want = r["q"].contiguous(), lin((r["q"], r["s"]))
            mid = lin((r["q"], r["s"]), mx_out=True)
            assert torch.equal(lin((q, r["s"])), want)
            for pad in (16, 48, 128):
                wide = torch.full((M, K + pad), 0x7F, dtype=torch.uint8, device=DEV)
                wide[:, :K] = q
                w = torch.full((N, K + pad), 0x7F, dtype=torch.uint8, device=DEV)
                w[:, :K] = lin.wq
                got = mm.mxfp8_linear_fused((wide[:, :K], r["s"]), w[:, :K], lin.ws_mma, act="silu")
                assert torch.equal(got, want)
                m = mm.mxfp8_linear_fused((wide[:, :K], r["s"]), w[:, :K], lin.ws_mma, act="silu",
                                          mx_out=True)
                assert torch.equal(m[0], mid[0])
                assert np.array_equal(untile(m[1], M, N)[0], untile(mid[1], M, N)[0])
            with pytest.raises(mm.api._lib.MXMoEError):
                mm.mxfp8_linear_fused((torch.empty(M, K + 8, dtype=torch.uint8, device=DEV)[:, :K],
                                       r["s"]), lin.wq, lin.ws_mma)


def test_linear_rows_do_not_depend_on_their_neighbours(mm):
    """A row of NaN, of infinities and of zeros beside ordinary ones."""
    lin = mm.MXFP8FusedLinear.from_bf16(randn(2, 256, 512, scale=0.02).bfloat16())
    for M in (6, 300):
        x = randn(1, M, 512).bfloat16()
        want = lin(x)
        x[1], x[2], x[4, 7] = float("nan"), 0, float("inf")
        got = lin(x)
        keep = [i for i in range(M) if i not in (1, 2, 4)]
        assert torch.equal(got[keep], want[keep])
        assert got[1].isnan().all() and not got[2].any()


def test_linear_refusals(mm):
    lin = mm.MXFP8FusedLinear.from_bf16(randn(2, 64, 128).bfloat16())
    x = randn(1, 4, 128).bfloat16()
    r = mm.mx_add_rmsnorm_quant(x, torch.ones(128, device=DEV))
    for bad in (lambda: lin(x[:, :64].contiguous()), lambda: lin(x, residual=x),
                lambda: lin(x, residual=torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV),
                            mx_out=True),
                lambda: lin((r["q"], r["s"])),        # row-major scales
                lambda: lin(x.t().contiguous().t()),
                lambda: lin(x, out=torch.zeros(4, 32, dtype=torch.bfloat16, device=DEV)),
                lambda: mm.MXFP8FusedLinear(lin.wq, torch.zeros(64, 4, dtype=torch.uint8,
                                                                device=DEV), act="tanh")(x),
                lambda: mm.mxfp8_linear_fused(x, lin.wq, lin.ws_mma[:32])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        lin(x.float())


# ---------------------------------------------------------------- balance loss

def balance_case(seed, T, E, k, masked=0.0, scale=1.0):
    z = randn(seed, T, E, scale=scale) + 0.5 * randn(seed + 1, E)
    ids = torch.topk(z, k, dim=1).indices.to(torch.int32)
    mask = None
    if masked:
        mask = torch.from_numpy(np.random.default_rng(seed).random(T) >= masked).to(DEV)
    return z, ids, mask


def check_balance(mm, z, ids, mask=None, counts=None, coef=1.0):
    r = mm.moe_balance_loss(z, ids, mask=mask, counts=counts, coef=coef, grad=True)
    torch.cuda.synchronize()
    assert mm.device_status() == 0
    num = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    loss, own, grad = block.balance_loss(num(z), num(ids), num(mask), num(counts), coef)
    assert np.array_equal(num(r["counts"]), own)
    assert abs(float(r["loss"]) - loss) <= 2.0 ** -16 * abs(loss)
    T, E = z.shape
    n = T if mask is None else max(1, int(num(mask).sum()))
    c = own if counts is None else num(counts)
    f = c / max(1, c.sum())
    live = np.ones(T) if mask is None else num(mask)
    with np.errstate(invalid="ignore"):
        zz = np.where(live[:, None] != 0, num(z).astype(np.float64), 0)
        top = zz.max(1, keepdims=True)
        p = np.exp(zz - np.where(np.isneginf(top), 0, top))
        p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    size = abs(coef) * E / n * p * (f[None, :] + (p @ f)[:, None])
    assert np.all(np.abs(num(r["dlogits"]) - grad) <= 2.0 ** -16 * size + 1e-37)
    return r


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (64, 8, 2), (33, 6, 6), (100, 60, 4),
                                   (257, 128, 8), (1000, 256, 8), (300, 512, 3), (70, 1000, 32),
                                   (9, 1024, 32), (5000, 33, 5), (16384, 128, 8), (2048, 64, 1)])
@pytest.mark.parametrize("masked", [0.0, 0.3])
def test_balance(mm, T, E, k, masked):
    z, ids, mask = balance_case(T + E, T, E, k, masked)
    check_balance(mm, z, ids, mask)
    counts = torch.from_numpy(np.random.default_rng(1).integers(0, 10 ** 12, E)).to(DEV)
    check_balance(mm, z, ids, mask, counts, coef=0.01)


def test_balance_rows_apart_and_unaligned(mm):
    z, ids, _ = balance_case(3, 200, 160, 4)
    for off, E in ((0, 128), (3, 128), (4, 128), (1, 61)):
        v = z[:, off:off + E]
        i = torch.topk(v, 4, dim=1).indices.to(torch.int32)
        a = check_balance(mm, v, i)
        b = mm.moe_balance_loss(v.contiguous(), i, grad=True)
        assert torch.equal(a["dlogits"], b["dlogits"]) and torch.equal(a["loss"], b["loss"])
    with pytest.raises(ValueError):
        mm.moe_balance_loss(z.t(), ids)


@pytest.mark.parametrize("T,E", [(40, 16), (3000, 128)])
def test_balance_empty_and_infinite_rows(mm, T, E):
    z, ids, _ = balance_case(5, T, E, 2, scale=3.0)
    z[3] = float("-inf")                               # a row without an expert
    z[4, 1:] = float("-inf")                           # with one
    z[5, ::2] = float("-inf")
    z[6] = torch.finfo(torch.float32).min
    z[7] = torch.finfo(torch.float32).max
    z[8] *= 1e4
    check_balance(mm, z, ids)
    # masked tokens hold anything, their ids too
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    mask[::3] = False
    zm, im = z.clone(), ids.clone()
    zm[::3] = float("nan")
    im[::3] = -7
    a, b = check_balance(mm, z, ids, mask), mm.moe_balance_loss(zm, im, mask=mask, grad=True)
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["dlogits"], b["dlogits"])
    assert mm.device_status() == 0
    # NaN in a counted row reaches the loss and that row's gradient only
    zm = z.clone()
    zm[10, 3] = float("nan")
    r = mm.moe_balance_loss(zm, ids, grad=True)
    assert r["loss"].isnan() and r["dlogits"][10].isnan().all()
    assert torch.equal(r["dlogits"][11:], mm.moe_balance_loss(z, ids, grad=True)["dlogits"][11:])
    # nothing counted, nothing given
    r = mm.moe_balance_loss(zm, ids, mask=torch.zeros_like(mask), grad=True)
    assert float(r["loss"]) == 0 and not r["counts"].any() and not r["dlogits"].any()
    r = mm.moe_balance_loss(z, ids, counts=torch.zeros(E, dtype=torch.int64, device=DEV), grad=True)
    assert float(r["loss"]) == 0 and not r["dlogits"].any()
    r = mm.moe_balance_loss(z[:0], ids[:0], grad=True)
    assert float(r["loss"]) == 0 and not r["counts"].any() and r["dlogits"].shape == (0, E)


@pytest.mark.parametrize("T", [100, 4000])
def test_balance_reports_ids_out_of_range(mm, T):
    z, ids, _ = balance_case(6, T, 16, 2)
    bad = ids.clone()
    bad[T - 1, 1] = 16
    bad[0, 0] = -1
    r = mm.moe_balance_loss(z, bad)
    assert mm.device_status() == 8 and mm.device_status() == 0
    keep = (bad >= 0) & (bad < 16)
    assert np.array_equal(r["counts"].cpu().numpy(),
                          np.bincount(bad[keep].cpu().numpy(), minlength=16))


def test_balance_gradient_against_differences(mm):
    """Along random directions, differences of the oracle's loss."""
    z, ids, mask = balance_case(8, 300, 48, 4, 0.2)
    d = mm.moe_balance_loss(z, ids, mask=mask, grad=True)["dlogits"].cpu().numpy().astype(np.float64)
    z64, i, m = z.cpu().numpy().astype(np.float64), ids.cpu().numpy(), mask.cpu().numpy()
    rng = np.random.default_rng(0)
    for _ in range(5):
        v = rng.standard_normal(z64.shape)
        h = 1e-4
        num = (block.balance_loss(z64 + h * v, i, m)[0]
               - block.balance_loss(z64 - h * v, i, m)[0]) / (2 * h)
        # the kernel's 2^-16 per term, and h^2 times a third derivative of order 1
        assert abs(num - (d * v).sum()) <= 2.0 ** -16 * (np.abs(d * v)).sum() * 4 + h * h


def test_balance_autograd_and_determinism(mm):
    z, ids, mask = balance_case(9, 700, 64, 4, 0.1)
    r = mm.moe_balance_loss(z, ids, mask=mask, coef=0.5, grad=True)
    zl = z.clone().requires_grad_()
    a = mm.moe_balance_loss(zl, ids, mask=mask, coef=0.5)
    (3.0 * a["loss"]).backward()
    assert torch.equal(a["loss"].detach(), r["loss"]) and torch.equal(a["counts"], r["counts"])
    assert torch.equal(zl.grad, 3.0 * r["dlogits"])
    with torch.no_grad():
        assert not mm.moe_balance_loss(zl, ids, mask=mask)["loss"].requires_grad
    assert "dlogits" not in mm.moe_balance_loss(z, ids)
    for _ in range(5):
        s = mm.moe_balance_loss(z, ids, mask=mask, coef=0.5, grad=True)
        assert torch.equal(s["loss"], r["loss"]) and torch.equal(s["dlogits"], r["dlogits"])


def test_operators_in_a_graph(mm):
    """The block's calls captured into a CUDA graph replay on new inputs."""
    x, res = randn(1, 20, 512).bfloat16(), randn(2, 20, 512).bfloat16()
    w = torch.ones(512, device=DEV)
    fc1 = mm.MXFP8FusedLinear.from_bf16(randn(3, 1040, 512, scale=0.02).bfloat16(), act="silu")
    fc2 = mm.MXFP8FusedLinear.from_bf16(randn(4, 512, 1040, scale=0.02).bfloat16())
    z, ids, _ = balance_case(1, 500, 32, 2)

    def step():
        r = mm.mx_add_rmsnorm_quant(x, w, residual=res, mma_scales=True)
        out = fc2(fc1((r["q"], r["s"]), mx_out=True), residual=r["residual"])
        b = mm.moe_balance_loss(z, ids, grad=True)
        return out, b["loss"], b["dlogits"]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (11, 12):
        x.copy_(randn(seed, 20, 512))
        z.copy_(randn(seed, 500, 32))
        graph.replay()
        want = step()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert mm.device_status() == 0


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [40, 600])
def test_linear_activation_tails(mm, M, act):
    """The activations by themselves (the bias alone, from -16 to 16): nothing but the
    activation's error and the bf16 rounding is left.  Results below 2^-100, where the
    exponentials end, aside.  40 and 600 rows: the split and the pair kernel."""
    z = np.arange(-256, 256) / 16.0
    b = torch.from_numpy(z).to(DEV, torch.float32)
    lin = mm.MXFP8FusedLinear.from_bf16(torch.zeros(512, 64, device=DEV).bfloat16(), bias=b, act=act)
    got = f64(lin(torch.zeros(M, 64, device=DEV).bfloat16()))
    want = block.activation(act, z)
    assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(want) + 2.0 ** -100)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_linear_ragged_block_does_not_see_the_call_before(mm, act):
    """N % 32 == 16: the half block past N holds nothing of an earlier call's bias."""
    x, w = randn(1, 2048, 256).bfloat16(), randn(2, 1040, 256, scale=0.02).bfloat16()
    lin = mm.MXFP8FusedLinear.from_bf16(w, bias=randn(3, 1040), act=act)
    wide = randn(4, 1056, 256, scale=0.02).bfloat16()
    got = []
    for level in (-1e4, 0.0, float("nan")):
        before = mm.MXFP8FusedLinear.from_bf16(wide, bias=torch.full((1056,), level, device=DEV),
                                               act=act)
        before(x, mx_out=True)
        got.append(lin(x, mx_out=True))
    torch.cuda.synchronize()
    for q, s in got[1:]:
        assert torch.equal(q, got[0][0]) and torch.equal(s, got[0][1])


@pytest.mark.parametrize("M,H", [(1, 128), (37, 112), (37, 144), (35, 256), (9, 272), (5, 512)])
@pytest.mark.parametrize("mma_scales", [False, True])
def test_norm_several_rows_per_warp(mm, M, H, mma_scales):
    x, res = (randn(M + H + i, M, H, scale=3).bfloat16() for i in range(2))
    check_norm(mm, x, randn(H, H), None, mma_scales=mma_scales)
    check_norm(mm, x, randn(H, H).bfloat16(), res.float(), mma_scales=mma_scales)


@pytest.mark.parametrize("T,E,k", [(768, 256, 8), (769, 256, 8), (193, 1024, 3), (192, 1024, 3),
                                   (1024, 192, 2), (1030, 7, 3), (3000, 33, 4), (2000, 600, 8)])
def test_balance_kernel_choice_edges(mm, T, E, k):
    z, ids, mask = balance_case(T + E, T, E, k, 0.2)
    check_balance(mm, z, ids, mask)
