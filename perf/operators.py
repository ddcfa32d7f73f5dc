"""What is measured of the operators around the MXFP8 expert forward.

* norm: the residual's addition, the root-mean-square norm and the MXFP8 (e4m3
  payload, one e8m0 scale per 32 elements) output that the products read;
* linear: an MXFP8 product with bias, activation and residual in its epilogue;
* block: norm, product with activation, product with the residual, the two
  intermediates in MXFP8, as the dense part of a transformer block runs them;
* balance: the router's load-balance loss, per-expert counts and the gradient
  of the logits.

``run`` with ``own`` false computes them with elementary torch operations in
fp32, with ``own`` true through this package.  Weights are held as a model
holds them: MXFP8 payload and scales.  8-bit outputs are returned as tensors of
the 8-bit floating types whose values they hold.
"""

import math

import torch

own = False

EPS = 1e-6
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a 2048-wide model in decode: the latency of a norm
        dict(name="norm_token", op="norm", rows=1, hidden=2048, residual="bf16", weight="bf16",
             bf16_out=True, pad=0),
        # 16K tokens of the same model in prefill; the bf16 output feeds the router
        dict(name="norm_prefill", op="norm", rows=16384, hidden=2048, residual="bf16",
             weight="bf16", bf16_out=True, pad=0),
        # an odd batch of a 4304-wide layer (a last block of 16), residual stream and weight
        # in fp32, rows that are a slice of a wider tensor
        dict(name="norm_odd_fp32", op="norm", rows=777, hidden=4304, residual="fp32",
             weight="fp32", bf16_out=False, pad=48),
        # small ragged product: every edge of the tiles
        dict(name="linear_ragged", op="linear", rows=200, n=400, k=336, act="silu", bias=True,
             residual=True),
        # 32 tokens through a down projection in decode: bound by the weights' bytes
        dict(name="linear_decode", op="linear", rows=32, n=4096, k=12288, act="none", bias=False,
             residual=True),
        # 8K tokens through the same projection in prefill: bound by the tensor cores
        dict(name="linear_prefill", op="linear", rows=8192, n=4096, k=12288, act="none",
             bias=False, residual=True),
        # first layer of a vision MLP: short contraction, ragged width, wide output
        dict(name="linear_vision", op="linear", rows=16384, n=4304, k=1152, act="gelu_tanh",
             bias=True, residual=False),
        # one token through a whole dense block
        dict(name="block_token", op="block", rows=1, hidden=4096, inner=12288, act="silu",
             bias=False),
        # a vision MLP block over 16K patches
        dict(name="block_vision", op="block", rows=16384, hidden=1152, inner=4304,
             act="gelu_tanh", bias=True),
        # the router of a small layer, 64 tokens
        dict(name="balance_small", op="balance", rows=64, experts=8, k=2, masked=0.0,
             given_counts=False),
        # 16K tokens, 128 experts, top-8, with padding tokens
        dict(name="balance_prefill", op="balance", rows=16384, experts=128, k=8, masked=0.1,
             given_counts=False),
        # a packed training batch, 256 experts, counts summed over micro-batches
        dict(name="balance_batch", op="balance", rows=65536, experts=256, k=8, masked=0.02,
             given_counts=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("norm", "linear", "block", "balance"))
    if op == "norm":
        hidden = _log_int(rng, 64, 12288, 16)
        rows = _log_int(rng, 1, max(1, min(16384, 16384 * 2048 // hidden)))
        return dict(op=op, rows=rows, hidden=hidden, residual=rng.choice(("none", "bf16", "fp32")),
                    weight=rng.choice(("bf16", "fp32")), bf16_out=rng.random() < 0.5,
                    pad=rng.choice((0, 0, 16, 48)))
    if op == "linear":
        n, k = _log_int(rng, 64, 12288, 16), _log_int(rng, 64, 12288, 16)
        n = min(n, 4096 * 12288 // k // 16 * 16)
        rows = _log_int(rng, 1, 8192)
        return dict(op=op, rows=rows, n=n, k=k, act=rng.choice(ACTS), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    if op == "block":
        hidden, inner = _log_int(rng, 128, 4096, 16), _log_int(rng, 128, 12288, 16)
        rows = _log_int(rng, 1, max(1, min(16384, 16384 * 1152 * 4304 // (hidden * inner))))
        return dict(op=op, rows=rows, hidden=hidden, inner=inner, act=rng.choice(ACTS),
                    bias=rng.random() < 0.5)
    experts = _log_int(rng, 4, 512)
    rows = _log_int(rng, 1, min(65536, 65536 * 256 // experts))
    return dict(op=op, rows=rows, experts=experts, k=rng.randint(1, min(8, experts)),
                masked=rng.choice((0.0, 0.1, 0.5)), given_counts=rng.random() < 0.3)


def work(case):
    op, m = case["op"], case["rows"]
    mx = lambda rows, k: rows * (k + -(-k // 32))  # noqa: E731  payload and scales
    if op == "norm":
        h = case["hidden"]
        rsize = {"none": 0, "bf16": 2, "fp32": 4}[case["residual"]]
        wsize = {"bf16": 2, "fp32": 4}[case["weight"]]
        per_row = 2 * h + 2 * rsize * h + (2 * h if case["bf16_out"] else 0)
        return {"bytes": m * per_row + mx(m, h) + wsize * h, "flops": 6 * m * h}
    if op == "linear":
        n, k = case["n"], case["k"]
        return {"bytes": 2 * m * k + mx(n, k) + 2 * m * n * (2 if case["residual"] else 1)
                + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if op == "block":
        h, i = case["hidden"], case["inner"]
        return {"bytes": 6 * m * h + 2 * h + mx(i, h) + mx(h, i)
                + (2 * (h + i) if case["bias"] else 0), "flops": 4 * m * h * i + 6 * m * h}
    e, k = case["experts"], case["k"]
    return {"bytes": 8 * m * e + 4 * m * k + (m if case["masked"] else 0) + 8 * e + 4,
            "flops": 8 * m * e}


# ---------------------------------------------------------------- inputs

def _hidden(g, dev, rows, width):
    """Hidden states: N(0, 1), one channel in a hundred twenty times as large."""
    x = torch.randn(rows, width, generator=g, device=dev)
    x[:, torch.randperm(width, generator=g, device=dev)[:width // 100]] *= 20.0
    return x


def _weight(g, dev, n, k):
    """A projection's weight, N(0, 0.02) in bf16, held as MXFP8."""
    w = (torch.randn(n, k, generator=g, device=dev) * 0.02).bfloat16().float()
    return _mx_quantize(w)


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    op, m = case["op"], case["rows"]
    s = {"op": op, "case": dict(case)}
    if op == "norm":
        h = case["hidden"]
        x = _hidden(g, dev, m, h + case["pad"]).bfloat16()
        s["x"] = x[:, :h]
        s["residual"] = None
        if case["residual"] != "none":
            s["residual"] = (2 * randn(m, h)).to(
                torch.bfloat16 if case["residual"] == "bf16" else torch.float32)
        s["w"] = (1 + 0.1 * randn(h)).to(
            torch.bfloat16 if case["weight"] == "bf16" else torch.float32)
    elif op == "linear":
        n, k = case["n"], case["k"]
        s["x"] = _hidden(g, dev, m, k).bfloat16()
        s["wq"], s["ws"] = _weight(g, dev, n, k)
        s["bias"] = randn(n).bfloat16() if case["bias"] else None
        s["residual"] = (2 * randn(m, n)).bfloat16() if case["residual"] else None
    elif op == "block":
        h, i = case["hidden"], case["inner"]
        s["x"] = _hidden(g, dev, m, h).bfloat16()
        s["residual"] = (2 * randn(m, h)).bfloat16()
        s["w"] = (1 + 0.1 * randn(h)).bfloat16()
        s["w1q"], s["w1s"] = _weight(g, dev, i, h)
        s["w2q"], s["w2s"] = _weight(g, dev, h, i)
        s["b1"] = randn(i).bfloat16() if case["bias"] else None
        s["b2"] = randn(h).bfloat16() if case["bias"] else None
    else:
        e, k = case["experts"], case["k"]
        s["logits"] = randn(m, e) + 0.7 * randn(e)  # some experts are more popular
        s["ids"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
        s["mask"] = None
        if case["masked"]:
            s["mask"] = torch.rand(m, generator=g, device=dev) >= case["masked"]
        s["counts"] = None
        if case["given_counts"]:
            s["counts"] = torch.randint(0, 4 * m, (e,), generator=g, device=dev)
    if own:
        import mxfp8_block_scaled_moe_gb300 as mm
        s["mm"] = mm
        # load time, as a model does it: the weights' scales in the layout the products read
        if op == "linear":
            s["layer"] = mm.MXFP8FusedLinear(s["wq"], s["ws"], bias=s["bias"], act=case["act"])
        elif op == "block":
            s["fc1"] = mm.MXFP8FusedLinear(s["w1q"], s["w1s"], bias=s["b1"], act=case["act"])
            s["fc2"] = mm.MXFP8FusedLinear(s["w2q"], s["w2s"], bias=s["b2"])
    return s


# ---------------------------------------------------------------- plain form

def _mx_quantize(x):
    """fp32 [.., K] -> (e4m3 payload, uint8 e8m0 scales [.., ceil(K/32)])."""
    k = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -k % 32)).unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 9, -127).clamp(-127, 127)
    q = torch.ldexp(b, -exponent[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.flatten(-2)[..., :k].contiguous(), (exponent + 127).to(torch.uint8)


def _mx_values(q, s):
    """The fp32 values an MXFP8 tensor holds."""
    k = q.shape[-1]
    scale = (s.int() - 127).repeat_interleave(32, -1)[..., :k]
    return torch.ldexp(q.float(), scale)


def _act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _plain_norm(x, residual, w):
    """(the new residual, in its type, and the normed rows in bf16)"""
    h = x.float()
    stream = None
    if residual is not None:
        stream = (h + residual.float()).to(residual.dtype)
        h = stream.float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    return stream, (h * r * w.float()).bfloat16()


def _plain_linear(x, wq, ws, bias, act):
    """x: the fp32 values of an MXFP8 tensor; the fp32 result before the residual"""
    z = x @ _mx_values(wq, ws).t()
    return _act(act, z if bias is None else z + bias.float())


def _plain(s):
    op, case = s["op"], s["case"]
    if op == "norm":
        stream, y = _plain_norm(s["x"], s["residual"], s["w"])
        q, scale = _mx_quantize(y.float())
        return _norm_outputs(case, q, scale, y, stream)
    if op == "linear":
        v = _plain_linear(_mx_values(*_mx_quantize(s["x"].float())), s["wq"], s["ws"], s["bias"],
                          case["act"])
        return (v if s["residual"] is None else v + s["residual"].float()).bfloat16()
    if op == "block":
        stream, y = _plain_norm(s["x"], s["residual"], s["w"])
        v = _plain_linear(_mx_values(*_mx_quantize(y.float())), s["w1q"], s["w1s"], s["b1"],
                          case["act"])
        v = _plain_linear(_mx_values(*_mx_quantize(v)), s["w2q"], s["w2s"], s["b2"], "none")
        return (v + stream.float()).bfloat16()
    logits, e = s["logits"], case["experts"]
    live = torch.ones_like(logits[:, 0]) if s["mask"] is None else s["mask"].float()
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    chosen = (s["ids"][:, :, None] == torch.arange(e, device=logits.device)).sum(1)
    counts = (chosen * live.long()[:, None]).sum(0)
    used = (counts if s["counts"] is None else s["counts"]).double()
    f = (used / used.sum().clamp(min=1)).float()
    n = live.sum().clamp(min=1)
    loss = e * (f * ((p * live[:, None]).sum(0) / n)).sum()
    grad = e / n * live[:, None] * p * (f - (p * f).sum(1, keepdim=True))
    return {"loss": loss, "counts": counts, "dlogits": grad}


def _norm_outputs(case, q, scale, y, stream):
    out = {"q": q.view(torch.float8_e4m3fn), "s": scale.view(torch.float8_e8m0fnu)}
    if case["bf16_out"]:
        out["y"] = y
    if stream is not None:
        out["residual"] = stream
    return out


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    op, case, mm = s["op"], s["case"], s["mm"]
    if op == "norm":
        r = mm.mx_add_rmsnorm_quant(s["x"], s["w"], residual=s["residual"], eps=EPS,
                                    bf16_out=case["bf16_out"])
        return _norm_outputs(case, r["q"], r["s"], r.get("y"), r.get("residual"))
    if op == "linear":
        return s["layer"](s["x"], residual=s["residual"])
    if op == "block":
        r = mm.mx_add_rmsnorm_quant(s["x"], s["w"], residual=s["residual"], eps=EPS,
                                    mma_scales=True)
        inner = s["fc1"]((r["q"], r["s"]), mx_out=True)
        return s["fc2"](inner, residual=r["residual"])
    return mm.moe_balance_loss(s["logits"], s["ids"], mask=s["mask"], counts=s["counts"],
                               grad=True)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits

def _round_e4m3(v):
    """float64 -> the nearest e4m3 values (ties to even, saturating at 448)."""
    power = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    power = power - (torch.exp2(power) > v.abs().clamp(min=2.0 ** -6)).double()
    step = torch.exp2(power - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _mx_exact(v):
    """float64 [M, K] -> (payload values, scales as powers of two, what they stand for)"""
    m, k = v.shape
    blocks = -(-k // 32)
    wide = v.new_zeros(m, blocks * 32)
    wide[:, :k] = v
    wide = wide.view(m, blocks, 32)
    top = wide.abs().max(2).values
    safe = top.clamp(min=2.0 ** -150)
    power = torch.floor(torch.log2(safe))
    power = power + (torch.exp2(power + 1) <= safe).double() - (torch.exp2(power) > safe).double()
    scale = torch.exp2((power - 8).clamp(-127, 127))
    q = _round_e4m3(wide / scale[:, :, None])
    flat = lambda t: t.reshape(m, blocks * 32)[:, :k]  # noqa: E731
    return flat(q), scale, flat(q * scale[:, :, None])


def _held(q, s):
    """What a weight's payload and scales stand for, in float64."""
    scale = torch.exp2(s.double() - 127)
    return q.double() * scale.repeat_interleave(32, 1)[:, :q.shape[1]]


def _norm_exact(s):
    h = s["x"].double()
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(s["residual"].dtype).double()
    y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / h.shape[1] + EPS) * s["w"].double()
    return h, y


def _act_exact(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h, y = _norm_exact(s)
        q, scale, _ = _mx_exact(y.bfloat16().double())
        return _norm_exact_outputs(case, q, scale, y, h)
    if op == "linear":
        z = _mx_exact(s["x"].double())[2] @ _held(s["wq"], s["ws"]).t()
        if s["bias"] is not None:
            z = z + s["bias"].double()
        v = _act_exact(case["act"], z)
        return v if s["residual"] is None else v + s["residual"].double()
    if op == "block":
        h, y = _norm_exact(s)
        z = _mx_exact(y.bfloat16().double())[2] @ _held(s["w1q"], s["w1s"]).t()
        if s["b1"] is not None:
            z = z + s["b1"].double()
        z = _mx_exact(_act_exact(case["act"], z))[2] @ _held(s["w2q"], s["w2s"]).t()
        if s["b2"] is not None:
            z = z + s["b2"].double()
        return z + h
    e = case["experts"]
    p = torch.softmax(s["logits"].double(), 1)
    ids = s["ids"].long()
    if s["mask"] is not None:
        p = p * s["mask"].double()[:, None]
        ids = ids[s["mask"]]
    n = max(1, ids.shape[0])
    counts = torch.bincount(ids.reshape(-1), minlength=e)
    used = (counts if s["counts"] is None else s["counts"]).double()
    f = used / max(1.0, float(used.sum()))
    loss = e * float((f * p.sum(0)).sum()) / n
    grad = p * (f[None, :] - p @ f[:, None]) * (e / n)
    return {"loss": torch.tensor(loss, dtype=torch.float64), "counts": counts, "dlogits": grad}


def _norm_exact_outputs(case, q, scale, y, h):
    out = {"q": q, "s": scale}
    if case["bf16_out"]:
        out["y"] = y
    if case["residual"] != "none":
        out["residual"] = h
    return out
