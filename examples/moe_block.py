"""One MoE block of a transformer on MXFP8 weights, and its router's training.

The block is what stands between two attentions: the residual's addition and RMS
norm, the routed experts, and a dense expert that every token passes through.
Its launches hand each other MXFP8 directly; bf16 exists only where it is read
as such (the router's input, the residual stream, the block's result).

    (q, s), y, residual = norm(x + residual)     MXFP8 for the dense expert, bf16 for the router
    routed              = experts(y, y . gate^T)
    next x              = down(silu(up(q, s))) + routed      the sum in the epilogue

Expert and dense weights are frozen MXFP8; the bf16 gate is what a fine-tuning
run trains.  `balance_step` lowers its load-balance loss by one step of gradient
descent, with the logits' gradient from the same launches as the loss.

    python examples/moe_block.py [--tokens 4096] [--steps 30]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import mxfp8_block_scaled_moe_gb300 as mm  # noqa: E402


class MoEBlock:
    """norm bf16 or fp32 [H], gate bf16 [E, H], w13 bf16 [E, 2I, H], w2 bf16 [E, H, I],
    up bf16 [S, H] and down bf16 [H, S] of the dense expert; k experts per token."""

    def __init__(self, norm, gate, w13, w2, up, down, k, eps=1e-6):
        self.norm, self.eps, self.k = norm, eps, k
        self.gate = gate.float()           # the trained copy; the router reads bf16
        self.experts = mm.MXFP8MoELayer.from_bf16(w13, w2, k)
        self.up = mm.MXFP8FusedLinear.from_bf16(up, act="silu")
        self.down = mm.MXFP8FusedLinear.from_bf16(down)

    def normed(self, x, residual):
        return mm.mx_add_rmsnorm_quant(x, self.norm, residual=residual, eps=self.eps,
                                       bf16_out=True, mma_scales=True)

    def route(self, y):
        return mm.moe_router_gate_topk(y, self.gate.bfloat16(), self.k, logits=True)

    def forward(self, x, residual):
        """x, residual bf16 [T, H] -> (the next block's x, the residual stream)."""
        n = self.normed(x, residual)
        routed = self.experts(n["y"], self.route(n["y"])["logits"])
        return self.down(self.up((n["q"], n["s"]), mx_out=True), residual=routed), n["residual"]

    __call__ = forward

    def balance_step(self, x, residual, mask=None, coef=1.0, rate=0.5):
        """One step of gradient descent on the load-balance loss of these tokens
        (mask: True where a token counts).  rate counts in logits: normed rows have a
        square of about H, so that a gate's step moves its logits by H times as much.
        Returns the loss and the counts before the step."""
        y = self.normed(x, residual)["y"]
        r = self.route(y)
        b = mm.moe_balance_loss(r["logits"], r["topk_ids"], mask=mask, coef=coef, grad=True)
        self.gate -= rate / y.shape[1] * (b["dlogits"].t() @ y.float())
        return b["loss"], b["counts"]


def random_block(E=128, H=2048, I=768, S=1536, k=8, device="cuda", seed=0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def w(*shape):
        return (torch.randn(*shape, generator=g, device=device) * 0.02).bfloat16()

    return MoEBlock(torch.ones(H, device=device), w(E, H) + w(E, 1), w(E, 2 * I, H), w(E, H, I),
                    w(S, H), w(H, S), k)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    torch.manual_seed(1)
    block = random_block()
    H = block.norm.numel()
    # hidden states with a common direction: some experts are chosen far too often
    x = (torch.randn(a.tokens, H, device="cuda") + torch.randn(H, device="cuda")).bfloat16()
    residual = torch.randn(a.tokens, H, device="cuda").bfloat16()
    mask = torch.arange(a.tokens, device="cuda") % 16 != 15  # every 16th token is padding
    for i in range(a.steps):
        loss, counts = block.balance_step(x, residual, mask)
        if i % 5 == 0 or i == a.steps - 1:
            c = counts.double()
            print(f"step {i:3d}  loss {loss.item():.4f}  busiest expert "
                  f"{(c.max() / c.mean()).item():.2f} x the mean")
    for T in (1, 32, a.tokens):
        xs, rs = x[:T].contiguous(), residual[:T].contiguous()
        graph = torch.cuda.CUDAGraph()
        block(xs, rs)  # workspaces and kernels are there before the capture
        with torch.cuda.graph(graph):
            out, _ = block(xs, rs)
        for _ in range(3):
            graph.replay()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"{T:6d} tokens  {start.elapsed_time(end) * 50:9.1f} us a block, "
              f"result {'finite' if out.isfinite().all().item() else 'NOT FINITE'}")
    if mm.device_status() != 0:
        raise RuntimeError("a kernel reported an error")


if __name__ == "__main__":
    main()
