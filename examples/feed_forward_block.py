"""A transformer's feed-forward sub-layer on the library's operators.

    y = x + W_down^T (silu(W_gate^T n) * (W_up^T n)),  n = layer_norm(x)

followed by a linear head.  `python examples/feed_forward_block.py` trains the
pair on synthetic data with plain SGD (forward, backward and update all on the
operators' results), then feeds it one token at a time and compares with the
batch.  Needs a GB300 and the built library.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_f32_gb300 as dg  # noqa: E402


class FeedForward:
    """Parameters in `dtype`, with float32 copies that the updates accumulate in."""

    def __init__(self, width, hidden, outputs, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            return torch.randn((rows, cols), generator=gen, device="cuda") * rows ** -0.5

        self.master = {
            "norm_w": torch.ones(width, device="cuda"), "norm_b": torch.zeros(width, device="cuda"),
            "w_gate": weight(width, hidden), "w_up": weight(width, hidden),
            "w_down": weight(hidden, width), "head_w": weight(width, outputs),
            "head_b": torch.zeros(outputs, device="cuda"),
        }
        self.dtype = dtype
        self.p = {k: v.to(dtype) for k, v in self.master.items()}

    def forward(self, x, keep=False):
        p = self.p
        n, mean, rstd = dg.layer_norm(x, p["norm_w"], p["norm_b"], return_stats=True)
        block = dg.gated_ffn(n, p["w_gate"], p["w_up"], p["w_down"], residual=x, return_saved=keep)
        y, g, u = block if keep else (block, None, None)
        out = dg.linear(y, p["head_w"], bias=p["head_b"])
        return (out, (x, n, mean, rstd, g, u, y)) if keep else out

    def backward(self, dout, saved):
        """Gradients of every parameter, and of x."""
        p, (x, n, mean, rstd, g, u, y) = self.p, saved
        grads = {}
        dy, grads["head_w"], grads["head_b"] = dg.linear_backward(dout, y, p["head_w"])
        dn, grads["w_gate"], grads["w_up"], grads["w_down"] = dg.gated_ffn_backward(
            dy, n, p["w_gate"], p["w_up"], p["w_down"], g, u)
        # the skip connection's gradient is dy itself
        dx, grads["norm_w"], grads["norm_b"] = dg.layer_norm_backward(
            dn, x, p["norm_w"], mean, rstd, dresidual=dy)
        return grads, dx

    def step(self, x, target, lr):
        """One SGD step on mean((out - target)^2); returns the loss before it."""
        out, saved = self.forward(x, keep=True)
        diff = out.float() - target
        # loss scale 1: the gradient of the sum, scaled down in the update
        grads, _ = self.backward(diff.to(self.dtype), saved)
        for k, g in grads.items():
            self.master[k].add_(g.float(), alpha=-lr * 2.0 / diff.numel() * diff.shape[-1])
            self.p[k] = self.master[k].to(self.dtype)
        return diff.square().mean()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1408)
    ap.add_argument("--outputs", type=int, default=128)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--lr", type=float, default=0.1)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.tokens, a.width), generator=gen, device="cuda").to(torch.bfloat16)
    teacher = FeedForward(a.width, a.hidden, a.outputs, seed=2)
    target = teacher.forward(x).float()
    model = FeedForward(a.width, a.hidden, a.outputs, seed=3)
    losses = [model.step(x, target, a.lr).item() for _ in range(a.steps)]
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps of {a.tokens} tokens")
    batch = model.forward(x[:8])
    single = torch.stack([model.forward(x[i]) for i in range(8)])
    off = ((batch.float() - single.float()).norm() / batch.float().norm()).item()
    print(f"one token at a time against the batch: relative difference {off:.2e}")
    if not (losses[-1] < 0.5 * losses[0] and off < 1e-2):
        raise SystemExit("the block did not train, or its single-token form differs")


if __name__ == "__main__":
    main()
