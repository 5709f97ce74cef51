"""A transformer's feed-forward sub-layer on the library's operators.

    y = x + W_down^T (silu(W_gate^T n) * (W_up^T n)),  n = layer_norm(x)

followed by a linear head.  `python examples/feed_forward_block.py` trains the
pair on synthetic data with plain SGD (forward, backward and update all on the
operators' results), then feeds it one token at a time and compares with the
batch.  `--update orthogonal` steps the block's weights with the orthogonalised
momentum instead, `--int8` serves the trained pair with its weights in 8-bit
integers too.  Needs a GB300 and the built library.
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
        self.momentum = {k: torch.zeros_like(self.master[k]) for k in ("w_gate", "w_up", "w_down")}
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

    def quantised(self):
        """The products' weights in 8-bit integers, each output's with a scale of its own."""
        return {k: dg.quantize_int8(self.p[k], transpose=True) for k in ("w_gate", "w_up", "w_down", "head_w")}

    def forward_int8(self, x, q):
        p = self.p
        n = dg.layer_norm(x, p["norm_w"], p["norm_b"])
        y = dg.gated_ffn_int8(n, *q["w_gate"], *q["w_up"], *q["w_down"], residual=x)
        return dg.linear_int8(y, *q["head_w"], bias=p["head_b"])

    def step(self, x, target, lr, orthogonal_lr=None):
        """One step on mean((out - target)^2); returns the loss before it.  SGD, but for the block's
        matrices where orthogonal_lr is given: their momentum, orthogonalised."""
        out, saved = self.forward(x, keep=True)
        diff = out.float() - target
        # loss scale 1: the gradient of the sum, scaled down in the update
        grads, _ = self.backward(diff.to(self.dtype), saved)
        for k, g in grads.items():
            if orthogonal_lr is not None and k in self.momentum:
                w, m = self.master[k], self.momentum[k].mul_(0.9).add_(g)
                # every singular value of the update is about 1: sized for the matrix's shape
                size = max(1.0, w.shape[1] / w.shape[0]) ** 0.5
                dg.orthogonalize(m, scale=-orthogonal_lr * size, residual=w, out=w)
                self.p[k] = w.to(self.dtype)
                continue
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
    ap.add_argument("--update", choices=("sgd", "orthogonal"), default="sgd")
    ap.add_argument("--orthogonal-lr", type=float, default=0.02)
    ap.add_argument("--int8", action="store_true")
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.tokens, a.width), generator=gen, device="cuda").to(torch.bfloat16)
    teacher = FeedForward(a.width, a.hidden, a.outputs, seed=2)
    target = teacher.forward(x).float()
    model = FeedForward(a.width, a.hidden, a.outputs, seed=3)
    orthogonal_lr = a.orthogonal_lr if a.update == "orthogonal" else None
    losses = [model.step(x, target, a.lr, orthogonal_lr).item() for _ in range(a.steps)]
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps of {a.tokens} tokens")
    batch = model.forward(x[:8])
    single = torch.stack([model.forward(x[i]) for i in range(8)])
    off = ((batch.float() - single.float()).norm() / batch.float().norm()).item()
    print(f"one token at a time against the batch: relative difference {off:.2e}")
    if a.int8:
        q = model.quantised()
        served = torch.stack([model.forward_int8(x[i], q) for i in range(8)])
        lost = ((batch.float() - served.float()).norm() / batch.float().norm()).item()
        bits = sum(v.numel() for v, _ in q.values())
        print(f"in 8-bit integers ({bits} bytes of weights): relative difference {lost:.2e}")
        if not lost < 0.1:
            raise SystemExit("the 8-bit form differs")
    if not (losses[-1] < 0.5 * losses[0] and off < 1e-2):
        raise SystemExit("the block did not train, or its single-token form differs")


if __name__ == "__main__":
    main()
