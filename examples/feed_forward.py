"""Train a gated feed-forward block in FP8, then serve it token by token.

    python -m examples.feed_forward [--steps N]

Training fits a fixed batch: ``GatedFFN`` runs both of its products, forward and
backward, on E4M3 blocks; the down projection is an ordinary layer; before each
optimizer step ``clip_grad_norm`` bounds the gradients' common norm.

Serving packs the trained weights once -- gate and up as E4M3 blocks
(``weight_quant``), down to four bits (``fp4_weight_quant``) -- and then needs
two calls a token: ``gated_ffn`` and ``fp4_gemv``.
"""

import argparse

import torch

import fp8_block_scaled_quant_amd as fb


class FeedForward(torch.nn.Module):
    """``y = (silu(x W_gate^T) * (x W_up^T)) W_down^T``"""

    def __init__(self, features: int, hidden: int, scale_fmt=None, device=None):
        super().__init__()
        self.gated = fb.GatedFFN(features, hidden, torch.bfloat16, scale_fmt, device)
        self.down = torch.nn.Linear(hidden, features, bias=False, dtype=torch.bfloat16, device=device)

    def forward(self, x):
        return self.down(self.gated(x))


class Decoder:
    """The trained block with packed weights, for the few rows of a decode step."""

    def __init__(self, model: FeedForward):
        self.scale_fmt = model.gated.scale_fmt
        self.gate = fb.weight_quant(model.gated.w_gate.detach())
        self.up = fb.weight_quant(model.gated.w_up.detach())
        self.down = fb.fp4_weight_quant(model.down.weight.detach())

    def __call__(self, x):
        h = fb.gated_ffn(x, *self.gate, *self.up, self.scale_fmt, x.dtype)
        return fb.fp4_gemv(h, *self.down, x.dtype)


def train(model: FeedForward, x, target, steps: int, max_norm: float = 0.05, lr: float = 1e-3):
    """The loss before each step, and the gradients' norms."""
    optimizer = torch.optim.AdamW(model.parameters(), lr=lr)
    losses, norms = [], []
    for _ in range(steps):
        optimizer.zero_grad(set_to_none=True)
        loss = torch.nn.functional.mse_loss(model(x).float(), target)
        loss.backward()
        norms.append(fb.clip_grad_norm([p.grad for p in model.parameters()], max_norm))
        optimizer.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), torch.stack(norms).tolist()


def run(features=1024, hidden=2048, tokens=512, steps=30, device="cuda:0"):
    """Train, then decode the first tokens one at a time: the losses, the norms,
    and both ways' outputs of these tokens."""
    torch.manual_seed(0)
    model = FeedForward(features, hidden, "ue8m0", device)
    x = torch.randn(tokens, features, device=device).bfloat16()
    target = torch.randn(tokens, features, device=device)
    losses, norms = train(model, x, target, steps)
    decode = Decoder(model)
    one_by_one = torch.cat([decode(x[i:i + 1]) for i in range(4)])
    with torch.no_grad():
        together = model(x)[:4]
    return losses, norms, one_by_one, together


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=30)
    losses, norms, one_by_one, together = run(steps=parser.parse_args().steps)
    for i in range(0, len(losses), 5):
        print(f"step {i}: loss {losses[i]:.4f}, gradient norm {norms[i]:.4f}")
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    off = (one_by_one.float() - together.float()).norm() / together.float().norm()
    print(f"decode with the 4-bit down projection differs by {100 * off:.1f}% (2-norm)")


if __name__ == "__main__":
    main()
