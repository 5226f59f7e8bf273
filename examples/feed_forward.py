"""A feed-forward block built from the library's operators, dense and with experts: a few training
steps and one decoding step on synthetic data.

  x' = x + gate * N(y) w_post, h = N(x') w_pre          block_norm: both norms in one pass
  a  = h W13^T                                          linear: gate and up projections
  z  = silu(a_gate) * a_up                              glu
  y' = z W2^T + b                                       linear: down projection
and with experts, between the norm and the next block,
  rows, offsets = sort of the router's choices          moe_sort
  z = glu(permute(h) W13[e]^T),  y' = combine(z W2[e]^T, weights)
With `save` the projections and the GLU between them are one op, feed_forward, which keeps gate and up for
the backward as BF16 with four more bits ("bf16") or as 8-bit codes ("mxfp8") and forms z again.

`torch.ops.glu_mx` carries the gradients.  Run on a GPU: python examples/feed_forward.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import glu_activation_microscaling_amd.torch_ops  # noqa: E402,F401  (registers torch.ops.glu_mx)

ops = torch.ops.glu_mx


def make_params(width, inner, experts=0, seed=0, device="cuda"):
    """Parameters of one block, BF16: norms, router (with experts), and the two projections."""
    g = torch.Generator(device=device).manual_seed(seed)

    def n(*shape, scale):
        t = torch.randn(shape, generator=g, device=device) * scale
        return t.to(torch.bfloat16).requires_grad_(True)

    lead = (experts,) if experts else ()
    ones = torch.ones(width, device=device, dtype=torch.bfloat16)
    p = dict(gate=(0.5 * ones).requires_grad_(True), w_post=ones.clone().requires_grad_(True),
             w_pre=ones.clone().requires_grad_(True), w13=n(*lead, 2 * inner, width, scale=width ** -0.5),
             w2=n(*lead, width, inner, scale=inner ** -0.5), b2=n(*lead, width, scale=0.02))
    if experts:
        p["router"] = n(experts, width, scale=width ** -0.5)
    return p


def feed_forward(x, y, p, choices=0, save=None):
    """One block on the residual stream x [M, width] and the previous block's output y: the new
    stream x' and this block's output.  choices > 0 takes that many experts a token; save says what
    the projections keep for the backward (None: the projections and the GLU one by one)."""
    x_out, h, _ = ops.block_norm(x, y, p["gate"], p["w_pre"], None, p["w_post"], True)
    inner = p["w13"].shape[-2] // 2
    if not choices:
        if save is not None:
            return x_out, ops.feed_forward(h, p["w13"], p["w2"], None, p["b2"], None, "swiglu", "split", save)[0]
        a, _ = ops.linear(h, p["w13"])
        z = ops.glu(a[:, :inner], a[:, inner:], "swiglu", "split")
        out, _ = ops.linear(z, p["w2"], p["b2"])
        return x_out, out
    logits = (h @ p["router"].t()).float()
    top, ids = torch.topk(logits, choices, dim=1)
    weights = torch.softmax(top, dim=1)
    rows, offsets = ops.moe_sort(ids, p["router"].shape[0])
    xs = ops.moe_permute(h, rows, offsets)
    if save is not None:
        ys, _, _ = ops.feed_forward(xs, p["w13"], p["w2"], None, p["b2"], offsets, "swiglu", "split", save)
        return x_out, ops.moe_combine(ys, rows, offsets, weights)
    a, _ = ops.linear(xs, p["w13"], None, None, offsets)
    z = ops.glu(a[:, :inner], a[:, inner:], "swiglu", "split")
    ys, _ = ops.linear(z, p["w2"], p["b2"], None, offsets)
    return x_out, ops.moe_combine(ys, rows, offsets, weights)


def train(tokens=512, width=256, inner=512, experts=0, choices=0, steps=8, lr=0.2, seed=0, save=None):
    """Fits the block's output to a fixed target by plain gradient descent; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, y, target = (torch.randn((tokens, width), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    p = make_params(width, inner, experts, seed)
    losses = []
    for _ in range(steps):
        x_out, out = feed_forward(x, y, p, choices, save)
        loss = (x_out.float() + out.float() - target.float()).square().mean()
        grads = torch.autograd.grad(loss * tokens, list(p.values()))
        with torch.no_grad():
            for t, d in zip(p.values(), grads):
                t -= lr * d / tokens ** 0.5
        losses.append(float(loss.detach()))
    return losses


def main():
    experts = dict(experts=8, choices=2)
    for name, kw in (("dense", {}), ("8 experts, 2 a token", experts), ("dense, 8-bit checkpoints", dict(save="mxfp8")),
                     ("8 experts, 8-bit checkpoints", dict(experts, save="mxfp8"))):
        losses = train(**kw)
        print(f"{name}: loss " + " ".join(f"{v:.4f}" for v in losses))
        with torch.no_grad():   # one new token
            p = make_params(256, 512, kw.get("experts", 0))
            one = torch.randn(1, 256, device="cuda").to(torch.bfloat16)
            x_out, out = feed_forward(one, one, p, kw.get("choices", 0), kw.get("save") and "none")
            print(f"{name}: one token -> {tuple(out.shape)}, mean square {float(out.float().square().mean()):.4f}")


if __name__ == "__main__":
    main()
