"""One pre-norm linear layer trained in 8 bits with an orthogonalised update:

    h = layer_norm(x);  y = h . W (8-bit product);  loss = mean (y - target)^2 / 2
    dh, dW = the product's backward (8-bit);  dx, dgamma, dbeta = the norm's
    momentum = beta momentum + dW;  W -= lr * orthogonalize(momentum), tile by tile

W is held in fp32 and in 8 bits (a scale for each 128 x 128 block), as the step
that follows reads it; its momentum is orthogonalised in N column tiles, the tiles
that ``TiledLinear`` would stream for a W too large for the device.  Last, the
trained layer answers for single tokens, and the same W goes through the
host-streamed bf16 operator for comparison.

    python examples/prenorm_layer.py [--tokens T] [--width K] [--out M] [--tiles N] [--steps S]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def train(tl, T: int, K: int, M: int, N: int, steps: int, lr: float = 0.02, beta: float = 0.9, seed: int = 0) -> dict:
    """Train the layer on a fixed batch of a hidden layer's outputs; returns the
    losses and the trained parameters."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (randn(T, K) * torch.exp(0.3 * randn(K)) + 0.2).bfloat16()
    hidden = torch.nn.functional.layer_norm(x.float(), (K,)) @ (randn(K, M) / K ** 0.5)
    gamma, beta_n = torch.ones(K, device="cuda"), torch.zeros(K, device="cuda")
    master = randn(K, M) / K ** 0.5
    momentum = torch.zeros(N, K, M // N, device="cuda")
    # Muon's scale: an update whose elements do not depend on the tile's shape
    scale = max(1.0, K / (M // N)) ** 0.5
    losses = []
    for _ in range(steps):
        wq, ws = tl.fp8_quantize(master, "tile")
        h, mean, rstd = tl.layer_norm(x, gamma.bfloat16(), beta_n.bfloat16())
        y = tl.fp8_linear(h, wq, ws)
        diff = y.float() - hidden
        losses.append(diff.square().mean())
        dy = (diff / T).bfloat16()
        dh, dw = tl.fp8_linear_backward(h, dy, wq, ws)
        _, dgamma, dbeta = tl.layer_norm_backward(dh, x, mean, rstd, gamma.bfloat16())
        momentum.mul_(beta).add_(dw.view(K, N, M // N).permute(1, 0, 2))
        update = tl.orthogonalize(momentum, scale=scale)
        master.view(K, N, M // N).sub_(update.permute(1, 0, 2).float(), alpha=lr)
        gamma.sub_(dgamma, alpha=lr)
        beta_n.sub_(dbeta, alpha=lr)
    tl.check_operators()
    return {"losses": [float(v) for v in losses], "x": x, "gamma": gamma, "beta": beta_n, "master": master}


def answer(tl, layer: dict, tokens) -> "object":
    """The trained layer's y for each of a few tokens, one at a time, as a server would."""
    import torch
    wq, ws = tl.fp8_quantize(layer["master"], "tile")
    rows = []
    for t in tokens:
        h, _, _ = tl.layer_norm(layer["x"][t:t + 1], layer["gamma"].bfloat16(), layer["beta"].bfloat16())
        rows.append(tl.fp8_linear(h, wq, ws))
    tl.check_operators()
    return torch.cat(rows)


def streamed(tl, layer: dict, N: int):
    """The same layer with its W in bf16 tiles in host memory, through the ring."""
    import torch
    master = layer["master"]
    K, M = master.shape
    w, dw = tl.PinnedBuffer(K * M), tl.PinnedBuffer(K * M)
    w.tensor.view(N, K, M // N).copy_(master.view(K, N, M // N).permute(1, 0, 2).bfloat16().cpu())
    op = tl.TiledLinear(K, M, N, min(1, N - 1), w, dw)
    h, _, _ = tl.layer_norm(layer["x"], layer["gamma"].bfloat16(), layer["beta"].bfloat16())
    y = op.forward(h)
    torch.cuda.synchronize()
    op.close()
    w.close()
    dw.close()
    return y


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--out", type=int, default=4096)
    ap.add_argument("--tiles", type=int, default=4)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    import __graft_entry__
    __graft_entry__.build()
    from offload_streamed_gb300 import tiled_linear as tl
    layer = train(tl, a.tokens, a.width, a.out, a.tiles, a.steps)
    print("loss: %.4f -> %.4f in %d steps" % (layer["losses"][0], layer["losses"][-1], a.steps))
    few = answer(tl, layer, range(4))
    full = streamed(tl, layer, a.tiles)[:4]
    print("8-bit single tokens against the streamed bf16 layer: %.4f of its norm apart"
          % float((few.float() - full.float()).norm() / full.float().norm()))


if __name__ == "__main__":
    main()
