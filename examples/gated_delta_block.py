"""A small gated-delta language block on the library's operators: prefill of a right-padded batch, decoding from
a pool of states, and one training step's gradients.

    python examples/gated_delta_block.py

Per layer: block norm (the norm before), projections, gated delta rule, gated RMS norm of its output, output projection;
the next layer's block norm adds the projection to the residual. Projections are plain matrix products.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mamba_ssd_selective_gb300 import binding as ops  # noqa: E402

DIM, HEADS, GROUPS, P, N, LAYERS = 768, 24, 12, 64, 128, 2
SIZES = (GROUPS * N, GROUPS * N, HEADS * P, HEADS, HEADS, HEADS * P)  # q, k, v, decay, beta, gate


def make_layer(gen):
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda") * s[0] ** -0.5  # noqa: E731
    ones = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    return dict(w_in=rand(DIM, sum(SIZES)).bfloat16(), w_out=rand(HEADS * P, DIM).bfloat16(), A=1 + 15 * torch.rand(
        HEADS, generator=gen, device="cuda"), dt_bias=torch.full((HEADS,), -4.0, device="cuda"),
        unit=torch.full((GROUPS * N,), N ** -0.5, device="cuda"), norm=ones(HEADS * P), pre=ones(DIM), post=ones(DIM),
        scale=torch.full((DIM,), 0.5, device="cuda"))


def project(layer, x):
    """x[rows, DIM] -> q, k (norm 1 per group), v, g, beta and the gate, each [rows, ...]."""
    q, k, v, a, b, z = (s.contiguous() for s in (x @ layer["w_in"]).split(SIZES, -1))
    q, k = (ops.gated_rmsnorm(s, None, layer["unit"], group=N, eps=1e-6 / N).view(-1, GROUPS, N) for s in (q, k))
    g = (-layer["A"] * torch.nn.functional.softplus(a.float() + layer["dt_bias"])).to(x.dtype)
    return q, k, v.view(-1, HEADS, P), g, torch.sigmoid(b), z


def run(layers, x, delta):
    """x[rows, DIM] through the layers; delta(i, q, k, v, g, beta) is layer i's rule over [rows, ...]."""
    res = torch.zeros_like(x, dtype=torch.float32)
    y, post, scale = x, None, None
    for i, layer in enumerate(layers):
        h, res = ops.block_norm(y, res, layer["pre"], post_weight=post, scale=scale)
        q, k, v, g, beta, z = project(layer, h)
        o = delta(i, q, k, v, g, beta)
        y = ops.gated_rmsnorm(o.reshape(-1, HEADS * P), z, layer["norm"], group=P) @ layer["w_out"]
        post, scale = layer["post"], layer["scale"]
    return ops.block_norm(y, res, layers[0]["pre"], post_weight=post, scale=scale)[0]


def prefill(layers, x, lens, pools, slots):
    """x[B, L, DIM] right-padded to lens; leaves the layers' states in their pools at `slots`."""
    B, L, _ = x.shape

    def delta(i, q, k, v, g, beta):
        t = [s.reshape(B, L, *s.shape[1:]) for s in (q, k, v, g, beta)]
        y, state = ops.gated_delta_chunked(*t, seqlens=lens)
        pools[i][slots.long()] = state
        return y

    return run(layers, x.reshape(B * L, DIM), delta).reshape(B, L, DIM)


def decode(layers, x, pools, slots):
    """One token x[B, DIM] of each row; rows with slot -1 are idle."""
    return run(layers, x, lambda i, *t: ops.gated_delta_step(pools[i], *t, slots=slots))


def train_gradients(layer, x):
    """Gradients of sum(out^2) / 2 of one layer's core (rule, then block norm) with respect to its tokens and residual."""
    B, L, _ = x.shape
    h, res = ops.block_norm(x.reshape(B * L, DIM), torch.zeros(B * L, DIM, device="cuda"), layer["pre"])
    t = [s.reshape(B, L, *s.shape[1:]) for s in project(layer, h)[:5]]
    y, _ = ops.gated_delta_chunked(*t)
    o = y.reshape(B * L, -1) @ layer["w_out"]
    norm = dict(post_weight=layer["post"], scale=layer["scale"])
    out, _ = ops.block_norm(o, res, layer["pre"], **norm)
    gn = ops.block_norm_bwd(o, res, out, layer["pre"], **norm)
    dy = (gn["dy"] @ layer["w_out"].T).reshape(y.shape)
    return {**gn, **ops.gated_delta_chunked_bwd(*t, dy, want_dinit=False)}


def main():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    layers = [make_layer(gen) for _ in range(LAYERS)]
    B, L, new = 3, 150, 4
    lens = torch.tensor([150, 1, 97], dtype=torch.int32, device="cuda")
    x = torch.randn(B, L + new, DIM, generator=gen, device="cuda").bfloat16()
    pools = [torch.zeros(5, HEADS, P, N, device="cuda") for _ in layers]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    prefill(layers, x[:, :L].contiguous(), lens, pools, slots)
    # the tokens after each prompt, one at a time, against one pass over the longer sequence of row 0
    ys = [decode(layers, x[:, L + i].contiguous(), pools, slots) for i in range(new)]
    whole = prefill(layers, x[:1].contiguous(), None, [torch.zeros_like(p) for p in pools], slots[:1])
    err = float((torch.stack([y[0] for y in ys]) - whole[0, L:]).float().norm() / whole[0, L:].float().norm())
    grads = train_gradients(layers[0], x)
    torch.cuda.synchronize()
    print(f"decode against one pass: {err:.1e}; gradients: "
          + ", ".join(f"|{n}| {float(g.float().norm()):.3g}" for n, g in grads.items() if g is not None))
    return err


if __name__ == "__main__":
    sys.exit(0 if main() < 2e-2 else 1)
