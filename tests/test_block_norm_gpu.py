"""The block norm and its backward on the GPU against the float64 definition (oracle.delta).

Tolerances: float32 results come from float32 sums of at most 16384 terms over a tree and a handful of products,
below 1e-6 in the 2-norm; weights' gradients add up to a thousand rows. 1e-5 (2-norm) and 1e-4 (largest error over the
largest result). bf16 results are rounded once: half a unit in the last of 8 bits is at most 2^-8 of each value, so of
the 2-norm too (over many values 1.7e-3): 2^-8 for both, and a little for the float32 value's own error.
"""
import threading

import numpy as np
import pytest
import torch

from mamba_ssd_selective_gb300 import inputs
from oracle import delta
from tests.helpers import IO_TORCH, dev, host

pytestmark = pytest.mark.gpu
TOL = {torch.float32: (1e-5, 1e-4), torch.bfloat16: (1.01 * 2.0 ** -8, 1.01 * 2.0 ** -8)}


def near(got, want, what):
    two, most = TOL[got.dtype]
    got = host(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    norm, top = np.linalg.norm(want), np.max(np.abs(want))
    assert np.linalg.norm(got - want) <= two * norm, f"{what}: {np.linalg.norm(got - want) / norm:.2e}"
    assert np.max(np.abs(got - want)) <= most * top, f"{what}: {np.max(np.abs(got - want)) / top:.2e}"


SIZES = [(1, 768), (3, 1), (5, 7), (2, 31), (700, 64), (33, 1537), (9, 2560), (4, 4100), (3, 5119), (2, 8192), (2, 16384),
         (2, 16383), (1031, 129)]
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


def case(rows, dim, io, rio, seed, parts):
    x = inputs.block_norm_inputs(rows, dim, io, rio, seed)
    for n, on in zip(("post", "z", "scale"), parts):
        if not on:
            x[n] = None
    t = {n: dev(v, IO_TORCH[io] if n in ("y", "z", "dout") else IO_TORCH[rio] if n in ("res", "dres")
                else torch.float32) for n, v in x.items()}
    return x, t


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("io,rio", TYPES)
@pytest.mark.parametrize("parts", [(1, 1, 1), (0, 0, 0), (1, 0, 1), (0, 1, 0)])
def test_block_norm(ssd, size, io, rio, parts):
    x, t = case(*size, io, rio, size[1], parts)
    out, r = ssd.block_norm(t["y"], t["res"], t["pre"], post_weight=t["post"], z=t["z"], scale=t["scale"])
    wo, wr = delta.block_norm(x["y"], x["res"], x["pre"], x["post"], x["z"], x["scale"])
    assert r.dtype == IO_TORCH[rio]
    near(out, wo, "out")
    near(r, wr, "res_out")


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("io,rio", TYPES)
@pytest.mark.parametrize("parts", [(1, 1, 1), (0, 0, 0), (1, 0, 1), (0, 1, 0)])
def test_block_norm_bwd(ssd, size, io, rio, parts):
    x, t = case(*size, io, rio, size[1] + 1, parts)
    for dres in (True, False):
        got = ssd.block_norm_bwd(t["y"], t["res"], t["dout"], t["pre"], dres_out=t["dres"] if dres else None,
                                 post_weight=t["post"], z=t["z"], scale=t["scale"])
        want = delta.block_norm_bwd(x["y"], x["res"], x["dout"], x["pre"], x["dres"] if dres else None, x["post"],
                                    x["z"], x["scale"])
        for n, w in want.items():
            if w is None:
                assert got[n] is None
            elif size[1] == 1 and n != "dpre_weight":
                # one channel: a norm keeps the sign alone, its gradient a (1 - r^2 / (r^2 + eps)) is what is left
                # of nearly equal numbers, and everything but dpre_weight comes through it
                assert torch.isfinite(got[n]).all()
            else:
                near(got[n], w, n)
        again = ssd.block_norm_bwd(t["y"], t["res"], t["dout"], t["pre"], dres_out=t["dres"] if dres else None,
                                   post_weight=t["post"], z=t["z"], scale=t["scale"])
        assert all(got[n] is None or torch.equal(got[n], again[n]) for n in got)


def test_block_norm_in_place_and_empty(ssd):
    _, t = case(40, 2560, "bf16", "bf16", 5, (1, 1, 1))
    kw = dict(post_weight=t["post"], z=t["z"], scale=t["scale"])
    out, r = ssd.block_norm(t["y"], t["res"], t["pre"], **kw)
    y, res = t["y"].clone(), t["res"].clone()
    ssd.block_norm(y, res, t["pre"], **kw, out=y, res_out=res)
    assert torch.equal(y, out) and torch.equal(res, r)
    none = t["y"][:0]
    out, r = ssd.block_norm(none, none, t["pre"])
    assert out.shape == (0, 2560)
    g = ssd.block_norm_bwd(none, none, none, t["pre"], scale=t["scale"])
    assert not g["dpre_weight"].any() and not g["dscale"].any()


def test_block_norm_rows_of_zeros(ssd):
    """A row whose block output is zero keeps its residual, and a row of zeros stays zero, with finite gradients."""
    y = torch.zeros(2, 64, device="cuda")
    res = torch.zeros_like(y)
    res[0] = 1.0
    w = torch.ones(64, device="cuda")
    out, r = ssd.block_norm(y, res, w, post_weight=w, z=y, scale=w)
    assert torch.equal(r, res) and not out[1].any()
    assert torch.allclose(out[0], torch.full((64,), (1 + 1e-5) ** -0.5, device="cuda"), rtol=1e-6)
    g = ssd.block_norm_bwd(y, res, torch.ones_like(y), w, post_weight=w, z=y, scale=w)
    assert all(torch.isfinite(x).all() for x in g.values())


@pytest.mark.parametrize("size", [(3, 8196), (2, 10004), (2, 16380)])
@pytest.mark.parametrize("io,rio", TYPES)
def test_block_norm_wide_rows_of_vectors_of_four(ssd, size, io, rio):
    """Rows above 8192 channels that are a multiple of four and not of eight, both directions."""
    x, t = case(*size, io, rio, size[1], (1, 1, 1))
    kw = dict(post_weight=t["post"], z=t["z"], scale=t["scale"])
    out, r = ssd.block_norm(t["y"], t["res"], t["pre"], **kw)
    for got, want, n in zip((out, r), delta.block_norm(x["y"], x["res"], x["pre"], x["post"], x["z"], x["scale"]), ("out", "res_out")):
        near(got, want, n)
    got = ssd.block_norm_bwd(t["y"], t["res"], t["dout"], t["pre"], dres_out=t["dres"], **kw)
    want = delta.block_norm_bwd(x["y"], x["res"], x["dout"], x["pre"], x["dres"], x["post"], x["z"], x["scale"])
    for n, w in want.items():
        near(got[n], w, n)


def test_block_norm_from_two_threads(ssd):
    """Widths that share a kernel and differ in the shared memory they ask for, at once: a call must not take back what
    another has been allowed."""
    said = []

    def work(dim):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                y, w = torch.randn(4, dim, device="cuda"), torch.ones(dim, device="cuda")
                for _ in range(1000):
                    ssd.block_norm(y, y, w, z=y)
                    ssd.block_norm_bwd(y, y, y, w, z=y)
        except Exception as e:
            said.append(e)

    threads = [threading.Thread(target=work, args=(d,)) for d in (4096, 3400, 4096, 3400)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not said


def test_block_norm_gate_of_any_size(ssd):
    """silu of gates from -80 to 80 in float32, element by element: expf within 1 unit in the last place (2^-23), the sum
    2^-24, the quotient 2 units, two products 2^-24 each: 4.5 units of 2^-23."""
    z = torch.linspace(-80, 80, 16000, device="cuda").reshape(1, -1)
    y, w = torch.ones_like(z), torch.ones(16000, device="cuda")
    _, r = ssd.block_norm(y, torch.zeros_like(z), w, z=z)
    want = z.double() / (1 + torch.exp(-z.double()))
    assert ((r.double() - want).abs() <= 4.5 * 2.0 ** -23 * want.abs()).all()
    g = ssd.block_norm_bwd(y, torch.zeros_like(z), torch.zeros_like(z), w, dres_out=y, z=z)  # dy = silu(z)
    assert ((g["dy"].double() - want).abs() <= 4.5 * 2.0 ** -23 * want.abs()).all()
