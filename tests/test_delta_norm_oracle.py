"""The float64 definitions of the gated delta rule and the block norm: their
gradients against central differences, and the rule against its closed cases.

A central difference of step h of a smooth f has error h^2 f''' / 6 + eps |f| / h;
with h = 1e-5, |f| and its derivatives of order 1 to 100, that is below 1e-7, so
gradients have to agree to 1e-6 of their largest entry.
"""
import numpy as np
import pytest

from mamba_ssd_selective_gb300 import inputs
from oracle import delta

H = 1e-5


def differences(f, x):
    g = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + H
        up = f()
        x[i] = old - H
        g[i] = (up - f()) / (2 * H)
        x[i] = old
    return g


def close(a, b):
    assert np.max(np.abs(a - b)) <= 1e-6 * max(1.0, np.max(np.abs(b)))


@pytest.mark.parametrize("seqlens", [None, [5, 0]])
def test_delta_gradient_against_differences(seqlens):
    d = inputs.delta_inputs(2, 5, 4, 2, 3, 4, io_dtype="f32", seed=1, init_state=True, rate=5.0)
    r = np.random.default_rng(2)
    dy, df = r.standard_normal(d["v"].shape), r.standard_normal(d["init"].shape)
    got = delta.delta_seq_bwd(*(d[n] for n in ("q", "k", "v", "g", "beta")), dy, d["init"], df, seqlens)

    def f():
        y, S = delta.delta_seq(*(d[n] for n in ("q", "k", "v", "g", "beta")), d["init"], seqlens)
        return (dy * y).sum() + (df * S).sum()

    for n in ("q", "k", "v", "g", "beta", "init"):
        close(got["d" + n], differences(f, d[n]))


def test_delta_rule_stores_and_replaces():
    """With no decay and beta 1 a key's value is read back exactly, and a second write replaces it."""
    k = np.zeros((1, 3, 1, 4))
    k[0, 0, 0, 1] = k[0, 1, 0, 2] = k[0, 2, 0, 1] = 1.0
    v = np.arange(1.0, 7.0).reshape(1, 3, 1, 2)
    y, S = delta.delta_seq(k, k, v, np.zeros((1, 3, 1)), np.ones((1, 3, 1)), scale=1.0)
    assert np.array_equal(y, v)
    assert np.array_equal(S[0, 0], [[0, 5, 3, 0], [0, 6, 4, 0]])


@pytest.mark.parametrize("post,z,scale", [(1, 1, 1), (0, 1, 1), (1, 0, 0), (0, 0, 0)])
def test_block_norm_gradient_against_differences(post, z, scale):
    x = inputs.block_norm_inputs(3, 5, "f32", "f32", seed=3)
    opt = dict(post=x["post"] if post else None, z=x["z"] if z else None, scale=x["scale"] if scale else None)
    got = delta.block_norm_bwd(x["y"], x["res"], x["dout"], x["pre"], x["dres"], **opt)

    def f():
        out, r = delta.block_norm(x["y"], x["res"], x["pre"], **opt)
        return (x["dout"] * out).sum() + (x["dres"] * r).sum()

    for n, at in (("dy", "y"), ("dres", "res"), ("dpre_weight", "pre"), ("dz", "z"), ("dpost_weight", "post"),
                  ("dscale", "scale")):
        if got[n] is not None:
            close(got[n], differences(f, x[at]))
