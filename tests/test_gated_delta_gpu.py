"""The gated delta rule on the GPU against its float64 definition (oracle.delta).

Tolerances, from the formats: 2-norm of the error over the 2-norm of the result, and the largest error over
the largest result.
* float32 inputs: sums of up to 256 float32 terms and a recurrence that is a contraction for keys of norm 1;
  each step adds rounding of a few 2^-24, so 1e-5 (2-norm) and 1e-4 (largest) leave a factor above ten.
* bf16 inputs, results in bf16: rounding the result is 2^-8 of a value at most and 1.7e-3 in the 2-norm; up to four operands
  of the products before it are rounded to bf16 as well (1.7e-3 each, independent), together below 4e-3: 6e-3
  (2-norm), and 2e-2 for the largest error, the bf16 parity bound of the scans.
* bf16 inputs, float32 states: their operands are held as pairs of bf16 (2^-17 and below), a few in a row: 1e-5 and 1e-4.
"""
import numpy as np
import pytest
import torch

from mamba_ssd_selective_gb300 import inputs
from oracle import delta
from tests.helpers import IO_TORCH, dev, host

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")
TOL = {"f32": (1e-5, 1e-4), "bf16": (6e-3, 2e-2), "state": (1e-5, 1e-4)}


def near(got, want, kind, what):
    got = host(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    two, most = TOL[kind]
    if not want.size:
        return
    norm, top = np.linalg.norm(want), np.max(np.abs(want))
    if not top:
        assert not np.any(got), what
        return
    assert np.linalg.norm(got - want) <= two * norm, f"{what}: {np.linalg.norm(got - want) / norm:.2e} > {two}"
    assert np.max(np.abs(got - want)) <= most * top, f"{what}: {np.max(np.abs(got - want)) / top:.2e} > {most}"


def tokens(d, io):
    return {n: dev(d[n], IO_TORCH[io]) for n in NAMES}


def lens_of(seqlens):
    return None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device="cuda")


# B, L, H, G, P, N: one token, around the 64-token chunk and its 16-token blocks, odd sizes, one head per group,
# heads sharing a group in odd and even numbers, state rows above and below 64, columns that are no multiple of 8
SHAPES = [(1, 1, 1, 1, 64, 128), (2, 17, 2, 1, 64, 128), (1, 63, 3, 1, 64, 128), (1, 64, 2, 2, 64, 128),
          (2, 65, 4, 2, 64, 128), (1, 130, 2, 1, 128, 128), (3, 200, 6, 2, 64, 128), (1, 193, 3, 3, 128, 64),
          (2, 100, 4, 4, 48, 64), (1, 77, 2, 1, 33, 20), (1, 70, 3, 1, 200, 128), (1, 65, 2, 1, 16, 7),
          (1, 40, 1, 1, 64, 200), (1, 33, 2, 1, 8, 250), (1, 700, 2, 1, 64, 128), (1, 129, 8, 1, 64, 72)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("init", [False, True])
def test_chunked(ssd, io, shape, init):
    B, L, H, G, P, N = shape
    d = inputs.delta_inputs(B, L, H, G, P, N, io, seed=L, init_state=init)
    yr, Sr = delta.delta_seq(*(d[n] for n in NAMES), d["init"])
    y, S = ssd.gated_delta_chunked(**tokens(d, io), init_state=dev(d["init"]))
    near(y, yr, io, "y")
    near(S, Sr, "state", "final_state")
    if io == "bf16":
        y, S = ssd.gated_delta_chunked(**tokens(d, io), init_state=dev(d["init"]), simt=True)
        near(y, yr, io, "y, CUDA cores")
        near(S, Sr, "state", "final_state, CUDA cores")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["strong decay", "no decay", "steep decay", "mean key", "beta"])
def test_chunked_extremes(ssd, io, what):
    """Decays that underflow within a chunk, none at all, keys with a common direction, beta of 0 and 1."""
    d = inputs.delta_inputs(2, 330, 4, 2, 64, 128, io, seed=5, init_state=True,
                            rate={"strong decay": 20.0, "no decay": 0.0, "steep decay": 400.0}.get(what, 1.0),
                            mean_key=0.5 if what == "mean key" else 0.0)
    if what == "beta":
        d["beta"] = np.round(d["beta"])
    yr, Sr = delta.delta_seq(*(d[n] for n in NAMES), d["init"])
    y, S = ssd.gated_delta_chunked(**tokens(d, io), init_state=dev(d["init"]))
    near(y, yr, io, "y")
    near(S, Sr, "state", "final_state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P", [64, 128])
def test_chunked_seqlens_hide_what_is_past_them(ssd, io, P):
    lens = [150, 0, 1, 64, 127]
    d = inputs.delta_inputs(5, 150, 4, 2, P, 128, io, seed=6, init_state=True)
    yr, Sr = delta.delta_seq(*(d[n] for n in NAMES), d["init"], lens)
    t = tokens(d, io)
    for n, x in t.items():
        for b, m in enumerate(lens):
            x[b, m:] = float("nan") if b % 2 else float("inf")
    y, S = ssd.gated_delta_chunked(**t, init_state=dev(d["init"]), seqlens=lens_of(lens))
    near(y, yr, io, "y")
    near(S, Sr, "state", "final_state")
    over = lens_of([999, -3, 1, 64, 127])
    y2, S2 = ssd.gated_delta_chunked(**t, init_state=dev(d["init"]), seqlens=over)
    assert torch.equal(y, y2) and torch.equal(S, S2)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_chunked_empty_sequences_and_state_in_place(ssd, io):
    d = inputs.delta_inputs(2, 90, 4, 2, 64, 128, io, seed=7, init_state=True)
    t, init = tokens(d, io), dev(d["init"])
    y, S = ssd.gated_delta_chunked(**{n: x[:, :0].contiguous() for n, x in t.items()}, init_state=init)
    assert y.shape == (2, 0, 4, 64) and torch.equal(S, init)
    _, S = ssd.gated_delta_chunked(**{n: x[:, :0].contiguous() for n, x in t.items()})
    assert not S.any()
    _, want = ssd.gated_delta_chunked(**t, init_state=init)
    _, got = ssd.gated_delta_chunked(**t, init_state=init, final_state=init)
    assert got is init and torch.equal(got, want)
    y, S = ssd.gated_delta_chunked(**t, want_final_state=False)
    assert S is None


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_chunked_is_reproducible_and_splits(ssd, io):
    """Bitwise the same twice and for each sequence alone; two halves give the whole up to rounding."""
    d = inputs.delta_inputs(3, 256, 4, 2, 64, 128, io, seed=8, init_state=True)
    t, init = tokens(d, io), dev(d["init"])
    y, S = ssd.gated_delta_chunked(**t, init_state=init, scale=0.5)
    y2, S2 = ssd.gated_delta_chunked(**t, init_state=init, scale=0.5)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    y1, S1 = ssd.gated_delta_chunked(**{n: x[1:2].contiguous() for n, x in t.items()}, init_state=init[1:2], scale=0.5)
    assert torch.equal(y[1:2], y1) and torch.equal(S[1:2], S1)
    ya, Sa = ssd.gated_delta_chunked(**{n: x[:, :100].contiguous() for n, x in t.items()}, init_state=init, scale=0.5)
    yb, Sb = ssd.gated_delta_chunked(**{n: x[:, 100:].contiguous() for n, x in t.items()}, init_state=Sa, scale=0.5)
    near(torch.cat([ya, yb], 1), host(y), io, "y")
    near(Sb, host(S), "state", "final_state")


def test_chunked_on_another_stream(ssd):
    d = inputs.delta_inputs(1, 300, 4, 2, 64, 128, "bf16", seed=9)
    t = tokens(d, "bf16")
    want, _ = ssd.gated_delta_chunked(**t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = ssd.gated_delta_chunked(**t)
    side.synchronize()
    assert torch.equal(want, got)


# ----------------------------------------------------------------------- backward

BWD = [(1, 1, 1, 1, 64, 128), (2, 17, 2, 1, 64, 128), (1, 64, 2, 2, 64, 128), (2, 65, 4, 2, 64, 128),
       (1, 130, 3, 1, 64, 128), (1, 130, 2, 1, 128, 128), (3, 200, 6, 2, 64, 128), (1, 193, 2, 2, 128, 64),
       (1, 77, 2, 1, 33, 20), (1, 65, 2, 1, 16, 7), (1, 40, 2, 1, 64, 200), (1, 500, 8, 1, 64, 128)]
GRADS = ("dq", "dk", "dv", "dg", "dbeta")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", BWD)
@pytest.mark.parametrize("states", [False, True])
def test_backward(ssd, io, shape, states):
    B, L, H, G, P, N = shape
    d = inputs.delta_inputs(B, L, H, G, P, N, io, seed=L + 1, init_state=states)
    r = np.random.default_rng(L)
    dy = inputs.round_to(r.standard_normal(d["v"].shape), io)
    df = inputs.round_to(0.1 * r.standard_normal((B, H, P, N)), "f32") if states else None
    want = delta.delta_seq_bwd(*(d[n] for n in NAMES), dy, d["init"], df)
    for simt in ([False, True] if io == "bf16" else [False]):
        got = ssd.gated_delta_chunked_bwd(**tokens(d, io), dy=dev(dy, IO_TORCH[io]), init_state=dev(d["init"]),
                                          dfinal_state=dev(df), simt=simt)
        for n in GRADS:
            assert got[n].dtype == IO_TORCH[io]
            near(got[n], want[n], io, f"{n}, simt={simt}")
        near(got["dinit"], want["dinit"], "state", f"dinit, simt={simt}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rate,mean_key", [(0.0, 0.0), (20.0, 0.0), (400.0, 0.0), (1.0, 0.5)])
def test_backward_extremes(ssd, io, rate, mean_key):
    d = inputs.delta_inputs(1, 200, 4, 2, 64, 128, io, seed=11, init_state=True, rate=rate, mean_key=mean_key)
    r = np.random.default_rng(12)
    dy = inputs.round_to(r.standard_normal(d["v"].shape), io)
    df = inputs.round_to(0.1 * r.standard_normal(d["init"].shape), "f32")
    want = delta.delta_seq_bwd(*(d[n] for n in NAMES), dy, d["init"], df)
    got = ssd.gated_delta_chunked_bwd(**tokens(d, io), dy=dev(dy, IO_TORCH[io]), init_state=dev(d["init"]),
                                      dfinal_state=dev(df))
    for n in GRADS:
        near(got[n], want[n], io, n)
    near(got["dinit"], want["dinit"], "state", "dinit")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_backward_seqlens(ssd, io):
    lens = [130, 0, 1, 64]
    d = inputs.delta_inputs(4, 130, 4, 2, 64, 128, io, seed=13, init_state=True)
    r = np.random.default_rng(14)
    dy = inputs.round_to(r.standard_normal(d["v"].shape), io)
    df = inputs.round_to(0.1 * r.standard_normal(d["init"].shape), "f32")
    want = delta.delta_seq_bwd(*(d[n] for n in NAMES), dy, d["init"], df, lens)
    t, dyt = tokens(d, io), dev(dy, IO_TORCH[io])
    for x in (*t.values(), dyt):
        for b, m in enumerate(lens):
            x[b, m:] = float("nan")
    got = ssd.gated_delta_chunked_bwd(**t, dy=dyt, init_state=dev(d["init"]), dfinal_state=dev(df),
                                      seqlens=lens_of(lens))
    again = ssd.gated_delta_chunked_bwd(**t, dy=dyt, init_state=dev(d["init"]), dfinal_state=dev(df),
                                        seqlens=lens_of(lens))
    for n in GRADS:
        near(got[n], want[n], io, n)
        assert torch.equal(got[n], again[n])
    near(got["dinit"], want["dinit"], "state", "dinit")
    empty = ssd.gated_delta_chunked_bwd(**{n: x[:, :0].contiguous() for n, x in t.items()}, dy=dyt[:, :0].contiguous(),
                                        dfinal_state=dev(df))
    assert torch.equal(empty["dinit"], dev(df))


def test_backward_against_differences(ssd):
    """The float32 backward against central differences of the float32 forward along random directions. With steps
    of 1e-2 of the inputs' size the third-order term is about 1e-4 of the derivative and rounding 2^-24 |f| / 1e-2,
    below 1e-3 of it for these sizes: 1e-2."""
    d = inputs.delta_inputs(1, 60, 2, 1, 16, 24, "f32", seed=15, init_state=True)
    t, init = tokens(d, "f32"), dev(d["init"])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rnd = lambda x: torch.randn(x.shape, generator=gen, device="cuda")  # noqa: E731
    dy, df = rnd(t["v"]), rnd(init)
    got = ssd.gated_delta_chunked_bwd(**t, dy=dy, init_state=init, dfinal_state=df)

    def f(over):
        y, S = ssd.gated_delta_chunked(**{**t, **{n: x for n, x in over.items() if n != "init"}},
                                       init_state=over.get("init", init))
        return float((dy.double() * y.double()).sum() + (df.double() * S.double()).sum())

    for n, x in [*t.items(), ("init", init)]:
        way = got["d" + n] / got["d" + n].norm()  # along the gradient: the derivative is its norm
        h = 1e-2 * float(x.norm()) / x.numel() ** 0.5
        slope = (f({n: x + h * way}) - f({n: x - h * way})) / (2 * h)
        assert abs(slope - float(got["d" + n].norm())) <= 1e-2 * abs(slope), n


# --------------------------------------------------------------------------- step

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 24, 12, 64, 128), (7, 4, 2, 128, 128), (3, 6, 6, 33, 20), (2, 2, 1, 16, 7),
                                   (65, 8, 1, 64, 128), (2, 3, 1, 50, 256), (5, 2, 2, 8, 133)])
def test_step(ssd, io, shape):
    B, H, G, P, N = shape
    d = inputs.delta_inputs(B, 1, H, G, P, N, io, seed=21)
    one = {n: d[n][:, 0] for n in NAMES}
    S0 = inputs.round_to(0.2 * np.random.default_rng(3).standard_normal((B + 2, H, P, N)), "f32")
    t = {n: dev(x, IO_TORCH[io]) for n, x in one.items()}
    yr, Sr = delta.delta_step(S0, **one)
    state = dev(S0)
    other = torch.zeros_like(state)
    y = ssd.gated_delta_step(state, **t, new_state=other)
    near(y, yr, io, "y")
    near(other[:B], Sr[:B], "state", "new_state")
    assert not other[B:].any() and torch.equal(state, dev(S0))
    y2 = ssd.gated_delta_step(state, **t)
    assert torch.equal(y, y2) and torch.equal(state[:B], other[:B]) and torch.equal(state[B:], dev(S0)[B:])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_slots(ssd, io):
    """Rows in any order over a pool; rows outside it are idle whatever they hold."""
    B, H, G, P, N, S = 6, 4, 2, 64, 128, 9
    d = inputs.delta_inputs(B, 1, H, G, P, N, io, seed=22)
    one = {n: d[n][:, 0] for n in NAMES}
    S0 = inputs.round_to(0.2 * np.random.default_rng(4).standard_normal((S, H, P, N)), "f32")
    slots = [8, -1, 0, 9, 3, -7]
    yr, Sr = delta.delta_step(S0, **one, slots=slots)
    t = {n: dev(x, IO_TORCH[io]) for n, x in one.items()}
    for x in t.values():
        x[1] = float("nan")
        x[3] = float("inf")
    state = dev(S0)
    y = ssd.gated_delta_step(state, **t, slots=lens_of(slots))
    near(y, yr, io, "y")
    near(state, Sr, "state", "state")
    assert torch.equal(state[[1, 2, 4, 5, 6, 7]], dev(S0)[[1, 2, 4, 5, 6, 7]])


def test_steps_follow_the_chunked_rule(ssd):
    """Tokens one by one against the whole sequence at once, from the same state."""
    d = inputs.delta_inputs(2, 70, 4, 2, 64, 128, "bf16", seed=23, init_state=True)
    t = tokens(d, "bf16")
    y, S = ssd.gated_delta_chunked(**t, init_state=dev(d["init"]))
    state = dev(d["init"])
    ys = [ssd.gated_delta_step(state, **{n: x[:, i].contiguous() for n, x in t.items()}) for i in range(70)]
    near(torch.stack(ys, 1), host(y), "bf16", "y")
    near(state, host(S), "state", "state")


def test_step_in_a_long_pool(ssd):
    """Offsets that pass 32 bits: the last states of a pool of 9 GB."""
    H, P, N = 80, 64, 128
    S = (9 << 30) // (4 * H * P * N)
    assert S * H * P * N > 1 << 31
    state = torch.zeros((S, H, P, N), dtype=torch.float32, device="cuda")
    d = inputs.delta_inputs(2, 1, H, 1, P, N, "bf16", seed=24)
    one = {n: d[n][:, 0] for n in NAMES}
    t = {n: dev(x, torch.bfloat16) for n, x in one.items()}
    y = ssd.gated_delta_step(state, **t, slots=lens_of([S - 1, S - 2]))
    yr, Sr = delta.delta_step(np.zeros((2, H, P, N)), **one)
    near(y, yr, "bf16", "y")
    near(state[S - 1], Sr[0], "state", "state")
    near(state[S - 2], Sr[1], "state", "state")
    assert not state[:16].any()


def test_example_block(ssd):
    """The example: prefill, decode and gradients together; decoding agrees with one pass over the whole sequence."""
    import importlib.util
    import os
    from tests.conftest import ROOT
    spec = importlib.util.spec_from_file_location("gated_delta_block", os.path.join(ROOT, "examples", "gated_delta_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main() < 2e-2


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P", [64, 128])
def test_backward_where_beta_is_zero(ssd, io, P):
    """Tokens that write nothing still have a gradient with respect to beta."""
    d = inputs.delta_inputs(2, 140, 4, 2, P, 128, io, seed=17, init_state=True)
    d["beta"][:, ::5] = 0.0
    d["beta"][1] = 0.0
    r = np.random.default_rng(18)
    dy = inputs.round_to(r.standard_normal(d["v"].shape), io)
    df = inputs.round_to(0.1 * r.standard_normal(d["init"].shape), "f32")
    want = delta.delta_seq_bwd(*(d[n] for n in NAMES), dy, d["init"], df)
    got = ssd.gated_delta_chunked_bwd(**tokens(d, io), dy=dev(dy, IO_TORCH[io]), init_state=dev(d["init"]),
                                      dfinal_state=dev(df))
    for n in GRADS:
        near(got[n], want[n], io, n)


@pytest.mark.parametrize("shape", [(1, 1, 2, 1, 64, 128), (4, 1, 40, 10, 64, 128), (2, 20, 40, 20, 128, 64), (1, 130, 2, 1, 64, 128)])
@pytest.mark.parametrize("simt", [False, True])
def test_first_decay_has_no_gradient_without_a_state(ssd, shape, simt):
    d = inputs.delta_inputs(*shape, "bf16", seed=41)
    t = tokens(d, "bf16")
    dy = torch.ones_like(t["v"])
    got = ssd.gated_delta_chunked_bwd(**t, dy=dy, simt=simt)
    assert (got["dg"][:, 0] == 0).all()
    got = ssd.gated_delta_chunked_bwd(**t, dy=dy, init_state=torch.ones(shape[0], shape[2], shape[4], shape[5], device="cuda"), simt=simt)
    assert (got["dg"][:, 0] != 0).any()


# more chains than SMs: they are cut between CTAs, and the state is handed on between them
MANY = [(1, 400, 160, 160, 64, 128), (5, 330, 64, 32, 64, 128), (1, 130, 100, 100, 200, 128), (2, 200, 80, 80, 128, 64)]
# and few chains of many chunks, which are cut into pieces that run at once
FEW = [(1, 1500, 2, 1, 64, 128), (2, 1100, 2, 2, 128, 128), (1, 1281, 3, 1, 48, 64), (5, 1300, 1, 1, 64, 128), (1, 1024, 4, 1, 200, 40)]


# with the slow decay the state of one piece is still felt in the next
@pytest.mark.parametrize("shape,rate", [(s, 1.0) for s in MANY + FEW] + [(s, 0.01) for s in FEW])
@pytest.mark.parametrize("ragged", [False, True])
def test_chains_cut_between_blocks(ssd, shape, rate, ragged):
    B, L, H, G, P, N = shape
    lens = [[L, 0, 70, 1, L - 1][i % 5] for i in range(B)] if ragged else None
    d = inputs.delta_inputs(B, L, H, G, P, N, "bf16", seed=31, init_state=True, rate=rate)
    t, init = tokens(d, "bf16"), dev(d["init"])
    for n, x in t.items():
        for b, m in enumerate(lens or []):
            x[b, m:] = float("nan")
    y, S = ssd.gated_delta_chunked(**t, init_state=init, seqlens=lens_of(lens))
    yr, Sr = delta.delta_seq(*(d[n] for n in NAMES), d["init"], lens)
    near(y, yr, "bf16", "y")
    near(S, Sr, "state", "final_state")
    if P > 128:
        return
    r = np.random.default_rng(32)
    dy = inputs.round_to(r.standard_normal(d["v"].shape), "bf16")
    df = inputs.round_to(0.1 * r.standard_normal(d["init"].shape), "f32")
    want = delta.delta_seq_bwd(*(d[n] for n in NAMES), dy, d["init"], df, lens)
    dyt = dev(dy, torch.bfloat16)
    for b, m in enumerate(lens or []):
        dyt[b, m:] = float("nan")
    got = ssd.gated_delta_chunked_bwd(**t, dy=dyt, init_state=init, dfinal_state=dev(df), seqlens=lens_of(lens))
    for n in GRADS:
        near(got[n], want[n], "bf16", n)
    near(got["dinit"], want["dinit"], "state", "dinit")


@pytest.mark.parametrize("shape", FEW + [(1, 1301, 8, 8, 128, 128)])
@pytest.mark.parametrize("ragged", [False, True])
def test_state_in_place_where_chains_are_cut(ssd, shape, ragged):
    """A pool updated in place: the pieces of a chain run at once, and only the last one may write the state."""
    B, L, H, G, P, N = shape
    lens = lens_of([[L - 130, L, 0, 70, 1][i % 5] for i in range(B)]) if ragged else None
    d = inputs.delta_inputs(B, L, H, G, P, N, "bf16", seed=33, init_state=True, rate=0.01)
    t, init = tokens(d, "bf16"), dev(d["init"])
    y, S = ssd.gated_delta_chunked(**t, init_state=init, seqlens=lens)
    state = init.clone()
    y2, S2 = ssd.gated_delta_chunked(**t, init_state=state, final_state=state, seqlens=lens)
    assert S2 is state and torch.equal(y, y2) and torch.equal(S, S2)
    y, S = ssd.gated_delta_chunked(**t, seqlens=lens)
    y2, S2 = ssd.gated_delta_chunked(**t, init_state=torch.zeros_like(init), seqlens=lens)
    assert torch.equal(y, y2) and torch.equal(S, S2)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("beta", [2.0 ** -40, 2.0 ** -70, 2.0 ** -120, 2.0 ** -126, 2.0 ** -133, -2.0 ** -120])
def test_backward_where_beta_is_tiny(ssd, io, beta):
    """Tokens that write next to nothing, down to the least bf16: their dbeta has the size of the others'. (Their dv is
    beta times that, below the normal numbers, and is not asked for.)"""
    d = inputs.delta_inputs(1, 100, 4, 2, 64, 128, io, seed=19, init_state=True)
    d["beta"][:, ::3] = beta
    r = np.random.default_rng(20)
    dy = inputs.round_to(r.standard_normal(d["v"].shape), io)
    want = delta.delta_seq_bwd(*(d[n] for n in NAMES), dy, d["init"])
    got = ssd.gated_delta_chunked_bwd(**tokens(d, io), dy=dev(dy, IO_TORCH[io]), init_state=dev(d["init"]))
    for n in GRADS:
        near(got[n], want[n], io, n)
    near(got["dbeta"][:, ::3], want["dbeta"][:, ::3], io, "dbeta of those tokens")


@pytest.mark.parametrize("how", ["small", "fast"])
def test_backward_head_by_head(ssd, how):
    """Heads of one group whose gradients or decays lie far apart, each head's dg and dbeta against its own size: dg of
    the last four is what is left of sums with the first four, whose gradients are a thousand times theirs."""
    d = inputs.delta_inputs(2, 300, 8, 1, 64, 128, "bf16", seed=61, init_state=True)
    dy = np.random.default_rng(62).standard_normal(d["v"].shape)
    if how == "small":
        dy[:, :, 4:] *= 1e-3
    else:
        d["g"][:, :, 4:] = inputs.round_to(100 * d["g"][:, :, 4:], "bf16")
    dy = inputs.round_to(dy, "bf16")
    want = delta.delta_seq_bwd(*(d[n] for n in NAMES), dy, d["init"])
    got = ssd.gated_delta_chunked_bwd(**tokens(d, "bf16"), dy=dev(dy, torch.bfloat16), init_state=dev(d["init"]))
    for n in ("dv", "dg", "dbeta"):
        for h in range(8):
            near(got[n][:, :, h], want[n][:, :, h], "bf16", f"{n} of head {h}")
