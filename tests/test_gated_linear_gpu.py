"""The gated linear recurrence, its backward, its step and values in 8 bits on the GPU against the float64 definitions
(oracle.linear).

Tolerances. float32: the gates are within about 4 units of 2^-24 of their values, w within 6 of its own, and h sums over
a memory of about 1 / w tokens what an error of w per token makes of it, w times as much: 6 units again; beta adds 4, the
sums over a run and its joints 4: 20 units of 2^-24, 1.2e-6 of the largest term; the gradients have the product of two such
sums. 1e-5 (2-norm) and 1e-4 (largest error over the largest result). bf16 inputs take approximate exponentials, within
37 units at |r| = 30 and 8 at |r| = 5, so float32 results of bf16 inputs get the same; bf16 results are rounded once: at most
2^-8 of each value, so of the 2-norm too, and 1e-5 for the float32 value's own error.
"""
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from mamba_ssd_selective_gb300 import inputs
from oracle import linear
from tests.conftest import ROOT
from tests.helpers import IO_TORCH, dev, host

pytestmark = pytest.mark.gpu
TOL = {torch.float32: (1e-5, 1e-4), torch.bfloat16: (2.0 ** -8 + 1e-5, 2.0 ** -8 + 1e-4)}
SIZES = [(1, 1, 1), (2, 3, 5), (1, 16, 64), (3, 17, 65), (2, 64, 2), (1, 65, 130), (2, 127, 33), (1, 128, 64), (2, 129, 66),
         (4, 300, 1), (3, 777, 97), (1, 2049, 34), (1, 5000, 6), (70, 9, 7)]


def near(got, want, what):
    two, most = TOL[got.dtype]
    got = host(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    norm, top = np.linalg.norm(want), np.max(np.abs(want), initial=0.0)
    assert np.linalg.norm(got - want) <= two * norm, f"{what}: {np.linalg.norm(got - want) / norm:.2e}"
    assert np.max(np.abs(got - want), initial=0.0) <= most * top, f"{what}: {np.max(np.abs(got - want)) / top:.2e}"


def case(size, io, seed=0, rate=1.0, ragged=False):
    """float64 inputs, the same on the device (with NaN past the sequences' ends), and the lengths."""
    d = inputs.linear_inputs(*size, io, seed=seed, rate=rate)
    t = {n: dev(v, IO_TORCH[io] if n in ("x", "r", "i", "dy") else torch.float32) for n, v in d.items()}
    lens = None
    if ragged:
        B, L, _ = size
        lens = np.random.default_rng(seed).integers(0, L + 1, B)
        lens[0], lens[-1] = L + 3, -2  # brought into [0, L]
        for b in range(B):
            for n in ("x", "r", "i", "dy"):
                t[n][b, max(0, lens[b]):] = float("nan")
        t["seqlens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return d, t, lens


def tokens(t):
    return [t[n] for n in ("x", "r", "i", "lam")]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [1.0, 40.0])
@pytest.mark.parametrize("ragged", [False, True])
def test_chunked(ssd, size, io, rate, ragged):
    d, t, lens = case(size, io, size[1], rate, ragged)
    for init in (False, True):
        kept = ssd.gated_linear_checkpoint(t["x"], packed=False)
        y, final = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"] if init else None, seqlens=t.get("seqlens"), **kept)
        wy, wf, ws = linear.linear_seq(d["x"], d["r"], d["i"], d["lam"], 8.0, d["init"] if init else None, lens)
        near(y, wy, "y")
        near(final, wf, "final")
        near(kept["states"], ws, "states")
        y2, none = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"] if init else None, seqlens=t.get("seqlens"),
                                            want_final_state=False)
        assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [1.0, 40.0])
@pytest.mark.parametrize("ragged", [False, True])
def test_backward(ssd, size, io, rate, ragged):
    d, t, lens = case(size, io, size[1] + 1, rate, ragged)
    args = [d[n] for n in ("x", "r", "i", "lam", "dy")]
    for init, dfinal in ((True, True), (False, False)):
        h0, df = (t["init"] if init else None), (t["dfinal"] if dfinal else None)
        want = linear.linear_seq_bwd(*args, 8.0, d["init"] if init else None, d["dfinal"] if dfinal else None, lens)
        kw = dict(dfinal_state=df, seqlens=t.get("seqlens"))
        got = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], init_state=h0, **kw)
        for n, w in want.items():
            near(got[n], w, n)
        kept = ssd.gated_linear_checkpoint(t["x"], packed=False)
        ssd.gated_linear_chunked(*tokens(t), init_state=h0, seqlens=t.get("seqlens"), **kept)
        again = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], **kept, **kw, want_dinit=False)
        assert again["dinit"] is None and all(torch.equal(got[n], again[n]) for n in want if n != "dinit")


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("ragged", [False, True])
def test_checkpoint_in_8_bits(ssd, size, io, ragged):
    """The forward's 8 bits are pack8's, bit for bit, and change nothing else; the backward from them is the definition's at the
    values that they stand for."""
    d, t, lens = case(size, io, size[1] + 2, 1.0, ragged)
    kw = dict(init_state=t["init"], seqlens=t.get("seqlens"))
    y, final = ssd.gated_linear_chunked(*tokens(t), **kw)
    kept = ssd.gated_linear_checkpoint(t["x"])
    y2, final2 = ssd.gated_linear_chunked(*tokens(t), **kw, **kept)
    assert torch.equal(y, y2) and torch.equal(final, final2)
    for z, n in enumerate(("x", "r", "i")):
        values, scales = ssd.pack8(t[n], seqlens=t.get("seqlens"))
        q, code = linear.pack8(d[n], lens)
        assert np.array_equal(host(values), q) and np.array_equal(host(scales), code), n
        assert torch.equal(kept["values"][z], values) and torch.equal(kept["scales"][z], scales), n
        d[n] = linear.unpack8(q, code)
        assert np.array_equal(host(ssd.unpack8(values, scales, IO_TORCH[io])), d[n]), n
    got = ssd.gated_linear_chunked_bwd_packed(lam=t["lam"], dy=t["dy"], dfinal_state=t["dfinal"], seqlens=t.get("seqlens"), **kept)
    want = linear.linear_seq_bwd(d["x"], d["r"], d["i"], d["lam"], d["dy"], 8.0, d["init"], d["dfinal"], lens,
                                 states=host(kept["states"]))
    for n, w in want.items():
        near(got[n], w, n)


@pytest.mark.parametrize("D", [1, 6, 33, 768, 2561])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step(ssd, D, io):
    B, S = 5, 9
    d, t, _ = case((B, 1, D), io, D)
    one = [t[n][:, 0].contiguous() for n in ("x", "r", "i")]
    pool = np.float32(np.random.default_rng(D).standard_normal((S, D))).astype(np.float64)
    slots = np.array([7, -1, 0, S, 3])
    ref = [d[n][:, 0] for n in ("x", "r", "i")]
    for sl in (None, slots):
        wy, wp = linear.linear_step(pool, *ref, d["lam"], 8.0, sl)
        state, new = dev(pool), torch.full((S, D), 77.0, device="cuda")
        on = None if sl is None else torch.tensor(sl, dtype=torch.int32, device="cuda")
        y = ssd.gated_linear_step(state, *one, t["lam"], slots=on, new_state=new)
        near(y, wy, "y")
        used = list(range(B)) if sl is None else [7, 0, 3]
        near(new[used], wp[used], "new states")
        rest = [s for s in range(S) if s not in used]
        assert (new[rest] == 77.0).all() and torch.equal(state, dev(pool))
        same = ssd.gated_linear_step(state, *one, t["lam"], slots=on, y=one[0].clone())
        assert torch.equal(same, y) and torch.equal(state[used], new[used]) and torch.equal(state[rest], dev(pool)[rest])


def test_step_goes_on_where_a_sequence_ends(ssd):
    """A right-padded prefill into a pool, then tokens one at a time, against one pass over the longer sequences."""
    B, L, new, D = 3, 150, 5, 96
    d, t, _ = case((B, L + new, D), "f32", 3)
    lens = [150, 1, 77]
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = [t[n][:, :L].contiguous() for n in ("x", "r", "i")]
    _, final = ssd.gated_linear_chunked(*first, t["lam"], init_state=t["init"], seqlens=seqlens)
    pool, slots = torch.zeros(5, D, device="cuda"), torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = final
    whole = {n: d[n].copy() for n in ("x", "r", "i")}
    ys = []
    for s in range(new):
        ys.append(ssd.gated_linear_step(pool, *(t[n][:, L + s].contiguous() for n in ("x", "r", "i")), t["lam"], slots=slots))
        for n, w in whole.items():
            for b in range(B):
                w[b, lens[b] + s] = d[n][b, L + s]
    wy, wf, _ = linear.linear_seq(*whole.values(), d["lam"], 8.0, d["init"], [n + new for n in lens])
    near(torch.stack(ys, 1), np.stack([wy[b, lens[b]:lens[b] + new] for b in range(B)]), "tokens")
    near(pool[slots.long()], wf, "states")


def test_training_step_beside_the_gated_delta_rule(ssd):
    """Two layers, a gated delta rule on the recurrence's outputs, with every activation that the backward reads again in 8
    bits: the gradients are the ones of the plain chain at those values."""
    B, L, H, N = 2, 200, 4, 16
    d, t, _ = case((B, L, H * N), "bf16", 8)
    kept = ssd.gated_linear_checkpoint(t["x"])
    h, _ = ssd.gated_linear_chunked(*tokens(t), **kept)
    r = inputs.delta_inputs(B, L, H, H, N, N, "bf16", seed=9)
    tok = {n: dev(r[n], torch.bfloat16) for n in ("q", "k", "g", "beta")}
    v8 = ssd.pack8(h.view(B, L, H, N))
    dv = ssd.gated_delta_chunked_bwd(v=ssd.unpack8(*v8), dy=t["dy"].view(B, L, H, N), **tok)["dv"]
    got = ssd.gated_linear_chunked_bwd_packed(lam=t["lam"], dy=dv.view(B, L, H * N), **kept)
    back = [linear.unpack8(*linear.pack8(d[n])) for n in ("x", "r", "i")]
    want = linear.linear_seq_bwd(*back, d["lam"], host(dv).reshape(B, L, -1), states=host(kept["states"]))
    for n in ("dx", "dr", "di", "dlam"):
        near(got[n], want[n], n)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gates_of_any_size(ssd, io):
    """r and i from -80 to 80 and lam from -40 to 40, every channel on its own scale; at -200 a gate counts as shut."""
    B, L, D = 2, 90, 64
    d = inputs.linear_inputs(B, L, D, io, seed=4)
    d["r"] = inputs.round_to(np.random.default_rng(1).uniform(-80, 80, (B, L, D)) * (np.arange(D) % 4 / 3), io)
    d["i"] = inputs.round_to(np.random.default_rng(2).uniform(-80, 80, (B, L, D)) * (np.arange(D) // 4 % 4 / 3), io)
    d["lam"] = inputs.round_to(np.linspace(-40, 40, D), "f32")
    t = {n: dev(v, IO_TORCH[io] if n in ("x", "r", "i", "dy") else torch.float32) for n, v in d.items()}
    args = [d[n] for n in ("x", "r", "i", "lam")]
    y, final = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"])
    wy, wf, _ = linear.linear_seq(*args, 8.0, d["init"])
    got = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], init_state=t["init"])
    want = linear.linear_seq_bwd(*args, d["dy"], 8.0, d["init"])
    # exp of |x| <= 80 by the special function unit: 2 + 1.2 |x| units of 2^-23, 1.2e-5; beta has half of rho's and iota all of its
    # own, w all of rho's: 2.4e-5 of the terms, 1e-4 with what cancels
    tol = 1e-4 if io == "f32" else 2.0 ** -8 + 1e-4
    for n, g, w in [("y", y, wy), ("final", final, wf)] + [(n, got[n], want[n]) for n in want]:
        g, axes = host(g), tuple(range(w.ndim - 1))
        assert np.isfinite(g).all(), n
        assert (np.abs(g - w).max(axes) <= tol * np.abs(w).max(axes) + 1e-30).all(), n
    t["r"].fill_(-200.0)
    y, final = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"])
    assert torch.equal(final, t["init"]) and torch.equal(y, t["init"].to(y.dtype)[:, None].expand_as(y))
    got = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], init_state=t["init"])
    assert not got["dx"].any() and not got["dr"].any() and not got["dlam"].any() and all(torch.isfinite(g).all() for g in got.values())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_channel(ssd, bad):
    B, L, D = 2, 300, 70
    _, t, _ = case((B, L, D), "bf16", 6)
    kept, kept2 = ssd.gated_linear_checkpoint(t["x"]), ssd.gated_linear_checkpoint(t["x"])
    y, _ = ssd.gated_linear_chunked(*tokens(t), **kept)
    g = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], **{"states": kept["states"]})
    t["x"][1, 200, 9] = bad
    y2, _ = ssd.gated_linear_chunked(*tokens(t), **kept2)
    g2 = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], **{"states": kept2["states"]})
    p2 = ssd.gated_linear_chunked_bwd_packed(lam=t["lam"], dy=t["dy"], **kept2)
    assert not torch.isfinite(y2[1, 200:, 9]).any()
    y2[1, 200:, 9] = y[1, 200:, 9]
    assert torch.equal(y, y2)
    others = [c for c in range(D) if c != 9]
    for n in ("dx", "dr", "di"):
        assert torch.equal(g[n][0], g2[n][0]) and torch.equal(g[n][1][:, others], g2[n][1][:, others]), n
        assert torch.isfinite(p2[n][:, :, others].float()).all() and torch.isfinite(p2[n][0].float()).all()
    assert torch.equal(g["dlam"][others], g2["dlam"][others])
    assert (kept2["scales"][0, 1, 12, 9] == 255) and not kept2["values"][0, 1, 192:208, 9].any()
    assert torch.isnan(ssd.unpack8(kept2["values"][0], kept2["scales"][0])[1, 192:208, 9]).all()
    kept2["values"][0, 1, 192:208, 9], kept2["scales"][0, 1, 12, 9] = kept["values"][0, 1, 192:208, 9], kept["scales"][0, 1, 12, 9]
    assert torch.equal(kept["values"], kept2["values"]) and torch.equal(kept["scales"], kept2["scales"])


def test_pack8_values_of_any_size(ssd):
    """Powers from the least float32 to the largest, ties, and group maxima on both sides of 127 2^e."""
    r = np.random.default_rng(5)
    x = np.ldexp(r.uniform(-1, 1, (3, 70, 301)), r.integers(-148, 126, (1, 1, 301)))
    x[:, :, :20] = np.ldexp(r.integers(-254, 255, (3, 70, 20)) / 2.0, np.arange(20) * 12 - 130)  # whole and halves: ties
    x[:, :, 20] = 127.0
    x[:, 1::16, 20] = np.nextafter(np.float32(127), np.float32(128))
    x[:, :, 21:23] = 0.0
    x = np.float32(x).astype(np.float64)
    for io in ("f32", "bf16"):
        v = inputs.round_to(x, io)
        q, code = linear.pack8(v)
        values, scales = ssd.pack8(dev(v, IO_TORCH[io]))
        assert np.array_equal(host(values), q) and np.array_equal(host(scales), code), io
        assert np.array_equal(host(ssd.unpack8(values, scales, IO_TORCH[io])), linear.unpack8(q, code)), io
        assert np.array_equal(host(ssd.unpack8(values, scales, torch.float32)), linear.unpack8(q, code)), io
    w, s = ssd.pack8(dev(v, torch.float32).view(3, 70, 7, 43))
    assert w.shape == (3, 70, 7, 43) and s.shape == (3, 5, 7, 43) and np.array_equal(host(w).reshape(q.shape), q)


@pytest.mark.parametrize("L", [5, 130, 1111])
def test_a_sequence_alone_is_bitwise_the_one_in_a_batch(ssd, L):
    B, D = 40, 200
    d, t, _ = case((B, L, D), "bf16", 7)
    kept = ssd.gated_linear_checkpoint(t["x"])
    y, final = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"], **kept)
    g = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], states=kept["states"], dfinal_state=t["dfinal"])
    for b in (0, 17, 39):
        one = [t[n][b:b + 1].contiguous() for n in ("x", "r", "i")]
        k1 = ssd.gated_linear_checkpoint(one[0])
        y1, f1 = ssd.gated_linear_chunked(*one, t["lam"], init_state=t["init"][b:b + 1].contiguous(), **k1)
        assert torch.equal(y1[0], y[b]) and torch.equal(f1[0], final[b]) and torch.equal(k1["states"][0], kept["states"][b])
        g1 = ssd.gated_linear_chunked_bwd(*one, t["lam"], t["dy"][b:b + 1].contiguous(), states=k1["states"],
                                          dfinal_state=t["dfinal"][b:b + 1].contiguous())
        assert all(torch.equal(g1[n][0], g[n][b]) for n in ("dx", "dr", "di", "dinit"))


def test_empty_calls(ssd):
    lam = torch.zeros(6, device="cuda")
    h0, none = torch.randn(3, 6, device="cuda"), torch.zeros(3, 0, 6, device="cuda")
    y, final = ssd.gated_linear_chunked(none, none, none, lam, init_state=h0, **ssd.gated_linear_checkpoint(none))
    assert y.shape == none.shape and torch.equal(final, h0)
    for kw in ({}, dict(states=torch.zeros(3, 0, 6, device="cuda"))):
        g = ssd.gated_linear_chunked_bwd(none, none, none, lam, none, dfinal_state=h0, **kw)
        assert torch.equal(g["dinit"], h0) and torch.equal(g["dlam"], lam)
    g = ssd.gated_linear_chunked_bwd_packed(lam=lam, dy=none, **ssd.gated_linear_checkpoint(none))
    assert not g["dinit"].any() and not g["dlam"].any()
    none = torch.zeros(0, 5, 6, device="cuda")
    y, final = ssd.gated_linear_chunked(none, none, none, lam)
    assert y.shape == (0, 5, 6) and final.shape == (0, 6)
    assert not ssd.gated_linear_chunked_bwd(none, none, none, lam, none)["dlam"].any()
    assert ssd.gated_linear_step(h0, none[:, 0], none[:, 0], none[:, 0], lam).shape == (0, 6)
    v, s = ssd.pack8(none)
    assert ssd.unpack8(v, s).shape == none.shape


def test_captured_and_replayed(ssd):
    """Two graphs of a training step and a decode step, replayed with other inputs, one after the other."""
    graphs = []
    for size, seed in (((2, 333, 66), 1), ((1, 1000, 31), 2)):
        _, t, _ = case(size, "bf16", seed)
        pool = t["init"].clone()
        one = [t[n][:, 0].contiguous() for n in ("x", "r", "i")]

        def step(t=t, pool=pool, one=one):
            kept = ssd.gated_linear_checkpoint(t["x"])
            y, final = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"], **kept)
            g = ssd.gated_linear_chunked_bwd_packed(lam=t["lam"], dy=t["dy"], dfinal_state=t["dfinal"], **kept)
            g2 = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], init_state=t["init"])
            return [y, final, *g.values(), *g2.values(), ssd.gated_linear_step(pool, *one, t["lam"], new_state=torch.empty_like(pool))]

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out, step, t))
    for again in range(2):
        for graph, out, step, t in graphs:
            t["x"].copy_(torch.randn_like(t["x"]))
            t["dy"].mul_(0.5)
            graph.replay()
        for graph, out, step, t in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_on_another_stream(ssd):
    """A call held up on its stream, while the current stream overwrites what was let go of."""
    _, t, _ = case((3, 700, 510), "bf16", 9)

    def call(t, stream=None):
        kept = ssd.gated_linear_checkpoint(t["x"])
        y, final = ssd.gated_linear_chunked(*tokens(t), stream=stream, **kept)
        g = ssd.gated_linear_chunked_bwd_packed(lam=t["lam"], dy=t["dy"], stream=stream, **kept)
        g2 = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], stream=stream)
        return [y, final, *g.values(), *g2.values(), ssd.unpack8(*ssd.pack8(t["x"], stream=stream), stream=stream)]

    want = call(t)
    copies = {n: v.clone() for n, v in t.items()}
    torch.cuda.synchronize()
    side, held = torch.cuda.Stream(), torch.cuda.Event()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        held.record()
    got = call(copies, side)
    del copies
    junk = [torch.full((1 << k,), 0x7f, dtype=torch.uint8, device="cuda") for k in range(10, 26) for _ in range(3)]
    assert not held.query()
    torch.cuda.synchronize()
    del junk
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits(ssd):
    """2.3 G elements a tensor: the last sequence is bitwise the one alone."""
    B, L, D = 3, 30000, 25600
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    x, r, i = (torch.empty(B, L, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(3))
    lam = torch.full((D,), -6.0, device="cuda")
    kept = ssd.gated_linear_checkpoint(x)
    y, final = ssd.gated_linear_chunked(x, r, i, lam, **kept)
    one = [v[2:] for v in (x, r, i)]
    k1 = ssd.gated_linear_checkpoint(one[0])
    y1, f1 = ssd.gated_linear_chunked(*one, lam, **k1)
    assert torch.equal(y[2:], y1) and torch.equal(final[2:], f1) and torch.equal(kept["states"][2:], k1["states"])
    assert torch.equal(kept["values"][:, 2:], k1["values"]) and torch.equal(kept["scales"][:, 2:], k1["scales"])
    del y1
    g = ssd.gated_linear_chunked_bwd_packed(lam=lam, dy=y, **kept)
    g1 = ssd.gated_linear_chunked_bwd_packed(lam=lam, dy=y[2:], **k1)
    assert all(torch.equal(g[n][2:], g1[n]) for n in ("dx", "dr", "di", "dinit"))
    del g, g1, kept
    v, s = ssd.pack8(x)
    assert torch.equal(v[2:], k1["values"][0]) and torch.equal(ssd.unpack8(v, s)[2:], ssd.unpack8(v[2:], s[2:]))


# widths whose rows are multiples of 16 bytes, tiles of fewer than 64 channels, lengths on both sides of a block's 64 tokens and of
# clusters of 16 of them, and more sequences and tiles than the device holds clusters
WIDE = [(1, 1, 8), (2, 63, 16), (2, 64, 72), (3, 65, 200), (2, 1025, 24), (1, 5000, 72), (300, 70, 136), (5, 130, 16), (2, 200, 1000)]


@pytest.mark.parametrize("size", WIDE)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [1.0, 40.0])
@pytest.mark.parametrize("ragged", [False, True])
def test_wide_rows(ssd, size, io, rate, ragged):
    """The forward, its states and 8 bits, and both backwards."""
    d, t, lens = case(size, io, size[1] + size[2], rate, ragged)
    args = [d[n] for n in ("x", "r", "i", "lam")]
    kept = ssd.gated_linear_checkpoint(t["x"])
    y, final = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"], seqlens=t.get("seqlens"), **kept)
    wy, wf, ws = linear.linear_seq(*args, 8.0, d["init"], lens)
    near(y, wy, "y")
    near(final, wf, "final")
    near(kept["states"], ws, "states")
    y2, final2 = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"], seqlens=t.get("seqlens"))
    assert torch.equal(y, y2) and torch.equal(final, final2)
    kw = dict(dfinal_state=t["dfinal"], seqlens=t.get("seqlens"))
    want = linear.linear_seq_bwd(*args, d["dy"], 8.0, d["init"], d["dfinal"], lens)
    for how in (dict(init_state=t["init"]), dict(states=kept["states"])):
        got = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], **how, **kw)
        for n, w in want.items():
            near(got[n], w, n)
    back = []
    for z, n in enumerate(("x", "r", "i")):
        q, code = linear.pack8(d[n], lens)
        assert np.array_equal(host(kept["values"][z]), q) and np.array_equal(host(kept["scales"][z]), code), n
        back.append(linear.unpack8(q, code))
    got = ssd.gated_linear_chunked_bwd_packed(lam=t["lam"], dy=t["dy"], **kept, **kw)
    want = linear.linear_seq_bwd(*back, d["lam"], d["dy"], 8.0, d["init"], d["dfinal"], lens, states=host(kept["states"]))
    for n, w in want.items():
        near(got[n], w, n)
    assert ssd.gated_linear_status() == ssd.SSD_OK


@pytest.mark.parametrize("D", [64, 65, 520])
def test_states_updated_in_place(ssd, D):
    d, t, lens = case((30, 100, D), "bf16", 11, 1.0, True)
    want = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"], seqlens=t["seqlens"])
    for _ in range(3):
        state = t["init"].clone()
        got = ssd.gated_linear_chunked(*tokens(t), init_state=state, final_state=state, seqlens=t["seqlens"])
        assert got[1] is state and torch.equal(got[0], want[0]) and torch.equal(state, want[1])


@pytest.mark.parametrize("D", [72, 33])
def test_gates_that_are_not_finite(ssd, D):
    """NaN or an infinity in r or i: NaN (or a gate that is open or shut) in its channel from there on, the others near what they were."""
    _, t, _ = case((2, 200, D), "bf16", 12)
    want, _ = ssd.gated_linear_chunked(*tokens(t))
    others = [c for c in range(D) if c != 7]
    for n in ("r", "i"):
        for bad in (float("nan"), float("inf"), -float("inf")):
            u = dict(t, **{n: t[n].clone()})
            u[n][1, 100, 7] = bad
            y, _ = ssd.gated_linear_chunked(*tokens(u))
            g = ssd.gated_linear_chunked_bwd(*tokens(u), t["dy"])
            assert torch.isnan(y[1, 100:, 7]).all() if bad != bad else torch.isfinite(y).all()
            assert torch.equal(y[0], want[0]) and torch.equal(y[1, :96], want[1, :96])
            diff = (y[1][:, others].float() - want[1][:, others].float()).abs()
            assert (diff <= 2.0 ** -7 * want[1][:, others].float().abs() + 1e-5).all()
            assert all(torch.isfinite(v.float()[..., others]).all() for v in g.values())
            if bad == bad:
                assert all(torch.isfinite(v.float()).all() for v in g.values())


FIRST_CALL = """
import torch
from mamba_ssd_selective_gb300 import binding as ops
x, lam = torch.randn(2, 300, 128, device="cuda").bfloat16(), torch.full((128,), -5.0, device="cuda")
side = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    kept = ops.gated_linear_checkpoint(x)
    y, final = ops.gated_linear_chunked(x, x, x, lam, **kept)
    g = ops.gated_linear_chunked_bwd_packed(lam=lam, dy=x, **kept)
    g2 = ops.gated_linear_chunked_bwd(x, x, x, lam, x)
graph.replay()
torch.cuda.synchronize()
kept2 = ops.gated_linear_checkpoint(x)
y2, _ = ops.gated_linear_chunked(x, x, x, lam, **kept2)
g3 = ops.gated_linear_chunked_bwd_packed(lam=lam, dy=x, **kept2)
assert torch.equal(y, y2) and all(torch.equal(g[n], g3[n]) for n in g) and torch.equal(kept["values"], kept2["values"])
assert torch.isfinite(g2["dlam"]).all()
"""


def test_first_call_of_a_process_is_captured(ssd):
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_from_two_threads(ssd):
    """First and later calls of two host threads, each on its stream."""
    said = []

    def work(D):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                _, t, _ = case((2, 400, D), "bf16", D)
                want = None
                for _ in range(50):
                    kept = ssd.gated_linear_checkpoint(t["x"])
                    y, _ = ssd.gated_linear_chunked(*tokens(t), **kept)
                    g = ssd.gated_linear_chunked_bwd_packed(lam=t["lam"], dy=t["dy"], **kept)
                    got = [y, *(v for v in g.values() if v is not None)]
                    assert want is None or all(torch.equal(a, b) for a, b in zip(got, want))
                    want = got
        except BaseException as e:  # noqa: B902
            said.append(e)

    threads = [threading.Thread(target=work, args=(D,)) for D in (64, 520, 33, 64)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not said


@pytest.mark.parametrize("B,D", [(255, 1024), (66, 5120), (1000, 333)])
def test_step_of_many_rows(ssd, B, D):
    """Batches of which a thread takes several rows, some of them idle: rows as they are one by one."""
    _, t, _ = case((B, 1, D), "bf16", 14)
    one = [t[n][:, 0].contiguous() for n in ("x", "r", "i")]
    pool = torch.randn(B + 7, D, device="cuda")
    slots = torch.randperm(B + 7, device="cuda")[:B].to(torch.int32)
    slots[::9] = -1
    slots[4::9] = B + 7
    new, want = pool.clone(), pool.clone()
    y = ssd.gated_linear_step(new, *one, t["lam"], slots=slots)
    for b in range(B):
        yb = ssd.gated_linear_step(want, *(v[b:b + 1] for v in one), t["lam"], slots=slots[b:b + 1].clone()) if D % 8 == 0 else \
            ssd.gated_linear_step(want, *(v[b:b + 1].clone() for v in one), t["lam"], slots=slots[b:b + 1].clone())
        assert torch.equal(yb[0], y[b])
    assert torch.equal(new, want)
