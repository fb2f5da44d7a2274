"""The gated linear recurrence and values in 8 bits without a GPU: the float64 definitions against central differences and
closed cases, and the refusals of the C ABI (before any CUDA call) and of the binding.

A central difference of step h of a smooth f has error h^2 f''' / 6 + eps |f| / h; with h = 1e-5, |f| and its derivatives of
order 1 to 100, that is below 1e-7, so gradients have to agree to 1e-6 of their largest entry.
"""
import ctypes

import numpy as np
import pytest
import torch

from mamba_ssd_selective_gb300 import binding, inputs
from mamba_ssd_selective_gb300 import build as nvbuild
from oracle import linear
from tests import test_stream_argument as streams

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p(1 << 20)  # an aligned address that no refused call may touch
H = 1e-5


# ------------------------------------------------------------ the definitions

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


@pytest.mark.parametrize("seqlens", [None, [7, 0, 3]])
@pytest.mark.parametrize("rate", [1.0, 30.0])
def test_gradient_against_differences(seqlens, rate):
    d = inputs.linear_inputs(3, 7, 2, "f32", seed=1, rate=rate)
    args = [d[n] for n in ("x", "r", "i", "lam")]
    got = linear.linear_seq_bwd(*args, d["dy"], 8.0, d["init"], d["dfinal"], seqlens)

    def f():
        y, final, _ = linear.linear_seq(*args, 8.0, d["init"], seqlens)
        return (d["dy"] * y).sum() + (d["dfinal"] * final).sum()

    for n in ("x", "r", "i", "lam", "init"):
        want = differences(f, d[n])
        assert np.max(np.abs(got["d" + n] - want)) <= 1e-6 * max(1.0, np.max(np.abs(want))), n


def test_closed_cases():
    """An open gate that forgets at once gives sigmoid(i) x; one that is shut keeps the state."""
    x = np.arange(1.0, 7.0).reshape(1, 3, 2)
    y, final, _ = linear.linear_seq(x, np.full(x.shape, 50.0), np.full(x.shape, 50.0), np.full(2, 50.0))
    assert np.allclose(y, x, rtol=1e-12) and np.allclose(final, x[:, -1])
    y, final, states = linear.linear_seq(x, np.full(x.shape, -800.0), x, np.zeros(2), init=[[3.0, -4.0]])
    assert (y == [3.0, -4.0]).all() and (states == [3.0, -4.0]).all()
    y, final, _ = linear.linear_seq(x, x, x, np.zeros(2), init=[[3.0, -4.0]], seqlens=[0])
    assert not y.any() and (final == [3.0, -4.0]).all()


def test_pack8_definition():
    x = np.zeros((1, 40, 3))
    x[0, :16, 0] = np.arange(16) * 127 / 15
    x[0, 3, 1] = 127.5  # above 127: the next power of two
    x[0, 35, 2] = -np.inf
    q, code = linear.pack8(x)
    assert code[0, :, 0].tolist() == [127, 0, 0] and code[0, 0, 1] == 128 and q[0, 3, 1] == 64
    assert code[0, :, 2].tolist() == [0, 0, 255] and not q[..., 2].any()
    back = linear.unpack8(q, code)
    assert np.isnan(back[0, 32:, 2]).all() and np.isfinite(back[0, :32]).all()
    assert np.max(np.abs(back[0, :16, 0] - x[0, :16, 0])) <= 0.5
    q, code = linear.pack8(x, seqlens=[4])
    assert not q[0, 4:].any() and code[0, 0, 0] == 125 and not code[0, 1:].any()  # 25.4 = 101.6 2^-2


# --------------------------------------------------------------- the refusals

@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return binding.load()


IN, OUT = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)


def fwd(lib, B=2, L=100, D=64, io=1, c=8.0, bad=None):
    a = [IN] * 4 + [OUT] * 7
    if bad:
        a[bad[0]] = bad[1]
    return lib.ssd_gated_linear_chunked(B, L, D, io, *a[:4], c, *a[4:], None)


def bwd(lib, B=2, L=100, D=64, io=1, c=8.0, bad=None, bytes_=1 << 40):
    a = [IN] * 8 + [OUT] * 7
    if bad:
        a[bad[0]] = bad[1]
    return lib.ssd_gated_linear_chunked_bwd(B, L, D, io, *a[:4], c, *a[4:15], bytes_, None)


def bwd_packed(lib, B=2, L=100, D=64, io=1, c=8.0, bad=None, bytes_=1 << 40):
    a = [IN] * 6 + [OUT] * 7
    if bad:
        a[bad[0]] = bad[1]
    return lib.ssd_gated_linear_chunked_bwd_packed(B, L, D, io, *a[:3], c, *a[3:13], bytes_, None)


def step(lib, B=2, L=1, D=64, io=1, c=8.0, bad=None, nslots=2):
    a = [P] * 8
    if bad:
        a[bad[0]] = bad[1]
    return lib.ssd_gated_linear_step(B, D, io, nslots, *a[:5], c, *a[5:8], None)


def pack(lib, B=2, L=100, D=64, io=1, c=8.0, bad=None):
    a = [P] * 4
    if bad:
        a[bad[0]] = bad[1]
    return lib.ssd_pack8(B, L, D, io, *a, None)


def unpack(lib, B=2, L=100, D=64, io=1, c=8.0, bad=None):
    a = [P] * 3
    if bad:
        a[bad[0]] = bad[1]
    return lib.ssd_unpack8(B, L, D, io, *a, None)


CALLS = [fwd, bwd, bwd_packed, step, pack, unpack]


@pytest.mark.parametrize("call", CALLS)
def test_sizes_are_refused(lib, call):
    assert call(lib, B=-1) == INVALID
    assert call(lib, D=0) == INVALID
    assert call(lib, io=2) == INVALID
    assert lib.ssd_last_error()
    assert call(lib, B=65536) == UNSUPPORTED
    assert call(lib, D=32 * 65535 + 1) == UNSUPPORTED
    if call is not step:
        assert call(lib, L=-1) == INVALID
        assert call(lib, L=1 << 31) == UNSUPPORTED
    if call not in (pack, unpack):
        for c in (0.0, -1.0, float("nan"), float("inf")):
            assert call(lib, c=c) == INVALID


@pytest.mark.parametrize("call,needed,total", [
    (fwd, (0, 1, 2, 3, 6), 11), (bwd, (0, 1, 2, 3, 7, 9, 10, 11, 12, 14), 15), (bwd_packed, (0, 1, 2, 3, 5, 7, 8, 9, 10, 12), 13),
    (step, (0, 1, 2, 3, 4, 6, 7), 8), (pack, (0, 2, 3), 4), (unpack, (0, 1, 2), 3)])
def test_missing_and_misaligned_pointers(lib, call, needed, total):
    for i in needed:
        assert call(lib, bad=(i, None)) == INVALID, i
    for i in range(total):
        assert call(lib, bad=(i, ctypes.c_void_p((1 << 20) + 4))) == INVALID, i


def test_results_in_the_place_of_inputs(lib):
    assert fwd(lib, bad=(6, IN)) == INVALID
    for i in (9, 10, 11):
        assert bwd(lib, bad=(i, IN)) == INVALID
    for i in (7, 8, 9):
        assert bwd_packed(lib, bad=(i, IN)) == INVALID


def test_values_and_scales_go_together(lib):
    assert fwd(lib, bad=(9, None)) == INVALID
    assert fwd(lib, bad=(10, None)) == INVALID


def test_workspace(lib):
    size = lib.ssd_gated_linear_chunked_bwd_workspace_size
    assert size(2, 100, 64, 1, 0) - size(2, 100, 64, 1, 1) >= 2 * 2 * 64 * 4
    assert size(2, 100, 0, 1, 0) == 0 and size(2, 100, 64, 3, 0) == 0 and size(70000, 1, 1, 1, 0) == 0
    assert bwd(lib, bytes_=size(2, 100, 64, 1, 1) - 1) == INVALID
    assert bwd(lib, bad=(5, None), bytes_=size(2, 100, 64, 1, 0) - 1) == INVALID
    assert bwd_packed(lib, bytes_=size(2, 100, 64, 1, 1) - 1) == INVALID
    assert bwd(lib, bad=(14, ctypes.c_void_p((1 << 20) + 16))) == INVALID


def test_step_pools(lib):
    assert step(lib, bad=(5, None), nslots=1) == INVALID
    assert step(lib, nslots=-1) == INVALID


def test_empty_calls_are_fine(lib):
    assert lib.ssd_gated_linear_chunked(0, 5, 4, 1, *[None] * 4, 8.0, *[None] * 8) == OK
    assert lib.ssd_gated_linear_step(0, 4, 1, 0, *[None] * 5, 8.0, *[None] * 4) == OK
    for B, L in ((0, 5), (2, 0)):
        assert lib.ssd_pack8(B, L, 4, 1, *[None] * 5) == OK
        assert lib.ssd_unpack8(B, L, 4, 1, *[None] * 4) == OK


def test_binding_refuses_other_tensors():
    B, L, D = 2, 70, 6
    z = torch.zeros
    t = dict(x=z(B, L, D), r=z(B, L, D), i=z(B, L, D), lam=z(D))
    for n, x, err in [("r", z(B, L, D + 1), ValueError), ("i", z(B, L, D, dtype=torch.bfloat16), TypeError),
                      ("r", z(B, D, L).transpose(1, 2), ValueError), ("lam", z(D + 1), ValueError), ("i", None, TypeError),
                      ("lam", None, TypeError), ("lam", z(D, dtype=torch.bfloat16), TypeError), ("x", z(B, D), ValueError),
                      ("r", [1], TypeError)]:
        with pytest.raises(err):
            binding.gated_linear_chunked(**{**t, n: x})
    kept = binding.gated_linear_checkpoint(t["x"])
    assert {n: tuple(k.shape) for n, k in kept.items()} == dict(states=(B, 2, D), values=(3, B, L, D), scales=(3, B, 5, D))
    for bad in (dict(kept, scales=None), dict(kept, states=z(B, 1, D)), dict(kept, values=z(B, L, D, dtype=torch.int8)),
                dict(seqlens=z(B, dtype=torch.int64)), dict(init_state=z(D, B)), dict(y=z(B, L, D + 1)),
                dict(final_state=z(B, D, dtype=torch.bfloat16))):
        with pytest.raises((ValueError, TypeError)):
            binding.gated_linear_chunked(**t, **bad)
    for bad in (dict(dy=z(B, L, D, dtype=torch.bfloat16)), dict(dy=t["x"], states=z(B, 2, D + 1)), dict(dy=t["x"], dfinal_state=z(D))):
        with pytest.raises((ValueError, TypeError)):
            binding.gated_linear_chunked_bwd(**t, **bad)
    for bad in (dict(states=None), dict(values=kept["values"].to(torch.uint8)), dict(scales=None), dict(dy=z(B, L))):
        with pytest.raises((ValueError, TypeError)):
            binding.gated_linear_chunked_bwd_packed(**{**kept, "lam": t["lam"], "dy": t["x"], **bad})
    with pytest.raises(TypeError):
        binding.gated_linear_chunked(**{n: x.half() for n, x in t.items() if n != "lam"}, lam=t["lam"])
    one = {n: x[:, 0].contiguous() if n != "lam" else x for n, x in t.items()}
    for bad in (dict(state=z(1, D)), dict(state=z(3, D + 1)), dict(state=z(3, D), slots=z(B)), dict(state=z(3, D), y=z(3, D))):
        with pytest.raises((ValueError, TypeError)):
            binding.gated_linear_step(**one, **bad)
    v, s = z(B, L, D, dtype=torch.int8), z(B, 5, D, dtype=torch.uint8)
    for f in (lambda: binding.pack8(z(L, D)), lambda: binding.pack8(t["x"].half()), lambda: binding.pack8(t["x"], values=v[:1]),
              lambda: binding.pack8(t["x"][..., ::2]), lambda: binding.pack8(t["x"], scales=s[:, :4]),
              lambda: binding.unpack8(v, s[:, :4].contiguous()), lambda: binding.unpack8(v, s, torch.float16),
              lambda: binding.unpack8(v, s, out=t["x"]), lambda: binding.unpack8(s, s), lambda: binding.unpack8(v, None)):
        with pytest.raises((ValueError, TypeError)):
            f()


# ------------------------------------------------------------ another stream

def calls(make):
    """name -> arguments of every entry point that makes tensors, from make(*shape)."""
    B, L, D = 2, 70, 6
    i8 = lambda *s: make(*s).to(torch.int8)  # noqa: E731
    u8 = lambda *s: make(*s).to(torch.uint8)  # noqa: E731
    tok, lam = dict(x=make(B, L, D), r=make(B, L, D), i=make(B, L, D)), make(D)
    kept = dict(states=make(B, 2, D), values=i8(3, B, L, D), scales=u8(3, B, 5, D))
    return dict(
        gated_linear_chunked=dict(tok, lam=lam, **kept), gated_linear_chunked_bwd=dict(tok, lam=lam, dy=make(B, L, D)),
        gated_linear_chunked_bwd_packed=dict(kept, lam=lam, dy=make(B, L, D)),
        gated_linear_step=dict(state=make(B, D), x=make(B, D), r=make(B, D), i=make(B, D), lam=lam),
        pack8=dict(x=make(B, L, D)), unpack8=dict(values=i8(B, L, D), scales=u8(B, 5, D)))


@pytest.mark.parametrize("name", sorted(calls(torch.zeros)))
def test_what_a_call_makes_belongs_to_its_stream(monkeypatch, name):
    monkeypatch.setattr(streams, "calls", calls)
    streams.test_what_a_call_makes_belongs_to_its_stream(monkeypatch, name)


@pytest.mark.parametrize("stream", [None, streams.FakeStream()])
@pytest.mark.parametrize("name", sorted(calls(torch.zeros)))
def test_tensors_in_host_memory_are_refused(monkeypatch, name, stream):
    monkeypatch.setattr(streams, "calls", calls)
    streams.test_tensors_in_host_memory_are_refused(monkeypatch, name, stream)
