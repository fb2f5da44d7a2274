"""The binding's `stream` argument: a call on another stream than torch's current one.

Without a GPU, torch's stream functions and the library are replaced by records of what was called: every tensor that a
call makes has to be made while `stream` is current (the allocator hands memory out in the order of the stream it was
made on), and what was given or is returned has to be marked as used on the other stream. With one, the calls are held up
on their stream while the current stream overwrites all memory that was let go of.
"""
import contextlib

import pytest
import torch

from mamba_ssd_selective_gb300 import binding, inputs
from tests.helpers import IO_TORCH, dev

B, L, H, G, P, N, D = 2, 3, 4, 2, 8, 16, 24


def calls(make):
    """name -> arguments of every entry point that makes tensors, from make(*shape)."""
    x, dt, A, Bm, C = make(B, L, H, P), make(B, L, H), make(H), make(B, L, G, N), make(B, L, G, N)
    tok = dict(q=make(B, L, G, N), k=make(B, L, G, N), v=make(B, L, H, P), g=make(B, L, H), beta=make(B, L, H))
    one = dict(q=make(B, G, N), k=make(B, G, N), v=make(B, H, P), g=make(B, H), beta=make(B, H))
    norm = dict(y=make(5, D), res=make(5, D), pre_weight=make(D), post_weight=make(D), z=make(5, D), scale=make(D))
    Cc = H * P + 2 * G * N
    return dict(
        ssd_scan_chunked=dict(x=x, dt=dt, A=A, B=Bm, C=C, chunk_size=128),
        ssd_scan_chunked_bwd=dict(x=x, dt=dt, A=A, B=Bm, C=C, dy=make(B, L, H, P), D=make(H)),
        ssd_decode_step=dict(state=make(B, H, P, N), x=make(B, H, P), dt=make(B, H), A=A, B=make(B, G, N), C=make(B, G, N)),
        selective_scan_diag=dict(x=make(B, L, D), dt=make(B, L, D), A=make(D, N), B=make(B, L, N), C=make(B, L, N)),
        conv1d_step=dict(x=make(B, D), conv_state=make(B, D, 4), weight=make(D, 4)),
        gated_rmsnorm=dict(y=make(B, D), z=make(B, D), weight=make(D)),
        decode_layer_step=dict(xBC=make(B, Cc), conv_state=make(B, Cc, 4), conv_weight=make(Cc, 4), conv_bias=make(Cc), dt=make(B, H),
                               A=A, D=make(H), ssm_state=make(B, H, P, N), z=make(B, H * P), norm_weight=make(H * P)),
        gated_delta_chunked=tok, gated_delta_chunked_bwd=dict(tok, dy=make(B, L, H, P)),
        gated_delta_step=dict(one, state=make(B, H, P, N)), block_norm=norm,
        block_norm_bwd=dict(norm, dout=make(5, D)))


class FakeStream:
    cuda_stream = 77


@pytest.mark.parametrize("name", sorted(calls(torch.zeros)))
def test_what_a_call_makes_belongs_to_its_stream(monkeypatch, name):
    here, side, current, made, used = FakeStream(), FakeStream(), [], [], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def recorded(f):
        def g(*a, **kw):
            made.append((current[-1] if current else None, f(*a, **kw)))
            return made[-1][1]
        return g

    class Library:
        def __getattr__(self, f):
            return lambda *a: 4096 if f.endswith("_size") else 0

    args = calls(torch.zeros)[name]
    monkeypatch.setattr(binding, "_elsewhere", lambda stream, device: stream is not None, raising=False)
    monkeypatch.setattr(binding, "_stream", lambda stream, device: 0)
    monkeypatch.setattr(binding, "load", Library)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1] if current else here)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: used.append((t, s)))
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, recorded(getattr(torch, f)))
    out = getattr(binding, name)(**args, stream=side)
    out = [t for t in (out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)) if t is not None]
    assert made and all(s is side for s, _ in made)
    for t in args.values():
        assert not isinstance(t, torch.Tensor) or any(u is t and s is side for u, s in used)
    assert out and all(any(u is t and s is here for u, s in used) for t in out)


@pytest.mark.parametrize("stream", [None, FakeStream()])
@pytest.mark.parametrize("name", sorted(calls(torch.zeros)))
def test_tensors_in_host_memory_are_refused(monkeypatch, name, stream):
    """By their device, whatever the stream, before the library gets a pointer."""
    class Library:
        def __getattr__(self, f):
            return lambda *a: 4096 if f.endswith("_size") else pytest.fail(f"{f} was called")

    monkeypatch.setattr(binding, "load", Library)
    with pytest.raises(ValueError, match="CUDA device"):
        getattr(binding, name)(**calls(torch.zeros)[name], stream=stream)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["chunked", "backward", "norm_bwd", "scan"])
def test_memory_let_go_of_while_the_call_waits(ssd, what):
    d = inputs.delta_inputs(2, 1100, 4, 2, 64, 128, "bf16", seed=51, init_state=True)
    tok = {n: dev(d[n], IO_TORCH["bf16"]) for n in ("q", "k", "v", "g", "beta")}
    n = inputs.block_norm_inputs(700, 2560, "bf16", "f32", seed=52)
    norm = {k: dev(x, IO_TORCH["bf16"] if k in ("y", "z", "dout") else torch.float32) for k, x in n.items()}
    s = inputs.ssd_inputs(2, 1100, 4, 64, 128, 2, io_dtype="bf16", seed=53)
    scan = {k: dev(s[k], torch.float32 if k == "A" else IO_TORCH["bf16"]) for k in ("x", "dt", "A", "B", "C")}

    def call(c, stream=None):
        if what == "chunked":
            return ssd.gated_delta_chunked(**c, stream=stream)
        if what == "backward":
            return tuple(ssd.gated_delta_chunked_bwd(**c, dy=c["v"], stream=stream).values())
        if what == "norm_bwd":
            return tuple(ssd.block_norm_bwd(c["y"], c["res"], c["dout"], c["pre"], dres_out=c["dres"], post_weight=c["post"],
                                            z=c["z"], scale=c["scale"], stream=stream).values())
        return ssd.ssd_scan_chunked(**c, stream=stream)

    def overwrite():
        return [torch.full((1 << k,), 0x7f, dtype=torch.uint8, device="cuda") for k in range(10, 28) for _ in range(3)]

    given = {"norm_bwd": norm, "scan": scan}.get(what, tok)
    want = call(given)
    overwrite()  # what this allocates is at hand below
    side, held = torch.cuda.Stream(), torch.cuda.Event()
    copies = {k: x.clone() for k, x in given.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 100 ms
        held.record()
    got = call(copies, side)
    del copies
    junk = overwrite()
    assert not held.query()  # the call has not begun, and its memory could have been overwritten
    torch.cuda.synchronize()
    del junk
    assert len(got) == len(want) and all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))
