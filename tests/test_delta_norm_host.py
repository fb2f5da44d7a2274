"""Refusals of the gated delta rule and the block norm: the C ABI turns down
bad calls before any CUDA call, and the binding turns down tensors of another
shape, type or layout. No GPU needed."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from mamba_ssd_selective_gb300 import binding
from mamba_ssd_selective_gb300 import build as nvbuild
from tests.conftest import ROOT

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p(1 << 20)  # an aligned address that no refused call may touch


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return binding.load()


def dims(**kw):
    base = dict(batch=2, seqlen=100, nheads=4, headdim=64, dstate=128, ngroups=2, io_dtype=1, flags=0)
    base.update(kw)
    return binding.ssd_dims(**base)


def chunked(lib, d, ptrs=None, scale=1.0, ws=P, bytes_=1 << 30):
    p = dict(q=P, k=P, v=P, g=P, beta=P, init=P, seqlens=P, y=P, final=P)
    p.update(ptrs or {})
    return lib.ssd_gated_delta_chunked(ctypes.byref(d), p["q"], p["k"], p["v"], p["g"], p["beta"], p["init"],
                                       p["seqlens"], scale, p["y"], p["final"], ws, bytes_, None)


def backward(lib, d, bad=None, scale=1.0, ws=P, bytes_=1 << 40):
    a = [P] * 15
    if bad is not None:
        a[bad[0]] = bad[1]
    return lib.ssd_gated_delta_chunked_bwd(ctypes.byref(d), *a[:7], scale, *a[7:15], ws, bytes_, None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(nheads=0), INVALID), (dict(headdim=0), INVALID),
    (dict(dstate=0), INVALID), (dict(ngroups=3), INVALID), (dict(io_dtype=2), INVALID), (dict(flags=2), INVALID),
    (dict(flags=8), INVALID), (dict(dstate=257), UNSUPPORTED), (dict(headdim=65536), UNSUPPORTED),
    (dict(seqlen=1 << 31), UNSUPPORTED)])
def test_delta_sizes_are_refused(lib, kw, want):
    d = dims(**kw)
    assert chunked(lib, d) == want
    assert backward(lib, d) == want
    assert lib.ssd_gated_delta_workspace_size(ctypes.byref(d)) == 0
    assert lib.ssd_gated_delta_chunked_bwd_workspace_size(ctypes.byref(d)) == 0
    assert lib.ssd_last_error()


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "y"])
def test_delta_missing_and_misaligned_pointers(lib, name):
    assert chunked(lib, dims(), {name: None}) == INVALID
    assert chunked(lib, dims(), {name: ctypes.c_void_p((1 << 20) + 4)}) == INVALID


def test_delta_backward_pointers(lib):
    for i in (0, 1, 2, 3, 4, 7, 9, 10, 11, 12, 13):
        assert backward(lib, dims(), (i, None)) == INVALID, i
    for i in range(15):
        assert backward(lib, dims(), (i, ctypes.c_void_p((1 << 20) + 2))) == INVALID, i


def test_delta_workspace_and_scale(lib):
    d = dims()
    need = lib.ssd_gated_delta_workspace_size(ctypes.byref(d))
    assert need > 0
    assert chunked(lib, d, ws=None) == INVALID
    assert chunked(lib, d, ws=ctypes.c_void_p((1 << 20) + 16)) == INVALID
    assert chunked(lib, d, bytes_=need - 1) == INVALID
    need = lib.ssd_gated_delta_chunked_bwd_workspace_size(ctypes.byref(d))
    assert backward(lib, d, bytes_=need - 1) == INVALID
    for s in (float("nan"), float("inf")):
        assert chunked(lib, d, scale=s) == INVALID
        assert backward(lib, d, scale=s) == INVALID
    assert lib.ssd_gated_delta_chunked(None, *[P] * 7, 1.0, P, P, P, 1 << 20, None) == INVALID


def test_delta_empty_batch_is_fine(lib):
    assert chunked(lib, dims(batch=0), {n: None for n in ("q", "k", "v", "g", "beta", "y")}, ws=None, bytes_=0) == OK


def test_delta_step_refusals(lib):
    def step(d, nslots=2, slots=P, **bad):
        p = [bad.get(n, P) for n in ("state", "q", "k", "v", "g", "beta")]
        return lib.ssd_gated_delta_step(ctypes.byref(d), nslots, *p, slots, bad.get("scale", 1.0), bad.get("new", P),
                                        bad.get("y", P), None)

    assert step(dims(), nslots=1, slots=None) == INVALID
    assert step(dims(), nslots=-1) == INVALID
    assert step(dims(dstate=300)) == UNSUPPORTED
    assert step(dims(flags=2)) == INVALID
    for n in ("state", "q", "k", "v", "g", "beta", "new", "y"):
        assert step(dims(), **{n: None}) == INVALID
        assert step(dims(), **{n: ctypes.c_void_p((1 << 20) + 8)}) == INVALID
    assert step(dims(), scale=float("inf")) == INVALID
    assert step(dims(batch=0), nslots=0, slots=None) == OK


def test_block_norm_refusals(lib):
    def fwd(rows=3, dim=64, io=1, rio=1, eps=1e-5, bad=None):
        a = [P] * 8
        if bad:
            a[bad[0]] = bad[1]
        return lib.ssd_block_norm(rows, dim, io, rio, *a[:6], eps, a[6], a[7], None)

    def bwd(rows=3, dim=64, io=1, rio=1, eps=1e-5, bad=None, bytes_=1 << 30):
        a = [P] * 15
        if bad:
            a[bad[0]] = bad[1]
        return lib.ssd_block_norm_bwd(rows, dim, io, rio, *a[:6], eps, *a[6:15], bytes_, None)

    for f in (fwd, bwd):
        assert f(rows=-1) == INVALID
        assert f(dim=0) == INVALID
        assert f(io=3) == INVALID
        assert f(io=0, rio=1) == INVALID
        assert f(eps=-1.0) == INVALID
        assert f(eps=float("nan")) == INVALID
        assert f(dim=16385) == UNSUPPORTED
        assert f(rows=1 << 31) == UNSUPPORTED
    assert fwd(rows=0) == OK
    for i in (0, 1, 5, 6, 7):
        assert fwd(bad=(i, None)) == INVALID
    for i in (0, 1, 5, 6, 8, 9, 10, 11, 12, 13, 14):
        assert bwd(bad=(i, None)) == INVALID, i
    for i in range(14):
        assert bwd(bad=(i, ctypes.c_void_p((1 << 20) + 4))) == INVALID, i
    assert bwd(bytes_=64) == INVALID


def test_binding_refuses_other_tensors():
    B, L, H, G, Pd, N = 2, 5, 4, 2, 8, 16
    t = dict(q=torch.zeros(B, L, G, N), k=torch.zeros(B, L, G, N), v=torch.zeros(B, L, H, Pd), g=torch.zeros(B, L, H),
             beta=torch.zeros(B, L, H))
    for n, x, err in [("k", torch.zeros(B, L, G, N + 1), ValueError), ("g", torch.zeros(B, L, G), ValueError),
                      ("beta", torch.zeros(B, L, H, dtype=torch.bfloat16), TypeError),
                      ("v", torch.zeros(B, H, L, Pd).transpose(1, 2), ValueError), ("q", None, AttributeError),
                      ("k", [1], TypeError)]:
        with pytest.raises(err):
            binding.gated_delta_chunked(**{**t, n: x})
    with pytest.raises(TypeError):
        binding.gated_delta_chunked(**t, seqlens=torch.zeros(B, dtype=torch.int64))
    with pytest.raises(ValueError):
        binding.gated_delta_chunked(**t, init_state=torch.zeros(B, H, N, Pd))
    with pytest.raises(TypeError):
        binding.gated_delta_chunked(**{n: x.half() for n, x in t.items()})
    one = {n: x[:, 0].contiguous() for n, x in t.items()}
    with pytest.raises(ValueError):
        binding.gated_delta_step(torch.zeros(1, H, Pd, N), **one)
    y = torch.zeros(3, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.block_norm(y, y.half(), torch.ones(8))
    with pytest.raises(ValueError):
        binding.block_norm(y, y, torch.ones(7))
    with pytest.raises(ValueError):
        binding.block_norm(y[:, ::2], y[:, ::2], torch.ones(4))
    with pytest.raises(TypeError):
        binding.block_norm_bwd(y, y, y.float(), torch.ones(8))


WIDTHS = """
import ctypes
from mamba_ssd_selective_gb300 import binding
lib, P = binding.load(), ctypes.c_void_p(1 << 20)
for io, rio in ((0, 0), (1, 1), (1, 0)):
    for dim in range(1, 16385):
        for f in (lambda: lib.ssd_block_norm(3, dim, io, rio, *[P] * 6, 1e-5, P, P, None),
                  lambda: lib.ssd_block_norm_bwd(3, dim, io, rio, *[P] * 6, 1e-5, *[P] * 9, 1 << 40, None)):
            assert f() == binding.SSD_ERR_CUDA, (dim, io, rio)
            assert b"invalid argument" not in lib.ssd_last_error(), (dim, io, rio, lib.ssd_last_error())
"""


def test_block_norm_has_a_kernel_for_every_width(lib):
    """In a process that sees no GPU the calls end at the first CUDA call, with the driver's error; a width without a
    kernel is turned down before it as an invalid argument."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", WIDTHS], env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
