"""What a gated-linear kernel leaves when one of its bounded waits runs out. The debug build, in a child process, has a barrier count
bytes that nothing sends: the wait ends after 0.1 or 0.2 s, the kernel goes on to its end, and the context stays usable."""
import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

# 32 chunks of 64 tokens and one tile: a cluster of several blocks, in two steps or more
CHILD = r"""
import sys
import torch
from mamba_ssd_selective_gb300 import binding as ops
assert ops.lib_path().endswith("libssdscan_dbg.so")
TILES, RUNS = 1, 2


def data(io, D, L=2000, B=1):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(D)
    t = {n: torch.randn(B, L, D, generator=gen, device="cuda").to(io) for n in ("x", "r", "i", "dy")}
    t.update(lam=torch.full((D,), -5.0, device="cuda"), init=torch.randn(B, D, generator=gen, device="cuda"))
    return t


def forward(t):
    kept = ops.gated_linear_checkpoint(t["x"])
    y, final = ops.gated_linear_chunked(t["x"], t["r"], t["i"], t["lam"], init_state=t["init"], **kept)
    plain, _ = ops.gated_linear_chunked(t["x"], t["r"], t["i"], t["lam"], init_state=t["init"])
    return dict(kept, y=y, final=final, plain=plain)


def backward(t, kept):
    g = ops.gated_linear_chunked_bwd(t["x"], t["r"], t["i"], t["lam"], t["dy"], states=kept["states"])
    p = ops.gated_linear_chunked_bwd_packed(kept["values"], kept["scales"], kept["states"], t["lam"], t["dy"])
    return dict(g, **{"packed_" + n: v for n, v in p.items()})


def same(a, b):
    return all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in a)


CASES = [(torch.bfloat16, 64, TILES), (torch.bfloat16, 64, RUNS), (torch.float32, 64, TILES), (torch.bfloat16, 33, RUNS), (torch.bfloat16, 66, RUNS)]
"""

ENDS = CHILD + r"""
for io, D, what in CASES:
    t = data(io, D)
    want = forward(t)
    grads = backward(t, want)
    assert ops.gated_linear_status() == ops.SSD_OK
    for rank in (0, 1):
        for step in (0, 1):
            ops.ssd_debug_linear_withhold(what, rank, step)
            got = forward(t)
            torch.cuda.synchronize()
            assert ops.gated_linear_status() == ops.SSD_ERR_TIMEOUT, (io, D, what, rank, step)
            assert ops.gated_linear_status() == ops.SSD_OK
            if step > 0 or rank > 0:  # the first block's tokens before that
                for n in ("y", "plain"):
                    assert torch.equal(got[n][:, :64], want[n][:, :64]), (io, D, what, rank, step, n)
            backward(t, want)
            torch.cuda.synchronize()
            assert ops.gated_linear_status() == ops.SSD_ERR_TIMEOUT, (io, D, what, rank, step)
            ops.ssd_debug_linear_withhold(0)
            again = forward(t)
            assert same(again, want) and same(backward(t, again), grads)
            assert ops.gated_linear_status() == ops.SSD_OK
print("ok")
"""


TOLD = CHILD + r"""
import threading
t = data(torch.bfloat16, 64)
streams = [torch.cuda.Stream() for _ in range(3)]
TIMEOUT, OK = ops.SSD_ERR_TIMEOUT, ops.SSD_OK
for again in range(2):
    assert [ops.gated_linear_status(s) for s in (None, *streams)] == [OK] * 4
    ops.ssd_debug_linear_withhold(RUNS, 1, 0)
    ops.gated_linear_chunked(t["x"], t["r"], t["i"], t["lam"], stream=streams[1])
    ops.ssd_debug_linear_withhold(0)
    torch.cuda.synchronize()
    # others ask first, more than once, and from another thread
    assert ops.gated_linear_status(streams[0]) == TIMEOUT and ops.gated_linear_status(streams[0]) == OK
    said = []
    thread = threading.Thread(target=lambda: said.extend(ops.gated_linear_status(s) for s in (streams[2], streams[2], None)))
    thread.start()
    thread.join()
    assert said == [TIMEOUT, OK, TIMEOUT], said
    assert ops.gated_linear_status(streams[1]) == TIMEOUT
print("ok")
"""

LOST = CHILD + r"""
def right_or_nan(got, want, what):
    got, want = got.float(), want.float()
    assert ((got == want) | torch.isnan(got)).all(), what


def right_or_lost(got, want, what):  # in 8 bits
    lost = (got["scales"] == 255)
    kept = ~lost.repeat_interleave(16, 2)[:, :, :got["values"].shape[2]]
    assert torch.equal(got["scales"][~lost], want["scales"][~lost]) and torch.equal(got["values"][kept], want["values"][kept]), what
    assert not got["values"][~kept].any(), what


for io, D, what in CASES:
    t = data(io, D)
    want = forward(t)
    grads = backward(t, want)
    L = t["x"].shape[1]
    for rank in (0, 1, 2):
        for step in (0, 1):
            case = (io, D, what, rank, step)
            ops.ssd_debug_linear_withhold(what, rank, step)
            got = forward(t)
            g = backward(t, want)
            ops.ssd_debug_linear_withhold(0)
            for n in ("y", "plain", "states", "final"):
                right_or_nan(got[n], want[n], (*case, n))
            right_or_lost(got, want, case)
            for n in g:
                right_or_nan(g[n], grads[n], (*case, n))
                assert n.endswith("dinit") or torch.isnan(g[n].float()).any(), (*case, n)
            if step > 0:
                continue
            # from the block whose wait ran out; all of the others' where its run was not known, else from the next step on
            first = 64 * rank
            lost = slice(first, None) if what == TILES else slice(first, min(first + 64, L))
            for n in ("y", "plain"):
                assert torch.isnan(got[n][:, lost]).all() and torch.isnan(got[n][:, -1]).all(), (*case, n)
                assert torch.equal(got[n][:, :first], want[n][:, :first]), (*case, n)
            assert torch.isnan(got["final"]).all(), case
            if what == TILES:
                assert torch.isnan(got["states"][:, rank:]).all() and (got["scales"][:, :, first // 16:first // 16 + 4] == 255).all(), case
                for n in ("dx", "dr", "di", "dlam", "dinit", "packed_dx", "packed_dlam", "packed_dinit"):
                    assert torch.isnan(g[n][:, 0] if g[n].dim() == 3 else g[n]).all(), (*case, n)
assert ops.gated_linear_status() == ops.SSD_ERR_TIMEOUT
print("ok")
"""


@pytest.fixture(scope="module")
def debug_library(cuda_device):
    from mamba_ssd_selective_gb300 import build
    return build.build(debug_bounds=True)


def run(child):
    r = subprocess.run([sys.executable, "-c", child], capture_output=True, text=True, cwd=ROOT, timeout=300,
                       env=dict(os.environ, SSD_DEBUG_BOUNDS_LIB="1"))
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-3000:]


def test_a_kernel_whose_wait_runs_out_ends_and_leaves_the_rest_as_it_was(debug_library):
    run(ENDS)


def test_what_is_not_known_is_nan(debug_library):
    """Every number is right or NaN (scale 255 in 8 bits), and what hangs on tiles that did not come is NaN."""
    run(LOST)


def test_every_stream_that_asks_is_told(debug_library):
    run(TOLD)
