"""Calls of the gated linear recurrence and of values in 8 bits that are refused before any CUDA call."""
import ctypes

import pytest

from mamba_ssd_selective_gb300 import binding
from mamba_ssd_selective_gb300 import build as nvbuild


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return binding.load()


def test_no_wait_is_made_to_run_out_in_a_release_build(lib):
    assert lib.ssd_debug_linear_withhold(0, 0, 0) == binding.SSD_ERR_UNSUPPORTED
    for bad in ((3, 0, 0), (1, -1, 0), (1, 0, -1)):
        assert lib.ssd_debug_linear_withhold(*bad) == binding.SSD_ERR_INVALID_ARG
    with pytest.raises(binding.SsdError):
        binding.ssd_debug_linear_withhold(1)


# -------------------------------------- results that share memory with something
# name -> elements and bytes of each, in the order of the call, at B = 3, L = 70, D = 48 and bf16 (a pool of 5 states)

B, L, D, S = 3, 70, 48, 5
TOK, STATE, STATES, VALUES, SCALES, LAM, LENS = 2 * B * L * D, 4 * B * D, 4 * B * 2 * D, 3 * B * L * D, 3 * B * 5 * D, 4 * D, 4 * B
WS = 9472  # ssd_gated_linear_chunked_bwd_workspace_size with states
CALLS = dict(
    chunked=(dict(x=TOK, r=TOK, i=TOK, lam=LAM, init_state=STATE, seqlens=LENS),
             dict(y=TOK, final_state=STATE, states=STATES, values=VALUES, scales=SCALES)),
    bwd=(dict(x=TOK, r=TOK, i=TOK, lam=LAM, states=STATES, seqlens=LENS, dy=TOK, dfinal_state=STATE),
         dict(dx=TOK, dr=TOK, di=TOK, dlam=LAM, dinit_state=STATE, workspace=WS)),
    bwd_packed=(dict(values=VALUES, scales=SCALES, lam=LAM, states=STATES, seqlens=LENS, dy=TOK, dfinal_state=STATE),
                dict(dx=TOK, dr=TOK, di=TOK, dlam=LAM, dinit_state=STATE, workspace=WS)),
    step=(dict(state=4 * S * D, x=2 * B * D, r=2 * B * D, i=2 * B * D, lam=LAM, slots=LENS), dict(new_state=4 * S * D, y=2 * B * D)),
    pack8=(dict(x=TOK, seqlens=LENS), dict(values=TOK // 2, scales=SCALES // 3)),
    unpack8=(dict(values=TOK // 2, scales=SCALES // 3), dict(out=TOK)))
IN_PLACE = {("chunked", "final_state", "init_state"), ("bwd", "dinit_state", "dfinal_state"), ("bwd_packed", "dinit_state", "dfinal_state"),
            ("step", "new_state", "state"), ("step", "y", "x"), ("step", "y", "r"), ("step", "y", "i")}


def call(lib, name, at):
    p = {n: ctypes.c_void_p(a) for n, a in at.items()}
    get = lambda *names: [p[n] for n in names]  # noqa: E731
    if name == "chunked":
        return lib.ssd_gated_linear_chunked(B, L, D, 1, *get("x", "r", "i", "lam"), 8.0,
                                            *get("init_state", "seqlens", "y", "final_state", "states", "values", "scales"), None)
    out = ("dx", "dr", "di", "dlam", "dinit_state", "workspace")
    if name == "bwd":
        return lib.ssd_gated_linear_chunked_bwd(B, L, D, 1, *get("x", "r", "i", "lam"), 8.0, None,
                                                *get("states", "seqlens", "dy", "dfinal_state", *out), WS, None)
    if name == "bwd_packed":
        return lib.ssd_gated_linear_chunked_bwd_packed(B, L, D, 1, *get("values", "scales", "lam"), 8.0,
                                                       *get("states", "seqlens", "dy", "dfinal_state", *out), WS, None)
    if name == "step":
        return lib.ssd_gated_linear_step(B, D, 1, S, *get("state", "x", "r", "i", "lam"), 8.0, *get("slots", "new_state", "y"), None)
    if name == "pack8":
        return lib.ssd_pack8(B, L, D, 1, *get("x", "seqlens", "values", "scales"), None)
    return lib.ssd_unpack8(B, L, D, 1, *get("values", "scales", "out"), None)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_results_that_share_memory_are_refused(lib, name):
    """Every result over every other buffer of the call: at its start, and by its last and first 16 bytes (a workspace: by 256)."""
    assert WS == lib.ssd_gated_linear_chunked_bwd_workspace_size(B, L, D, 1, 1)
    inputs, results = CALLS[name]
    sizes = {**inputs, **results}
    apart = {n: (k + 1) << 24 for k, n in enumerate(sizes)}
    for n in results:
        for m in sizes:
            if m == n:
                continue
            spots = [apart[m], apart[m] + (sizes[m] - 1) // 16 * 16, apart[m] - (sizes[n] - 1) // 16 * 16]
            if n == "workspace":
                spots = [apart[m], apart[m] + (sizes[m] - 1) // 256 * 256, apart[m] - (sizes[n] - 256)]
            for k, at in enumerate(spots):
                if k == 0 and (name, n, m) in IN_PLACE:
                    continue
                assert call(lib, name, {**apart, n: at}) == binding.SSD_ERR_INVALID_ARG, (n, m, k)
                assert b"shares memory" in lib.ssd_last_error(), (n, m, k, lib.ssd_last_error())
