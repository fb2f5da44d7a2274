"""Calls of the gated linear recurrence and of values in 8 bits that are refused before any CUDA call."""
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
