"""CPU check of the distillation's smallest temperatures (no call here touches a GPU)."""
import os

import pytest

from selective_state_space_naju_amd import binding as nb

FAKE = 0x100000  # a 256-byte aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nb.LIB_PATH):
        pytest.fail("libnaju.so is not built (run __graft_entry__.build())")
    return nb.lib()


@pytest.mark.parametrize("tau", [1e-45, 1e-39, 4e-39])
def test_temperatures_without_a_finite_reciprocal_are_refused(lib, tau):
    args = (4, 100, 8, nb.BF16, FAKE, 100, FAKE, FAKE, tau)
    for status in (lib.naju_distill_fwd(*args, FAKE, FAKE, None),
                   lib.naju_distill_bwd(*args, FAKE, FAKE, FAKE, 100, None),
                   lib.naju_distill_fwd_bwd(*args, FAKE, FAKE, FAKE, FAKE, 100, None)):
        assert status == nb.EINVAL and "temperature" in nb.last_error()


def test_the_smallest_temperatures_with_one_are_taken(lib):
    args = (0, 100, 8, nb.BF16, None, 100, None, None)  # no rows: nothing is launched
    for tau in (5e-39, 1e-30, 3e38):
        assert lib.naju_distill_fwd(*args, tau, None, None, None) == nb.OK
