"""CPU checks of the strides that one token a row may have (no call here touches a GPU): the limit on
the distance of a chunk's tokens is none on the distance of the batch's rows."""
import pytest

from selective_state_space_naju_amd import binding as nb

FAKE = 0x100000  # a 256-byte aligned non-null address; never dereferenced


def fwd(L, ldq=256, ldk=128, ldv=64, a=None):
    return nb.lib().naju_linattn_fwd(2, L, 4, 2, 64, 32, nb.BF16, FAKE, ldq, FAKE, ldk, FAKE, ldv,
                                     a, None, None, 1.0, FAKE, None, FAKE, 1 << 40, None)


def bwd(L, ldq=256, ldk=128, ldv=64, a=None):
    return nb.lib().naju_linattn_bwd(2, L, 4, 2, 64, 32, nb.BF16, FAKE, ldq, FAKE, ldk, FAKE, ldv,
                                     a, None, None, 1.0, FAKE, None, FAKE, FAKE, FAKE, None, FAKE,
                                     1 << 40, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("name", ["ldq", "ldk", "ldv"])
def test_distance_of_rows(call, name):
    for ld in ((1 << 20) + 8, 2048000, 1 << 32, 1 << 40):
        # (the strides are looked at before log_decay, which is missing)
        assert call(1, **{name: ld}) == nb.EINVAL and "log_decay" in nb.last_error()
        assert call(2, **{name: ld}) == nb.EINVAL and "token stride of " + name[2:] in \
            nb.last_error()
    for ld in ((1 << 40) + 8, 2048001, 8):
        assert call(1, **{name: ld}) == nb.EINVAL and "token stride of " + name[2:] in \
            nb.last_error()
