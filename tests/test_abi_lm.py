"""CPU checks of the entry points around the mixer layer: argument validation
through the C ABI (no call here touches a GPU)."""
import os

import pytest

from selective_state_space_naju_amd import binding as nb

FAKE = 0x100000  # a 256-byte aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nb.LIB_PATH):
        pytest.fail("libnaju.so is not built (run __graft_entry__.build())")
    return nb.lib()


def expect(status, want, text=""):
    assert status == want, nb.last_error()
    assert text in nb.last_error(), nb.last_error()


def test_embed_fwd_refusals(lib):
    def call(T=10, V=50, d=64, io=nb.BF16, ids=FAKE, W=FAKE, out=FAKE):
        return lib.naju_embed_fwd(T, V, d, io, ids, W, 1.0, out, None)
    expect(call(T=-1), nb.EINVAL, "negative size")
    expect(call(io=9), nb.EINVAL, "io dtype")
    expect(call(T=2 ** 29), nb.EINVAL, "too large")
    expect(call(V=2 ** 31), nb.EINVAL, "too large")
    expect(call(d=2 ** 21), nb.EINVAL, "too large")
    expect(call(ids=None), nb.EINVAL, "ids is NULL")
    expect(call(ids=FAKE + 2), nb.EINVAL, "aligned")
    expect(call(W=None), nb.EINVAL, "W is NULL")
    expect(call(out=FAKE + 1), nb.EINVAL, "aligned")
    assert call(T=0, ids=None, W=None, out=None) == nb.OK
    assert call(d=0, ids=None, W=None, out=None) == nb.OK


def test_embed_bwd_refusals(lib):
    def call(T=10, V=50, d=64, io=nb.BF16, ids=FAKE, dout=FAKE, acc=0, dW=FAKE, ws=FAKE,
             wsb=1 << 40):
        return lib.naju_embed_bwd(T, V, d, io, ids, dout, 1.0, acc, dW, ws, wsb, None)
    expect(call(d=-1), nb.EINVAL, "negative size")
    expect(call(io=2), nb.EINVAL, "io dtype")
    expect(call(T=2 ** 29), nb.EINVAL, "too large")
    expect(call(ids=None), nb.EINVAL, "ids is NULL")
    expect(call(dout=None), nb.EINVAL, "dout is NULL")
    expect(call(dW=None), nb.EINVAL, "dW is NULL")
    expect(call(dW=FAKE + 2), nb.EINVAL, "aligned")
    expect(call(ws=None), nb.EWORKSPACE, "workspace is NULL")
    expect(call(ws=FAKE + 16), nb.EINVAL, "256-byte")
    expect(call(wsb=64), nb.EWORKSPACE, "needs")
    assert call(V=0, ids=None, dout=None, dW=None, ws=None) == nb.OK
    assert call(T=0, acc=1, ids=None, dout=None, ws=None) == nb.OK
    size = lib.naju_embed_bwd_workspace_bytes
    assert size(16384, 50000, 768) >= 4 * 4 * 16384
    assert size(-1, 5, 5) == 0 and size(2 ** 29, 5, 5) == 0
    assert size(2 ** 28, 2 ** 30, 2 ** 20) > 2 ** 40  # no overflow at the limits
