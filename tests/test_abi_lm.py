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


def test_distill_refusals(lib):
    def args(R=4, V=100, k=8, io=nb.BF16, logits=FAKE, ld=None, ids=FAKE, t=FAKE, tau=1.0):
        return (R, V, k, io, logits, V if ld is None else ld, ids, t, tau)

    def fwd(loss=FAKE, lse=FAKE, **kw):
        return lib.naju_distill_fwd(*args(**kw), loss, lse, None)

    def bwd(lse=FAKE, g=FAKE, d=FAKE, ldd=100, **kw):
        return lib.naju_distill_bwd(*args(**kw), lse, g, d, ldd, None)

    def both(g=FAKE, loss=FAKE, lse=FAKE, d=FAKE, ldd=100, **kw):
        return lib.naju_distill_fwd_bwd(*args(**kw), g, loss, lse, d, ldd, None)
    for call in (fwd, bwd, both):
        expect(call(R=-1), nb.EINVAL, "negative size")
        expect(call(k=-1), nb.EINVAL, "negative size")
        expect(call(io=3), nb.EINVAL, "io dtype")
        expect(call(k=513), nb.EUNSUPPORTED, "teacher entries")
        for tau in (0.0, -1.0, float("nan"), float("inf")):
            expect(call(tau=tau), nb.EINVAL, "temperature")
        expect(call(ld=99), nb.EINVAL, "row stride of logits")
        expect(call(V=2 ** 31), nb.EINVAL, "too large")
        expect(call(logits=None), nb.EINVAL, "logits is NULL")
        expect(call(logits=FAKE + 1), nb.EINVAL, "aligned")
        expect(call(ids=None), nb.EINVAL, "t_ids is NULL")
        expect(call(t=None), nb.EINVAL, "t_logits is NULL")
        expect(call(lse=None), nb.EINVAL, "lse is NULL")
        assert call(R=0, logits=None, ids=None, t=None) == nb.OK
        assert call(V=0, logits=None, ids=None, t=None) == nb.OK
    expect(fwd(loss=None), nb.EINVAL, "loss is NULL")
    for call in (bwd, both):
        expect(call(g=None), nb.EINVAL, "g is NULL")
        expect(call(d=None), nb.EINVAL, "dlogits is NULL")
        expect(call(ldd=99), nb.EINVAL, "row stride of dlogits")


def test_logits_refusals(lib):
    def call(R=4, V=100, io=nb.BF16, logits=FAKE, ld=100, hist=FAKE, H=10, lengths=None, rep=None,
             pres=None, freq=None, ids=FAKE, bias=FAKE, n=3, mask=None, out=FAKE, best=FAKE,
             ws=FAKE, wsb=1 << 30):
        return lib.naju_logits_process(R, V, io, logits, ld, hist, H, lengths, rep, pres, freq,
                                       ids, bias, n, mask, out, best, ws, wsb, None)
    expect(call(R=-1), nb.EINVAL, "negative size")
    expect(call(H=-1), nb.EINVAL, "negative size")
    expect(call(n=-1), nb.EINVAL, "negative size")
    expect(call(R=2 ** 25), nb.EINVAL, "too large")
    expect(call(io=4), nb.EINVAL, "io dtype")
    expect(call(H=2 ** 20), nb.EUNSUPPORTED, "history_len")
    expect(call(n=4095), nb.EUNSUPPORTED, "n_bias")
    expect(call(ld=99), nb.EINVAL, "row stride")
    expect(call(logits=None), nb.EINVAL, "logits is NULL")
    expect(call(out=None), nb.EINVAL, "out is NULL")
    expect(call(hist=None), nb.EINVAL, "history is NULL")
    expect(call(ids=None), nb.EINVAL, "bias_ids is NULL")
    expect(call(bias=None), nb.EINVAL, "bias is NULL")
    for name in ("lengths", "rep", "pres", "freq", "mask"):
        expect(call(**{name: FAKE + 2}), nb.EINVAL, "aligned")
    expect(call(best=FAKE + 2), nb.EINVAL, "best is not")
    expect(call(ws=None), nb.EWORKSPACE, "workspace is NULL")
    expect(call(wsb=16), nb.EWORKSPACE, "needs")
    assert call(R=0, logits=None, out=None, ws=None) == nb.OK
    assert lib.naju_logits_workspace_bytes(100) >= 1600
    assert lib.naju_logits_workspace_bytes(-1) == 0


def test_w4_refusals(lib):
    def lin(R=2, K=64, N=10, G=32, x=FAKE, q=FAKE, s=FAKE, z=None, bias=None, res=None, y=FAKE):
        return lib.naju_w4_linear(R, K, N, G, x, q, s, z, bias, res, y, None)

    def quant(K=64, N=10, G=32, io=nb.F32, W=FAKE, q=FAKE, s=FAKE, z=None):
        return lib.naju_w4_quantize(K, N, G, io, W, q, s, z, None)
    for call in (lin, quant):
        expect(call(K=-2), nb.EINVAL, "negative size")
        expect(call(K=63), nb.EUNSUPPORTED, "odd")
        expect(call(G=16), nb.EUNSUPPORTED, "group")
        expect(call(N=2 ** 27), nb.EINVAL, "too large")
        expect(call(q=None), nb.EINVAL, "qweight is NULL")
        expect(call(s=FAKE + 1), nb.EINVAL, "aligned")
        assert call(N=0, q=None, s=None) == nb.OK
    expect(lin(R=-1), nb.EINVAL, "negative size")
    expect(lin(R=2 ** 21), nb.EINVAL, "too large")
    expect(lin(x=None), nb.EINVAL, "x is NULL")
    expect(lin(y=None), nb.EINVAL, "y is NULL")
    expect(lin(bias=FAKE + 2), nb.EINVAL, "aligned")
    expect(lin(res=FAKE + 1), nb.EINVAL, "aligned")
    expect(quant(io=5), nb.EINVAL, "io dtype")
    expect(quant(W=None), nb.EINVAL, "W is NULL")
    assert lin(R=0, x=None, y=None) == nb.OK
    assert quant(K=0, W=None) == nb.OK


def test_binding_refuses_tensors_in_host_memory(lib):
    import torch
    ids, W = torch.zeros(3, dtype=torch.int32), torch.zeros(5, 8)
    x, t = torch.zeros(3, 5), torch.zeros(3, 2)
    t_ids, g = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3)
    q, s = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.bfloat16)
    for call in (lambda: nb.embed_fwd(ids, W), lambda: nb.embed_bwd(ids, torch.zeros(3, 8), 5),
                 lambda: nb.distill_fwd(x, t_ids, t), lambda: nb.distill_fwd_bwd(x, t_ids, t, g),
                 lambda: nb.distill_bwd(x, t_ids, t, g, g), lambda: nb.logits_process(x),
                 lambda: nb.w4_linear(torch.zeros(2, 32, dtype=torch.bfloat16), q, s, 32),
                 lambda: nb.w4_quantize(W)):
        with pytest.raises(ValueError, match="GPU"):
            call()
