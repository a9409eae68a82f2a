"""CPU checks of the entry points of the rest of a layer: argument validation
through the C ABI and the binding (no call here touches a GPU), and pins of
their fp64 definitions."""
import os

import numpy as np
import pytest
import torch

from oracle import layer
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


def test_res_norm_fwd_refusals(lib):
    def call(T=10, d=64, io=nb.BF16, xio=nb.F32, x=FAKE, y=FAKE, z=FAKE, s=FAKE, wo=FAKE, wi=FAKE,
             eps=1e-6, new=FAKE, xn=FAKE):
        return lib.naju_res_norm_fwd(T, d, io, xio, x, y, z, s, wo, wi, eps, new, xn, None)
    expect(call(T=-1), nb.EINVAL, "negative size")
    expect(call(T=2 ** 41), nb.EINVAL, "too large")
    expect(call(io=3), nb.EINVAL, "io dtype")
    expect(call(xio=7), nb.EINVAL, "io dtype")
    expect(call(io=nb.F32, xio=nb.BF16), nb.EUNSUPPORTED, "fp32")
    for d in (1, 3, 8193):
        expect(call(d=d), nb.EUNSUPPORTED, "d_model")
    for eps in (-1.0, float("nan"), float("inf")):
        expect(call(eps=eps), nb.EINVAL, "eps")
    expect(call(x=None), nb.EINVAL, "x is NULL")
    expect(call(x=FAKE + 2), nb.EINVAL, "aligned")
    expect(call(y=None, new=None), nb.EINVAL, "need y")
    expect(call(new=None), nb.EINVAL, "go together")
    expect(call(xn=None), nb.EINVAL, "go together")
    expect(call(y=FAKE + 1), nb.EINVAL, "aligned")
    expect(call(s=FAKE + 2), nb.EINVAL, "aligned")
    expect(call(y=None, z=None, s=None, wo=None, wi=None, new=None, xn=None), nb.EINVAL,
           "nothing to compute")
    assert call(T=0, x=None) == nb.OK
    assert call(d=0, x=None) == nb.OK


def test_res_norm_bwd_refusals(lib):
    def call(T=10, d=64, io=nb.BF16, xio=nb.F32, gio=nb.F32, dxn=FAKE, dnew=FAKE, x=FAKE, y=FAKE,
             z=FAKE, s=FAKE, wo=FAKE, wi=FAKE, eps=1e-6, dx=FAKE, dy=FAKE, dz=FAKE, ds=FAKE,
             dwo=FAKE, dwi=FAKE, ws=FAKE, wsb=1 << 40):
        return lib.naju_res_norm_bwd(T, d, io, xio, gio, dxn, dnew, x, y, z, s, wo, wi, eps, dx,
                                     dy, dz, ds, dwo, dwi, ws, wsb, None)
    expect(call(d=-1), nb.EINVAL, "negative size")
    expect(call(gio=2), nb.EINVAL, "io dtype")
    expect(call(io=nb.F32, gio=nb.BF16), nb.EUNSUPPORTED, "fp32")
    expect(call(d=2), nb.EUNSUPPORTED, "d_model")
    expect(call(dxn=None), nb.EINVAL, "go together")
    expect(call(dxn=None, wi=None, dwi=None, dnew=None), nb.EINVAL, "no gradient")
    expect(call(s=None), nb.EINVAL, "dscale needs")
    expect(call(wo=None), nb.EINVAL, "dw_post needs")
    expect(call(wi=None, dxn=None), nb.EINVAL, "dw_pre needs")
    expect(call(x=None), nb.EINVAL, "x_new is NULL")
    for k in ("dx", "dy", "dz"):
        expect(call(**{k: None}), nb.EINVAL, k + " is NULL")
        expect(call(**{k: FAKE + 1}), nb.EINVAL, "aligned")
    expect(call(ws=None), nb.EWORKSPACE, "workspace is NULL")
    expect(call(wsb=64), nb.EWORKSPACE, "needs")
    expect(call(ws=FAKE + 16), nb.EINVAL, "256-byte")
    assert call(d=0, ws=None) == nb.OK
    assert call(T=0, ds=None, dwo=None, dwi=None, dxn=None, dnew=None, ws=None) == nb.OK
    size = lib.naju_res_norm_bwd_workspace_bytes
    assert size(16384, 768) >= 512 * 3 * 768 * 4
    assert size(-1, 768) == 0 and size(10, 3) == 0


def test_binding_refuses_what_does_not_fit(lib):
    x, w = torch.zeros(3, 8), torch.ones(8)
    with pytest.raises(ValueError, match="GPU"):
        nb.res_norm_fwd(x, w_pre=w)
    with pytest.raises(ValueError, match="GPU"):
        nb.res_norm_bwd(x, None, x, w_pre=w)


# ------------------------------------------------------------- pins of the definitions
def test_norm_definitions():
    """A norm without weight brings any row to unit mean square; the gradient of a norm is
    perpendicular to its input where eps is 0; SiLU(0) = 0 leaves the residual."""
    rng = np.random.default_rng(1)
    x, y, d = rng.standard_normal((3, 4, 50))
    new, xn = layer.res_norm_fwd(x, y, np.zeros_like(y), w_pre=np.ones(50), eps=0.0)
    assert np.array_equal(new, x)
    assert np.allclose((xn * xn).mean(1), 1.0, rtol=1e-12)
    g = layer.res_norm_bwd(d, None, x, w_pre=np.ones(50), eps=0.0)
    assert np.abs((g["dx"] * x).sum(1)).max() < 1e-12
    assert np.allclose(g["dw_pre"], (d * xn).sum(0))


def test_adamw_refusals(lib):
    def tensor(**kw):
        t = dict(n=1000, p=FAKE, g=FAKE * 2, m=FAKE * 3, v=FAKE * 4, m_scale=FAKE * 5,
                 v_scale=FAKE * 6)
        t.update(kw)
        return nb.AdamwTensor(**{k: v for k, v in t.items() if v is not None})

    def call(*ts, n=None, io=nb.F32, bits=32, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1, step=1,
             step_dev=None, lr_dev=None, gs=None):
        table = (nb.AdamwTensor * max(1, len(ts)))(*ts)
        return lib.naju_adamw_step(len(ts) if n is None else n, table, io, bits, lr, b1, b2, eps,
                                   wd, step, step_dev, lr_dev, gs, None)
    expect(call(n=-1), nb.EINVAL, "negative size")
    expect(call(n=2 ** 25), nb.EINVAL, "too large")
    expect(call(tensor(), io=5), nb.EINVAL, "io dtype")
    expect(call(tensor(), bits=16), nb.EUNSUPPORTED, "state_bits")
    for kw in (dict(b1=1.0), dict(b2=-0.1), dict(b1=float("nan"))):
        expect(call(tensor(), **kw), nb.EINVAL, "beta")
    expect(call(tensor(), eps=-1.0), nb.EINVAL, "eps")
    expect(call(tensor(), lr=float("inf")), nb.EINVAL, "lr")
    expect(call(tensor(), wd=float("nan")), nb.EINVAL, "weight_decay")
    expect(call(tensor(), step=0), nb.EINVAL, "steps count from 1")
    for k in ("step_dev", "lr_dev", "gs"):
        expect(call(tensor(), **{k: FAKE + 2}), nb.EINVAL, "aligned")
    for k in ("p", "g", "m", "v"):
        expect(call(tensor(**{k: None})), nb.EINVAL, k + " is NULL")
        expect(call(tensor(**{k: FAKE + 2})), nb.EINVAL, "aligned")
    expect(call(tensor(n=-1)), nb.EINVAL, "elements")
    expect(call(tensor(n=2 ** 43)), nb.EINVAL, "elements")
    expect(call(tensor(m_scale=None), bits=8), nb.EINVAL, "m_scale is NULL")
    expect(call(tensor(copy=FAKE + 1)), nb.EINVAL, "aligned")
    # the same parameter twice, and two that overlap by one element
    expect(call(tensor(), tensor()), nb.EINVAL, "overlap")
    expect(call(tensor(p=FAKE + 4 * 999), tensor(p=2 * FAKE + 64), tensor()), nb.EINVAL, "overlap")
    assert call() == nb.OK
    assert call(tensor(n=0, p=None, g=None, m=None, v=None)) == nb.OK


def test_adamw_binding_refusals(lib):
    p = [torch.zeros(5)]
    with pytest.raises(ValueError, match="GPU"):
        nb.adamw_step(p, p, p, p, 1, 1e-3)
    nb.adamw_step([], [], [], [], 1, 1e-3)


def test_adamw_definition():
    """One step from zero states moves every parameter by lr against its gradient's sign; zero
    gradients leave weight decay alone; the 8-bit type's values."""
    p, g = np.array([1.0, 2.0, 3.0]), np.array([0.5, -2.0, 1e-3])
    q, m, v = layer.adamw(p, g, 0 * p, 0 * p, 1, 0.1, weight_decay=0.0, eps=0.0)
    assert np.allclose(q, p - 0.1 * np.sign(g), rtol=1e-12)
    q, _, _ = layer.adamw(p, 0 * g, 0 * p, 0 * p, 3, 0.1, weight_decay=0.5)
    assert np.allclose(q, p * 0.95)
    vals = layer.e4m3_values()
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(vals, t) and vals[-1] == 448


def lin_args(B=2, L=100, H=4, Hk=2, dk=64, dv=32, io=nb.BF16, q=FAKE, ldq=256, k=FAKE, ldk=128,
             v=FAKE, ldv=64, a=FAKE, state=None, lengths=None, scale=0.125):
    return (B, L, H, Hk, dk, dv, io, q, ldq, k, ldk, v, ldv, a, state, lengths, scale)


def test_linattn_refusals(lib):
    def fwd(o=FAKE, so=FAKE, ws=FAKE, wsb=1 << 40, **kw):
        return lib.naju_linattn_fwd(*lin_args(**kw), o, so, ws, wsb, None)

    def bwd(do=FAKE, ds=None, dq=FAKE, dk_=FAKE, dv_=FAKE, dst=FAKE, ws=FAKE, wsb=1 << 40, **kw):
        return lib.naju_linattn_bwd(*lin_args(**kw), do, ds, dq, dk_, dv_, dst, ws, wsb, None)
    for call in (fwd, bwd):
        expect(call(B=-1), nb.EINVAL, "negative size")
        expect(call(L=-1), nb.EINVAL, "negative size")
        expect(call(io=2), nb.EINVAL, "io dtype")
        expect(call(Hk=3), nb.EINVAL, "no multiple")
        expect(call(Hk=0), nb.EINVAL, "no multiple")
        for d in (0, 4, 20, 264):
            expect(call(dk=d), nb.EUNSUPPORTED, "multiples of 8")
            expect(call(dv=d), nb.EUNSUPPORTED, "multiples of 8")
        expect(call(L=2 ** 31), nb.EINVAL, "too large")
        expect(call(B=2 ** 21), nb.EINVAL, "too large")
        expect(call(scale=float("nan")), nb.EINVAL, "scale")
        expect(call(ldq=248), nb.EINVAL, "token stride of q")
        expect(call(ldk=132), nb.EINVAL, "token stride of k")
        expect(call(ldv=56), nb.EINVAL, "token stride of v")
        for name in ("q", "k", "v"):
            expect(call(**{name: None}), nb.EINVAL, name + " is NULL")
            expect(call(**{name: FAKE + 8}), nb.EINVAL, "aligned")
        expect(call(a=None), nb.EINVAL, "log_decay is NULL")
        expect(call(lengths=FAKE + 2), nb.EINVAL, "aligned")
        expect(call(state=FAKE + 2), nb.EINVAL, "aligned")
        assert call(B=0, q=None) == nb.OK
        assert call(H=0, Hk=0, q=None) == nb.OK
        # a long sequence of few heads is cut, and needs the workspace
        expect(call(L=65536, ws=None), nb.EWORKSPACE, "workspace is NULL")
        expect(call(L=65536, wsb=256), nb.EWORKSPACE, "needs")
    expect(fwd(o=None), nb.EINVAL, "o is NULL")
    expect(bwd(dq=None), nb.EINVAL, "dq is NULL")
    expect(bwd(dv_=FAKE + 4), nb.EINVAL, "aligned")
    expect(bwd(do=None), nb.EINVAL, "dout is NULL")
    expect(bwd(wsb=64), nb.EWORKSPACE, "needs")  # (shared heads)
    f, g = lib.naju_linattn_fwd_workspace_bytes, lib.naju_linattn_bwd_workspace_bytes
    assert f(8, 64, 96, 96, 128, 128) == 0 and f(1, 65536, 16, 16, 128, 128) >= 16 * 65536
    assert g(2, 100, 4, 2, 64, 32) >= 2 * 100 * 4 * (64 + 32) * 4
    assert f(-1, 1, 1, 1, 8, 8) == 0 and g(1, 1, 1, 1, 9, 8) == 0


def test_linattn_step_refusals(lib):
    def call(B=2, H=4, Hk=2, dk=64, dv=32, io=nb.BF16, q=FAKE, k=FAKE, v=FAKE, a=FAKE, s=FAKE,
             scale=1.0, o=FAKE, so=FAKE):
        return lib.naju_linattn_step(B, H, Hk, dk, dv, io, q, k, v, a, s, scale, o, so, None)
    expect(call(B=-1), nb.EINVAL, "negative size")
    expect(call(dk=12), nb.EUNSUPPORTED, "multiples of 8")
    expect(call(Hk=3), nb.EINVAL, "no multiple")
    expect(call(s=None), nb.EINVAL, "state is NULL")
    expect(call(s=FAKE + 8), nb.EINVAL, "aligned")
    expect(call(so=None), nb.EINVAL, "state_out is NULL")
    expect(call(o=FAKE + 1), nb.EINVAL, "aligned")
    assert call(B=0, q=None, s=None) == nb.OK


def test_linattn_binding_refusals(lib):
    q, a = torch.zeros(2, 5, 4, 16), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        nb.linattn_fwd(q, q, q, a)
    with pytest.raises(ValueError, match="GPU"):
        nb.linattn_bwd(q, q, q, a, q)
    with pytest.raises(ValueError, match="GPU"):
        nb.linattn_step(q[0], q[0], q[0], a, torch.zeros(5, 4, 16, 16))
    # strides: parts of a joint projection pass, other orders do not
    joint = torch.zeros(2, 5, 3, 4, 16)
    assert nb._req_tokens(joint[:, :, 1], "q", (2, 5, 4, 16), q.dtype, q.device) == 192
    assert nb._req_tokens(joint[:, :1, 1], "q", (2, 1, 4, 16), q.dtype, q.device) == 960
    for bad in (q.transpose(1, 2).contiguous().transpose(1, 2), joint[:, ::2, 0],
                joint[:, :, 0, :, ::2], q.expand(2, 5, 4, 16)[:, :, :1].expand(2, 5, 4, 16)):
        with pytest.raises(ValueError):
            nb._req_tokens(bad, "q", tuple(bad.shape), q.dtype, q.device)


def test_linattn_definition():
    """Without decay it is causal attention without softmax; with decay 0 only the token itself
    counts; two halves with the state carried are the whole; gradients are differences."""
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 2, 7, 2, 3))
    v, do = rng.standard_normal((2, 2, 7, 2, 4))
    o, s = layer.linattn_fwd(q, k, v, np.zeros(2), scale=0.5)
    scores = np.einsum("bihd,bjhd->bhij", q, k) * np.tril(np.ones((7, 7)))
    assert np.allclose(o, 0.5 * np.einsum("bhij,bjhe->bihe", scores, v))
    assert np.allclose(s, np.einsum("bjhd,bjhe->bhde", k, v))
    o, _ = layer.linattn_fwd(q, k, v, np.full(2, -np.inf))
    assert np.allclose(o, (q * k).sum(-1, keepdims=True) * v)
    a = np.array([-0.1, -1.0])
    whole, end = layer.linattn_fwd(q, k, v, a)
    o1, s1 = layer.linattn_fwd(q[:, :3], k[:, :3], v[:, :3], a)
    o2, s2 = layer.linattn_fwd(q[:, 3:], k[:, 3:], v[:, 3:], a, state=s1)
    assert np.allclose(np.concatenate([o1, o2], 1), whole) and np.allclose(s2, end)
    s0, ds = rng.standard_normal((2, 2, 2, 3, 4))
    n = np.array([7, 4])

    def loss(q, k, v, s0):
        o, s = layer.linattn_fwd(q, k, v, a, s0, n, 0.7)
        return (o * do).sum() + (s * ds).sum()
    g = layer.linattn_bwd(q, k, v, a, do, s0, ds, n, 0.7)
    base = dict(q=q, k=k, v=v, s0=s0)
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "dstate")):
        way = rng.standard_normal(base[name].shape)
        up, down = (loss(**{**base, name: base[name] + h * way}) for h in (1e-5, -1e-5))
        assert abs((g[key] * way).sum() - (up - down) / 2e-5) < 1e-6
