"""The norms around a block with its gate and residual scale, forward and backward, against the
fp64 definitions, and the gradients against differences."""
import itertools

import numpy as np
import pytest
import torch

from gpu_helpers import dev, f32_dev, host, to_dev
from oracle import layer
from selective_state_space_naju_amd import binding as nb

pytestmark = pytest.mark.gpu

TYPES = {"f32": ("f32", "f32", "f32"), "bf16": ("bf16", "bf16", "bf16"),
         "bf16_x32": ("bf16", "f32", "bf16"), "bf16_g32": ("bf16", "bf16", "f32"),
         "bf16_x32_g32": ("bf16", "f32", "f32")}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # the largest relative error of one rounding


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


def rounded(rng, shape, io, std=1.0):
    """Values of the io type, as floats."""
    x = torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32))
    return (x.bfloat16() if io == "bf16" else x).double().numpy()


def close(name, got, want, io, d, size=None):
    """An output is rounded once; before that it passed about 20 fp32 operations, a sum over d
    channels among them (its relative error is at most d roundings, in practice about sqrt d; the
    terms of a mean of squares are positive).  Differences of terms are held to the size of the
    terms: `size`, the output's own where it is not given."""
    got = host(got)
    assert got.shape == want.shape
    scale = np.abs(want) if size is None else size
    bound = HALF[io] * np.abs(want) + (32 + d ** 0.5) * 2.0 ** -24 * scale + 1e-30
    err = np.abs(got - want)
    worst = float((err / bound).max()) if err.size else 0.0
    print("  %-8s worst %.3f of the bound" % (name, worst), flush=True)
    assert worst <= 1.0, name


def case(R, d, types, gate, post, scale, seed):
    io, x_io, g_io = TYPES[types]
    rng = np.random.default_rng(seed)
    c = dict(x=rounded(rng, (R, d), x_io, 2.0), y=rounded(rng, (R, d), io, 0.7),
             z=rounded(rng, (R, d), io) if gate else None,
             scale=rounded(rng, (d,), "f32") if scale else None,
             w_post=1 + rounded(rng, (d,), "f32", 0.1) if post else None,
             w_pre=1 + rounded(rng, (d,), "f32", 0.1),
             dxn=rounded(rng, (R, d), g_io), dx=rounded(rng, (R, d), g_io))
    for k in ("w_post", "w_pre"):
        if c[k] is not None:
            c[k] = c[k].astype(np.float32).astype(np.float64)
    return c


def on_dev(c, types):
    io, x_io, g_io = TYPES[types]
    kind = dict(x=x_io, y=io, z=io, dxn=g_io, dx=g_io, scale="f32", w_post="f32", w_pre="f32")
    return {k: None if v is None else to_dev(v, kind[k]) for k, v in c.items()}


def check_fwd(R, d, types, gate=True, post=True, scale=True, seed=0):
    io, x_io, _ = TYPES[types]
    c = case(R, d, types, gate, post, scale, seed)
    t = on_dev(c, types)
    x, xn = nb.res_norm_fwd(t["x"], t["y"], t["z"], scale=t["scale"], w_post=t["w_post"],
                            w_pre=t["w_pre"])
    wx, wn = layer.res_norm_fwd(c["x"], c["y"], c["z"], c["scale"], c["w_post"], c["w_pre"])
    add = np.abs(wx - c["x"]) + np.abs(c["x"])
    close("x_new", x, wx, x_io, d, add)
    # (xn's error has that of x', magnified by the norm)
    close("xn", xn, wn, io, d, np.abs(wn) + add * np.abs(wn) / np.maximum(np.abs(wx), 1e-30))


def check_bwd(R, d, types, gate=True, post=True, scale=True, seed=0, pre=True, later=True):
    io, x_io, g_io = TYPES[types]
    c = case(R, d, types, gate, post, scale, seed)
    t = on_dev(c, types)
    kw = dict(scale="scale", w_post="w_post")
    got = nb.res_norm_bwd(t["dxn"] if pre else None, t["dx"] if later else None, t["x"], t["y"],
                          t["z"], w_pre=t["w_pre"] if pre else None,
                          dtype=None, **{k: t[v] for k, v in kw.items()})
    want = layer.res_norm_bwd(c["dxn"] if pre else None, c["dx"] if later else None, c["x"],
                              c["y"], c["z"], c["scale"], c["w_post"],
                              c["w_pre"] if pre else None)
    # the size of the terms that each output is a sum of: a row's largest for the outputs that a
    # mean was taken off, the sum of magnitudes over rows for the vectors' gradients
    rowmax = lambda x: np.abs(x).max(axis=1, keepdims=True) + 0 * x  # noqa: E731
    dx = rowmax(c["dx"]) * later + rowmax(want["dx"])
    close("dx", got["dx"], want["dx"], g_io, d, dx)
    sc = 1.0 if c["scale"] is None else np.abs(c["scale"])
    close("dy", got["dy"], want["dy"], io, d, rowmax(want["dy"]) * 4 + dx * sc)
    if gate:
        n = np.abs(c["y"]) * (3 if post else 1)
        close("dz", got["dz"], want["dz"], io, d, np.abs(want["dz"]) + dx * sc * n)
    for k, used in (("dw_pre", pre), ("dw_post", post), ("dscale", scale)):
        if not used:
            assert got[k] is None
            continue
        terms = (np.abs(c["dxn"]) * 4).sum(0) if k == "dw_pre" else (dx * 6 * (
            sc if k == "dw_post" else 1.0)).sum(0)
        # (a sum over R rows on top)
        close(k, got[k], want[k], "f32", d + R, terms)


@pytest.mark.parametrize("types", sorted(TYPES))
@pytest.mark.parametrize("R,d", [(1, 4), (5, 7), (3, 255), (9, 257), (6, 510), (2, 768), (3, 770),
                                 (4, 1023), (3, 1027), (2, 2049), (2, 4095), (2, 4098),
                                 (3, 8191), (2, 8192)])
def test_forward(R, d, types):
    check_fwd(R, d, types, seed=R * d)


@pytest.mark.parametrize("types", sorted(TYPES))
@pytest.mark.parametrize("R,d", [(1, 4), (5, 7), (3, 255), (9, 257), (6, 510), (2, 768), (3, 770),
                                 (4, 1023), (3, 1027), (2, 2049), (2, 4095), (2, 4098),
                                 (3, 8191), (2, 8192)])
def test_backward(R, d, types):
    check_bwd(R, d, types, seed=R * d)


@pytest.mark.parametrize("d", [96, 1027])
@pytest.mark.parametrize("gate,post,scale", list(itertools.product([False, True], repeat=3)))
def test_every_combination(gate, post, scale, d):
    check_fwd(5, d, "bf16_x32", gate, post, scale, seed=1)
    check_bwd(5, d, "bf16_g32", gate, post, scale, seed=2)
    check_bwd(5, d, "f32", gate, post, scale, seed=3, pre=False)
    check_bwd(5, d, "f32", gate, post, scale, seed=4, later=False)


@pytest.mark.parametrize("R,d", [(13003, 40), (2601, 600), (2600, 1500), (1100, 2050), (600, 5001)])
def test_more_rows_than_workgroups_hold(R, d):
    """Workgroups walk over rows, and their sums are joined."""
    check_fwd(R, d, "bf16", seed=5)
    check_bwd(R, d, "bf16_x32", seed=6)


def test_norm_alone_and_residual_alone():
    x = torch.randn(3, 7, 96, device=dev())
    w = torch.rand(96, device=dev()) + 0.5
    same, xn = nb.res_norm_fwd(x, w_pre=w, dtype=torch.bfloat16)
    assert same is x and xn.dtype == torch.bfloat16 and xn.shape == x.shape
    _, want = layer.res_norm_fwd(host(x).reshape(21, 96), w_pre=host(w))
    close("xn", xn.reshape(21, 96), want, "bf16", 96)
    y = torch.randn(3, 7, 96, device=dev()).bfloat16()
    new, none = nb.res_norm_fwd(x, y)
    assert none is None and torch.equal(new, x + y.float())
    g = nb.res_norm_bwd(xn, None, x, w_pre=w, dtype=torch.bfloat16)
    assert g["dy"] is None and g["dx"].dtype == torch.bfloat16
    g = nb.res_norm_bwd(None, x, x, y)
    assert torch.equal(g["dx"], x) and torch.equal(g["dy"], x.bfloat16())


def test_gradients_are_differences():
    """The loss sum(x_new * dx) + sum(xn * dxn) changes along a direction as the gradients say:
    with fp64 definitions for the loss, the gradients' fp32 error (about 1e-6) and the difference
    quotient's (the step squared, 1e-8, times third derivatives of some units) are all there is."""
    R, d = 6, 37
    c = case(R, d, "f32", True, True, True, 11)
    new, _ = layer.res_norm_fwd(c["x"], c["y"], c["z"], c["scale"], c["w_post"], c["w_pre"])
    t = on_dev(c, "f32")
    got = nb.res_norm_bwd(t["dxn"], t["dx"], f32_dev(new), t["y"], t["z"], scale=t["scale"],
                          w_post=t["w_post"], w_pre=t["w_pre"])

    def loss(**over):
        a = {**c, **over}
        x, xn = layer.res_norm_fwd(a["x"], a["y"], a["z"], a["scale"], a["w_post"], a["w_pre"])
        return (x * c["dx"]).sum() + (xn * c["dxn"]).sum()
    rng = np.random.default_rng(5)
    for k, gk in (("x", "dx"), ("y", "dy"), ("z", "dz"), ("scale", "dscale"),
                  ("w_post", "dw_post"), ("w_pre", "dw_pre")):
        way = rng.standard_normal(c[k].shape)
        h = 1e-4
        diff = (loss(**{k: c[k] + h * way}) - loss(**{k: c[k] - h * way})) / (2 * h)
        g = host(got[gk])
        size = np.abs(g * way).sum()
        print("  %-8s %.3e against %.3e" % (gk, (g * way).sum(), diff), flush=True)
        assert abs((g * way).sum() - diff) <= 1e-5 * size + 1e-6


def test_extreme_rows():
    """Rows of zeros give zeros; NaN and infinity stay in their row; huge gates are SiLU's limits."""
    d = 130
    x = torch.zeros(5, d, device=dev())
    y = torch.zeros(5, d, device=dev())
    z = torch.zeros(5, d, device=dev())
    w = torch.ones(d, device=dev())
    x[1] = 1.0
    y[1], z[1, 0], z[1, 1] = 2.0, 100.0, -100.0
    x[2, 3] = float("nan")
    y[3, 5] = float("inf")
    y[4] = -1.0
    new, xn = nb.res_norm_fwd(x, y, z, w_post=w, w_pre=w)
    assert (xn[0] == 0).all() and (new[0] == 0).all()
    assert abs(float(new[1, 0]) - 101.0) < 1e-4 and abs(float(new[1, 1]) - 1.0) < 1e-6
    assert torch.isnan(xn[2]).all() and torch.isnan(xn[3]).any()
    assert torch.isfinite(xn[4]).all() and torch.isfinite(xn[:2]).all()
    g = nb.res_norm_bwd(torch.ones_like(x), torch.ones_like(x), x, y, z, w_post=w, w_pre=w)
    for k in ("dx", "dy", "dz"):
        for r in (0, 1, 4):
            assert torch.isfinite(g[k][r]).all(), k


def test_no_tokens():
    w = torch.ones(64, device=dev())
    x = torch.zeros(0, 64, device=dev())
    _, xn = nb.res_norm_fwd(x, x, w_pre=w)
    assert xn.shape == (0, 64)
    g = nb.res_norm_bwd(x, x, x, x, scale=w, w_pre=w)
    assert (g["dw_pre"] == 0).all() and (g["dscale"] == 0).all()


def test_repeats_give_equal_bits():
    c = on_dev(case(3001, 200, "bf16", True, True, True, 3), "bf16")
    runs = [nb.res_norm_bwd(c["dxn"], c["dx"], c["x"], c["y"], c["z"], scale=c["scale"],
                            w_post=c["w_post"], w_pre=c["w_pre"]) for _ in range(3)]
    for r in runs[1:]:
        for k in r:
            assert torch.equal(r[k], runs[0][k]), k


def test_rows_behind_the_last_are_untouched():
    """Outputs inside larger buffers: what lies around them stays."""
    R, d = 5, 77
    c = on_dev(case(R, d, "bf16", True, True, True, 9), "bf16")
    keep = {k: torch.full((R + 2, d), 7.0, device=dev()).bfloat16() for k in ("x", "xn", "dx",
                                                                            "dy", "dz")}
    inside = {k: t[1:-1] for k, t in keep.items()}
    L, st = nb.lib(), torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()  # noqa: E731
    nb.check(L.naju_res_norm_fwd(R, d, nb.BF16, nb.BF16, p(c["x"]), p(c["y"]), p(c["z"]),
                                 p(c["scale"]), p(c["w_post"]), p(c["w_pre"]), 1e-6,
                                 p(inside["x"]), p(inside["xn"]), st))
    ws = nb.Workspace(L.naju_res_norm_bwd_workspace_bytes(R, d), dev())
    nb.check(L.naju_res_norm_bwd(R, d, nb.BF16, nb.BF16, nb.BF16, p(c["dxn"]), p(c["dx"]),
                                 p(c["x"]), p(c["y"]), p(c["z"]), p(c["scale"]), p(c["w_post"]),
                                 p(c["w_pre"]), 1e-6, p(inside["dx"]), p(inside["dy"]),
                                 p(inside["dz"]), None, None, None, p(ws.tensor), ws.nbytes, st))
    x, xn = nb.res_norm_fwd(c["x"], c["y"], c["z"], scale=c["scale"], w_post=c["w_post"],
                            w_pre=c["w_pre"])
    assert torch.equal(inside["x"], x) and torch.equal(inside["xn"], xn)
    for t in keep.values():
        assert (t[0] == 7).all() and (t[-1] == 7).all()


def test_graph_replays():
    c = on_dev(case(300, 96, "bf16", True, True, True, 21), "bf16")

    def step():
        x, xn = nb.res_norm_fwd(c["x"], c["y"], c["z"], scale=c["scale"], w_post=c["w_post"],
                                w_pre=c["w_pre"])
        return [x, xn] + list(nb.res_norm_bwd(c["dxn"], c["dx"], x, c["y"], c["z"],
                                              scale=c["scale"], w_post=c["w_post"],
                                              w_pre=c["w_pre"]).values())
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in range(4):
        c["y"].copy_(torch.randn(300, 96, device=dev()).bfloat16())
        want = step()
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), n
