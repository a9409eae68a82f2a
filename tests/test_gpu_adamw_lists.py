"""The lists that the update takes: whatever does not fit is refused by name, before anything is
written; tuples, parameters and subclasses are taken as lists of tensors are."""
import pytest
import torch

from gpu_helpers import dev
from selective_state_space_naju_amd import binding as nb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


SHAPES = [(3, 5), (300,), (), (2, 0), (16, 40)]


def lists(bits):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    c = {"p": [torch.randn(s, generator=g, device=dev()) for s in SHAPES],
         "g": [torch.randn(s, generator=g, device=dev()) for s in SHAPES]}
    st = torch.float32 if bits == 32 else torch.float8_e4m3fn
    for k in ("m", "v"):
        c[k] = [torch.zeros(s, device=dev()).to(st) for s in SHAPES]
        if bits == 8:
            c[k + "_scale"] = [torch.zeros(-(-t.numel() // 256), device=dev()) for t in c["p"]]
    c["copy"] = [torch.zeros(s, device=dev(), dtype=torch.bfloat16) for s in SHAPES]
    return c


def step(c, **kw):
    scales = {k: c[k] for k in ("m_scale", "v_scale") if k in c}
    nb.adamw_step(c["p"], c["g"], c["m"], c["v"], 1, 0.1, copies=c["copy"], **scales, **kw)


DEFECTS = {
    "missing": (lambda t: None, "required"),
    "host": (lambda t: t.cpu(), "must be on"),
    "type": (lambda t: t.to(torch.float16), "expected"),
    "strided": (lambda t: torch.cat([t, t], dim=-1)[..., ::2], "contiguous"),
    "longer": (lambda t: torch.cat([t, t], dim=-1), "expected"),
    "number": (lambda t: 3.0, "required"),
}


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("defect", sorted(DEFECTS))
def test_what_does_not_fit_is_named(bits, defect):
    change, text = DEFECTS[defect]
    for k in lists(bits):
        c = lists(bits)
        i = 4
        c[k] = list(c[k])
        x = c[k][i]
        if x.dtype == torch.float8_e4m3fn and defect in ("strided", "longer"):
            c[k][i] = change(x.view(torch.uint8)).view(torch.float8_e4m3fn)
        else:
            c[k][i] = change(x)
        kept = [t.clone() for t in lists(bits)["p"]]
        with pytest.raises((ValueError, TypeError), match=text) as e:
            step(c)
        if not (k == "p" and defect == "longer"):  # (there it is the others that do not fit)
            assert str(e.value).startswith("%s[%d]" % (k, i)), (k, str(e.value))
        for j, t in enumerate(kept):
            if not (k == "p" and j == i):
                assert torch.equal(c["p"][j], t)


def test_a_gradient_of_another_shape_is_named():
    c = lists(32)
    c["g"][0] = c["g"][0].t().contiguous()
    with pytest.raises(ValueError, match=r"g\[0\]: expected shape"):
        step(c)


def test_lists_of_other_lengths_are_refused():
    for k in ("g", "m", "v", "copy"):
        c = lists(32)
        c[k] = c[k][:-1]
        with pytest.raises(ValueError, match="expected 5 tensors, got 4"):
            step(c)


def test_sparse_tensors_are_refused():
    c = lists(32)
    c["g"][4] = c["g"][4].to_sparse()
    with pytest.raises((ValueError, RuntimeError)):
        step(c)


@pytest.mark.parametrize("bits", [32, 8])
def test_tuples_and_parameters(bits):
    a, b = lists(bits), lists(bits)
    step(a)
    b["p"] = torch.nn.ParameterList(b["p"])
    for k in ("g", "m", "v"):
        b[k] = tuple(b[k])
    step(b)
    for k in a:
        for x, y in zip(a[k], b[k]):
            view = (lambda t: t.view(torch.uint8)) if x.dtype == torch.float8_e4m3fn else (
                lambda t: t)
            assert torch.equal(view(x), view(y.detach())), k
