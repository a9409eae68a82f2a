"""GPU parity of the 4-bit linear layer and the quantisation against fp64 definitions.

Tolerance, derived before the first run.  The codes enter the matrix cores as
128 + q (at most 143) and 128 + z times the sum of x is taken off per group, so
each fp32 rounding is at most 2^-24 times 144 sum |x| s over a group.  A group of
up to 128 inputs passes through at most four products of 32 (a few roundings
each) and the sum of x through as many: 32 roundings are allowed for.  Over the
groups and the splits of the inputs the sums are of the result's size, with one
rounding per group.  Then bias, residual and one rounding to bf16 (2^-8 with the
fp32 roundings): |err| <= 2^-8 (|y| + tail) + tail, with
tail = 32 2^-24 144 sum_k |x_k| s_k + groups 2^-23 (sum |x w| + |bias| + |res|).
"""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, f32_dev, host, to_dev
from oracle import lm
from selective_state_space_naju_amd import binding as nb
from selective_state_space_naju_amd import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


def u8(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.uint8)).to(dev())


def draw(R, K, N, G, seed, zeros, extra):
    rng = np.random.default_rng(seed)
    ng = -(-K // G)
    x = inputs.bf16_round(rng.standard_normal((R, K), dtype=np.float32) + np.float32(0.3))
    q = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    s = inputs.bf16_round((rng.uniform(0.2, 1.8, (N, ng)) * 0.02).astype(np.float32))
    z = rng.integers(0, 16, (N, ng)).astype(np.uint8) if zeros else None
    bias = rng.standard_normal(N).astype(np.float32) if extra else None
    res = inputs.bf16_round(rng.standard_normal((R, N), dtype=np.float32)) if extra else None
    return x, q, s, z, bias, res


def call(x, q, s, G, z, bias, res):
    return nb.w4_linear(to_dev(x, "bf16"), u8(q), to_dev(s, "bf16"), G,
                        None if z is None else u8(z), None if bias is None else f32_dev(bias),
                        None if res is None else to_dev(res, "bf16"))


def check(y, x, q, s, G, z, bias, res):
    K = x.shape[1]
    ref = lm.w4_linear(x, q, s, G, z, bias, res)
    group = np.arange(K) // G
    sk = np.abs(s.astype(np.float64))[:, group]
    ax = np.abs(x.astype(np.float64))
    add = (0 if bias is None else np.abs(bias)) + (0 if res is None else np.abs(res))
    tail = 32 * 2.0 ** -24 * 144 * (ax @ sk.T)
    tail = tail + s.shape[1] * 2.0 ** -23 * (ax @ np.abs(lm.w4_weights(q, s, G, z)).T + add)
    err = np.abs(host(y) - ref)
    bound = 2.0 ** -8 * (np.abs(ref) + tail) + tail + 1e-30
    print("  worst error %.3f of the bound" % (err / bound).max(), flush=True)
    assert np.all(err <= bound)


CASES = [  # rows, d_in, d_out, group, zeros, bias and residual
    (1, 2, 1, 32, False, False),
    (1, 64, 16, 64, False, True),
    (3, 34, 5, 32, True, False),
    (1, 130, 17, 128, True, True),
    (2, 768, 1536, 64, False, False),
    (1, 1536, 16, 128, False, True),
    (16, 1030, 33, 64, True, True),
    (17, 1024, 48, 32, True, False),
    (32, 2050, 100, 128, False, True),
    (33, 510, 31, 64, True, True),
    (64, 1600, 130, 32, False, False),
    (65, 514, 47, 128, True, True),
    (130, 258, 19, 64, False, True),
    (5, 4100, 301, 32, True, False),
    (4, 98, 66000, 32, True, True),
    (20, 646, 65600, 64, False, True),
    (40, 384, 70001, 128, True, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "r%d_k%d_n%d_g%d_z%d_e%d" % c)
def test_w4_linear(case):
    R, K, N, G, zeros, extra = case
    print("w4", case, flush=True)
    a = draw(R, K, N, G, 31, zeros, extra)
    check(call(*a[:3], G, *a[3:]), *a[:3], G, *a[3:])


def test_w4_unaligned_tensors():
    """Codes, scales and zeros that start at any byte or element."""
    R, K, N, G = 3, 200, 40, 64
    x, q, s, z, bias, _ = draw(R, K, N, G, 32, True, True)
    qd = torch.zeros(q.size + 3, dtype=torch.uint8, device=dev())[3:].view(N, K // 2)
    sd = torch.zeros(s.size + 1, dtype=torch.bfloat16, device=dev())[1:].view(s.shape)
    xd = torch.zeros(x.size + 1, dtype=torch.bfloat16, device=dev())[1:].view(x.shape)
    zd = torch.zeros(z.size + 1, dtype=torch.uint8, device=dev())[1:].view(z.shape)
    qd.copy_(u8(q)), sd.copy_(to_dev(s, "bf16")), xd.copy_(to_dev(x, "bf16")), zd.copy_(u8(z))
    check(nb.w4_linear(xd, qd, sd, G, zd, f32_dev(bias)), x, q, s, G, z, bias, None)


def test_w4_outlier_inputs():
    """A few inputs a thousand times the others, under codes of weight zero and others."""
    R, K, N, G = 4, 512, 64, 128
    x, q, s, _, _, _ = draw(R, K, N, G, 33, False, False)
    x[:, [5, 300]] = 1000.0
    q[:, 2] = (q[:, 2] & 0x0F) | 0x80  # input 5: weight 0
    check(call(x, q, s, G, None, None, None), x, q, s, G, None, None, None)


def test_w4_non_finite_inputs_stay_in_their_row():
    x, q, s, _, _, _ = draw(3, 256, 50, 64, 34, False, False)
    clean = host(call(x, q, s, 64, None, None, None))
    x[1, 17] = np.inf
    got = host(call(x, q, s, 64, None, None, None))
    assert not np.isfinite(got[1]).any()
    assert np.array_equal(got[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("case", [(64, 16, 64, "f32"), (130, 33, 128, "bf16"), (34, 300, 32, "f32"),
                                  (768, 1536, 64, "bf16")], ids=lambda c: "k%d_n%d_g%d_%s" % c)
def test_w4_quantize(case, zeros):
    """Every weight is within half a step of its code, the steps follow the group's extremes."""
    K, N, G, io = case
    rng = np.random.default_rng(35)
    W = rng.standard_normal((K, N)).astype(np.float32) * rng.uniform(0.01, 2, N).astype(np.float32)
    W[:min(G, K), 0] = 0.0       # a group of zeros
    W[:, N - 1] = np.abs(W[:, N - 1])  # one sign only
    W = inputs.bf16_round(W) if io == "bf16" else W
    print("w4_quantize", case, zeros, flush=True)
    q, s, z = nb.w4_quantize(to_dev(W, io), G, zeros=zeros)
    back = lm.w4_weights(q.cpu().numpy(), host(s), G, None if z is None else z.cpu().numpy())
    sd = host(s)
    ng = -(-K // G)
    for g in range(ng):
        w = W[g * G:(g + 1) * G].astype(np.float64)
        lo, hi = np.minimum(w.min(0), 0), np.maximum(w.max(0), 0)
        step = (hi - lo) / 15 if zeros else np.maximum(hi, -lo) / 7
        assert np.allclose(sd[:, g], step, rtol=2.0 ** -8, atol=0)
        # half a step (and, with zeros, half a step of z's own rounding); the scale's rounding
        # moves the ends of the range by up to 15 2^-9 steps
        slack = (1.0 if zeros else 0.5) + 15 * 2.0 ** -8
        assert np.all(np.abs(back[:, g * G:(g + 1) * G].T - w) <= slack * sd[:, g] + 1e-12)


def test_w4_quantize_then_linear_equals_the_dequantised_product():
    rng = np.random.default_rng(36)
    W = to_dev(rng.standard_normal((384, 100)).astype(np.float32) * 0.05, "bf16")
    x = to_dev(rng.standard_normal((6, 384)).astype(np.float32), "bf16")
    for zeros in (False, True):
        q, s, z = nb.w4_quantize(W, 64, zeros=zeros)
        a = [x, q, s, z]
        xn, qn, sn = host(x), q.cpu().numpy(), host(s)
        zn = None if z is None else z.cpu().numpy()
        check(nb.w4_linear(a[0], a[1], a[2], 64, a[3]), xn, qn, sn, 64, zn, None, None)


def test_w4_repeats_bit_for_bit_and_on_another_stream():
    a = draw(9, 1000, 555, 64, 37, True, True)
    first = call(*a[:3], 64, *a[3:])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        again = call(*a[:3], 64, *a[3:])
    s.synchronize()
    assert torch.equal(first, again)


def test_w4_empty_and_refusals():
    x, q, s, _, _, _ = draw(2, 64, 10, 32, 38, False, False)
    X, Q, S = to_dev(x, "bf16"), u8(q), to_dev(s, "bf16")
    assert nb.w4_linear(X[:0], Q, S, 32).shape == (0, 10)
    assert nb.w4_linear(X, Q[:0], S[:0], 32).shape == (2, 0)
    e = torch.empty(2, 0, dtype=torch.bfloat16, device=dev())
    bias = torch.randn(10, device=dev())
    y = nb.w4_linear(e, torch.empty(10, 0, dtype=torch.uint8, device=dev()),
                     torch.empty(10, 0, dtype=torch.bfloat16, device=dev()), 32, None, bias)
    assert torch.equal(y, bias.bfloat16().expand(2, 10))
    with pytest.raises(TypeError):
        nb.w4_linear(X.float(), Q, S, 32)
    with pytest.raises(ValueError):
        nb.w4_linear(X, Q[:, :-1].contiguous(), S, 32)
    with pytest.raises(ValueError):
        nb.w4_linear(X, Q, S, 64)
    with pytest.raises(ValueError):
        nb.w4_linear(X[:, :-1].contiguous(), Q, S, 32)
    with pytest.raises(nb.NajuError):
        nb.w4_linear(X, Q, torch.empty(10, 4, dtype=torch.bfloat16, device=dev()), 16)
    with pytest.raises(nb.NajuError):
        nb.w4_quantize(torch.randn(63, 4, device=dev()), 32)
