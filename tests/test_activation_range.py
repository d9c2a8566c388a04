"""The activations and their slopes over every BF16 number of [-128, 128], far
tails included, against float64.

The bound: half a BF16 step, 2^-8 of the value, and half the least BF16 number,
2^-134; FP32 arithmetic, whose exponents reach 150 and are computed with at most six
roundings of 2^-24 (150 * 6 * 2^-24 * ln 2 = 3.7e-5 < 2^-14 of every term, with
room for the approximate instructions and the fitted polynomial, a few 2^-21); and the
gradual underflow of the logistic and the density below 2^-126, 2^-150 absolute,
which a factor of at most 2^9 (|z| times the inner slope, where either is so small)
multiplies."""
import math

import pytest
import torch

import block_scaled_fp8_fp8blk_b200 as fb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAMES = ["relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fb.read_device_error() == 0


def numbers():
    """Every BF16 number of magnitude up to 128, [1, n] with n a multiple of 8."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[v.float().abs() <= 128]
    return torch.cat([v, v[:-v.numel() % 8]]).view(1, -1).to(DEV)


def terms(name, z):
    """act(z), and the two terms whose sum is act'(z), in float64."""
    z = z.double()
    zero = torch.zeros_like(z)
    if name == "relu":
        return z.clamp(min=0), ((z > 0).double(), zero)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * cdf, (cdf, z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    c1, c3 = (2 * math.sqrt(2 / math.pi), 2 * math.sqrt(2 / math.pi) * 0.044715) if name == "gelu_tanh" else (1.0, 0.0)
    t = c1 * z + c3 * z ** 3
    s, rest = torch.sigmoid(t), torch.sigmoid(-t)
    return z * s, (s, z * s * rest * (c1 + 3 * c3 * z * z))


def check(got, parts, what):
    want = sum(parts)
    size = sum(p.abs() for p in parts)
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -14 * size + 2.0 ** -134 + 2.0 ** -141
    off = (got.double() - want).abs() - tol
    assert bool(torch.isfinite(off).all()), what
    i = off.argmax().item()
    assert off[i] <= 0, f"{what}: {got[i].item():.3e} for {want[i].item():.3e}"


@pytest.mark.parametrize("name", NAMES)
def test_backward_over_every_number(name):
    z = numbers()
    n = z.shape[1]
    one = torch.ones_like(z)
    value, slope = terms(name, z[0])
    out = fb.gated_backward(one, z, one, activation=name)
    padded = -(-n // 128) * 128
    check(out[0, :n], slope, "act'")
    check(out[0, padded:padded + n], (value,), "act")
    dz, dbias = fb.epilogue_backward(one, z, activation=name)
    check(dz[0], slope, "dz")
    check(dbias.to(torch.bfloat16), slope, "dbias")


@pytest.mark.parametrize("mode", ["w8a16", "w8a8", "empty"])
@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("name", NAMES)
def test_forward_over_every_number(mode, M, name):
    """Through the linears (zero activations, so that z is the bias) and through the
    empty product."""
    z = numbers()
    n, k = z.shape[1], 0 if mode == "empty" else 128
    q = torch.full((n, k), 0x38, dtype=torch.uint8, device=DEV)
    s = torch.ones((-(-n // 128), -(-k // 128)), device=DEV)
    x = torch.zeros((M, k), dtype=torch.bfloat16, device=DEV)
    f = fb.linear_w8a8_epilogue if mode == "w8a8" else fb.linear_w8a16_epilogue
    y = f(x, q, s, bias=z[0], activation=name)
    value, _ = terms(name, z[0])
    for row in (y[0], y[M - 1]):
        check(row, (value,), name)


@pytest.mark.parametrize("name", NAMES)
def test_gated_backward_products_beyond_fp32(name):
    """dh u is beyond FP32, dg is not: the slope is 0 (the exact one of relu, or
    below 1e-300) or, at the last z, so small that dg is an ordinary number."""
    z = [-1e4, -200.0, -60.0, -25.0]
    g = torch.tensor([z + z], device=DEV).to(torch.bfloat16)
    big = torch.full_like(g, 1e20)
    out = fb.gated_backward(big, g, big, activation=name)
    a, slope = terms(name, g[0])
    want = big[0].double() ** 2 * sum(slope)
    near = want.abs() < 1e38
    assert near[0] and near[1]
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -14 * big[0].double() ** 2 * sum(p.abs() for p in slope) + 2.0 ** -134
    tol = tol + 2.0 ** -140 * big[0].double() ** 2      # the slope's own underflow, multiplied
    assert bool(((out[0, :8].double() - want).abs() <= tol)[near].all()), (out[0, :8], want)
    du = big[0].double() * a
    assert bool(((out[0, 128:136].double() - du).abs() <= 2.0 ** -7 * du.abs() + 2.0 ** -114).all())
