"""The feed-forward operators on the GPU -- the gated linear, the linear with
an epilogue, their backward passes, the transposed weight and the weight
gradient -- against plain float64 forms.

Tolerances count roundings. Half a BF16 step is 2^-8 of the value. A sum over
K on the tensor cores is at most 2 roundings per MMA step inside a 128-wide
slab (8 steps for BF16) and one per slab outside, each at most 2^-23 of the sum
of magnitudes S, so |sum - exact| <= acc(K) S with acc(K) = (16 + K/128) 2^-22
(a factor two to spare); over tokens the steps are 16 long. The activations
change that by at most their slope (below 1.13 in magnitude) and add FP32
errors of a few 2^-21 relative."""
import math

import numpy as np
import pytest
import torch

import block_scaled_fp8_fp8blk_b200 as fb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = 2.0 ** -8        # half a BF16 step, relative
SLOPE = 1.13            # largest |act'|
FP32 = 2.0 ** -19       # FP32 arithmetic of an activation, relative
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    fb.lib()
    yield
    assert fb.read_device_error() == 0, "a kernel reported a timed-out wait"


def up(a, b):
    return -(-a // b) * b


def acc(n):
    return (16 + n / 128) * 2.0 ** -22


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def rows(t, align=8, extra=0):
    """t in a buffer with padded rows (the padding holds NaN)."""
    r, c = t.shape
    buf = torch.full((max(r, 1), up(max(c, 1), align) + extra), float("nan"), dtype=t.dtype, device=DEV)
    buf[:r, :c] = t.to(DEV)
    return buf[:r, :c]


def normal(g, m, n, sigma=1.0, extra=0):
    return rows((torch.randn(m, n, generator=g) * sigma).to(torch.bfloat16), 8, extra)


def weight(g, n, k, sigma=0.02, ldq=None):
    w = rows((torch.randn(n, k, generator=g) * sigma).to(torch.bfloat16))
    return fb.quantize_weight(w, ldq=ldq)


def dequantized(q, s):
    n, k = q.shape
    blocks = s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return q.contiguous().view(torch.float8_e4m3fn).double() * blocks


def activations(mode, x):
    """x in float64 as the product sees it."""
    if mode == "w8a16" or x.numel() == 0:
        return x.double()
    qx, sx = fb.quantize_act(x)  # bit-exact against the oracle in its own tests
    m, k = x.shape
    s = sx[:, :m].t().double().repeat_interleave(128, 1)[:, :k]
    return qx.contiguous().view(torch.float8_e4m3fn).double() * s


def act(name, z):
    """(act(z), act'(z)) in float64."""
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
        sn = torch.sigmoid(-2 * c * (z + 0.044715 * z ** 3))
        return z * s, s + z * s * sn * 2 * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    return z, torch.ones_like(z)


def within(got, want, tol, what):
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.numel() == 0:
        return
    assert bool(torch.isfinite(got.double()).all()), f"{what}: not finite"
    excess = ((got.double() - want).abs() - tol).max().item()
    assert excess <= 0, f"{what}: off by {excess:.3e} more than the bound"


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


FUNCS = {("linear", "w8a16"): fb.linear_w8a16_epilogue, ("linear", "w8a8"): fb.linear_w8a8_epilogue,
         ("gated", "w8a16"): fb.gated_linear_w8a16, ("gated", "w8a8"): fb.gated_linear_w8a8}


def run_gated(mode, M, K, N, name="silu", keep=False, seed=1, sigma=0.02, extra=0):
    g = gen(seed)
    x = normal(g, M, K, extra=extra)
    wg, wu = weight(g, N, K, sigma), weight(g, N, K, sigma)
    out = torch.full((M, up(N, 8) + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    kept = [torch.full((M, up(N, 8) + 8), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    FUNCS["gated", mode](x, *wg, *wu, activation=name, out=out[:, :N],
                         preact=tuple(t[:, :N] for t in kept) if keep else None)
    xd = activations(mode, x)
    dg, du = dequantized(*wg), dequantized(*wu)
    gd, ud = xd @ dg.T, xd @ du.T
    eg, eu = acc(K) * (xd.abs() @ dg.abs().T), acc(K) * (xd.abs() @ du.abs().T)
    a = act(name, gd)[0]
    h = a * ud
    tol = HALF * h.abs() + FP32 * h.abs() + (SLOPE * eg) * (ud.abs() + eu) + a.abs() * eu + 1e-37
    within(out[:, :N], h, tol, "h")
    assert (out[:, N:] == 7.0).all(), "wrote past N"
    if keep:
        within(kept[0][:, :N], gd, HALF * gd.abs() + 1.01 * eg + 1e-37, "g")
        within(kept[1][:, :N], ud, HALF * ud.abs() + 1.01 * eu + 1e-37, "u")
        assert all((t[:, N:] == 7.0).all() for t in kept)
    return x, wg, wu, out[:, :N], kept


GATED_SHAPES = [(1, 128, 64), (1, 1000, 1000), (7, 129, 65), (16, 640, 512), (17, 256, 1), (33, 384, 200),
                (64, 1024, 640), (100, 130, 72), (128, 512, 320), (129, 300, 72), (200, 16, 130),
                (300, 1000, 1000), (512, 640, 9500), (700, 2048, 257)]


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("M,K,N", GATED_SHAPES)
def test_gated_linear(mode, M, K, N):
    run_gated(mode, M, K, N, "silu", keep=(M + N) % 2 == 0, seed=M + K + N)


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("M", [3, 150])
def test_gated_activations(mode, name, M):
    run_gated(mode, M, 384, 200, name, keep=True, seed=5)


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_gated_large_preactivations(mode, name):
    """Pre-activations of hundreds: the gates saturate to 0 and to the identity."""
    run_gated(mode, 40, 512, 96, name, keep=True, seed=6, sigma=20.0)


@pytest.mark.parametrize("M", [64, 300])
def test_gated_w8a8_products_are_the_linears(M):
    """g and u are bit for bit what the W8A8 linear gives for each weight."""
    x, wg, wu, _, kept = run_gated("w8a8", M, 640, 400, keep=True)
    for t, w in zip(kept, (wg, wu)):
        assert same_bits(t[:, :400], fb.linear_w8a8(x, *w))


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
def test_gated_raster_groups(mode):
    """9000 tokens with K = 3000: two unequal raster groups."""
    run_gated(mode, 9000, 3000, 200, seed=8)


def run_linear(mode, M, K, N, name="none", bias=False, residual=False, keep=False, in_place=False,
               seed=2, sigma=0.02):
    g = gen(seed)
    x = normal(g, M, K)
    w = weight(g, N, K, sigma)
    b = normal(g, 1, N, 0.5)[0].contiguous() if bias else None
    out = torch.full((M, up(N, 8) + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    r = normal(g, M, N, extra=8) if residual or in_place else None
    rd = r.double() if r is not None else 0.0
    if in_place:
        out[:, :N] = r
        r = out[:, :N]
    z = torch.full((M, up(N, 8) + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    FUNCS["linear", mode](x, *w, bias=b, activation=name, residual=r, out=out[:, :N],
                          preact=z[:, :N] if keep else None)
    xd, wd = activations(mode, x), dequantized(*w)
    zd = xd @ wd.T + (b.double() if bias else 0.0)
    ez = acc(K) * (xd.abs() @ wd.abs().T) + 2.0 ** -23 * zd.abs()
    a = act(name, zd)[0]
    y = a + rd
    within(out[:, :N], y, HALF * y.abs() + FP32 * (a.abs() + y.abs()) + SLOPE * ez + 1e-37, "y")
    assert (out[:, N:] == 7.0).all(), "wrote past N"
    if keep:
        within(z[:, :N], zd, HALF * zd.abs() + 1.01 * ez + 1e-37, "z")
        assert (z[:, N:] == 7.0).all()
    return x, w, out[:, :N]


LINEAR_SHAPES = [(1, 128, 128), (1, 8192, 640), (5, 1, 9), (16, 640, 512), (31, 384, 257), (64, 1000, 1000),
                 (128, 512, 384), (129, 300, 72), (333, 1000, 1000), (512, 2048, 1280), (300, 128, 19000)]


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("M,K,N", LINEAR_SHAPES)
def test_linear_epilogue(mode, M, K, N):
    run_linear(mode, M, K, N, ACTS[(M + N) % 5], bias=True, residual=True, keep=M % 2 == 1, seed=M + N)


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("M", [4, 260])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("parts", ["", "bias", "residual", "in_place", "keep"])
def test_linear_epilogue_parts(mode, M, name, parts):
    run_linear(mode, M, 300, 136, name, **({parts: True} if parts else {}))


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("M,K,N", [(4, 300, 137), (100, 700, 333), (260, 300, 137), (9000, 3000, 200)])
def test_linear_epilogue_everything_at_once(mode, M, K, N):
    """Bias, activation, kept z and the residual updated in place; the last size
    walks two unequal raster groups."""
    run_linear(mode, M, K, N, "gelu_tanh", bias=True, keep=True, in_place=True, seed=17)


# Few tiles and many K slabs: W8A8 shares a tile among 2, 4 or 8 SMs.
SPLIT_SHAPES = [(1, 8192, 640), (40, 8192, 256), (128, 2560, 5120), (100, 4100, 2570), (300, 2100, 1000),
                (129, 16000, 130), (1, 25600, 5120), (256, 2048, 9000)]


@pytest.mark.parametrize("M,K,N", SPLIT_SHAPES)
def test_few_tiles_and_many_slabs(M, K, N):
    run_linear("w8a8", M, K, N, "silu", bias=True, keep=True, in_place=True, seed=K)
    run_linear("w8a8", M, K, N, residual=True, seed=K + 1)
    run_gated("w8a8", M, K, N // 2, "gelu", keep=True, seed=K + 2)
    x, w, first = run_linear("w8a8", M, K, N, "gelu", seed=K + 3)
    for _ in range(3):
        assert same_bits(fb.linear_w8a8_epilogue(x, *w, activation="gelu"), first)


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("M", [1, 50, 129, 300])
def test_rows_behind_the_last_token_stay(mode, M):
    """Buffers of more rows than tokens: what lies behind is not written."""
    g = gen(18)
    K, N = 256, 200
    w, wu = weight(g, N, K), weight(g, N, K)
    x, r = normal(g, M + 9, K)[:M], normal(g, M + 9, N)[:M]
    big = [torch.full((M + 9, N), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(5)]
    y, z, h, a, b = (t[:M] for t in big)
    FUNCS["linear", mode](x, *w, residual=r, preact=z, out=y)
    FUNCS["gated", mode](x, *w, *wu, preact=(a, b), out=h)
    assert all((t[M:] == 7.0).all() and not (t[:M] == 7.0).all() for t in big)
    dgu = torch.full((M + 9, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    fb.gated_backward(h, a, b, out=dgu[:M])
    fb.epilogue_backward(h, z, activation="silu", dz=y)
    assert (dgu[M:] == 7.0).all() and (big[0][M:] == 7.0).all()
    dw = torch.full((N + 9, K), 7.0, device=DEV)
    fb.linear_grad_weight(y, x, out=dw[:N])
    qt = torch.full((K + 9, 208), 0xA5, dtype=torch.uint8, device=DEV)
    fb.transpose_weight(*w, qt=qt[:K, :N])
    assert (dw[N:] == 7.0).all() and (qt[K:] == 0xA5).all()


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
def test_offsets_beyond_32_bits(mode):
    """Activations of more than 2^32 bytes (and 2^31 elements): rows at both ends."""
    M, K, N = 70000, 64, 32768
    g = gen(19)
    w, wu = weight(g, N, K), weight(g, N, K)
    x = normal(g, M, K)
    rows_ = torch.cat([torch.arange(3), torch.arange(65500, 65560), torch.arange(M - 3, M)]).to(DEV)
    y = torch.ones((M, N), dtype=torch.bfloat16, device=DEV)
    FUNCS["linear", mode](x, *w, residual=y, out=y)
    xd = activations(mode, x[rows_].contiguous())
    zd, ud = xd @ dequantized(*w).T, xd @ dequantized(*wu).T
    within(y[rows_], zd + 1, HALF * (zd + 1).abs() + 1e-4, "y")
    kept = tuple(torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    FUNCS["gated", mode](x, *w, *wu, activation="silu", preact=kept, out=y)
    a, s = act("silu", zd)
    within(y[rows_], a * ud, HALF * (a * ud).abs() + 1e-4, "h")
    within(kept[1][rows_], ud, HALF * ud.abs() + 1e-4, "u")
    dgu = fb.gated_backward(y, *kept)
    d, gg, uu = (t[rows_].double() for t in (y, *kept))
    a, s = act("silu", gg)
    within(dgu[rows_, :N], d * uu * s, HALF * (d * uu * s).abs() + 1e-6, "dg")
    within(dgu[rows_, N:], d * a, HALF * (d * a).abs() + 1e-6, "du")
    dz, db = fb.epilogue_backward(y, kept[0], activation="silu", dz=y)
    within(dz[rows_], d * s, HALF * (d * s).abs() + 1e-6, "dz")
    dw = fb.linear_grad_weight(dz, x)
    cols = [0, 1, N - 1]
    want = dz[:, cols].double().T @ x.double()
    within(dw[cols], want, (M / 8 + 16) * 2.0 ** -22 * (dz[:, cols].double().abs().T @ x.double().abs()), "dw")


def test_weights_beyond_32_bits():
    """Weight gradients and transposed codes of more than 2^31 elements."""
    g = gen(20)
    N, K = 70000, 32768
    dz, x = normal(g, 16, N), normal(g, 16, K)
    dw = fb.linear_grad_weight(dz, x)
    sel = [0, 65536, N - 1]
    want = dz[:, sel].double().T @ x.double()
    within(dw[sel], want, 10 * 2.0 ** -22 * (dz[:, sel].double().abs().T @ x.double().abs()), "dw")
    del dw
    q = torch.arange(251, dtype=torch.uint8, device=DEV).repeat(N * K // 251 + 1)[:N * K].view(N, K)
    s = torch.rand((-(-N // 128), K // 128), device=DEV)
    qt, st = fb.transpose_weight(q, s)
    for k in (0, 4097, K - 1):
        assert torch.equal(qt[k], q[:, k])
    assert torch.equal(st, s.t())


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("M", [1, 48, 128, 300])
def test_empty_epilogue_is_the_linear(mode, M):
    """Without bias, activation and residual the result is the linear's: bit for
    bit where the slabs are added in the same order (always at these sizes,
    but for W8A16 up to 128 tokens, where the plain call splits the tiles that
    this one runs whole), else the same sum in another order, rounded."""
    x, w, y = run_linear(mode, M, 640, 1000)
    plain = (fb.linear_w8a16 if mode == "w8a16" else fb.linear_w8a8)(x, *w)
    if mode == "w8a8" or M > 128:
        assert same_bits(y, plain)
    xd, wd = activations(mode, x), dequantized(*w)
    within(y, plain.double(), 2 * HALF * plain.double().abs() + 2 * acc(640) * (xd.abs() @ wd.abs().T), "order")


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
def test_linear_epilogue_edges(mode):
    """Empty sizes write nothing; K = 0 gives act(bias) + residual; no
    workspace above 128 tokens runs every W8A16 tile whole."""
    g = gen(3)
    f, gf = FUNCS["linear", mode], FUNCS["gated", mode]
    w, wu = weight(g, 200, 256), weight(g, 200, 256)
    empty = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    assert f(empty, *w, activation="gelu").shape == (0, 200)
    assert gf(empty, *w, *wu).shape == (0, 200)
    q0, s0 = torch.empty((200, 0), dtype=torch.uint8, device=DEV), torch.empty((2, 0), device=DEV)
    x0 = torch.empty((5, 0), dtype=torch.bfloat16, device=DEV)
    b, r = normal(g, 1, 200)[0].contiguous(), normal(g, 5, 200)
    z = torch.empty((5, 200), dtype=torch.bfloat16, device=DEV)
    y = f(x0, q0, s0, bias=b, activation="silu", residual=r, preact=z)
    want = act("silu", b.double())[0] + r.double()
    within(y, want, HALF * want.abs() + 1e-6, "K = 0")
    assert same_bits(z, b.expand(5, 200))
    kept = tuple(torch.ones((5, 200), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    h = gf(x0, q0, s0, q0, s0, preact=kept)
    assert not h.any() and not kept[0].any() and not kept[1].any()
    q1, s1 = torch.empty((0, 256), dtype=torch.uint8, device=DEV), torch.empty((0, 2), device=DEV)
    assert f(normal(g, 3, 256), q1, s1).shape == (3, 0)
    assert gf(normal(g, 3, 256), q1, s1, q1, s1).shape == (3, 0)


def test_w8a16_without_optional_workspace():
    """Above 128 tokens the workspace only enables the split last wave: without
    it the same values come from whole tiles, within the tolerance."""
    g = gen(4)
    M, K, N = 300, 640, 1000
    x, wg, wu, r = normal(g, M, K), weight(g, N, K), weight(g, N, K), normal(g, M, N)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    for f in (lambda ws: fb.linear_w8a16_epilogue(x, *wg, activation="gelu", residual=r, workspace=ws),
              lambda ws: fb.gated_linear_w8a16(x, *wg, *wu, workspace=ws)):
        a, b = f(None).double(), f(none).double()
        assert ((a - b).abs() <= 2 * HALF * a.abs() + 1e-3).all()


def test_scales_and_strides_of_the_halves_of_a_fused_weight():
    """A fused [2N, K] weight as its two halves, with a padded row stride."""
    g = gen(9)
    M, K, N = 70, 300, 256
    q, s = weight(g, 2 * N, K, ldq=352)
    x = normal(g, M, K, extra=16)
    h = fb.gated_linear_w8a16(x, q[:N], s[:2], q[N:], s[2:])
    w = dequantized(q, s)
    a, b = x.double() @ w[:N].T, x.double() @ w[N:].T
    want = act("silu", a)[0] * b
    within(h, want, HALF * want.abs() + 1e-4, "fused weight")


# ------------------------------------------------------------------ backward
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("M,N", [(1, 8), (3, 1), (77, 1000), (200, 128), (5, 2049), (1, 25600)])
def test_gated_backward(name, M, N):
    g = gen(M + N)
    dh, gg, u = normal(g, M, N, 0.1, extra=8), normal(g, M, N, 3.0), normal(g, M, N, 3.0)
    Np = up(N, 128)
    out = torch.full((M, 2 * Np + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    fb.gated_backward(dh, gg, u, activation=name, out=out[:, :2 * Np])
    a, s = act(name, gg.double())
    dg, du = dh.double() * u.double() * s, dh.double() * a
    # the slope's FP32 error: a few 2^-22 of its terms, which reach 1 + |z|
    es = 2.0 ** -20 * (1 + gg.double().abs()) * (dh.double() * u.double()).abs()
    within(out[:, :N], dg, HALF * dg.abs() + es + 1e-37, "dg")
    within(out[:, Np:Np + N], du, (HALF + FP32) * du.abs() + 1e-37, "du")
    assert not out[:, N:Np].any() and not out[:, Np + N:2 * Np].any(), "padding columns"
    assert (out[:, 2 * Np:] == 7.0).all()


def test_gated_backward_saturated():
    """Gates far out on both sides, where exp overflows: finite, and 0 or dh u."""
    gg = torch.tensor([[-3e38, -1e13, -200.0, -101.0, 101.0, 200.0, 1e13, 3e38]], device=DEV).to(torch.bfloat16)
    ones = torch.ones_like(gg)
    for name in ("gelu", "gelu_tanh", "silu"):
        out = fb.gated_backward(ones, gg, ones, activation=name)
        assert out[0, :8].tolist() == [0, 0, 0, 0, 1, 1, 1, 1], name
        assert torch.equal(out[0, 128:136].double(), torch.where(gg[0] > 0, gg[0], 0 * gg[0]).double()), name


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("M,N", [(1, 8), (3, 1), (77, 1000), (4096, 40), (513, 2049), (9, 25600)])
def test_epilogue_backward(name, M, N):
    g = gen(M * 3 + N)
    dy, z = normal(g, M, N, 0.1, extra=8), normal(g, M, N, 2.0)
    out = torch.full((M, up(N, 8) + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    dz, db = fb.epilogue_backward(dy, z, activation=name, dz=out[:, :N])
    d = dy.double() * act(name, z.double())[1]
    e = 2.0 ** -20 * (1 + z.double().abs()) * dy.double().abs()
    within(dz, d, HALF * d.abs() + e + 1e-37, "dz")
    assert (out[:, N:] == 7.0).all()
    # FP32 sums: fewer than M/8 + 8 + 2368 additions, each half an FP32 step of the magnitudes
    within(db, d.sum(0), (M / 8 + 2400) * 2.0 ** -24 * d.abs().sum(0) + e.sum(0) + 1e-37, "dbias")
    again = fb.epilogue_backward(dy, z, activation=name)[1]
    assert torch.equal(db, again), "the sum's order is fixed"


def test_epilogue_backward_forms():
    g = gen(12)
    dy, z = normal(g, 50, 300), normal(g, 50, 300)
    want = fb.epilogue_backward(dy, z, activation="gelu")
    only = fb.epilogue_backward(dy, z, activation="gelu", bias_grad=False)
    assert only[1] is None and same_bits(only[0], want[0])
    a, b = rows(dy.clone()), rows(z.clone())
    assert same_bits(fb.epilogue_backward(a, z, activation="gelu", dz=a)[0], want[0])    # over dy
    assert same_bits(fb.epilogue_backward(dy, b, activation="gelu", dz=b)[0], want[0])   # over z
    same, db = fb.epilogue_backward(dy)
    assert same is dy
    within(db, dy.double().sum(0), 1e-4 * dy.double().abs().sum(0), "plain sums")
    copy = rows(torch.zeros_like(dy))
    assert same_bits(fb.epilogue_backward(dy, dz=copy, bias_grad=False)[0], dy)
    none = torch.empty((0, 40), dtype=torch.bfloat16, device=DEV)
    assert torch.equal(fb.epilogue_backward(none)[1], torch.zeros(40, device=DEV))


@pytest.mark.parametrize("N,K", [(1, 1), (3, 200), (128, 128), (130, 257), (1000, 1000), (384, 2048), (2051, 130)])
def test_transpose_weight(N, K):
    g = gen(N + K)
    q, s = weight(g, N, K)
    buf = torch.full((K, up(N, 16) + 16), 0xA5, dtype=torch.uint8, device=DEV)
    qt, st = fb.transpose_weight(q, s, qt=buf[:, :N])
    assert torch.equal(qt, q.t()) and torch.equal(st, s.t())
    assert (buf[:, N:] == 0xA5).all(), "wrote past N"
    q2, s2 = weight(g, N, K)
    both = torch.full((K, 2 * up(N, 128)), 0xA5, dtype=torch.uint8, device=DEV)
    qt, st = fb.transpose_gated_weights(q, s, q2, s2, qt=both)
    Np, NB = up(N, 128), -(-N // 128)
    assert torch.equal(qt[:, :N], q.t()) and torch.equal(qt[:, Np:Np + N], q2.t())
    assert not qt[:, N:Np].any() and not qt[:, Np + N:].any()
    assert torch.equal(st[:, :NB], s.t()) and torch.equal(st[:, NB:], s2.t())


GRAD_SHAPES = [(1, 8, 8), (1, 256, 256), (5, 1, 1), (16, 640, 512), (63, 257, 130), (64, 128, 384), (65, 300, 72),
               (77, 1000, 1000), (200, 2048, 640), (512, 1280, 2048), (1030, 520, 264), (4096, 384, 640), (2050, 257, 129), (20000, 40, 72)]


@pytest.mark.parametrize("M,N,K", GRAD_SHAPES)
@pytest.mark.parametrize("form", ["fp32", "add", "bf16"])
def test_linear_grad_weight(M, N, K, form):
    g = gen(M + N + K)
    dz, x = normal(g, M, N, 0.1, extra=8), normal(g, M, K, extra=8)
    dtype = torch.bfloat16 if form == "bf16" else torch.float32
    out = torch.full((N, up(K, 8) + 8), 7.0, dtype=dtype, device=DEV)
    before = torch.randn(N, K, generator=g).to(DEV)
    if form == "add":
        out[:, :K] = before
    fb.linear_grad_weight(dz, x, out=out[:, :K], accumulate=form == "add")
    want = dz.double().T @ x.double()
    tol = (M / 16 + 8) * 2.0 ** -22 * (dz.double().abs().T @ x.double().abs()) + 1e-37
    if form == "bf16":
        tol = tol + HALF * want.abs()
    if form == "add":
        want = want + before.double()
        tol = tol + 2.0 ** -23 * want.abs()
    within(out[:, :K], want, tol, form)
    assert (out[:, K:] == 7.0).all(), "wrote past K"


def test_linear_grad_weight_edges():
    g = gen(13)
    x, z = torch.empty((0, 40), dtype=torch.bfloat16, device=DEV), torch.empty((0, 24), dtype=torch.bfloat16, device=DEV)
    assert not fb.linear_grad_weight(z, x).any()
    out = torch.ones((24, 40), device=DEV)
    fb.linear_grad_weight(z, x, out=out, accumulate=True)
    assert (out == 1).all()
    dz, x = normal(g, 300, 520), normal(g, 300, 1000)
    first = fb.linear_grad_weight(dz, x)
    for _ in range(4):
        assert torch.equal(fb.linear_grad_weight(dz, x), first)
    # split over the tokens or whole: the same sums, in another order
    dz, x = normal(g, 1500, 520), normal(g, 1500, 300)
    assert fb.linear_grad_weight_workspace_size(1500, 520, 300) > 0
    split = fb.linear_grad_weight(dz, x)
    whole = fb.linear_grad_weight(dz, x, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    within(split, whole.double(), (1500 / 8 + 16) * 2.0 ** -22 * (dz.double().abs().T @ x.double().abs()), "split")


# ---------------------------------------------------------- used together
def block_reference(x, wg, wu, wd, dy):
    """The gated feed-forward block y = x' + down(silu(gate x) * up x) in
    float64: y's branch, and the gradients of <y, dy>."""
    g, u = x @ wg.T, x @ wu.T
    a, s = act("silu", g)
    h = a * u
    dh = dy @ wd
    dg, du = dh * u * s, dh * a
    return h @ wd.T, dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ h


@pytest.mark.parametrize("M,K,N", [(1, 256, 384), (77, 1000, 1000), (260, 640, 1280)])
def test_training_step_of_a_block(M, K, N):
    """Forward and backward of a whole block with the operators as a training
    step uses them; gradients against the formula's and against differences."""
    g = gen(M)
    x, res, dy = normal(g, M, K), normal(g, M, K), normal(g, M, K, 0.1)
    wg, wu, wd = weight(g, N, K, 0.05), weight(g, N, K, 0.05), weight(g, K, N, 0.05)
    Np = up(N, 128)
    kept = tuple(torch.empty((M, up(N, 8)), dtype=torch.bfloat16, device=DEV)[:, :N] for _ in range(2))
    h = fb.gated_linear_w8a16(x, *wg, *wu, preact=kept)
    y = fb.linear_w8a16_epilogue(h, *wd, residual=res)
    dz, _ = fb.epilogue_backward(dy, bias_grad=False)
    dh = fb.linear_w8a16(dz, *fb.transpose_weight(*wd))
    dwd = fb.linear_grad_weight(dz, h)
    dgu = fb.gated_backward(dh, *kept)
    dx = fb.linear_w8a16(dgu, *fb.transpose_gated_weights(*wg, *wu))
    dwg, dwu = (fb.linear_grad_weight(dgu[:, c:c + N], x) for c in (0, Np))

    wgd, wud, wdd = (dequantized(*w) for w in (wg, wu, wd))
    ref = block_reference(x.double(), wgd, wud, wdd, dy.double())

    def close(got, want, what, n):
        # n BF16 roundings on the way (each half a step of a term, independent):
        # relative Frobenius error of at most n half steps
        err = (got.double() - want).norm() / want.norm()
        assert err <= n * HALF, f"{what}: {err:.2e}"

    close(y.double() - res.double(), ref[0], "y", 2 + res.double().norm() / ref[0].norm())
    close(dx, ref[1], "dx", 5)      # g, u, dh, dg/du, dx
    close(dwg, ref[2], "dwg", 4)
    close(dwu, ref[3], "dwu", 4)
    close(dwd, ref[4], "dwd", 1)

    # differences of <y, dy> along random directions, in float64
    def loss(xx, a, b, c):
        gg, uu = xx @ a.T, xx @ b.T
        return ((act("silu", gg)[0] * uu) @ c.T * dy.double()).sum()

    args = [x.double(), wgd, wud, wdd]
    for i, grad in enumerate((dx, dwg, dwu, dwd)):
        v = grad.double() / grad.double().norm()   # along the gradient itself
        eps = 1e-4
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - eps * v, args[i] + eps * v
        slope = (loss(*hi) - loss(*lo)) / (2 * eps)
        assert abs(slope - grad.double().norm()) <= 5 * HALF * grad.double().norm(), i


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
def test_block_in_a_captured_graph_and_on_other_streams(mode):
    """The forward and backward calls captured into a graph, replayed on new
    inputs, and run on two side streams at once (each with its own
    workspace), give what eager calls give."""
    g = gen(21)
    M, K, N = 40, 640, 512
    wg, wu, wd = weight(g, N, K), weight(g, N, K), weight(g, K, N)
    wt, wdt = fb.transpose_gated_weights(*wg, *wu), fb.transpose_weight(*wd)
    lin = FUNCS["linear", mode]
    gat = FUNCS["gated", mode]

    def step(x, dy):
        kept = tuple(torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        h = gat(x, *wg, *wu, preact=kept)
        y = lin(h, *wd, residual=x)
        dz, db = fb.epilogue_backward(dy)
        dgu = fb.gated_backward(fb.linear_w8a16(dz, *wdt), *kept)
        return [h, y, db, dgu, fb.linear_w8a16(dgu, *wt), fb.linear_grad_weight(dgu[:, :N], x)]

    inputs = [(normal(g, M, K).contiguous(), normal(g, M, K).contiguous()) for _ in range(3)]
    want = [[t.clone() for t in step(*i)] for i in inputs]
    x, dy = inputs[0][0].clone(), inputs[0][1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, dy)
    for i, w in zip(inputs, want):
        x.copy_(i[0])
        dy.copy_(i[1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s, i in zip(streams, inputs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(step(*i))
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("M", [1, 64, 128, 700])
def test_repeated_calls_are_bit_identical(mode, M):
    """A race in a ring or in the gate/up trade shows up as differing rows."""
    g = gen(M)
    K, N = 2560, 9600
    x, wg, wu, r = normal(g, M, K), weight(g, N, K), weight(g, N, K), normal(g, M, N)
    for f in (lambda: FUNCS["gated", mode](x, *wg, *wu),
              lambda: FUNCS["linear", mode](x, *wg, activation="gelu", residual=r)):
        first = f()
        for _ in range(5):
            assert same_bits(f(), first)


@pytest.mark.parametrize("mode", ["w8a16", "w8a8"])
@pytest.mark.parametrize("name", ACTS)
def test_a_bad_weight_scale_shows(mode, name):
    """A scale of NaN is outside the contract, but it must not turn into numbers:
    its block's outputs are NaN and no others."""
    g = gen(40)
    M, K, N = 20, 384, 300
    x, (q, s), wu = normal(g, M, K), weight(g, N, K), weight(g, N, K)
    s[1, 2] = float("nan")
    y = FUNCS["linear", mode](x, q, s, activation=name)
    h = FUNCS["gated", mode](x, q, s, *wu, activation=name)
    for t in (y, h):
        assert torch.isnan(t[:, 128:256]).all()
        assert torch.isfinite(t[:, :128]).all() and torch.isfinite(t[:, 256:]).all()


@pytest.mark.parametrize("name", ACTS)
def test_a_nan_stays_one_backward(name):
    """A kept value of NaN reaches its own gradients and no others."""
    g = gen(41)
    M, N = 5, 140
    dh, z, u = normal(g, M, N), normal(g, M, N), normal(g, M, N)
    z[2, 7] = float("nan")
    here = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    here[2, 7] = True
    out = fb.gated_backward(dh, z, u, activation=name)
    at = lambda t: torch.equal(torch.isnan(t), here)
    assert at(out[:, 256:256 + N]), "du"
    if name in ("gelu", "gelu_tanh", "silu"):
        assert at(out[:, :N]) and at(fb.epilogue_backward(dh, z, activation=name, bias_grad=False)[0])
    else:       # slopes of 0 and 1
        assert torch.equal(out[2, 7].float(), (dh[2, 7].float() * u[2, 7].float()).to(torch.bfloat16).float())


def test_refusals_of_the_binding():
    g = gen(30)
    x, (q, s) = normal(g, 4, 256), weight(g, 200, 256)
    with pytest.raises(ValueError, match="activation"):
        fb.linear_w8a16_epilogue(x, q, s, activation="tanh")
    with pytest.raises(ValueError, match="residual"):
        fb.linear_w8a16_epilogue(x, q, s, residual=normal(g, 4, 199))
    with pytest.raises(ValueError, match="bias"):
        fb.linear_w8a16_epilogue(x, q, s, bias=torch.zeros(200, device=DEV))
    with pytest.raises(ValueError, match="codes"):
        fb.gated_linear_w8a8(x, q, s, q[:100], s)
    with pytest.raises(ValueError, match="scales"):
        fb.gated_linear_w8a8(x, q, s, q, s[:1])
    with pytest.raises(ValueError, match="x: expected torch.bfloat16"):
        fb.gated_linear_w8a16(x.float(), q, s, q, s)
    with pytest.raises(ValueError, match="stride"):
        fb.linear_w8a16_epilogue(x, q, s, residual=normal(g, 200, 4).t())
    with pytest.raises(ValueError, match="overlap"):
        fb.linear_w8a16_epilogue(x, q, s, residual=normal(g, 1, 200).expand(4, 200))
    with pytest.raises(ValueError, match="overlap"):
        fb.linear_grad_weight(x[:1].expand(4, 256), x)
    with pytest.raises(ValueError, match="z: needed"):
        fb.epilogue_backward(x, activation="gelu")
    with pytest.raises(ValueError, match="accumulate"):
        fb.linear_grad_weight(x, x, accumulate=True)
    with pytest.raises(fb.Fp8BlkError, match="WORKSPACE"):
        fb.gated_linear_w8a8(x, q, s, q, s, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
