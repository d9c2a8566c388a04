"""Tiles shared by several SMs, element by element against float64: the W8A16 split
and its fix-up with an epilogue (up to 128 tokens), and the W8A8 clusters of two.
test_schedule.py checks on the host that the rules do split these sizes so.

The bounds are those of test_feed_forward.py; a split adds at most one FP32 addition per
slab, 2^-24 of the sum of magnitudes each."""
import pytest
import torch

import block_scaled_fp8_fp8blk_b200 as fb
from test_feed_forward import (DEV, FP32, FUNCS, HALF, SLOPE, acc, act, activations, dequantized, gen, normal,
                               run_gated, run_linear, same_bits, up, weight, within)

# (tokens, inputs, outputs of the linear; the gated pair has half as many)
W8A16_SPLIT = [(M, K, N) for M in (1, 16, 20, 50, 100, 128)
               for K, N in ((8192, 640), (4100, 1000), (8192, 5120), (4100, 25630))]
W8A16_LAST_WAVE = [(300, 4100, 1000), (129, 8192, 642), (700, 1000, 5000)]
W8A8_TWO = [(16, 8192, 16384), (200, 5000, 8100), (130, 6000, 8000), (1, 5000, 16900)]


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fb.read_device_error() == 0


def nans(mode, M, N, K):
    return torch.full((max(1, fb.workspace_size(mode, M, N, K) // 4),), float("nan"), device=DEV)


def buffer(M, N):
    return torch.full((M, up(N, 8) + 8), 7.0, dtype=torch.bfloat16, device=DEV)


def adds(K):
    return acc(K) + K / 128 * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", W8A16_SPLIT + W8A16_LAST_WAVE)
def test_w8a16_split_linear(M, K, N):
    """Bias, gelu, z kept and the residual updated in place, then a residual alone; the
    partials' workspace starts as NaN."""
    g = gen(M + K + N)
    x, w = normal(g, M, K), weight(g, N, K)
    b = normal(g, 1, N, 0.5)[0].contiguous()
    r = normal(g, M, N)
    y, z = buffer(M, N), buffer(M, N)
    y[:, :N] = r
    fb.linear_w8a16_epilogue(x, *w, bias=b, activation="gelu", residual=y[:, :N], preact=z[:, :N], out=y[:, :N],
                             workspace=nans(0, M, N, K))
    xd, wd = x.double(), dequantized(*w)
    sd, size = xd @ wd.T, xd.abs() @ wd.abs().T
    zd = sd + b.double()
    ez = adds(K) * size + 2.0 ** -23 * zd.abs()
    a = act("gelu", zd)[0]
    want = a + r.double()
    within(z[:, :N], zd, HALF * zd.abs() + 1.01 * ez + 1e-37, "z")
    within(y[:, :N], want, HALF * want.abs() + FP32 * (a.abs() + want.abs()) + SLOPE * ez + 1e-37, "y")
    assert (y[:, N:] == 7.0).all() and (z[:, N:] == 7.0).all(), "wrote past N"
    only = fb.linear_w8a16_epilogue(x, *w, residual=r, workspace=nans(0, M, N, K))
    want = sd + r.double()
    within(only, want, HALF * want.abs() + adds(K) * size + 2.0 ** -23 * want.abs() + 1e-37, "residual alone")
    for _ in range(3):
        assert same_bits(only, fb.linear_w8a16_epilogue(x, *w, residual=r, workspace=nans(0, M, N, K)))


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", W8A16_SPLIT + W8A16_LAST_WAVE)
def test_w8a16_split_gated(M, K, N):
    """g and u kept, and without them; the partials' workspace starts as NaN."""
    N //= 2
    g = gen(M + K + N)
    x, wg, wu = normal(g, M, K), weight(g, N, K), weight(g, N, K)
    h, kg, ku = (buffer(M, N) for _ in range(3))
    fb.gated_linear_w8a16(x, *wg, *wu, out=h[:, :N], preact=(kg[:, :N], ku[:, :N]), workspace=nans(0, M, 2 * N, K))
    xd, dg, du = x.double(), dequantized(*wg), dequantized(*wu)
    gd, ud = xd @ dg.T, xd @ du.T
    eg, eu = (adds(K) * (xd.abs() @ d.abs().T) for d in (dg, du))
    a = act("silu", gd)[0]
    want = a * ud
    tol = (HALF + FP32) * want.abs() + SLOPE * eg * (ud.abs() + eu) + a.abs() * eu + 1e-37
    within(kg[:, :N], gd, HALF * gd.abs() + 1.01 * eg + 1e-37, "g")
    within(ku[:, :N], ud, HALF * ud.abs() + 1.01 * eu + 1e-37, "u")
    within(h[:, :N], want, tol, "h")
    assert all((t[:, N:] == 7.0).all() for t in (h, kg, ku)), "wrote past N"
    for _ in range(3):
        assert same_bits(h[:, :N], fb.gated_linear_w8a16(x, *wg, *wu, workspace=nans(0, M, 2 * N, K)))


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", W8A8_TWO)
def test_w8a8_clusters_of_two(M, K, N):
    run_linear("w8a8", M, K, N, "silu", bias=True, keep=True, in_place=True, seed=K)
    run_gated("w8a8", M, K, N // 2, "gelu", keep=True, seed=K + 2)
    x, w, first = run_linear("w8a8", M, K, N, "gelu", residual=False, seed=K + 3)
    x2, wg, wu, h, _ = run_gated("w8a8", M, K, N // 2, "silu", seed=K + 4)
    for _ in range(3):
        assert same_bits(fb.linear_w8a8_epilogue(x, *w, activation="gelu"), first)
        assert same_bits(fb.gated_linear_w8a8(x2, *wg, *wu), h)
