"""The weight gradient where a pair of SMs walks several tiles: its two accumulators are
handed back and filled again, while the stages of the next tile run on. Compared in full,
and repeated bit for bit."""
import pytest
import torch

import block_scaled_fp8_fp8blk_b200 as fb
from test_feed_forward import DEV, HALF, gen, normal, up, within

pytestmark = pytest.mark.gpu

PAIRS = 74  # pairs of SMs of a B200: an accumulator is used again from the third tile of a pair on


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fb.read_device_error() == 0


# 800 tiles of 8 stages; 760 of 8, ragged on every side; 200 of 18; 216 of 1; 1600 of 2
SIZES = [(512, 5120, 10240), (500, 4841, 10001), (1100, 5120, 2560), (40, 3000, 4600), (100, 10240, 10240)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("form", ["fp32", "add", "bf16"])
def test_many_tiles_per_pair(M, N, K, form):
    assert up(N, 256) // 256 * (up(K, 256) // 256) > 2 * PAIRS
    g = gen(M + N + K)
    dz, x = normal(g, M, N, 0.1, extra=8), normal(g, M, K, extra=8)
    dtype = torch.bfloat16 if form == "bf16" else torch.float32
    out = torch.full((N + 3, up(K, 8) + 8), 7.0, dtype=dtype, device=DEV)
    before = torch.randn(N, K, generator=g).to(DEV) if form == "add" else None
    if form == "add":
        out[:N, :K] = before
    fb.linear_grad_weight(dz, x, out=out[:N, :K], accumulate=form == "add")
    want = dz.double().T @ x.double()
    # FP32 sums, 16 tokens a step: M / 16 + 8 roundings, each at most 2^-23 of the
    # magnitudes (a factor two to spare)
    tol = (M / 16 + 8) * 2.0 ** -22 * (dz.double().abs().T @ x.double().abs()) + 1e-37
    if form == "bf16":
        tol = tol + HALF * want.abs()
    if form == "add":
        want = want + before.double()
        tol = tol + 2.0 ** -23 * want.abs()
    within(out[:N, :K], want, tol, form)
    assert (out[:, K:] == 7.0).all() and (out[N:] == 7.0).all(), "wrote past the gradient"
    first = fb.linear_grad_weight(dz, x, dtype=dtype)
    if form != "add":
        assert torch.equal(first, out[:N, :K])
    for _ in range(4):
        assert torch.equal(fb.linear_grad_weight(dz, x, dtype=dtype), first)
