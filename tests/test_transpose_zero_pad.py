"""The transposed weight with its columns padded to whole blocks."""
import pytest
import torch

import block_scaled_fp8_fp8blk_b200 as fb
from test_feed_forward import DEV, gen, normal, same_bits, up, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fb.read_device_error() == 0


@pytest.mark.parametrize("N,K", [(1, 1), (3, 200), (128, 128), (130, 257), (1000, 1000), (383, 2048), (2051, 130)])
def test_columns_past_n_are_zero(N, K):
    q, s = weight(gen(N + K), N, K)
    Np = up(N, 128)
    buf = torch.full((K + 3, Np + 32), 0xA5, dtype=torch.uint8, device=DEV)
    qt, st = fb.transpose_weight(q, s, qt=buf[:K, :Np], zero_pad=True)
    assert torch.equal(qt[:, :N], q.t()) and torch.equal(st, s.t())
    assert not qt[:, N:].any()
    assert (buf[:, Np:] == 0xA5).all() and (buf[K:] == 0xA5).all(), "wrote past the padding"
    made, made_s = fb.transpose_weight(q, s, zero_pad=True)
    assert made.shape == (K, Np) and torch.equal(made, qt) and torch.equal(made_s, st)


def test_a_padded_operand_gives_the_same_product():
    """dz in a buffer of whole blocks with ones behind its columns."""
    g = gen(5)
    M, N, K = 40, 300, 512
    q, s = weight(g, N, K)
    dz = torch.ones((M, up(N, 128)), dtype=torch.bfloat16, device=DEV)
    dz[:, :N] = normal(g, M, N)
    want = fb.linear_w8a16(dz[:, :N], *fb.transpose_weight(q, s))
    assert same_bits(fb.linear_w8a16(dz, *fb.transpose_weight(q, s, zero_pad=True)), want)


def test_refusals():
    q, s = weight(gen(6), 200, 256)
    with pytest.raises(ValueError, match="codes"):
        fb.transpose_weight(q, s, qt=torch.empty((256, 208), dtype=torch.uint8, device=DEV)[:, :200], zero_pad=True)
    with pytest.raises(ValueError, match="codes"):
        fb.transpose_weight(q, s, qt=torch.empty((256, 256), dtype=torch.uint8, device=DEV))
