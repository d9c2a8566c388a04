"""W8A16 above 128 tokens whose last wave of tiles has fewer K slabs than the
GPU has SMs: the split of those slabs must leave no SM without one inside a
split tile, or the fix-up adds a partial that nobody wrote."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_fp8blk_b200 as fb
import oracle
from block_scaled_fp8_fp8blk_b200 import workloads as W
from helpers import bf16_to_f64, check_linear, weight_bits, x_bits

DEV = "cuda:0"


def ranges(U, G):
    return [(U * c // G, U * (c + 1) // G) for c in range(G)]


@pytest.mark.parametrize("U", [1, 2, 5, 10, 40, 147, 148, 149, 1000])
def test_every_sharing_sm_has_a_slab(U):
    """The rule on the host: min(SMs, slabs) SMs share, each has at least one
    slab, and together they cover all of them in order."""
    S = min(148, U)
    r = ranges(U, S)
    assert all(a < b for a, b in r)
    assert r[0][0] == 0 and r[-1][1] == U and all(r[i][1] == r[i + 1][0] for i in range(S - 1))


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(512, 640, 19000), (300, 128, 19000), (512, 1000, 9500)])
def test_last_wave_with_few_slabs(M, K, N):
    torch.cuda.set_device(0)
    wl = W.Workload(f"m{M}_k{K}_n{N}", M, K, N)
    wb, xb = weight_bits(wl), x_bits(wl)
    q, s = oracle.quantize_weight(wb)
    x, w = wl.x_bf16().to(DEV), wl.weight_bf16().to(DEV)
    q_d, s_d = fb.quantize_weight(w)
    ws = torch.full((fb.workspace_size(0, M, N, K) // 4,), float("nan"), device=DEV)
    y = fb.linear_w8a16(x, q_d, s_d, workspace=ws)
    rows = np.arange(0, M, 37)
    check_linear(bf16_to_f64(y)[rows], oracle.linear_w8a16(xb, q, s, N, K, rows=rows), wl.name)
    assert fb.read_device_error() == 0
