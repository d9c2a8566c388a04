"""Refusals of the feed-forward calls that need no GPU: bad arguments are
rejected before any CUDA call (addresses below are never dereferenced), and
the binding refuses tensors that are not on the current CUDA device."""
import pytest
import torch

import block_scaled_fp8_fp8blk_b200 as fb
from block_scaled_fp8_fp8blk_b200 import build as fbuild

P = 1 << 20
P2, P3, P4 = 2 << 20, 3 << 20, 4 << 20
PM = P + 2


@pytest.fixture(scope="module")
def lib():
    fbuild.build_cuda()
    return fb.lib()


def caller(f, names, values):
    def call(**kw):
        a = dict(zip(names, values))
        assert set(kw) <= set(a), set(kw) - set(a)
        a.update(kw)
        return f(*a.values())
    return call


@pytest.mark.parametrize("mode", [0, 1])
def test_linear_epilogue_validation(lib, mode):
    M, N, K = 64, 384, 256
    ws = fb.workspace_size(mode, M, N, K)
    names = "x ldx q ldq s y ldy M N K ep ws wsb st".split()
    f = lib.fp8blk_linear_w8a8_epilogue if mode else lib.fp8blk_linear_w8a16_epilogue

    def ep(**kw):
        d = dict(bias=P, activation=4, residual=P2, ldr=N, preact=P3, ldp=N)
        d.update(kw)
        return fb.Epilogue(*d.values())

    call = caller(f, names, (P, K, P, K, P, P4, N, M, N, K, ep(), P, ws, None))
    assert call(ep=None) == 1
    assert call(ep=ep(activation=5)) == 1 and call(ep=ep(activation=-1)) == 1
    assert call(M=-1) == 1 and call(x=None) == 1 and call(q=None) == 1 and call(y=None) == 1
    assert call(ldx=K - 8) == 1 and call(ldq=K - 16) == 1 and call(ldy=N - 8) == 1
    assert call(ldx=K + 4) == 2 and call(ldq=K + 8) == 2 and call(ldy=N + 4) == 2 and call(x=PM) == 2
    assert call(ep=ep(bias=P + 1)) == 2
    assert call(ep=ep(ldr=N - 8)) == 1 and call(ep=ep(ldr=N + 4)) == 2 and call(ep=ep(residual=PM)) == 2
    assert call(ep=ep(ldp=N - 8)) == 1 and call(ep=ep(ldp=N + 4)) == 2 and call(ep=ep(preact=PM)) == 2
    assert call(ep=ep(residual=P4, ldr=N + 8)) == 1        # over y, but with another stride
    assert call(ep=ep(preact=P4)) == 1 and call(ep=ep(preact=P2)) == 1
    assert call(ws=None) == 4 and call(wsb=ws - 1) == 4 and call(ws=P + 16) == 4
    assert call(M=0) == 0 and call(N=0) == 0
    assert call(M=0, ep=ep(activation=9)) == 1


@pytest.mark.parametrize("mode", [0, 1])
def test_gated_linear_validation(lib, mode):
    M, N, K = 64, 200, 256
    ws = fb.workspace_size(mode, M, 2 * N, K)
    names = "x ldx qg sg qu su ldq act h ldh g u ldgu M N K ws wsb st".split()
    f = lib.fp8blk_gated_linear_w8a8 if mode else lib.fp8blk_gated_linear_w8a16
    call = caller(f, names, (P, K, P, P, P, P, K, 4, P, N, P2, P3, N, M, N, K, P, ws, None))
    assert call(act=7) == 1 and call(M=-1) == 1 and call(N=2 ** 31) == 1
    for n in ("x", "qg", "sg", "qu", "su", "h"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: P + 1}) == 2, n
    assert call(g=None) == 1 and call(u=None) == 1 and call(u=P2) == 1 and call(g=P) == 1
    assert call(ldgu=N - 8) == 1 and call(ldgu=N + 4) == 2 and call(g=PM) == 2
    assert call(ldh=N - 8) == 1 and call(ldq=K - 16) == 1 and call(ldq=K + 8) == 2
    assert call(ws=None) == 4 and call(wsb=ws - 1) == 4
    assert call(M=0) == 0 and call(N=0) == 0


def test_gated_backward_validation(lib):
    M, N = 64, 200
    names = "dh lddh g u ldgu act dgu lddgu M N st".split()
    call = caller(lib.fp8blk_gated_backward, names, (P, N, P, P, N, 4, P, 512, M, N, None))
    assert call(act=5) == 1 and call(M=-1) == 1 and call(N=-1) == 1 and call(M=2 ** 31) == 1
    for n in ("dh", "g", "u", "dgu"):
        assert call(**{n: None}) == 1 and call(**{n: PM}) == 2
    assert call(lddh=N - 8) == 1 and call(ldgu=N - 8) == 1 and call(lddgu=504) == 1
    assert call(lddh=N + 4) == 2 and call(ldgu=N + 4) == 2 and call(lddgu=516) == 2
    assert call(M=0) == 0 and call(N=0) == 0


def test_epilogue_backward_validation(lib):
    M, N = 640, 200
    ws = fb.epilogue_backward_workspace_size(M, N)
    assert ws > 0 and fb.epilogue_backward_workspace_size(-1, N) == 0
    assert fb.epilogue_backward_workspace_size(8, N) == 0          # one run of rows: no partial sums
    names = "dy lddy z ldz act dz lddz db M N ws wsb st".split()
    call = caller(lib.fp8blk_epilogue_backward, names, (P, N, P2, N, 2, P3, N, P, M, N, P, ws, None))
    assert call(act=5) == 1 and call(M=-1) == 1 and call(N=2 ** 31) == 1
    assert call(dy=None) == 1 and call(z=None) == 1
    assert call(lddy=N - 8) == 1 and call(ldz=N - 8) == 1 and call(lddz=N - 8) == 1
    assert call(lddy=N + 4) == 2 and call(ldz=N + 4) == 2 and call(lddz=N + 4) == 2
    assert call(dy=PM) == 2 and call(z=PM) == 2 and call(dz=PM) == 2 and call(db=PM) == 2
    assert call(dz=P, lddz=N + 8) == 1 and call(dz=P2, lddz=N + 8) == 1   # in place, other stride
    assert call(ws=None) == 4 and call(wsb=ws - 1) == 4 and call(ws=P + 16) == 4
    assert call(N=0) == 0 and call(M=0, db=None) == 0
    assert call(act=0, dz=P, db=None) == 0                         # dz = dy already: nothing to do


def test_transpose_weight_validation(lib):
    N, K = 200, 300
    names = "q ldq s N K qt ldqt stt ldst pad st".split()
    call = caller(lib.fp8blk_transpose_weight, names, (P, 304, P, N, K, P, 256, P, 2, 1, None))
    assert call(N=-1) == 1 and call(pad=2) == 1
    for n in ("q", "s", "qt", "stt"):
        assert call(**{n: None}) == 1 and call(**{n: P + 1}) == 2
    assert call(ldq=288) == 1 and call(ldq=312) == 2
    assert call(ldqt=208) == 1 and call(ldqt=264) == 2 and call(ldst=1) == 1
    assert call(N=0) == 0 and call(K=0) == 0


def test_transpose_gated_weights_validation(lib):
    N, K = 200, 300
    names = "qg sg qu su ldq N K qt ldqt stt st".split()
    call = caller(lib.fp8blk_transpose_gated_weights, names, (P, P, P, P, 304, N, K, P, 512, P, None))
    assert call(N=-1) == 1 and call(K=-1) == 1
    for n in ("qg", "sg", "qu", "su", "qt", "stt"):
        assert call(**{n: None}) == 1 and call(**{n: P + 1}) == 2
    assert call(ldq=288) == 1 and call(ldq=312) == 2 and call(ldqt=496) == 1 and call(ldqt=520) == 2
    assert call(N=0) == 0 and call(K=0) == 0


def test_linear_grad_weight_validation(lib):
    M, N, K = 64, 200, 304
    names = "dz lddz x ldx dw lddw fp32 add M N K ws wsb st".split()
    call = caller(lib.fp8blk_linear_grad_weight, names, (P, N, P, K, P, K, 1, 0, M, N, K, None, 0, None))
    assert call(M=-1) == 1 and call(fp32=2) == 1 and call(add=2) == 1
    assert call(fp32=0, add=1) == 1                                # sums are added in FP32 only
    assert call(dz=None) == 1 and call(x=None) == 1 and call(dw=None) == 1
    assert call(lddz=N - 8) == 1 and call(ldx=K - 8) == 1 and call(lddw=K - 8) == 1
    assert call(lddz=N + 4) == 2 and call(ldx=K + 4) == 2 and call(lddw=K + 2) == 2
    assert call(fp32=0, lddw=K + 4) == 2
    assert call(dz=PM) == 2 and call(x=PM) == 2 and call(dw=PM) == 2
    assert call(N=0) == 0 and call(K=0) == 0 and call(M=0, add=1) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    q, s = torch.zeros((128, 128), dtype=torch.uint8), torch.zeros((1, 1))
    for f in (lambda: fb.linear_w8a16_epilogue(x, q, s), lambda: fb.linear_w8a8_epilogue(x, q, s),
              lambda: fb.gated_linear_w8a16(x, q, s, q, s), lambda: fb.gated_linear_w8a8(x, q, s, q, s),
              lambda: fb.gated_backward(x, x, x), lambda: fb.epilogue_backward(x),
              lambda: fb.transpose_weight(q, s), lambda: fb.transpose_gated_weights(q, s, q, s),
              lambda: fb.linear_grad_weight(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_overlapping_rows_are_refused():
    """A broadcast tensor has row stride 0: its rows are not [rows, cols] memory."""
    wide = torch.zeros((1, 128), dtype=torch.bfloat16).expand(4, 128)
    with pytest.raises(ValueError, match="overlap"):
        fb._ld(wide)
    assert fb._ld(torch.zeros((1, 128)).expand(1, 128)) == 128
    assert fb._ld(torch.zeros((3, 1)).expand(3, 1)) == 1 and fb._ld(torch.zeros((0, 5))) == 5


def test_linear_grad_weight_workspace_size(lib):
    """A workspace where few 256 x 256 tiles meet many tokens: runs of at least
    eight 64-token stages, all (tile, run) units at once on 74 pairs of SMs."""
    size = fb.linear_grad_weight_workspace_size
    assert size(4096, 25600, 5120) == 0 and size(200, 256, 256) == 0 and size(-1, 8, 8) == 0
    assert size(2048, 1024, 1024) == 4 * 1024 * 1024 * 4        # 16 tiles: 4 runs of 8 stages
    assert size(1023, 256, 256) == 2 * 256 * 256 * 4            # 16 stages: 2 runs of 8
    assert size(960, 256, 256) == 0                             # 15 stages
    assert size(4096, 300, 130) == 8 * 512 * 132 * 4            # rows and columns padded
    assert size(1 << 20, 1, 1) == 74 * 256 * 4 * 4 and size(4096, 0, 130) == 0
