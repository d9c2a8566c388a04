"""An output given the pointer of an input is refused before any launch (the addresses
below are never dereferenced): with the residual stream, out = x where inputs and
outputs have one size is an easy mistake, and tiles would read what others wrote."""
import pytest

import block_scaled_fp8_fp8blk_b200 as fb
from block_scaled_fp8_fp8blk_b200 import build as fbuild

A = [(i + 1) << 20 for i in range(12)]  # distinct addresses


@pytest.fixture(scope="module")
def lib():
    fbuild.build_cuda()
    return fb.lib()


def refused(f, names, values, pairs):
    """Every (output, input) pair with one pointer; the call with distinct ones is not made."""
    for out, inp in pairs:
        a = dict(zip(names.split(), values))
        a[out] = a[inp]
        assert f(*a.values()) == 1, (out, inp)


@pytest.mark.parametrize("mode", [0, 1])
def test_linear_epilogue(lib, mode):
    M, N, K = 64, 256, 256
    f = lib.fp8blk_linear_w8a8_epilogue if mode else lib.fp8blk_linear_w8a16_epilogue
    ws = fb.workspace_size(mode, M, N, K)

    def call(x=A[0], y=A[1], bias=A[2], residual=A[3], preact=A[4]):
        ep = fb.Epilogue(bias, 4, residual, N, preact, N)
        return f(x, K, A[5], K, A[6], y, N, M, N, K, ep, A[7], ws, None)

    assert call(y=A[0]) == 1 and call(preact=A[0]) == 1
    assert call(y=A[0], residual=A[0]) == 1                 # the residual stream updated in place
    assert call(y=A[5]) == 1 and call(y=A[6]) == 1 and call(preact=A[5]) == 1
    assert call(y=A[2]) == 1 and call(preact=A[2]) == 1 and call(preact=A[3]) == 1 and call(preact=A[1]) == 1


@pytest.mark.parametrize("mode", [0, 1])
def test_gated_linear(lib, mode):
    M, N, K = 64, 256, 256
    f = lib.fp8blk_gated_linear_w8a8 if mode else lib.fp8blk_gated_linear_w8a16
    refused(f, "x ldx qg sg qu su ldq act h ldh g u ldgu M N K ws wsb st",
            (A[0], K, A[1], A[2], A[3], A[4], K, 4, A[5], N, A[6], A[7], N, M, N, K, A[8],
             fb.workspace_size(mode, M, 2 * N, K), None),
            [("h", "g"), ("h", "u"), ("g", "u")] +
            [(out, inp) for out in "hgu" for inp in ("x", "qg", "sg", "qu", "su")])


def test_backward(lib):
    M, N, K = 64, 256, 256
    refused(lib.fp8blk_gated_backward, "dh lddh g u ldgu act dgu lddgu M N st",
            (A[0], N, A[1], A[2], N, 4, A[3], 512, M, N, None), [("dgu", "dh"), ("dgu", "g"), ("dgu", "u")])
    refused(lib.fp8blk_epilogue_backward, "dy lddy z ldz act dz lddz db M N ws wsb st",
            (A[0], N, A[1], N, 2, A[2], N, A[3], M, N, A[4], 1 << 20, None), [("db", "dy"), ("db", "z"), ("db", "dz")])
    refused(lib.fp8blk_transpose_weight, "q ldq s N K qt ldqt stt ldst pad st",
            (A[0], K, A[1], N, K, A[2], N, A[3], 2, 0, None), [("qt", "q"), ("stt", "s")])
    refused(lib.fp8blk_transpose_gated_weights, "qg sg qu su ldq N K qt ldqt stt st",
            (A[0], A[1], A[2], A[3], K, N, K, A[4], 2 * N, A[5], None),
            [("qt", "qg"), ("qt", "qu"), ("stt", "sg"), ("stt", "su")])
    refused(lib.fp8blk_linear_grad_weight, "dz lddz x ldx dw lddw fp32 add M N K ws wsb st",
            (A[0], N, A[1], K, A[2], K, 1, 0, M, N, K, None, 0, None), [("dw", "dz"), ("dw", "x")])
