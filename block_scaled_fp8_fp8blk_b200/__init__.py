"""Python binding of the fp8blk C ABI (``include/fp8blk.h``).

Argument marshalling only: every step runs in ``libfp8blk.so`` (hand-written
sm_100a kernels). PyTorch supplies device memory and the current stream.
There is no fallback: if the library is missing or the device is not
compute capability 10.x, the calls raise.

Tensors are 2-D, row-major with unit column stride; the row stride is the
leading dimension, so padded buffers are passed as column slices of a wider
tensor (e.g. ``q = buf[:, :K]`` with ``buf`` of shape ``[N, ldq]``).
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "Fp8BlkError", "lib", "quantize_weight", "dequantize", "quantize_act", "linear_w8a16",
    "linear_w8a8", "linear_w8a8_quantized", "workspace_size", "encode_e4m3", "read_device_error",
    "version", "LinearJob", "stream_slot_bytes", "streamed_linears", "selftest_wait_timeout",
    "LinearArgs", "linear_sequence",
    "ACTIVATIONS", "Epilogue", "linear_w8a16_epilogue", "linear_w8a8_epilogue",
    "gated_linear_w8a16", "gated_linear_w8a8", "gated_backward", "epilogue_backward",
    "epilogue_backward_workspace_size", "transpose_weight", "transpose_gated_weights",
    "linear_grad_weight", "linear_grad_weight_workspace_size",
    "LIB_PATH", "EXPORTS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8blk.so")

STATUS = {
    0: "FP8BLK_OK", 1: "FP8BLK_ERR_INVALID_ARG", 2: "FP8BLK_ERR_ALIGNMENT",
    3: "FP8BLK_ERR_UNSUPPORTED_DEVICE", 4: "FP8BLK_ERR_WORKSPACE", 5: "FP8BLK_ERR_CUDA",
    6: "FP8BLK_ERR_TIMEOUT",
}

_i64, _p, _sz, _int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_st = ctypes.c_int


class LinearJob(ctypes.Structure):
    """fp8blk_linear_job: one linear of a streamed sequence (host weights)."""
    _fields_ = [("mode", ctypes.c_int32), ("q_host", _p), ("scale_host", _p), ("ldq", _i64),
                ("x", _p), ("ldx", _i64), ("y", _p), ("ldy", _i64),
                ("M", _i64), ("N", _i64), ("K", _i64)]


class LinearArgs(ctypes.Structure):
    """fp8blk_linear_args: one linear of a sequence (device weights)."""
    _fields_ = [("mode", ctypes.c_int32), ("x", _p), ("ldx", _i64), ("q", _p), ("ldq", _i64),
                ("scale_inv", _p), ("y", _p), ("ldy", _i64), ("M", _i64), ("N", _i64), ("K", _i64)]


class Epilogue(ctypes.Structure):
    """fp8blk_epilogue: what follows a linear's product."""
    _fields_ = [("bias", _p), ("activation", ctypes.c_int32), ("residual", _p), ("ldr", _i64),
                ("preact", _p), ("ldp", _i64)]


# fp8blk_activation by name
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_i32 = ctypes.c_int32
_linear_epilogue_args = [_p, _i64, _p, _i64, _p, _p, _i64, _i64, _i64, _i64,
                         ctypes.POINTER(Epilogue), _p, _sz, _p]
_gated_linear_args = [_p, _i64, _p, _p, _p, _p, _i64, _i32, _p, _i64, _p, _p, _i64, _i64, _i64, _i64,
                      _p, _sz, _p]

# name -> (restype, argtypes), mirroring include/fp8blk.h
EXPORTS = {
    "fp8blk_quantize_weight": (_st, [_p, _i64, _i64, _i64, _p, _i64, _p, _p]),
    "fp8blk_dequantize": (_st, [_p, _i64, _p, _i64, _i64, _p, _i64, _p]),
    "fp8blk_quantize_act": (_st, [_p, _i64, _i64, _i64, _p, _i64, _p, _i64, _p]),
    "fp8blk_linear_w8a16": (_st, [_p, _i64, _p, _i64, _p, _p, _i64, _i64, _i64, _i64, _p, _sz, _p]),
    "fp8blk_linear_w8a8": (_st, [_p, _i64, _p, _i64, _p, _p, _i64, _i64, _i64, _i64, _p, _sz, _p]),
    "fp8blk_linear_w8a8_noalloc": (_st, [_p, _i64, _p, _i64, _p, _p, _i64, _i64, _i64, _i64, _p]),
    "fp8blk_linear_w8a8_quantized": (_st, [_p, _i64, _p, _i64, _p, _i64, _p, _p, _i64, _i64, _i64, _i64, _p]),
    "fp8blk_workspace_size": (_sz, [_int, _i64, _i64, _i64]),
    "fp8blk_stream_slot_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8blk_linear_sequence": (_st, [ctypes.POINTER(LinearArgs), _i64, _p, _sz, _p]),
    "fp8blk_streamed_linears": (_st, [ctypes.POINTER(LinearJob), _i64, _p, _sz, ctypes.c_int32,
                                      _p, _sz, _p, _p, ctypes.POINTER(_p)]),
    "fp8blk_linear_w8a16_epilogue": (_st, _linear_epilogue_args),
    "fp8blk_linear_w8a8_epilogue": (_st, _linear_epilogue_args),
    "fp8blk_gated_linear_w8a16": (_st, _gated_linear_args),
    "fp8blk_gated_linear_w8a8": (_st, _gated_linear_args),
    "fp8blk_gated_backward": (_st, [_p, _i64, _p, _p, _i64, _i32, _p, _i64, _i64, _i64, _p]),
    "fp8blk_epilogue_backward": (_st, [_p, _i64, _p, _i64, _i32, _p, _i64, _p, _i64, _i64, _p, _sz, _p]),
    "fp8blk_epilogue_backward_workspace_size": (_sz, [_i64, _i64]),
    "fp8blk_transpose_weight": (_st, [_p, _i64, _p, _i64, _i64, _p, _i64, _p, _i64, _i32, _p]),
    "fp8blk_transpose_gated_weights": (_st, [_p, _p, _p, _p, _i64, _i64, _i64, _p, _i64, _p, _p]),
    "fp8blk_linear_grad_weight": (_st, [_p, _i64, _p, _i64, _p, _i64, _i32, _i32, _i64, _i64, _i64, _p,
                                        _sz, _p]),
    "fp8blk_linear_grad_weight_workspace_size": (_sz, [_i64, _i64, _i64]),
    "fp8blk_encode_e4m3": (_st, [_p, _i64, _p, _p]),
    "fp8blk_read_device_error": (_st, [ctypes.POINTER(ctypes.c_uint32)]),
    "fp8blk_selftest_wait_timeout": (_st, [_i64, _p]),
    "fp8blk_status_string": (ctypes.c_char_p, [_int]),
    "fp8blk_version": (_int, []),
}

_lib = None


class Fp8BlkError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call} failed: {STATUS.get(status, status)}")


def lib() -> ctypes.CDLL:
    """The loaded libfp8blk.so (loaded once; raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "python -m block_scaled_fp8_fp8blk_b200.build")
        import torch  # noqa: F401  (loads the CUDA runtime the library shares)
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(handle, name)
            f.restype, f.argtypes = res, args
        _lib = handle
    return _lib


def _check(status: int, call: str) -> None:
    if status != 0:
        raise Fp8BlkError(status, call)


def _cdiv(a: int, b: int) -> int:
    return -(-a // b)


def _round_up(a: int, b: int) -> int:
    return _cdiv(a, b) * b


def _stream():
    """The raw handle of the current stream of the current CUDA device."""
    import torch
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ld(t) -> int:
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError("expected unit column stride")
    if ld >= cols:
        return ld or 1
    if rows > 1:
        raise ValueError("rows overlap: expected a row stride of at least the columns")
    return cols or 1


def _padded(rows: int, cols: int, ld: int, dtype, device):
    import torch
    buf = torch.empty((rows, ld), dtype=dtype, device=device)
    return buf if ld == cols else buf[:, :cols]


def version() -> int:
    return int(lib().fp8blk_version())


def workspace_size(mode: int, M: int, N: int, K: int) -> int:
    return int(lib().fp8blk_workspace_size(mode, M, N, K))


def quantize_weight(w, q=None, scale_inv=None, ldq: int | None = None):
    """BF16 w [N, K] -> (q uint8 [N, K] with row stride ldq, scale_inv float32 [NB, KB])."""
    import torch
    N, K = w.shape
    if q is None:
        q = _padded(N, K, ldq or _round_up(max(K, 1), 16), torch.uint8, w.device)
    if scale_inv is None:
        scale_inv = torch.empty((_cdiv(N, 128), _cdiv(K, 128)), dtype=torch.float32, device=w.device)
    _check(lib().fp8blk_quantize_weight(w.data_ptr(), N, K, _ld(w), q.data_ptr(), _ld(q),
                                        scale_inv.data_ptr(), _stream()), "fp8blk_quantize_weight")
    return q, scale_inv


def dequantize(q, scale_inv, out=None):
    import torch
    N, K = q.shape
    if out is None:
        out = _padded(N, K, _round_up(max(K, 1), 8), torch.bfloat16, q.device)
    _check(lib().fp8blk_dequantize(q.data_ptr(), _ld(q), scale_inv.data_ptr(), N, K,
                                   out.data_ptr(), _ld(out), _stream()), "fp8blk_dequantize")
    return out


def quantize_act(x, qx=None, sx=None):
    """BF16 x [M, K] -> (qx uint8 [M, K], sx float32 [KB, ldsx] with ldsx = round_up(M, 4))."""
    import torch
    M, K = x.shape
    if qx is None:
        qx = _padded(M, K, _round_up(max(K, 1), 16), torch.uint8, x.device)
    if sx is None:
        sx = torch.empty((_cdiv(K, 128), _round_up(max(M, 1), 4)), dtype=torch.float32, device=x.device)
    _check(lib().fp8blk_quantize_act(x.data_ptr(), M, K, _ld(x), qx.data_ptr(), _ld(qx),
                                     sx.data_ptr(), sx.stride(0), _stream()), "fp8blk_quantize_act")
    return qx, sx


def _linear(mode: int, name: str, x, q, scale_inv, out, workspace):
    import torch
    M, K = x.shape
    N = q.shape[0]
    if q.shape[1] != K:
        raise ValueError("x and q disagree on K")
    if out is None:
        out = _padded(M, N, _round_up(max(N, 1), 8), torch.bfloat16, x.device)
    if workspace is None:
        need = workspace_size(mode, M, N, K)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(getattr(lib(), name)(x.data_ptr(), _ld(x), q.data_ptr(), _ld(q), scale_inv.data_ptr(),
                                out.data_ptr(), _ld(out), M, N, K, ws_ptr, ws_len, _stream()), name)
    return out


def linear_w8a16(x, q, scale_inv, out=None, workspace=None):
    """y = x . dequant(q, scale_inv)^T with BF16 activations; y BF16 [M, N]."""
    return _linear(0, "fp8blk_linear_w8a16", x, q, scale_inv, out, workspace)


def linear_w8a8(x, q, scale_inv, out=None, workspace=None):
    """y = x . dequant(q, scale_inv)^T with x quantized per 1x128 K-group to E4M3."""
    return _linear(1, "fp8blk_linear_w8a8", x, q, scale_inv, out, workspace)


def linear_w8a8_quantized(qx, sx, q, scale_inv, M=None, out=None):
    """W8A8 linear on (qx, sx) from quantize_act; M defaults to qx.shape[0]."""
    import torch
    M = qx.shape[0] if M is None else M
    K = qx.shape[1]
    N = q.shape[0]
    if out is None:
        out = _padded(M, N, _round_up(max(N, 1), 8), torch.bfloat16, qx.device)
    _check(lib().fp8blk_linear_w8a8_quantized(qx.data_ptr(), _ld(qx), sx.data_ptr(), sx.stride(0),
                                              q.data_ptr(), _ld(q), scale_inv.data_ptr(),
                                              out.data_ptr(), _ld(out), M, N, K, _stream()),
           "fp8blk_linear_w8a8_quantized")
    return out


def linear_sequence(jobs, workspace=None):
    """Runs linears back to back with their weight streams overlapping the
    kernels before them (fp8blk_linear_sequence). jobs: list of
    (mode, x, q, scale_inv, y) with mode 0 = W8A16, 1 = W8A8, all CUDA
    tensors as for linear_w8a16 / linear_w8a8. The workspace (allocated here
    if None) must cover the largest workspace_size over the jobs."""
    import torch
    arr = (LinearArgs * max(1, len(jobs)))()
    need = 0
    for i, (mode, x, q, s, y) in enumerate(jobs):
        M, K = x.shape
        N = q.shape[0]
        if q.shape[1] != K or y.shape != (M, N):
            raise ValueError("job shapes disagree")
        arr[i] = LinearArgs(mode, x.data_ptr(), _ld(x), q.data_ptr(), _ld(q), s.data_ptr(),
                            y.data_ptr(), _ld(y), M, N, K)
        need = max(need, workspace_size(mode, M, N, K))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=jobs[0][1].device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().fp8blk_linear_sequence(arr, len(jobs), ws_ptr, ws_len, _stream()),
           "fp8blk_linear_sequence")


def stream_slot_bytes(N: int, K: int, ldq: int) -> int:
    return lib().fp8blk_stream_slot_bytes(N, K, ldq)


def streamed_linears(jobs, slots, slot_bytes: int, nslots: int, workspace, compute, copy, events):
    """Run linears whose weights are in (pinned) host memory through nslots
    device weight slots (fp8blk_streamed_linears).

    jobs: list of (mode, q_host, s_host, x, y) with mode 0 = W8A16, 1 = W8A8,
    q_host uint8 [N, K] / s_host float32 (CPU tensors, pinned for overlap;
    q_host's row stride is ldq), x BF16 [M, K] and y BF16 [M, N] on the GPU.
    slots: uint8 CUDA tensor of nslots * slot_bytes; compute / copy:
    torch.cuda.Stream; events: 2 * nslots torch.cuda.Event (created here by
    a first record on `compute` if they have no handle yet).
    """
    arr = (LinearJob * max(1, len(jobs)))()
    for i, (mode, qh, sh, x, y) in enumerate(jobs):
        M, K = x.shape
        N = qh.shape[0]
        if qh.shape[1] != K or y.shape != (M, N):
            raise ValueError("job shapes disagree")
        arr[i] = LinearJob(mode, qh.data_ptr(), sh.data_ptr(), _ld(qh), x.data_ptr(), _ld(x),
                           y.data_ptr(), _ld(y), M, N, K)
    for e in events:
        if not e.cuda_event:
            e.record(compute)
    ev = (_p * max(1, len(events)))(*[e.cuda_event for e in events])
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().fp8blk_streamed_linears(arr, len(jobs), slots.data_ptr(), slot_bytes, nslots,
                                         ws_ptr, ws_len, compute.cuda_stream, copy.cuda_stream, ev),
           "fp8blk_streamed_linears")


# ------------------------------------------------- feed-forward operators
# (Small layers are bound by the host: the checks below read each tensor's
# properties once, and work out a message only for a refusal.)
def _matrix(t, rows, cols, dtype, dev, what):
    """Leading dimension of a 2-D operand [rows, cols] of the dtype on CUDA device dev."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == (rows, cols):
        ld, step = t.stride()
        if step != 1 and cols > 1:
            raise ValueError(f"{what}: expected unit column stride")
        if ld >= cols:
            return ld or 1
        if rows > 1:
            raise ValueError(f"{what}: rows overlap (row stride {ld}, {cols} columns)")
        return cols or 1
    if t.dtype is not dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, expected cuda:{dev}")
    raise ValueError(f"{what}: expected shape {(rows, cols)}, got {tuple(t.shape)}")


def _device(t, what):
    """The index of the current CUDA device, on which t must be."""
    import torch
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{what}: on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return dev


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"unknown activation {name!r}: one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


def _dims(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a 2-D tensor")
    return t.shape


def _weight(q, s, N, K, dev, what):
    """Leading dimension of a block-FP8 weight's codes [N, K], its scales checked."""
    import torch
    _scales(s, N, K, dev, what)
    return _matrix(q, N, K, torch.uint8, dev, what + " codes")


def _scales(s, N, K, dev, what):
    import torch
    if N and K and not (s.shape == ((N + 127) // 128, (K + 127) // 128) and s.is_contiguous()):
        raise ValueError(f"{what} scales: expected a contiguous [{_cdiv(N, 128)}, {_cdiv(K, 128)}] grid")
    if s.dtype is not torch.float32 or s.get_device() != dev:
        raise ValueError(f"{what} scales: expected float32 on cuda:{dev}")


def _scratch(workspace, size, dims, dev):
    """(tensor kept alive, pointer, bytes) of a workspace; if None, one of
    size(*dims) bytes allocated here."""
    if workspace is None:
        need = size(*dims)
        if not need:
            return None, None, 0
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), need
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _new(rows, cols, align, dtype, dev):
    """A new matrix whose rows are a multiple of align elements apart, and its
    leading dimension."""
    import torch
    ld = (max(cols, 1) + align - 1) // align * align
    buf = torch.empty((rows, ld), dtype=dtype, device=dev)
    return (buf if ld == cols else buf[:, :cols]), ld


def _output(out, rows, cols, align, dtype, dev, what="out"):
    """out and its leading dimension, made here if None."""
    if out is None:
        return _new(rows, cols, align, dtype, dev)
    return out, _matrix(out, rows, cols, dtype, dev, what)


def _linear_epilogue(mode, name, x, q, scale_inv, bias, activation, residual, preact, out, workspace):
    import torch
    act = _activation(activation)
    bf16 = torch.bfloat16
    M, K = _dims(x, "x")
    N = _dims(q, "q")[0]
    dev = _device(x, "x")
    ldx = _matrix(x, M, K, bf16, dev, "x")
    ldq = _weight(q, scale_inv, N, K, dev, "weight")
    ep = Epilogue(None, act, None, 0, None, 0)
    if bias is not None:
        if not (bias.shape == (N,) and bias.dtype is bf16 and bias.is_contiguous() and bias.get_device() == dev):
            raise ValueError(f"bias: expected {N} contiguous BF16 values on cuda:{dev}")
        ep.bias = bias.data_ptr()
    if residual is not None:
        ep.residual, ep.ldr = residual.data_ptr(), _matrix(residual, M, N, bf16, dev, "residual")
    if preact is not None:
        ep.preact, ep.ldp = preact.data_ptr(), _matrix(preact, M, N, bf16, dev, "preact")
    out, ldy = _output(out, M, N, 8, bf16, dev)
    workspace, ws, ws_len = _scratch(workspace, workspace_size, (mode, M, N, K), dev)
    _check(getattr(lib(), name)(x.data_ptr(), ldx, q.data_ptr(), ldq, scale_inv.data_ptr(),
                                out.data_ptr(), ldy, M, N, K, ctypes.byref(ep), ws, ws_len,
                                _stream()), name)
    return out


def linear_w8a16_epilogue(x, q, scale_inv, bias=None, activation="none", residual=None, preact=None,
                          out=None, workspace=None):
    """y = act(x . dequant(W)^T + bias) + residual, BF16 activations; y BF16 [M, N].

    bias BF16 [N]; residual BF16 [M, N], which out may be itself; preact BF16
    [M, N] receives z = x . dequant(W)^T + bias for epilogue_backward."""
    return _linear_epilogue(0, "fp8blk_linear_w8a16_epilogue", x, q, scale_inv, bias, activation,
                            residual, preact, out, workspace)


def linear_w8a8_epilogue(x, q, scale_inv, bias=None, activation="none", residual=None, preact=None,
                         out=None, workspace=None):
    """linear_w8a16_epilogue with x quantized per 1x128 K-group to E4M3."""
    return _linear_epilogue(1, "fp8blk_linear_w8a8_epilogue", x, q, scale_inv, bias, activation,
                            residual, preact, out, workspace)


def _gated_linear(mode, name, x, q_gate, s_gate, q_up, s_up, activation, out, preact, workspace):
    import torch
    act = _activation(activation)
    bf16 = torch.bfloat16
    M, K = _dims(x, "x")
    N = _dims(q_gate, "q_gate")[0]
    dev = _device(x, "x")
    ldx = _matrix(x, M, K, bf16, dev, "x")
    ldq = _weight(q_gate, s_gate, N, K, dev, "gate weight")
    if _weight(q_up, s_up, N, K, dev, "up weight") != ldq:
        raise ValueError("q_gate and q_up: expected one row stride")
    g = u = None
    ldgu = 0
    if preact is not None:
        g, u = preact
        ldgu = _matrix(g, M, N, bf16, dev, "g")
        if _matrix(u, M, N, bf16, dev, "u") != ldgu:
            raise ValueError("g and u: expected one row stride")
    out, ldh = _output(out, M, N, 8, bf16, dev)
    workspace, ws, ws_len = _scratch(workspace, workspace_size, (mode, M, 2 * N, K), dev)
    _check(getattr(lib(), name)(x.data_ptr(), ldx, q_gate.data_ptr(), s_gate.data_ptr(),
                                q_up.data_ptr(), s_up.data_ptr(), ldq, act, out.data_ptr(), ldh,
                                g.data_ptr() if g is not None else None,
                                u.data_ptr() if u is not None else None, ldgu, M, N, K, ws, ws_len,
                                _stream()), name)
    return out


def gated_linear_w8a16(x, q_gate, s_gate, q_up, s_up, activation="silu", out=None, preact=None,
                       workspace=None):
    """h = act(x . dequant(Wg)^T) * (x . dequant(Wu)^T), BF16 activations; h BF16 [M, N].

    Both weights [N, K] with one row stride (a fused [2N, K] weight with
    N % 128 == 0 is passed as its two halves). preact: a pair (g, u) of BF16
    [M, N] with one row stride, which receive the two products for
    gated_backward. The workspace is that of 2 N outputs."""
    return _gated_linear(0, "fp8blk_gated_linear_w8a16", x, q_gate, s_gate, q_up, s_up, activation,
                         out, preact, workspace)


def gated_linear_w8a8(x, q_gate, s_gate, q_up, s_up, activation="silu", out=None, preact=None,
                      workspace=None):
    """gated_linear_w8a16 with x quantized per 1x128 K-group to E4M3."""
    return _gated_linear(1, "fp8blk_gated_linear_w8a8", x, q_gate, s_gate, q_up, s_up, activation,
                         out, preact, workspace)


def gated_backward(dh, g, u, activation="silu", out=None):
    """dgu BF16 [M, 2 Np], Np = round_up(N, 128): dg = dh u act'(g) in columns
    [0, N), du = dh act(g) in [Np, Np + N), zeros between. dx is then
    linear_w8a16(dgu, *transpose_gated_weights(...))."""
    import torch
    act = _activation(activation)
    bf16 = torch.bfloat16
    M, N = _dims(dh, "dh")
    dev = _device(dh, "dh")
    lddh = _matrix(dh, M, N, bf16, dev, "dh")
    ldgu = _matrix(g, M, N, bf16, dev, "g")
    if _matrix(u, M, N, bf16, dev, "u") != ldgu:
        raise ValueError("g and u: expected one row stride")
    width = 2 * _round_up(N, 128)
    out, ldo = _output(out, M, width, 8, bf16, dev)
    _check(lib().fp8blk_gated_backward(dh.data_ptr(), lddh, g.data_ptr(), u.data_ptr(), ldgu, act,
                                       out.data_ptr(), ldo, M, N, _stream()), "fp8blk_gated_backward")
    return out


def epilogue_backward_workspace_size(M: int, N: int) -> int:
    return int(lib().fp8blk_epilogue_backward_workspace_size(M, N))


def epilogue_backward(dy, z=None, activation="none", dz=None, bias_grad=True, workspace=None):
    """(dz, dbias): dz = dy act'(z) in BF16, dbias float32 [N] its column sums
    before rounding (None without bias_grad). z is the kept preact (not needed
    for "none", whose dz is dy itself unless a dz is given). dz may be dy or z."""
    import torch
    act = _activation(activation)
    bf16 = torch.bfloat16
    M, N = _dims(dy, "dy")
    dev = _device(dy, "dy")
    lddy = _matrix(dy, M, N, bf16, dev, "dy")
    ldz = 0
    if z is not None:
        ldz = _matrix(z, M, N, bf16, dev, "z")
    elif act != 0:
        raise ValueError("z: needed for every activation but none")
    if dz is None and act == 0:
        dz, lddz = dy, lddy
    else:
        dz, lddz = _output(dz, M, N, 8, bf16, dev, "dz")
    dbias, ws, ws_len = None, None, 0
    if bias_grad:
        dbias = torch.empty(N, dtype=torch.float32, device=dev)
        workspace, ws, ws_len = _scratch(workspace, epilogue_backward_workspace_size, (M, N), dev)
    _check(lib().fp8blk_epilogue_backward(dy.data_ptr(), lddy, z.data_ptr() if z is not None else None,
                                          ldz, act, dz.data_ptr(), lddz,
                                          dbias.data_ptr() if bias_grad else None, M, N, ws, ws_len,
                                          _stream()), "fp8blk_epilogue_backward")
    return dz, dbias


def transpose_weight(q, scale_inv, qt=None, st=None, zero_pad=False):
    """(qt, st): the transposed block-FP8 weight, codes [K, N] and scales
    [ceil(K/128), ceil(N/128)], exact. dx = linear_w8a16(dz, qt, st).

    zero_pad: codes [K, Np] with Np = round_up(N, 128), zeros in the columns past
    N, for a dz in a buffer of Np columns whose last ones hold any numbers."""
    import torch
    N, K = _dims(q, "q")
    dev = _device(q, "q")
    ldq = _weight(q, scale_inv, N, K, dev, "weight")
    cols = _round_up(N, 128) if zero_pad else N
    if st is None:
        st = torch.empty((_cdiv(K, 128), _cdiv(N, 128)), dtype=torch.float32, device=dev)
    if qt is None:
        qt, ldqt = _new(K, cols, 16, torch.uint8, dev)
        _scales(st, K, N, dev, "transposed weight")
    else:
        ldqt = _weight(qt, st, K, cols, dev, "transposed weight")
    _check(lib().fp8blk_transpose_weight(q.data_ptr(), ldq, scale_inv.data_ptr(), N, K, qt.data_ptr(),
                                         ldqt, st.data_ptr(), st.shape[1], int(bool(zero_pad)), _stream()),
           "fp8blk_transpose_weight")
    return qt, st


def transpose_gated_weights(q_gate, s_gate, q_up, s_up, qt=None, st=None):
    """(qt, st): both transposed weights of a gated linear side by side, codes
    [K, 2 Np] (Np = round_up(N, 128), zero codes between), the layout that
    gated_backward's output multiplies."""
    import torch
    N, K = _dims(q_gate, "q_gate")
    dev = _device(q_gate, "q_gate")
    ldq = _weight(q_gate, s_gate, N, K, dev, "gate weight")
    if _weight(q_up, s_up, N, K, dev, "up weight") != ldq:
        raise ValueError("q_gate and q_up: expected one row stride")
    NB = _cdiv(N, 128)
    Np = 128 * NB
    if qt is None:
        qt = torch.empty((K, 2 * Np), dtype=torch.uint8, device=dev)
    if st is None:
        st = torch.empty((_cdiv(K, 128), 2 * NB), dtype=torch.float32, device=dev)
    ldqt = _weight(qt, st, K, 2 * Np, dev, "transposed weight")
    _check(lib().fp8blk_transpose_gated_weights(q_gate.data_ptr(), s_gate.data_ptr(), q_up.data_ptr(),
                                                s_up.data_ptr(), ldq, N, K, qt.data_ptr(), ldqt,
                                                st.data_ptr(), _stream()),
           "fp8blk_transpose_gated_weights")
    return qt, st


def linear_grad_weight_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().fp8blk_linear_grad_weight_workspace_size(M, N, K))


def linear_grad_weight(dz, x, out=None, accumulate=False, dtype=None, workspace=None):
    """dw [N, K] = dz^T . x over the tokens of dz BF16 [M, N] and x BF16 [M, K],
    FP32 sums of the products of the BF16 values given; float32 unless out or
    dtype says BF16. accumulate adds to a float32 out."""
    import torch
    bf16, f32 = torch.bfloat16, torch.float32
    M, N = _dims(dz, "dz")
    K = _dims(x, "x")[1]
    dev = _device(dz, "dz")
    lddz = _matrix(dz, M, N, bf16, dev, "dz")
    ldx = _matrix(x, M, K, bf16, dev, "x")
    dtype = dtype or (out.dtype if out is not None else f32)
    if dtype not in (bf16, f32):
        raise ValueError(f"dw: expected float32 or bfloat16, got {dtype}")
    if accumulate and (out is None or dtype != f32):
        raise ValueError("accumulate: needs a float32 out")
    out, lddw = _output(out, N, K, 4 if dtype == f32 else 8, dtype, dev)
    workspace, ws, ws_len = _scratch(workspace, linear_grad_weight_workspace_size, (M, N, K), dev)
    _check(lib().fp8blk_linear_grad_weight(dz.data_ptr(), lddz, x.data_ptr(), ldx, out.data_ptr(), lddw,
                                           int(dtype == f32), int(accumulate), M, N, K, ws, ws_len,
                                           _stream()), "fp8blk_linear_grad_weight")
    return out


def encode_e4m3(v):
    import torch
    out = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check(lib().fp8blk_encode_e4m3(v.data_ptr(), v.numel(), out.data_ptr(), _stream()),
           "fp8blk_encode_e4m3")
    return out


def selftest_wait_timeout(limit_cycles: int = 2_000_000) -> None:
    """Launches the failure-detection self-test (a bounded wait that runs out)."""
    _check(lib().fp8blk_selftest_wait_timeout(limit_cycles, _stream()),
           "fp8blk_selftest_wait_timeout")


def read_device_error() -> int:
    """Reads and clears the device error word (synchronizes the device)."""
    word = ctypes.c_uint32(0)
    st = lib().fp8blk_read_device_error(ctypes.byref(word))
    if st not in (0, 6):
        raise Fp8BlkError(st, "fp8blk_read_device_error")
    return int(word.value)
