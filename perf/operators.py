"""The feed-forward operators of the block-FP8 linear layer, case by case.

Four operators, each with W an E4M3 code matrix and one FP32 scale per
128 x 128 block (W[n, k] = code * scale):

* ``gated``           h = act(x Wg^T) * (x Wu^T), and the BF16 pre-activations
                      g, u where a training step keeps them;
* ``gated_backward``  from dh and the kept g, u: dg, du, dx, dWg, dWu (or dx
                      alone when the weights are frozen);
* ``linear``          z = x W^T + bias, y = act(z) + residual, and z where a
                      training step keeps it;
* ``linear_backward`` from dy and the kept z: dz, dbias, dx, dW.

``mode`` is "w8a16" (BF16 activations) or "w8a8" (activations quantized to E4M3
per token and group of 128 inputs, scale = group maximum / 448).
"""
import math

import torch

own = False

BLOCK = 128
FP8_MAX = 448.0


def listed():
    """The cases: hidden 5120, feed-forward 25600, attention 8192 -> 5120 and
    fused query/key/value 10240, plus ragged ones of about 1000."""
    return [
        # one token being generated: the weights' stream is the whole cost
        _gated("gated_w8a16_m1", "w8a16", 1, 5120, 25600),
        # a batch of 64 sequences, one token each
        _gated("gated_w8a16_m64", "w8a16", 64, 5120, 25600),
        # a prompt of ordinary length in a training step that keeps g and u
        _gated("gated_w8a16_m512_kept", "w8a16", 512, 5120, 25600, keep=True),
        # sizes that fill no tile and no block, with the other usual gate
        _gated("gated_w8a8_ragged", "w8a8", 77, 1000, 1000, act="gelu_tanh"),
        # a long prompt, or many short ones packed
        _gated("gated_w8a8_m4096", "w8a8", 4096, 5120, 25600),
        # gradient through a frozen layer (adapters or embeddings being trained)
        _gated_backward("gated_backward_frozen_ragged", 300, 1000, 1000, frozen=True),
        # a training step of the whole layer
        _gated_backward("gated_backward_m2048", 2048, 5120, 25600),
        # attention output of one token, added to the residual stream
        _linear("linear_w8a16_o_proj_m1", "w8a16", 1, 8192, 5120, residual=True),
        # down projection of a prompt, added to the residual stream
        _linear("linear_w8a8_down_m512", "w8a8", 512, 25600, 5120, residual=True),
        # first layer of a plain feed-forward block with bias, kept for training
        _linear("linear_w8a16_ragged_kept", "w8a16", 333, 1000, 1000, bias=True, act="gelu", keep=True),
        # a small layer's training step, ragged
        _linear_backward("linear_backward_ragged", 77, 1000, 1000, act="gelu"),
        # a projection's training step without activation
        _linear_backward("linear_backward_qkv_m512", 512, 5120, 10240),
    ]


def _gated(name, mode, m, k, n, act="silu", keep=False):
    return dict(name=name, op="gated", mode=mode, m=m, k=k, n=n, act=act, keep=keep)


def _gated_backward(name, m, k, n, act="silu", frozen=False):
    return dict(name=name, op="gated_backward", m=m, k=k, n=n, act=act, frozen=frozen)


def _linear(name, mode, m, k, n, bias=False, act="none", residual=False, keep=False):
    return dict(name=name, op="linear", mode=mode, m=m, k=k, n=n, bias=bias, act=act,
                residual=residual, keep=keep)


def _linear_backward(name, m, k, n, act="none"):
    return dict(name=name, op="linear_backward", m=m, k=k, n=n, act=act)


def draw(rng):
    op = rng.choice(["gated", "gated", "linear", "linear", "gated_backward", "linear_backward"])
    m = round(math.exp(rng.uniform(0.0, math.log(4096))))
    k = round(math.exp(rng.uniform(math.log(64), math.log(8192))))
    n = round(math.exp(rng.uniform(math.log(64), math.log(25600))))
    if rng.random() < 0.5:  # half of the layers are whole blocks, half are not
        k, n = max(BLOCK, k // BLOCK * BLOCK), max(BLOCK, n // BLOCK * BLOCK)
    # no dearer than the largest listed case
    limit = (2048 if op.endswith("backward") else 4096) * 5120 * 25600
    m = max(1, min(m, limit // (k * n)))
    acts = ["relu", "gelu", "gelu_tanh", "silu"]
    if op == "gated":
        c = _gated("", rng.choice(["w8a16", "w8a8"]), m, k, n, rng.choice(acts), rng.random() < 0.3)
    elif op == "gated_backward":
        c = _gated_backward("", m, k, n, rng.choice(acts), rng.random() < 0.3)
    elif op == "linear":
        c = _linear("", rng.choice(["w8a16", "w8a8"]), m, k, n, rng.random() < 0.5,
                    rng.choice(["none"] + acts), rng.random() < 0.5, rng.random() < 0.3)
    else:
        c = _linear_backward("", m, k, n, rng.choice(["none"] + acts))
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs
def _up(a, b):
    return -(-a // b) * b


def _over_448(t):
    """t / 448, correctly rounded (a Python scalar divisor becomes a product
    with its rounded reciprocal, which moves values lying on a border)."""
    return t / torch.full_like(t, FP8_MAX)


def _rows(t, align):
    """t in a buffer whose rows are a multiple of `align` elements apart."""
    r, c = t.shape
    buf = torch.zeros((r, _up(c, align)), dtype=t.dtype, device=t.device)
    buf[:, :c] = t
    return buf[:, :c]


def _weight(gen, n, k):
    """A BF16 weight N(0, 0.02^2) in the serialized form: codes and scales."""
    w = (torch.randn((n, k), generator=gen, device="cuda") * 0.02).to(torch.bfloat16).float()
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    pad = torch.zeros((nb * BLOCK, kb * BLOCK), device="cuda")
    pad[:n, :k] = w
    blocks = pad.view(nb, BLOCK, kb, BLOCK)
    scale = _over_448(blocks.abs().amax(dim=(1, 3)))
    q = (blocks / torch.where(scale == 0, 1.0, scale)[:, None, :, None]).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).view(nb * BLOCK, kb * BLOCK)[:n, :k]
    return _rows(q, 16), scale.contiguous()


def _activations(gen, m, k):
    """N(0, 1) with one channel in a hundred twenty times larger."""
    x = torch.randn((m, k), generator=gen, device="cuda")
    loud = torch.randperm(k, generator=gen, device="cuda")[:k // 100]
    x[:, loud] *= 20.0
    return _rows(x.to(torch.bfloat16), 8)


def _normal(gen, m, n, sigma):
    return _rows((torch.randn((m, n), generator=gen, device="cuda") * sigma).to(torch.bfloat16), 8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    m, k, n = case["m"], case["k"], case["n"]
    st = {"case": case, "x": _activations(gen, m, k)}
    gated = case["op"].startswith("gated")
    st["w"] = [_weight(gen, n, k) for _ in range(2 if gated else 1)]
    if case["op"] == "gated_backward":
        # pre-activations of the size the forward pass gives, small gradients
        st["g"], st["u"] = _normal(gen, m, n, 1.5), _normal(gen, m, n, 1.5)
        st["dh"] = _normal(gen, m, n, 0.01)
    elif case["op"] == "linear_backward":
        st["z"] = _normal(gen, m, n, 1.5) if case["act"] != "none" else None
        st["dy"] = _normal(gen, m, n, 0.01)
    elif case["op"] == "linear":
        st["bias"] = _normal(gen, 1, n, 0.1)[0] if case["bias"] else None
        st["residual"] = _normal(gen, m, n, 1.0) if case["residual"] else None
    if own:
        _prepare_own(case, st)
    return st


def _prepare_own(case, st):
    """What a program keeps beside its tensors: output buffers and workspaces,
    and for frozen weights their transposed codes (laid out once)."""
    import block_scaled_fp8_fp8blk_b200 as fb

    m, k, n = case["m"], case["k"], case["n"]

    def scratch(mode, rows, outs, ins):
        return torch.empty(fb.workspace_size(0 if mode == "w8a16" else 1, rows, outs, ins),
                           dtype=torch.uint8, device="cuda")

    if case["op"] == "gated":
        st["workspace"] = scratch(case["mode"], m, 2 * n, k)
    elif case["op"] == "linear":
        st["workspace"] = scratch(case["mode"], m, n, k)
    elif case["op"] == "gated_backward":
        st["workspace"] = scratch("w8a16", m, k, 2 * _up(n, BLOCK))
        if case["frozen"]:
            st["wt"] = fb.transpose_gated_weights(*st["w"][0], *st["w"][1])
    else:
        st["workspace"] = scratch("w8a16", m, k, n)


# ---------------------------------------------------------------- the passes
def run(state):
    case = state["case"]
    return (_own if own else _plain)[case["op"]](case, state)


def _own_gated(case, st):
    import block_scaled_fp8_fp8blk_b200 as fb

    f = fb.gated_linear_w8a16 if case["mode"] == "w8a16" else fb.gated_linear_w8a8
    kept = None
    if case["keep"]:
        m, n = case["m"], case["n"]
        kept = tuple(torch.empty((m, _up(n, 8)), dtype=torch.bfloat16, device="cuda")[:, :n]
                     for _ in range(2))
    h = f(st["x"], *st["w"][0], *st["w"][1], activation=case["act"], preact=kept,
          workspace=st["workspace"])
    return [h, *kept] if kept else [h]


def _own_gated_backward(case, st):
    import block_scaled_fp8_fp8blk_b200 as fb

    n = case["n"]
    dgu = fb.gated_backward(st["dh"], st["g"], st["u"], activation=case["act"])
    # trained weights change from step to step, so they are transposed here
    wt = st["wt"] if case["frozen"] else fb.transpose_gated_weights(*st["w"][0], *st["w"][1])
    dx = fb.linear_w8a16(dgu, *wt, workspace=st["workspace"])
    if case["frozen"]:
        return [dx]
    dg, du = dgu[:, :n], dgu[:, _up(n, BLOCK):_up(n, BLOCK) + n]
    return [dg, du, dx, *(fb.linear_grad_weight(d, st["x"], dtype=torch.bfloat16) for d in (dg, du))]


def _own_linear(case, st):
    import block_scaled_fp8_fp8blk_b200 as fb

    f = fb.linear_w8a16_epilogue if case["mode"] == "w8a16" else fb.linear_w8a8_epilogue
    kept = None
    if case["keep"]:
        m, n = case["m"], case["n"]
        kept = torch.empty((m, _up(n, 8)), dtype=torch.bfloat16, device="cuda")[:, :n]
    y = f(st["x"], *st["w"][0], bias=st["bias"], activation=case["act"], residual=st["residual"],
          preact=kept, workspace=st["workspace"])
    return [y] if kept is None else [y, kept]


def _own_linear_backward(case, st):
    import block_scaled_fp8_fp8blk_b200 as fb

    dz, dbias = fb.epilogue_backward(st["dy"], st["z"], activation=case["act"])
    dx = fb.linear_w8a16(dz, *fb.transpose_weight(*st["w"][0]), workspace=st["workspace"])
    return [dz, dbias, dx, fb.linear_grad_weight(dz, st["x"], dtype=_grad_dtype(case))]


def _grad_dtype(case):
    """32 bits where dz is the BF16 gradient that was given; where dz is itself
    rounded to BF16 on its way into the product, so is the result."""
    return torch.float32 if case["act"] == "none" else torch.bfloat16


_own = {"gated": _own_gated, "gated_backward": _own_gated_backward, "linear": _own_linear,
        "linear_backward": _own_linear_backward}


def _blocks(s, n, k):
    return s.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def _dequantized(w):
    q, s = w
    return q.contiguous().view(torch.float8_e4m3fn).float() * _blocks(s, *q.shape)


def _input(case, st):
    """x in 32 bits; for w8a8 after its quantization per token and group."""
    x = st["x"].float()
    if case["mode"] == "w8a16":
        return x
    m, k = x.shape
    groups = torch.nn.functional.pad(x, (0, _up(k, BLOCK) - k)).view(m, -1, BLOCK)
    s = _over_448(groups.abs().amax(dim=2, keepdim=True))
    q = (groups / torch.where(s == 0, 1.0, s)).to(torch.float8_e4m3fn)
    return (q.float() * s).view(m, -1)[:, :k]


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return (0.5 * torch.erfc(-z / math.sqrt(2.0))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1.0 - s) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _bf16(*ts):
    return [t.to(torch.bfloat16) for t in ts]


def _plain_gated(case, st):
    x = _input(case, st)
    g, u = (x @ _dequantized(w).T for w in st["w"])
    h = _act(case["act"], g) * u
    return _bf16(h, g, u) if case["keep"] else _bf16(h)


def _plain_gated_backward(case, st):
    g, u, dh, x = (st[name].float() for name in ("g", "u", "dh", "x"))
    dg = dh * u * _act_slope(case["act"], g)
    du = dh * _act(case["act"], g)
    dx = dg @ _dequantized(st["w"][0]) + du @ _dequantized(st["w"][1])
    if case["frozen"]:
        return _bf16(dx)
    return _bf16(dg, du, dx, dg.T @ x, du.T @ x)


def _plain_linear(case, st):
    z = _input(case, st) @ _dequantized(st["w"][0]).T
    if st["bias"] is not None:
        z = z + st["bias"].float()
    y = _act(case["act"], z)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return _bf16(y, z) if case["keep"] else _bf16(y)


def _plain_linear_backward(case, st):
    dz, x = st["dy"].float(), st["x"].float()
    if st["z"] is not None:
        dz = dz * _act_slope(case["act"], st["z"].float())
    dx = dz @ _dequantized(st["w"][0])
    return [*_bf16(dz), dz.sum(0), *_bf16(dx), (dz.T @ x).to(_grad_dtype(case))]


_plain = {"gated": _plain_gated, "gated_backward": _plain_gated_backward,
          "linear": _plain_linear, "linear_backward": _plain_linear_backward}


# ------------------------------------------------------------ the definition
def _code_values():
    """The 256 E4M3 values: bias 7, three mantissa bits, no infinities."""
    v = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        a = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v.append(-a if c >> 7 else a)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_weight(w):
    q, s = w
    n, k = q.shape
    rows = torch.arange(n, device="cuda") // BLOCK
    cols = torch.arange(k, device="cuda") // BLOCK
    return _code_values()[q.long()] * s.double()[rows][:, cols]


def _nearest_e4m3(v):
    """Nearest E4M3 value to |v| <= 448, ties to the even mantissa."""
    exponent = torch.frexp(v)[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return (torch.round(v / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_input(case, st):
    x = st["x"].double()
    if case["mode"] == "w8a16":
        return x
    out = torch.empty_like(x)
    for k0 in range(0, x.shape[1], BLOCK):
        part = x[:, k0:k0 + BLOCK]
        top = part.abs().max(dim=1, keepdim=True)[0]
        s = (top / torch.full_like(top, FP8_MAX)).float().double()  # a 32-bit scale
        ratio = torch.where(s > 0, part / s, 0.0).float().double()  # a 32-bit quotient
        out[:, k0:k0 + BLOCK] = _nearest_e4m3(ratio) * s
    return out


def _exact_act(name, z):
    """(act(z), act'(z))"""
    if name == "relu":
        return z.clamp(min=0.0), torch.heaviside(z, torch.zeros_like(z))
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * (0.5 * math.sqrt(2.0 / math.pi))
    if name == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        # 1 + t without cancellation where t is near -1
        onep = 2.0 * torch.sigmoid(2.0 * a * (z + 0.044715 * z ** 3))
        return 0.5 * z * onep, 0.5 * onep + 0.5 * z * onep * (1.0 - t) * a * (1.0 + 0.134145 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    return z, torch.ones_like(z)


def exact(case, seed):
    st = prepare(case, seed)
    op, act = case["op"], case["act"]
    if op == "gated":
        x = _exact_input(case, st)
        g, u = (torch.einsum("mk,nk->mn", x, _exact_weight(w)) for w in st["w"])
        h = _exact_act(act, g)[0] * u
        return [h, g, u] if case["keep"] else [h]
    if op == "linear":
        z = torch.einsum("mk,nk->mn", _exact_input(case, st), _exact_weight(st["w"][0]))
        if case["bias"]:
            z = z + st["bias"].double()
        y = _exact_act(act, z)[0]
        if case["residual"]:
            y = y + st["residual"].double()
        return [y, z] if case["keep"] else [y]
    x = st["x"].double()
    if op == "gated_backward":
        a, slope = _exact_act(act, st["g"].double())
        dh = st["dh"].double()
        parts = [dh * st["u"].double() * slope, dh * a]
        dx = sum(torch.einsum("mn,nk->mk", p, _exact_weight(w)) for p, w in zip(parts, st["w"]))
        if case["frozen"]:
            return [dx]
        return [*parts, dx, *(torch.einsum("mn,mk->nk", p, x) for p in parts)]
    dz = st["dy"].double()
    if st["z"] is not None:
        dz = dz * _exact_act(act, st["z"].double())[1]
    return [dz, dz.sum(0), torch.einsum("mn,nk->mk", dz, _exact_weight(st["w"][0])),
            torch.einsum("mn,mk->nk", dz, x)]


# ------------------------------------------------------------------ the work
def work(case):
    m, k, n, op = case["m"], case["k"], case["n"], case["op"]
    x, y = 2 * m * k, 2 * m * n
    w = n * k + 4 * -(-n // BLOCK) * -(-k // BLOCK)
    if op == "gated":
        return {"bytes": x + 2 * w + y + (2 * y if case["keep"] else 0), "flops": 4 * m * n * k}
    if op == "linear":
        extra = (2 * n if case["bias"] else 0) + y * (int(case["residual"]) + int(case["keep"]))
        return {"bytes": x + w + y + extra, "flops": 2 * m * n * k}
    if op == "gated_backward":
        if case["frozen"]:
            return {"bytes": 3 * y + 2 * w + x, "flops": 4 * m * n * k}
        return {"bytes": 3 * y + 2 * w + x + 2 * y + x + 4 * n * k, "flops": 8 * m * n * k}
    kept = y if case["act"] != "none" else 0
    dw = _grad_dtype(case).itemsize * n * k
    return {"bytes": y + kept + x + w + y + 4 * n + x + dw, "flops": 4 * m * n * k}
