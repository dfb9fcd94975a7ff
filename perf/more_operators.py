"""The operators around the quantised linears, case by case: the root-mean-square norm that adds the
residual and gives rotated codes, and the gated product of two projections.

norm: h = x + residual, rounded to the type and kept; the row h / rms(h) * weight goes through the
block rotation (Walsh-Hadamard, 128 wide, stages 1, 2, 4, ... in binary32) and is quantised with one
scale a row. The norm's factor is one positive number a row and a row's codes do not change with
such a factor, so it enters the scale alone.
gated: y = act(g) * u of the gate's and the up projection's row, both from one matrix of codes in
which 16 gate rows and 16 up rows lie in turn.

Codes are an intermediate of every pass: the norm's are taken by the projection behind it, as in a
layer. With `own` false, run() is the plain form (elementary torch operations in binary32); with
`own` true it makes the calls of this package.
"""
import torch

own = False

_TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------------------ the cases
def listed():
    def case(name, op, M, K, N, bits, dtype, act="none", residual=True, bias=False, tiles="int", weight="same"):
        return dict(name=name, op=op, M=M, K=K, N=N, bits=bits, dtype=dtype, act=act, residual=residual, bias=bias,
                    tiles=tiles, weight=weight)

    return [
        # Norm, then a projection: one ViT-L image (72 x 72 patches) and its output projection.
        case("norm_image", "norm", 5184, 1024, 1024, 8, "f16", bias=True),
        # The tokens of two DiT images and the fused projection of queries, keys and values.
        case("norm_dit", "norm", 8192, 1536, 4608, 8, "bf16"),
        # A batch of eight images.
        case("norm_batch", "norm", 41472, 1024, 1024, 8, "f16", bias=True),
        # A ragged prompt, a width of 17 blocks, no residual yet (a first layer), 4-bit codes, binary32 weights.
        case("norm_ragged", "norm", 777, 2176, 528, 4, "bf16", residual=False, weight="f32"),
        # A single token's gated product: latency, and the weights' bytes.
        case("gated_one", "gated", 1, 4096, 11264, 8, "bf16", act="silu"),
        # Eight sequences with five drafted tokens each, 4-bit codes.
        case("gated_drafts", "gated", 40, 2048, 5120, 4, "f16", act="silu"),
        # An image's tokens, an odd width of the hidden layer, biases.
        case("gated_image", "gated", 5184, 1024, 2736, 8, "f16", act="gelu_erf", bias=True),
        # A DiT block's feed-forward layer.
        case("gated_dit", "gated", 8192, 1536, 4096, 8, "bf16", act="gelu_tanh", bias=True),
        # 4-bit codes on the matrix cores' 6-bit floats.
        case("gated_w4", "gated", 5184, 4096, 4096, 4, "f16", act="silu", tiles="fp6"),
        # Norm and gated product, as a layer has them: a single token with 4-bit codes.
        case("block_one", "block", 1, 4096, 11264, 4, "bf16", act="silu"),
        # A decode step of 64 sequences.
        case("block_batch", "block", 64, 4096, 11264, 8, "bf16", act="silu"),
        # A long prompt.
        case("block_prompt", "block", 16384, 4096, 8192, 8, "bf16", act="silu"),
    ]


def _log_between(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("norm", "gated", "gated", "block"))
    K = 128 * _log_between(rng, 1, 64)
    N = 16 * _log_between(rng, 1, 704)
    M = _log_between(rng, 1, 41472)
    per_token = K * N * (1 if op == "norm" else 2)
    M = max(1, min(M, 16384 * 4096 * 8192 // per_token, (1 << 28) // K, (1 << 28) // N))
    bits = rng.choice((8, 8, 4))
    return dict(op=op, M=M, K=K, N=N, bits=bits, dtype=rng.choice(("f16", "bf16")),
                act="none" if op == "norm" else rng.choice(("silu", "silu", "gelu_erf", "gelu_tanh", "none")),
                residual=rng.random() < 0.8, bias=rng.random() < 0.4,
                tiles=rng.choice(("int", "fp6")) if bits == 4 else "int", weight=rng.choice(("same", "f32")))


def _rows(case):
    """Rows of the weights: the gated product has two for an output."""
    return case["N"] * (1 if case["op"] == "norm" else 2)


def work(case):
    M, K, N = case["M"], case["K"], case["N"]
    rows = _rows(case)
    moved = M * K * 2 + rows * K * case["bits"] // 8 + rows * 4 * (2 if case["bias"] else 1) + M * N * 2
    flops = 2 * M * rows * K
    if case["op"] != "gated":
        moved += (2 * M * K * 2 if case["residual"] else 0) + K * (4 if case["weight"] == "f32" else 2)
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------------------- the plain form
def _rotate(x):
    """Unnormalised Walsh-Hadamard transform of blocks of 128 along the last axis."""
    h = 1
    while h < 128:
        y = x.reshape(*x.shape[:-1], x.shape[-1] // (2 * h), 2, h)
        a, b = y[..., 0, :], y[..., 1, :]
        x = torch.stack((a + b, a - b), dim=-2).reshape(x.shape)
        h *= 2
    return x


_NORM = torch.tensor(128.0, dtype=torch.float64).rsqrt().float().item()


def _quantise(x, bits):
    """Rows of the last axis -> (codes as binary32, scales)."""
    top = 127.0 if bits == 8 else 7.0
    u = _rotate(x)
    a = u.abs().amax(-1)
    top_of = torch.full_like(a, top)
    inv = top_of / a
    zero = torch.isinf(inv)
    inv = torch.where(zero, torch.zeros_like(inv), inv)
    scale = torch.where(zero, torch.zeros_like(a), (a * _NORM) / top_of)
    return torch.round(u * inv[..., None]), scale


def _pack(codes, bits):
    if bits == 8:
        return codes.to(torch.int8)
    c = codes.to(torch.int16).reshape(*codes.shape[:-1], -1, 2) & 15
    return (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8)


def _unpack(raw, bits):
    """Bytes -> codes as binary32."""
    if bits == 8:
        return raw.float()
    return ((torch.stack((raw & 15, raw >> 4), dim=-1) ^ 8).float() - 8.0).flatten(-2)


def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu_erf":
        return 0.5 * g * torch.erfc(g * -0.5 ** 0.5)
    if act == "gelu_tanh":
        return g * torch.sigmoid(1.5957691216057308 * (g + 0.044715 * g * g * g))
    return g


def _plain(s, case):
    x, out = s["X"], {}
    row = x.float()
    if case["op"] != "gated":
        h = x
        if case["residual"]:
            h = (x.float() + s["residual"].float()).to(x.dtype)
            out["h"] = h
        row = h.float()
        r = torch.rsqrt(row.square().mean(-1) + EPS)
        row = row * s["weight"].float()
    codes, scale = _quantise(row, case["bits"])
    if case["op"] != "gated":
        scale = scale * r
    y = torch.matmul(codes, _unpack(s["Wq"], case["bits"]).t()) * (scale[:, None] * s["w_scale"])
    if case["bias"]:
        y = y + s["bias"]
    if case["op"] != "norm":
        both = y.view(y.shape[0], -1, 2, 16)
        y = (_act(both[:, :, 0], case["act"]) * both[:, :, 1]).reshape(y.shape[0], -1)
    out["y"] = y.to(x.dtype)
    return out


# -------------------------------------------------------------------------------- inputs, a pass
def _tokens(gen, M, K, dtype, dev):
    """Activations with a few large channels, as the layers see them."""
    x = torch.randn(M, K, generator=gen, device=dev)
    big = torch.randint(0, K, (max(1, K // 100),), generator=gen, device=dev)
    x[:, big] *= 30.0
    return x.to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)
    M, K, rows, dtype = case["M"], case["K"], _rows(case), _TORCH[case["dtype"]]
    state = dict(case=case, X=_tokens(gen, M, K, dtype, dev))
    if case["op"] != "gated":
        state["weight"] = (1.0 + 0.2 * torch.randn(K, generator=gen, device=dev)).to(
            torch.float32 if case["weight"] == "f32" else dtype)
        if case["residual"]:
            state["residual"] = _tokens(gen, M, K, dtype, dev)
    # Gate and up rows of one size: the interleaved matrix is as random as the two.
    W = torch.randn(rows, K, generator=gen, device=dev) * (1.5 / K ** 0.5 if case["op"] != "gated" else 0.02)
    codes, state["w_scale"] = _quantise(W, case["bits"])
    state["Wq"] = _pack(codes, case["bits"])
    if case["bias"]:
        state["bias"] = 0.1 * torch.randn(rows, generator=gen, device=dev)
    if own:
        import w4a4_integer_quantized_amd as rq
        state["rq"] = rq
        state["act"] = {"none": rq.RQ_ACT_NONE, "silu": rq.RQ_ACT_SILU, "gelu_erf": rq.RQ_ACT_GELU_ERF,
                        "gelu_tanh": rq.RQ_ACT_GELU_TANH}[case["act"]]
        if case["tiles"] == "fp6":
            state["W6"], _ = rq.quantize_weights(W, bits=4, w_layout=rq.RQ_W_FP6)
    return state


def run(state):
    case = state["case"]
    if not own:
        return _plain(state, case)
    rq, bits, bias = state["rq"], case["bits"], state.get("bias")
    fp6 = case["tiles"] == "fp6"
    Wq, w_layout = (state["W6"], rq.RQ_W_FP6) if fp6 else (state["Wq"], rq.RQ_W_ROWS)
    if case["op"] == "gated":
        return {"y": rq.rotq_gated_linear(state["X"], Wq, state["w_scale"], bias, bits=bits, w_layout=w_layout, act=state["act"])}
    layout = rq.RQ_X_FP6 if fp6 else rq.RQ_X_TILED
    Xq, x_scale, h = rq.norm_rotate_quantize(state["X"], state.get("residual"), state["weight"], eps=EPS, bits=bits,
                                             x_layout=layout)
    out = {"h": h} if case["residual"] else {}
    if case["op"] == "norm":
        out["y"] = rq.gemm_dequant(Xq, x_scale, Wq, state["w_scale"], bias, bits=bits, K=case["K"],
                                   out_dtype=_TORCH[case["dtype"]], x_layout=layout, w_layout=w_layout)
    else:
        out["y"] = rq.gemm_gated(Xq, x_scale, Wq, state["w_scale"], bias, bits=bits, K=case["K"],
                                 out_dtype=_TORCH[case["dtype"]], x_layout=layout, w_layout=w_layout, act=state["act"])
    return out


# ------------------------------------------------------------------------ the definition, 64 bits
def _codes64(raw, bits):
    x = raw.view(torch.int8)
    if bits == 8:
        return x.double()
    return torch.stack(((x << 4) >> 4, x >> 4), dim=-1).double().reshape(raw.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    x, top, out = s["X"], 127.0 if case["bits"] == 8 else 7.0, {}
    j = torch.arange(128, device=x.device)
    odd = sum(((j[:, None] & j[None, :]) >> b) & 1 for b in range(7)) % 2
    R = (1.0 - 2.0 * odd.double()) / 128.0 ** 0.5
    W = _codes64(s["Wq"], case["bits"])
    sw = s["w_scale"].double()
    if case["op"] != "gated" and case["residual"]:
        out["h"] = x.double() + s["residual"].double()
    ys = []
    for at in range(0, case["M"], 4096):
        h = x[at:at + 4096].double()
        r = 1.0
        if case["op"] != "gated":
            if case["residual"]:
                h = out["h"][at:at + 4096].to(x.dtype).double()     # what is kept is what is normalised
            r = (h.pow(2).sum(1, keepdim=True) / case["K"] + EPS).pow(-0.5)
            h = h * s["weight"].double()
        u = torch.matmul(h.view(-1, 128), R).view(h.shape)
        a = u.abs().amax(1, keepdim=True)
        codes = torch.round(u * torch.where(a > 0, top / a, 0.0))
        y = (codes @ W.t()) * (a / top * r) * sw
        if case["bias"]:
            y = y + s["bias"].double()
        if case["op"] != "norm":
            y = y.unflatten(1, (-1, 32))
            g, up = y[:, :, :16], y[:, :, 16:]
            if case["act"] == "silu":
                g = g / (1.0 + torch.exp(-g))
            elif case["act"] == "gelu_erf":
                g = g * 0.5 * (1.0 + torch.erf(g / 2.0 ** 0.5))
            elif case["act"] == "gelu_tanh":
                g = 0.5 * g * (1.0 + torch.tanh((2.0 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
            y = (g * up).flatten(1)
        ys.append(y)
    out["y"] = torch.cat(ys)
    return out
