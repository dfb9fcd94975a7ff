"""The operators around the quantised linears and the cache, case by case: the root-mean-square norm
that adds the residual and gives rotated codes, the gated product of two projections, and the cache
held to a budget: attention weights added up for each token, and pages written anew with the tokens
that had most.

norm: h = x + residual, rounded to the type and kept; the row h / rms(h) * weight goes through the
block rotation (Walsh-Hadamard, 128 wide, stages 1, 2, 4, ... in binary32) and is quantised with one
scale a row. The norm's factor is one positive number a row and a row's codes do not change with
such a factor, so it enters the scale alone.
gated: y = act(g) * u of the gate's and the up projection's row, both from one matrix of codes in
which 16 gate rows and 16 up rows lie in turn.

Codes are an intermediate there: the norm's are taken by the projection behind it, as in a layer.
weigh: weights[s, g, j] = keep * weights[s, g, j] + the sum over a sequence's query rows and the heads
of key head g of exp(scale * q . K_j - lse), lse as attention gave it.
evict: for each sequence and key head the first and the most recent tokens and, of the others, those
with the largest weights, as many as the budget has room for, written in order into new pages. Bytes
of a page are moved as they are.

A cache is a uint8 tensor [pages, bytes of a page]. A page holds, for each of its heads, `page`
tokens: their K codes row by row, their V codes with four tokens interleaved by the byte, the K
scales and the V scales (binary32). With `own` false, run() is the plain form (elementary torch operations in binary32); with
`own` true it makes the calls of this package.
"""
import random

import torch

own = False

_TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------------------ the cases
def listed():
    def case(name, op, M, K, N, bits, dtype, act="none", residual=True, bias=False, tiles="int", weight="same"):
        return dict(name=name, op=op, M=M, K=K, N=N, bits=bits, dtype=dtype, act=act, residual=residual, bias=bias,
                    tiles=tiles, weight=weight)

    def weigh(name, seqs, q, kv, ragged, q_heads, heads, dim, bits, page, dtype, causal, window=0, keep=1.0):
        return dict(name=name, op="weigh", seqs=seqs, q=q, kv=kv, ragged=ragged, q_heads=q_heads, heads=heads, dim=dim,
                    bits=bits, page=page, dtype=dtype, causal=causal, window=window, keep=keep)

    def evict(name, seqs, kv, ragged, heads, dim, bits, page, budget, first, recent):
        return dict(name=name, op="evict", seqs=seqs, q=1, kv=kv, ragged=ragged, heads=heads, dim=dim, bits=bits, page=page,
                    budget=budget, first=first, recent=recent)

    return [
        # Norm, then a projection: the tokens of eight ViT-L images (72 x 72 patches) and their output projection.
        case("norm_batch", "norm", 41472, 1024, 1024, 8, "f16", bias=True),
        # A ragged prompt, a width of 17 blocks, no residual yet (a first layer), 4-bit codes, binary32 weights.
        case("norm_ragged", "norm", 777, 2176, 528, 4, "bf16", residual=False, weight="f32"),
        # A single token's gated product: latency, and the weights' bytes.
        case("gated_one", "gated", 1, 4096, 11264, 8, "bf16", act="silu"),
        # Eight sequences with five drafted tokens each, 4-bit codes.
        case("gated_drafts", "gated", 40, 2048, 5120, 4, "f16", act="silu"),
        # An image's tokens, an odd width of the hidden layer, biases.
        case("gated_image", "gated", 5184, 1024, 2736, 8, "f16", act="gelu_erf", bias=True),
        # 4-bit codes on the matrix cores' 6-bit floats.
        case("gated_w4", "gated", 5184, 4096, 4096, 4, "f16", act="silu", tiles="fp6"),
        # Norm and gated product, as a layer has them: a decode step of 64 sequences.
        case("block_batch", "block", 64, 4096, 11264, 8, "bf16", act="silu"),
        # A long prompt.
        case("block_prompt", "block", 16384, 4096, 8192, 8, "bf16", act="silu"),
        # A serving batch's step: one new token each, lengths all different.
        weigh("weigh_batch", 64, 1, 8192, 1, 32, 8, 128, 4, 64, "bf16", True),
        # Prompts that come in chunks over what is cached already.
        weigh("weigh_chunks", 4, 2048, 9000, 4, 32, 8, 128, 4, 64, "bf16", True, keep=0.0),
        # That batch's caches brought down to a budget.
        evict("evict_batch", 64, 8192, 1, 8, 128, 4, 64, 2048, 4, 256),
        # Few very long caches.
        evict("evict_long", 4, 131072, 2, 8, 128, 4, 256, 16384, 16, 4096),
    ]


def _log_between(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("norm", "gated", "gated", "block", "weigh", "evict"))
    if op in ("weigh", "evict"):
        return _draw_cache(rng, op)
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


def _draw_cache(rng, op):
    dim, bits, page = rng.choice((64, 128, 128, 256)), rng.choice((4, 4, 8)), rng.choice((16, 32, 64, 128, 256))
    heads, ragged = rng.randint(1, 12), rng.randint(0, 1 << 20) if rng.random() < 0.8 else 0
    if op == "evict":
        kv = _log_between(rng, 1, 131072)
        seqs = min(_log_between(rng, 1, 64), max(1, 64 * 8192 * 8 * 128 // (kv * heads * dim)))
        budget = _log_between(rng, 1, kv)
        first = rng.choice((0, 0, 1, 4, 16))
        recent = rng.choice((0, 1, budget // 8, budget // 3))
        return dict(op=op, seqs=seqs, q=1, kv=kv, ragged=ragged, heads=heads, dim=dim, bits=bits, page=page, budget=budget,
                    first=min(first, budget - recent), recent=recent)
    group = rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 12, 16))
    if rng.random() < 0.5:   # single tokens and drafts over long caches
        q, kv = rng.choice((1, 1, 1, 2, 3, 6)), _log_between(rng, 1, 65536)
        seqs = min(_log_between(rng, 1, 64), max(1, 64 * 8192 * 8 * 128 // (kv * heads * dim)))
    else:                    # prompts
        q = _log_between(rng, 7, 4096)
        kv = min(q + rng.choice((0, _log_between(rng, 1, 4096))), 8192)
        seqs = rng.randint(1, 6)
        most = 12 * 4096 * 4096 * 128
        while seqs > 1 and seqs * heads * group * q * kv * dim > most:
            seqs -= 1
        while heads > 1 and seqs * heads * group * q * kv * dim > most:
            heads -= 1
        while seqs * heads * group * q * kv * dim > most:
            q, kv = q // 2, kv // 2
    causal = rng.random() < 0.7
    window = _log_between(rng, 1, max(2, kv)) if causal and rng.random() < 0.3 else 0
    return dict(op=op, seqs=seqs, q=q, kv=kv, ragged=ragged, q_heads=heads * group, heads=heads, dim=dim, bits=bits, page=page,
                dtype=rng.choice(("f16", "bf16")), causal=causal, window=window, keep=rng.choice((0.0, 0.5, 1.0, 1.0)))


def _lengths(case):
    """(query tokens, cached tokens) of each sequence; they follow from the case alone. The last
    sequence has the case's own lengths; a ragged batch's others are shorter."""
    n, q, kv = case["seqs"], case["q"], case["kv"]
    if not case["ragged"]:
        return [q] * n, [kv] * n
    rng = random.Random(case["ragged"])
    qs = [q if q < 8 else rng.randint(1, q) for _ in range(n - 1)] + [q]
    return qs, [rng.randint(min(x, kv), kv) for x in qs[:-1]] + [kv]


def _attended(case):
    """Pairs of a query token and a cached token it attends to, and the cached tokens that are
    attended to at all, over all sequences."""
    pairs = keys = 0
    for q, kv in zip(*_lengths(case)):
        if not case["causal"]:
            pairs, keys = pairs + q * kv, keys + kv
            continue
        first = kv - q + 1   # keys up to the first query's own position
        w = case["window"] or kv
        lo = [max(0, first + i) for i in (0, q - 1)]
        pairs += sum(min(max(0, first + i), w) for i in range(q))
        keys += lo[1] - max(0, lo[0] - w)
    return pairs, keys


def _rows(case):
    """Rows of the weights: the gated product has two for an output."""
    return case["N"] * (1 if case["op"] == "norm" else 2)


def work(case):
    if case["op"] == "weigh":
        pairs, keys = _attended(case)
        qs, kvs = _lengths(case)
        row = case["dim"] * case["bits"] // 8 + 4
        return {"bytes": keys * case["heads"] * row + sum(qs) * case["q_heads"] * (case["dim"] * 2 + 4) + keys // case["page"] * 4
                + sum(kvs) * case["heads"] * (8 if case["keep"] else 4), "flops": 2 * pairs * case["q_heads"] * case["dim"]}
    if case["op"] == "evict":
        kvs = _lengths(case)[1]
        kept = sum(min(x, case["budget"]) for x in kvs)
        row = 2 * (case["dim"] * case["bits"] // 8 + 4)
        return {"bytes": case["heads"] * (sum(kvs) * 4 + kept * (2 * row + 2 * 4 + 4)), "flops": case["heads"] * sum(kvs)}
    M, K, N = case["M"], case["K"], case["N"]
    rows = _rows(case)
    moved = M * K * 2 + rows * K * case["bits"] // 8 + rows * 4 * (2 if case["bias"] else 1) + M * N * 2
    flops = 2 * M * rows * K
    if case["op"] != "gated":
        moved += (2 * M * K * 2 if case["residual"] else 0) + K * (4 if case["weight"] == "f32" else 2)
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------------------- the plain form
def _rotate(x, block=128):
    """Unnormalised Walsh-Hadamard transform of blocks along the last axis."""
    h = 1
    while h < block:
        y = x.reshape(*x.shape[:-1], x.shape[-1] // (2 * h), 2, h)
        a, b = y[..., 0, :], y[..., 1, :]
        x = torch.stack((a + b, a - b), dim=-2).reshape(x.shape)
        h *= 2
    return x


def _norm(block):
    return torch.tensor(float(block), dtype=torch.float64).rsqrt().float().item()


def _quantise(x, bits, block=128):
    """Rows of the last axis -> (codes as binary32, scales)."""
    top = 127.0 if bits == 8 else 7.0
    u = _rotate(x, block)
    a = u.abs().amax(-1)
    top_of = torch.full_like(a, top)
    inv = top_of / a
    zero = torch.isinf(inv)
    inv = torch.where(zero, torch.zeros_like(inv), inv)
    scale = torch.where(zero, torch.zeros_like(a), (a * _norm(block)) / top_of)
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


def _row_bytes(case):
    return case["dim"] * case["bits"] // 8


def _head_bytes(case):
    return case["page"] * (2 * _row_bytes(case) + 8)


def _parts(blocks, case):
    """Views of head blocks [..., head bytes]: K codes [..., page, row], V codes [..., page / 4, row, 4],
    scales [..., 2, page] as bytes of four."""
    page, row = case["page"], _row_bytes(case)
    return (blocks[..., :page * row].unflatten(-1, (page, row)), blocks[..., page * row:2 * page * row].unflatten(-1, (page // 4, row, 4)),
            blocks[..., 2 * page * row:].unflatten(-1, (2, page, 4)))


def _weigh(s, case):
    n, heads, dim, page, top = case["seqs"], case["heads"], case["dim"], case["page"], min(128, case["dim"])
    group, span = case["q_heads"] // heads, s["pages"].shape[1] * page
    k, _, scales = _parts(s["cache"].view(-1, heads, _head_bytes(case))[s["pages"].clamp(min=0).long()], case)
    scale = scales[..., 0, :, :].contiguous().view(torch.float32)[..., 0]        # [seqs, pages, heads, page]
    K = _rotate(_unpack(k.view(torch.int8) if case["bits"] == 8 else k, case["bits"]), top)
    K = ((scale * top ** -0.5)[..., None] * K).transpose(1, 2).flatten(2, 3)     # [seqs, heads, tokens, dim]
    j = torch.arange(span, device=K.device)
    there = j[None] < s["kv_len"][:, None]
    K = torch.where(there[:, None, :, None], K, 0.0)
    # Query rows, padded to the longest sequence's.
    q0, q1 = s["q_start"][:-1, None], s["q_start"][1:, None]
    i = torch.arange(s["max_q_len"], device=K.device)[None]
    row = (q0 + i).clamp(max=s["Q"].shape[0] - 1).long()
    Q = s["Q"].float()[row].view(n, -1, heads, group, dim).permute(0, 2, 3, 1, 4)
    lse = s["lse"][row].view(n, -1, heads, group).permute(0, 2, 3, 1)
    S = torch.matmul(Q.reshape(n, heads, -1, dim), K.transpose(2, 3).contiguous()) * dim ** -0.5
    pos = (s["kv_len"][:, None] - (q1 - q0) + i)[:, :, None]
    ok = there[:, None] & (i < q1 - q0)[:, :, None]
    if case["causal"]:
        ok = ok & (j <= pos)
        if case["window"]:
            ok = ok & (j > pos - case["window"])
    P = torch.exp(S.view(n, heads, group, -1, span) - lse[..., None]).masked_fill(~ok[:, None, None], 0.0).sum((2, 3))
    if case["keep"]:
        old = s["weights"]
        if case["causal"]:   # the newest tokens had none before
            old = torch.where((j >= s["kv_len"][:, None] - (q1 - q0))[:, None], 0.0, old)
        P = P + case["keep"] * old
    s["weights"].copy_(torch.where(there[:, None], P, s["weights"]))
    return s["weights"]


def _evict(s, case):
    n, heads, page, W = case["seqs"], case["heads"], case["page"], s["weights"].shape[2]
    j, length = torch.arange(W, device=s["weights"].device), s["kv_len"][:, None, None]
    key = torch.where((j < case["first"]) | (j >= length - case["recent"]), float("inf"), s["weights"])
    key = torch.where(j < length, key, -1.0)
    order = torch.sort(key, dim=2, descending=True, stable=True)[1][:, :, :case["budget"]]
    if W < case["budget"]:
        order = torch.nn.functional.pad(order, (0, case["budget"] - W), value=W)
    at = torch.arange(case["budget"], device=j.device)
    kept = torch.sort(torch.where(at < length, order, 1 << 30), dim=2)[0]
    valid = kept < (1 << 30)
    src = kept.clamp(max=W - 1)
    # Only what is there is written: places behind a sequence's last token keep what they held.
    b, h, i = torch.nonzero(valid, as_tuple=True)
    j = src[b, h, i]
    blocks = s["cache"].view(-1, heads, _head_bytes(case))
    k, v, scales = _parts(blocks, case)
    from_page, to_page = s["pages"][b, j // page].long(), s["new_pages"][b, i // page].long()
    f, t = j % page, i % page
    new = k[from_page, h, f], v[from_page, h, f // 4, :, f % 4], scales[from_page, h, :, f]
    k[to_page, h, t], v[to_page, h, t // 4, :, t % 4], scales[to_page, h, :, t] = new
    s["new_weights"][b, h, i] = s["weights"][b, h, j]
    return {"cache": s["cache"], "kept": torch.where(valid, kept, -1).int(), "kv_len": s["kv_len"].clamp(max=case["budget"]),
            "weights": s["new_weights"]}


# -------------------------------------------------------------------------------- inputs, a pass
def _tokens(gen, M, K, dtype, dev):
    """Activations with a few large channels, as the layers see them."""
    x = torch.randn(M, K, generator=gen, device=dev)
    big = torch.randint(0, K, (max(1, K // 100),), generator=gen, device=dev)
    x[:, big] *= 30.0
    return x.to(dtype)


def _prepare_cache(case, gen, dev):
    heads, dim, page, bits = case["heads"], case["dim"], case["page"], case["bits"]
    qs, kvs = _lengths(case)
    most, need = -(-max(kvs) // page), [-(-x // page) for x in kvs]
    new = -(-case["budget"] // page) if case["op"] == "evict" else 0
    total = sum(need) + len(kvs) * new + 2
    # Pages as a reused pool holds them: bytes of whatever was there, in any order.
    cache = torch.randint(0, 256, (total, heads * _head_bytes(case)), generator=gen, device=dev, dtype=torch.uint8)
    order = torch.randperm(total, generator=gen, device=dev).int()
    pages = torch.full((len(kvs), most), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
    kv_len = torch.tensor(kvs, dtype=torch.int32, device=dev)
    # What tokens got so far: a few have most of it, many next to nothing, some the same.
    weights = torch.exp(2.5 * torch.randn(len(kvs), heads, most * page, generator=gen, device=dev))
    weights = torch.where(weights < 0.02, 0.0, weights)
    state = dict(cache=cache, pages=pages, kv_len=kv_len, weights=weights)
    if case["op"] == "evict":
        state.update(new_pages=order[at:at + len(kvs) * new].view(len(kvs), new).contiguous(),
                     new_weights=torch.zeros(len(kvs), heads, new * page, device=dev))
        return state
    weights *= sum(qs) * case["q_heads"] / heads / sum(kvs) / 20.0     # about what one call adds
    k, _, scales = _parts(cache.view(total, heads, _head_bytes(case)), case)
    K = torch.randn(total, heads, page, dim, generator=gen, device=dev)
    big = torch.randint(0, dim, (1, heads, 1, 2), generator=gen, device=dev).expand(total, -1, page, -1)
    K.scatter_(3, big, K.gather(3, big) * 6.0)
    codes, s = _quantise(K, bits, min(128, dim))
    k.copy_(_pack(codes, bits).view(torch.uint8))
    scales[:, :, 0] = s.view(torch.uint8).view(total, heads, page, 4)
    Q = torch.randn(sum(qs), case["q_heads"], dim, generator=gen, device=dev).to(_TORCH[case["dtype"]])
    starts = [0]
    for x in qs:
        starts.append(starts[-1] + x)
    state.update(Q=Q, q_start=torch.tensor(starts, dtype=torch.int32, device=dev), max_q_len=max(qs), max_kv_len=max(kvs))
    # The rows' log-sums, as attention returns them.
    lse, group = torch.empty(sum(qs), case["q_heads"], device=dev), case["q_heads"] // heads
    for b, (q, kv) in enumerate(zip(qs, kvs)):
        ok = _mask(case, q, kv, dev)
        rows = _keys64(state, case, b, kv).float()
        for h in range(heads):
            S = Q[starts[b]:starts[b + 1], h * group:(h + 1) * group].float().transpose(0, 1) @ rows[:, h].t().contiguous() * dim ** -0.5
            lse[starts[b]:starts[b + 1], h * group:(h + 1) * group] = torch.logsumexp(S.masked_fill(~ok, float("-inf")), 2).t()
    state["lse"] = lse
    return state


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)
    if case["op"] in ("weigh", "evict"):
        state = _prepare_cache(case, gen, dev)
        if own:
            import w4a4_integer_quantized_amd as rq
            state["rq"], state["cfg"] = rq, rq.make_kv_cfg(case["heads"], case["dim"], page_size=case["page"], bits=case["bits"])
        state["case"] = case
        return state
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
        return (_weigh if case["op"] == "weigh" else _evict if case["op"] == "evict" else _plain)(state, case)
    if case["op"] == "weigh":
        state["rq"].kv_attention_weights(
            state["Q"], state["lse"], state["cache"], state["pages"], state["kv_len"], state["cfg"], state["weights"],
            keep=case["keep"], q_start=state["q_start"], causal=case["causal"], window=case["window"],
            max_q_len=state["max_q_len"], max_kv_len=state["max_kv_len"])
        return state["weights"]
    if case["op"] == "evict":
        kept, kv_len = state["rq"].kv_evict(state["cache"], state["pages"], state["kv_len"], state["weights"], state["cfg"],
                                            case["budget"], state["new_pages"], state["new_weights"], first=case["first"],
                                            recent=case["recent"])
        return {"cache": state["cache"], "kept": kept, "kv_len": kv_len, "weights": state["new_weights"]}
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


def _mask(case, q, kv, dev):
    """[q, kv]: whether a query attends to a token."""
    behind = (kv - q + torch.arange(q, device=dev))[:, None] - torch.arange(kv, device=dev)
    ok = torch.ones(q, kv, dtype=torch.bool, device=dev)
    if case["causal"]:
        ok = behind >= 0
        if case["window"]:
            ok &= behind < case["window"]
    return ok


def _keys64(s, case, b, kv):
    """The keys [kv, heads, dim] that the cache stands for in sequence b."""
    page, row, dim, n = case["page"], _row_bytes(case), case["dim"], min(128, case["dim"])
    block = s["cache"].view(-1, case["heads"], _head_bytes(case))[s["pages"][b, :-(-kv // page)].long()]
    codes = _codes64(block[:, :, :page * row].reshape(-1, row), case["bits"]).view(-1, case["heads"], page, dim)
    scale = block[:, :, 2 * page * row:2 * page * row + 4 * page].contiguous().view(torch.float32).double()
    j = torch.arange(n, device=codes.device)
    odd = sum(((j[:, None] & j[None, :]) >> i) & 1 for i in range(7)) % 2
    K = torch.matmul((codes * scale[..., None]).view(-1, n), (1.0 - 2.0 * odd.double()) / n ** 0.5)
    return K.view(-1, case["heads"], page, dim).transpose(1, 2).flatten(0, 1)[:kv]


def _exact_weigh(s, case):
    out, group = s["weights"].double(), case["q_heads"] // case["heads"]
    at = 0
    for b, (q, kv) in enumerate(zip(*_lengths(case))):
        K, ok = _keys64(s, case, b, kv), _mask(case, q, kv, out.device)
        for g in range(case["heads"]):
            p = 0.0
            for h in range(g * group, (g + 1) * group):
                L = s["Q"][at:at + q, h].double() @ K[:, g].t() / case["dim"] ** 0.5
                p = p + torch.where(ok, torch.exp(L - s["lse"][at:at + q, h].double()[:, None]), 0.0).sum(0)
            old = case["keep"] * out[b, g, :kv]
            if case["causal"]:
                old[kv - q if kv > q else 0:] = 0.0
            out[b, g, :kv] = old + p
        at += q
    return out


def _exact_evict(s, case):
    kept = torch.full((case["seqs"], case["heads"], case["budget"]), -1, dtype=torch.int32, device=s["weights"].device)
    weights = s["new_weights"].double()
    for b, kv in enumerate(_lengths(case)[1]):
        for g in range(case["heads"]):
            w = s["weights"][b, g, :kv].double()
            if kv <= case["budget"]:
                take = torch.arange(kv, device=w.device)
            else:
                lo, hi = case["first"], kv - case["recent"]
                n = case["budget"] - case["first"] - case["recent"]
                # The n-th largest; everything above it, and of those beside it the first.
                edge = torch.topk(w[lo:hi], n)[0].min() if n else float("inf")
                take = w > edge
                beside = (w == edge) & (torch.arange(kv, device=w.device) >= lo) & (torch.arange(kv, device=w.device) < hi)
                take[:lo], take[hi:] = False, False
                room = n - int(take.sum())
                take |= beside & (beside.cumsum(0) <= room)
                take[:lo], take[hi:] = True, True
                take = take.nonzero()[:, 0]
            kept[b, g, :take.numel()] = take.int()
            weights[b, g, :take.numel()] = w[take]
    return {"cache": None, "kept": kept, "kv_len": None, "weights": weights}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("weigh", "evict"):
        return (_exact_weigh if case["op"] == "weigh" else _exact_evict)(s, case)
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
