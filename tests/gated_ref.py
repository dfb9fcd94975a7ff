"""The gated product's plain implementation for the tests: exact integer accumulators and everything
behind them in 64 bits, with the bound that a binary32 epilogue and one rounding keep."""
import torch

U32 = 2.0 ** -24
ACTS = ("none", "gelu_erf", "gelu_tanh", "silu")      # by their RQ_ACT_* values


def _act(g, act):
    """(A(g), A'(g), relative error of a binary32 evaluation of A at g)."""
    if act == "none":
        return g, torch.ones_like(g), torch.zeros_like(g)
    if act == "silu":
        # exp(-|g|) with its argument rounded (|g| log2 e, then + 32) and a few roundings and native ulps.
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), (16 + 4 * g.abs()) * U32
    if act == "gelu_erf":
        # As act_window() of the plain linears' tests.
        phi = 0.5 * torch.erfc(-g / 2 ** 0.5)
        return g * phi, phi + g * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5, 2.0 ** -18 + g * g / 2 * 2.0 ** -19
    u = (2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(2 * u)
    return g * s, s + g * s * (1 - s) * 2 * (2 / torch.pi) ** 0.5 * (1 + 3 * 0.044715 * g * g), 2.0 ** -18 + u.abs() * 2.0 ** -18


def reference(xc, xs, wc, ws, bias, act, dtype):
    """(y, bound) float64 [M, N] on the operands' device: codes xc [M, K] and wc [2 N, K] int8 in the
    interleaved order, scales float32, bias float32 [2 N] or None."""
    acc = xc.double() @ wc.double().t().contiguous()         # exact: below 2^53
    v = acc * (ws[None] * xs[:, None]).double()              # the scales' product is rounded to binary32
    if bias is not None:
        v = v + bias.double()
    v = v.view(v.shape[0], -1, 2, 16)
    g, u = v[:, :, 0].flatten(1), v[:, :, 1].flatten(1)
    a, da, w = _act(g, act)
    y = a * u
    half, small = (2.0 ** -11, 2.0 ** -25) if dtype == torch.float16 else (2.0 ** -8, 2.0 ** -134)
    # g and u are rounded once (their fma), A to w, the product once; what is below binary32's normal
    # range may be taken for zero in A. Then one rounding to the output type.
    inner = (da * g * u).abs() * U32 + y.abs() * (w + 2 * U32) + u.abs() * 2.0 ** -126
    return y, inner * (1 + half) + y.abs() * half + small


def check(got, y, bound):
    top = 65500.0 if got.dtype == torch.float16 else float("inf")
    got = got.double()
    bad = ~((got - y).abs() <= bound) & (y.abs() < top)
    assert not bool(bad.any()), "%d of %d off, the worst %.3g times its bound" % (
        int(bad.sum()), bad.numel(), float(((got - y).abs() / bound).nan_to_num(posinf=0).max()))
