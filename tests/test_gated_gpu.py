"""The gated product of two projections on the GPU, over every kernel that a call may take."""
import numpy as np
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests import gated_ref, norm_ref
from tests.gpu_util import fp6_tile, need_gpu, tile_codes

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def _operands(M, K, N, bits, seed, bias=True):
    """Codes and scales (device) as the quantizers give them, of inputs whose products are about 1."""
    gen = torch.Generator("cuda").manual_seed(seed)
    top = 127 if bits == 8 else 7
    xc = torch.randint(-top, top + 1, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    wc = torch.randint(-top, top + 1, (2 * N, K), generator=gen, device="cuda", dtype=torch.int8)
    unit = 3.0 / (K ** 0.5 * top * top)        # a product of uniform codes is about top^2 / 3
    xs = (0.5 + torch.rand(M, generator=gen, device="cuda")) * unit
    ws = 0.5 + torch.rand(2 * N, generator=gen, device="cuda")
    b = torch.randn(2 * N, generator=gen, device="cuda") if bias else None
    return xc, xs, wc, ws, b


def _packed(codes, bits):
    if bits == 8:
        return codes
    c = codes.to(torch.int16) & 15
    return (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8)


def _x_buffer(xc, bits, layout):
    M, K = xc.shape
    if layout == rq.RQ_X_ROWS:
        return _packed(xc, bits).contiguous()
    if layout == rq.RQ_X_TILED:
        return torch.from_numpy(tile_codes(_packed(xc, bits).cpu().numpy(), M, K, bits)).cuda()
    return torch.from_numpy(fp6_tile(xc.cpu().numpy(), 256)).cuda()


def _run(M, K, N, bits, layout, dtype, act, bias=True, seed=0):
    xc, xs, wc, ws, b = _operands(M, K, N, bits, seed + M + K + N, bias)
    fp6 = layout == rq.RQ_X_FP6
    Wq = torch.from_numpy(fp6_tile(wc.cpu().numpy(), 128)).cuda() if fp6 else _packed(wc, bits).contiguous()
    out = torch.full((M + 3, N), -7.0, dtype=TORCH[dtype], device="cuda")
    Y = rq.gemm_gated(_x_buffer(xc, bits, layout), xs, Wq, ws, b, bits=bits, K=K, x_layout=layout,
                      w_layout=rq.RQ_W_FP6 if fp6 else rq.RQ_W_ROWS, act=gated_ref.ACTS.index(act), out=out[:M])
    y, bound = gated_ref.reference(xc, xs, wc, ws, b, act, TORCH[dtype])
    gated_ref.check(Y, y, bound)
    assert bool((out[M:] == -7.0).all())
    return Y


LAYOUTS = [(8, rq.RQ_X_ROWS), (8, rq.RQ_X_TILED), (4, rq.RQ_X_ROWS), (4, rq.RQ_X_TILED), (4, rq.RQ_X_FP6)]


@pytest.mark.parametrize("bits,layout", LAYOUTS)
@pytest.mark.parametrize("M,K,N", [(1, 128, 16), (1, 4096, 528), (2, 2176, 80), (5, 384, 48), (16, 1024, 1040), (17, 640, 16),
                                   (31, 8192, 32), (33, 1152, 272), (64, 2048, 528), (65, 1024, 64), (127, 512, 112), (90, 1152, 528),
                                   (255, 1536, 16), (256, 256, 144), (300, 1024, 1040), (700, 896, 1024)])
def test_sizes(M, K, N, bits, layout):
    need_gpu()
    print("gated", M, K, N, bits, layout, flush=True)
    k = M + N // 16 + bits
    _run(M, K, N, bits, layout, ("f16", "bf16")[k % 2], gated_ref.ACTS[k % 4], bias=k % 3 > 0)


@pytest.mark.parametrize("bits,layout", LAYOUTS)
@pytest.mark.parametrize("M,K,N", [(4103, 1024, 1040), (4103, 1536, 1040), (4103, 2048, 1040), (4103, 3200, 1040), (2303, 6400, 2064)])
def test_more_tiles_than_cus(M, K, N, bits, layout):
    need_gpu()
    print("gated", M, K, N, bits, layout, flush=True)
    _run(M, K, N, bits, layout, "f16" if bits == 8 else "bf16", "silu")


@pytest.mark.parametrize("M", [1, 20, 40, 64, 90, 128])
@pytest.mark.parametrize("N", [4096, 4112, 6144, 11264, 16000])
def test_few_tokens_over_many_rows(M, N):
    """Workgroups of one to four blocks, the last of them not full; 128 tokens on either side of the tiles."""
    need_gpu()
    _run(M, 640, N, 8, rq.RQ_X_TILED, "bf16", "silu")
    _run(M, 384, N, 4, rq.RQ_X_ROWS, "f16", "none")
    _run(M, 384, N, 4, rq.RQ_X_FP6, "bf16", "gelu_tanh")


@pytest.mark.parametrize("act", gated_ref.ACTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M", [1, 20, 400])
def test_activations(M, dtype, act):
    need_gpu()
    for bits, layout in LAYOUTS:
        _run(M, 1024, 272, bits, layout, dtype, act, bias=True, seed=1)
        _run(M, 256, 48, bits, layout, dtype, act, bias=False, seed=2)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gates_of_any_size(M):
    """Gates from far below zero, where the activation vanishes, to far above; products out of fp16's range."""
    need_gpu()
    for act in gated_ref.ACTS:
        for dtype in ("f16", "bf16"):
            xc, xs, wc, ws, _ = _operands(M, 256, 64, 8, 5)
            b = torch.zeros(128, device="cuda")
            b.view(-1, 2, 16)[:, 0] = torch.linspace(-120.0, 60.0, 64, device="cuda").view(-1, 16)
            b.view(-1, 2, 16)[:, 1] = 30.0
            Y = rq.gemm_gated(xc, xs, wc, ws, b, act=gated_ref.ACTS.index(act), out_dtype=TORCH[dtype])
            y, bound = gated_ref.reference(xc, xs, wc, ws, b, act, TORCH[dtype])
            gated_ref.check(Y, y, bound)
    xs = xs * 1e4
    Y = rq.gemm_gated(xc, xs, wc, ws, None, act=rq.RQ_ACT_NONE)
    y, _ = gated_ref.reference(xc, xs, wc, ws, None, "none", torch.float16)
    over = y.abs() > 65536.0
    assert bool(over.any()) and bool(torch.isinf(Y[over]).all()) and torch.equal(Y[over] > 0, y[over] > 0)


@pytest.mark.parametrize("w_layout,bits", [(rq.RQ_W_ROWS, 8), (rq.RQ_W_ROWS, 4), (rq.RQ_W_FP6, 4)])
@pytest.mark.parametrize("M", [1, 9, 64, 333])
def test_from_the_activations(M, w_layout, bits):
    """rotq_gated_linear: codes as rotate_quantize gives them, weights as quantize_gated_weights does."""
    need_gpu()
    K, N = 1152, 144
    gen = torch.Generator("cuda").manual_seed(M)
    X = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16)
    gate, up = (torch.randn(N, K, generator=gen, device="cuda") * 0.03 for _ in range(2))
    b = torch.randn(2 * N, generator=gen, device="cuda")
    Wq, ws = rq.quantize_gated_weights(gate, up, bits=bits, w_layout=w_layout)
    Wr, wr = rq.quantize_gated_weights(gate, up, bits=bits)
    assert torch.equal(ws, wr)
    Xr, xs = rq.rotate_quantize(X, bits=bits)
    xc = torch.from_numpy(norm_ref.codes_of(Xr, M, K, bits, rq.RQ_X_ROWS, rq)).cuda()
    wc = torch.from_numpy(norm_ref.codes_of(Wr, 2 * N, K, bits, rq.RQ_X_ROWS, rq)).cuda()
    # The interleaved rows are those of the two matrices.
    for part, W in enumerate((gate, up)):
        c, s = rq.quantize_weights(W, bits=bits)
        assert torch.equal(Wr.view(-1, 2, 16, Wr.shape[1])[:, part].reshape(c.shape), c)
        assert torch.equal(ws.view(-1, 2, 16)[:, part].flatten(), s)
    y, bound = gated_ref.reference(xc, xs, wc, ws, b, "silu", torch.bfloat16)
    Y = rq.rotq_gated_linear(X, Wq, ws, b, bits=bits, w_layout=w_layout)
    gated_ref.check(Y, y, bound)
    ws_buf = torch.full((rq.workspace_size(M, K, bits, w_layout),), 0xAA, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(Y)
    assert rq.rotq_gated_linear(X, Wq, ws, b, bits=bits, w_layout=w_layout, workspace=ws_buf, out=out) is out
    assert torch.equal(out, Y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = rq.rotq_gated_linear(X, Wq, ws, b, bits=bits, w_layout=w_layout, stream=side)
    side.synchronize()
    assert torch.equal(again, Y)


def test_other_scale_rules():
    need_gpu()
    gen = torch.Generator("cuda").manual_seed(3)
    gate, up = (torch.randn(64, 256, generator=gen, device="cuda") * s for s in (0.1, 0.4))
    for mode in (rq.RQ_W_MSE, rq.RQ_W_TENSOR):
        Wq, ws = rq.quantize_gated_weights(gate, up, w_scale_mode=mode)
        c, s = rq.quantize_weights(rq.interleave_gated(gate, up), w_scale_mode=mode)
        assert torch.equal(Wq, c) and torch.equal(ws, s)
    assert bool((ws == ws[0]).all())


@pytest.mark.parametrize("M", [1, 30, 200])
def test_a_feed_forward_layer(M):
    """Norm with the residual, gated product, down projection and the next residual, each step against
    its reference on what the step before gave."""
    need_gpu()
    K, N = 1024, 1408
    gen = torch.Generator("cuda").manual_seed(M)
    dt = torch.bfloat16
    x, res = (torch.randn(M, K, generator=gen, device="cuda").to(dt) for _ in range(2))
    w = (1 + 0.1 * torch.randn(K, generator=gen, device="cuda")).to(dt)
    gate, up = (torch.randn(N, K, generator=gen, device="cuda") * 0.03 for _ in range(2))
    down = torch.randn(K, N, generator=gen, device="cuda") * 0.03
    for bits, xl, wl in ((8, rq.RQ_X_TILED, rq.RQ_W_ROWS), (4, rq.RQ_X_FP6, rq.RQ_W_FP6)):
        Wq, ws = rq.quantize_gated_weights(gate, up, bits=bits, w_layout=wl)
        Dq, ds = rq.quantize_weights(down, bits=bits, w_layout=wl)
        Xq, xs, h = rq.norm_rotate_quantize(x, res, w, bits=bits, x_layout=xl)
        y = rq.gemm_gated(Xq, xs, Wq, ws, bits=bits, K=K, out_dtype=dt, x_layout=xl, w_layout=wl)
        z = rq.rotq_linear(y, Dq, ds, bits=bits, w_layout=wl)
        Zq, zs, h2 = rq.norm_rotate_quantize(z, h, w, bits=bits, x_layout=xl, out=h.clone())
        assert torch.equal(h.cpu(), norm_ref.hidden(x.cpu(), res.cpu()))
        codes, scale = norm_ref.reference(h.cpu(), w.cpu(), 1e-6, bits)
        assert np.array_equal(norm_ref.codes_of(Xq, M, K, bits, xl, rq), codes)
        wc = torch.from_numpy(norm_ref.codes_of(rq.quantize_gated_weights(gate, up, bits=bits)[0], 2 * N, K, bits, rq.RQ_X_ROWS, rq))
        gated_ref.check(y, *gated_ref.reference(torch.from_numpy(codes).cuda(), xs, wc.cuda(), ws, None, "silu", dt))
        yc, ys = rq.rotate_quantize(y, bits=bits)
        yc = torch.from_numpy(norm_ref.codes_of(yc, M, N, bits, rq.RQ_X_ROWS, rq)).cuda().double()
        dc = torch.from_numpy(norm_ref.codes_of(rq.quantize_weights(down, bits=bits)[0], K, N, bits, rq.RQ_X_ROWS, rq)).cuda().double()
        exact = (yc @ dc.t().contiguous()) * (ys[:, None] * ds[None]).double()
        assert bool(((z.double() - exact).abs() <= exact.abs() * (2.0 ** -8 + 2.0 ** -20)).all())
        assert torch.equal(h2.cpu(), norm_ref.hidden(z.cpu(), h.cpu()))
        codes, _ = norm_ref.reference(h2.cpu(), w.cpu(), 1e-6, bits)
        assert np.array_equal(norm_ref.codes_of(Zq, M, K, bits, xl, rq), codes)


@pytest.mark.parametrize("M", [1, 48, 300])
def test_captured_layer(M):
    """A captured feed-forward layer, replayed with other inputs and eager work between."""
    need_gpu()
    K, N = 1024, 528
    gen = torch.Generator("cuda").manual_seed(M)
    x, res = (torch.randn(M, K, generator=gen, device="cuda").half() for _ in range(2))
    gate, up = (torch.randn(N, K, generator=gen, device="cuda") * 0.03 for _ in range(2))
    Wq, ws = rq.quantize_gated_weights(gate, up)

    def layer():
        Xq, xs, h = rq.norm_rotate_quantize(x, res, None, x_layout=rq.RQ_X_TILED)
        return h, rq.gemm_gated(Xq, xs, Wq, ws, K=K, x_layout=rq.RQ_X_TILED), rq.rotq_gated_linear(x, Wq, ws)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for _ in range(4):
        x.copy_(torch.randn(M, K, generator=gen, device="cuda"))
        want = layer()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_rows_and_equal_bits():
    need_gpu()
    xc, xs, wc, ws, b = _operands(70, 1024, 272, 8, 1)
    assert rq.gemm_gated(xc[:0], xs[:0], wc, ws, b).shape == (0, 272)
    assert rq.rotq_gated_linear(torch.empty((0, 1024), dtype=torch.float16, device="cuda"), wc, ws, b).shape == (0, 272)
    first = rq.gemm_gated(xc, xs, wc, ws, b)
    for _ in range(3):
        assert torch.equal(rq.gemm_gated(xc, xs, wc, ws, b), first)
    # A row's outputs do not depend on the rows beside it.
    for m in (1, 7, 16, 17, 33, 64):
        assert torch.equal(rq.gemm_gated(xc[:m].contiguous(), xs[:m].contiguous(), wc, ws, b), first[:m])
