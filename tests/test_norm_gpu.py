"""rq_norm_rotate_quantize on the GPU: h and codes exactly, scales within the bound of their sums."""
import numpy as np
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests import norm_ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

LAYOUTS = [(8, rq.RQ_X_ROWS), (8, rq.RQ_X_TILED), (4, rq.RQ_X_ROWS), (4, rq.RQ_X_TILED), (4, rq.RQ_X_FP6)]


def _case(M, K, dtype, residual, weight, seed):
    gen = torch.Generator().manual_seed(seed)
    t = norm_ref.TORCH[dtype]
    x = torch.randn(M, K, generator=gen)
    x[:, torch.randint(0, K, (max(1, K // 100),), generator=gen)] *= 30.0
    r = torch.randn(M, K, generator=gen).to(t) if residual else None
    w = (1.0 + 0.3 * torch.randn(K, generator=gen)).to(t if weight == "same" else torch.float32) if weight else None
    return x.to(t), r, w


def _check(Xq, scale, h, weight, eps, bits, layout, K):
    M = h.shape[0]
    codes, ref = norm_ref.reference(h, weight, eps, bits)
    got = norm_ref.codes_of(Xq, M, K, bits, layout, rq)
    assert np.array_equal(got, codes), "codes differ in %d places" % int((got != codes).sum())
    s = scale.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(s - ref) <= norm_ref.scale_error(K) * ref), np.abs(s / np.where(ref == 0, 1, ref) - 1).max()


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("bits,layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 128), (17, 128), (300, 256), (5, 640), (67, 1024), (33, 1152), (257, 1536), (19, 2176),
                                 (9, 2944), (4, 4096), (7, 5120), (3, 8192), (2, 8320), (3, 16384), (2, 16512), (1, 131072)])
def test_against_the_definition(M, K, dtype, bits, layout):
    need_gpu()
    print("norm", M, K, dtype, bits, layout, flush=True)
    k = K // 128 + bits + layout
    x, r, w = _case(M, K, dtype, k % 3 > 0, (None, "same", "f32")[k % 3 if dtype != "f32" else 2 * (k % 2)], K + M)
    h = norm_ref.hidden(x, r)
    X, R, W = _cuda(x, r, w)
    Xq, scale, H = rq.norm_rotate_quantize(X, R, W, eps=1e-5, bits=bits, x_layout=layout)
    if r is None:
        assert H is X
    assert torch.equal(H.cpu(), h)
    _check(Xq, scale, h, w, 1e-5, bits, layout, K)


@pytest.mark.parametrize("K", [1024, 4096, 16512])
def test_residual_and_weight_in_every_combination(K):
    need_gpu()
    for dtype in ("f16", "bf16"):
        for residual in (False, True):
            for weight in (None, "same", "f32"):
                x, r, w = _case(21, K, dtype, residual, weight, 7)
                h = norm_ref.hidden(x, r)
                X, R, W = _cuda(x, r, w)
                Xq, scale, H = rq.norm_rotate_quantize(X, R, W, bits=8, x_layout=rq.RQ_X_TILED)
                assert torch.equal(H.cpu(), h)
                _check(Xq, scale, h, w, 1e-6, 8, rq.RQ_X_TILED, K)


@pytest.mark.parametrize("K", [1024, 6144, 17408])
def test_h_in_the_place_of_an_input(K):
    need_gpu()
    x, r, w = _case(37, K, "bf16", True, "same", 3)
    h = norm_ref.hidden(x, r)
    for place in ("residual", "x", "both"):
        X, R, W = _cuda(x, r, w)
        if place == "both":
            R, h2 = X, norm_ref.hidden(x, x)
        else:
            h2 = h
        out = R if place == "residual" else X
        Xq, scale, H = rq.norm_rotate_quantize(X, R, W, out=out)
        assert H is out and torch.equal(out.cpu(), h2)
        _check(Xq, scale, h2, w, 1e-6, 8, rq.RQ_X_ROWS, K)
    X, = _cuda(x)
    out = torch.empty_like(X)
    _, _, H = rq.norm_rotate_quantize(X, None, W, out=out)
    assert H is out and torch.equal(out, X)


@pytest.mark.parametrize("K", [128, 1280, 4096, 16512])
def test_rows_with_strides_and_what_lies_between(K):
    need_gpu()
    M = 35
    x, r, w = _case(M, K, "f16", True, "f32", 5)
    h = norm_ref.hidden(x, r)
    both = torch.full((M, 2 * K + 24), -3.0, dtype=torch.float16, device="cuda")
    X, H = both[:, :K], both[:, K + 16:2 * K + 16]       # beside each other in one buffer
    X.copy_(x)
    W, = _cuda(w)
    R = torch.empty((M, K + 8), dtype=torch.float16, device="cuda")[:, 8:]
    R.copy_(r)
    Xq, scale, got = rq.norm_rotate_quantize(X, R, W, out=H, bits=4)
    assert torch.equal(got.cpu(), h) and torch.equal(X.cpu(), x)
    rest = torch.cat((both[:, K:K + 16], both[:, 2 * K + 16:]), 1)
    assert bool((rest == -3.0).all())
    _check(Xq, scale, h, w, 1e-6, 4, rq.RQ_X_ROWS, K)
    # One row for all of them.
    row = R[:1].expand(M, K)
    assert row.stride(0) == 0
    Xq, scale, got = rq.norm_rotate_quantize(X, row, W)
    h = norm_ref.hidden(x, r[:1].expand(M, K))
    assert torch.equal(got.cpu(), h)
    _check(Xq, scale, h, w, 1e-6, 8, rq.RQ_X_ROWS, K)


@pytest.mark.parametrize("bits,layout", LAYOUTS)
def test_rows_past_the_last_are_left(bits, layout):
    """Codes of rows past M, in the layouts that have them (pad rows of a panel), and what follows."""
    need_gpu()
    M, K = 19, 640
    x, r, w = _case(M, K, "bf16", True, "same", 9)
    X, R, W = _cuda(x, r, w)
    cfg = rq.make_cfg(bits, x_layout=layout)
    need = rq.rq_codes_bytes(M, K, cfg)
    buf = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((M + 300,), 7.0, device="cuda")
    H = torch.full((M + 5, K), 7.0, dtype=torch.bfloat16, device="cuda")
    p = rq.rq_norm_params(X.data_ptr(), R.data_ptr(), W.data_ptr(), H.data_ptr(), buf.data_ptr(), scale.data_ptr(), M, K, K, K, K,
                          rq.RQ_BF16, rq.RQ_BF16, 1e-6)
    assert rq.rq_norm_rotate_quantize(p, cfg, torch.cuda.current_stream().cuda_stream) == rq.RQ_OK
    torch.cuda.synchronize()
    assert bool((scale[M:] == 7.0).all()) and bool((H[M:] == 7.0).all()) and bool((buf[need:] == 0x5A).all())
    if layout == rq.RQ_X_TILED:
        panel = buf[:need].view(-1, 256, 64)
        assert bool((panel[:, M:] == 0x5A).all())
    if layout == rq.RQ_X_FP6:
        sl = buf[:need].view(-1, 256 * 48)
        assert bool((sl[:, M * 32:256 * 32] == 0x5A).all()) and bool((sl[:, 256 * 32 + M * 16:] == 0x5A).all())
    h = norm_ref.hidden(x, r)
    _check(buf[:need].view(M, -1) if layout == rq.RQ_X_ROWS else buf[:need], scale[:M], h, w, 1e-6, bits, layout, K)


@pytest.mark.parametrize("K", [512, 1024, 8192, 16512])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_any_size(K, dtype):
    """Squares beyond binary32's range and below it, zeros, one value alone, with and without eps."""
    need_gpu()
    t = norm_ref.TORCH[dtype]
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(12, K, generator=gen)
    sizes = torch.tensor([1e30, 3e18, 1e-3, 1e-20, 1e-25, 1e-30, 0.0, 1.0, 1e25, 1e-12, 2e19, 1e-35])
    x = (x * sizes[:, None]).to(t)
    x[7] = 0
    x[7, 5] = 1.0
    for eps in (0.0, 1e-6, 1e-30):
        X, = _cuda(x)
        for out in (None, torch.empty_like(X), X.clone()):
            src = out if out is not None and torch.equal(out, X) else X     # the last: in place
            Xq, scale, _ = rq.norm_rotate_quantize(src, None, None, eps=eps, out=out)
            _check(Xq, scale, x, None, eps, 8, rq.RQ_X_ROWS, K)


def test_a_row_that_is_no_number_touches_no_other():
    need_gpu()
    x, r, w = _case(40, 1024, "f16", True, "same", 2)
    h = norm_ref.hidden(x, r)
    x[11, 3], r[20, 100] = float("nan"), float("inf")
    X, R, W = _cuda(x, r, w)
    Xq, scale, H = rq.norm_rotate_quantize(X, R, W)
    keep = [i for i in range(40) if i not in (11, 20)]
    assert torch.equal(H.cpu()[keep], h[keep])
    _check(Xq[keep], scale[keep], h[keep], w, 1e-6, 8, rq.RQ_X_ROWS, 1024)


def test_no_rows():
    need_gpu()
    X = torch.empty((0, 256), dtype=torch.float16, device="cuda")
    for layout in (rq.RQ_X_ROWS, rq.RQ_X_TILED):
        Xq, scale, H = rq.norm_rotate_quantize(X, X, None, x_layout=layout)
        assert scale.shape == (0,) and H.shape == (0, 256)


def test_rows_past_4_gib():
    need_gpu()
    M, K = (1 << 21) + 3, 1024
    X = torch.full((M, K), 0.5, dtype=torch.float16, device="cuda")
    rows = [0, 1 << 20, M - 300, M - 1]
    x, r, _ = _case(len(rows), K, "f16", True, None, 4)
    X[rows] = x.cuda()
    R = torch.zeros_like(X)
    R[rows] = r.cuda()
    Xq, scale, H = rq.norm_rotate_quantize(X, R, None)
    h = norm_ref.hidden(x, r)
    assert torch.equal(H[rows].cpu(), h)
    _check(Xq[rows], scale[rows], h, None, 1e-6, 8, rq.RQ_X_ROWS, K)
    assert bool((H[1:1 << 20] == 0.5).all())


def test_streams_and_a_captured_call():
    need_gpu()
    x, r, w = _case(130, 2176, "bf16", True, "same", 6)
    X, R, W = _cuda(x, r, w)
    h = norm_ref.hidden(x, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    Xq, scale, H = rq.norm_rotate_quantize(X, R, W, stream=side)
    side.synchronize()
    assert torch.equal(H.cpu(), h)
    _check(Xq, scale, h, w, 1e-6, 8, rq.RQ_X_ROWS, 2176)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Xq2, scale2, H2 = rq.norm_rotate_quantize(X, R, W, x_layout=rq.RQ_X_TILED)
    for i in range(4):
        X.copy_(torch.roll(x, i, 0))
        R.copy_(torch.roll(r, i, 0))
        eager = rq.norm_rotate_quantize(X, R, W, x_layout=rq.RQ_X_TILED)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = norm_ref.codes_of(Xq2, 130, 2176, 8, rq.RQ_X_TILED, rq)
        assert np.array_equal(got, norm_ref.codes_of(eager[0], 130, 2176, 8, rq.RQ_X_TILED, rq))
        assert torch.equal(scale2, eager[1]) and torch.equal(H2, eager[2])


def test_equal_calls_give_equal_bits():
    need_gpu()
    x, r, w = _case(513, 5120, "f16", True, "f32", 8)
    X, R, W = _cuda(x, r, w)
    first = rq.norm_rotate_quantize(X, R, W)
    for _ in range(3):
        again = rq.norm_rotate_quantize(X, R, W)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_codes_feed_the_products():
    """Norm, then gemm_dequant and rotq's own GEMM layouts: the same as a linear over codes given by hand."""
    need_gpu()
    x, r, w = _case(300, 1024, "f16", True, "same", 12)
    X, R, W = _cuda(x, r, w)
    Wl = torch.randn(256, 1024, generator=torch.Generator().manual_seed(1)).cuda() * 0.03
    for bits, layout, wl in ((8, rq.RQ_X_TILED, rq.RQ_W_ROWS), (8, rq.RQ_X_ROWS, rq.RQ_W_ROWS), (4, rq.RQ_X_FP6, rq.RQ_W_FP6)):
        Wq, ws = rq.quantize_weights(Wl, bits=bits, w_layout=wl)
        Xq, scale, _ = rq.norm_rotate_quantize(X, R, W, bits=bits, x_layout=layout)
        Y = rq.gemm_dequant(Xq, scale, Wq, ws, bits=bits, K=1024, x_layout=layout, w_layout=wl)
        codes, ref = norm_ref.reference(norm_ref.hidden(x, r), w, 1e-6, bits)
        wc = norm_ref.codes_of(rq.quantize_weights(Wl, bits=bits)[0], 256, 1024, bits, rq.RQ_X_ROWS, rq)
        exact = (codes.astype(np.float64) * ref[:, None]) @ (wc.astype(np.float64) * ws.cpu().numpy().astype(np.float64)[:, None]).T
        y = Y.cpu().double().numpy()
        # One rounding to fp16 and a few of binary32; below fp16's normal range a step is 2^-24.
        assert np.all(np.abs(y - exact) <= (2.0 ** -11 + 2.0 ** -19) * np.abs(exact) + 2.0 ** -25)


@pytest.mark.parametrize("M", [3, 65537])
def test_one_residual_row_in_a_gap_of_h(M):
    need_gpu()
    K = 256
    x, r, w = _case(M, K, "bf16", True, "same", 11)
    X, W = _cuda(x, w)
    both = torch.full((M, 2 * K), -3.0, dtype=torch.bfloat16, device="cuda")
    both[0, K:] = r[0].cuda()
    keep = both[:, K:].clone()
    row = both[:1, K:].expand(M, K)
    Xq, scale, H = rq.norm_rotate_quantize(X, row, W, out=both[:, :K])
    h = norm_ref.hidden(x, r[:1].expand(M, K))
    assert torch.equal(H.cpu(), h) and torch.equal(both[:, K:], keep)
    _check(Xq[:50], scale[:50], h[:50], w, 1e-6, 8, rq.RQ_X_ROWS, K)
    _check(Xq[-50:], scale[-50:], h[-50:], w, 1e-6, 8, rq.RQ_X_ROWS, K)
