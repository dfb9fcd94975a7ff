"""The gated product's checks and weight layout (no GPU: refused calls launch nothing)."""
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests.test_abi import A, GB


def _gemm(cfg=None, M=16, N=32, K=256, y_dtype=rq.RQ_F16, **kw):
    p = dict(Xq=A, x_scale=A + GB, Wq=A + 2 * GB, w_scale=A + 3 * GB, bias=A + 4 * GB, Y=A + 5 * GB)
    p.update(kw)
    return rq.rq_gemm_gated(p["Xq"], p["x_scale"], p["Wq"], p["w_scale"], p["bias"], M, N, K, cfg or rq.make_cfg(8, act=rq.RQ_ACT_SILU),
                            p["Y"], y_dtype, None)


def _linear(cfg=None, M=16, N=32, K=256, x_dtype=rq.RQ_F16, ws_bytes=None, **kw):
    p = dict(X=A, Wq=A + 2 * GB, w_scale=A + 3 * GB, bias=A + 4 * GB, Y=A + 5 * GB, ws=A + 6 * GB)
    p.update(kw)
    cfg = cfg or rq.make_cfg(8, act=rq.RQ_ACT_SILU)
    if ws_bytes is None:
        ws_bytes = rq.rq_rotq_linear_workspace_size(M, K, cfg)
    return rq.rq_rotq_gated_linear(p["X"], x_dtype, M, K, p["Wq"], p["w_scale"], N, p["bias"], cfg, p["Y"], p["ws"], ws_bytes, None)


SHARED = [
    (dict(K=200), rq.RQ_EUNSUPPORTED), (dict(N=24), rq.RQ_EUNSUPPORTED), (dict(N=0), rq.RQ_EUNSUPPORTED), (dict(M=-1), rq.RQ_EINVAL),
    (dict(N=1 << 30), rq.RQ_EUNSUPPORTED), (dict(M=1 << 25, N=1 << 14), rq.RQ_EUNSUPPORTED),
    (dict(Wq=None), rq.RQ_EINVAL), (dict(w_scale=None), rq.RQ_EINVAL), (dict(Y=None), rq.RQ_EINVAL),
    (dict(Wq=A + 2 * GB + 8), rq.RQ_EINVAL), (dict(bias=A + 4 * GB + 4), rq.RQ_EINVAL), (dict(Y=A + 5 * GB + 2), rq.RQ_EINVAL),
    (dict(Y=A + 2 * GB + 64 * 256 - 16), rq.RQ_EINVAL), (dict(Y=A + 3 * GB + 128), rq.RQ_EINVAL), (dict(Y=A + 4 * GB), rq.RQ_EINVAL),
    (dict(Y=A), rq.RQ_EINVAL),
    (dict(cfg=rq.make_cfg(8, act=4)), rq.RQ_EINVAL), (dict(cfg=rq.make_cfg(8, act=-1)), rq.RQ_EINVAL),
    (dict(cfg=rq.make_cfg(6)), rq.RQ_EUNSUPPORTED), (dict(cfg=rq.make_cfg(8, w_layout=rq.RQ_W_FP6)), rq.RQ_EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(Xq=None), rq.RQ_EINVAL), (dict(Xq=A + 4), rq.RQ_EINVAL), (dict(x_scale=None), rq.RQ_EINVAL), (dict(x_scale=A + GB + 2), rq.RQ_EINVAL),
    (dict(Y=A + GB), rq.RQ_EINVAL), (dict(y_dtype=rq.RQ_F32), rq.RQ_EUNSUPPORTED), (dict(y_dtype=5), rq.RQ_EINVAL),
    (dict(cfg=rq.make_cfg(4, x_layout=rq.RQ_X_FP6)), rq.RQ_EINVAL), (dict(cfg=rq.make_cfg(4, w_layout=rq.RQ_W_FP6)), rq.RQ_EINVAL),
])
def test_gemm_refused(kw, status):
    assert _gemm(**kw) == status
    assert rq.load().rq_last_error_detail().decode()


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(X=None), rq.RQ_EINVAL), (dict(X=A + 4), rq.RQ_EINVAL), (dict(ws=None), rq.RQ_EINVAL), (dict(ws=A + 6 * GB + 8), rq.RQ_EINVAL),
    (dict(ws_bytes=100), rq.RQ_EWORKSPACE), (dict(ws=A + 16), rq.RQ_EINVAL), (dict(ws=A + 5 * GB), rq.RQ_EINVAL),
    (dict(ws=A + 2 * GB), rq.RQ_EINVAL), (dict(ws=A + 3 * GB), rq.RQ_EINVAL), (dict(ws=A + 4 * GB), rq.RQ_EINVAL),
    (dict(x_dtype=rq.RQ_F32), rq.RQ_EUNSUPPORTED), (dict(x_dtype=7), rq.RQ_EINVAL),
])
def test_linear_refused(kw, status):
    assert _linear(**kw) == status
    assert rq.load().rq_last_error_detail().decode()


def test_no_rows_launch_nothing():
    for act in range(4):
        assert _gemm(rq.make_cfg(8, act=act), M=0) == rq.RQ_OK
        assert _linear(rq.make_cfg(4, w_layout=rq.RQ_W_FP6, act=act), M=0) == rq.RQ_OK


def test_silu_belongs_to_the_gated_products():
    """One configuration serves the whole block, but a plain linear does not apply SiLU."""
    cfg = rq.make_cfg(8, act=rq.RQ_ACT_SILU)
    assert rq.rq_codes_bytes(5, 256, cfg) == 5 * 256 and rq.rq_weight_bytes(64, 256, cfg) == 64 * 256
    assert rq.rq_rotq_linear_workspace_size(300, 1024, cfg) == rq.rq_rotq_linear_workspace_size(300, 1024, rq.make_cfg(8))
    assert rq.rq_rotate_quantize(A, rq.RQ_F16, 0, 128, cfg, A + GB, A + 2 * GB, None) == rq.RQ_OK
    assert rq.rq_gemm_dequant(A, A + GB, A + 2 * GB, A + 3 * GB, None, 16, 32, 128, cfg, A + 4 * GB, rq.RQ_F16, None) == rq.RQ_EINVAL
    assert rq.rq_rotq_linear_noalloc(A, rq.RQ_F16, 16, 128, A + GB, A + 2 * GB, 32, None, cfg, A + 3 * GB, None) == rq.RQ_EINVAL


def test_interleaved_rows():
    gate, up = torch.arange(48 * 2).view(48, 2), -torch.arange(48 * 2).view(48, 2)
    both = rq.interleave_gated(gate, up)
    for row in range(96):
        i, r = divmod(row, 32)
        assert torch.equal(both[row], (gate if r < 16 else up)[16 * i + r % 16])
    assert torch.equal(rq.interleave_gated(gate[:, 0], up[:, 0]), both[:, 0])
    for bad in ((gate[:40], up[:40]), (gate, up[:32]), (gate, up.float()), (gate[None], up[None])):
        with pytest.raises(ValueError):
            rq.interleave_gated(*bad)


def test_wrapper_refusals():
    X = torch.zeros(4, 256, dtype=torch.float16)
    Xq, xs, Wq, ws, b = torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4), torch.zeros(64, 256, dtype=torch.int8), torch.zeros(64), torch.zeros(64)
    with pytest.raises(ValueError, match="device tensor"):
        rq.rotq_gated_linear(X, Wq, ws, b)
    with pytest.raises(ValueError, match="device tensor"):
        rq.gemm_gated(Xq, xs, Wq, ws, b)
    for kw in (dict(w_scale=torch.zeros(48)), dict(w_scale=ws.half()), dict(bias=torch.zeros(32)), dict(Wq=Wq[:32]),
               dict(out=torch.zeros(4, 64, dtype=torch.float16)), dict(out=torch.zeros(4, 32, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            rq.rotq_gated_linear(**{**dict(X=X, Wq=Wq, w_scale=ws, bias=b), **kw})
    for bad in (X.float(), X[:, :128].t(), X[0], torch.zeros(4, 512, dtype=torch.float16)[:, ::2]):
        with pytest.raises(ValueError):
            rq.rotq_gated_linear(bad, Wq, ws, b)
    with pytest.raises(ValueError):
        rq.rotq_gated_linear(X, Wq, ws, b, workspace=torch.zeros(100, dtype=torch.uint8))
    for kw in (dict(Xq=Xq[:3]), dict(x_scale=xs.half()), dict(out_dtype=torch.float32), dict(out=torch.zeros(4, 32)),
               dict(out=torch.zeros(4, 32, dtype=torch.float16), out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            rq.gemm_gated(**{**dict(Xq=Xq, x_scale=xs, Wq=Wq, w_scale=ws, bias=b), **kw})
