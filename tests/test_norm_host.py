"""rq_norm_rotate_quantize's checks (no GPU: refused calls launch nothing)."""
import ctypes
import re

import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests.test_abi import A, GB, HEADER


def _params(**kw):
    p = dict(X=A, residual=A + GB, weight=A + 2 * GB, H=A + 3 * GB, Xq=A + 4 * GB, x_scale=A + 5 * GB, M=16, K=256, x_stride=256,
             residual_stride=256, h_stride=256, dtype=rq.RQ_BF16, w_dtype=rq.RQ_BF16, eps=1e-6)
    p.update(kw)
    return rq.rq_norm_params(*p.values())


def _status(cfg=None, **kw):
    return rq.rq_norm_rotate_quantize(_params(**kw), cfg or rq.make_cfg(8), None)


def test_struct_matches_header():
    body = re.search(r"typedef struct \{([^{}]*)\} rq_norm_params;", open(HEADER).read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip(" *") for line in body.split(";") if line.strip() for n in re.sub(r"^(const )?\w+ ", "", line.strip()).split(",")]
    assert [n for n, _ in rq.rq_norm_params._fields_] == names
    assert ctypes.sizeof(rq.rq_norm_params) == 6 * 8 + 5 * 8 + 2 * 4 + 4 + 4


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), rq.RQ_EINVAL), (dict(Xq=None), rq.RQ_EINVAL), (dict(x_scale=None), rq.RQ_EINVAL),
    (dict(X=A + 8), rq.RQ_EINVAL), (dict(residual=A + GB + 2), rq.RQ_EINVAL), (dict(weight=A + 2 * GB + 4), rq.RQ_EINVAL),
    (dict(H=A + 3 * GB + 8), rq.RQ_EINVAL), (dict(x_scale=A + 5 * GB + 2), rq.RQ_EINVAL),
    (dict(dtype=3), rq.RQ_EINVAL), (dict(w_dtype=rq.RQ_F16), rq.RQ_EINVAL), (dict(w_dtype=9), rq.RQ_EINVAL),
    (dict(eps=-1.0), rq.RQ_EINVAL), (dict(eps=float("nan")), rq.RQ_EINVAL), (dict(eps=float("inf")), rq.RQ_EINVAL),
    (dict(M=-1), rq.RQ_EINVAL), (dict(K=200), rq.RQ_EUNSUPPORTED), (dict(K=131200), rq.RQ_EUNSUPPORTED),
    (dict(x_stride=-8), rq.RQ_EINVAL), (dict(x_stride=257), rq.RQ_EINVAL), (dict(x_stride=(1 << 26) + 8), rq.RQ_EINVAL),
    (dict(residual_stride=4), rq.RQ_EINVAL), (dict(h_stride=248), rq.RQ_EINVAL), (dict(h_stride=0), rq.RQ_EINVAL),
    (dict(M=1 << 27, K=8192, x_stride=0, residual=None, H=None), rq.RQ_EUNSUPPORTED),      # 2^32 threads
    (dict(H=A + 16), rq.RQ_EINVAL), (dict(H=A, h_stride=512), rq.RQ_EINVAL), (dict(H=A + GB + 16 * 256), rq.RQ_EINVAL),
    (dict(H=A, x_stride=0), rq.RQ_EINVAL), (dict(H=A + 2 * GB), rq.RQ_EINVAL),
    (dict(Xq=A), rq.RQ_EINVAL), (dict(Xq=A + 3 * GB + 512), rq.RQ_EINVAL), (dict(x_scale=A + 4 * GB + 16), rq.RQ_EINVAL),
    (dict(x_scale=A + 2 * GB), rq.RQ_EINVAL),
    (dict(X=A, H=A + 4096 * 2, M=40, x_stride=8192, h_stride=4096), rq.RQ_EINVAL),         # rows that meet further down
])
def test_refused(kw, status):
    assert _status(**kw) == status
    assert rq.load().rq_last_error_detail().decode()


def test_refused_configurations():
    assert _status(rq.make_cfg(5)) == rq.RQ_EUNSUPPORTED
    assert _status(rq.make_cfg(8, x_layout=rq.RQ_X_FP6)) == rq.RQ_EUNSUPPORTED
    assert _status(rq.make_cfg(8, x_layout=4)) == rq.RQ_EINVAL
    assert rq.load().rq_norm_rotate_quantize(None, ctypes.byref(rq.make_cfg(8)), None) == rq.RQ_EINVAL
    assert rq.load().rq_norm_rotate_quantize(ctypes.byref(_params()), None, None) == rq.RQ_EINVAL


def test_no_rows_launch_nothing():
    assert _status(M=0) == rq.RQ_OK
    assert _status(M=0, X=None, Xq=None) == rq.RQ_OK


def test_wrapper_refusals():
    X = torch.zeros(4, 256, dtype=torch.float16)
    R = torch.zeros(4, 256, dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        rq.norm_rotate_quantize(X, R)
    for bad in (X[0], X.double(), X.t()):
        with pytest.raises(ValueError):
            rq.norm_rotate_quantize(bad)
    for bad in (R[:3], R.float(), R[:, :128], torch.zeros(256, 4, dtype=torch.float16).t()):
        with pytest.raises(ValueError):
            rq.norm_rotate_quantize(X, bad)
        with pytest.raises(ValueError):
            rq.norm_rotate_quantize(X, R, out=bad)
    for bad in (torch.zeros(255), torch.zeros(256, dtype=torch.bfloat16), torch.zeros(512)[::2], torch.zeros(1, 256)):
        with pytest.raises(ValueError, match="weight"):
            rq.norm_rotate_quantize(X, R, bad)


@pytest.mark.parametrize("M", [65536, 65537])
def test_inputs_in_the_gaps_of_h(M):
    """X between H's rows, met by none: a single row repeated at any M, rows of another stride up to 65536 of them (not worked
    out beyond). The residual, looked at after X, lies on H's rows, so that no call here launches."""
    kw = dict(M=M, H=A, h_stride=512, residual=A + 512 + 16, residual_stride=512, Xq=A + 4 * GB, x_scale=A + 6 * GB)
    detail = lambda: rq.load().rq_last_error_detail().decode()  # noqa: E731
    assert _status(X=A + 512, x_stride=0, **kw) == rq.RQ_EINVAL and "residual" in detail()
    assert _status(X=A + 512 + 1024 * (M - 1), x_stride=0, **kw) == rq.RQ_EINVAL and "residual" in detail()
    for at in (496, 1024 - 496, 1024 * (M - 1), 1024 * (M - 1) - 496, 1024 * (M - 1) + 496):   # on one of H's rows, or its first or last bytes
        assert _status(X=A + at, x_stride=0, **kw) == rq.RQ_EINVAL and "overlaps X" in detail(), at
    apart = _status(X=A + 512, x_stride=1024, **kw)
    if M <= 65536:
        assert apart == rq.RQ_EINVAL and "residual" in detail()
    else:
        assert apart == rq.RQ_EUNSUPPORTED and "X" in detail()
