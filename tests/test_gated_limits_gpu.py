"""The gated product on the GPU at the longest K, where the sums come closest to their integers' ends."""
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests import gated_ref
from tests.gpu_util import fp6_tile, need_gpu
from tests.test_gated_gpu import LAYOUTS, TORCH, _packed, _x_buffer

pytestmark = pytest.mark.gpu

K = 131072


@pytest.mark.parametrize("bits,layout", LAYOUTS)
@pytest.mark.parametrize("M", [1, 17, 40, 64, 90, 128, 129])
@pytest.mark.parametrize("N", [16, 48])
def test_codes_all_at_their_ends(M, N, bits, layout):
    """Sums of +-K top^2 (2^31 - 2^25 for 8 bits; 49 K for 4, held times 256 or as binary32), and of rows that turn half way."""
    need_gpu()
    print("gated", M, N, bits, layout, flush=True)
    top = 127 if bits == 8 else 7
    xc = torch.full((M, K), top, dtype=torch.int8, device="cuda")
    xc[1::2] = -top
    wc = torch.full((2 * N, K), top, dtype=torch.int8, device="cuda")
    wc[1::3] = -top
    wc[2::5, K // 2:] *= -1
    gen = torch.Generator("cuda").manual_seed(M + N)
    xs = (1 + torch.rand(M, generator=gen, device="cuda")) / (K * top * top)
    ws, b = (0.5 + torch.rand(2 * N, generator=gen, device="cuda") for _ in range(2))
    fp6, dtype = layout == rq.RQ_X_FP6, ("f16", "bf16")[(M + N // 16) % 2]
    Wq = torch.from_numpy(fp6_tile(wc.cpu().numpy(), 128)).cuda() if fp6 else _packed(wc, bits).contiguous()
    X = _x_buffer(xc, bits, layout)
    for act in ("silu", "none"):
        Y = rq.gemm_gated(X, xs, Wq, ws, b, bits=bits, K=K, x_layout=layout, w_layout=rq.RQ_W_FP6 if fp6 else rq.RQ_W_ROWS,
                          act=gated_ref.ACTS.index(act), out_dtype=TORCH[dtype])
        # (K top^2 and 0 are binary32 numbers: the sums' conversion rounds nothing.)
        gated_ref.check(Y, *gated_ref.reference(xc, xs, wc, ws, b, act, TORCH[dtype]))
