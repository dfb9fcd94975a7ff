"""The norm's plain implementation for the tests: h and the codes from their binary32 definition
(exact), the scale's factor in 64 bits."""
import numpy as np
import torch

import oracle
from tests.gpu_util import fp6_untile, untile_codes

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24


def hidden(x, residual):
    """x + residual (CPU tensors) rounded once to their type."""
    if residual is None:
        return x
    return (x.double() + residual.double()).to(x.dtype) if x.dtype == torch.float32 else (x.float() + residual.float()).to(x.dtype)


def reference(h, weight, eps, bits):
    """(codes int8 [M, K], scales float64 [M]) of rows h."""
    v = h.float()
    if weight is not None:
        v = v * weight.float()
    codes, scale = oracle.quantize_rows(v.numpy(), oracle.F32, bits)[:2]
    mean = (h.double() ** 2).mean(1).numpy() + eps
    s = scale.astype(np.float64)
    return codes, np.where(s == 0.0, 0.0, s / np.sqrt(np.where(mean == 0.0, 1.0, mean)))


def scale_error(K):
    """Relative bound of a scale: a lane adds 8 squares a block into one sum (a rounding each), over
    at most 4 blocks of a row, or ceil(blocks / 16) where the row has more than 128; sums are joined in at
    most 4 + 2 + 8 steps. The factor's root halves that. Then the mean, eps added, root,
    reciprocal and product round once each."""
    blocks = K // 128
    chain = 8 * (4 if blocks <= 128 else -(-blocks // 16)) + 14
    return (chain / 2 + 5) * U32


def codes_of(Xq, M, K, bits, layout, rq):
    """Codes int8 [M, K] of a buffer in any layout."""
    flat = Xq.cpu().contiguous().numpy()
    if layout == rq.RQ_X_FP6:
        return fp6_untile(flat, M, K, 256)
    if layout == rq.RQ_X_TILED:
        flat = untile_codes(flat, M, K, bits)
    return flat.view(np.int8) if bits == 8 else oracle.unpack_int4(flat, K)
