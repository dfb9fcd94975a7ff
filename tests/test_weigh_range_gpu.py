"""rq_kv_attention_weights on the GPU: large queries over small keys and the other way round, logits as ever."""
import pytest
import torch

from tests import evict_ref
from tests.test_weigh_gpu import _call, _check, _run

pytestmark = pytest.mark.gpu


def _rescale(c, factor):
    """Every key of a cache times a power of two."""
    c.scale = c.scale * factor
    blocks = c.bytes.view(c.pages, c.heads, c.block)
    at = 2 * c.page * c.row
    blocks[:, :, at:at + 4 * c.page] = c.scale.contiguous().view(torch.uint8).view(c.pages, c.heads, -1)


@pytest.mark.parametrize("exponent", [119, 100, 40, -40, -90])
@pytest.mark.parametrize("dim,bits", [(64, 8), (128, 4), (128, 8), (256, 4)])
@pytest.mark.parametrize("q", [1, 5, 40])
def test_queries_and_keys_at_opposite_ends(q, dim, bits, exponent):
    """bf16 queries times 2^e over keys times 2^-e: each product of the two is as it was, and nothing in between leaves
    binary32. In a second call every second token's query is 1 or 2^8 less than that: a tile of rows of two sizes. (Not more: a
    logit of 2^40 is known to 2^16 from its log-sum, which bounds no exponential.)"""
    for every in (1, 2):
        d = _call([q, q], [90, 200], dim, bits, group=3, dtype="bf16", seed=q)
        _rescale(d["c"], 2.0 ** -exponent)
        size = torch.full((2 * q, 1, 1), 2.0 ** min(0, exponent - 8), dtype=torch.float64, device="cuda")
        size[::every] = 2.0 ** exponent
        d["Q"] = (d["Q"].double() * size).bfloat16()
        d["lse"] = evict_ref.logsums(d["c"], d["Q"], d["pages"], d["kv_len"], d["starts"], True, 0, d["scale"]).float()
        assert bool(torch.isfinite(d["Q"]).all()) and bool(torch.isfinite(d["lse"]).all())
        _check(d, _run(d))
