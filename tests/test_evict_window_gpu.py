"""Attention with a window over a cache that was brought down to a budget, on the GPU."""
import numpy as np
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests import kv_ref
from tests.gpu_util import need_gpu
from tests.test_evict_gpu import _ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [1, 17, 40])
@pytest.mark.parametrize("bits", [4, 8])
def test_recent_tokens_cover_a_window(bits, window):
    """With recent >= window - 1 the tokens behind the eviction attend to what they would have attended to without it."""
    need_gpu()
    heads, group, dim, page, n, more, budget = 2, 3, 128, 16, 200, 45, 64
    rng = np.random.default_rng(bits + window)
    cfg = rq.make_kv_cfg(heads, dim, page, bits)
    c = kv_ref.Cache(40, heads, dim, page, bits, rng)
    cache = c.flat().cuda()
    order = rng.permutation(40)
    pages, new_pages = order[:16][None], order[16:23][None]
    at = np.arange(n + more)
    slots = pages[0][at // page] * page + at % page
    k, v = (torch.from_numpy(rng.normal(size=(n + more, heads, dim))).bfloat16() for _ in range(2))
    c.write(k.float().numpy(), v.float().numpy(), slots)
    rq.kv_cache_write(k[:n].cuda(), v[:n].cuda(), torch.from_numpy(slots[:n]).cuda(), cache, cfg)
    W = torch.from_numpy(rng.random((1, heads, 16 * page)).astype(np.float32)).cuda()
    _, length = rq.kv_evict(cache, _ints(pages), _ints([n]), W, cfg, budget, _ints(new_pages), first=4, recent=window - 1)
    assert length.tolist() == [budget]
    at = budget + np.arange(more)
    rq.kv_cache_write(k[n:].cuda(), v[n:].cuda(), torch.from_numpy(new_pages[0][at // page] * page + at % page).cuda(), cache, cfg)
    Q = torch.from_numpy(rng.normal(size=(more, heads * group, dim))).bfloat16()
    O, lse = rq.kv_attention(Q.cuda(), cache, _ints(new_pages), _ints([budget + more]), cfg, window=window, return_lse=True)
    ref, ref_lse, _, tol, lse_tol = kv_ref.attention(Q.float().numpy(), c, pages, [n + more], [0, more], "bf16", window=window)
    assert np.all(np.abs(O.cpu().double().numpy() - ref) <= tol) and np.all(np.abs(lse.cpu().double().numpy() - ref_lse) <= lse_tol)
