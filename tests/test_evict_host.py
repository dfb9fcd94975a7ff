"""The checks of the operators that hold a cache to a budget (no GPU: refused calls launch nothing)."""
import ctypes
import re

import numpy as np
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests import evict_ref
from tests.test_abi import A, GB, HEADER


def _evict(cfg=None, ws=None, ws_bytes=0, **kw):
    p = dict(cache=A, kv_len=A + GB, pages=A + 2 * GB, new_pages=A + 3 * GB, weights=A + 4 * GB, new_weights=A + 5 * GB,
             new_kv_len=A + 6 * GB, kept=A + 7 * GB, num_pages=100, seqs=4, max_pages=20, new_max_pages=5, budget=300, first=4, recent=32)
    p.update(kw)
    return rq.rq_kv_evict(rq.rq_kv_evict_params(*p.values()), cfg or rq.make_kv_cfg(2, 128, 64, 4), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), rq.RQ_EINVAL), (dict(cache=A + 8), rq.RQ_EINVAL), (dict(kv_len=None), rq.RQ_EINVAL), (dict(pages=None), rq.RQ_EINVAL),
    (dict(new_pages=None), rq.RQ_EINVAL), (dict(weights=None), rq.RQ_EINVAL), (dict(new_kv_len=None), rq.RQ_EINVAL), (dict(kept=None), rq.RQ_EINVAL),
    (dict(weights=A + 4 * GB + 4), rq.RQ_EINVAL), (dict(pages=A + 2 * GB + 2), rq.RQ_EINVAL), (dict(kept=A + 7 * GB + 1), rq.RQ_EINVAL),
    (dict(new_weights=A + 5 * GB + 2), rq.RQ_EINVAL),
    (dict(seqs=-1), rq.RQ_EINVAL), (dict(max_pages=-1), rq.RQ_EINVAL), (dict(new_max_pages=-1), rq.RQ_EINVAL), (dict(first=-1), rq.RQ_EINVAL),
    (dict(recent=-1), rq.RQ_EINVAL), (dict(budget=0), rq.RQ_EINVAL), (dict(budget=321), rq.RQ_EINVAL), (dict(first=290), rq.RQ_EINVAL),
    (dict(first=(1 << 31) - 1, recent=(1 << 31) - 1), rq.RQ_EINVAL),
    (dict(seqs=70000), rq.RQ_EUNSUPPORTED), (dict(max_pages=1 << 25), rq.RQ_EUNSUPPORTED), (dict(num_pages=0), rq.RQ_EINVAL),
    (dict(cfg=rq.make_kv_cfg(200, 128, 64, 4), seqs=60000), rq.RQ_EUNSUPPORTED),                                     # workgroups
    (dict(seqs=60000, new_max_pages=20000, budget=1 << 20), rq.RQ_EUNSUPPORTED),
    (dict(cfg=rq.make_kv_cfg(2, 96, 64, 4)), rq.RQ_EUNSUPPORTED),
    (dict(kept=A + 64), rq.RQ_EINVAL), (dict(new_kv_len=A + GB), rq.RQ_EINVAL), (dict(kept=A + 3 * GB), rq.RQ_EINVAL),
    (dict(new_weights=A + 4 * GB), rq.RQ_EINVAL), (dict(new_weights=A + 7 * GB), rq.RQ_EINVAL), (dict(new_kv_len=A + 7 * GB + 64), rq.RQ_EINVAL),
    (dict(weights=A + 4096), rq.RQ_EINVAL), (dict(pages=A + 16), rq.RQ_EINVAL),
    (dict(max_pages=200), rq.RQ_EWORKSPACE), (dict(max_pages=200, ws=A + 8 * GB, ws_bytes=1000), rq.RQ_EWORKSPACE),
    (dict(max_pages=200, ws_bytes=GB), rq.RQ_EINVAL), (dict(max_pages=200, ws=A + 8 * GB + 4, ws_bytes=GB), rq.RQ_EINVAL),
    (dict(max_pages=200, ws=A + 4 * GB, ws_bytes=GB), rq.RQ_EINVAL), (dict(max_pages=200, ws=A + 7 * GB, ws_bytes=GB), rq.RQ_EINVAL),
    (dict(max_pages=200, ws=A + 64, ws_bytes=GB), rq.RQ_EINVAL),
])
def test_eviction_refused(kw, status):
    assert _evict(**kw) == status
    assert rq.load().rq_last_error_detail().decode()


def test_nothing_to_evict():
    assert _evict(seqs=0) == rq.RQ_OK
    cfg = rq.make_kv_cfg(2, 128, 64, 4)
    assert rq.load().rq_kv_evict(None, ctypes.byref(cfg), None, 0, None) == rq.RQ_EINVAL
    assert rq.load().rq_kv_evict(ctypes.byref(rq.rq_kv_evict_params()), None, None, 0, None) == rq.RQ_EINVAL


def test_struct_matches_header():
    body = re.search(r"typedef struct \{([^{}]*)\} rq_kv_evict_params;", open(HEADER).read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip(" *") for line in body.split(";") if line.strip() for n in re.sub(r"^(const )?\w+ ", "", line.strip()).split(",")]
    assert [n for n, _ in rq.rq_kv_evict_params._fields_] == names
    assert ctypes.sizeof(rq.rq_kv_evict_params) == 8 * 8 + 8 + 6 * 4


def _weigh(cfg=None, weights=A + 6 * GB, keep=1.0, ws=A + 8 * GB, ws_bytes=1 << 40, cache=A + 5 * GB, num_pages=100, **kw):
    p = dict(Q=A, O=None, lse=A + GB, q_start=A + 2 * GB, kv_len=A + 3 * GB, pages=A + 4 * GB, total_q=8, q_token_stride=512,
             q_head_stride=128, o_token_stride=0, o_head_stride=0, max_q_len=0, max_kv_len=0, dtype=rq.RQ_BF16, q_heads=4, seqs=4,
             max_pages=20, causal=1, window=0, softmax_scale=0.1)
    p.update(kw)
    return rq.rq_kv_attention_weights(rq.rq_kv_attention_params(*p.values()), cfg or rq.make_kv_cfg(2, 128, 64, 4), cache, num_pages,
                                      weights, keep, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), rq.RQ_EINVAL), (dict(lse=None), rq.RQ_EINVAL), (dict(kv_len=None), rq.RQ_EINVAL), (dict(pages=None), rq.RQ_EINVAL),
    (dict(weights=None), rq.RQ_EINVAL), (dict(Q=A + 2), rq.RQ_EINVAL), (dict(lse=A + GB + 2), rq.RQ_EINVAL), (dict(weights=A + 6 * GB + 1), rq.RQ_EINVAL),
    (dict(keep=-0.5), rq.RQ_EINVAL), (dict(keep=float("nan")), rq.RQ_EINVAL), (dict(keep=float("inf")), rq.RQ_EINVAL),
    (dict(dtype=rq.RQ_F32), rq.RQ_EUNSUPPORTED), (dict(q_heads=5), rq.RQ_EINVAL), (dict(window=3, causal=0), rq.RQ_EINVAL),
    (dict(softmax_scale=0.0), rq.RQ_EINVAL), (dict(total_q=9, q_start=None), rq.RQ_EINVAL), (dict(q_token_stride=4), rq.RQ_EINVAL),
    (dict(seqs=0, total_q=3), rq.RQ_EINVAL), (dict(num_pages=0), rq.RQ_EINVAL), (dict(cache=None), rq.RQ_EINVAL),
    (dict(weights=A), rq.RQ_EINVAL), (dict(weights=A + GB), rq.RQ_EINVAL), (dict(weights=A + 4 * GB + 64), rq.RQ_EINVAL),
    (dict(weights=A + 5 * GB), rq.RQ_EINVAL),
    (dict(total_q=600, ws=A + 6 * GB), rq.RQ_EINVAL), (dict(total_q=600, ws=A), rq.RQ_EINVAL), (dict(total_q=600, ws=A + 8 * GB + 4), rq.RQ_EINVAL),
    (dict(total_q=600, ws_bytes=1000), rq.RQ_EWORKSPACE),
    (dict(cfg=rq.make_kv_cfg(2, 128, 64, 5)), rq.RQ_EUNSUPPORTED),
    (dict(cfg=rq.make_kv_cfg(64, 128, 16, 4), q_heads=64, seqs=60000, total_q=60000, max_pages=4096, num_pages=10), rq.RQ_EUNSUPPORTED),
])
def test_weights_refused(kw, status):
    assert _weigh(**kw) == status
    assert rq.load().rq_last_error_detail().decode()


def test_weights_of_nothing():
    assert _weigh(seqs=0, total_q=0) == rq.RQ_OK
    assert _weigh(max_pages=0, Q=None, lse=None) == rq.RQ_OK


def test_workspaces():
    cfg = rq.make_kv_cfg(2, 128, 64, 4)
    assert rq.kv_attention_weights_workspace_size(4, 8, 4, 100, cfg) == 0                 # single tokens
    assert rq.kv_attention_weights_workspace_size(64, 8, 4, 100, cfg, max_q_len=8, ragged=True) == 0
    # 4 heads of 16 rows' tiles: 4 operand steps of 2 KB and 256 bytes a tile, and a spare tile a sequence.
    # And the sums of three shares of the rows: 250 ranges of tokens of 8 (sequence, head) pairs are 2000 workgroups.
    got = rq.kv_attention_weights_workspace_size(4000, 8, 4, 1000, cfg, max_q_len=1000, ragged=True)
    query = (4000 * 4 // 16 + 4 + 1) * 2 * (4 * 2048 + 256)
    assert got == -(-query // 256) * 256 + 3 * 8 * 64000 * 4
    assert rq.kv_attention_weights_workspace_size(-1, 8, 4, 100, cfg) == 0


def test_eviction_workspaces():
    cfg = rq.make_kv_cfg(2, 128, 64, 4)
    word = 2 + 2 * 2048 + 1024
    assert rq.kv_evict_workspace_size(4, 64, cfg) == 0                                          # 4096 tokens
    assert rq.kv_evict_workspace_size(4, 65, cfg) == 8 * 4 * (4 + 2 * word)                     # two parts
    assert rq.kv_evict_workspace_size(4, 10000, cfg) == 8 * 4 * (4 + 32 * word)                 # the most parts
    assert rq.kv_evict_workspace_size(64, 10000, cfg) == 128 * 4 * (4 + 2 * word)               # 256 workgroups
    assert rq.kv_evict_workspace_size(65, 10000, cfg) == 0
    assert rq.kv_evict_workspace_size(0, 10000, cfg) == 0 and rq.kv_evict_workspace_size(-1, -1, cfg) == 0
    assert rq.kv_evict_workspace_size(4, 1 << 30, cfg) == 0 and rq.kv_evict_workspace_size(4, 100, rq.make_kv_cfg(2, 96, 64, 4)) == 0


def test_wrapper_refusals():
    cfg = rq.make_kv_cfg(2, 128, 64, 4)
    i32 = torch.int32
    cache = torch.zeros((10, rq.rq_kv_page_bytes(cfg)), dtype=torch.uint8)
    ok = dict(pages=torch.zeros((2, 3), dtype=i32), kv_len=torch.zeros(2, dtype=i32), weights=torch.zeros(2, 2, 192), budget=100,
              new_pages=torch.zeros((2, 2), dtype=i32))
    with pytest.raises(ValueError, match="device tensors"):
        rq.kv_evict(cache, cfg=cfg, **ok)
    for kw in (dict(pages=ok["pages"][0]), dict(pages=ok["pages"].long()), dict(kv_len=torch.zeros(3, dtype=i32)), dict(weights=torch.zeros(2, 2, 191)),
               dict(weights=torch.zeros(2, 1, 192)), dict(new_pages=torch.zeros((3, 2), dtype=i32)), dict(new_weights=torch.zeros(2, 2, 192)),
               dict(kept=torch.zeros((2, 2, 99), dtype=i32)), dict(new_kv_len=torch.zeros(2))):
        with pytest.raises(ValueError):
            rq.kv_evict(cache, cfg=cfg, **{**ok, **kw})
    with pytest.raises(ValueError):
        rq.kv_evict(cache[:, :-1], cfg=cfg, **ok)
    Q = torch.zeros(4, 6, 128, dtype=torch.bfloat16)
    ok = dict(Q=Q, lse=torch.zeros(4, 6), cache=cache, pages=torch.zeros((2, 3), dtype=i32), kv_len=torch.zeros(2, dtype=i32), cfg=cfg,
              weights=torch.zeros(2, 2, 192))
    with pytest.raises(ValueError, match="device tensors"):
        rq.kv_attention_weights(**ok)
    for kw in (dict(Q=Q.float()), dict(Q=Q[0]), dict(lse=torch.zeros(4, 5)), dict(lse=torch.zeros(4, 6).double()), dict(pages=ok["pages"][0]),
               dict(weights=torch.zeros(2, 2, 128)), dict(weights=torch.zeros(2, 2, 192).half()), dict(q_start=torch.zeros(2, dtype=i32))):
        with pytest.raises(ValueError):
            rq.kv_attention_weights(**{**ok, **kw})


def test_the_reference_itself():
    """Its layout round trip, and its choice against the definition by counting."""
    rng = np.random.default_rng(0)
    b = rng.integers(0, 256, (3, 2, 32 * (2 * 64 + 8)), dtype=np.uint8)
    k, v, s = evict_ref.tokens(b, 32, 64)
    assert np.array_equal(evict_ref.blocks(k, v, s), b)
    assert v[1, 1, 5, 9] == b[1, 1, 32 * 64 + (5 // 4 * 64 + 9) * 4 + 5 % 4]
    w = rng.integers(0, 5, 50).astype(np.float32)
    stay = evict_ref.choose(w, 50, 20, 3, 4)
    assert len(stay) == 20 and set(range(3)) <= set(stay) and set(range(46, 50)) <= set(stay)
    inner = [j for j in stay if 3 <= j < 46]
    for j in inner:
        ahead = sum(w[i] > w[j] or (w[i] == w[j] and i < j) for i in range(3, 46))
        assert ahead < 13


@pytest.mark.parametrize("seqs,rows,heads,group", [(1, 2048, 8, 4), (4, 1024, 8, 4), (1, 2813, 8, 16), (2, 700, 1, 16)])
def test_weights_workspaces_go_by_lengths_not_by_the_table(seqs, rows, heads, group):
    """A call of known lengths shares out its rows, and needs the same workspace, whatever its page table could hold."""
    cfg = rq.make_kv_cfg(heads, 128, 64, 4)
    need = [rq.kv_attention_weights_workspace_size(seqs * rows, heads * group, seqs, tokens // 64, cfg, max_q_len=rows, max_kv_len=rows,
                                                   ragged=True) for tokens in (4096, 65536, 131072, 139264, 1 << 20, 1 << 30)]
    query = (seqs * rows * group // 16 + seqs + 1) * heads * (4 * 2048 + 256)
    assert len(set(need)) == 1 and need[0] > -(-query // 256) * 256
    # Without lengths the table's count: the sums of 6000 workgroups of 256 tokens, and of one turn more, at most.
    for tokens in (4096, 65536, 131072, 139264, 1 << 20, 1 << 30):
        sums = rq.kv_attention_weights_workspace_size(seqs * rows, heads * group, seqs, tokens // 64, cfg, max_q_len=rows, ragged=True) \
            - -(-query // 256) * 256
        assert 0 <= sums <= 2 * 6000 * 256 * 4
