"""rq_kv_evict on the GPU: the choice and the bytes exactly."""
import numpy as np
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests import evict_ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _case(kv_len, budget, dim=128, bits=4, page=16, heads=2, seed=0, spare=0):
    need_gpu()
    rng = np.random.default_rng(seed)
    row = dim * bits // 8
    need = [-(-n // page) for n in kv_len]
    new = -(-budget // page) + spare
    total = sum(need) + new * len(kv_len) + 2
    raw = rng.integers(0, 256, (total, heads * page * (2 * row + 8)), dtype=np.uint8)
    order = rng.permutation(total).astype(np.int32)
    pages = np.full((len(kv_len), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
    new_pages = order[at:at + new * len(kv_len)].reshape(len(kv_len), new)
    weights = np.exp(2 * rng.normal(size=(len(kv_len), heads, pages.shape[1] * page))).astype(np.float32)
    weights[rng.random(weights.shape) < 0.3] = 0.0
    return dict(raw=raw, pages=pages, new_pages=new_pages, weights=weights, kv_len=list(kv_len), budget=budget, heads=heads, page=page,
                row=row, cfg=rq.make_kv_cfg(heads, dim, page, bits))


def _check(d, first=0, recent=0, with_weights=True):
    cache = torch.from_numpy(d["raw"]).cuda()
    new_span = d["new_pages"].shape[1] * d["page"]
    out = torch.full((len(d["kv_len"]), d["heads"], new_span), -5.0, device="cuda") if with_weights else None
    W = torch.from_numpy(d["weights"]).cuda()
    kept, length = rq.kv_evict(cache, _ints(d["pages"]), _ints(d["kv_len"]), W, d["cfg"], d["budget"], _ints(d["new_pages"]), out,
                               first=first, recent=recent)
    raw, want, lengths = evict_ref.evict(d["raw"], d["heads"], d["page"], d["row"], d["pages"], d["kv_len"], d["weights"], d["budget"],
                                         d["new_pages"], first, recent)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(length.cpu().numpy(), lengths)
    assert np.array_equal(cache.cpu().numpy(), raw)
    if with_weights:
        o = out.cpu().numpy()
        for b, n in enumerate(lengths):
            for h in range(d["heads"]):
                assert np.array_equal(o[b, h, :n], d["weights"][b, h, want[b, h, :n]], equal_nan=True)
                assert np.all(o[b, h, n:] == -5.0)
    return cache, kept, length


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_every_row_width(dim, bits, page):
    print("evict", dim, bits, page, flush=True)
    _check(_case([5, 100, 37, 38, 39, 1, 0, 200], 37, dim, bits, page, heads=3, seed=dim + bits), first=3, recent=10)


@pytest.mark.parametrize("budget", [1, 2, 3, 4, 5, 63, 64, 65, 130, 299, 300, 301])
def test_budgets(budget):
    d = _case([300, 64, 65, 301, 7], budget, seed=budget, spare=budget % 2)
    _check(d)
    _check(d, recent=min(budget, 1))
    _check(d, first=budget // 2, recent=budget - budget // 2)
    _check(d, first=budget // 3, recent=budget // 3, with_weights=False)


@pytest.mark.parametrize("n", [4095, 4096, 4097, 8191, 20000])
def test_long_rows(n):
    """Several passes of the workgroup over a row."""
    d = _case([n, 4100, 3000], 2500, dim=64, page=128, heads=2, seed=n)
    _check(d, first=4, recent=300)


@pytest.mark.parametrize("n", [16385, 40001, 131071])
def test_rows_in_parts(n):
    """Few rows whose choice is shared by many workgroups: cuts of a row in front of, inside and behind what stays."""
    d = _case([n, n // 3, 900, 1001], 1000, dim=64, page=256, heads=1, seed=n)
    assert rq.kv_evict_workspace_size(4, d["pages"].shape[1], d["cfg"]) > 0
    _check(d, first=4, recent=300)
    _check(d, first=600, recent=400)
    d["weights"][:] = np.round(d["weights"])       # many of one size
    _check(d, recent=1)
    d = _case([n], n - 7, dim=64, page=256, heads=1, seed=n)
    _check(d, first=n // 2, recent=n // 3)
    d["weights"][:] = 0.0
    _check(d)


def test_many_long_rows():
    """As many rows as workgroups are wanted: one each, several passes long."""
    d = _case([4500] * 130 + [9000], 64, dim=64, page=512, heads=2, seed=11)
    assert rq.kv_evict_workspace_size(131, d["pages"].shape[1], d["cfg"]) == 0
    _check(d, recent=16)


@pytest.mark.parametrize("kind", ["zeros", "ones", "steps", "specials", "near", "negative", "rising", "falling"])
def test_weights_of_every_kind(kind):
    """Ties go to the first; NaN is below all; -0 is 0; infinities; weights that differ in their last bit only."""
    d = _case([5000, 1000, 700], 600, dim=64, page=64, seed=4)
    rng = np.random.default_rng(1)
    w = d["weights"]
    if kind == "zeros":
        w[:] = 0.0
    elif kind == "ones":
        w[:] = 1.0
    elif kind == "steps":
        w[:] = rng.integers(0, 4, w.shape)
    elif kind == "specials":
        pick = rng.random(w.shape)
        w[pick < 0.3] = np.nan
        w[(pick >= 0.3) & (pick < 0.5)] = -np.inf
        w[(pick >= 0.5) & (pick < 0.7)] = -0.0
        w[(pick >= 0.7) & (pick < 0.9)] = 0.0
        w[pick > 0.97] = np.inf
    elif kind == "near":
        w[:] = np.float32(1.0) + rng.integers(0, 8, w.shape).astype(np.float32) * np.float32(2.0 ** -23)
    elif kind == "negative":
        w[:] = rng.normal(size=w.shape)
    else:
        w[:] = np.arange(w.shape[-1]) * (1 if kind == "rising" else -1)
    _check(d, first=2, recent=50)
    _check(d)


def test_tables_are_not_trusted():
    d = _case([200, 150, 90], 64, seed=3)
    d["pages"][0, 3], d["pages"][1, 0], d["pages"][2, 1] = len(d["raw"]), -3, (1 << 31) - 1
    d["new_pages"][0, 1], d["new_pages"][2, 0] = -1, len(d["raw"]) + 7
    _check(d, recent=8)
    d["kv_len"] = [-4, 1 << 30, 90]      # cut to nothing, and to the table
    _check(d, recent=8)


def test_no_pages_and_no_sequences():
    d = _case([0, 0], 16)
    d["pages"] = d["pages"][:, :0]
    d["weights"] = d["weights"][:, :, :0]
    _check(d)
    cache = torch.from_numpy(d["raw"]).cuda()
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    kept, n = rq.kv_evict(cache, none, _ints([]), torch.empty((0, 2, 32), device="cuda"), d["cfg"], 16, none)
    assert kept.shape == (0, 2, 16) and n.shape == (0,)
    assert np.array_equal(cache.cpu().numpy(), d["raw"])


def test_streams_outputs_and_replays():
    d = _case([500, 333], 100, seed=6)
    W, pages, new_pages, kv_len = torch.from_numpy(d["weights"]).cuda(), _ints(d["pages"]), _ints(d["new_pages"]), _ints(d["kv_len"])
    cache, want, length = _check(d, first=1, recent=9)
    other = torch.from_numpy(d["raw"]).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kept, n = torch.empty_like(want), torch.empty_like(length)
    got = rq.kv_evict(other, pages, kv_len, W, d["cfg"], 100, new_pages, first=1, recent=9, kept=kept, new_kv_len=n, stream=side)
    side.synchronize()
    assert got[0] is kept and got[1] is n and torch.equal(kept, want) and torch.equal(n, length) and torch.equal(other, cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq.kv_evict(other, pages, kv_len, W, d["cfg"], 100, new_pages, first=1, recent=9, kept=kept, new_kv_len=n)
    for i in range(4):
        d["weights"] = np.roll(d["weights"], 7, 2)
        W.copy_(torch.from_numpy(d["weights"]))
        other.copy_(torch.from_numpy(d["raw"]))
        cache, want, _ = _check(d, first=1, recent=9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want) and torch.equal(other, cache)


def test_parts_in_a_graph_and_given_a_workspace():
    d = _case([9000, 12000], 500, dim=64, page=256, heads=2, seed=6)
    W, pages, new_pages, kv_len = torch.from_numpy(d["weights"]).cuda(), _ints(d["pages"]), _ints(d["new_pages"]), _ints(d["kv_len"])
    need = rq.kv_evict_workspace_size(2, pages.shape[1], d["cfg"])
    other, space = torch.from_numpy(d["raw"]).cuda(), torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    cache, want, _ = _check(d, first=1, recent=9)
    kept, n = torch.empty_like(want), torch.empty_like(kv_len)
    args = dict(first=1, recent=9, kept=kept, new_kv_len=n, workspace=space)
    with pytest.raises(ValueError, match="workspace"):
        rq.kv_evict(other, pages, kv_len, W, d["cfg"], 500, new_pages, **{**args, "workspace": space[:need - 1]})
    rq.kv_evict(other, pages, kv_len, W, d["cfg"], 500, new_pages, **args)
    assert torch.equal(kept, want) and torch.equal(other, cache) and bool((space[need:] == 255).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq.kv_evict(other, pages, kv_len, W, d["cfg"], 500, new_pages, **args)
    for i in range(4):
        d["weights"] = np.roll(d["weights"], 7, 2)
        W.copy_(torch.from_numpy(d["weights"]))
        other.copy_(torch.from_numpy(d["raw"]))
        space.fill_(i)
        cache, want, _ = _check(d, first=1, recent=9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want) and torch.equal(other, cache)


def test_offsets_past_32_bits():
    need_gpu()
    d = _case([700], 300, dim=256, bits=8, page=256, heads=4, seed=9)
    small, want, _ = _check(d, first=4, recent=30)
    pages = (5 << 30) // d["raw"].shape[1]
    at = np.array([0, pages - 1, pages // 2, pages - 2, 1, pages - 3, pages - 4, 2])[:len(d["raw"])]
    assert len(at) == len(d["raw"])
    big = torch.empty((pages, d["raw"].shape[1]), dtype=torch.uint8, device="cuda")
    big[torch.from_numpy(at).cuda()] = torch.from_numpy(d["raw"]).cuda()
    move = lambda t: _ints(np.where(t >= 0, at[np.maximum(t, 0)], -1))  # noqa: E731
    kept, _ = rq.kv_evict(big, move(d["pages"]), _ints(d["kv_len"]), torch.from_numpy(d["weights"]).cuda(), d["cfg"], 300,
                          move(d["new_pages"]), first=4, recent=30)
    assert torch.equal(kept, want) and torch.equal(big[torch.from_numpy(at).cuda()], small)


def test_weights_past_4_gib():
    """A page table of 2^28 tokens: a head's weights, and the places kept, by the parts of a row and past 32 bits of bytes."""
    d = _case([1000], 300, dim=64, page=256, heads=8, seed=10, spare=1)
    _, want, _ = _check(d, first=4, recent=30)
    wide = torch.full((1, 1 << 20), -1, dtype=torch.int32, device="cuda")
    wide[:, :d["pages"].shape[1]] = _ints(d["pages"])
    W = torch.zeros(1, 8, 1 << 28, device="cuda")
    W[:, :, :d["weights"].shape[2]] = torch.from_numpy(d["weights"]).cuda()
    cache = torch.from_numpy(d["raw"]).cuda()
    kept, n = rq.kv_evict(cache, wide, _ints([1000]), W, d["cfg"], 300, _ints(d["new_pages"]), first=4, recent=30)
    assert torch.equal(kept, want) and n.tolist() == [300]
    raw, _, _ = evict_ref.evict(d["raw"], 8, 256, d["row"], d["pages"], [1000], d["weights"], 300, d["new_pages"], 4, 30)
    assert np.array_equal(cache.cpu().numpy(), raw)


def test_sequences_that_share_pages():
    """A prefix that several sequences have in the same pages is copied for each."""
    d = _case([300, 250, 90], 64, page=16, seed=12)
    d["pages"][1, :8] = d["pages"][0, :8]
    d["pages"][2, :3] = d["pages"][0, :3]
    _check(d, first=4, recent=10)


@pytest.mark.parametrize("kw", [dict(first=(1 << 32) + 3), dict(recent=1 << 32), dict(first=-(1 << 32)), dict(recent=1 << 63),
                                dict(budget=(1 << 32) + 64), dict(budget=(1 << 31) - 1), dict(budget=97), dict(budget=0)])
def test_counts_beyond_the_calls_integers(kw):
    """Refused, not cut to 32 bits; and no room is made for more places than new_pages have."""
    d = _case([200, 150], 96, seed=2)
    cache = torch.from_numpy(d["raw"]).cuda()
    args = {**dict(budget=96, first=4, recent=8), **kw}
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    with pytest.raises(rq.ConvRotError):
        rq.kv_evict(cache, _ints(d["pages"]), _ints(d["kv_len"]), torch.from_numpy(d["weights"]).cuda(), d["cfg"], new_pages=_ints(d["new_pages"]),
                    **args)
    assert torch.cuda.max_memory_allocated() - held < 1 << 24
    assert np.array_equal(cache.cpu().numpy(), d["raw"])
