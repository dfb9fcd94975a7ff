"""rq_kv_attention_weights on the GPU against 64 bits, and attention, weights and eviction together."""
import numpy as np
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests import evict_ref, kv_ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def _call(q_len, kv_len, dim=128, bits=4, page=16, heads=2, group=2, dtype="bf16", causal=True, window=0, keep=1.0, seed=0,
          scale=None, extra=1, q_scale=1.0):
    need_gpu()
    need = sum(-(-n // page) for n in kv_len) + 2
    c = evict_ref.Pages(need, heads, dim, page, bits, seed)
    pages, _ = evict_ref.table(c, kv_len, extra, seed)
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    starts = [0] + list(np.cumsum(q_len))
    Q = (torch.randn(starts[-1], heads * group, dim, generator=gen, device="cuda") * q_scale).to(TORCH[dtype])
    span = pages.shape[1] * page
    old = torch.exp(torch.randn(len(kv_len), heads, span, generator=gen, device="cuda"))
    s = dim ** -0.5 if scale is None else scale
    lse = evict_ref.logsums(c, Q, pages, kv_len, starts, causal, window, s).float()
    return dict(c=c, cfg=rq.make_kv_cfg(heads, dim, page, bits), Q=Q, lse=lse, pages=pages, kv_len=kv_len, starts=starts, old=old,
                keep=keep, causal=causal, window=window, scale=s)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run(d, **kw):
    out = d["old"].clone()
    args = dict(keep=d["keep"], q_start=_ints(d["starts"]), causal=d["causal"], window=d["window"], softmax_scale=d["scale"])
    args.update(kw)
    rq.kv_attention_weights(d["Q"], d["lse"], d["c"].bytes, d["pages"], _ints(d["kv_len"]), d["cfg"], out, **args)
    return out


def _check(d, got, **kw):
    want, tol = evict_ref.weigh(d["c"], d["Q"], d["lse"], d["pages"], d["kv_len"], d["starts"], d["old"], d["keep"], d["causal"],
                                d["window"], d["scale"], **kw)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), "%d of %d off, the worst %.3g times its bound" % (
        int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / tol).nan_to_num(posinf=0.0).max()))
    for b, n in enumerate(d["kv_len"]):
        assert torch.equal(got[b, :, n:], d["old"][b, :, n:])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_single_tokens_at_every_length(dim, bits, dtype):
    kv = [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513]
    d = _call([1] * len(kv), kv, dim, bits, dtype=dtype, seed=dim + bits)
    print("weigh", dim, bits, dtype, flush=True)
    _check(d, _run(d))
    _check(d, _run(d, q_start=None, max_kv_len=max(kv)))


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("group", [1, 4, 7, 33])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40), (True, 1 << 30)])
def test_ragged_chunks(page, group, causal, window):
    d = _call([1, 30, 0, 7, 64, 5], [40, 30, 17, 100, 333, 3], page=page, group=group, causal=causal, window=window, dtype="f16")
    _check(d, _run(d))
    _check(d, _run(d, max_q_len=64, max_kv_len=333))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompts(dim, bits):
    d = _call([700, 90], [700, 1500], dim, bits, page=32, heads=1, group=3, keep=0.0, seed=3)
    d["old"].fill_(float("nan"))
    got = _run(d, max_q_len=700, max_kv_len=1500)
    d["old"].zero_()
    got2 = got.clone()
    for b, n in enumerate(d["kv_len"]):
        assert bool(got[b, :, n:].isnan().all())
        got2[b, :, n:] = 0.0
    _check(d, got2)


@pytest.mark.parametrize("kv", [600, 5000])
@pytest.mark.parametrize("window", [0, 77])
def test_rows_in_shares(kv, window):
    """Few ranges of tokens and many rows: the rows are split and joined."""
    d = _call([600], [kv], heads=1, group=4, window=window, seed=5)
    assert rq.kv_attention_weights_workspace_size(600, 4, 1, d["pages"].shape[1], d["cfg"], ragged=True) > \
        (600 * 4 // 16 + 2) * (4 * 2048 + 256)
    _check(d, _run(d))


@pytest.mark.parametrize("window", [1, 59, 128, 129, 2000])
@pytest.mark.parametrize("q", [1, 2, 50])
def test_long_caches_and_short_windows(q, window):
    """Whole ranges of tokens that no row attends to: what was there before, times keep."""
    d = _call([q] * 3, [3000, 2048, 300], window=window, keep=0.5, seed=window)
    _check(d, _run(d))
    d["keep"] = 0.0
    d["old"].fill_(float("nan"))
    got = _run(d)
    for b, n in enumerate(d["kv_len"]):
        assert bool(got[b, :, n:].isnan().all()) and not bool(got[b, :, :n].isnan().any())
        assert not bool(got[b, :, :max(n - q + 1 - window, 0)].any())


@pytest.mark.parametrize("window", [0, 3000])
def test_more_ranges_than_workgroups(window):
    """Single tokens over a batch whose every workgroup walks over several ranges."""
    kv = [9000 - 37 * i for i in range(20)]
    d = _call([1] * 20, kv, dim=64, page=256, heads=4, group=2, window=window, seed=8)
    _check(d, _run(d))


@pytest.mark.parametrize("q", [1, 3, 20, 100])
def test_what_was_there_before(q):
    """keep, and the places of the newest tokens, which hold anything."""
    for keep in (0.0, 0.25, 1.0, 3.0):
        for causal in (True, False):
            d = _call([q, q], [q + 50, q], keep=keep, causal=causal)
            if causal:
                for b, n in enumerate(d["kv_len"]):
                    d["old"][b, :, n - q:n] = float("nan")
            got = _run(d)
            d["old"] = torch.nan_to_num(d["old"])
            _check(d, got)


@pytest.mark.parametrize("q", [2, 40])
def test_rows_that_count_for_nothing(q):
    d = _call([q, q], [100, 90])
    lse, Q = d["lse"].clone(), d["Q"]
    lse[0, 1], lse[1, 0], lse[q, 2], lse[q + 1, 3] = float("nan"), float("-inf"), float("inf"), float("-inf")
    Q[q + 1, 0, 5], Q[1, 1, 7] = float("nan"), float("inf")
    d["lse"] = lse
    _check(d, _run(d))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e38])
@pytest.mark.parametrize("q", [1, 40])
def test_tokens_that_nobody_attends_to(q, value):
    """Never written in front of a window: their sums stay what was kept of them."""
    d = _call([q], [400], window=60)
    d["c"].spoil(d["pages"], 0, range(0, 400 - q - 60 + 1), value)
    _check(d, _run(d))


@pytest.mark.parametrize("size", [1e-3, 30.0, 1e4])
@pytest.mark.parametrize("q", [1, 40])
def test_logits_of_any_size(q, size):
    for dtype in ("f16", "bf16"):
        d = _call([q], [200], dtype=dtype, q_scale=size)
        _check(d, _run(d))


@pytest.mark.parametrize("q_len", [[1, 1, 1], [40, 70, 3]])
def test_tables_are_not_trusted(q_len):
    d = _call(q_len, [100, 150, 64], page=16, extra=2)
    pages = d["pages"].clone()
    pages[0, 2], pages[1, 3], pages[2, 0] = d["c"].pages, -5, (1 << 31) - 1
    d["pages"] = pages
    _check(d, _run(d))
    span = pages.shape[1] * 16
    # Lengths beyond the table are cut to it, and below 0 to nothing.
    out = d["old"].clone()
    rq.kv_attention_weights(d["Q"], d["lse"], d["c"].bytes, pages, _ints([-7, 1 << 30, 64]), d["cfg"], out, q_start=_ints(d["starts"]))
    torch.cuda.synchronize()
    assert torch.equal(out[0], d["old"][0])
    # Rows outside [0, total_q) do not exist.
    total = d["Q"].shape[0]
    for starts in ([-9, 1 << 30, 5, 2], [total, total, total + 1, 3], [3, 2, 1, 0]):
        out = d["old"].clone()
        rq.kv_attention_weights(d["Q"], d["lse"], d["c"].bytes, pages, _ints([100, span, 64]), d["cfg"], out, q_start=_ints(starts))
        torch.cuda.synchronize()


def test_hints_that_are_too_small_or_absent():
    d = _call([3, 1], [3000, 500], page=64)
    full = _run(d)
    _check(d, full)
    for hint in (1, 64, 500, 2999):
        assert torch.equal(_run(d, max_kv_len=hint), full)
    d = _call([60, 30], [300, 200])
    _check(d, _run(d, max_q_len=20), max_q=20)
    _check(d, _run(d, max_kv_len=100))


def test_no_rows_no_pages_no_sequences():
    d = _call([0, 0], [30, 40], keep=0.5)
    _check(d, _run(d))
    need_gpu()
    empty = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    rq.kv_attention_weights(d["Q"], d["lse"], d["c"].bytes, empty, _ints([0, 0]), d["cfg"], d["old"][:, :, :0].contiguous(),
                            q_start=_ints([0, 0, 0]))
    rq.kv_attention_weights(d["Q"], d["lse"], d["c"].bytes, empty[:0], _ints([]), d["cfg"], d["old"][:0, :, :0].contiguous())


def test_strided_queries_streams_and_a_callers_workspace():
    d = _call([50, 20], [200, 300], group=2, heads=3, dim=64)
    want = _run(d)
    wide = torch.zeros((70, 9, 64 + 8), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8, :64] = d["Q"]
    keep = d["Q"]
    d["Q"] = wide[:, 2:8, :64]
    assert torch.equal(_run(d), want)
    d["Q"] = keep
    need = rq.kv_attention_weights_workspace_size(70, 6, 2, d["pages"].shape[1], d["cfg"], ragged=True)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(_run(d, workspace=ws), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _run(d, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for _ in range(3):
        assert torch.equal(_run(d), want)


@pytest.mark.parametrize("q", [1, 50])
def test_captured_and_replayed(q):
    """A decode step: attention, its weights, and the next; replayed over growing caches."""
    d = _call([q, q], [300, 500], page=64, extra=3)
    kv_len, starts, out = _ints(d["kv_len"]), _ints(d["starts"]), d["old"].clone()
    cfg, c = d["cfg"], d["c"]

    def step(w):
        O, lse = rq.kv_attention(d["Q"], c.bytes, d["pages"], kv_len, cfg, q_start=starts, return_lse=True)
        rq.kv_attention_weights(d["Q"], lse, c.bytes, d["pages"], kv_len, cfg, w, q_start=starts)
        return O, lse

    step(out)
    torch.cuda.synchronize()
    out.copy_(d["old"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(out)
    mine = d["old"].clone()
    out.copy_(d["old"])
    for i in range(4):
        kv_len.sub_(i)
        want = step(mine)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        # (V is anything here, so O may be NaN: its bits.)
        assert torch.equal(out, mine) and torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits():
    need_gpu()
    cfg = rq.make_kv_cfg(8, 128, 256, 8)
    small = evict_ref.Pages(6, 8, 128, 256, 8, seed=2)
    pages = (5 << 30) // small.bytes.shape[1]
    cache = torch.empty((pages, small.bytes.shape[1]), dtype=torch.uint8, device="cuda")
    at = torch.tensor([0, pages - 1, pages // 2, pages - 2, 1, pages - 3], device="cuda")
    cache[at] = small.bytes
    Q = torch.randn(3, 16, 128, generator=torch.Generator("cuda").manual_seed(1), device="cuda").half()
    few = torch.tensor([[1, 2, 5, 3]], dtype=torch.int32, device="cuda")
    lse = evict_ref.logsums(small, Q, few, [1000], [0, 3], True, 0, 128 ** -0.5).float()
    out = torch.zeros(1, 8, 1024, device="cuda")
    want = out.clone()
    rq.kv_attention_weights(Q, lse, small.bytes, few, _ints([1000]), cfg, want)
    rq.kv_attention_weights(Q, lse, cache, at[few.long()].int(), _ints([1000]), cfg, out)
    assert torch.equal(out, want) and bool((out[:, :, :1000] > 0).any())


@pytest.mark.parametrize("q", [3, 60])
def test_weights_past_4_gib(q):
    """A page table of 2^28 tokens: the last head's sums lie 7 GiB behind the first's."""
    need_gpu()
    cfg = rq.make_kv_cfg(8, 64, 256, 4)
    c = evict_ref.Pages(6, 8, 64, 256, 4, seed=2)
    Q = torch.randn(q, 16, 64, generator=torch.Generator("cuda").manual_seed(1), device="cuda").half()
    few = torch.tensor([[1, 2, 5, 3]], dtype=torch.int32, device="cuda")
    lse = evict_ref.logsums(c, Q, few, [1000], [0, q], True, 0, 64 ** -0.5).float()
    want = torch.zeros(1, 8, 1024, device="cuda")
    rq.kv_attention_weights(Q, lse, c.bytes, few, _ints([1000]), cfg, want, max_kv_len=1000)
    table = torch.full((1, 1 << 20), -1, dtype=torch.int32, device="cuda")
    table[:, :4] = few
    out = torch.zeros(1, 8, 1 << 28, device="cuda")
    rq.kv_attention_weights(Q, lse, c.bytes, table, _ints([1000]), cfg, out, max_kv_len=1000)
    # (The rows may be shared out otherwise: sums of at most 2 q weights of at most 1 in another order.)
    assert float((out[:, :, :1024] - want).abs().max()) <= 2 * q * 2 * q * 2.0 ** -24 and bool((want[:, :, :1000] > 0).any())
    assert not bool(out[:, :, 1000:].any())


@pytest.mark.parametrize("q", [1, 40])
def test_sequences_that_share_pages(q):
    d = _call([q] * 3, [300, 250, 90], page=16, keep=0.5, seed=12)
    d["pages"][1, :8] = d["pages"][0, :8]
    d["pages"][2, :3] = d["pages"][0, :3]
    d["lse"] = evict_ref.logsums(d["c"], d["Q"], d["pages"], d["kv_len"], d["starts"], True, 0, d["scale"]).float()
    _check(d, _run(d))


@pytest.mark.parametrize("bits,dim,dtype", [(4, 128, "bf16"), (8, 64, "f16"), (4, 256, "f16")])
def test_attention_weights_and_eviction_together(bits, dim, dtype):
    """A prompt written, attended to and weighed, brought down to a budget, and single tokens after that over
    what stayed: attention over the new pages is attention over the tokens kept."""
    need_gpu()
    heads, group, page, n, budget = 2, 2, 16, 230, 96
    rng = np.random.default_rng(dim + bits)
    cfg = rq.make_kv_cfg(heads, dim, page, bits)
    c = kv_ref.Cache(30, heads, dim, page, bits, rng)
    cache = c.flat().cuda()
    order = rng.permutation(30)
    pages, new_pages = order[:15][None], order[15:22][None]
    slots = pages[0][np.arange(n + 1) // page] * page + np.arange(n + 1) % page
    k, v = (torch.from_numpy(rng.normal(size=(n, heads, dim))).to(TORCH[dtype]) for _ in range(2))
    rq.kv_cache_write(k.cuda(), v.cuda(), torch.from_numpy(slots[:n]).cuda(), cache, cfg)
    c.write(k.float().numpy(), v.float().numpy(), slots[:n])
    Q = torch.from_numpy(rng.normal(size=(n, heads * group, dim))).to(TORCH[dtype])
    W = torch.zeros(1, heads, 15 * page, device="cuda")
    tables = _ints(pages)
    O, lse = rq.kv_attention(Q.cuda(), cache, tables, _ints([n]), cfg, return_lse=True)
    rq.kv_attention_weights(Q.cuda(), lse, cache, tables, _ints([n]), cfg, W)
    # Every row gives away 1: as near as lse is to the sum (its error is the attention's, below 2^-8).
    assert abs(float(W.double().sum()) / (n * heads * group) - 1) < 2.0 ** -8
    new_w = torch.zeros(1, heads, 7 * page, device="cuda")
    before = cache.clone()
    kept, length = rq.kv_evict(cache, tables, _ints([n]), W, cfg, budget, _ints(new_pages), new_w, first=4, recent=16)
    assert length.tolist() == [budget]
    raw, want, _ = evict_ref.evict(before.cpu().numpy(), heads, page, c.row, pages, [n], W.cpu().numpy(), budget, new_pages, 4, 16)
    assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(cache.cpu().numpy(), raw)
    assert torch.equal(new_w[0, :, :budget], W[0].gather(1, kept[0].long()))
    # One more token, behind the budget, then attention over what there is.
    at = budget
    slot = int(new_pages[0, at // page]) * page + at % page
    k1, v1 = (torch.from_numpy(rng.normal(size=(1, heads, dim))).to(TORCH[dtype]) for _ in range(2))
    rq.kv_cache_write(k1.cuda(), v1.cuda(), torch.tensor([slot]).cuda(), cache, cfg)
    held = kv_ref.Cache(30, heads, dim, page, bits, rng)
    held.codes, held.scale = c.codes.copy(), c.scale.copy()
    held.write(k1.float().numpy(), v1.float().numpy(), [slot])
    for h in range(heads):
        for i in range(budget):
            s = int(new_pages[0, i // page]) * page + i % page
            for part in range(2):
                held.codes[part, s, h] = c.codes[part, slots[want[0, h, i]], h]
                held.scale[part, s, h] = c.scale[part, slots[want[0, h, i]], h]
    q1 = torch.from_numpy(rng.normal(size=(1, heads * group, dim))).to(TORCH[dtype])
    O, lse = rq.kv_attention(q1.cuda(), cache, _ints(new_pages), _ints([budget + 1]), cfg, return_lse=True)
    ref, ref_lse, _, tol, lse_tol = kv_ref.attention(q1.float().numpy(), held, new_pages, [budget + 1], [0, 1], dtype)
    assert np.all(np.abs(O.cpu().double().numpy() - ref) <= tol) and np.all(np.abs(lse.cpu().double().numpy() - ref_lse) <= lse_tol)
    rq.kv_attention_weights(q1.cuda(), lse, cache, _ints(new_pages), _ints([budget + 1]), cfg, new_w)
    grown = new_w[0, :, :budget] - W[0].gather(1, kept[0].long())
    assert bool((grown >= 0).all())
