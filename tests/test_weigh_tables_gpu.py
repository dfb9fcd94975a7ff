"""rq_kv_attention_weights on the GPU: rows in shares whatever the page table's width, lengths beyond the hint."""
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests import evict_ref
from tests.test_weigh_gpu import _call, _check, _ints, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q,kv,group", [([700], [900], 3), ([400, 90, 0, 640], [1200, 90, 33, 640], 4)])
def test_tables_wider_than_the_sequences(q, kv, group):
    """The same call with tables of 2^12 to 2^20 tokens: the same shares of rows, workspace and bits."""
    got = []
    for extra in (0, 3, 2048, 16384):
        d = _call(q, kv, heads=2, group=group, page=64, extra=extra, keep=0.0, seed=21)
        print("table", d["pages"].shape[1] * 64, flush=True)
        hints = dict(max_q_len=max(q), max_kv_len=max(kv))
        out = _run(d, **hints)
        _check(d, out)
        need = rq.kv_attention_weights_workspace_size(sum(q), 2 * group, len(q), d["pages"].shape[1], d["cfg"], ragged=True, **hints)
        got.append((need, [out[b, :, :n] for b, n in enumerate(kv)]))
    for need, out in got[1:]:
        assert need == got[0][0] and all(torch.equal(x, y) for x, y in zip(out, got[0][1]))


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 90), (False, 0)])
@pytest.mark.parametrize("hint", [1, 256, 300])
def test_lengths_beyond_the_hint(hint, causal, window):
    """Rows are shared out for the first tokens only; those of a longer sequence's others are added up by one workgroup."""
    for keep in (0.0, 0.5):
        d = _call([300, 520, 128, 0], [2000, 513, 256, 700], heads=1, group=5, page=32, causal=causal, window=window, keep=keep, seed=hint)
        assert rq.kv_attention_weights_workspace_size(948, 5, 4, d["pages"].shape[1], d["cfg"], max_kv_len=hint, ragged=True) > \
            (948 * 5 // 16 + 5) * (4 * 2048 + 256) + 256
        _check(d, _run(d, max_kv_len=hint))


def test_the_most_shares():
    """700 tiles of rows over three ranges of tokens: 64 shares, joined, and in a workspace whose ends are left alone."""
    d = _call([700], [705], heads=1, group=16, page=64, keep=0.5, seed=4)
    need = rq.kv_attention_weights_workspace_size(700, 16, 1, d["pages"].shape[1], d["cfg"], ragged=True)
    span = d["pages"].shape[1] * 64
    assert need == -(-(700 + 2) * (4 * 2048 + 256) // 256) * 256 + 64 * (-(-span // 256) * 256) * 4
    space = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    got = _run(d, workspace=space[256:256 + need])
    _check(d, got)
    assert bool((space[:256] == 0xFF).all()) and bool((space[256 + need:] == 0xFF).all())
    assert torch.equal(_run(d), got)


def _inside(t):
    """A copy of t within a buffer of one number, and that buffer's ends."""
    big = torch.full((t.numel() + 2048,), 0x55, dtype=torch.uint8, device="cuda") if t.dtype == torch.uint8 else \
        torch.full((t.numel() + 2048,), -77.0, dtype=t.dtype, device="cuda")
    view = big[1024:1024 + t.numel()].view(t.shape)
    view.copy_(t)
    return view, (big[:1024], big[1024 + t.numel():])


@pytest.mark.parametrize("q_len", [[1, 1, 1], [9, 0, 7], [40, 70, 3], [300, 333, 40]])
def test_what_untrusted_tables_give_and_leave(q_len):
    """Starts and lengths outside their ranges count as cut to them; nothing beside the sequences' sums and the workspace is
    written. (Sequences whose rows lie over one another need not be right, but stay within them.)"""
    d = _call(q_len, [100, 150, 64], page=16, extra=2, keep=0.5)
    pages = d["pages"].clone()
    pages[0, 2], pages[1, 3], pages[2, 0] = d["c"].pages, -5, (1 << 31) - 1
    d["pages"] = pages
    total, span = d["Q"].shape[0], pages.shape[1] * 16
    need = rq.kv_attention_weights_workspace_size(total, 4, 3, pages.shape[1], d["cfg"], ragged=True)
    good = [d["starts"][i] for i in range(4)]
    calls = [([-9, 1 << 30, 5, 2], [100, span, 64]), ([total, total, total + 1, 3], [100, span, 64]), ([3, 2, 1, 0], [100, span, 64]),
             ([-(1 << 31), 2, 2, (1 << 31) - 1], [span, 0, 37]), (good, [-7, 1 << 30, 64]), (good, [-(1 << 31), span + 1, (1 << 31) - 1]),
             ([0, total, 0, total], [100, span, 64])]
    for starts, lengths in calls:
        print("tables", q_len, starts, lengths, flush=True)
        out, ends = _inside(d["old"])
        space, spaces_ends = _inside(torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda"))
        rq.kv_attention_weights(d["Q"], d["lse"], d["c"].bytes, pages, _ints(lengths), d["cfg"], out, keep=0.5, q_start=_ints(starts),
                                workspace=space)
        torch.cuda.synchronize()
        assert all(bool((x == -77.0).all()) for x in ends) and all(bool((x == 0x55).all()) for x in spaces_ends)
        rows = [min(max(x, 0), total) for x in starts]
        for b in range(3):
            n = min(max(lengths[b], 0), span)
            assert torch.equal(out[b, :, n:], d["old"][b, :, n:])
            if starts[:3] == [0, total, 0] or n == 0:
                continue
            one = dict(d, pages=pages[b:b + 1], kv_len=[n], starts=[rows[b], max(rows[b], rows[b + 1])], old=d["old"][b:b + 1])
            _check(one, out[b:b + 1])


def test_shares_captured_and_replayed_over_growing_lengths():
    """Replays whose lengths pass the hint that the call was captured with, with eager work between."""
    d = _call([300, 90], [700, 256], heads=2, group=3, page=32, extra=40, keep=0.5, seed=6)
    rest = torch.randperm(d["c"].pages, device="cuda")[:8].int()
    d["pages"][:, 22:30], d["pages"][1, 8:22] = rest, d["pages"][0, :14]
    kv_len, out = _ints(d["kv_len"]), d["old"].clone()
    args = dict(keep=0.5, q_start=_ints(d["starts"]), max_q_len=300, max_kv_len=512)

    def step(w):
        rq.kv_attention_weights(d["Q"], d["lse"], d["c"].bytes, d["pages"], kv_len, d["cfg"], w, **args)

    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for lengths in ([700, 256], [511, 100], [512, 513], [900, 700], [0, 257]):
        d["kv_len"] = lengths
        kv_len.copy_(_ints(lengths))
        d["lse"].copy_(evict_ref.logsums(d["c"], d["Q"], d["pages"], lengths, d["starts"], True, 0, d["scale"]).float())
        mine = d["old"].clone()
        step(mine)
        out.copy_(d["old"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mine)
        _check(d, out)


def test_two_calls_at_once():
    """Calls on two streams, each with the workspace that it takes for itself."""
    a = _call([500], [800], heads=2, group=4, page=32, keep=0.0, seed=7)
    b = _call([400, 200], [900, 300], heads=1, group=6, dim=64, page=16, keep=0.0, seed=8)
    want = [_run(a), _run(b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[d["old"].clone() for _ in range(10)] for d in (a, b)]
    tables = [(_ints(d["kv_len"]), _ints(d["starts"])) for d in (a, b)]
    torch.cuda.synchronize()
    for i in range(10):
        for d, out, s, (n, q) in zip((a, b), outs, streams, tables):
            rq.kv_attention_weights(d["Q"], d["lse"], d["c"].bytes, d["pages"], n, d["cfg"], out[i], keep=0.0, q_start=q, stream=s)
    torch.cuda.synchronize()
    for d, out, w in zip((a, b), outs, want):
        _check(d, w)
        assert all(torch.equal(x, w) for x in out)
