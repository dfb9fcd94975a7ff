"""The cache operators on the GPU against the plain implementation in 64 bits (tests.kv_ref): the
cache's bytes exactly, rows read back and attention within bounds derived from the arithmetic."""
import numpy as np
import pytest
import torch

import w4a4_integer_quantized_amd as rq
from tests import kv_ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

DIMS, BITS = [64, 128, 256], [4, 8]


def make(dim, bits, page=16, heads=2, pages=8, seed=0):
    need_gpu()
    rng = np.random.default_rng(seed + dim + bits + page)
    c = kv_ref.Cache(pages, heads, dim, page, bits, rng)
    return rng, c, rq.make_kv_cfg(heads, dim, page, bits)


def rows(rng, tokens, heads, dim, dtype):
    """Rows of a type (exact in it) with scales all over, a few of zeros; the same values on the CPU."""
    x = rng.normal(size=(tokens, heads, dim)) * np.exp(rng.normal(size=(tokens, heads, 1)))
    x[rng.random((tokens, heads)) < 0.05] = 0.0
    t = torch.from_numpy(x).to(kv_ref.TORCH[dtype])
    return t, t.float().numpy()


# --------------------------------------------------------------------------------- write, read
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("dim", DIMS)
def test_write_is_exact_and_keeps_the_rest(dim, bits, dtype, page):
    rng, c, cfg = make(dim, bits, page, heads=3, pages=1024 // page)
    dev = c.flat().cuda()
    for tokens in (1, 3, 37, 300):
        k, k32 = rows(rng, tokens, 3, dim, dtype)
        v, v32 = rows(rng, tokens, 3, dim, dtype)
        slots = rng.permutation(c.pages * page)[:tokens]
        if tokens > 3:      # runs of neighbours from any offset on, and slots outside the cache
            slots = (np.arange(tokens) + 5) % (c.pages * page)
            slots[7], slots[11], slots[12] = -1, c.pages * page, -(1 << 62)
        rq.kv_cache_write(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), dev, cfg)
        c.write(k32, v32, slots)
        assert torch.equal(dev.cpu(), c.flat()), tokens


@pytest.mark.parametrize("bits", BITS)
def test_write_takes_slices_of_one_projection(bits):
    rng, c, cfg = make(128, bits, 32, heads=3)
    x = torch.from_numpy(rng.normal(size=(21, 5 * 128 + 6 * 128 + 8))).to(torch.bfloat16)
    k, v = x[:, 5 * 128:8 * 128].view(21, 3, 128), x[:, 8 * 128:11 * 128].view(21, 3, 128)
    xd = x.cuda()
    kd, vd = xd[:, 5 * 128:8 * 128].view(21, 3, 128), xd[:, 8 * 128:11 * 128].view(21, 3, 128)
    slots = rng.permutation(8 * 32)[:21]
    dev = c.flat().cuda()
    rq.kv_cache_write(kd, vd, torch.from_numpy(slots).cuda(), dev, cfg)
    c.write(k.float().numpy(), v.float().numpy(), slots)
    assert torch.equal(dev.cpu(), c.flat())
    # One row for every head and token (strides of zero).
    one = x[:1, :128].view(1, 1, 128)
    rq.kv_cache_write(one.cuda().expand(21, 3, 128), vd, torch.from_numpy(slots).cuda(), dev, cfg)
    c.write(np.broadcast_to(one.float().numpy(), (21, 3, 128)), v.float().numpy(), slots)
    assert torch.equal(dev.cpu(), c.flat())


def test_rows_of_128_hold_the_activation_quantizers_codes():
    need_gpu()
    x = torch.randn(256, 128, device="cuda").bfloat16()
    for bits in BITS:
        cfg = rq.make_kv_cfg(1, 128, 256, bits)
        cache = rq.kv_cache_alloc(1, cfg)
        rq.kv_cache_write(x[:, None], x[:, None], torch.arange(256, device="cuda"), cache, cfg)
        codes, scale = rq.rotate_quantize(x, bits=bits)
        raw = 128 * bits // 8
        assert torch.equal(cache[0, :256 * raw].view(256, raw), codes.view(torch.uint8))
        assert torch.equal(cache[0, 512 * raw:512 * raw + 1024].view(torch.float32), scale)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("dim", DIMS)
def test_read(dim, bits, out):
    rng, c, cfg = make(dim, bits, 32, heads=3)
    _, k = rows(rng, 200, 3, dim, "f32")
    _, v = rows(rng, 200, 3, dim, "f32")
    where = rng.permutation(8 * 32)[:200]
    c.write(k, v, where)
    dev = c.flat().cuda()
    for tokens in (1, 5, 200):
        slots = where[:tokens].copy()
        if tokens > 1:
            slots[1], slots[2], slots[3] = -1, 8 * 32, slots[0]     # outside the cache, and one twice
        got = rq.kv_cache_read(dev, torch.from_numpy(slots).cuda(), cfg, out_dtype=kv_ref.TORCH[out])
        ok = (slots >= 0) & (slots < 8 * 32)
        s = np.where(ok, slots, 0)
        for part, (g, want) in enumerate(zip(got, c.rows(slots))):
            assert g.dtype == kv_ref.TORCH[out] and g.shape == (tokens, 3, dim)
            tol = kv_ref.read_error(dim, c.scale[part][s], c.codes[part][s], out) * ok[:, None, None]
            tol = tol + kv_ref.EPS[out] * (np.abs(want) + tol)
            assert np.all(np.abs(g.cpu().double().numpy() - want) <= tol)


def test_read_into_strided_outputs():
    rng, c, cfg = make(64, 4, 16, heads=3)
    _, k = rows(rng, 50, 3, 64, "f32")
    c.write(k, -k, np.arange(50))
    dev = c.flat().cuda()
    slots = torch.arange(50).cuda()
    K, V = rq.kv_cache_read(dev, slots, cfg, out_dtype=torch.float16)
    both = torch.full((50, 2, 3, 72), 7.0, dtype=torch.float16, device="cuda")
    rq.kv_cache_read(dev, slots, cfg, out=(both[:, 0, :, :64], both[:, 1, :, :64]))
    assert torch.equal(both[:, 0, :, :64], K) and torch.equal(both[:, 1, :, :64], V) and torch.all(both[..., 64:] == 7.0)
    turned = torch.empty((3, 50, 64), dtype=torch.float16, device="cuda").transpose(0, 1)
    rq.kv_cache_read(dev, slots, cfg, out=(turned, torch.empty_like(V)))
    assert torch.equal(turned, K)


# ------------------------------------------------------------------------------------- attention
def fill(rng, c, kv_len, spread=1.0):
    """Pages in any order for each sequence, keys and values written; entries not needed are -1."""
    need = [-(-n // c.page) for n in kv_len]
    order = rng.permutation(c.pages)
    assert sum(need) <= c.pages
    pages = np.full((len(kv_len), max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
        if kv_len[b]:
            j = np.arange(kv_len[b])
            _, k = rows(rng, kv_len[b], c.heads, c.dim, "f32")
            _, v = rows(rng, kv_len[b], c.heads, c.dim, "f32")
            c.write(k * np.float32(spread), v, pages[b][j // c.page].astype(np.int64) * c.page + j % c.page)
    return pages


def check(c, cfg, Q, pages, kv_len, q_len, dtype, causal=True, window=0, scale=None, before=0, after=0, level=True, **kw):
    """One call against the reference; rows before and after the sequences must stay as they were.
    level: the inputs are random and of one size, so that roundings are independent and add in
    squares: beside the bound of each element, the 2-norm of all errors is well within 2 eps."""
    starts = before + np.concatenate(([0], np.cumsum(q_len))).astype(np.int32)
    assert Q.shape[0] == starts[-1] + after
    q = torch.from_numpy(Q).to(kv_ref.TORCH[dtype])
    want, lse, there, tol, lse_tol = kv_ref.attention(q.float().numpy(), c, pages, kv_len, starts, dtype, causal, window, scale)
    out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    got, got_lse = rq.kv_attention(q.cuda(), c.flat().cuda(), torch.from_numpy(pages).cuda(),
                                   torch.tensor(kv_len, dtype=torch.int32).cuda(), cfg, q_start=torch.from_numpy(starts).cuda(),
                                   causal=causal, window=window, softmax_scale=scale, return_lse=True, out=out, **kw)
    assert got is out
    got, got_lse = got.cpu().double().numpy(), got_lse.cpu().double().numpy()
    assert np.all(got[~there] == 3.0)
    err = np.abs(got - want)[there]
    bad = err > tol[there]
    assert not bad.any(), "worst %g of its bound, %d of %d outside" % ((err / np.maximum(tol[there], 1e-300)).max(), bad.sum(), bad.size)
    if level:
        assert np.linalg.norm(err) <= 2 * kv_ref.EPS[dtype] * np.linalg.norm(want)
    empty = np.isneginf(lse[there])
    assert np.array_equal(np.isneginf(got_lse[there]), empty)
    assert np.all(np.abs(got_lse[there][~empty] - lse[there][~empty]) <= lse_tol[there][~empty])
    assert np.all(got[there][empty] == 0.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("dim", DIMS)
def test_single_tokens_at_every_length(dim, bits, dtype):
    kv_len = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, 300]
    rng, c, cfg = make(dim, bits, 16, heads=2, pages=64)
    pages = fill(rng, c, kv_len)
    for group in (1, 3, 16):
        Q = rng.normal(size=(len(kv_len), 2 * group, dim))
        check(c, cfg, Q, pages, kv_len, [1] * len(kv_len), dtype)


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("group", [1, 4, 7])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40)])
def test_ragged_chunks(page, group, causal, window):
    """Sequences with no query rows, no keys, more query rows than keys (rows that attend to nothing),
    and rows of no sequence before and behind."""
    q_len, kv_len = [5, 0, 33, 7, 1, 20], [70, 40, 33, 3, 0, 150]
    rng, c, cfg = make(128, 4, page, heads=2, pages=1536 // page)
    pages = fill(rng, c, kv_len)
    Q = rng.normal(size=(sum(q_len) + 5, 2 * group, 128))
    for kw in ({}, dict(max_q_len=max(q_len), max_kv_len=max(kv_len)), dict(max_kv_len=1)):
        check(c, cfg, Q, pages, kv_len, q_len, "bf16", causal, window, before=2, after=3, **kw)


@pytest.mark.parametrize("kv", [100, 5000])
def test_rows_beyond_max_q_len_are_left(kv):
    rng, c, cfg = make(64, 4, 16, heads=1, pages=700)
    q_len, kv_len = [9, 2, 70], [kv, 60, kv]
    pages = torch.from_numpy(fill(rng, c, kv_len)).cuda()
    n, starts = torch.tensor(kv_len, dtype=torch.int32).cuda(), torch.tensor([0, 9, 11, 81], dtype=torch.int32).cuda()
    Q = torch.randn(81, 3, 64, device="cuda").half()
    dev = c.flat().cuda()
    for most in (1, 5, 9, 69):
        out = torch.full_like(Q, 3.0)
        rq.kv_attention(Q, dev, pages, n, cfg, q_start=starts, max_q_len=most, out=out)
        whole = rq.kv_attention(Q, dev, pages, n, cfg, q_start=starts)
        for a, b in ((0, 9), (9, 11), (11, 81)):
            e = min(b, a + most)
            assert torch.all(out[e:b] == 3.0)
            assert torch.all((out[a:e] - whole[a:e]).abs() <= 1e-3 * whole.abs().max())     # the split may differ


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("dim", DIMS)
def test_prompts(dim, bits, dtype):
    """Many rows of one sequence: its own prompt, and a chunk over what is there already."""
    q_len, kv_len = [150, 130], [150, 260]
    rng, c, cfg = make(dim, bits, 32, heads=1, pages=16)
    pages = fill(rng, c, kv_len)
    Q = rng.normal(size=(sum(q_len), 2, dim)) * 2
    check(c, cfg, Q, pages, kv_len, q_len, dtype, True)
    check(c, cfg, Q, pages, kv_len, q_len, dtype, True, window=100)
    check(c, cfg, Q, pages, kv_len, q_len, dtype, False, scale=0.3)


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1, 1 << 40])
@pytest.mark.parametrize("rows", [12, 140])
def test_windows_wider_than_any_cache(rows, window):
    """As none at all, also where rows lie before position 0."""
    kv_len, q_len = [5, 40], [rows, rows - 3]
    rng, c, cfg = make(64, 4, 16, heads=2, pages=8)
    pages = fill(rng, c, kv_len)
    check(c, cfg, rng.normal(size=(sum(q_len), 4, 64)), pages, kv_len, q_len, "bf16", window=window)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,bits", [(64, 8), (128, 4), (256, 4)])
def test_long_caches_are_split(dim, bits, dtype):
    kv_len = [3000, 1, 777]
    rng, c, cfg = make(dim, bits, 64, heads=1, pages=64)
    pages = fill(rng, c, kv_len)
    Q = rng.normal(size=(3, 4, dim))
    assert rq.kv_attention_workspace_size(3, 4, 3, pages.shape[1], cfg, ragged=True) > 0
    check(c, cfg, Q, pages, kv_len, [1, 1, 1], dtype)
    Q = rng.normal(size=(9, 4, dim))
    check(c, cfg, Q, pages, kv_len, [4, 1, 4], dtype, before=0)
    check(c, cfg, Q, pages, kv_len, [4, 1, 4], dtype, window=900, max_q_len=4)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,bits", [(64, 4), (128, 8), (128, 4), (256, 8)])
def test_chunks_over_long_caches_are_split(dim, bits, dtype):
    kv_len, q_len = [2500, 70, 1300], [25, 1, 19]
    rng, c, cfg = make(dim, bits, 64, heads=1, pages=64)
    pages = fill(rng, c, kv_len)
    assert rq.kv_attention_workspace_size(45, 4, 3, pages.shape[1], cfg, ragged=True, max_q_len=25) > 0
    Q = rng.normal(size=(sum(q_len) + 3, 4, dim))
    check(c, cfg, Q, pages, kv_len, q_len, dtype, before=1, after=2, max_q_len=25)
    check(c, cfg, Q, pages, kv_len, q_len, dtype, before=1, after=2, window=600)
    check(c, cfg, Q, pages, kv_len, q_len, dtype, causal=False, before=1, after=2, max_kv_len=2500)


@pytest.mark.parametrize("group", [33, 64, 65, 128])
@pytest.mark.parametrize("page", [16, 1024])
def test_many_heads_share_one(group, page):
    rng, c, cfg = make(64, 4, page, heads=1, pages=max(4, 512 // page))
    kv_len = [137, 1, 300]
    pages = fill(rng, c, kv_len)
    Q = rng.normal(size=(3, group, 64))
    check(c, cfg, Q, pages, kv_len, [1, 1, 1], "bf16")
    Q = rng.normal(size=(9, group, 64))
    check(c, cfg, Q, pages, kv_len, [3, 2, 4], "f16")


@pytest.mark.parametrize("rows_", [1, 40])
@pytest.mark.parametrize("bits", BITS)
def test_extremes(bits, rows_):
    """A key that takes nearly all the weight and whose value is tiny, values of very different sizes,
    logits that are large, queries of zeros, tiny and large ones."""
    rng, c, cfg = make(128, bits, 16, heads=1, pages=16)
    kv_len = [200]
    pages = fill(rng, c, kv_len, spread=2.0)
    q = rng.normal(size=(rows_, 5, 128))
    k = (q[0, 0] * 4)[None, None].astype(np.float32)
    slot = pages[0][3 // 16].astype(np.int64) * 16 + 3
    c.write(k, np.full((1, 1, 128), 1e-6, np.float32) * rng.normal(size=(1, 1, 128)).astype(np.float32), np.array([slot]))
    for at, size in ((20, 1e4), (70, 1e-4), (150, 1e6), (199, 3e-9)):
        slot = pages[0][at // 16].astype(np.int64) * 16 + at % 16
        kk = rng.normal(size=(1, 1, 128)).astype(np.float32)
        c.write(kk, rng.normal(size=(1, 1, 128)).astype(np.float32) * np.float32(size), np.array([slot]))
    q[:, 1] = 0.0
    q[:, 2] *= 1e-7
    q[:, 3] *= 30.0
    check(c, cfg, q, pages, kv_len, [rows_], "bf16", level=False)
    check(c, cfg, q, pages, kv_len, [rows_], "f16", causal=False, scale=1.0 / 128, level=False)


def test_bytes_of_unused_tokens_do_not_matter():
    """NaN, infinite and largest scales, any codes, behind every length and on pages of nobody."""
    rng, c, cfg = make(64, 4, 16, heads=2, pages=32)
    kv_len, q_len = [37, 100, 1], [2, 20, 1]
    used = rng.bit_generator.state
    outs = []
    for filler in (0x00, 0xFF, 0x7F):
        rng.bit_generator.state = used
        c.bytes[:] = filler
        pages = fill(rng, c, kv_len)
        Q = rng.normal(size=(23, 4, 64))
        check(c, cfg, Q, pages, kv_len, q_len, "f16")
        out = rq.kv_attention(torch.from_numpy(Q).half().cuda(), c.flat().cuda(), torch.from_numpy(pages).cuda(),
                              torch.tensor(kv_len, dtype=torch.int32).cuda(), cfg,
                              q_start=torch.tensor([0, 2, 22, 23], dtype=torch.int32).cuda())
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("q_len", [[1, 1, 1], [40, 70, 3]])
def test_tables_are_not_trusted(q_len):
    """Page indexes outside the cache hide their tokens, lengths are cut to the table's, and query
    rows to what there is."""
    rng, c, cfg = make(128, 4, 16, heads=2, pages=32)
    kv_len = [112, 150, 90]      # the first fills its pages: no token behind it was never written
    pages = fill(rng, c, kv_len)
    pages[0, 1], pages[1, 0], pages[1, 9], pages[2, 5] = -5, 1 << 30, 32, -(1 << 31)
    Q = rng.normal(size=(sum(q_len), 4, 128))
    check(c, cfg, Q, pages, kv_len, q_len, "bf16", causal=False)
    check(c, cfg, Q, pages, kv_len, q_len, "bf16")
    check(c, cfg, Q, pages, [1 << 30, 150, -7], q_len, "bf16", causal=False)
    q = torch.from_numpy(Q).bfloat16().cuda()
    args = (c.flat().cuda(), torch.from_numpy(pages).cuda(), torch.tensor(kv_len, dtype=torch.int32).cuda(), cfg)
    for starts in ([0, 1, 1 << 30, 2], [-9, 1, 2, sum(q_len)], [5, 4, 3, 2], [1 << 30] * 4):
        rq.kv_attention(q, *args, q_start=torch.tensor(starts, dtype=torch.int32).cuda())
    torch.cuda.synchronize()


def test_no_pages_and_no_rows():
    rng, c, cfg = make(64, 4)
    dev = c.flat().cuda()
    Q = torch.randn(3, 4, 64, device="cuda").half()
    none = torch.zeros((3, 0), dtype=torch.int32, device="cuda")
    n = torch.full((3,), 9, dtype=torch.int32, device="cuda")
    out, lse = rq.kv_attention(Q, dev, none, n, cfg, return_lse=True)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    out = rq.kv_attention(Q[:0], dev, none, n, cfg)
    assert out.shape == (0, 4, 64)
    e = torch.zeros(0, dtype=torch.int64, device="cuda")
    rq.kv_cache_write(Q[:0, :2], Q[:0, :2], e, dev, cfg)
    K, V = rq.kv_cache_read(dev, e, cfg)
    assert K.shape == (0, 2, 64)
    torch.cuda.synchronize()
    assert torch.equal(dev.cpu(), c.flat())


def test_strided_queries_and_outputs():
    rng, c, cfg = make(64, 4, 16, heads=2)
    kv_len = [90]
    pages = fill(rng, c, kv_len)
    x = torch.randn(33, 8, 72, device="cuda").half()
    args = (c.flat().cuda(), torch.from_numpy(pages).cuda(), torch.tensor(kv_len, dtype=torch.int32).cuda(), cfg)
    want = rq.kv_attention(x[..., :64].contiguous(), *args)
    assert torch.equal(rq.kv_attention(x[..., :64], *args), want)
    wide = torch.zeros(33, 8, 80, device="cuda").half()
    rq.kv_attention(x[..., :64], *args, out=wide[..., :64])
    assert torch.equal(wide[..., :64], want) and torch.all(wide[..., 64:] == 0)
    turned = torch.zeros(8, 33, 64, device="cuda").half().transpose(0, 1)
    rq.kv_attention(x[..., :64].transpose(0, 1).contiguous().transpose(0, 1), *args, out=turned)
    assert torch.equal(turned, want)


# ------------------------------------------------------------------- streams, graphs, large caches
def big_call(seed, rows_=4, q=1, dim=128, dtype=torch.bfloat16):
    need_gpu()
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    cfg = rq.make_kv_cfg(2, dim, 64, 4)
    cache = rq.kv_cache_alloc(rows_ * 64, cfg)
    K = torch.randn(rows_ * 4096, 2, dim, generator=g, device="cuda").bfloat16()
    rq.kv_cache_write(K, K.flip(0), torch.arange(rows_ * 4096, device="cuda"), cache, cfg)
    pages = torch.arange(rows_ * 64, dtype=torch.int32, device="cuda").view(rows_, 64)
    n = torch.tensor([4096 - 501 * b for b in range(rows_)], dtype=torch.int32, device="cuda")
    Q = torch.randn(rows_ * q, 8, dim, generator=g, device="cuda").to(dtype)
    return Q, cache, pages, n, cfg


@pytest.mark.parametrize("q", [1, 50])
def test_two_streams_at_once(q):
    a, b = big_call(1, q=q), big_call(2, q=q)
    want = rq.kv_attention(*a), rq.kv_attention(*b)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, args in enumerate((a, b)):
            if i == 0:
                got[i].append(rq.kv_attention(*args, stream=s[i]))
            else:
                with torch.cuda.stream(s[i]):
                    got[i].append(rq.kv_attention(*args))
    torch.cuda.synchronize()
    for i in range(2):
        for x in got[i]:
            assert torch.equal(x, want[i])


@pytest.mark.parametrize("q", [1, 50])
def test_captured_and_replayed(q):
    """Write, attention and read in one graph, replayed over changed inputs with eager calls in between."""
    Q, cache, pages, n, cfg = big_call(3, q=q)
    eager_cache = cache.clone()
    K = torch.randn(8, 2, 128, device="cuda").bfloat16()
    slots = torch.arange(0, 8 * 300, 300, device="cuda")

    def step(c):
        rq.kv_cache_write(K, K, slots, c, cfg)
        return rq.kv_attention(Q, c, pages, n, cfg, return_lse=True) + rq.kv_cache_read(c, slots, cfg)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache)
    for k in range(5):
        Q.copy_(torch.randn_like(Q))
        K.copy_(torch.randn_like(K))
        slots.copy_(torch.arange(k, k + 8 * 300, 300, device="cuda"))
        n.copy_(torch.tensor([4000 - 37 * k, 4096, 5, 64 * k], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        want = step(eager_cache)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        assert torch.equal(cache, eager_cache)


def test_many_sequences_without_hints():
    """A ragged batch of single tokens whose longest the call is not told: launched as if any sequence had all rows."""
    rng, c, cfg = make(64, 8, 16, heads=2, pages=400)
    kv_len = [int(x) for x in rng.integers(0, 60, 90)]
    pages = fill(rng, c, kv_len)
    Q = rng.normal(size=(90, 4, 64))
    check(c, cfg, Q, pages, kv_len, [1] * 90, "f16")


def test_equal_calls_give_equal_bits():
    for q in (1, 50):
        args = big_call(4, q=q)
        first = rq.kv_attention(*args, return_lse=True)
        for _ in range(3):
            again = rq.kv_attention(*args, return_lse=True)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_callers_workspace():
    Q, cache, pages, n, cfg = big_call(5)
    need = rq.kv_attention_workspace_size(4, 8, 4, 64, cfg)
    assert need > 0
    want = rq.kv_attention(Q, cache, pages, n, cfg)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")    # NaN: nothing has to be cleared
    assert torch.equal(rq.kv_attention(Q, cache, pages, n, cfg, workspace=ws), want)
    assert torch.all(ws[need:] == 0xFF)
    with pytest.raises(ValueError):
        rq.kv_attention(Q, cache, pages, n, cfg, workspace=ws[:need - 1])


@pytest.mark.parametrize("q", [1, 40])
def test_offsets_past_32_bits(q):
    """A cache of over 8 GiB, pages at its far end; its tokens' copies near the start give equal bits."""
    need_gpu()
    cfg = rq.make_kv_cfg(8, 256, 256, 8)
    pages = (9 << 30) // rq.rq_kv_page_bytes(cfg)
    cache = rq.kv_cache_alloc(pages, cfg)
    K = torch.randn(1000, 8, 256, device="cuda").half()
    V = torch.randn(1000, 8, 256, device="cuda").half()
    far = (pages - 4) * 256
    for at in (0, far):
        rq.kv_cache_write(K, V, torch.arange(at, at + 1000, device="cuda"), cache, cfg)
    assert torch.equal(cache[:3], cache[pages - 4:pages - 1])
    near, gone = (rq.kv_cache_read(cache, torch.arange(at, at + 1000, device="cuda"), cfg) for at in (0, far))
    assert torch.equal(near[0], gone[0]) and torch.equal(near[1], gone[1])
    Q = torch.randn(q, 8, 256, device="cuda").half()
    n = torch.tensor([1000], dtype=torch.int32, device="cuda")
    outs = [rq.kv_attention(Q, cache, torch.arange(at, at + 4, dtype=torch.int32, device="cuda")[None], n, cfg)
            for at in (0, pages - 4)]
    assert torch.equal(outs[0], outs[1])


# --------------------------------------------------------------------------------- used together
@pytest.mark.parametrize("bits", BITS)
def test_a_block_with_its_cache(bits):
    """qkv projection, keys and values into the cache, attention, out projection, over a prompt and
    then token by token, each on the framework's own paths; every step against the plain forms."""
    need_gpu()
    rng = np.random.default_rng(7)
    dim, heads, kv_heads, width = 64, 4, 2, 256
    W = torch.from_numpy(rng.normal(0, 0.06, size=((heads + 2 * kv_heads) * dim, width)).astype(np.float32)).cuda()
    Wo = torch.from_numpy(rng.normal(0, 0.06, size=(width, heads * dim)).astype(np.float32)).cuda()
    Wq, ws = rq.quantize_weights(W, bits=8)
    Wqo, wso = rq.quantize_weights(Wo, bits=8)
    c = kv_ref.Cache(8, kv_heads, dim, 16, bits, rng)
    cfg = rq.make_kv_cfg(kv_heads, dim, 16, bits)
    dev = c.flat().cuda()
    pages = np.array([[5, 2, 7, 0]], np.int32)
    x = torch.from_numpy(rng.normal(size=(40, width))).to(torch.bfloat16).cuda()
    done = 0
    for step in (33, 1, 1, 4, 1):
        rows_ = x[done:done + step]
        qkv = rq.rotq_linear(rows_, Wq, ws, bits=8).view(step, heads + 2 * kv_heads, dim)
        Q, K, V = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        j = np.arange(done, done + step)
        slots = pages[0][j // 16].astype(np.int64) * 16 + j % 16
        rq.kv_cache_write(K, V, torch.from_numpy(slots).cuda(), dev, cfg)
        done += step
        n = torch.tensor([done], dtype=torch.int32).cuda()
        O = rq.kv_attention(Q, dev, torch.from_numpy(pages).cuda(), n, cfg, max_kv_len=done)
        Y = rq.rotq_linear(O.reshape(step, heads * dim), Wqo, wso, bits=8)
        assert Y.shape == (step, width) and torch.isfinite(Y.float()).all()
        c.write(K.float().cpu().numpy(), V.float().cpu().numpy(), slots)
        assert torch.equal(dev.cpu(), c.flat())
        want, _, _, tol, _ = kv_ref.attention(Q.float().cpu().numpy(), c, pages, [done], [0, step], "bf16")
        assert np.all(np.abs(O.double().cpu().numpy() - want) <= tol)


def test_more_tokens_than_one_launch_takes():
    need_gpu()
    tokens, cfg = (1 << 27) + 37, rq.make_kv_cfg(1, 64, 16, 4)
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB of device memory")
    at = torch.tensor([0, 1, (1 << 27) - 1, 1 << 27, tokens - 1])
    x = torch.randn(5, 1, 64).bfloat16()
    slots = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")
    slots[at.cuda()] = torch.arange(5, device="cuda") * 3
    rows_in = torch.empty((tokens, 1, 64), dtype=torch.bfloat16, device="cuda")
    rows_in[at.cuda()] = x.cuda()
    small, cache = (rq.kv_cache_alloc(1, cfg) for _ in range(2))
    rq.kv_cache_write(x.cuda(), x.cuda(), torch.arange(5, device="cuda") * 3, small, cfg)
    rq.kv_cache_write(rows_in, rows_in, slots, cache, cfg)
    want = rq.kv_cache_read(small, torch.arange(5, device="cuda") * 3, cfg)[0]
    K, V = rq.kv_cache_read(cache, slots, cfg, out=(rows_in, torch.empty_like(rows_in)))
    assert torch.equal(K[at.cuda()], want) and torch.equal(V[at.cuda()], want)
    assert not K[5:4096].any() and not K[-30:-1].any() and not V[-30:-1].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("q", [1, 5, 150])
def test_a_query_that_is_no_number_stays_alone(q, bad):
    """Its own row is no number either; the others', in its tile and elsewhere, keep their bits."""
    kv_len = [200, 170]
    rng, c, cfg = make(128, 4, 16, heads=2, pages=32)
    pages = torch.from_numpy(fill(rng, c, kv_len)).cuda()
    n, dev = torch.tensor(kv_len, dtype=torch.int32, device="cuda"), c.flat().cuda()
    for dtype in (torch.float16, torch.bfloat16):
        Q = torch.from_numpy(rng.normal(size=(2 * q, 4, 128))).to(dtype).cuda()
        want, want_lse = rq.kv_attention(Q, dev, pages, n, cfg, return_lse=True)
        Q[q, 1, 7] = bad
        got, lse = rq.kv_attention(Q, dev, pages, n, cfg, return_lse=True)
        assert got[q, 1].isnan().all()
        got[q, 1], lse[q, 1] = want[q, 1], want_lse[q, 1]
        assert torch.equal(got, want) and torch.equal(lse, want_lse)


def spoil(c, pages, b, tokens, value):
    """Scales of a sequence's tokens as bytes that nobody wrote may read: `value`. What the reference takes
    for these tokens is as bad."""
    for t in tokens:
        p, i = int(pages[b][t // c.page]), t % c.page
        for part in range(2):
            at = 2 * c.page * c.row + (part * c.page + i) * 4
            c.bytes[p, :, at:at + 4] = np.frombuffer(np.float32(value).tobytes(), np.uint8)
            c.scale[part, p * c.page + i] = value


UNWRITTEN = [float("nan"), float("inf"), float("-inf"), 3.0e38]


@pytest.mark.filterwarnings("ignore:invalid value")
@pytest.mark.parametrize("value", UNWRITTEN)
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("dim,bits", [(128, 4), (64, 8), (256, 4)])
@pytest.mark.parametrize("q_len,kv_len,window,split", [
    ([2, 1, 1], [200, 75, 33], 40, False), ([70, 66, 3], [200, 150, 90], 33, False),
    ([2, 1, 1], [2900, 70, 1], 1500, True), ([40, 33, 1], [2100, 70, 1], 1500, True)])
def test_tokens_in_front_of_a_window_do_not_matter(q_len, kv_len, window, split, dim, bits, page, value):
    """Tokens that no row attends to, in a tile with some that rows do: never written, or given back."""
    rng, c, cfg = make(dim, bits, page, heads=1, pages=4096 // page)
    pages = fill(rng, c, kv_len)
    for b, (q, n) in enumerate(zip(q_len, kv_len)):
        spoil(c, pages, b, range(max(0, n - q + 1 - window)), value)
    need = rq.kv_attention_workspace_size(sum(q_len), 2, len(q_len), pages.shape[1], cfg, ragged=True, window=window,
                                          max_q_len=max(q_len))
    assert (need > 0) == split
    Q = rng.normal(size=(sum(q_len), 2, dim))
    for dtype in ("f16", "bf16"):
        check(c, cfg, Q, pages, kv_len, q_len, dtype, window=window, max_q_len=max(q_len))


@pytest.mark.parametrize("value", UNWRITTEN)
@pytest.mark.parametrize("q,kv,pad", [(5, 100, 3), (3, 64, 1), (20, 2900, 6), (90, 90, 40), (150, 1000, 30)])
def test_padding_at_a_sequences_end_does_not_matter(q, kv, pad, value):
    """A batch of equal lengths whose shorter sequences end in padding tokens, skipped by their slots of -1: rows in
    front of the padding keep their bits. (The padding's own rows attend to what nobody wrote.)"""
    rng, c, cfg = make(128, 4, 16, heads=2, pages=400)
    pages = fill(rng, c, [kv, kv])
    args = [torch.from_numpy(pages).cuda(), torch.tensor([kv, kv], dtype=torch.int32).cuda(), cfg]
    for dtype in (torch.float16, torch.bfloat16):
        Q = torch.from_numpy(rng.normal(size=(2 * q, 4, 128))).to(dtype).cuda()
        want, want_lse = rq.kv_attention(Q, c.flat().cuda(), *args, return_lse=True)
        kept = c.bytes.copy()
        spoil(c, pages, 0, range(kv - pad, kv), value)
        got, lse = rq.kv_attention(Q, c.flat().cuda(), *args, return_lse=True)
        c.bytes[:] = kept
        real = torch.arange(2 * q) < q - pad
        real[q:] = True
        assert torch.equal(got[real], want[real]) and torch.equal(lse[real], want_lse[real])


@pytest.mark.parametrize("kv,split", [(200, False), (3000, True)])
@pytest.mark.parametrize("q", [1, 5, 80])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_no_number_is_not_one_that_attends_to_nothing(bad, q, kv, split):
    """O and lse of its row are NaN however the keys are split; all others keep their bits."""
    rng, c, cfg = make(128, 4, 16, heads=1, pages=400)
    pages = torch.from_numpy(fill(rng, c, [kv, kv - 30])).cuda()
    n, dev = torch.tensor([kv, kv - 30], dtype=torch.int32, device="cuda"), c.flat().cuda()
    assert (rq.kv_attention_workspace_size(2 * q, 2, 2, pages.shape[1], cfg) > 0) == split
    for dtype in (torch.float16, torch.bfloat16):
        Q = torch.from_numpy(rng.normal(size=(2 * q, 2, 128))).to(dtype).cuda()
        want, want_lse = rq.kv_attention(Q, dev, pages, n, cfg, return_lse=True)
        Q[q, 1, 7] = bad
        got, lse = rq.kv_attention(Q, dev, pages, n, cfg, return_lse=True)
        assert got[q, 1].isnan().all() and lse[q, 1].isnan()
        got[q, 1], lse[q, 1] = want[q, 1], want_lse[q, 1]
        assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("at", [3, 150])
@pytest.mark.parametrize("kv,split", [(200, False), (3000, True)])
@pytest.mark.parametrize("q", [1, 5, 80])
def test_a_logit_beyond_binary32_is_not_dropped(q, kv, split, at):
    """One key whose logits are infinite: no finite result of the other keys takes its place."""
    rng, c, cfg = make(128, 4, 16, heads=1, pages=400)
    pages = fill(rng, c, [kv])
    k = np.zeros((1, 1, 128), np.float32)
    k[0, 0, 0] = 3e38
    c.write(k, np.ones((1, 1, 128), np.float32), pages[0][[at // 16]].astype(np.int64) * 16 + at % 16)
    dev, n = c.flat().cuda(), torch.tensor([kv], dtype=torch.int32, device="cuda")
    assert (rq.kv_attention_workspace_size(q, 2, 1, pages.shape[1], cfg) > 0) == split
    for dtype in (torch.float16, torch.bfloat16):
        Q = torch.from_numpy(np.abs(rng.normal(size=(q, 2, 128))) + 100.0).to(dtype).cuda()
        out, lse = rq.kv_attention(Q, dev, torch.from_numpy(pages).cuda(), n, cfg, return_lse=True, causal=False)
        assert out.isnan().all() and (lse.isnan() | lse.isposinf()).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 20, 2.0 ** 25, 2.0 ** 29, 2.0 ** 36, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("q,kv", [(1, 1), (1, 200), (5, 3000), (80, 150), (80, 3000)])
@pytest.mark.parametrize("dim,bits", [(128, 4), (64, 8)])
def test_logits_of_any_size(dim, bits, q, kv, size, sign):
    """Logits so far apart that a row's result is one key's value (or the mean of two equal keys' values), whatever
    the size of the logits and of the values. With a single weight (two equal ones) in the rotated domain: its
    rounding u of each |value|, spread over the block by the way back, 16 roundings of binary32, the output's."""
    rng, c, cfg = make(dim, bits, 16, heads=1, pages=400)
    pages = fill(rng, c, [kv])
    a = rng.normal(size=dim)
    slots = pages[0][np.arange(kv) // 16].astype(np.int64) * 16 + np.arange(kv) % 16
    m = sign * (1.0 + rng.permutation(kv) / max(kv, 2))
    if kv > 1:
        top2 = np.sort(m)[-2:]
        m[m == top2[0]] = top2[1]                  # the two largest are equal: the same codes and scale
    # |a|^2 dim^-1/2 m size, base 2: about `size`
    k = (a[None] * (m * size / (np.dot(a, a) * dim ** -0.5 * np.log2(np.e)))[:, None])[:, None].astype(np.float32)
    v = (rng.normal(size=(kv, 1, dim)) * 10.0 ** rng.uniform(-3, 3, size=(kv, 1, 1))).astype(np.float32)
    c.write(k, v, slots)
    assert (rq.kv_attention_workspace_size(q, 2, 1, pages.shape[1], cfg) > 0) == (kv > 1000)
    R, B = kv_ref.matrix(dim), min(128, dim)
    held = [(c.codes[p][slots, 0].astype(np.float64) * c.scale[p][slots, 0][:, None].astype(np.float64)) for p in range(2)]
    for dtype in ("f16", "bf16"):
        Q = torch.from_numpy(a[None, None] * (1.0 + rng.random((q, 2, 1)))).to(kv_ref.TORCH[dtype])
        L = (Q.double().numpy() @ R) @ held[0].T * dim ** -0.5                      # q, 2, kv
        order = np.sort(L, axis=-1)
        best = order[..., -1:]
        two = L == best
        assert (two.sum(-1) == min(kv, 2)).all()
        if kv > 2:
            assert ((best - order[..., -3:-2]) >= 2.0 ** -13 * np.abs(best)).all() and ((best - order[..., -3:-2]) * size >= 0).all()
        if kv > 2 and size < 2.0 ** 20:      # the others count for something: only the large ones are this test's
            continue
        P = two / two.sum(-1, keepdims=True)
        want = P @ (held[1] @ R)
        u = 2.0 ** -22 if dtype == "f16" else 2.0 ** -11
        rot = (P @ np.abs(held[1])) * (u + 16 * kv_ref.U32)
        e = np.repeat(rot.reshape(q, 2, -1, B).sum(-1) / np.sqrt(B), B, axis=-1)
        tol = e + kv_ref.EPS[dtype] * (np.abs(want) + e) + (2.0 ** -25 if dtype == "f16" else 0.0)
        out, lse = rq.kv_attention(Q.cuda(), c.flat().cuda(), torch.from_numpy(pages).cuda(),
                                   torch.tensor([kv], dtype=torch.int32).cuda(), cfg, causal=False, return_lse=True)
        assert np.all(np.abs(out.cpu().double().numpy() - want) <= tol)
        # lse: the logit's own error, R q in fp16 and dim sums, and that of its logarithm to base 2
        want_lse = best[..., 0] + np.log(two.sum(-1))
        A = np.abs(Q.double().numpy() @ R) @ np.abs(held[0]).T * dim ** -0.5
        assert np.all(np.abs(lse.cpu().double().numpy() - want_lse) <= (u + 2 * (dim + 32) * kv_ref.U32) * A.max(-1) + 2.0 ** -16)


@pytest.mark.parametrize("size", [2.0 ** 23, 2.0 ** 31, 2.0 ** 50])
@pytest.mark.parametrize("behind", [False, True])
@pytest.mark.parametrize("q,kv", [(1, 200), (5, 3200), (80, 160), (80, 3200)])
def test_large_and_ordinary_logits_in_one_row(q, kv, behind, size):
    """Keys with very negative logits, in front of or behind ordinary ones: as if they were not there. One with a very
    large logit: as if the others were not there. And the same rows beside rows that are not touched by them."""
    rng, c, cfg = make(128, 4, 16, heads=1, pages=400)
    pages = fill(rng, c, [kv])
    a = rng.normal(size=128)
    a *= np.sqrt(128) / np.linalg.norm(a)                               # |a|^2 / sqrt(128) = 11.3
    far = np.arange(kv - 64, kv) if behind else np.arange(64)           # whole pages
    slots = lambda j: pages[0][j // 16].astype(np.int64) * 16 + j % 16
    low = (a[None, None] * -size * (1.0 + rng.random((64, 1, 1)))).astype(np.float32)
    c.write(low, rng.normal(size=(64, 1, 128)).astype(np.float32) * 100, slots(far))
    near_pages = pages[:, :-4] if behind else pages[:, 4:]
    n = torch.tensor([kv], dtype=torch.int32).cuda()
    for dtype in ("f16", "bf16"):
        Q = rng.normal(size=(q, 2, 128))
        Q = Q - (Q @ a)[..., None] * a / 128 + a                         # each q . a = 128
        Q = torch.from_numpy(Q).to(kv_ref.TORCH[dtype])
        Qf = Q.float().numpy()
        want, lse, _, tol, lse_tol = kv_ref.attention(Qf, c, near_pages, [kv - 64], [0, q], dtype, causal=False)
        got, got_lse = rq.kv_attention(Q.cuda(), c.flat().cuda(), torch.from_numpy(pages).cuda(), n, cfg, causal=False, return_lse=True)
        assert np.all(np.abs(got.cpu().double().numpy() - want) <= tol)
        assert np.all(np.abs(got_lse.cpu().double().numpy() - lse) <= lse_tol)
        # One row's queries turned to the other side: its logits are large, the other rows keep their bits.
        Q2 = Q.clone()
        Q2[q // 2, 1] = -Q2[q // 2, 1]
        got2, lse2 = rq.kv_attention(Q2.cuda(), c.flat().cuda(), torch.from_numpy(pages).cuda(), n, cfg, causal=False, return_lse=True)
        R = kv_ref.matrix(128)
        L = Q2[q // 2, 1].double().numpy() @ (c.codes[0][slots(far), 0].astype(np.float64) * c.scale[0][slots(far), 0][:, None] @ R).T
        best = np.argsort(L)
        assert L[best[-1]] - L[best[-2]] > 1e-5 * L[best[-1]]
        v = c.codes[1][slots(far[best[-1:]]), 0][0].astype(np.float64) * c.scale[1][slots(far[best[-1:]]), 0]
        u = 2.0 ** -22 if dtype == "f16" else 2.0 ** -11
        e = np.abs(v).sum() / np.sqrt(128) * (u + 16 * kv_ref.U32)
        err = np.abs(got2[q // 2, 1].cpu().double().numpy() - v @ R)
        if (L[best[-1]] - L[best[-2]]) * 128 ** -0.5 > 60:
            assert np.all(err <= e + kv_ref.EPS[dtype] * (np.abs(v @ R) + e) + 2.0 ** -25)
        got2[q // 2, 1], lse2[q // 2, 1] = got[q // 2, 1], got_lse[q // 2, 1]
        assert torch.equal(got2, got) and torch.equal(lse2, got_lse)
