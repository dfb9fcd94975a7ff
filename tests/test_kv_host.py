"""The cache operators on the CPU: sizes, refusals before any launch, and the tests' own plain
implementation against the oracle and the definition."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import w4a4_integer_quantized_amd as rq
from tests import kv_ref

A = 0x10000          # fake, 16-byte aligned "device addresses": only compared, never touched
GB = 1 << 30


# ------------------------------------------------------------------------ the plain implementation
@pytest.mark.parametrize("bits", [8, 4])
def test_rows_of_128_are_the_quantizers_own(bits):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(37, 128)).astype(np.float32) * np.exp(rng.normal(size=(37, 1))).astype(np.float32)
    x[3] = 0.0
    x[4] = 0.0
    x[4, 5] = 1e-38        # q_max / absmax is infinite: a zero row
    x[5] = 0.0
    x[5, 0] = 7.0
    codes, scale = kv_ref.quantise(x, bits)
    want = oracle.quantize_rows(x, oracle.F32, bits)
    got_codes, got_scale = want[0], want[1]
    assert np.array_equal(codes, got_codes) and np.array_equal(scale, got_scale)
    assert scale[3] == 0 and scale[4] == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bits", [8, 4])
def test_held_rows_are_near_the_rows(dim, bits):
    """Half a code step an element in the rotated domain; the rotation keeps 2-norms."""
    rng = np.random.default_rng(dim + bits)
    x = rng.normal(size=(9, 3, dim))
    c = kv_ref.Cache(2, 3, dim, 16, bits, rng)
    c.write(x, x, np.arange(9))
    for got, s in zip(c.rows(np.arange(9)), c.scale):
        err = np.linalg.norm(got - x, axis=-1)
        assert np.all(err <= 0.5 * s[:9] * np.sqrt(dim) * (1 + 1e-5))


def test_rotation_is_orthogonal():
    for dim in (64, 128, 256):
        R = kv_ref.matrix(dim)
        assert np.allclose(R @ R.T, np.eye(dim), atol=1e-12) and np.allclose(R, R.T)
        x = np.random.default_rng(0).normal(size=(4, dim)).astype(np.float32)
        assert np.allclose(kv_ref.wht32(x) * kv_ref.norm32(dim), x @ R, atol=1e-5)


# ----------------------------------------------------------------------------------------- sizes
@pytest.mark.parametrize("bits,dim,heads,page", [(4, 128, 8, 64), (8, 64, 1, 16), (4, 256, 3, 1024), (4, 64, 65535, 16)])
def test_page_bytes(bits, dim, heads, page):
    got = rq.rq_kv_page_bytes(rq.make_kv_cfg(heads, dim, page, bits))
    assert got == heads * page * (2 * dim * bits // 8 + 8) and got % 128 == 0


@pytest.mark.parametrize("kw", [dict(bits=3), dict(bits=16), dict(head_dim=96), dict(head_dim=0), dict(page_size=48),
                                dict(page_size=8), dict(page_size=2048), dict(page_size=0), dict(page_size=-16),
                                dict(kv_heads=0), dict(kv_heads=65536), dict(kv_heads=-1)])
def test_bad_configurations(kw):
    cfg = rq.make_kv_cfg(**{**dict(kv_heads=8, head_dim=128), **kw})
    assert rq.rq_kv_page_bytes(cfg) == 0
    assert write(cfg=cfg) == rq.RQ_EUNSUPPORTED
    assert read(cfg=cfg) == rq.RQ_EUNSUPPORTED
    assert attend(cfg=cfg)[0] == rq.RQ_EUNSUPPORTED


# -------------------------------------------------------------------------------------- refusals
# Each call below is refused on the host, or has no tokens: nothing is launched.
def write(**kw):
    a = dict(K=A, V=A + GB, dtype=rq.RQ_BF16, tokens=0, kt=1024, kh=128, vt=1024, vh=128, slots=A + 2 * GB,
             cfg=rq.make_kv_cfg(8, 128), cache=A + 3 * GB, pages=100)
    a.update(kw)
    return rq.rq_kv_cache_write(a["K"], a["V"], a["dtype"], a["tokens"], a["kt"], a["kh"], a["vt"], a["vh"], a["slots"],
                                a["cfg"], a["cache"], a["pages"], None)


def read(**kw):
    a = dict(K=A, V=A + GB, dtype=rq.RQ_BF16, tokens=0, kt=1024, kh=128, vt=1024, vh=128, slots=A + 2 * GB,
             cfg=rq.make_kv_cfg(8, 128), cache=A + 3 * GB, pages=100)
    a.update(kw)
    return rq.rq_kv_cache_read(a["cache"], a["pages"], a["slots"], a["tokens"], a["cfg"], a["K"], a["V"], a["dtype"],
                               a["kt"], a["kh"], a["vt"], a["vh"], None)


def test_no_tokens_is_no_work():
    assert write() == rq.RQ_OK and read() == rq.RQ_OK
    assert write(K=None, V=None, slots=None) == rq.RQ_OK   # tensors of no tokens may have no address
    assert attend(total_q=0)[0] == rq.RQ_OK


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw,status", [
    (dict(K=None), rq.RQ_EINVAL), (dict(V=None), rq.RQ_EINVAL), (dict(slots=None), rq.RQ_EINVAL),
    (dict(cache=None), rq.RQ_EINVAL), (dict(K=A + 8), rq.RQ_EINVAL), (dict(V=A + GB + 2), rq.RQ_EINVAL),
    (dict(slots=A + 2 * GB + 4), rq.RQ_EINVAL), (dict(cache=A + 3 * GB + 4), rq.RQ_EINVAL),
    (dict(pages=0), rq.RQ_EINVAL), (dict(pages=-1), rq.RQ_EINVAL), (dict(pages=1 << 31), rq.RQ_EUNSUPPORTED),
    (dict(tokens=-1), rq.RQ_EINVAL), (dict(tokens=1 << 31), rq.RQ_EUNSUPPORTED), (dict(dtype=7), rq.RQ_EINVAL),
    (dict(kt=1025), rq.RQ_EINVAL), (dict(vh=4), rq.RQ_EINVAL), (dict(kh=-128), rq.RQ_EINVAL),
    (dict(kt=1 << 41), rq.RQ_EINVAL), (dict(vt=1 << 40, tokens=1 << 20), rq.RQ_EUNSUPPORTED),
    (dict(cache=A), rq.RQ_EINVAL), (dict(cache=A + GB + 16), rq.RQ_EINVAL), (dict(cache=A + 2 * GB), rq.RQ_EINVAL)])
def test_bad_rows_are_refused(call, kw, status):
    assert call(**{**dict(tokens=5), **kw}) == status
    assert rq.load().rq_last_error_detail()


def test_sizes_that_do_not_fit_64_bits():
    big = rq.make_kv_cfg(65535, 256, 1024, 8)
    for call in (write, read):
        assert call(tokens=1, cfg=big, pages=(1 << 31) - 1, kt=65535 * 256, vt=65535 * 256, kh=256, vh=256) == rq.RQ_EUNSUPPORTED
    assert attend(cfg=big, q_heads=65535, num_pages=(1 << 31) - 1)[0] == rq.RQ_EUNSUPPORTED
    # every sequence launched as if it had all rows: more workgroups than a launch holds
    many = dict(total_q=1 << 24, seqs=65535, q_heads=64, cfg=rq.make_kv_cfg(64, 64), qt=4096, ot=4096, qh=64, oh=64, O=A + (1 << 42),
                lse=None, ws=None)
    assert attend(**many)[0] == rq.RQ_EUNSUPPORTED


def test_the_stride_of_a_single_row_is_not_looked_at():
    one = rq.make_kv_cfg(1, 128)
    assert read(tokens=1, kt=3, vt=0, cfg=one, kh=7, vh=1, slots=None) == rq.RQ_EINVAL
    assert "slots" in rq.load().rq_last_error_detail().decode()      # all that is wrong with it


@pytest.mark.parametrize("kw", [dict(kt=512), dict(kh=64), dict(kt=0), dict(vh=0), dict(kt=128, kh=128), dict(V=A)])
def test_output_rows_may_not_overlap(kw):
    assert read(**{**dict(tokens=5), **kw}) == rq.RQ_EINVAL


def attend(**kw):
    a = dict(Q=A, O=A + GB, lse=A + 2 * GB, q_start=A + 3 * GB, kv_len=A + 4 * GB, pages=A + 5 * GB, total_q=7, qt=4096,
             qh=128, ot=4096, oh=128, max_q=0, max_kv=0, dtype=rq.RQ_BF16, q_heads=32, seqs=3, max_pages=4, causal=1, window=0,
             scale=0.1, cfg=rq.make_kv_cfg(8, 128), cache=A + 8 * GB, num_pages=100, ws=A + 20 * GB, ws_bytes=None)
    a.update(kw)
    p = rq.rq_kv_attention_params(a["Q"], a["O"], a["lse"], a["q_start"], a["kv_len"], a["pages"], a["total_q"], a["qt"],
                                  a["qh"], a["ot"], a["oh"], a["max_q"], a["max_kv"], a["dtype"], a["q_heads"], a["seqs"],
                                  a["max_pages"], a["causal"], a["window"], a["scale"])
    need = rq.rq_kv_attention_workspace_size(p, a["cfg"])
    if a["ws_bytes"] is None:
        a["ws_bytes"] = need
    return rq.rq_kv_attention(p, a["cfg"], a["cache"], a["num_pages"], a["ws"], a["ws_bytes"], None), need


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), rq.RQ_EINVAL), (dict(O=None), rq.RQ_EINVAL), (dict(kv_len=None), rq.RQ_EINVAL),
    (dict(pages=None), rq.RQ_EINVAL), (dict(cache=None), rq.RQ_EINVAL), (dict(Q=A + 8), rq.RQ_EINVAL),
    (dict(O=A + GB + 8), rq.RQ_EINVAL), (dict(kv_len=A + 4 * GB + 2), rq.RQ_EINVAL), (dict(lse=A + 2 * GB + 1), rq.RQ_EINVAL),
    (dict(q_start=A + 3 * GB + 2), rq.RQ_EINVAL), (dict(pages=A + 5 * GB + 2), rq.RQ_EINVAL),
    (dict(dtype=rq.RQ_F32), rq.RQ_EUNSUPPORTED), (dict(dtype=9), rq.RQ_EINVAL), (dict(total_q=-1), rq.RQ_EINVAL),
    (dict(seqs=-1), rq.RQ_EINVAL), (dict(seqs=0), rq.RQ_EINVAL), (dict(seqs=65536, total_q=65536), rq.RQ_EUNSUPPORTED),
    (dict(max_pages=-1), rq.RQ_EINVAL), (dict(max_pages=1 << 25), rq.RQ_EUNSUPPORTED), (dict(window=-1), rq.RQ_EINVAL),
    (dict(window=5, causal=0), rq.RQ_EINVAL), (dict(q_heads=0), rq.RQ_EINVAL), (dict(q_heads=12), rq.RQ_EINVAL),
    (dict(q_heads=-8), rq.RQ_EINVAL), (dict(total_q=1 << 27), rq.RQ_EUNSUPPORTED), (dict(total_q=1 << 62), rq.RQ_EUNSUPPORTED),
    (dict(scale=0.0), rq.RQ_EINVAL), (dict(scale=-1.0), rq.RQ_EINVAL), (dict(scale=float("nan")), rq.RQ_EINVAL),
    (dict(scale=float("inf")), rq.RQ_EINVAL), (dict(q_start=None), rq.RQ_EINVAL), (dict(qt=4097), rq.RQ_EINVAL),
    (dict(oh=64), rq.RQ_EINVAL), (dict(ot=128), rq.RQ_EINVAL), (dict(O=A), rq.RQ_EINVAL), (dict(O=A + 8 * GB), rq.RQ_EINVAL),
    (dict(lse=A + GB), rq.RQ_EINVAL), (dict(lse=A + 5 * GB), rq.RQ_EINVAL), (dict(num_pages=0), rq.RQ_EINVAL)])
def test_bad_attention_calls_are_refused(kw, status):
    assert attend(**kw)[0] == status
    assert rq.load().rq_last_error_detail()


def test_workspace_is_checked():
    big = dict(total_q=3, seqs=3, max_pages=2048)
    st, need = attend(**big, ws_bytes=0)
    assert need > 0 and st == rq.RQ_EWORKSPACE
    assert attend(**big, ws_bytes=need - 1)[0] == rq.RQ_EWORKSPACE
    assert attend(**big, ws=None, ws_bytes=need)[0] == rq.RQ_EINVAL
    assert attend(**big, ws=A + 20 * GB + 4, ws_bytes=need + 16)[0] == rq.RQ_EINVAL
    assert attend(**big, ws=A, ws_bytes=need)[0] == rq.RQ_EINVAL            # on Q
    assert attend(**big, ws=A + GB, ws_bytes=need)[0] == rq.RQ_EINVAL       # on O
    for ragged in (False, True):
        assert rq.kv_attention_workspace_size(3, 32, 3, 2048, rq.make_kv_cfg(8, 128), ragged=ragged) > 0


def test_null_pointers():
    lib = rq.load()
    none = ctypes.POINTER(rq.rq_kv_config)()
    p = rq.rq_kv_attention_params()
    assert lib.rq_kv_page_bytes(none) == 0
    assert lib.rq_kv_attention_workspace_size(ctypes.byref(p), none) == 0
    assert lib.rq_kv_attention(None, ctypes.byref(rq.make_kv_cfg(8, 128)), A, 1, None, 0, None) == rq.RQ_EINVAL
    assert lib.rq_kv_cache_write(A, A, 1, 1, 128, 128, 128, 128, A, none, A, 1, None) == rq.RQ_EINVAL


# ------------------------------------------------------------- wrappers (CPU tensors get no further)
def test_wrappers_check_their_tensors():
    cfg = rq.make_kv_cfg(2, 64, page_size=16)
    cache = rq.kv_cache_alloc(3, cfg, device="cpu")
    assert cache.shape == (3, rq.rq_kv_page_bytes(cfg)) and cache.dtype == torch.uint8
    K = torch.zeros(5, 2, 64)
    slots = torch.arange(5)
    bad = [(K[:, :1], K, slots, cache), (K, K.half(), slots, cache), (K.double(), K.double(), slots, cache),
           (K, K[:4], slots, cache), (K, K, slots.int(), cache), (K, K, slots[:4], cache), (K, K, slots, cache[:, :-1]),
           (K, K, slots, cache.view(torch.int8)), (K.transpose(1, 2), K, slots, cache), (K[0], K[0], slots, cache),
           (K, K, slots, cache)]        # the last: tensors that are not on a device
    for args in bad:
        with pytest.raises(ValueError):
            rq.kv_cache_write(*args, cfg)
    for kw in (dict(out_dtype=torch.float64), dict(out=(K, K.half())), dict(out=(K, K[:3])), dict(out=(K, K), out_dtype=torch.float16), {}):
        with pytest.raises(ValueError):
            rq.kv_cache_read(cache, slots, cfg, **kw)
    Q = torch.zeros(5, 4, 64, dtype=torch.float16)
    pages, n = torch.zeros(5, 2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    for args, kw in [((Q.float(), cache, pages, n), {}), ((Q[0], cache, pages, n), {}), ((Q, cache, pages.long(), n), {}),
                     ((Q, cache, pages, n[:4]), {}), ((Q, cache, pages[0], n), {}), ((Q, cache, pages, n), dict(q_start=n)),
                     ((Q, cache, pages, n), dict(out=Q.bfloat16())), ((Q[..., :32], cache, pages, n), {}), ((Q, cache, pages, n), {})]:
        with pytest.raises(ValueError):
            rq.kv_attention(*args, cfg, **kw)
    with pytest.raises(rq.ConvRotError):
        rq.kv_cache_alloc(3, rq.make_kv_cfg(2, 96), device="cpu")


def test_windows_of_any_width():
    cfg = rq.make_kv_cfg(8, 128)
    whole = rq.kv_attention_workspace_size(3, 32, 3, 2048, cfg)
    assert whole > 0
    for window in (1 << 30, (1 << 31) - 1, 1 << 31, (1 << 32) + 1, 1 << 40):
        assert rq.kv_attention_workspace_size(3, 32, 3, 2048, cfg, window=window) == whole
    for window in (-1, -(1 << 32) + 1):
        assert rq.kv_attention_workspace_size(3, 32, 3, 2048, cfg, window=window) == 0


def test_attention_grids_beyond_the_hardwares():
    """2^32 threads: 512 sequences of as many as 2^18 rows each, 8 heads, are 2^25 workgroups."""
    big = dict(total_q=1 << 18, seqs=512)
    assert attend(**big)[0] == rq.RQ_EUNSUPPORTED
    assert attend(**big, max_q=600, O=A)[0] == rq.RQ_EINVAL        # fits; refused later, for O on Q


# K and V read back into one buffer: accepted where no row of one meets a row of the other. Such calls are
# then refused for their missing slots.
def apart(**kw):
    st = read(**{**dict(tokens=5, slots=None), **kw})
    detail = rq.load().rq_last_error_detail().decode()
    assert st != rq.RQ_OK
    return detail == "slots is NULL", st


H, D, T, E = 8, 128, 5, 2      # heads, dim, tokens of the calls below, bytes an element


@pytest.mark.parametrize("kw", [
    dict(V=A + H * D * E, kt=2 * H * D, vt=2 * H * D),                                   # [T, 2, H, D]
    dict(K=A + H * D * E, V=A, kt=2 * H * D, vt=2 * H * D),                              # V first
    dict(V=A + D * E, kt=2 * H * D, vt=2 * H * D, kh=2 * D, vh=2 * D),                   # [T, H, 2, D]
    dict(V=A + T * D * E, kt=D, vt=D, kh=2 * T * D, vh=2 * T * D),                       # [H, 2, T, D]
    dict(V=A + H * 192 * E, kt=H * 320, vt=H * 320, kh=192, vh=128),                     # wider keys, a row of both a token
    dict(V=A + 3 * D * E, kt=H * D * 4, vt=H * D * 4, kh=4 * D, vh=4 * D),               # the last of four parts
    dict(V=A + T * H * D * E), dict(K=A + T * H * D * E, V=A),                           # one behind the other
    dict(tokens=1, V=A + D * E, kh=2 * D, vh=2 * D, kt=0, vt=7),
    dict(tokens=1 << 20, V=A + (D << 20) * E, kt=D, vt=D, kh=2 * D << 20, vh=2 * D << 20, cache=A + (1 << 43))])
def test_outputs_beside_each_other(kw):
    assert apart(**kw)[0]


@pytest.mark.parametrize("kw", [
    dict(V=A + 4 * D * E, kt=12 * D, vt=12 * D), dict(K=A + 4 * D * E, V=A, kt=12 * D, vt=12 * D),   # heads 0 .. 7, 4 .. 11
    dict(V=A + H * D * E), dict(V=A + 4 * H * D * E), dict(K=A + 4 * H * D * E, V=A),                # by whole tokens
    dict(V=A + 16), dict(V=A + D * E - 16, kt=2 * H * D, vt=2 * H * D, kh=2 * D, vh=2 * D),          # by parts of a row
    dict(tokens=1, V=A + 64 * E), dict(V=A + (7 * 192 + 120) * E, kt=H * 320, vt=H * 320, kh=192, vh=128),
    dict(V=A + T * D * E - 16, kt=D, vt=D, kh=2 * T * D, vh=2 * T * D),
    dict(tokens=1 << 20, V=A + (D << 20) * E - 16, kt=D, vt=D, kh=2 * D << 20, vh=2 * D << 20, cache=A + (1 << 43))])
def test_outputs_that_meet_are_refused(kw):
    assert apart(**kw) == (False, rq.RQ_EINVAL)


def test_outputs_in_each_other_in_unlike_orders_are_refused():
    assert apart(V=A + H * D * E, kt=4 * H * D, vt=D, vh=4 * T * D) == (False, rq.RQ_EUNSUPPORTED)


def test_outputs_of_any_strides_against_their_elements():
    """Every call that is let through has no element twice; every one refused as overlapping has one."""
    rng = np.random.default_rng(0)
    met = free = 0
    for _ in range(4000):
        tokens, heads, dim = int(rng.integers(1, 5)), int(rng.integers(1, 4)), 64
        def strides():
            a = dim + 16 * int(rng.integers(0, 6))
            n = heads if rng.random() < 0.7 else tokens
            b = a * n + 64 * int(rng.integers(0, 8))
            return (b, a) if n == heads else (a, b)
        k = strides()
        v = k if rng.random() < 0.5 else ((k[0], k[1] + 16 * int(rng.integers(-3, 4))) if rng.random() < 0.5 else strides())
        shift = 16 * int(rng.integers(-60, 60))
        def elements(s):
            return (np.arange(tokens)[:, None, None] * s[0] + np.arange(heads)[None, :, None] * s[1] + np.arange(dim)).ravel()
        ke, ve = elements(k), elements(v) + shift
        if len(np.unique(ke)) < ke.size or len(np.unique(ve)) < ve.size:
            continue
        got, st = apart(tokens=tokens, K=A + 65536, V=A + 65536 + shift * E, kt=k[0], kh=k[1], vt=v[0], vh=v[1],
                        cfg=rq.make_kv_cfg(heads, dim))
        if "rows overlap" in rq.load().rq_last_error_detail().decode():
            continue        # neither axis lies inside the other: refused before
        meet = np.intersect1d(ke, ve).size > 0
        if got:
            assert not meet
        elif st == rq.RQ_EINVAL:
            assert meet
        else:
            assert st == rq.RQ_EUNSUPPORTED and k != v
        met, free = met + meet, free + (got and not meet)
    assert met > 300 and free > 300
