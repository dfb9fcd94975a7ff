"""Plain implementations for the tests of a cache held to a budget: attention weights added up in 64 bits,
with a bound of what the stated arithmetic may be off, and the choice and move of tokens on bytes."""
import numpy as np
import torch

from tests import kv_ref
from tests.kv_ref import U32


class Pages:
    """A cache on the device with codes and scales of every K row known; V's bytes are anything."""

    def __init__(self, pages, heads, dim, page, bits, seed=0, device="cuda"):
        gen = torch.Generator(device).manual_seed(seed)
        self.heads, self.dim, self.page, self.bits, self.pages, self.row = heads, dim, page, bits, pages, dim * bits // 8
        top = 127 if bits == 8 else 7
        self.block = page * (2 * self.row + 8)
        self.codes = torch.randint(-top, top + 1, (pages, heads, page, dim), generator=gen, device=device, dtype=torch.int8)
        # Keys of about unit elements: logits of a unit query spread over a few units.
        self.scale = torch.exp(0.5 * torch.randn(pages, heads, page, generator=gen, device=device)) * 2.0 / top
        self.bytes = torch.randint(0, 256, (pages, heads * self.block), generator=gen, device=device, dtype=torch.uint8)
        b = self.bytes.view(pages, heads, self.block)
        raw = self.codes.view(torch.uint8)
        if bits == 4:
            raw = (raw[..., 0::2] & 15) | (raw[..., 1::2] << 4)
        b[:, :, :page * self.row] = raw.reshape(pages, heads, -1)
        b[:, :, 2 * page * self.row:2 * page * self.row + 4 * page] = self.scale.contiguous().view(torch.uint8).view(pages, heads, -1)

    def spoil(self, table, b, tokens, value):
        """Scales of tokens of sequence b that were never written, as anything."""
        blocks = self.bytes.view(self.pages, self.heads, self.block)
        bits = torch.tensor(np.frombuffer(np.float32(value).tobytes(), np.uint8).copy(), device=blocks.device)
        for j in tokens:
            p, t = int(table[b, j // self.page]), j % self.page
            for part in range(2):
                at = 2 * self.page * self.row + (part * self.page + t) * 4
                blocks[p, :, at:at + 4] = bits

    def keys(self, table_row, n, head):
        """What K rows 0 .. n - 1 of a page table's row stand for, in the rotated domain (codes times scales),
        float64 [n, dim], and which of them are there."""
        j = torch.arange(n, device=self.codes.device)
        pg = table_row[j // self.page].long()
        ok = (pg >= 0) & (pg < self.pages)
        at = torch.where(ok, pg, 0)
        c = self.codes[at, head, j % self.page].double() * self.scale[at, head, j % self.page].double()[:, None]
        return c, ok


def table(cache, kv_len, extra=0, seed=0):
    """A page table [seqs, pages] of pages in any order, -1 behind a sequence's last, and the unused pages."""
    need = [-(-max(n, 0) // cache.page) for n in kv_len]
    order = torch.randperm(cache.pages, generator=torch.Generator().manual_seed(seed)).int()
    out = torch.full((len(kv_len), max(need + [1]) + extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        out[b, :n] = order[at:at + n]
        at += n
    return out.to(cache.codes.device), order[at:].to(cache.codes.device)


def mask(q, kv, causal, window, device):
    behind = (kv - q + torch.arange(q, device=device))[:, None] - torch.arange(kv, device=device)
    ok = torch.ones(q, kv, dtype=torch.bool, device=device)
    if causal:
        ok = behind >= 0
        if window:
            ok &= behind < window
    return ok


def logsums(cache, Q, pages, kv_len, q_start, causal, window, scale):
    """lse [total_q, q_heads], 64 bits."""
    R = torch.from_numpy(kv_ref.matrix(cache.dim)).to(Q.device)
    out = torch.full(Q.shape[:2], float("-inf"), dtype=torch.float64, device=Q.device)
    group = Q.shape[1] // cache.heads
    for b in range(len(kv_len)):
        q0, q1 = q_start[b], q_start[b + 1]
        for h in range(Q.shape[1]):
            K, there = cache.keys(pages[b], kv_len[b], h // group)
            ok = mask(q1 - q0, kv_len[b], causal, window, Q.device) & there
            L = (Q[q0:q1, h].double() @ R) @ K.t().contiguous() * scale
            out[q0:q1, h] = torch.logsumexp(L.masked_fill(~ok, float("-inf")), 1)
    return out


def weigh(cache, Q, lse, pages, kv_len, q_start, old, keep, causal, window, scale, max_q=None):
    """(weights, bound) float64 [seqs, heads, span] for lengths within the table.

    The bound: a logit's error as in kv_ref.attention with the queries in two fp16 parts (2^-22 an element,
    and 2^-33 of the row's largest where the second part is below fp16's normal range); the scale, 1 / sqrt B
    and log2 e 6 u of it; lse times log2 e one rounding each, 3 u of lse; the difference one, u of each; exp2 4 u,
    and nothing is left below 2^-126. A lane adds four rows' weights and these up over the tiles of 16 rows, then four
    lanes', the shares of rows and what was there: u each. (At most 64 shares, and an eighth of the tiles: those of one
    share and the shares are fewer together than all tiles in one chain.)"""
    R = torch.from_numpy(kv_ref.matrix(cache.dim)).to(Q.device)
    B, group = min(128, cache.dim), Q.shape[1] // cache.heads
    out, tol = old.double().clone(), torch.zeros_like(old, dtype=torch.float64)
    for b in range(len(kv_len)):
        q0, q1, n = q_start[b], q_start[b + 1], kv_len[b]
        rows = q1 - q0 if max_q is None else min(q1 - q0, max_q)
        for g in range(cache.heads):
            K, there = cache.keys(pages[b], n, g)
            sums = torch.zeros(n, dtype=torch.float64, device=Q.device)
            err = torch.zeros_like(sums)
            ok = (mask(q1 - q0, n, causal, window, Q.device) & there)[:rows]
            for h in range(g * group, (g + 1) * group):
                q = Q[q0:q0 + rows, h].double()
                fine = torch.isfinite(lse[q0:q0 + rows, h]) & torch.isfinite(q).all(1)
                q, s = torch.where(fine[:, None], q, 0.0), torch.where(fine, lse[q0:q0 + rows, h].double(), float("inf"))[:, None]
                rq = q @ R
                L = rq @ K.t().contiguous() * scale
                A = rq.abs() @ K.abs().t().contiguous() * scale
                spread = K.abs().sum(1)[None] * scale
                d = (2.0 ** -22 + (cache.dim + 8) * U32) * A + 8 * U32 * (q.abs().sum(1) / B ** 0.5)[:, None] * spread
                d = d + 2.0 ** -33 * rq.abs().amax(1)[:, None] * spread + 8 * U32 * L.abs() + 4 * U32 * torch.where(fine[:, None], s.abs(), 0.0)
                p = torch.where(ok, torch.exp(L - s), 0.0)
                sums += p.sum(0)
                err += (p * (torch.expm1(d) + 4 * U32)).sum(0) + rows * 2.0 ** -126
            before = torch.zeros_like(sums)
            if keep:
                before = keep * old[b, g, :n].double()
                if causal:
                    before[max(n - (q1 - q0), 0):] = 0.0
            out[b, g, :n] = before + sums
            tol[b, g, :n] = err + (rows * group / 16 + 24) * U32 * sums + 2 * U32 * out[b, g, :n].abs()
    return out, tol


def choose(weights, n, budget, first, recent):
    """The places that stay of n tokens with numpy float32 weights."""
    if n <= budget:
        return np.arange(n)
    lo, hi = first, n - recent
    w = weights[lo:hi].astype(np.float64)
    w = np.where(np.isnan(w), -np.inf, w) + 0.0
    # A NaN is below -inf too.
    order = np.lexsort((np.arange(hi - lo), np.isnan(weights[lo:hi]), -w))
    inner = lo + np.sort(order[:budget - first - recent])
    return np.concatenate((np.arange(lo), inner, np.arange(hi, n)))


def tokens(block, page, row):
    """(K rows, V rows, scales) of head blocks [..., bytes] (numpy, copies): [..., page, row] twice and [..., page, 2, 4]."""
    k = block[..., :page * row].reshape(*block.shape[:-1], page, row)
    v = block[..., page * row:2 * page * row].reshape(*block.shape[:-1], page // 4, row, 4)
    v = np.moveaxis(v, -1, -2).reshape(*block.shape[:-1], page, row)
    s = block[..., 2 * page * row:].reshape(*block.shape[:-1], 2, page, 4)
    return k.copy(), v.copy(), np.moveaxis(s, -3, -2).copy()


def blocks(k, v, s):
    """The inverse of tokens()."""
    page, row = k.shape[-2:]
    lead = k.shape[:-2]
    vv = np.moveaxis(v.reshape(*lead, page // 4, 4, row), -1, -2)
    return np.concatenate((k.reshape(*lead, -1), vv.reshape(*lead, -1), np.moveaxis(s, -2, -3).reshape(*lead, -1)), -1)


def evict(raw, heads, page, row, pages, kv_len, weights, budget, new_pages, first, recent):
    """(cache bytes, kept, new lengths) from numpy arrays; weights float32 [seqs, heads, span]."""
    total = raw.shape[0]
    k, v, s = tokens(raw.reshape(total, heads, -1), page, row)
    k0, v0, s0 = k.copy(), v.copy(), s.copy()
    kept = np.full((len(kv_len), heads, budget), -1, np.int32)
    lengths = []
    for b in range(len(kv_len)):
        n = min(max(int(kv_len[b]), 0), pages.shape[1] * page)
        lengths.append(min(n, budget))
        for h in range(heads):
            stay = choose(weights[b, h, :n], n, budget, first, recent)
            kept[b, h, :len(stay)] = stay
            for i, j in enumerate(stay):
                dst, src = new_pages[b, i // page], pages[b, j // page]
                if not 0 <= dst < total:
                    continue
                at, ok = j % page, 0 <= src < total
                k[dst, h, i % page] = k0[src, h, at] if ok else 0
                v[dst, h, i % page] = v0[src, h, at] if ok else 0
                s[dst, h, i % page] = s0[src, h, at] if ok else 0
    return blocks(k, v, s).reshape(raw.shape), kept, np.array(lengths, np.int32)
