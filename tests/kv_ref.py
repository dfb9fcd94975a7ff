"""The cache operators' plain implementation for the tests: the quantizer in binary32 (its steps
define the codes), everything that is computed from held codes in 64 bits, on the CPU."""
import numpy as np
import torch

EPS = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}      # half a step, relative
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24


def norm32(dim):
    return np.float32(1.0 / np.sqrt(np.float64(min(128, dim))))


def wht32(x):
    """Unnormalised transform of blocks of min(128, dim), stages 1, 2, 4, ... in binary32."""
    x = np.ascontiguousarray(x, np.float32).copy()
    dim, h = x.shape[-1], 1
    while h < min(128, dim):
        y = x.reshape(-1, dim // (2 * h), 2, h)
        a, b = y[:, :, 0].copy(), y[:, :, 1].copy()
        y[:, :, 0], y[:, :, 1] = a + b, a - b
        h *= 2
    return x


def matrix(dim):
    """The normalised rotation [dim, dim] (symmetric), 64 bits."""
    n = min(128, dim)
    H = np.ones((1, 1))
    while H.shape[0] < n:
        H = np.block([[H, H], [H, -H]])
    return np.kron(np.eye(dim // n), H / np.sqrt(n))


def quantise(x, bits):
    """Rows -> (codes int8, scales float32), every step one binary32 operation."""
    q = np.float32(127 if bits == 8 else 7)
    u = wht32(x)
    a = np.abs(u).max(-1)
    with np.errstate(divide="ignore", over="ignore"):
        inv = q / a
    zero = np.isinf(inv)
    inv = np.where(zero, np.float32(0), inv)
    scale = np.where(zero, np.float32(0), (a * norm32(x.shape[-1])) / q)
    return np.rint(u * inv[..., None]).astype(np.int8), scale.astype(np.float32)


def pack(codes, bits):
    if bits == 8:
        return codes.view(np.uint8)
    c = codes.astype(np.uint8) & 15
    return c[..., 0::2] | (c[..., 1::2] << 4)


class Cache:
    """A cache's bytes on the CPU, written token by token from the layout's description."""

    def __init__(self, pages, heads, dim, page, bits, rng):
        self.heads, self.dim, self.page, self.bits, self.pages = heads, dim, page, bits, pages
        self.row = dim * bits // 8
        self.block = page * (2 * self.row + 8)
        self.bytes = rng.integers(0, 256, (pages, heads, self.block), dtype=np.uint8)
        # what the slots hold: codes and scales, for the reference
        self.codes = np.zeros((2, pages * page, heads, dim), np.int8)
        self.scale = np.zeros((2, pages * page, heads), np.float32)

    def write(self, K, V, slots):
        for part, x in enumerate((K, V)):
            codes, scale = quantise(x, self.bits)
            raw = pack(codes, self.bits)
            for i, s in enumerate(slots):
                if not 0 <= s < self.pages * self.page:
                    continue
                self.codes[part, s], self.scale[part, s] = codes[i], scale[i]
                p, t = divmod(int(s), self.page)
                for h in range(self.heads):
                    b = self.bytes[p, h]
                    if part == 0:
                        b[t * self.row:(t + 1) * self.row] = raw[i, h]
                    else:
                        at = self.page * self.row + (t // 4) * self.row * 4 + t % 4
                        b[at:at + 4 * self.row:4] = raw[i, h]
                    at = 2 * self.page * self.row + (part * self.page + t) * 4
                    b[at:at + 4] = np.frombuffer(scale[i, h].tobytes(), np.uint8)

    def flat(self):
        return torch.from_numpy(self.bytes.reshape(self.pages, -1).copy())

    def rows(self, slots):
        """K and V [tokens, heads, dim] that the slots stand for, 64 bits; rows of slots outside are 0."""
        slots = np.asarray(slots)
        ok = (slots >= 0) & (slots < self.pages * self.page)
        s = np.where(ok, slots, 0)
        R = matrix(self.dim)
        return [np.where(ok[:, None, None], (self.codes[p][s].astype(np.float64) * self.scale[p][s][..., None].astype(np.float64)) @ R, 0.0)
                for p in range(2)]


def read_error(dim, scale, codes, out):
    """Bound of a read element's error: fl(1 / sqrt B), the product with the scale and the product
    with the (exact) transform round once each, then the output type's rounding of the value; below
    a type's normal range half its smallest step. [tokens, heads, 1], to add to eps * |value|."""
    big = np.abs(codes.astype(np.float64)).sum(-1) * scale.astype(np.float64) / np.sqrt(min(128, dim))
    tiny = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}[out]
    return (4 * U32 * big + tiny)[..., None]


def attention(Q, cache, pages, kv_len, q_start, dtype, causal=True, window=0, scale=None):
    """O [total_q, q_heads, dim] and lse in 64 bits, rows that are computed, and a bound of |O - kernel's|.

    The bound, from the arithmetic that convrot.h states. The transform of q in binary32: 7 stages, 8 u
    of the row's absolute sum; a logit's products and sums: dim + 8 steps, each u of sum |q_d k_d|. R q in
    fp16: 2^-11 an element (2^-22 in two parts), and 2^-25 / 2^8 of the row's largest below fp16's normal range. Logits in base
    2: the scale, 1 / sqrt B, log2 e: 6 u of |logit|, and of the row's largest, whose multiple is taken off. An error
    d of the logits changes a normalised weight by expm1(2 d) at most. exp2: 4 u and each rescaling of a
    partial sum 4 u (64 of them at most here). The weight's fp16: 2^-11 (2^-22 in two parts), and below fp16's
    normal range half of its smallest step, 2^-25, where the row's largest weight p s_v is at least 2^6: 2^-31 of
    that, a key, times a code. Sums over T keys: T u. These stand
    in the rotated domain; going back spreads a row's error over the block: sum / sqrt B. Then the output's half step."""
    total, q_heads, dim = Q.shape
    group = q_heads // cache.heads
    scale = dim ** -0.5 if scale is None else scale
    R, B = matrix(dim), min(128, dim)
    O = np.zeros((total, q_heads, dim))
    lse = np.full((total, q_heads), -np.inf)
    tol = np.zeros((total, q_heads, dim))
    lse_tol = np.zeros((total, q_heads))
    there = np.zeros(total, bool)
    uq = 2.0 ** -22 if dtype == "f16" else 2.0 ** -11
    for b in range(len(kv_len)):
        q0, q1 = int(q_start[b]), int(q_start[b + 1])
        n = min(max(int(kv_len[b]), 0), pages.shape[1] * cache.page)
        there[q0:q1] = True
        j = np.arange(n)
        pg = pages[b][j // cache.page].astype(np.int64) if n else np.zeros(0, np.int64)
        good = (pg >= 0) & (pg < cache.pages)
        slots = np.where(good, pg, 0) * cache.page + j % cache.page
        for h in range(q_heads):
            C = [cache.codes[p][slots, h // group].astype(np.float64) * cache.scale[p][slots, h // group][:, None].astype(np.float64) for p in range(2)]
            for i in range(q0, q1):
                q = Q[i, h].astype(np.float64)
                pos = n - (q1 - q0) + (i - q0)
                ok = good.copy()
                if causal:
                    ok &= j <= pos
                    if window:
                        ok &= j > pos - window
                if not ok.any():
                    continue
                rq = R @ q
                K, V = C[0][ok], C[1][ok]
                L = (K @ rq) * scale
                A = np.abs(K) @ np.abs(rq) * scale
                all_q = np.abs(q).sum() / np.sqrt(B)
                spread = np.abs(K).sum(1) * scale
                d = (uq + (dim + 8) * U32) * A + 8 * U32 * all_q * spread + 2.0 ** -33 * np.abs(rq).max() * spread
                d = d + 6 * U32 * (np.abs(L) + np.abs(L).max())
                m = L.max()
                P = np.exp(L - m)
                l = P.sum()
                P = P / l
                O[i, h] = R @ (P @ V)
                lse[i, h] = m + np.log(l)
                each = np.expm1(2 * d.max()) + uq + (len(L) + 4 + 64 * 4) * U32
                most = (P * cache.scale[1][slots, h // group][ok].astype(np.float64)).max()
                rot = P @ np.abs(V) * each + len(L) * 2.0 ** -31 * most * (127 if cache.bits == 8 else 7)
                blocks = rot.reshape(-1, B).sum(1) / np.sqrt(B)
                e = np.repeat(blocks, B) * (1 + 16 * U32)
                tol[i, h] = e + EPS[dtype] * (np.abs(O[i, h]) + e) + (2.0 ** -25 if dtype == "f16" else 0.0)
                lse_tol[i, h] = d.max() + (len(L) + 300) * U32 + 8 * U32 * (abs(lse[i, h]) + abs(m) + 1)
    return O, lse, there, tol, lse_tol
