"""Plain reference of the INT8 paged KV cache operators (numpy), written from
their definitions: the append in fp32 operation by operation (its codes,
scales and rotated queries are compared bit for bit) and in 64 bits, the
attention in 64 bits with a bound on what fp32 arithmetic may add."""
from __future__ import annotations

from dataclasses import dataclass, field

import numpy as np

from int8_gemm_token_b200 import synth

F = np.float32


@dataclass
class Cache:
    """Codes int8 [pages, heads, page, d] and scales fp32 [pages, heads]."""
    k: np.ndarray
    v: np.ndarray
    ks: np.ndarray
    vs: np.ndarray

    @property
    def page(self):
        return self.k.shape[2]

    @property
    def d(self):
        return self.k.shape[3]

    def copy(self):
        return Cache(self.k.copy(), self.v.copy(), self.ks.copy(), self.vs.copy())


@dataclass
class Seqs:
    table: np.ndarray            # int32 [batch, max_pages]
    start: np.ndarray            # int32 [batch + 1]
    kv: np.ndarray               # int32 [batch]
    spare: int = 0               # rows behind the last sequence
    tokens: int = field(init=False)

    def __post_init__(self):
        self.tokens = int(self.start[-1]) + self.spare

    @property
    def new(self):
        return np.diff(self.start)


def make_seqs(rng, new, ctx, page, spare=0, extra_pages=2, width_extra=1, kv=None):
    """Sequences with `new` tokens behind `ctx` cached ones, on shuffled pages; -> (Seqs, pages)."""
    kv = np.array([a + b for a, b in zip(new, ctx)] if kv is None else kv, dtype=np.int32)
    need = [-(-int(n) // page) for n in kv]
    pages = sum(need) + extra_pages
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(new), max(need + [1]) + width_extra), -1, dtype=np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return Seqs(table, np.concatenate([[0], np.cumsum(new)]).astype(np.int32), kv, spare), pages


def random_cache(rng, pages, heads, page, d):
    def codes():
        return np.clip(np.rint(rng.standard_normal((pages, heads, page, d), dtype=F) * 40), -127, 127).astype(np.int8)

    def scales():
        return rng.uniform(0.01, 0.04, (pages, heads)).astype(F)
    return Cache(codes(), codes(), scales(), scales())


def angles(positions, rot, base=10000.0):
    half = rot // 2
    a = np.arange(positions, dtype=np.float64)[:, None] * base ** (-np.arange(half, dtype=np.float64) / half)
    return np.cos(a).astype(F), np.sin(a).astype(F)


def rotate(x, cos, sin, interleaved, dtype=F):
    """x [..., d] turned by cos, sin [..., rot / 2]; each operation in `dtype`."""
    if cos is None:
        return x.astype(dtype)
    x, c, s = x.astype(dtype), cos.astype(dtype), sin.astype(dtype)
    half = c.shape[-1]
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


def _sym(x, r):
    with np.errstate(invalid="ignore"):
        return np.clip(np.rint(x * r), -127, 127).astype(np.int8)


def append(cache: Cache, s: Seqs, k, v, cos=None, sin=None, interleaved=False):
    """The cache after the append; k, v float32 [tokens, heads, d] (values of bf16)."""
    out = cache.copy()
    page = cache.page
    for b in range(len(s.kv)):
        n, q = int(s.kv[b]), int(s.new[b])
        first = n - q
        pos = max(first, 0)
        while pos < n:
            pi = pos // page
            end = min(n, (pi + 1) * page)
            p = int(s.table[b, pi])
            rows = slice(s.start[b] + pos - first, s.start[b] + end - first)
            for codes, scale, x, turn in ((out.k, out.ks, k, True), (out.v, out.vs, v, False)):
                x = x[rows].astype(F)
                if turn and cos is not None:
                    x = rotate(x, cos[pos:end][:, None], sin[pos:end][:, None], interleaved)
                old = pos % page
                for h in range(x.shape[1]):
                    s_old = scale[p, h] if old else F(0)
                    S = max(s_old, F(np.abs(x[:, h]).max() / F(127)))
                    with np.errstate(divide="ignore", over="ignore"):
                        r = F(1) / S if S > 0 else F(0)
                    if np.isinf(r):
                        S = r = F(0)
                    if old and S != s_old:
                        ratio = F(s_old / S) if S > 0 else F(0)
                        codes[p, h, :old] = _sym(codes[p, h, :old].astype(F), ratio)
                    codes[p, h, old:old + end - pos] = _sym(x[:, h], r)
                    scale[p, h] = S
            pos = end
    return out


def rotate_queries(s: Seqs, q, cos, sin, interleaved, keep):
    """bf16 bits of the rotated queries; `keep`: what rows of no sequence hold."""
    out = keep.copy()
    for b in range(len(s.kv)):
        for i in range(int(s.new[b])):
            t, pos = int(s.start[b]) + i, int(s.kv[b]) - int(s.new[b]) + i
            if pos < 0:
                out[t] = 0
                continue
            c = None if cos is None else cos[pos][None]
            out[t] = synth.bf16_bits(rotate(q[t], c, None if sin is None else sin[pos][None], interleaved))
    return out


def dense(cache: Cache, s_table_row, n, name):
    """float64 [heads, n, d]: the values of one sequence."""
    codes, scale = (cache.k, cache.ks) if name == "k" else (cache.v, cache.vs)
    m = -(-n // cache.page)
    if m == 0:
        return np.zeros((codes.shape[1], 0, cache.d))
    pages = s_table_row[:m].astype(np.int64)
    x = codes[pages].astype(np.float64) * scale[pages].astype(np.float64)[..., None, None]
    return np.concatenate(list(x), axis=1)[:, :n]


def gather(cache: Cache, table, first, start, keep):
    """float32 [rows, heads, d] of k and v: one product in fp32."""
    outs = []
    for codes, scale in ((cache.k, cache.ks), (cache.v, cache.vs)):
        out = keep.copy()
        for b in range(len(first)):
            for i in range(int(start[b + 1] - start[b])):
                pos = int(first[b]) + i
                p = int(table[b, pos // cache.page])
                out[start[b] + i] = codes[p, :, pos % cache.page].astype(F) * scale[p][:, None]
        outs.append(out)
    return outs


def few_rows(max_new, hq, cache: Cache, s: Seqs):
    """Whether the kernel for few query rows of a kv head takes the call (its products round to other formats)."""
    heads, max_kv = cache.k.shape[1], s.table.shape[1] * cache.page
    rows = int(max_new) * (hq // heads)
    return rows <= 32 or (rows <= 64 and (len(s.kv) * heads <= 64 or max_kv >= 4096))


def attention(cache: Cache, s: Seqs, q, scale, softcap=0.0, window=0, slopes=None, prefix=None, few=True):
    """(out, tolerance) float64 [tokens, q_heads, d], NaN in rows of no sequence.

    The tolerance counts what fp32 arithmetic may add, to first order. With
    u = 2^-23 (an fp32 step: the tensor core may truncate):
      a score is a sum of d exact products, off by at most d u sum|q k|
      (times its factor), and its few further operations by 8 u of the
      largest value that enters them: delta;
      a weight is exp(score): off by a factor 1 + 2 delta against the row's
      maximum, by 2^-21 in the exponential and, where it is rounded for the
      second product, by 2^-11 with `few` query rows of a kv head (fp16, and
      there by at least 2^-25 of the row's largest weight times scale, which
      meets a code of at most 127), else by 2^-8 (bf16);
      sums of n terms in fp32 by n u; the quotient by 2 u more.
    All of that times sum_j p_j |v_j| / sum_j p_j, then one rounding to bf16
    (2^-8 of the value). A relative bound ends where numbers do: against the
    row's maximum, whose weight is 1 (so the sum is at least 1), a weight
    below 2^-126 may become 0 and so may its product with v's scale, which
    moves the sum over v by at most 2^-126 |v_j| and 2^-126 |code_j|."""
    u = 2.0 ** -23
    weight_err = 2.0 ** -11 if few else 2.0 ** -8
    tokens, hq, d = q.shape
    heads = cache.k.shape[1]
    g = hq // heads
    out = np.full((tokens, hq, d), np.nan)
    tol = np.zeros((tokens, hq, d))
    for b in range(len(s.kv)):
        n, m = int(s.kv[b]), int(s.new[b])
        if m == 0:
            continue
        rows = slice(int(s.start[b]), int(s.start[b]) + m)
        kd, vd = dense(cache, s.table[b], n, "k"), dense(cache, s.table[b], n, "v")
        i = n - m + np.arange(m)[:, None]
        j = np.arange(n)[None]
        seen = j <= i
        if window:
            seen &= i - j < window
        if prefix is not None:
            seen |= j < prefix[b]
        seen &= i >= 0
        for h in range(hq):
            qh = q[rows, h].astype(np.float64)
            kh, vh = kd[h // g], vd[h // g]
            z = qh @ kh.T * scale
            delta = d * u * (np.abs(qh) @ np.abs(kh).T) * scale + 8 * u * np.abs(z)
            if softcap:
                z = softcap * np.tanh(z / softcap)
                delta = delta + 16 * u * softcap
            if slopes is not None:
                bias = float(slopes[h]) * (j - i)
                z = z + bias
                delta = delta + 8 * u * (np.abs(bias) + np.abs(z))
            z = np.where(seen, z, -np.inf)
            top = z.max(-1, keepdims=True, initial=-np.inf)
            p = np.exp(z - np.where(np.isinf(top), 0.0, top)) * seen
            l = p.sum(-1, keepdims=True)
            safe = np.where(l > 0, l, 1.0)
            out[rows, h] = p @ vh / safe
            dmax = np.where(seen, delta, 0.0).max(-1, keepdims=True, initial=0.0)
            rel = 2 * dmax + 8 * u * np.abs(np.where(np.isinf(top), 0.0, top)) + 2.0 ** -21 + weight_err + (n + 4) * u
            e = p @ np.abs(vh) / safe * rel
            if few:
                page = s.table[b, np.arange(n) // cache.page].astype(np.int64)
                largest = (p * cache.vs[page, h // g].astype(np.float64)).max(-1, keepdims=True, initial=0.0)
                e = e + 2.0 ** -25 * 127 * seen.sum(-1, keepdims=True) * largest / safe
            e = e + 2.0 ** -126 * (np.abs(vh).sum(0) + 127 * n)
            tol[rows, h] = e + 2.0 ** -8 * (np.abs(out[rows, h]) + e)
    return out, tol
