"""Attention with capped, biased and masked scores in binary64, row by row, and
how far a kernel's results may lie from it."""
import numpy as np

import kv_ref


def seen(n, pos, window=0, first=0, prefix=0):
    """Which of n tokens a row at position pos sees."""
    t = np.arange(n)
    sees = ((t <= pos) | (t < prefix)) & (t >= first)
    return sees & (pos - t < window) if window else sees


def scores(q, k, scale, pos, softcap=0.0, slope=None):
    """Scores of the rows q [rows, dim] at position pos against the tokens k."""
    s = scale * (q @ k.T)
    if softcap:
        s = softcap * np.tanh(s / softcap)
    if slope is not None:
        s = s - slope[:, None] * np.abs(pos - np.arange(len(k)))
    return s


def score_error(q, ka, scale, pos, softcap=0.0, slope=None):
    """How far a score may be off.  The rounding errors of its partial sums add
    like a random walk: 2^-22 of scale times the 2-norm of the products of q and
    the keys' sizes ka (kv_ref.attention_rows), for the largest token; the cap
    passes on no more.  The cap itself is off by a few 2^-24 of the capped score
    (a polynomial, or an exponential, a reciprocal and a product where the score
    is over half the cap: 2^-21), the bias by a rounding or two of its own size
    (2^-22)."""
    off = 2.0 ** -22 * abs(scale) * np.sqrt((q ** 2) @ (ka ** 2).T).max(1)
    if softcap:
        off = off + 2.0 ** -21 * np.minimum(softcap, abs(scale) * (np.abs(q) @ ka.T).max(1))
    return off if slope is None else off + 2.0 ** -22 * slope * (pos + len(ka))


def row(q, k, v, ka, va, sees, scale, pos, part, softcap=0.0, slope=None):
    """(out, lse, slack of out, slack of lse, weights) of the rows q [rows, dim]:
    the formula, and the errors of sums, weights and scores that
    kv_ref.attention_rows describes; `part` is what a weight's rounding may be
    off by, relative to it."""
    rows, n = len(q), int(sees.sum())
    if not n:
        return np.zeros_like(q), np.full(rows, -np.inf), np.zeros(rows), np.zeros(rows), np.zeros((rows, len(k)))
    s = np.where(sees, scores(q, k, scale, pos, softcap, slope), -np.inf)
    top = s.max(1, keepdims=True)
    w = np.exp(s - top)
    total = w.sum(1, keepdims=True)
    w /= total
    off = score_error(q, ka[sees], scale, pos, softcap, slope)
    va = np.where(sees[:, None], va, 0)
    v = np.where(sees[:, None], v, 0)
    slack = (2.0 ** -18 * np.linalg.norm(w @ va, axis=1) + part * np.sqrt((w ** 2) @ (va ** 2).sum(1))
             + 2 * off * np.linalg.norm(w @ np.abs(v), axis=1))
    lse = (top + np.log(total))[:, 0]
    return w @ v, lse, slack, off + 2.0 ** -21 * (1 + np.abs(lse)), w


def paged(q, cache, table, lengths, scale, softcap=0.0, slopes=None, window=0, first=None):
    """q [B, L, Hq, D] over a kv_ref.Cache -> out, lse, slack, slack of lse, and
    the weights [B, tokens] that the tokens gather."""
    B, L, Hq, D = q.shape
    pages, heads, page = cache.shape
    group = Hq // heads
    part = 2.0 ** -16 if cache.bits == 16 and cache.dtype == "bf16" else 2.0 ** -22
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    slack, lse_slack = np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    gathered, may = (np.zeros((B, table.shape[1] * page)) for _ in range(2))
    for b in range(B):
        n = min(max(0, int(lengths[b])), table.shape[1] * page)
        there = np.array([0 <= p < pages for p in table[b]]).repeat(page)[:n]
        for h in range(heads if n else 0):
            k, ka, v, va = (np.zeros((n, D)) for _ in range(4))
            for p in range(-(-n // page)):
                if 0 <= table[b, p] < pages:
                    at = slice(p * page, min(n, (p + 1) * page))
                    (k[at], ka[at]), (v[at], va[at]) = (cache.row(x, table[b, p], h, at.stop - at.start)
                                                        for x in "kv")
            mine = slice(h * group, (h + 1) * group)
            slope = None if slopes is None else slopes[mine]
            for i in range(L):
                pos = n - L + i
                sees = there & seen(n, pos, window, 0 if first is None else first[b])
                o, l, s, ls, w = row(q[b, i, mine], k, v, ka, va, sees, scale, pos, part, softcap, slope)
                out[b, i, mine], lse[b, i, mine], slack[b, i, mine], lse_slack[b, i, mine] = o, l, s, ls
                gathered[b, :n] += w.sum(0)
                # a weight carries its score's error, and that of the logarithm it is given
                may[b, :n] += ((2 * ls + 2.0 ** -20)[:, None] * w).sum(0)
    return out, lse, slack, lse_slack, gathered, may


def prompt(q, k, v, q_starts, k_starts, scale, dtype, softcap=0.0, slopes=None, window=0, first=None,
           prefix=None):
    """q [Tq, Hq, D] over k, v [Tk, H, D] -> out, lse, slack, slack of lse; rows
    behind the last sequence are NaN.  A weight is rounded to the 16-bit type
    once: half a unit in the last place."""
    Hq, group = q.shape[1], q.shape[1] // k.shape[1]
    part = kv_ref.rounding(dtype)
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    slack, lse_slack = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    for b in range(len(q_starts) - 1):
        n, keys = q_starts[b + 1] - q_starts[b], slice(k_starts[b], k_starts[b + 1])
        length = keys.stop - keys.start
        for i in range(n):
            at, pos = q_starts[b] + i, length - n + i
            sees = seen(length, pos, window, 0 if first is None else first[at],
                        0 if prefix is None else prefix[b])
            for h in range(Hq // group):
                mine = slice(h * group, (h + 1) * group)
                if not length:
                    out[at, mine], lse[at, mine] = 0, -np.inf
                    continue
                kh, vh = k[keys, h], v[keys, h]
                out[at, mine], lse[at, mine], slack[at, mine], lse_slack[at, mine], _ = row(
                    q[at, mine], kh, vh, np.abs(kh), np.abs(vh), sees, scale, pos, part, softcap,
                    None if slopes is None else slopes[mine])
    return out, lse, slack, lse_slack


def lse_off(got, ref, slack):
    """Worst logarithm over what it may be off by; 0 and inf where it sees nothing."""
    none = ref == -np.inf
    assert np.array_equal(got[none], ref[none])
    return (np.abs(got[~none] - ref[~none]) / slack[~none]).max() if (~none).any() else 0.0
