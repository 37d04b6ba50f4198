"""The cache and attention of the tests in binary64: packing by the CPU
oracle, everything else elementary numpy."""
import numpy as np

import oracle


def to_bits(x, dtype):
    """float64 -> uint16 patterns of f16 / bf16 and the exact values they hold."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64))
    t = t.to({"f16": torch.float16, "bf16": torch.bfloat16}[dtype])
    return t.view(torch.int16).numpy().view(np.uint16), t.double().numpy()


class Cache:
    """A paged cache on the host, bits 4 / 8 (codes, scales, biases) or 16."""

    def __init__(self, pages, heads, page, dim, group, bits, dtype="f16"):
        self.shape = (pages, heads, page)
        self.dim, self.group, self.bits, self.dtype = dim, group, bits, dtype
        self.parts = {}
        for n in "kv":
            if bits == 16:
                self.parts[n] = [np.zeros(self.shape + (dim,), np.uint16), None, None]
            else:
                self.parts[n] = [np.zeros(self.shape + (dim * bits // 32,), np.uint32),
                                 np.zeros(self.shape + (dim // group,), np.uint16),
                                 np.zeros(self.shape + (dim // group,), np.uint16)]

    def poison(self):
        """NaN scales and biases and the largest codes everywhere."""
        for n in "kv":
            p = self.parts[n]
            if self.bits == 16:
                p[0][:] = 0x7FFF
            else:
                p[0][:], p[1][:], p[2][:] = 0xFFFFFFFF, 0x7E00, 0xFE00

    def put(self, n, slot, rows_bits, rows):
        """Row [heads, dim] of one token, as bit patterns and as values."""
        page, at = slot // self.shape[2], slot % self.shape[2]
        if self.bits == 16:
            self.parts[n][0][page, :, at] = rows_bits
        else:
            for part, got in zip(self.parts[n], oracle.quantize(rows.astype(np.float32), self.group,
                                                                 self.bits)):
                part[page, :, at] = got

    def row(self, n, page, head, count):
        """(values, |bias| + 2^bits * scale) of the first `count` tokens of a page, binary64."""
        c, s, b = self.parts[n]
        if self.bits == 16:
            import torch
            t = torch.from_numpy(c[page, head, :count].view(np.int16).copy())
            v = t.view({"f16": torch.float16, "bf16": torch.bfloat16}[self.dtype]).double().numpy()
            return v, np.abs(v)
        v = oracle.dequantize_exact(c[page, head, :count], s[page, head, :count],
                                    b[page, head, :count], self.dim, self.group, self.bits)
        s64, b64 = (x[page, head, :count].view(np.float16).astype(np.float64) for x in (s, b))
        return v, np.repeat(np.abs(b64) + 2.0 ** self.bits * s64, self.group, axis=1)

    def device(self, null_biases=False):
        """The six arguments of the package's calls."""
        import torch
        out = []
        for n in "kv":
            c, s, b = self.parts[n]
            if self.bits == 16:
                dt = {"f16": torch.float16, "bf16": torch.bfloat16}[self.dtype]
                out += [torch.from_numpy(c.view(np.int16)).cuda().view(dt), None, None]
            else:
                out += [torch.from_numpy(c.view(np.int32)).cuda()]
                out += [torch.from_numpy(x.view(np.int16)).cuda().view(torch.float16) for x in (s, b)]
                if null_biases:
                    out[-1] = None
        return out


def attention(q, cache, table, lengths, scale):
    """q [B, L, Hq, D] -> (out, bound on the error before the output's own rounding).

    The bound's parts: a weight may be rounded to 11 bits once before its
    product (2^-11), and the binary32 arithmetic of scores, weights and sums
    may add as much again (2^-10 in all) of sum p (|b| + 2^bits s); a score
    carries at most 4 D 2^-24 of sum |q| (|b| + 2^bits s), which its weight
    then carries too.  A weight below the 11-bit format's normal range may be
    off by 2^-25 of the largest value (16 bits), or, scaled up by at least
    2^(bits-2) together with its group's scale, by 2^-23 of a step of one code
    times the number of codes: 2^-25 * 2^(2-bits) * 2^bits."""
    B, L, Hq, D = q.shape
    pages, heads, page = cache.shape
    group = Hq // heads
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = min(max(0, int(lengths[b])), table.shape[1] * page)
        for h in range(heads):
            ks, kas, vs, vas, at = [], [], [], [], []
            for p in range(-(-n // page)):
                count = min(page, n - p * page)
                if not 0 <= table[b, p] < pages:
                    continue
                k, ka = cache.row("k", table[b, p], h, count)
                v, va = cache.row("v", table[b, p], h, count)
                ks.append(k), kas.append(ka), vs.append(v), vas.append(va)
                at.append(np.arange(p * page, p * page + count))
            if not ks:
                continue
            k, ka, v, va, at = (np.concatenate(x) for x in (ks, kas, vs, vas, at))
            for i in range(L):
                sees = at <= n - L + i
                if not sees.any():
                    continue
                rows = slice(h * group, (h + 1) * group)
                s = scale * (q[b, i, rows] @ k[sees].T)
                off = 4 * D * 2.0 ** -24 * abs(scale) * (np.abs(q[b, i, rows]) @ ka[sees].T).max(1)
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                out[b, i, rows] = p @ v[sees]
                bound[b, i, rows] = ((2.0 ** -10 + 2 * off[:, None]) * (p @ va[sees])
                                     + sees.sum() * (2.0 ** -25 * np.abs(v[sees]).max()
                                                     if cache.bits == 16 else 2.0 ** -23))
    return out, bound


def rounding(dtype):
    """Unit roundoff of the output type."""
    return {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]


def attention_rows(q, cache, table, lengths, scale, change=None):
    """q [B, L, Hq, D] -> (out, slack [B, L, Hq]): the formula in binary64, and
    how far from it a result's row may lie, as the 2-norm over its D values,
    before the output's own rounding:

    * sums.  The values enter as p s code + p b, whose absolute values sum to at
      most V = p . (|b| + 2^bits s) (16 bits: p . |v|).  A wave adds its tiles
      into one binary32 sum, 64 of them at most in the tests, and a piece or a
      wave's share is rescaled and added a few more times: 64 * 2^-24 of V.
    * weights.  The two parts hold 2^-22 of a weight (bf16: 2^-16), rounded to
      either side, so that over the tokens of a row they add like a random walk:
      2^-22 (2^-16) of the 2-norm of p times the same sizes.
    * scores.  The rounding errors of one score's partial sums add like a random
      walk: 2^-22 of scale times the 2-norm over d of q_d (|b| + 2^bits s), for
      the largest token; a weight carries it once and the weights' sum once more.

    `change(p, sees)` gives other weights for the softmax's (to show what the
    comparison refuses)."""
    B, L, Hq, D = q.shape
    pages, heads, page = cache.shape
    group = Hq // heads
    part = 2.0 ** -16 if cache.bits == 16 and cache.dtype == "bf16" else 2.0 ** -22
    out, slack = np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        n = min(max(0, int(lengths[b])), table.shape[1] * page)
        for h in range(heads):
            rows = {"k": [], "v": [], "t": []}
            for p in range(-(-n // page)):
                if 0 <= table[b, p] < pages:
                    count = min(page, n - p * page)
                    for name in "kv":
                        rows[name].append(cache.row(name, table[b, p], h, count))
                    rows["t"].append(np.arange(p * page, p * page + count))
            if not rows["t"]:
                continue
            t = np.concatenate(rows["t"])
            (k, ka), (v, va) = ([np.concatenate(x) for x in zip(*rows[name])] for name in "kv")
            at = slice(h * group, (h + 1) * group)
            for i in range(L):
                sees = t <= n - L + i
                if not sees.any():
                    continue
                qi = q[b, i, at]
                s = scale * (qi @ k[sees].T)
                w = np.exp(s - s.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                if change:
                    w = change(w, t[sees])
                out[b, i, at] = w @ v[sees]
                of_sums = 2.0 ** -18 * np.linalg.norm(w @ va[sees], axis=1)
                of_weights = part * np.sqrt((w ** 2) @ (va[sees] ** 2).sum(1))
                score = 2.0 ** -22 * abs(scale) * np.sqrt((qi ** 2) @ (ka[sees] ** 2).T).max(1)
                of_scores = 2 * score * np.linalg.norm(w @ np.abs(v[sees]), axis=1)
                slack[b, i, at] = of_sums + of_weights + of_scores
    return out, slack


def rows_off(got, ref, slack, dtype):
    """Worst row of got against ref: the 2-norm of the error over what it may be,
    half as much again as the norm that rounding ref to the output's type leaves,
    the slack, and half a unit of fp16's smallest in every value."""
    own = np.linalg.norm(to_values(ref, dtype) - ref, axis=-1)
    off = np.linalg.norm(got - ref, axis=-1)
    return (off / (1.5 * own + slack + 2.0 ** -25 * np.sqrt(ref.shape[-1]))).max()


def to_values(x, dtype):
    """x rounded to f16 / bf16, in binary64."""
    return to_bits(x, dtype)[1]
