"""Rotary positions on the GPU: turned rows are those of the formula -- angles
in binary64, the turn in binary32 with a rounding after each operation -- bit
for bit, far positions among them, and lie within their own rounding of the
turn in binary64; a cache that keys are turned into is bit for bit the one that
the separate calls write."""
import numpy as np
import pytest

import kv_ref
from gpu_util import out_bits, out_to_f64, to_dev, torch_dtype
from test_gpu_kv import _cache_bits, _dev16, aq  # noqa: F401  (aq: the module's fixture)

pytestmark = pytest.mark.gpu


def _pairs(x, half, interleaved):
    part = x[..., :2 * half]
    return (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])


def _join(x, a, b, interleaved):
    y = x.copy()
    half = a.shape[-1]
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a, b
    else:
        y[..., :half], y[..., half:2 * half] = a, b
    return y


def _turned(x, positions, freqs, interleaved, factor, dtype):
    """(16-bit patterns by the rounded formula, the turn in binary64)."""
    angle = positions.astype(np.float64)[:, None, None] * freqs.astype(np.float64)
    cos, sin = np.cos(angle) * factor, np.sin(angle) * factor
    a, b = _pairs(x, len(freqs), interleaved)
    exact = _join(x, a * cos - b * sin, b * cos + a * sin, interleaved)
    c, s, a, b = (z.astype(np.float32) for z in (cos, sin, a, b))
    rounded = _join(x, (a * c - b * s).astype(np.float64), (b * c + a * s).astype(np.float64), interleaved)
    return kv_ref.to_bits(rounded, dtype)[0], exact


def _strided(bits, dtype, before, after):
    """Rows as a part of wider ones."""
    import torch
    t = _dev16(bits, dtype)
    T, H, D = t.shape
    wide = torch.full((T, before + H * D + after), 7.0, dtype=t.dtype, device="cuda")
    part = wide[:, before:before + H * D].unflatten(1, (H, D))
    part.copy_(t)
    return part


FAR = [0, 1, 2, 5, 1000, 65535, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -1, -77777, -(2 ** 31)]
SHAPES = [  # tokens, query heads, key heads, dim, rotary
    (1, 1, 1, 64, 64), (12, 8, 2, 128, 128), (37, 7, 1, 256, 256), (5, 3, 3, 256, 64),
    (600, 4, 2, 64, 32), (513, 1, 1, 128, 16), (70, 40, 8, 128, 96), (1100, 2, 1, 64, 48),
    (4100, 1, 1, 64, 64), (8200, 1, 2, 64, 64), (2050, 2, 2, 256, 256)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rotary", SHAPES)
def test_rows(aq, T, Hq, Hk, D, rotary, interleaved, dtype):
    rng = np.random.default_rng(T + D)
    positions = rng.integers(-2 ** 31, 2 ** 31, T).astype(np.int32)
    positions[:min(T, len(FAR))] = FAR[:T]
    positions[len(FAR):] %= 100000
    freqs = (10000.0 ** (-np.arange(rotary // 2) / (rotary // 2))).astype(np.float32)
    factor = 1.0 if T % 2 else 1.2079441541679836
    (qb, qx), (kb, kx) = (kv_ref.to_bits(rng.standard_normal((T, H, D)) * 3, dtype) for H in (Hq, Hk))
    q, k = _strided(qb, dtype, 8, 16), _dev16(kb, dtype)
    pos, fr = to_dev(positions), to_dev(freqs)
    got = aq.aq_rope(q, k, pos, fr, interleaved, factor)
    for y, x, b in ((got[0], qx, qb), (got[1], kx, kb)):
        want, exact = _turned(x, positions, freqs, interleaved, factor, dtype)
        assert np.array_equal(out_bits(y)[..., rotary:], b[..., rotary:])
        # numpy's and the kernel's cosines may differ in the last place of binary32, which
        # a value's rounding shows once in thousands
        assert (out_bits(y) != want).mean() < 1e-3
        # one rounding to 16 bits, and of binary32: two factors, two products, a sum
        size = 2.0 ** -22 * factor * 2 * np.abs(x).max(-1, keepdims=True)
        off = np.abs(out_to_f64(y) - exact) - kv_ref.rounding(dtype) * np.abs(exact) - 2.0 ** -25
        assert (off <= size).all()
    # in place, one side alone, and the rows beside stay
    alone = aq.aq_rope(None, k, pos, fr, interleaved, factor)
    assert alone[0] is None and np.array_equal(out_bits(alone[1]), out_bits(got[1]))
    same = aq.aq_rope(q, None, pos, fr, interleaved, factor, q_out=q)
    assert same[0] is q and same[1] is None and np.array_equal(out_bits(q.contiguous()), out_bits(got[0]))
    if T > 1:
        beside = q.as_strided((T, 8), (q.stride(0), 1), 0)
        assert (beside == 7).all()


CASES = [(T, Hq, H, D, G, page) for T, Hq, H, D, G, page in (
    (1, 4, 1, 64, 32, 16), (3, 10, 5, 64, 64, 48), (64, 32, 8, 128, 64, 16), (130, 2, 2, 128, 128, 32),
    (1030, 3, 3, 128, 32, 64), (9, 1, 1, 256, 64, 16), (2050, 4, 4, 256, 128, 16), (17, 0, 2, 256, 32, 96),
    (8200, 1, 1, 64, 32, 16), (33, 64, 40, 64, 64, 16))]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("T,Hq,H,D,G,page", CASES)
def test_append_is_turn_and_append(aq, T, Hq, H, D, G, page, bits, dtype):
    import torch
    rng = np.random.default_rng(T + D + bits)
    rotary = D // (1 if T % 2 else 2)
    pages = T // page + 4
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    drop = rng.random(T) < 0.15
    slots[drop] = rng.choice([-1, pages * page, -(1 << 40), 1 << 40], drop.sum())
    slots, positions = to_dev(slots), to_dev(rng.integers(0, 1 << 20, T).astype(np.int32))
    freqs, factor = aq.aq_rope_frequencies(rotary, 10000.0, "by_index", 4.0, 4096.0, 1.0, 32.0)
    x = rng.standard_normal((T, H, D))
    x[..., ::29] *= 6
    if bits == 8 and T > 2:
        x[1, 0, 3], x[2, 0, D - 1] = np.nan, np.inf  # a NaN stays with its group
    k = _strided(kv_ref.to_bits(x, dtype)[0], dtype, 16, 8)
    v = _strided(kv_ref.to_bits(rng.standard_normal((T, H, D)), dtype)[0], dtype, 0, 24)
    q = _dev16(kv_ref.to_bits(rng.standard_normal((T, Hq, D)), dtype)[0], dtype) if Hq else None
    for interleaved in (False, True):
        one, two = (kv_ref.Cache(pages, H, page, D, G, bits, dtype).device() for _ in range(2))
        turned = torch.zeros((T, H, D), dtype=k.dtype, device="cuda")
        got = aq.aq_rope_append(q, k, v, positions, freqs, slots, *one, G, bits, interleaved, factor,
                                k_out=turned)
        wq, wk = aq.aq_rope(q, k, positions, freqs, interleaved, factor)
        aq.aq_kv_append(wk, v, slots, *two, G, bits)
        assert (got is None) == (q is None)
        if q is not None:
            assert np.array_equal(out_bits(got), out_bits(wq))
        assert np.array_equal(out_bits(turned), out_bits(wk))
        for a, b in zip(one, two):
            if a is not None:
                assert np.array_equal(_cache_bits(a), _cache_bits(b))
        # without the turned keys, the same
        three = kv_ref.Cache(pages, H, page, D, G, bits, dtype).device()
        aq.aq_rope_append(q, k, v, positions, freqs, slots, *three, G, bits, interleaved, factor)
        assert all(np.array_equal(_cache_bits(a), _cache_bits(b)) for a, b in zip(one, three) if a is not None)


def test_refusals(aq):
    import torch
    q, k = (torch.zeros((3, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2))
    pos, fr = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    aq.aq_rope(q, k, pos, fr)
    for bad in (lambda: aq.aq_rope(None, None, pos, fr), lambda: aq.aq_rope(q, k[:2], pos, fr),
                lambda: aq.aq_rope(q, k.bfloat16(), pos, fr), lambda: aq.aq_rope(q, k, pos[:2], fr),
                lambda: aq.aq_rope(q, k, pos, fr, q_out=k), lambda: aq.aq_rope(q.cpu(), None, pos, fr),
                lambda: aq.aq_rope(q.transpose(0, 1), None, pos, fr)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: aq.aq_rope(q, k, pos.long(), fr), lambda: aq.aq_rope(q, k, pos, fr.half())):
        with pytest.raises(TypeError):
            bad()
    for n in (33, 12):
        with pytest.raises(aq.AQError):
            aq.aq_rope(q, k, pos, torch.ones(n, device="cuda"))
