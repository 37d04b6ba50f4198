"""Attention over the paged cache where its values are unusual: infinities and
NaN that some rows see and others do not, scales and scores far from one,
batches without a token, every form of the kernel.  Rows are compared by the
norm of their error, kv_ref.attention_rows says how large that may be."""
import numpy as np
import pytest

import kv_ref
import oracle
from gpu_util import out_to_f64
from test_gpu_kv import CASES, LONG, _attend, _build, aq  # noqa: F401  (aq: the module's fixture)

pytestmark = pytest.mark.gpu


def _queries(seed, shape, dtype, size=1.0):
    return kv_ref.to_bits(size * np.random.default_rng(seed).standard_normal(shape), dtype)


def _check(out, q, cache, table, lengths, dtype, scale=None, rows=None):
    """out against the formula, in the rows chosen."""
    got = out_to_f64(out)
    ref, slack = kv_ref.attention_rows(q, cache, table, lengths,
                                       q.shape[-1] ** -0.5 if scale is None else scale)
    if rows is not None:
        got, ref, slack = got[rows], ref[rows], slack[rows]
    assert np.isfinite(got).all()
    worst = kv_ref.rows_off(got, ref, slack, dtype)
    assert worst <= 1, f"worst row's error over its bound {worst:.3f}"


# ---- lanes that leave a branch ----------------------------------------------------------
def _compare(aq, lengths, per, heads, dim, G, bits, page, L, dtype, seed=61):
    cache, table = _build(lengths, heads, dim, G, bits, page, dtype, seed=seed)
    qb, q = _queries(seed + 1, (len(lengths), L, per * heads, dim), dtype)
    _check(_attend(aq, cache, table, lengths, qb, dtype, G), q, cache, table, lengths, dtype)


def test_heads_of_256_with_40_rows(aq):
    """This call once ended in a memory fault: lanes that the look-up of pages
    left out lost their thread's number, from which the rows' addresses are
    made (test_compiled_kernels.py has the check of the code itself)."""
    _compare(aq, [38] * 40, 5, 1, 256, 128, 8, 48, 8, "f16")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_heads_of_128_with_25_rows_of_16_bits(aq, dtype):
    """The form that holds the most registers."""
    _compare(aq, [100, 37, 6, 0], 5, 2, 128, 0, 16, 16, 5, dtype)


# ---- what a row does not see ------------------------------------------------------------
def _set_value(cache, table, b, t, head, bits16, d=slice(None)):
    """The value row of token t of sequence b, one head, as 16-bit patterns."""
    page = cache.shape[2]
    cache.parts["v"][0][table[b, t // page], head, t % page, d] = bits16


@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("L,per,dim", [(3, 2, 64), (8, 2, 128), (5, 5, 128), (3, 1, 256), (8, 5, 64)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_newer_values_stay_with_the_rows_that_see_them(aq, dtype, L, per, dim, what):
    """16-bit pages, several new tokens, one and two tiles of columns: a value
    of the newest or second newest token that is not finite leaves the rows of
    the tokens before it as they are."""
    lengths, heads = [100, 37, L + 1], 2
    cache, table = _build(lengths, heads, dim, 0, 16, 16, dtype, seed=L + dim)
    qb, q = _queries(51, (3, L, per * heads, dim), dtype)
    clean = _attend(aq, cache, table, lengths, qb, dtype, 0)
    _check(clean, q, cache, table, lengths, dtype)
    bad = {"nan": 0x7FFF, "inf": {"f16": 0x7C00, "bf16": 0x7F80}[dtype]}[what]
    for back in (1, 2):  # the newest token, the second newest
        dirty, _ = _build(lengths, heads, dim, 0, 16, 16, dtype, seed=L + dim)
        for b, n in enumerate(lengths):
            _set_value(dirty, table, b, n - back, 1, bad, slice(0, dim, 3))
        out = _attend(aq, dirty, table, lengths, qb, dtype, 0)
        got, want = out_to_f64(out), out_to_f64(clean)
        rest = np.arange(dim) % 3 != 0
        # the other head, and the tokens before: untouched
        assert np.array_equal(got[:, :, :per], want[:, :, :per])
        assert np.array_equal(got[:, :L - back, per:], want[:, :L - back, per:])
        # where it is seen, it is seen
        seen = got[:, L - back:, per:]
        assert not np.isfinite(seen[..., ~rest]).any()
        assert np.array_equal(seen[..., rest], want[:, L - back:, per:][..., rest])


@pytest.mark.parametrize("dim,per,L", [(64, 4, 1), (128, 4, 1), (128, 5, 5), (256, 4, 2), (64, 9, 4)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_infinite_values(aq, dtype, dim, per, L):
    """16-bit pages: an infinite value makes infinities of its sign in the rows
    that see it, however its weight is rounded; both signs in one place, NaN."""
    lengths, heads = [333, 40], 2
    cache, table = _build(lengths, heads, dim, 0, 16, 16, dtype, seed=81)
    qb, q = _queries(82, (2, L, per * heads, dim), dtype)
    clean = out_to_f64(_attend(aq, cache, table, lengths, qb, dtype, 0))
    inf = {"f16": 0x7C00, "bf16": 0x7F80}[dtype]
    for b, t, d, bits16 in ((0, 3, 5, inf), (0, 200, 6, inf | 0x8000), (0, 332 - L, 7, inf), (1, 20, 5, inf),
                            (0, 100, 9, inf), (0, 101, 9, inf | 0x8000)):
        _set_value(cache, table, b, t, 0, bits16, d)
    got = out_to_f64(_attend(aq, cache, table, lengths, qb, dtype, 0))
    want = clean.copy()
    want[0, :, :per, 5], want[0, :, :per, 6], want[0, :, :per, 7] = np.inf, -np.inf, np.inf
    want[0, :, :per, 9], want[1, :, :per, 5] = np.nan, np.inf
    assert np.array_equal(got, want, equal_nan=True)


# ---- weights and scales far from one ----------------------------------------------------
def _one_head(bits, dtype, G, dim, k, v, page=16):
    """A cache of one sequence and one head with the rows k and v [n, dim]."""
    n = k.shape[0]
    cache = kv_ref.Cache(-(-n // page), 1, page, dim, G or 32, bits, dtype)
    slots = np.arange(n)
    for name, x in (("k", k), ("v", v)):
        xb, xv = kv_ref.to_bits(x, dtype)
        if bits == 16:
            cache.parts[name][0][slots // page, 0, slots % page] = xb
        else:
            for part, got in zip(cache.parts[name], oracle.quantize(xv.astype(np.float32), G, bits)):
                part[slots // page, 0, slots % page] = got
    return cache, np.arange(-(-n // page), dtype=np.int32)[None]


@pytest.mark.parametrize("ahead", [9, 18])
@pytest.mark.parametrize("bits,G,dim,dtype", [(4, 32, 64, "bf16"), (8, 64, 128, "bf16"), (8, 128, 256, "bf16"),
                                              (16, 0, 128, "f16"), (16, 0, 64, "bf16")])
def test_many_small_weights_beside_one_large(aq, bits, G, dim, dtype, ahead):
    """One token whose value is 0 takes nearly all of the softmax, e^18 times
    the weight of each other: the result is what the others add."""
    n = 2500
    rng = np.random.default_rng(71)
    qb, q = _queries(72, (1, 1, 4, dim), dtype)
    k = 0.02 * rng.standard_normal((n, dim))
    v = rng.random((n, dim))
    q[0, 0, :] = q[0, 0, 0]  # all heads look the same way
    qb[0, 0, :] = qb[0, 0, 0]
    k[700] = q[0, 0, 0] * ahead / (dim ** -0.5 * (q[0, 0, 0] ** 2).sum())
    v[700] = 0
    cache, table = _one_head(bits, dtype, G, dim, k, v)
    _check(_attend(aq, cache, table, [n], qb, dtype, G), q, cache, table, [n], dtype)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("size", [3e-4, 3e-3, 300.0, 6e4])
def test_scales_of_any_size(aq, bits, size):
    """Scales of values, given and not made by the quantizer, up to fp16's
    largest and down among its subnormals; scores that spread over e^10."""
    n, dim, G = 300, 128, 64
    rng = np.random.default_rng(73)
    qb, q = _queries(74, (1, 2, 4, dim), "bf16", 3.0)
    cache, table = _one_head(bits, "bf16", G, dim, rng.standard_normal((n, dim)), np.ones((n, dim)))
    codes, scales, biases = cache.parts["v"]
    codes[:] = rng.integers(0, 1 << 32, codes.shape, dtype=np.uint32)
    scales[:] = (size * rng.uniform(0.01, 1, scales.shape)).astype(np.float16).view(np.uint16)
    biases[:] = (size * rng.uniform(-1, 1, biases.shape)).astype(np.float16).view(np.uint16)
    _check(_attend(aq, cache, table, [n], qb, "bf16", G), q, cache, table, [n], "bf16")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bits,G,dim", [(4, 64, 128), (8, 32, 64), (8, 64, 128), (8, 128, 256)])
def test_keys_far_from_zero(aq, bits, G, dim, dtype):
    """Keys that lie 100 to either side of zero, queries whose groups add up to
    little: the scores are what remains when the biases' large parts cancel."""
    n = 200
    rng = np.random.default_rng(91)
    x = 3 * rng.standard_normal((1, 2, 4, dim // G, G))
    x[..., -1] = -x[..., :-1].sum(-1)
    qb, q = kv_ref.to_bits(x.reshape(1, 2, 4, dim), dtype)
    k = rng.standard_normal((n, dim)) + np.where(rng.random((n, dim // G)) < 0.5, 100, -100).repeat(G, 1)
    cache, table = _one_head(bits, dtype, G, dim, k, rng.standard_normal((n, dim)))
    _check(_attend(aq, cache, table, [n], qb, dtype, G), q, cache, table, [n], dtype)


# ---- no tokens at all -------------------------------------------------------------------
@pytest.mark.parametrize("B", [1, 3, 70, 300])
@pytest.mark.parametrize("pages", [4, 40])  # up to 128 tokens, and more
@pytest.mark.parametrize("per,dim,bits,G", [(4, 64, 8, 32), (16, 256, 4, 64), (4, 128, 16, 0)])
def test_every_sequence_empty(aq, per, dim, bits, G, pages, B):
    """As a graph is captured before any token is there: zero rows, and the
    workspace serves the next call, with tables joined either way."""
    import torch
    cache = kv_ref.Cache(8, 1, 32, dim, G or 32, bits, "f16")
    cache.poison()
    table = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    parts = cache.device()
    for L in (1, 5):
        q = torch.ones((B, L, per, dim), dtype=torch.float16, device="cuda")
        out = torch.full_like(q, 7.0)
        aq.aq_paged_attention(q, *parts, table, lengths, G, bits, out=out, workspace=ws)
        assert not out.any()
    full = [700, 0, 31]
    cache, table = _build(full, 1, dim, G, bits, 32, "f16", seed=95)
    qb, q = _queries(96, (3, 1, per, dim), "f16")
    _check(_attend(aq, cache, table, full, qb, "f16", G, workspace=ws), q, cache, table, full, "f16")


# ---- queries of any size ----------------------------------------------------------------
@pytest.mark.parametrize("size", [1e8, 1e28, 3e33, 1e36])
@pytest.mark.parametrize("per", [4, 20])
@pytest.mark.parametrize("bits,G", [(4, 32), (8, 64), (16, 0)])
def test_large_queries(aq, bits, G, per, size):
    """bf16 queries far past fp16's range, scores within binary32's: one token
    takes all.  In every other head ordinary queries."""
    n, dim = 200, 128
    rng = np.random.default_rng(97)
    x = rng.standard_normal((1, 1, per, dim))
    x[:, :, ::2] *= size
    qb, q = kv_ref.to_bits(x, "bf16")
    cache, table = _one_head(bits, "bf16", G, dim, rng.standard_normal((n, dim)), rng.standard_normal((n, dim)))
    got = out_to_f64(_attend(aq, cache, table, [n], qb, "bf16", G))
    ref, slack = kv_ref.attention_rows(q, cache, table, [n], dim ** -0.5)
    # (the formula's weights of 0 and 1 leave no room for errors of the scores)
    slack[:, :, ::2] = 2.0 ** -14 * np.linalg.norm(ref[:, :, ::2], axis=-1)
    assert np.isfinite(got).all()
    assert kv_ref.rows_off(got, ref, slack, "bf16") <= 1


# ---- arguments --------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [8, 16])
def test_arrays_of_one_cache_have_its_shape(aq, bits):
    """As many elements in another shape are another cache's."""
    import torch
    parts = kv_ref.Cache(4, 2, 16, 64, 32, bits).device()
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    aq.aq_kv_read(slots, *parts, 32, bits)
    for i, t in enumerate(parts):
        if t is not None:
            pages, heads, page, last = t.shape
            for other in ((heads, pages, page, last), (pages * heads, 1, page, last), (pages, heads, page * last)):
                wrong = list(parts)
                wrong[i] = t.view(other)
                with pytest.raises(ValueError):
                    aq.aq_kv_read(slots, *wrong, 32, bits)


# ---- every form, within bounds that refuse other results --------------------------------
# bits, head size, group size, rows a key head (query heads, new tokens): one tile of
# columns, two, several slices
FORMS = [(bits, dim, G, per, L) for bits in (4, 8) for dim in (64, 128, 256) for G in (32, 64, 128)
         if G <= dim for per, L in ((3, 1), (5, 5))]
FORMS += [(16, dim, 0, per, L) for dim in (64, 128, 256) for per, L in ((3, 1), (5, 5))]
FORMS += [(8, 128, 128, 9, 8), (4, 64, 32, 33, 2), (8, 256, 128, 2, 8), (16, 128, 0, 9, 8)]
FORM_LENGTHS = [1, 31, 33, 129, 0, 400, 16]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bits,dim,G,per,L", FORMS)
def test_every_form(aq, bits, dim, G, per, L, dtype):
    _compare(aq, FORM_LENGTHS, per, 2, dim, G, bits, 32, L, dtype, seed=dim + L)


@pytest.mark.parametrize("lengths,per,heads,dim,G,bits,page,L,dtype", CASES + LONG)
def test_rows_of_long_and_short_sequences(aq, lengths, per, heads, dim, G, bits, page, L, dtype):
    _compare(aq, lengths, per, heads, dim, G, bits, page, L, dtype)
