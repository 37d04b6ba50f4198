"""Attention whose scores are capped, biased by distance and masked, of new
tokens over the paged cache and of prompts, and the weight that cached tokens
gather, on the GPU: rows by the norm of their error against the formula in
binary64 (scores_ref.py says how large it may be)."""
import numpy as np
import pytest

import kv_ref
import scores_ref
from gpu_util import out_bits, out_to_f64, to_dev
from test_gpu_attention import FORM_LENGTHS, FORMS, _queries, _set_value
from test_gpu_kv import CASES, _attend, _build, _dev16, aq  # noqa: F401  (aq: the module's fixture)

pytestmark = pytest.mark.gpu


def _device_scores(slopes, first):
    return {"slopes": None if slopes is None else to_dev(slopes.astype(np.float32)),
            "first": None if first is None else to_dev(np.array(first, np.int32))}


def _slopes(heads):
    return (2.0 ** (-8.0 * np.arange(1, heads + 1) / heads)).astype(np.float32).astype(np.float64)


def _paged(aq, lengths, per, heads, dim, G, bits, page, L, dtype, seed, softcap=0.0, slopes=False, window=0,
           first=None, scale=None, size=1.0):
    """Attention and gathered weights of one call, both compared."""
    import torch
    cache, table = _build(lengths, heads, dim, G, bits, page, dtype, seed=seed)
    B, Hq = len(lengths), per * heads
    qb, q = _queries(seed + 1, (B, L, Hq, dim), dtype, size)
    slopes = _slopes(Hq) if slopes else None
    more = dict(softcap=softcap, window=window, scale=scale, **_device_scores(slopes, first))
    parts, qd = cache.device(), _dev16(qb, dtype)
    tab, lens = to_dev(table), to_dev(np.array(lengths, np.int32))
    out, lse = aq.aq_paged_attention_masked(qd, *parts, tab, lens, G or 32, bits, return_lse=True, **more)
    scale = dim ** -0.5 if scale is None else scale
    ref, ref_lse, slack, lse_slack, gathered, may = scores_ref.paged(q, cache, table, lengths, scale, softcap,
                                                                     slopes, window, first)
    got = out_to_f64(out)
    assert np.isfinite(got).all()
    worst = kv_ref.rows_off(got, ref, slack, dtype)
    assert worst <= 1, f"worst row's error over its bound {worst:.3f}"
    worst = scores_ref.lse_off(lse.cpu().numpy().astype(np.float64), ref_lse, lse_slack)
    assert worst <= 1, f"worst logarithm over its bound {worst:.3f}"
    before = np.random.default_rng(seed + 2).random(gathered.shape).astype(np.float32)
    w = to_dev(before)
    aq.aq_kv_weigh(qd, lse, *parts, tab, lens, w, G or 32, bits, **more)
    w = w.cpu().numpy().astype(np.float64)
    off = np.abs(w - before - gathered) - may - 2.0 ** -24 * (before + gathered)
    assert off.max() <= 0, f"gathered weights off by {off.max():.3g} more than they may be"
    for b, n in enumerate(lengths):
        assert np.array_equal(w[b, max(n, 0):], before[b, max(n, 0):])
    return out, lse


# ---- new tokens over the cache ----------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bits,dim,G,per,L", FORMS)
def test_every_form(aq, bits, dim, G, per, L, dtype):
    _paged(aq, FORM_LENGTHS, per, 2, dim, G, bits, 32, L, dtype, seed=dim + L, softcap=5.0, slopes=True,
           window=150, first=[0, 3, 20, 33, 0, 270, 15])


@pytest.mark.parametrize("what", [dict(softcap=2.0), dict(softcap=50.0, size=20.0), dict(slopes=True),
                                  dict(window=1), dict(window=16), dict(window=33), dict(window=100000),
                                  dict(window=2 ** 31 - 1), dict(first=[0, 5, 300, 1, 64, 63, 2 ** 31 - 1]),
                                  dict(first=[-5, -2 ** 31, 0, 0, 0, 0, 0]), dict(softcap=1e-30),
                                  dict(softcap=1e30), dict(scale=-0.2), dict(scale=0.0),
                                  dict(slopes=True, softcap=10.0, window=40, first=[0, 1, 370, 2, 3, 4, 5])])
@pytest.mark.parametrize("bits,G,L,per", [(8, 64, 1, 4), (4, 32, 5, 5), (16, 0, 3, 2)])
def test_each_kind(aq, what, bits, G, L, per):
    lengths = [37, 5, 400, 1, 65, 128, 90]
    _paged(aq, lengths, per, 2, 128, G, bits, 16, L, "bf16", seed=3, **what)


def test_long_sequences_with_a_window(aq):
    """Units that begin far behind their first page, cut over many workgroups."""
    _paged(aq, [9000, 300, 12345], 4, 1, 64, 32, 8, 48, 2, "f16", seed=5, window=4000, slopes=True)
    _paged(aq, [20000], 4, 1, 128, 64, 4, 64, 1, "f16", seed=6, softcap=20.0, first=[7777])


@pytest.mark.parametrize("bits,G", [(8, 64), (16, 0)])
def test_without_any_it_is_the_plain_call(aq, bits, G):
    lengths = [100, 0, 37, 2000]
    cache, table = _build(lengths, 2, 128, G, bits, 16, "f16", seed=9)
    qb, _ = _queries(10, (4, 2, 8, 128), "f16")
    plain = _attend(aq, cache, table, lengths, qb, "f16", G or 32)
    out = aq.aq_paged_attention_masked(_dev16(qb, "f16"), *cache.device(), to_dev(table),
                                       to_dev(np.array(lengths, np.int32)), G or 32, bits)
    assert np.array_equal(out_bits(out), out_bits(plain))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("L,per,dim,window", [(1, 4, 128, 20), (4, 5, 64, 20), (3, 2, 256, 33), (8, 2, 128, 5)])
def test_odd_values_that_no_row_sees(aq, dtype, L, per, dim, window):
    """16-bit pages: values before the window, or newer than a row, that are not
    finite leave it as it is; keys too."""
    lengths = [100, 70]
    clean, table = _build(lengths, 2, dim, 0, 16, 16, dtype, seed=L + dim)
    dirty, _ = _build(lengths, 2, dim, 0, 16, 16, dtype, seed=L + dim)
    inf = {"f16": 0x7C00, "bf16": 0x7F80}[dtype]
    for b, n in enumerate(lengths):
        _set_value(dirty, table, b, n - L - window, 1, 0x7FFF)    # before what the oldest row sees
        _set_value(dirty, table, b, n - L - window - 3, 0, inf)
        dirty.parts["k"][0][table[b, 0], :, 2] = 0x7FFF
        dirty.parts["k"][0][table[b, 0], :, 3] = inf
    qb, _ = _queries(21, (2, L, per * 2, dim), dtype)
    lens = to_dev(np.array(lengths, np.int32))
    a, b = (aq.aq_paged_attention_masked(_dev16(qb, dtype), *c.device(), to_dev(table), lens, 32, 16,
                                         window=window, return_lse=True) for c in (clean, dirty))
    assert np.array_equal(out_bits(a[0]), out_bits(b[0])) and np.array_equal(out_bits(a[1]), out_bits(b[1]))
    # inside the window of some rows only: those that see it, and no others
    if L > 1:
        for b, n in enumerate(lengths):
            _set_value(dirty, table, b, n - L - window + 1, 1, 0x7FFF)  # the oldest row's last
        got = aq.aq_paged_attention_masked(_dev16(qb, dtype), *dirty.device(), to_dev(table), lens, 32, 16,
                                           window=window)
        got, want = out_to_f64(got), out_to_f64(a[0])
        assert np.isnan(got[:, 0, per:]).all()
        assert np.array_equal(got[:, 1:], want[:, 1:]) and np.array_equal(got[:, :, :per], want[:, :, :per])


@pytest.mark.parametrize("B", [1, 70])
def test_empty_sequences(aq, B):
    import torch
    cache = kv_ref.Cache(8, 1, 32, 64, 32, 8, "f16")
    cache.poison()
    table = torch.full((B, 40), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.ones((B, 3, 4, 64), dtype=torch.float16, device="cuda")
    out, lse = aq.aq_paged_attention_masked(q, *cache.device(), table, lengths, 32, 8, window=9, return_lse=True)
    assert not out.any() and (lse == -np.inf).all()
    w = torch.ones((B, 1280), device="cuda")
    aq.aq_kv_weigh(q, lse, *cache.device(), table, lengths, w, 32, 8, window=9)
    assert (w == 1).all()


def test_gathered_weights_of_few_tokens_of_a_row(aq):
    """Fewer weights than tokens: the others are not looked for."""
    import torch
    lengths = [100, 30]
    cache, table = _build(lengths, 1, 64, 32, 8, 16, "f16", seed=31)
    qb, _ = _queries(32, (2, 1, 4, 64), "f16")
    lens, q = to_dev(np.array(lengths, np.int32)), _dev16(qb, "f16")
    _, lse = aq.aq_paged_attention_masked(q, *cache.device(), to_dev(table), lens, 32, 8, return_lse=True)
    full, part = torch.zeros((2, 112), device="cuda"), torch.zeros((2, 52), device="cuda")
    for w in (full, part):
        aq.aq_kv_weigh(q, lse, *cache.device(), to_dev(table), lens, w, 32, 8)
    assert torch.equal(full[:, :52], part)
    assert abs(float(full.sum()) - 8) < 1e-4  # every row gives one


# ---- prompts ----------------------------------------------------------------------------
def _prompt(aq, n, past, Hq, H, D, dtype, seed=0, softcap=0.0, slopes=False, window=0, first=None, prefix=None,
            scale=None, extra=0, size=1.0, k=None, v=None):
    """Sequences of n[b] new tokens after past[b]; `extra` rows behind the last."""
    import torch
    rng = np.random.default_rng(seed)
    qs, ks = (np.cumsum([0] + list(x)).astype(np.int32) for x in (n, np.array(n) + past))
    Tq, Tk = qs[-1] + extra, ks[-1] + extra
    qb, qx = kv_ref.to_bits(size * rng.standard_normal((Tq, Hq, D)), dtype)
    kx, vx = (rng.standard_normal((Tk, H, D)) if x is None else x for x in (k, v))
    (kb, kx), (vb, vx) = (kv_ref.to_bits(x, dtype) for x in (kx, vx))
    wide = torch.zeros((Tk, 2 * H * D + 8), dtype=_dev16(kb, dtype).dtype, device="cuda")
    kd, vd = (wide[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)).copy_(_dev16(x, dtype))
              for i, x in enumerate((kb, vb)))
    sl = _slopes(Hq) if slopes else None
    more = dict(softcap=softcap, window=window, scale=scale, **_device_scores(sl, first),
                prefix=None if prefix is None else to_dev(np.array(prefix, np.int32)))
    out = torch.full((Tq, Hq, D), 7.0, dtype=kd.dtype, device="cuda")
    lse = torch.full((Tq, Hq), 7.0, device="cuda")
    call = lambda **o: aq.aq_prompt_attention(_dev16(qb, dtype), kd, vd, to_dev(qs), to_dev(ks), **more, **o)  # noqa: E731
    call(out=out, lse=lse)
    last = qs[-1]
    assert (out[last:] == 7).all() and (lse[last:] == 7).all()
    again = call()
    assert np.array_equal(out_bits(again[:last]), out_bits(out[:last]))
    ref = scores_ref.prompt(qx, kx, vx, qs, ks, D ** -0.5 if scale is None else scale, dtype, softcap, sl, window,
                            first, prefix)
    return out_to_f64(out)[:last], lse.cpu().numpy().astype(np.float64)[:last], [r[:last] for r in ref]


def _check_prompt(aq, n, past, Hq, H, D, dtype, **more):
    got, lse, (ref, ref_lse, slack, lse_slack) = _prompt(aq, n, past, Hq, H, D, dtype, **more)
    assert np.isfinite(got).all()
    worst = kv_ref.rows_off(got, ref, slack, dtype)
    assert worst <= 1, f"worst row's error over its bound {worst:.3f}"
    worst = scores_ref.lse_off(lse, ref_lse, lse_slack)
    assert worst <= 1, f"worst logarithm over its bound {worst:.3f}"


PROMPTS = [  # new tokens, tokens before them, query heads, key heads, dim
    ([1], [0], 1, 1, 64), ([1], [300], 8, 2, 128), ([2, 1, 5], [0, 64, 63], 4, 4, 256), ([61], [0], 8, 4, 64),
    ([33, 64, 65, 31], [0, 0, 0, 0], 4, 1, 128), ([100, 0, 7], [50, 20, 0], 10, 2, 64),
    ([257], [130], 5, 1, 128), ([300], [0], 2, 2, 256), ([129], [1], 16, 2, 256), ([3] * 70, [5] * 70, 2, 1, 64)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,past,Hq,H,D", PROMPTS)
def test_prompts(aq, n, past, Hq, H, D, dtype):
    _check_prompt(aq, n, past, Hq, H, D, dtype, seed=sum(n) + D, extra=3)


@pytest.mark.parametrize("what", [
    dict(softcap=3.0), dict(softcap=50.0, size=20.0), dict(slopes=True), dict(window=1), dict(window=50),
    dict(window=2 ** 31 - 1), dict(prefix=[40, 0, 1000]), dict(prefix=[-3, 64, 65], slopes=True),
    dict(first="documents"), dict(first="documents", prefix=[90, 30, 100], window=70, slopes=True, softcap=8.0),
    dict(scale=-0.1), dict(scale=0.0), dict(first="past"), dict(softcap=1e-30), dict(softcap=1e30)])
@pytest.mark.parametrize("Hq,H,D,dtype", [(8, 2, 128, "bf16"), (3, 1, 64, "f16"), (2, 2, 256, "f16")])
def test_kinds_of_prompts(aq, what, Hq, H, D, dtype):
    n, past = [150, 33, 70], [0, 90, 10]
    what = dict(what)
    if what.get("first") == "documents":
        rng = np.random.default_rng(1)
        what["first"] = np.concatenate([np.repeat(sorted([0, *rng.integers(0, m + p, 3)]),
                                                  np.diff(sorted([0, *rng.integers(0, m, 3), m])))
                                        for m, p in zip(n, past)])
    elif what.get("first") == "past":
        what["first"] = np.full(sum(n), 2 ** 31 - 1)  # no row sees anything
    _check_prompt(aq, n, past, Hq, H, D, dtype, seed=17, **what)


@pytest.mark.parametrize("n,past,Hq,H,D", [([2], [9000], 4, 1, 128), ([40], [5000], 4, 2, 64), ([5], [4000], 8, 1, 256),
                                           ([1, 3], [7000, 2000], 2, 1, 128), ([300], [4200], 1, 1, 64)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_few_rows_and_many_keys(aq, n, past, Hq, H, D, dtype):
    """Keys cut into parts, joined by a second launch; rows that see only one part."""
    _check_prompt(aq, n, past, Hq, H, D, dtype, seed=D)
    _check_prompt(aq, n, past, Hq, H, D, dtype, seed=D + 1, window=700, slopes=True, softcap=20.0)


def test_queries_without_keys_before_them(aq):
    """More queries than keys: the first ones stand before every token."""
    _check_prompt(aq, [50, 4], [-30, -4], 4, 2, 64, "f16", seed=2)


@pytest.mark.parametrize("D,Hq,H", [(64, 4, 1), (128, 4, 2), (256, 2, 1)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_odd_values_in_prompts(aq, dtype, D, Hq, H):
    """Infinite and NaN values reach the rows that see them, and no others, in
    tiles that all rows see and in those that only some do; keys as well."""
    n, past = [150, 40], [30, 0]
    rng = np.random.default_rng(8)
    k, v = rng.standard_normal((220, H, D)), rng.standard_normal((220, H, D))
    clean, lse0, (ref, *_) = _prompt(aq, n, past, Hq, H, D, dtype, seed=8, k=k, v=v, window=100)
    v[3, 0, 5], v[70, 0, 6], v[71, 0, 6], v[100, 0, 7] = np.inf, np.inf, -np.inf, np.nan
    v[179, 0, 8], v[180, 0, 9], v[219, 0, 10] = -np.inf, np.inf, np.nan
    got, lse, _ = _prompt(aq, n, past, Hq, H, D, dtype, seed=8, k=k, v=v, window=100)
    want = clean.copy()
    group = Hq // H
    for t, d, x in ((3, 5, np.inf), (70, 6, np.inf), (71, 6, -np.inf), (100, 7, np.nan), (179, 8, -np.inf),
                    (180, 9, np.inf), (219, 10, np.nan)):
        for row in range(190):
            b = row >= 150
            pos, at = (row - 150, t - 180) if b else (row + 30, t)
            if 0 <= at <= pos and pos - at < 100:
                want[row, :group, d] = x if np.isfinite(want[row, :group, d]).all() or x != x else np.nan
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(lse, lse0)
    k[50, 0, 0] = np.nan
    got, _, _ = _prompt(aq, n, past, Hq, H, D, dtype, seed=8, k=k, v=rng.standard_normal((220, H, D)), window=100)
    pos = np.arange(150) + 30
    sees = np.concatenate([(pos >= 50) & (pos - 50 < 100), np.zeros(40, bool)])
    assert np.isnan(got[sees][:, :group]).all() and np.isfinite(got[~sees]).all()
    assert np.isfinite(got[:, group:]).all()


@pytest.mark.parametrize("n,Hq", [(20, 2), (90, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_keys_in_parts(aq, n, Hq, D):
    """Keys cut into parts for workgroups of two and of four waves; infinite and NaN values in the
    first, an inner and the last tile of a part, seen by all rows, by some and by none."""
    past, window = 3000, 2990
    rng = np.random.default_rng(D + n)
    k, v = rng.standard_normal((past + n, 1, D)), rng.standard_normal((past + n, 1, D))
    _check_prompt(aq, [n], [past], Hq, 1, D, "f16", seed=9, k=k, v=v, softcap=30.0)
    clean, lse0, _ = _prompt(aq, [n], [past], Hq, 1, D, "f16", seed=9, k=k, v=v, window=window)
    odd = [(0, 1, np.nan), (12, 5, np.inf), (511, 6, -np.inf), (512, 7, np.inf), (1700, 8, np.nan),
           (past, 9, np.inf), (past + n - 1, 10, -np.inf)]
    for t, d, x in odd:
        v[t, 0, d] = x
    got, lse, _ = _prompt(aq, [n], [past], Hq, 1, D, "f16", seed=9, k=k, v=v, window=window)
    want = clean.copy()
    for t, d, x in odd:
        for row in range(n):
            if t <= past + row and past + row - t < window:
                want[row, :, d] = x
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(lse, lse0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_small_weights_beside_a_large_one(aq, dtype):
    """One token whose value is 0 takes nearly all of the softmax."""
    n, D = 600, 64
    rng = np.random.default_rng(71)
    k, v = 0.02 * rng.standard_normal((n, 1, D)), rng.random((n, 1, D))
    q = np.random.default_rng(4).standard_normal((n, 1, D))  # what _prompt makes of seed 4
    k[100, 0] = q[-1, 0] * 14 / (D ** -0.5 * (q[-1, 0] ** 2).sum())
    v[100] = 0
    _check_prompt(aq, [n], [0], 1, 1, D, dtype, seed=4, k=k, v=v)


def test_large_queries(aq):
    """bf16 queries far past fp16's range: one token takes all."""
    got, _, (ref, _, _, _) = _prompt(aq, [90], [0], 2, 1, 128, "bf16", seed=6, size=1e30)
    assert np.isfinite(got).all()
    off = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert off.max() < 2.0 ** -8


def test_starts_that_are_clamped(aq):
    """Starts past the rows, or descending, read and write nothing outside."""
    import torch
    q, k = (torch.randn((20, 2, 64), device="cuda").half() for _ in range(2))
    starts = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    want = aq.aq_prompt_attention(q, k, k, starts(0, 20), starts(0, 20))
    got = aq.aq_prompt_attention(q, k, k, starts(-5, 1 << 30), starts(-5, 1 << 30))
    assert torch.equal(want, got)
    out = torch.full_like(q, 7.0)
    aq.aq_prompt_attention(q, k, k, starts(15, 3, 3), starts(0, 9, 4), out=out)
    assert (out == 7).all()


def test_refusals(aq):
    import torch
    q, k = torch.zeros((4, 4, 64), dtype=torch.float16, device="cuda"), torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda")
    st = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    aq.aq_prompt_attention(q, k, k, st, st)
    for bad in (dict(q=q.bfloat16()), dict(v=k[:3]), dict(k_starts=st[:1]), dict(first=st), dict(prefix=st),
                dict(slopes=torch.zeros(3, device="cuda")), dict(out=k), dict(q=q.cpu()),
                dict(lse=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            aq.aq_prompt_attention(**{**dict(q=q, k=k, v=k, q_starts=st, k_starts=st), **bad})
    for bad in (dict(q_starts=st.long()), dict(first=torch.zeros(4, device="cuda"))):
        with pytest.raises(TypeError):
            aq.aq_prompt_attention(**{**dict(q=q, k=k, v=k, q_starts=st, k_starts=st), **bad})
    for bad in (dict(window=-1), dict(softcap=-2.0), dict(workspace=torch.zeros(0, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(aq.AQError):
            aq.aq_prompt_attention(q, k, k, st, st, **bad)
