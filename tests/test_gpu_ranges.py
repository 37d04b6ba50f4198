"""The calls around the cache at the ends of their ranges: caps and values far
from one, what a row does not see, rows past 31 bits, every share of the key
heads among the waves."""
import numpy as np
import pytest

import kv_ref
from gpu_util import out_bits, out_to_f64, to_dev
from test_gpu_attention import _queries
from test_gpu_kv import _build, _dev16, aq  # noqa: F401  (aq: the module's fixture)
from test_gpu_scores import _check_prompt, _paged, _prompt

pytestmark = pytest.mark.gpu


# ---- caps -------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,D,cap,scale", [
    ("f16", 128, 1e4, None), ("bf16", 128, 3e4, None), ("bf16", 64, 1e5, None), ("bf16", 128, 1e5, None),
    ("bf16", 256, 1e5, None), ("bf16", 128, 1e6, None), ("bf16", 64, 4e6, None), ("f16", 128, 50.0, 1e-4),
    ("bf16", 128, 50.0, 1e-5), ("f16", 128, 1e3, None), ("f16", 64, 50.0, 1e-3), ("f16", 256, 1e-4, None)])
def test_scores_near_caps_of_any_size(aq, dtype, D, cap, scale):
    """Scores of 0.13 of the cap times a normal variable, so up to 0.6 of it, in
    tiles that all rows see and in those that only some do."""
    size = 0.13 * cap if scale is None else 0.13 * cap / (scale * D ** 0.5)
    _check_prompt(aq, [150], [200], 2, 1, D, dtype, seed=D, softcap=cap, scale=scale, size=size)


# ---- gathered weights -------------------------------------------------------------------
@pytest.mark.parametrize("bits,G", [(4, 64), (8, 64), (16, 0)])
@pytest.mark.parametrize("odd", ["query", "key"])
def test_weights_of_tokens_that_other_rows_see(aq, bits, G, odd):
    """80 rows of one key head in three slices, the last with 16 columns to
    spare; its tile of the tokens 32 .. 63 is one that all of its rows see, the
    first row does not.  A query that is NaN, or a key and a query that give the
    first row alone a NaN, stay with the tokens of that row."""
    import torch
    n, L, per, dim = 64, 5, 16, 128
    cache, table = _build([n], 1, dim, G, bits, 16, "f16", seed=41)
    qb, _ = _queries(42, (1, L, per, dim), "f16")
    if odd == "query":
        qb[0, 0, 0, 7] = 0x7E00
    elif bits == 16:
        qb[0, :, :, 7], qb[0, 0, 0, 7] = 0xBC00, 0  # -1, and 0 that meets the infinite key
        cache.parts["k"][0][table[0, 3], 0, 60 - 48, 7] = 0x7C00
    else:
        pytest.skip("codes are finite")
    q, tab, lens = _dev16(qb, "f16"), to_dev(table), torch.tensor([n], dtype=torch.int32, device="cuda")
    parts, w = cache.device(), torch.zeros((1, n), device="cuda")
    _, lse = aq.aq_paged_attention_masked(q, *parts, tab, lens, G or 32, bits, return_lse=True)
    none = np.isnan(lse.cpu().numpy()[0])
    aq.aq_kv_weigh(q, lse, *parts, tab, lens, w, G or 32, bits)
    w = w.cpu().numpy()[0]
    if odd == "query":  # row 0 of token 0, which sees the tokens up to 59
        assert none[0, 0] and none.sum() == 1
        assert np.isnan(w[:60]).all() and np.isfinite(w[60:]).all() and (w[60:] > 0).all()
    else:  # the first row does not see token 60, to the others its score is -inf
        assert not none.any() and np.isfinite(w).all()
        assert w[60] == 0 and (np.delete(w, 60) > 0).all()


def test_rows_without_a_logarithm_add_nothing(aq):
    """A row whose lse is -inf adds nothing, whatever its query holds."""
    import torch
    cache, table = _build([100], 1, 64, 32, 8, 16, "f16", seed=43)
    qb, _ = _queries(44, (1, 1, 4, 64), "f16")
    tab, lens = to_dev(table), torch.tensor([100], dtype=torch.int32, device="cuda")
    parts = cache.device()
    _, lse = aq.aq_paged_attention_masked(_dev16(qb, "f16"), *parts, tab, lens, 32, 8, return_lse=True)
    lse[0, 0, 2] = -np.inf
    got = []
    for bad in (0x3C00, 0x7E00):
        qb[0, 0, 2] = bad
        w = torch.zeros((1, 112), device="cuda")
        aq.aq_kv_weigh(_dev16(qb, "f16"), lse, *parts, tab, lens, w, 32, 8)
        got.append(w)
    assert torch.equal(*got) and abs(float(got[0].sum()) - 3) < 1e-4


# ---- values near binary32's ends --------------------------------------------------------
@pytest.mark.parametrize("n,past,window", [([1], [0], 0), ([150, 1, 33], [30, 0, 200], 0), ([150], [200], 1),
                                           ([20], [3000], 0), ([90], [3000], 0)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_values_of_prompts(aq, D, n, past, window):
    """bf16 values around 1e36, and of one sign near the type's largest: sums of
    weights and values stay within binary32 where the result does."""
    rng = np.random.default_rng(D)
    keys = sum(n) + sum(past)
    k, v = rng.standard_normal((keys, 1, D)), rng.standard_normal((keys, 1, D))
    for x in (v * 1e36, 3.3e38 * (1 - rng.random(v.shape) / 16)):
        _check_prompt(aq, n, past, 2, 1, D, "bf16", seed=D, k=k, v=x, window=window)


@pytest.mark.parametrize("power", [-60, 100, 121])
def test_results_scale_with_the_values_of_prompts(aq, power):
    """Values times a power of two give the same results times it."""
    rng = np.random.default_rng(9)
    k, v = rng.standard_normal((350, 1, 128)), rng.standard_normal((350, 1, 128))
    a, b = (_prompt(aq, [150], [200], 2, 1, 128, "bf16", seed=3, k=k, v=x, softcap=20.0)[0]
            for x in (v, v * 2.0 ** power))
    assert np.array_equal(a * 2.0 ** power, b)


def test_scores_past_where_weights_have_room(aq):
    """Scores past 2^23 in powers of two that fall by 8 from tile to tile: what
    was summed is not raised as they fall."""
    n, D = 700, 64
    q = np.random.default_rng(4).standard_normal((1, 1, D))  # what _prompt makes of seed 4
    q0, q1 = (float(x) for x in kv_ref.to_bits(q, "bf16")[1][0, 0, :2])
    to_power = D ** 0.5 * np.log(2)
    k = np.zeros((n + 1, 1, D))
    k[:, 0, 0] = 1.2e7 * to_power / q0
    k[:, 0, 1] = -8 * to_power / q1 * (np.arange(n + 1) // 64)
    v = 1e36 * np.random.default_rng(5).standard_normal((n + 1, 1, D))
    got, lse, _ = _prompt(aq, [1], [n], 1, 1, D, "bf16", seed=4, k=k, v=v)
    assert np.isfinite(got).all() and np.abs(got).max() <= np.abs(v[:192]).max()
    assert lse.min() > 2.0 ** 23 * np.log(2)


@pytest.mark.parametrize("lengths,L,per,dim", [([1, 300, 33], 1, 4, 128), ([2500], 2, 2, 64), ([700], 5, 8, 256)])
@pytest.mark.parametrize("power", [-60, 100, 121])
def test_results_scale_with_the_values_of_pages(aq, power, lengths, L, per, dim):
    """bf16 pages whose values are those of another cache times a power of two: the
    same results times it, where sums of weights and values pass binary32
    unless the weights leave room too."""
    import torch
    got = []
    for times in (0, power):
        cache, table = _build(lengths, 1, dim, 0, 16, 16, "bf16", seed=51, poison=False)
        v = cache.parts["v"][0]
        v &= 0x7FFF  # (of one sign)
        v[:] = np.where(v & 0x7F80, v + (times << 7 & 0xFFFF), v).astype(np.uint16)
        qb, _ = _queries(52, (len(lengths), L, per, dim), "bf16", 0.3)
        args = (_dev16(qb, "bf16"), *cache.device(), to_dev(table), to_dev(np.array(lengths, np.int32)), 32, 16)
        got.append([out_to_f64(aq.aq_paged_attention(*args)), out_to_f64(aq.aq_paged_attention_masked(*args, softcap=9.0))])
    for a, b in zip(*got):
        assert np.isfinite(b).all() and np.array_equal(a * 2.0 ** power, b)


# ---- what a row does not see ------------------------------------------------------------
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("L,per,dim,window", [(1, 4, 128, 20), (4, 5, 64, 20), (3, 2, 256, 33), (8, 8, 128, 5)])
def test_scales_that_no_row_sees(aq, bits, L, per, dim, window):
    """Packed pages: scales and biases of tokens before the window, large,
    infinite or NaN, leave all results as they are to the last bit."""
    lengths = [100, 70]
    qb, _ = _queries(61, (2, L, per * 2, dim), "f16")
    lens, got = to_dev(np.array(lengths, np.int32)), []
    for odd in (None, 0x7BFF, 0x7C00, 0x7E00):
        cache, table = _build(lengths, 2, dim, 32, bits, 16, "f16", seed=L + dim)
        if odd:
            for b, n in enumerate(lengths):
                for t in range(max(0, n - L - window - 30), n - L - window + 1):
                    for part in (1, 2):
                        cache.parts["k"][part][table[b, t // 16], :, t % 16] = odd
                        cache.parts["v"][part][table[b, t // 16], :, t % 16] = odd
        out, lse = aq.aq_paged_attention_masked(_dev16(qb, "f16"), *cache.device(), to_dev(table), lens, 32, bits,
                                                window=window, return_lse=True)
        got.append((out_bits(out), out_bits(lse)))
    for out, lse in got[1:]:
        assert np.array_equal(out, got[0][0]) and np.array_equal(lse, got[0][1])


# ---- shares of the work -----------------------------------------------------------------
@pytest.mark.parametrize("bits,G", [(4, 64), (8, 64), (16, 0)])
@pytest.mark.parametrize("heads", [3, 4, 5, 7, 8, 9, 16])
def test_any_number_of_key_heads(aq, bits, G, heads):
    """Key heads go to eight, four, two or one of a workgroup's waves, and round
    again where there are more; strips of 512 tokens are used again."""
    _paged(aq, [700, 1, 0, 1333], 4, heads, 64, G and 32, bits, 16, 1, "f16", seed=heads, window=1200)
    _paged(aq, [577, 90], 9, heads, 128, G, bits, 48, 5, "bf16", seed=heads + 1, softcap=20.0, slopes=True)


def test_many_tokens_of_many_key_heads(aq):
    """Chunks of one sequence over the whole chip."""
    _paged(aq, [20011], 2, 5, 64, 64, 8, 64, 1, "f16", seed=71)
    _paged(aq, [9001, 12000], 3, 8, 64, 32, 4, 16, 2, "f16", seed=72, first=[17, 2300])


# ---- rows past 31 bits ------------------------------------------------------------------
@pytest.fixture(scope="module")
def vast():
    """One array for keys and values (4 bits, 69 GB of codes) of more than 2^31 rows."""
    import torch
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 77 GB of device memory")
    H, D, G, page = 8, 64, 64, 64
    pages = (1 << 31) // (H * page) + 9
    part = [torch.empty((pages, H, page, D // 8), dtype=torch.int32, device="cuda")]
    part += [torch.empty((pages, H, page, 1), dtype=torch.float16, device="cuda") for _ in range(2)]
    yield part, pages, H, D, G, page
    part.clear()
    torch.cuda.empty_cache()


def test_turned_keys_of_more_rows_than_31_bits(aq, vast):
    import torch
    part, pages, H, D, G, page = vast
    T, ids = 150, torch.tensor([pages - 1, 3, pages - 3], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(81)
    k = torch.randn((T, H, D), generator=gen, device="cuda").half()
    positions = torch.randint(0, 1 << 20, (T,), generator=gen, device="cuda", dtype=torch.int32)
    freqs, _ = aq.aq_rope_frequencies(D)
    t = torch.arange(T, device="cuda")
    small = kv_ref.Cache(3, H, page, D, G, 4).device()
    turned = aq.aq_rope(None, k, positions, freqs)[1]
    aq.aq_kv_append(turned, turned, t, *small, G, 4)
    # keys turned and values that are the same rows: both writes leave the same bits
    far = ids[t // page] * page + t % page
    out = torch.empty_like(k)
    aq.aq_rope_append(None, k, turned, positions, freqs, far, *part, *part, G, 4, k_out=out)
    assert torch.equal(out, turned)
    at = (t // page, slice(None), t % page)
    for x, y in zip(part, small):
        assert torch.equal(x[ids][at].view(torch.int16), y[at].view(torch.int16))


def test_rows_that_move_past_31_bits(aq, vast):
    import torch
    part, pages, H, D, G, page = vast
    old = torch.tensor([[pages - 1, 2, pages - 4], [pages - 2, pages - 6, 5]], dtype=torch.int32, device="cuda")
    new = torch.tensor([[7, pages - 7], [pages - 8, 9]], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(82)
    for x in part:
        y = torch.randint(-2 ** 15, 2 ** 15, (6, *x.shape[1:]), generator=gen, device="cuda")
        x[old.flatten().long()] = y.to(torch.int16).view(torch.float16) if x.dtype == torch.float16 else y.int()
    weights = torch.rand((2, 3 * page), generator=gen, device="cuda")
    lengths = torch.tensor([3 * page - 1, 2 * page + 5], dtype=torch.int32, device="cuda")
    kept, _, _ = aq.aq_kv_evict(weights, lengths, old, new, *part, *part, G, 4, keep=100, sinks=3, recent=9)
    to = torch.arange(100, device="cuda")
    for b in range(2):
        at = kept[b].long()
        for x in part:
            moved = x[new[b].long()][to // page, :, to % page]
            assert torch.equal(moved.view(torch.int16), x[old[b].long()][at // page, :, at % page].view(torch.int16))


# ---- scores that are not finite ---------------------------------------------------------
def test_infinite_scores(aq):
    """A score of +inf leaves no sum: the rows that see it are NaN, their
    logarithms too, and no others; -inf is a weight of 0; a cap bounds both."""
    import torch
    n, dim = 90, 64
    gen = torch.Generator(device="cuda").manual_seed(91)
    q, k, v = (torch.randn((n, 1, dim), generator=gen, device="cuda").half() for _ in range(3))
    k[40, 0, 7] = np.inf
    q[:, 0, 7] = 1.0
    st = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pages = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    cache = kv_ref.Cache(6, 1, 16, dim, 32, 16, "f16").device()
    aq.aq_kv_append(k, v, torch.arange(n, device="cuda"), *cache, 32, 16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")

    def both(q, **more):
        out, lse = aq.aq_prompt_attention(q, k, v, st, st, return_lse=True, **more)
        one = aq.aq_paged_attention_masked(q[None, -3:], *cache, pages, lens, 32, 16, return_lse=True, **more)
        return out, lse, *one

    out, lse, o1, l1 = both(q)
    sees = torch.arange(n, device="cuda") >= 40
    assert out[sees].isnan().all() and out[~sees].isfinite().all() and o1.isnan().all()
    assert lse[sees].isnan().all() and lse[~sees].isfinite().all() and l1.isnan().all()
    q[:, 0, 7] = -1.0
    got = both(q)
    assert all(x.isfinite().all() for x in got)
    w = torch.zeros((1, 96), device="cuda")
    aq.aq_kv_weigh(q[None, -3:], got[3], *cache, pages, lens, w, 32, 16)
    assert w[0, 40] == 0 and abs(float(w.sum()) - 3) < 1e-4
    for sign in (1.0, -1.0):
        q[:, 0, 7] = sign
        assert all(x.isfinite().all() for x in both(q, softcap=5.0))
