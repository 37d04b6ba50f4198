"""The calls around the cache at the ends of their ranges: caps and values far
from one, what a row does not see, rows past 31 bits, every share of the key
heads among the waves."""
import numpy as np
import pytest

import kv_ref
from gpu_util import out_bits, out_to_f64, to_dev
from test_gpu_attention import _queries
from test_gpu_kv import _build, _dev16, aq  # noqa: F401  (aq: the module's fixture)
from test_gpu_scores import _check_prompt, _prompt

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
