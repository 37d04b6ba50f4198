"""The calls around the cache at the ends of their ranges: caps and values far
from one, what a row does not see, rows past 31 bits, every share of the key
heads among the waves."""
import numpy as np
import pytest

from gpu_util import to_dev
from test_gpu_attention import _queries
from test_gpu_kv import _build, _dev16, aq  # noqa: F401  (aq: the module's fixture)
from test_gpu_scores import _check_prompt

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
