"""Attention over the paged cache where its values are unusual: infinities and
NaN that some rows see and others do not, scales and scores far from one,
batches without a token, every form of the kernel.  Rows are compared by the
norm of their error, kv_ref.attention_rows says how large that may be."""
import numpy as np
import pytest

import kv_ref
import oracle
from gpu_util import out_to_f64
from test_gpu_kv import _attend, _build, _dev16, aq  # noqa: F401  (aq: the module's fixture)

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
