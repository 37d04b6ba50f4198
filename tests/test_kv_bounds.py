"""What the comparison of attention's rows (kv_ref.attention_rows, rows_off)
refuses, in every case that the GPU tests compare: results of zero, equal
weights, the newest token or a piece of the sequence left out, a piece joined
with another weight.  And what it has to accept: the formula in binary32."""
import numpy as np
import pytest

import kv_ref
import test_gpu_attention as gpu
from test_gpu_kv import CASES, LONG, _build

EVERY = CASES + LONG + [(gpu.FORM_LENGTHS, per, 2, dim, G, bits, 32, L, dtype)
                        for bits, dim, G, per, L in gpu.FORMS for dtype in ("f16", "bf16")]


def _without(w, left_out):
    w = np.where(left_out, 0, w)
    return w / np.maximum(w.sum(1, keepdims=True), 1e-300)


def _piece(t):
    return (t >= 128) & (t < 256) if t[-1] > 256 else t < (t[-1] + 1) // 2


WRONG = {
    "zeros": lambda w, t: 0 * w,
    "equal weights": lambda w, t: np.full_like(w, 1 / w.shape[1]),
    "newest left out": lambda w, t: _without(w, t == t[-1]),
    "piece left out": lambda w, t: _without(w, _piece(t)),
    "piece at half its weight": lambda w, t: (lambda x: x / x.sum(1, keepdims=True))(
        np.where(_piece(t), w / 2, w)),
}


@pytest.mark.parametrize("lengths,per,heads,dim,G,bits,page,L,dtype", EVERY)
def test_wrong_results_are_refused(lengths, per, heads, dim, G, bits, page, L, dtype):
    # the sequence with the most tokens, and one head: the others are more of the same
    n = max(lengths)
    cache, table = _build([n], 1, dim, G, bits, page, dtype, seed=61)
    qb, q = kv_ref.to_bits(np.random.default_rng(62).standard_normal((1, L, per, dim)), dtype)
    ref, slack = kv_ref.attention_rows(q, cache, table, [n], dim ** -0.5)
    for what, change in WRONG.items():
        if n == 1 and what != "zeros":
            continue
        other, _ = kv_ref.attention_rows(q, cache, table, [n], dim ** -0.5, change)
        worst = kv_ref.rows_off(kv_ref.to_values(other, dtype), ref, slack, dtype)
        assert worst > 1, f"{what}: {worst:.3f}"
    assert kv_ref.rows_off(kv_ref.to_values(ref, dtype), ref, slack, dtype) <= 1
