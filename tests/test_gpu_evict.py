"""Eviction on the GPU: the kept tokens, their weights and rows against numpy's
stable sort and plain copies, exactly."""
import numpy as np
import pytest

import kv_ref
from gpu_util import to_dev
from test_gpu_kv import _cache_bits, aq  # noqa: F401  (aq: the module's fixture)

pytestmark = pytest.mark.gpu


def _choose(w, n, keep, sinks, recent):
    if n <= keep:
        return np.arange(n)
    between = np.arange(sinks, n - recent)
    rank = np.where(np.isnan(w[between]), -np.inf, w[between].astype(np.float64))
    rank = np.where(np.isnan(w[between]), -1e300, np.maximum(rank, -1e299))  # NaN below -inf
    best = between[np.argsort(-rank, kind="stable")[:keep - sinks - recent]]
    return np.sort(np.concatenate([np.arange(sinks), best, np.arange(n - recent, n)]))


def _run(aq, lengths, weights, keep, sinks, recent, heads=2, dim=64, G=32, bits=8, page=16, dtype="f16",
         seed=0, bad_pages=False, null_biases=False, capacity=None):
    import torch
    rng = np.random.default_rng(seed)
    B = len(lengths)
    old, new = (-(-max(1, x) // page) for x in (capacity or max(lengths), keep))
    pages = B * (old + new) + 2
    order = rng.permutation(pages).astype(np.int32)
    table, new_table = order[:B * old].reshape(B, old), order[B * old:B * (old + new)].reshape(B, new)
    if bad_pages:
        table[0, 0], new_table[-1, -1] = -1, pages
    cache = kv_ref.Cache(pages, heads, page, dim, G, bits, dtype)
    for n in "kv":
        for part in cache.parts[n]:
            if part is not None:
                part[:] = rng.integers(0, 1 << 16, part.shape)
    parts = cache.device(null_biases)
    w = to_dev(weights)
    given = to_dev(np.array(lengths, np.int32))
    kept, out_lengths, got = aq.aq_kv_evict(w, given, to_dev(table), to_dev(new_table), *parts, G, bits,
                                            keep=keep, sinks=sinks, recent=recent)
    cap = min(old * page, weights.shape[1])
    kept, got = kept.cpu().numpy(), got.cpu().numpy()
    want = {n: [None if p is None else p.copy() for p in cache.parts[n]] for n in "kv"}
    for b, n in enumerate(lengths):
        n = min(max(n, 0), cap)
        stay = _choose(weights[b], n, keep, sinks, recent)
        assert int(out_lengths[b]) == len(stay)
        assert np.array_equal(kept[b, :len(stay)], stay), (b, n)
        assert (kept[b, len(stay):] == -1).all() and not got[b, len(stay):].any()
        assert np.array_equal(got[b, :len(stay)], weights[b, stay], equal_nan=True)
        for to, at in enumerate(stay):
            src, dst = table[b, at // page], new_table[b, to // page]
            if 0 <= dst < pages:
                for name in "kv":
                    for part, whole in zip(want[name], cache.parts[name]):
                        if part is not None:
                            part[dst, :, to % page] = whole[src, :, at % page] if 0 <= src < pages else 0
    for i, (n, part) in enumerate((n, p) for n in "kv" for p in range(3)):
        if parts[i] is not None:
            assert np.array_equal(_cache_bits(parts[i]), want[n][part]), (n, part)


def _weights(rng, B, n, kind):
    w = np.exp(3 * rng.standard_normal((B, n)))
    if kind == "ties":
        w = np.round(w * 4) / 4
    if kind == "equal":
        w[:] = 0.5
    if kind == "odd":
        w = rng.choice([0.0, -0.0, np.inf, -np.inf, np.nan, 1.0, -1.0, 1e-45, -1e-45, 3e38], (B, n))
    return w.astype(np.float32)


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("lengths,keep,sinks,recent", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([2], 1, 1, 0), ([2], 1, 0, 1), ([17, 0, 5, 300], 16, 3, 4),
    ([64, 65, 66, 1000], 64, 0, 0), ([1023, 1024, 1025], 500, 500, 0), ([700, 3000], 333, 33, 300),
    ([5000], 4999, 4, 64), ([70, 80], 200, 10, 20), ([4097, 129, 2], 128, 1, 126)])
def test_choice(aq, lengths, keep, sinks, recent, kind):
    rng = np.random.default_rng(sum(lengths))
    width = -(-max(lengths) // 16) * 16
    _run(aq, lengths, _weights(rng, len(lengths), width, kind), keep, sinks, recent)


@pytest.mark.parametrize("bits,dim,G,heads,page", [
    (4, 64, 32, 1, 16), (4, 64, 64, 3, 48), (4, 128, 64, 8, 64), (4, 256, 32, 2, 16), (8, 64, 64, 5, 16),
    (8, 128, 128, 2, 32), (8, 256, 128, 1, 96), (8, 128, 32, 2, 16), (16, 64, 0, 2, 16), (16, 128, 0, 4, 80),
    (16, 256, 0, 1, 16)])
def test_rows(aq, bits, dim, G, heads, page):
    rng = np.random.default_rng(dim + bits)
    lengths = [333, 1, 150, 0, 260]
    _run(aq, lengths, _weights(rng, 5, 400, "ties"), 130, 4, 31, heads, dim, G or 32, bits, page, "bf16", 1)
    if bits != 16:
        _run(aq, lengths, _weights(rng, 5, 400, "ties"), 130, 4, 31, heads, dim, G, bits, page, seed=2,
             null_biases=True)


def test_pages_that_are_not_there(aq):
    rng = np.random.default_rng(5)
    _run(aq, [200, 100, 333], _weights(rng, 3, 336, "plain"), 90, 20, 10, bad_pages=True)


def test_lengths_past_the_table_and_the_weights(aq):
    rng = np.random.default_rng(6)
    _run(aq, [500, 40, -7], _weights(rng, 3, 336, "plain"), 90, 20, 10, capacity=320)
    _run(aq, [500, 40, 301], _weights(rng, 3, 300, "plain"), 90, 20, 10, capacity=320)


def test_long_sequence(aq):
    rng = np.random.default_rng(7)
    w = (rng.random((1, 131072)) ** 8).astype(np.float32)
    _run(aq, [131071], w, 3000, 4, 100, heads=1)


def test_lengths_in_place(aq):
    import torch
    cache = kv_ref.Cache(12, 1, 16, 64, 32, 8).device()
    tables = torch.arange(12, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([60, 7], dtype=torch.int32, device="cuda")
    w = torch.rand((2, 64), device="cuda")
    kept, new, _ = aq.aq_kv_evict(w, lengths, tables[:8].view(2, 4).contiguous(), tables[8:].view(2, 2).contiguous(),
                                  *cache, 32, 8, keep=30, recent=5, new_lengths=lengths)
    assert new is lengths and lengths.tolist() == [30, 7]
    assert kept[0, -5:].tolist() == [55, 56, 57, 58, 59] and kept[1, 7:].max() == -1
