"""The calls around the cache as a program uses them: one after the other in a
conversation (the example), captured into graphs that are replayed between eager
work, on streams of their own, two at once."""
import os
import sys

import numpy as np
import pytest

import kv_ref
from gpu_util import out_bits, out_to_f64, to_dev
from test_gpu_attention import _queries, _set_value
from test_gpu_kv import _build, _dev16, aq  # noqa: F401  (aq: the module's fixture)

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("bits,dtype", [(4, "f16"), (8, "bf16"), (16, "f16"), (16, "bf16")])
def test_conversation(aq, bits, dtype):
    import long_conversation
    import torch
    kind = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    off, block, evicted = long_conversation.converse(cache_bits=bits, dtype=kind)
    # q twice, the attention's output, both projections and y are each rounded to 11 or 8 bits: six
    # roundings, the sums over 512 terms of random sign grow slower than their largest value
    assert off < 6 * kv_ref.rounding(dtype) * 4
    assert evicted > 0 and block.positions.tolist() == [140, 77, 110]
    assert (block.lengths <= block.budget + 12).all()
    # every row of every step gave one in all, and what was evicted took its share along
    assert (block.weights.sum(1) <= 40 * block.q_heads + 1e-2).all() and (block.weights.sum(1) > 0).all()


def test_prompt_is_many_steps(aq):
    """A prompt's rows are what the same tokens give one at a time over a 16-bit cache."""
    import torch
    n, Hq, H, D = 70, 8, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((n, h, D), generator=gen, device="cuda").half() for h in (Hq, H, H))
    positions = torch.arange(n, dtype=torch.int32, device="cuda")
    freqs, factor = aq.aq_rope_frequencies(D)
    cache = kv_ref.Cache(5, H, 16, D, 32, 16, "f16").device()
    turned = torch.empty_like(k)
    q = aq.aq_rope_append(q, k, v, positions, freqs, positions.long(), *cache, 32, 16, factor=factor, k_out=turned)
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    slopes = torch.rand(Hq, generator=gen, device="cuda") * 0.1
    more = dict(softcap=8.0, window=33, slopes=slopes)
    out, lse = aq.aq_prompt_attention(q, turned, v, starts, starts, return_lse=True, **more)
    table = torch.arange(5, dtype=torch.int32, device="cuda")[None]
    for i in range(n):
        length = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        one, l1 = aq.aq_paged_attention_masked(q[None, i], *cache, table, length, 32, 16, return_lse=True, **more)
        # both are within half a rounding of the weights (and one of the result) of the formula
        assert (one[0].float() - out[i].float()).norm() <= 3 * 2.0 ** -11 * out[i].float().norm()
        assert (l1[0] - lse[i]).abs().max() < 1e-5


# ---- graphs, streams --------------------------------------------------------------------
def _calls(aq):
    """name -> (a call that gives its results, what to change between replays)."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(11)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    lengths = [100, 0, 37, 300]
    cache, table = _build(lengths, 2, 64, 32, 8, 16, "f16", seed=5)
    parts, tab, lens = cache.device(), to_dev(table), to_dev(np.array(lengths, np.int32))
    q = rand(4, 8, 64).half()
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    slopes = torch.rand(8, generator=gen, device="cuda")
    more = dict(softcap=10.0, slopes=slopes, window=50)
    first = lambda: aq.aq_paged_attention_masked(q, *parts, tab, lens, 32, 8, return_lse=True, workspace=ws, **more)  # noqa: E731

    def weigh():
        w = torch.zeros((4, tab.shape[1] * 16), device="cuda")
        aq.aq_kv_weigh(q, first()[1], *parts, tab, lens, w, 32, 8, **more)
        return [w]

    pq, pk = rand(90, 8, 64).half(), rand(2000, 2, 64).half()
    starts = torch.tensor([0, 40, 90], dtype=torch.int32, device="cuda")
    keys = torch.tensor([0, 1900, 1990], dtype=torch.int32, device="cuda")
    few = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    all_keys = torch.tensor([0, 2000], dtype=torch.int32, device="cuda")
    positions = torch.randint(0, 1 << 20, (90,), generator=gen, device="cuda", dtype=torch.int32)
    freqs, _ = aq.aq_rope_frequencies(64)
    weights = torch.rand((4, 320), generator=gen, device="cuda")
    slots = torch.randperm(1280, generator=gen, device="cuda")[:90]  # (the slots of a call differ)
    other = kv_ref.Cache(80, 2, 16, 64, 32, 8, "f16").device()

    def append():
        aq.aq_rope_append(None, pk[:90], pk[90:180], positions, freqs, slots, *other, 32, 8)
        return [other[0], other[1], other[2], other[3], other[4], other[5]]

    new = torch.arange(60, 80, dtype=torch.int32, device="cuda").view(4, 5)
    old = torch.arange(0, 60, dtype=torch.int32, device="cuda").view(4, 15)
    ev_lens = to_dev(np.array([200, 0, 37, 240], np.int32))

    def evict():
        return [*aq.aq_kv_evict(weights, ev_lens, old, new, *other, 32, 8, keep=70, sinks=3, recent=20), *other]

    def shake():
        q.copy_(rand(4, 8, 64))
        pq.copy_(rand(90, 8, 64))
        pk.copy_(rand(2000, 2, 64))
        weights.copy_(torch.rand((4, 320), generator=gen, device="cuda"))
        lens.sub_(1).clamp_(min=0)

    return {"masked": lambda: list(first()), "weigh": weigh, "append": append, "evict": evict,
            "rope": lambda: list(aq.aq_rope(pq, pk[:90], positions, freqs, True)),
            "prompt": lambda: list(aq.aq_prompt_attention(pq, pk, pk, starts, keys, return_lse=True, **more)),
            "prompt in parts": lambda: list(aq.aq_prompt_attention(pq[:2], pk, pk, few, all_keys, return_lse=True)),
            }, shake


@pytest.mark.parametrize("name", ["masked", "weigh", "append", "evict", "rope", "prompt", "prompt in parts"])
def test_captured_and_replayed(aq, name):
    import torch
    calls, shake = _calls(aq)
    call = calls[name]
    call()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        got = call()
    for _ in range(4):
        shake()
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        sum(t.float().sum() for t in want).item()  # (eager work between the replays)


@pytest.mark.parametrize("name", ["masked", "weigh", "append", "evict", "rope", "prompt", "prompt in parts"])
def test_on_another_stream(aq, name):
    import torch
    calls, shake = _calls(aq)
    call = calls[name]
    stream = torch.cuda.Stream()
    for _ in range(3):
        shake()
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            got = [t.clone() for t in call()]
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_two_prompts_at_once(aq):
    """Calls that make their own workspaces, on two streams."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k = (torch.randn((s, h, 128), generator=gen, device="cuda").half() for s, h in ((3, 4), (6000, 1)))
    starts = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    keys = torch.tensor([0, 6000], dtype=torch.int32, device="cuda")
    want = [aq.aq_prompt_attention(x, k, k, starts, keys) for x in (q, -q)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, (s, x) in enumerate(zip(streams, (q, -q))):
            got[i] = aq.aq_prompt_attention(x, k, k, starts, keys, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---- what one row has is not another's --------------------------------------------------
def test_a_nan_stays_with_the_tokens_of_its_row(aq):
    """A key that is NaN makes the weights of the rows that see it NaN, and of no
    token that only other rows see."""
    lengths, dim = [50], 64
    cache, table = _build(lengths, 1, dim, 0, 16, 16, "f16", seed=9)
    cache.parts["k"][0][table[0, 0], 0, 5] = 0x7FFF  # token 5
    qb, _ = _queries(10, (1, 8, 2, dim), "f16")
    q, tab, lens = _dev16(qb, "f16"), to_dev(table), to_dev(np.array(lengths, np.int32))
    import torch
    # rows 42 .. 49 look back 40 tokens: row 42 sees 3 .. 42, 43 from 4, 44 from 5, 45 from 6 on
    _, lse = aq.aq_paged_attention_masked(q, *cache.device(), tab, lens, 32, 16, window=40, return_lse=True)
    lse = lse.cpu().numpy()
    assert np.isnan(lse[0, :3]).all() and np.isfinite(lse[0, 3:]).all()
    w = torch.zeros((1, 64), device="cuda")
    aq.aq_kv_weigh(q, to_dev(lse), *cache.device(), tab, lens, w, 32, 16, window=40)
    w = w.cpu().numpy()[0]
    assert np.isnan(w[3:45]).all()       # some of the three see them
    assert np.isfinite(w[45:50]).all() and (w[45:50] > 0).all()
    assert not w[:3].any() and not w[50:].any()


@pytest.mark.parametrize("cap", [1e3, 1e6, 1e12, 1e30])
def test_a_cap_far_above_the_scores_changes_nothing(aq, cap):
    """Up to s^3 / (3 cap^2), here 2^-13 at most."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn((200, h, 128), generator=gen, device="cuda").half() for h in (4, 1, 1))
    st = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    slopes = torch.rand(4, generator=gen, device="cuda") * 0.1
    for more in (dict(), dict(slopes=slopes)):
        a, b = (aq.aq_prompt_attention(q, k, v, st, st, softcap=c, return_lse=True, **more)[1] for c in (0.0, cap))
        assert (a - b).abs().max() <= 2.0 ** -13 * (1e3 / cap) ** 2 + 2.0 ** -19
    cache, table = _build([200], 1, 128, 64, 8, 16, "f16", seed=3)
    args = (q[None, 199], *cache.device(), to_dev(table), torch.tensor([200], dtype=torch.int32, device="cuda"), 64, 8)
    a, b = (aq.aq_paged_attention_masked(*args, softcap=c, return_lse=True)[1] for c in (0.0, cap))
    assert (a - b).abs().max() <= 2.0 ** -13 * (1e3 / cap) ** 2 + 2.0 ** -19


def test_the_same_token_twice_in_a_table(aq):
    """Two sequences over one sequence's pages: each as alone."""
    import torch
    lengths = [90]
    cache, table = _build(lengths, 2, 64, 32, 4, 16, "bf16", seed=12)
    qb, _ = _queries(13, (1, 1, 8, 64), "bf16")
    q, parts = _dev16(qb, "bf16"), cache.device()
    lens = torch.tensor([90, 90, 60], dtype=torch.int32, device="cuda")
    tab = to_dev(table).expand(3, -1).contiguous()
    out, lse = aq.aq_paged_attention_masked(q.expand(3, -1, -1, -1).contiguous(), *parts, tab, lens, 32, 4, return_lse=True)
    assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1])
    w = torch.zeros((3, 96), device="cuda")
    aq.aq_kv_weigh(q.expand(3, -1, -1, -1).contiguous(), lse, *parts, tab, lens, w, 32, 4)
    assert torch.equal(w[0], w[1]) and abs(float(w[2].sum()) - 8) < 1e-4
