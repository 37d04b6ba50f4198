"""Refusals of the calls around the cache -- rotary positions, masked and prompt
attention, gathered weights, eviction: every bad argument comes back from the
host's checks before anything is enqueued, so these run without a GPU.  And
the frequencies, which are computed on the host."""
import ctypes
import math
import os

import numpy as np
import pytest

import group_wise_affine_aq_amd as aq
from test_kv_abi import ALIGN, BF16, F16, F32, INVALID, MIS, OK, P, UNSUPPORTED, cache

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(aq.lib_path()):
        pytest.skip("libaq.so not built (run python -m group_wise_affine_aq_amd.build)")
    return aq.load_library()


def given(x):
    return ctypes.byref(x) if x is not None and not isinstance(x, bytes) else x


def scores(softcap=0.0, window=0, slopes=None, first=None, prefix=None, lse=None):
    return aq._pack_scores(softcap, window, *(x or 0 for x in (slopes, first, prefix, lse)))


def masked(lib, c, sc=scores(), q=P, dt=F16, B=2, L=1, hq=8, qs=1024, table=P, mp=4, lengths=P, out=P,
           ws=P, wsb=64 << 20):
    return lib.aq_paged_attention_masked(q, dt, B, L, hq, qs, given(c), table, mp, lengths, 0.1, sc,
                                         out, ws, wsb, None)


def weigh(lib, c, sc=scores(lse=P), q=P, dt=F16, B=2, L=1, hq=8, qs=1024, table=P, mp=4, lengths=P,
          w=P, ws=64):
    return lib.aq_kv_weigh(q, dt, B, L, hq, qs, given(c), table, mp, lengths, 0.1, sc, w, ws, None)


def prompt(lib, sc=scores(), q=P, dt=F16, Tq=5, hq=8, qs=1024, k=P, ks=256, v=P, vs=256, Tk=9, hk=2,
           d=128, B=2, qst=P, kst=P, out=P, ws=P, wsb=64 << 20):
    return lib.aq_prompt_attention(q, dt, Tq, hq, qs, k, ks, v, vs, Tk, hk, d, B, qst, kst, 0.1, sc, out,
                                   ws, wsb, None)


def rotation(positions=P, freqs=P, rotary=128, interleaved=0, factor=1.0):
    return aq._pack_rotation(positions or 0, freqs or 0, rotary, interleaved, factor)


def rope(lib, r=rotation(), q=P, qs=1024, hq=8, k=P, ks=256, hk=2, dt=F16, T=3, d=128, qo=P, qos=1024,
         ko=P, kos=256):
    return lib.aq_rope(q, qs, hq, k, ks, hk, dt, T, d, r, qo, qos, ko, kos, None)


def append(lib, c, r=rotation(), q=P, qs=1024, hq=8, k=P, ks=256, v=P, vs=256, dt=F16, T=3, slots=P, qo=P,
           qos=1024, ko=None, kos=0):
    return lib.aq_rope_append(q, qs, hq, k, ks, v, vs, dt, T, r, slots, given(c), qo, qos, ko, kos, None)


def evict(lib, c, w=P, ws=64, lengths=P, B=2, table=P, mp=4, new=P, nmp=2, keep=20, sinks=2, recent=3,
          kept=P, nw=P, nl=P):
    return lib.aq_kv_evict(w, ws, lengths, B, table, mp, new, nmp, given(c), keep, sinks, recent, kept,
                           nw, nl, None)


@pytest.mark.parametrize("call", [masked, weigh, append, evict])
def test_cache_shape_errors(lib, call):
    assert call(lib, None) == INVALID
    for bad in (dict(num_pages=0), dict(page_size=0), dict(kv_heads=0), dict(head_dim=0), dict(bits=1),
                dict(bits=9), dict(group_size=0), dict(group_size=48), dict(group_size=128, head_dim=64),
                dict(bits=16, dtype=F32), dict(k_codes=None), dict(v_codes=None), dict(k_scales=None),
                dict(v_scales=None)):
        assert call(lib, cache(**bad)) == INVALID, bad
    for bad in (dict(bits=5), dict(head_dim=384), dict(page_size=24), dict(num_pages=1 << 31),
                dict(page_size=1 << 24), dict(kv_heads=1 << 28)):
        assert call(lib, cache(**bad)) == UNSUPPORTED, bad
    for bad in ("k_codes", "k_scales", "k_biases", "v_codes", "v_scales", "v_biases"):
        assert call(lib, cache(**{bad: MIS})) == ALIGN, bad


@pytest.mark.parametrize("call", [masked, weigh])
def test_new_tokens_errors(lib, call):
    c = cache()
    for bad in (dict(B=0), dict(L=0), dict(L=9), dict(hq=0), dict(hq=7), dict(dt=F32), dict(mp=0),
                dict(qs=1016), dict(qs=1028), dict(q=None), dict(table=None), dict(lengths=None)):
        assert call(lib, c, **bad) == INVALID, bad
    for bad in (dict(q=MIS), dict(table=MIS), dict(lengths=MIS)):
        assert call(lib, c, **bad) == ALIGN, bad
    for bad in (dict(mp=1 << 27), dict(B=1 << 24), dict(hq=1 << 24, qs=1 << 40), dict(qs=1 << 62)):
        assert call(lib, c, **bad) == UNSUPPORTED, bad
    assert call(lib, cache(bits=16, dtype=BF16), dt=F16) == INVALID


def test_scores_errors(lib):
    c = cache()
    calls = {masked: lambda **s: masked(lib, c, scores(**s)), prompt: lambda **s: prompt(lib, scores(**s)),
             weigh: lambda **s: weigh(lib, c, scores(**{"lse": P, **s}))}
    for name, call in calls.items():
        for bad in (dict(softcap=-1.0), dict(softcap=NAN), dict(softcap=INF), dict(softcap=1e-31),
                    dict(softcap=1e31), dict(window=-1)):
            assert call(**bad) == INVALID, (name, bad)
        for bad in ("slopes", "first", "lse"):
            assert call(**{bad: MIS}) == ALIGN, (name, bad)
        assert call(prefix=P) == INVALID or name is prompt
    assert prompt(lib, scores(prefix=MIS)) == ALIGN
    assert masked(lib, c, None) == prompt(lib, None) == weigh(lib, c, None) == INVALID


def test_masked_errors(lib):
    c = cache()
    for bad in (dict(out=None), dict(ws=None), dict(wsb=0), dict(wsb=-1)):
        assert masked(lib, c, **bad) == INVALID, bad
    for bad in (dict(out=MIS), dict(ws=MIS)):
        assert masked(lib, c, **bad) == ALIGN, bad


def test_weigh_errors(lib):
    c = cache()
    for bad in (dict(sc=scores()), dict(w=None), dict(ws=0), dict(ws=-4), dict(ws=63)):
        assert weigh(lib, c, **bad) == INVALID, bad
    assert weigh(lib, c, w=MIS) == ALIGN
    for bad in (dict(ws=1 << 62), dict(B=1 << 20, mp=1 << 20)):
        assert weigh(lib, c, **bad) == UNSUPPORTED, bad


def test_prompt_errors(lib):
    for bad in (dict(Tq=-1), dict(Tk=-1), dict(B=0), dict(hq=0), dict(hk=0), dict(hq=7), dict(dt=F32),
                dict(qs=1016), dict(qs=1028), dict(ks=248), dict(ks=260), dict(vs=0), dict(q=None),
                dict(k=None), dict(v=None), dict(qst=None), dict(kst=None), dict(out=None), dict(ws=None),
                dict(wsb=0)):
        assert prompt(lib, **bad) == INVALID, bad
    for bad in ("q", "k", "v", "qst", "kst", "out", "ws"):
        assert prompt(lib, **{bad: MIS}) == ALIGN, bad
    for bad in (dict(d=96, qs=1024), dict(d=192, qs=2048, ks=512, vs=512), dict(Tq=1 << 21), dict(Tk=1 << 23),
                dict(B=1 << 23), dict(ks=(1 << 23) + 8), dict(vs=1 << 40), dict(qs=1 << 62)):
        assert prompt(lib, **bad) == UNSUPPORTED, bad
    assert prompt(lib, Tq=0, q=None, k=None, v=None, out=None) == OK


def test_prompt_workspace(lib):
    ask = lib.aq_prompt_attention_workspace
    for bad in ((-1, 1, 1, 8, 2, 128), (1, 1, 0, 8, 2, 128), (1, 1, 1, 8, 3, 128), (1, 1, 1, 8, 2, 96)):
        assert ask(*bad) == -1, bad
    for shape in ((1, 1, 1, 1, 1, 64), (1, 1 << 20, 1, 8, 8, 128), (64, 1 << 20, 1, 8, 1, 256),
                  (16, 1 << 23, 16, 64, 1, 64), (8192, 8192, 1, 32, 8, 128), (500, 100000, 100, 128, 8, 256)):
        n = ask(*shape)
        assert 0 < n <= 64 << 20, (shape, n)
    with pytest.raises(aq.AQError):
        aq.aq_prompt_attention_workspace(1, 1, 1, 8, 3, 128)


def test_rope_errors(lib):
    for bad in (dict(T=-1), dict(hq=-1), dict(hk=-1), dict(dt=F32), dict(d=0), dict(r=None),
                dict(r=rotation(rotary=0)), dict(r=rotation(rotary=144)), dict(r=rotation(factor=NAN)),
                dict(r=rotation(factor=-INF)), dict(r=rotation(positions=None)), dict(r=rotation(freqs=None)),
                dict(qs=1016), dict(qs=1028), dict(qos=8), dict(ks=248), dict(kos=252), dict(q=None),
                dict(k=None), dict(qo=None), dict(ko=None)):
        assert rope(lib, **bad) == INVALID, bad
    for bad in (dict(r=rotation(rotary=24)), dict(d=96, r=rotation(rotary=32)), dict(T=1 << 40),
                dict(T=2, ks=1 << 62)):
        assert rope(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=MIS), dict(k=MIS), dict(qo=MIS), dict(ko=MIS), dict(r=rotation(positions=MIS)),
                dict(r=rotation(freqs=MIS))):
        assert rope(lib, **bad) == ALIGN, bad
    assert rope(lib, T=0, q=None, k=None, qo=None, ko=None, r=rotation(positions=None, freqs=None)) == OK
    assert rope(lib, hq=0, hk=0, q=None, k=None, qo=None, ko=None) == OK


def test_rope_append_errors(lib):
    c = cache()
    for bad in (dict(v=None), dict(slots=None), dict(vs=248), dict(T=-1), dict(dt=F32), dict(k=None),
                dict(q=None), dict(qo=None), dict(ko=P, kos=8), dict(r=rotation(rotary=256))):
        assert append(lib, c, **bad) == INVALID, bad
    for bad in (dict(v=MIS), dict(slots=MIS), dict(ko=MIS, kos=256)):
        assert append(lib, c, **bad) == ALIGN, bad
    assert append(lib, cache(k_biases=None)) == append(lib, cache(v_biases=None)) == INVALID
    assert append(lib, cache(bits=16, dtype=BF16), dt=F16) == INVALID
    assert append(lib, c, T=0, q=None, k=None, v=None, slots=None, qo=None) == OK


def test_evict_errors(lib):
    c = cache()
    for bad in (dict(B=0), dict(mp=0), dict(nmp=0), dict(ws=0), dict(keep=0), dict(sinks=-1),
                dict(recent=-1), dict(sinks=21), dict(sinks=10, recent=11), dict(keep=33),
                dict(w=None), dict(lengths=None), dict(table=None), dict(new=None), dict(kept=None),
                dict(nw=None), dict(nl=None), dict(sinks=1 << 62, recent=1 << 62)):
        assert evict(lib, c, **bad) == INVALID, bad
    for bad in ("w", "lengths", "table", "new", "kept", "nw", "nl"):
        assert evict(lib, c, **{bad: MIS}) == ALIGN, bad
    for bad in (dict(B=1 << 24), dict(mp=1 << 27), dict(nmp=1 << 27), dict(ws=(1 << 30) + 4),
                dict(keep=1 << 31, nmp=1 << 26), dict(B=1 << 20, keep=1 << 12, nmp=1 << 9)):
        assert evict(lib, c, **bad) == UNSUPPORTED, bad


def test_launches_of_more_threads_than_there_are(lib):
    """2^32 threads or more in one launch: refused before anything is enqueued."""
    c = cache(kv_heads=1, head_dim=64, group_size=64, bits=4)
    # moving: B * ceil(keep / 64) * kv_heads workgroups; choosing: B of 1024 threads
    for bad in (dict(B=1, keep=1 << 30, nmp=1 << 26), dict(B=1 << 14, keep=1 << 16, nmp=1 << 12),
                dict(B=1 << 22, keep=1, nmp=1, sinks=0, recent=0)):
        assert evict(lib, c, **bad) == UNSUPPORTED, bad
    assert evict(lib, cache(kv_heads=16, num_pages=1), B=1 << 20, keep=64, nmp=4) == UNSUPPORTED
    for T in (1 << 28, 0x7FFFFFF0):
        assert rope(lib, T=T) == append(lib, cache(), T=T) == UNSUPPORTED, T


# ---- frequencies ------------------------------------------------------------------------
def freqs(*args, **k):
    return aq.aq_rope_frequencies(*args, device="cpu", **k)


def test_frequencies_by_the_formulas(lib):
    R, base, s, ctx = 128, 10000.0, 8.0, 4096.0
    i = np.arange(R // 2)
    f = base ** (-2.0 * i / R)
    same = lambda got, want: np.array_equal(got.numpy(), want.astype(np.float32))  # noqa: E731
    assert same(freqs(R, base)[0], f) and freqs(R, base)[1] == 1.0
    assert same(freqs(R, base, "linear", s)[0], f / s)
    assert np.allclose(freqs(R, base, "base", s)[0], (base * s ** (R / (R - 2))) ** (-2.0 * i / R), rtol=1e-7)
    # the longest wave of "base" is the stretched one
    assert math.isclose(freqs(R, base, "base", s)[0][-1], f[-1] / s, rel_tol=1e-6)
    got, factor = freqs(R, base, "by_index", s, ctx, 1.0, 32.0)
    index = lambda r: R * math.log(ctx / (2 * math.pi * r)) / (2 * math.log(base))  # noqa: E731
    a, b = max(math.floor(index(32)), 0), min(math.ceil(index(1)), R - 1)
    g = np.clip((i - a) / (b - a), 0, 1)
    assert np.allclose(got, g * f / s + (1 - g) * f, rtol=1e-7)
    assert math.isclose(factor, 0.1 * math.log(s) + 1, rel_tol=1e-6)
    assert got[0] == 1.0 and math.isclose(got[-1], f[-1] / s, rel_tol=1e-6)
    got, factor = freqs(R, 500000.0, "by_turns", s, ctx, 1.0, 4.0)
    f = 500000.0 ** (-2.0 * i / R)
    g = 1 - np.clip((ctx * f / (2 * math.pi) - 1) / 3, 0, 1)
    assert np.allclose(got, g * f / s + (1 - g) * f, rtol=1e-7) and factor == 1.0


def test_frequencies_are_made_on_the_host(lib):
    """Where tensors are made on another device by default, too: the library
    fills host memory."""
    import torch
    with torch.device("meta"):
        got, factor = freqs(128, 500000.0, "by_turns", 8.0, 4096.0, 1.0, 4.0)
    want = freqs(128, 500000.0, "by_turns", 8.0, 4096.0, 1.0, 4.0)
    assert got.device.type == "cpu" and torch.equal(got, want[0]) and factor == want[1]


def test_frequencies_errors(lib):
    for bad in (dict(rotary=2), dict(rotary=7), dict(rotary=-4), dict(base=1.0), dict(base=NAN), dict(base=INF),
                dict(kind="linear", stretch=0.5), dict(kind="base", stretch=INF),
                dict(kind="by_index", stretch=2.0, ctx=0.0, low=1.0, high=2.0),
                dict(kind="by_turns", stretch=2.0, ctx=100.0, low=2.0, high=2.0),
                dict(kind="by_turns", stretch=2.0, ctx=100.0, low=0.0, high=2.0)):
        with pytest.raises(aq.AQError):
            freqs(**{"rotary": 64, **bad})
    assert lib.aq_rope_frequencies(64, 1e4, 5, 2.0, 1.0, 1.0, 2.0, P, None) == INVALID
    assert lib.aq_rope_frequencies(64, 1e4, -1, 2.0, 1.0, 1.0, 2.0, P, None) == INVALID
    assert lib.aq_rope_frequencies(64, 1e4, 0, 2.0, 1.0, 1.0, 2.0, None, None) == INVALID
    with pytest.raises(KeyError):
        freqs(64, kind="other")


# ---- the tests' own formulas -------------------------------------------------------------
def test_reference_is_the_formula():
    """scores_ref.row against the formula written out token by token."""
    import scores_ref
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((2, 8)), rng.standard_normal((11, 8)), rng.standard_normal((11, 8))
    slope = np.array([0.3, 0.7])
    for pos, window, first, prefix in ((10, 0, 0, 0), (4, 3, 0, 7), (6, 0, 5, 0), (2, 0, 4, 0), (-2, 0, 0, 3)):
        sees = scores_ref.seen(11, pos, window, first, prefix)
        out, lse, *_ = scores_ref.row(q, k, v, np.abs(k), np.abs(v), sees, 0.5, pos, 0.0, 2.0, slope)
        for h in range(2):
            w = {}
            for t in range(11):
                if (t <= pos or t < prefix) and t >= first and (not window or pos - t < window):
                    s = 2.0 * math.tanh(0.5 * float(q[h] @ k[t]) / 2.0) - slope[h] * abs(pos - t)
                    w[t] = math.exp(s)
            total = sum(w.values())
            if w:
                assert np.allclose(out[h], sum(x * v[t] for t, x in w.items()) / total, rtol=1e-12)
                assert math.isclose(lse[h], math.log(total), rel_tol=1e-12)
            else:
                assert not out[h].any() and lse[h] == -math.inf


@pytest.mark.parametrize("named", [False, True])
def test_calls_run_on_the_device_of_their_tensors(monkeypatch, named):
    """Whether the first tensor is passed by position or by name, or stands behind a None."""
    import contextlib
    import torch

    class There(torch.Tensor):
        is_cuda = property(lambda self: True)
        device = property(lambda self: "the second")
        get_device = lambda self: 1  # noqa: E731

    entered = []

    @contextlib.contextmanager
    def device(x):
        entered.append(x)
        yield

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    x = torch.zeros(2).as_subclass(There)
    call = aq._on_its_device(lambda q, k, stream=None: (q, k))
    assert (call(q=None, k=x) if named else call(None, x)) == (None, x) and entered == ["the second"]
    assert (call(k=None, q=x) if named else call(x, None)) == (x, None) and len(entered) == 2
    assert call(None, None) == (None, None) and len(entered) == 2
