"""Refusals of the cache and attention entry points: every bad argument comes
back from the host's checks before anything is enqueued, so these run without
a GPU.  The formula of the tests' own reference is checked here too."""
import ctypes
import os

import numpy as np
import pytest

import group_wise_affine_aq_amd as aq
import kv_ref
import oracle

OK, INVALID, UNSUPPORTED, ALIGN = 0, -1, -2, -3
F32, F16, BF16 = 0, 1, 2
P, MIS = 0x10000, 0x10008  # never dereferenced; MIS is not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(aq.lib_path()):
        pytest.skip("libaq.so not built (run python -m group_wise_affine_aq_amd.build)")
    return aq.load_library()


def cache(**k):
    f = dict(k_codes=P, k_scales=P, k_biases=P, v_codes=P, v_scales=P, v_biases=P, num_pages=9,
             page_size=16, kv_heads=2, head_dim=128, group_size=64, bits=8, dtype=0)
    assert not set(k) - set(f)
    return aq._KVCache(*{**f, **k}.values())


def append(lib, c, k=P, v=P, dt=F16, T=3, ks=256, vs=256, slots=P):
    return lib.aq_kv_append(k, v, dt, T, ks, vs, slots, ctypes.byref(c) if c else None, None)


def read(lib, c, slots=P, T=3, k=P, v=P, dt=F16):
    return lib.aq_kv_read(slots, T, ctypes.byref(c) if c else None, k, v, dt, None)


def attend(lib, c, q=P, dt=F16, B=2, L=1, hq=8, qs=1024, table=P, mp=4, lengths=P, out=P, ws=P,
           wsb=64 << 20):
    return lib.aq_paged_attention(q, dt, B, L, hq, qs, ctypes.byref(c) if c else None, table, mp,
                                  lengths, 0.1, out, ws, wsb, None)


@pytest.mark.parametrize("call", [append, read, attend])
def test_cache_shape_errors(lib, call):
    assert call(lib, None) == INVALID
    for bad in (dict(num_pages=0), dict(page_size=0), dict(kv_heads=0), dict(head_dim=0),
                dict(num_pages=-1), dict(kv_heads=-2), dict(bits=1), dict(bits=9), dict(bits=0),
                dict(bits=-4), dict(group_size=0), dict(group_size=16), dict(group_size=48),
                dict(group_size=128, head_dim=64), dict(bits=16, dtype=F32),
                dict(bits=16, dtype=7), dict(k_codes=None), dict(v_codes=None),
                dict(k_scales=None), dict(v_scales=None)):
        assert call(lib, cache(**bad)) == INVALID, bad
    for bad in (dict(bits=5), dict(bits=2), dict(head_dim=384), dict(head_dim=192),
                dict(page_size=8), dict(page_size=24), dict(num_pages=1 << 31),
                dict(page_size=1 << 24), dict(kv_heads=1 << 28), dict(kv_heads=1 << 30)):
        assert call(lib, cache(**bad)) == UNSUPPORTED, bad
    for bad in ("k_codes", "k_scales", "k_biases", "v_codes", "v_scales", "v_biases"):
        assert call(lib, cache(**{bad: MIS})) == ALIGN, bad


def test_append_errors(lib):
    c = cache()
    for bad in (dict(T=-1), dict(dt=F32), dict(dt=9), dict(k=None), dict(v=None),
                dict(slots=None), dict(ks=255), dict(ks=248), dict(vs=0), dict(vs=-256),
                dict(ks=260)):
        assert append(lib, c, **bad) == INVALID, bad
    for bad in (dict(k=MIS), dict(v=MIS), dict(slots=MIS)):
        assert append(lib, c, **bad) == ALIGN, bad
    for bad in (dict(T=1 << 50), dict(ks=1 << 62), dict(T=1 << 30, vs=1 << 40)):
        assert append(lib, c, **bad) == UNSUPPORTED, bad
    # the writer needs somewhere to put biases; 16 bits needs neither them nor scales
    assert append(lib, cache(k_biases=None)) == INVALID
    assert append(lib, cache(v_biases=None)) == INVALID
    none = dict(k_scales=None, k_biases=None, v_scales=None, v_biases=None, group_size=0)
    assert append(lib, cache(bits=16, dtype=BF16, **none), dt=F16) == INVALID
    assert append(lib, cache(bits=16, dtype=BF16, **none), dt=BF16, T=0) == OK
    assert append(lib, c, T=0, k=None, v=None, slots=None) == OK


def test_read_errors(lib):
    c = cache()
    for bad in (dict(T=-1), dict(dt=3), dict(dt=-1), dict(k=None), dict(v=None),
                dict(slots=None)):
        assert read(lib, c, **bad) == INVALID, bad
    for bad in (dict(k=MIS), dict(v=MIS), dict(slots=MIS)):
        assert read(lib, c, **bad) == ALIGN, bad
    assert read(lib, c, T=1 << 50) == UNSUPPORTED
    assert read(lib, cache(k_biases=None, v_biases=None), T=0) == OK
    assert read(lib, c, T=0, slots=None, k=None, v=None) == OK


def test_attention_errors(lib):
    c = cache()
    for bad in (dict(B=0), dict(B=-1), dict(L=0), dict(L=9), dict(hq=0), dict(hq=7), dict(hq=-2),
                dict(dt=F32), dict(mp=0), dict(qs=1016), dict(qs=1028), dict(qs=0), dict(q=None),
                dict(table=None), dict(lengths=None), dict(out=None), dict(ws=None),
                dict(wsb=-1), dict(wsb=0)):
        assert attend(lib, c, **bad) == INVALID, bad
    for bad in (dict(q=MIS), dict(table=MIS), dict(lengths=MIS), dict(out=MIS), dict(ws=MIS)):
        assert attend(lib, c, **bad) == ALIGN, bad
    for bad in (dict(mp=1 << 27), dict(mp=1 << 60), dict(B=1 << 24), dict(B=1 << 21, L=1),
                dict(B=1 << 60), dict(hq=1 << 24, qs=1 << 40), dict(qs=1 << 62)):
        assert attend(lib, c, **bad) == UNSUPPORTED, bad
    assert attend(lib, cache(bits=16, dtype=BF16), dt=F16) == INVALID


def test_workspace_bytes(lib):
    ask = lib.aq_paged_attention_workspace
    for bad in ((0, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 9, 8, 2, 128), (1, 1, 8, 3, 128),
                (1, 1, 8, 2, 96), (1, 1, 0, 2, 128), (1 << 24, 1, 8, 2, 128)):
        assert ask(*bad) == -1, bad
    for B, L, hq, hkv, D in ((1, 1, 1, 1, 64), (7, 3, 35, 5, 64), (64, 8, 128, 8, 256),
                             (1 << 18, 1, 32, 8, 128), (1 << 20, 1, 8, 1, 256),
                             ((1 << 24) - 1, 1, 1, 1, 64)):
        n = ask(B, L, hq, hkv, D)
        assert 0 < n <= 64 << 20, (B, L, hq, hkv, D, n)
    with pytest.raises(aq.AQError):
        aq.aq_paged_attention_workspace(1, 1, 8, 3, 128)


def test_reference_attention_is_the_formula():
    """kv_ref.attention against the formula written out token by token."""
    rng = np.random.default_rng(0)
    B, L, Hq, H, D, page, G = 2, 3, 4, 2, 64, 16, 32
    lengths, table = [21, 2], np.array([[2, 0, -1], [3, 1, -1]], np.int32)
    c = kv_ref.Cache(4, H, page, D, G, 8)
    dense = {}
    for b, n in enumerate(lengths):
        for t in range(n):
            for name in "kv":
                bits, x = kv_ref.to_bits(rng.standard_normal((H, D)), "f16")
                c.put(name, int(table[b, t // page]) * page + t % page, bits, x)
                packed = oracle.quantize(x.astype(np.float32), G, 8)
                dense[b, t, name] = oracle.dequantize_exact(*packed, D, G, 8)
    q = rng.standard_normal((B, L, Hq, D))
    out, bound = kv_ref.attention(q, c, table, lengths, 0.125)
    for b, n in enumerate(lengths):
        for i in range(L):
            for h in range(Hq):
                seen = [t for t in range(n) if t <= n - L + i]
                if not seen:
                    assert not out[b, i, h].any()
                    continue
                w = np.exp([0.125 * q[b, i, h] @ dense[b, t, "k"][h // 2] for t in seen])
                ref = sum(x * dense[b, t, "v"][h // 2] for x, t in zip(w, seen)) / w.sum()
                assert np.allclose(out[b, i, h], ref, rtol=1e-12, atol=1e-14)
                assert (bound[b, i, h] > 0).all()
