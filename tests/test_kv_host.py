"""The K/V cache's entry points without a GPU: refusals before anything is
enqueued, and the plain reference against definitions worked by hand."""
import ctypes

import numpy as np
import pytest

from oracle import kv


@pytest.fixture(scope="module")
def b():
    from bitmap_encoded_unstructured_ie_gb300 import binding, build
    build.build()
    binding.load()
    return binding


P = 1 << 20                                    # any aligned address: refused calls read nothing


def cache(b, **kw):
    f = dict(elem=b.US_I8, D=128, Hkv=8, page_size=64, num_pages=10, B=2, max_pages=4, reserved=0, k=P, v=P, scale=P,
             page_table=P)
    f.update(kw)
    return b.us_kv_cache(*(f[n] for n, _ in b.us_kv_cache._fields_))


def calls(b, c, T=2, ld=1024, off=P, pos=P, max_n=4, K=P, V=P):
    lib, r = b.load(), ctypes.byref(c) if c is not None else None
    return (lib.us_kv_write(r, K, ld, V, ld, T, off, pos, max_n, None),
            lib.us_kv_read(r, T, off, pos, max_n, K, ld, V, ld, None),
            lib.us_kv_commit(r, T, off, K, pos, max_n, None) if ld == 1024 and V == P else None,
            lib.us_attn_kv(r, K, ld, 8, T, off, pos, None, max_n, 0.1, V, ld, P, 1 << 40, None))


@pytest.mark.parametrize("kw,code", [
    (dict(elem=0), 1), (dict(elem=2), 1), (dict(elem=9), 1), (dict(D=96), 2), (dict(D=256), 2), (dict(D=0), 1),
    (dict(Hkv=0), 1), (dict(Hkv=2000), 3), (dict(page_size=8), 1), (dict(page_size=48), 1), (dict(page_size=2048), 1),
    (dict(num_pages=0), 1), (dict(B=0), 1), (dict(B=1025), 3), (dict(max_pages=0), 1), (dict(max_pages=1 << 24), 3),
    (dict(reserved=1), 1), (dict(k=None), 1), (dict(v=P + 8), 1), (dict(scale=None), 1), (dict(page_table=P + 4), 1)])
def test_bad_caches_are_refused(b, kw, code):
    assert set(calls(b, cache(b, **kw))) == {code}
    n = ctypes.c_size_t()
    assert b.load().us_attn_kv_workspace_bytes(ctypes.byref(cache(b, **kw)), 8, 1, ctypes.byref(n)) == code


@pytest.mark.parametrize("kw", [dict(T=-1), dict(off=None), dict(pos=None), dict(off=P + 4), dict(max_n=0), dict(ld=1016),
                                dict(ld=1028), dict(K=None), dict(K=P + 2), dict(V=None)])
def test_bad_calls_are_refused(b, kw):
    assert set(calls(b, cache(b), **kw)) - {None} == {1}


def test_other_refusals(b):
    lib, c = b.load(), cache(b)
    r = ctypes.byref(c)
    assert calls(b, None) == (1, 1, 1, 1)
    assert lib.us_kv_commit(r, 2, P, P, P, 65, None) == b.US_ERR_UNSUPPORTED
    attn = lambda Hq=8, mask=None, max_n=1, scale=0.1, ws=P, wsb=1 << 40: lib.us_attn_kv(  # noqa: E731
        r, P, 4096 * 128, Hq, 2, P, P, mask, max_n, scale, P, 4096 * 128, ws, wsb, None)
    assert attn(Hq=12) == 1 and attn(Hq=0) == 1 and attn(Hq=8192) == b.US_ERR_TOO_LARGE
    assert attn(mask=P, max_n=65) == b.US_ERR_UNSUPPORTED and attn(mask=P + 8) == 1
    assert attn(scale=float("nan")) == 1 and attn(scale=float("inf")) == 1
    assert lib.us_attn_kv_workspace_bytes(r, 8, 1, None) == 1


def test_no_tokens_is_no_work(b):
    lib, r = b.load(), ctypes.byref(cache(b))
    assert lib.us_kv_write(r, None, 0, None, 0, 0, P, P, 1, None) == 0
    assert lib.us_kv_read(r, 0, P, P, 1, None, 0, None, 0, None) == 0
    assert lib.us_kv_commit(r, 0, P, None, P, 1, None) == 0
    assert lib.us_attn_kv(r, None, 0, 8, 0, P, P, None, 1, 1.0, None, 0, None, 0, None) == 0


def test_matrices_of_weights_do_not_take_int8(b):
    n = ctypes.c_size_t()
    d = b.us_bitmap(64, 64, 64, 64, b.US_I8, 0, P, P, P, 64, 0, 0)
    assert b.load().us_workspace_bytes(b.US_OP_SPMM_F16, ctypes.byref(d), 1, 0, ctypes.byref(n)) == 1


def test_reference_quantisation_by_hand():
    c, s = kv.quantise(np.array([[7.0, 0.5, 1.5, -2.5, -7.0, 0.0]]), kv.I4)
    assert s[0] == 1 and c[0].tolist() == [7, 0, 2, -2, -7, 0]
    c, s = kv.quantise(np.array([[254.0, 1.0, 3.0, -5.0]]), kv.I8)
    assert s[0] == 2 and c[0].tolist() == [127, 0, 2, -2]
    c, s = kv.quantise(np.array([[0.0, -0.0]]), kv.I8)
    assert s[0] == 1 and (c == 0).all()
    x = np.random.default_rng(0).standard_normal((50, 64)).astype(np.float16)
    for e in (kv.I4, kv.I8):
        c, s = kv.quantise(x, e)
        assert np.array_equal(kv.unpack(kv.pack(c, e), e), c)
        assert (np.abs(c * s.astype(float)[:, None] - x) <= 0.5 * s.astype(float)[:, None] * (1 + 2.0 ** -10)).all()


def test_reference_attention_by_hand():
    """Equal scores give the mean of what a row sees; one large score its value."""
    r = kv.Cache(kv.I8, 64, 1, 16, 1, [[0]])
    for p in range(3):
        r.k[0, 0, p, 0], r.v[0, 0, p] = 10 * p, p + 1
    one = np.zeros((2, 1, 64))
    out, mag, _ = kv.attend(r, 0, one, 1, [[1, 0], [1, 1]], 1.0)
    assert np.allclose(out[0], 1.5) and np.allclose(out[1], 2.0) and np.allclose(mag, out)
    one[:, :, 0] = 10
    out, _, _ = kv.attend(r, 0, one, 1, [[0, 0], [0, 1]], 1.0)
    assert np.allclose(out[0], 1) and np.allclose(out[1], 3)
    out, _, _ = kv.attend(r, 0, one[:1], 0, [[0]], 1.0)
    assert (out == 0).all()
