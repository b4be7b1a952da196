"""Page pool, norm and rotation, latent cache and its attention without a GPU: refusals
before anything is enqueued, the binding's checks, and the plain reference by hand."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import lat
from tests.test_kv_binding import OnGpu, OnOther, on_gpu
from tests.test_kv_host import P, cache


@pytest.fixture(scope="module")
def b():
    from bitmap_encoded_unstructured_ie_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def made(struct, **kw):
    return struct(*(kw[n] for n, _ in struct._fields_))


def pool(b, **kw):
    return made(b.us_kv_pool, **(dict(B=2, page_size=64, num_pages=10, max_pages=4, page_table=P, held=P, free_pages=P, free_count=P) | kw))


def rope(b, **kw):
    return made(b.us_rope, **(dict(style=0, R=64, eps=1e-6, reserved=0, turns=P) | kw))


def heads(b, **kw):
    return made(b.us_heads, **(dict(x=P, ld=1024, hs=128, y=P, ldy=1024, hsy=128, w=P, H=8, reserved=0) | kw))


def lcache(b, **kw):
    return made(b.us_lat_cache, **(dict(Dc=512, Dr=64, page_size=64, num_pages=10, B=2, max_pages=4, rows=P, page_table=P) | kw))


def rows(b, **kw):
    return made(b.us_attn_kv_rows, **(dict(Dn=128, Dr=64, Dv=128, H=4, K=P, ldk=1024, hsk=256, KR=P, ldkr=64, V=P, ldv=1024, hsv=256, S=100) | kw))


def ref(x):
    return ctypes.byref(x) if x is not None else None


PAGES = [(dict(page_size=8), 1), (dict(page_size=48), 1), (dict(page_size=2048), 1), (dict(num_pages=0), 1), (dict(B=0), 1),
         (dict(B=1025), 3), (dict(max_pages=0), 1), (dict(max_pages=1 << 24), 3), (dict(page_table=None), 1), (dict(page_table=P + 4), 1)]


@pytest.mark.parametrize("kw,code", PAGES + [(dict(num_pages=(1 << 30) + 1), 3)])
def test_bad_pools_are_refused(b, kw, code):
    lib, p = b.load(), pool(b, **kw)
    assert lib.us_kv_reserve(ref(p), P, None) == code
    assert lib.us_kv_slots(ref(p), 3, P, P, 2, P, None) == code


def test_pool_calls(b):
    lib = b.load()
    assert lib.us_kv_reserve(None, P, None) == 1 and lib.us_kv_reserve(ref(pool(b)), None, None) == 1
    for kw in (dict(held=None), dict(free_pages=P + 8), dict(free_count=None)):
        assert lib.us_kv_reserve(ref(pool(b, **kw)), P, None) == 1
    p = pool(b, held=None, free_pages=None, free_count=None)      # slots do not need them
    assert lib.us_kv_slots(ref(p), 0, P, P, 1, None, None) == 0
    for args in ((-1, P, P, 1, P), (1, None, P, 1, P), (1, P, P + 4, 1, P), (1, P, P, 0, P), (1, P, P, 1, None), (1, P, P, 1, P + 8)):
        assert lib.us_kv_slots(ref(p), *args, None) == 1
    assert lib.us_kv_slots(ref(p), 1, P, P, 1 << 30, P, None) == 3


ROPES = [dict(style=2), dict(R=-16), dict(R=8), dict(R=144), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
         dict(reserved=1), dict(turns=None), dict(turns=P + 8)]
HEADS = [dict(x=None), dict(x=P + 2), dict(y=P + 8), dict(w=P + 4), dict(ld=1020), dict(hs=124), dict(hs=120), dict(ld=512),
         dict(ldy=1016), dict(hsy=100), dict(H=0), dict(reserved=1), dict(ld=-1024), dict(hs=0)]


@pytest.mark.parametrize("kw", ROPES)
def test_bad_rotations_are_refused(b, kw):
    lib, r, h = b.load(), rope(b, **kw), heads(b)
    assert lib.us_norm_rope(ref(r), 128, ref(h), None, 2, 3, P, P, None, 2, None) == 1
    assert lib.us_kv_append(ref(cache(b)), ref(r), ref(h), ref(h), P, 1024, 3, P, P, None, 2, None) == 1
    assert lib.us_lat_write(ref(lcache(b)), ref(r), P, 576, P, 3, P, P, None, 2, None) == 1


@pytest.mark.parametrize("kw", HEADS)
def test_bad_heads_are_refused(b, kw):
    lib, r, h, good = b.load(), rope(b), heads(b, **kw), heads(b)
    for q, k in ((h, None), (None, h), (good, h), (h, good)):
        assert lib.us_norm_rope(ref(r), 128, ref(q), ref(k), 2, 3, P, P, None, 2, None) == 1
    c = cache(b)
    assert lib.us_kv_append(ref(c), ref(r), ref(h), ref(good), P, 1024, 3, P, P, None, 2, None) == 1
    assert lib.us_kv_append(ref(c), ref(r), None, ref(h), P, 1024, 3, P, P, None, 2, None) == 1


def test_norm_rope_and_append_calls(b):
    lib, r, h, c = b.load(), rope(b), heads(b), cache(b)
    nr = lambda D=128, q=h, k=h, B=2, T=3, off=P, pos=P, depth=None, n=2: lib.us_norm_rope(  # noqa: E731
        ref(r), D, ref(q), ref(k), B, T, off, pos, depth, n, None)
    for kw in (dict(D=0), dict(D=4), dict(D=264), dict(D=100), dict(q=None, k=None), dict(B=0), dict(T=-1), dict(off=None),
               dict(pos=P + 4), dict(depth=P + 4), dict(n=0), dict(D=32)):
        assert nr(**kw) == 1, kw
    assert nr(B=1025) == 3 and nr(n=1 << 30) == 3 and nr(q=heads(b, H=5000, ld=5000 * 128, ldy=5000 * 128)) == 3
    assert nr(q=heads(b, y=None)) == 1
    assert lib.us_norm_rope(None, 128, ref(h), None, 2, 3, P, P, None, 2, None) == 1
    assert nr(T=0) == 0
    ap = lambda C=c, q=h, k=h, V=P, ldv=1024, T=3: lib.us_kv_append(ref(C), ref(r), ref(q), ref(k), V, ldv, T, P, P, None, 2, None)  # noqa: E731
    assert ap(C=None) == 1 and ap(k=None) == 1 and ap(k=heads(b, H=4)) == 1 and ap(V=None) == 1 and ap(ldv=1016) == 1
    assert ap(C=cache(b, D=96)) == 2 and ap(q=heads(b, y=None)) == 1 and ap(T=0) == 0


@pytest.mark.parametrize("kw,code", PAGES + [(dict(Dc=128), 2), (dict(Dc=576), 2), (dict(Dr=32), 2), (dict(Dc=0), 1), (dict(Dr=-64), 1),
                                             (dict(rows=None), 1), (dict(rows=P + 8), 1),
                                             (dict(page_size=1024, num_pages=1 << 21), 3)])
def test_bad_latent_caches_are_refused(b, kw, code):
    lib, c, n = b.load(), lcache(b, **kw), ctypes.c_size_t()
    r = rope(b, R=0, turns=None)
    assert lib.us_lat_write(ref(c), ref(r), P, 4096, P, 3, P, P, None, 2, None) == code
    assert lib.us_lat_read(ref(c), 3, P, P, 2, P, 4096, None) == code
    assert lib.us_lat_commit(ref(c), 3, P, P, P, 2, None) == code
    assert lib.us_attn_lat(ref(c), P, 4096, 4, 3, P, P, None, 2, 0.1, P, 4096, P, 1 << 40, None) == code
    assert lib.us_attn_lat_workspace_bytes(ref(c), 4, 2, ctypes.byref(n)) == code


def test_latent_calls(b):
    lib, c, r = b.load(), lcache(b), rope(b)
    w = lambda X=P, ldx=576, wt=P, T=3, off=P, pos=P, depth=None, n=2, rp=r: lib.us_lat_write(  # noqa: E731
        ref(c), ref(rp), X, ldx, wt, T, off, pos, depth, n, None)
    for kw in (dict(X=None), dict(X=P + 8), dict(ldx=568), dict(ldx=580), dict(wt=P + 2), dict(T=-1), dict(off=P + 4), dict(pos=None),
               dict(depth=P + 8 - 4), dict(n=0), dict(rp=rope(b, R=32)), dict(rp=None)):
        assert w(**kw) == 1, kw
    assert w(T=0) == 0 and w(n=1 << 30) == 3
    assert lib.us_lat_read(ref(c), 3, P, P, 2, P, 568, None) == 1 and lib.us_lat_read(ref(c), 0, P, P, 2, None, 0, None) == 0
    assert lib.us_lat_commit(ref(c), 3, P, P, P, 65, None) == 2 and lib.us_lat_commit(ref(c), 3, P, None, P, 2, None) == 1
    at = lambda Q=P, ldq=8 * 576, Hq=8, T=3, mask=None, n=2, scale=0.1, O=P, ldo=4096, ws=P, wsb=1 << 40: lib.us_attn_lat(  # noqa: E731
        ref(c), Q, ldq, Hq, T, P, P, mask, n, scale, O, ldo, ws, wsb, None)
    for kw in (dict(Q=None), dict(ldq=8 * 576 - 8), dict(Hq=0), dict(T=-1), dict(mask=P + 8), dict(n=0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(O=P + 2), dict(ldo=4088)):
        assert at(**kw) == 1, kw
    assert at(Hq=1025) == 3 and at(mask=P, n=65) == 2 and at(n=1 << 28) == 3
    assert at(ws=None) == 4 and at(wsb=1000) == 4 and at(ws=P + 8) == 4 and at(T=0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(Dn=96), 2), (dict(Dr=32), 2), (dict(Dv=64), 2), (dict(Dn=0), 1), (dict(Dr=0), 1), (dict(Dv=-1), 1), (dict(H=0), 1),
    (dict(H=1025), 3), (dict(K=None), 1), (dict(K=P + 8), 1), (dict(ldk=888), 1), (dict(ldk=1020), 1), (dict(hsk=64), 1),
    (dict(KR=None), 1), (dict(ldkr=56), 1), (dict(V=P + 2), 1), (dict(ldv=512), 1), (dict(hsv=130), 1), (dict(S=0), 1),
    (dict(S=(1 << 30) + 1), 3)])
def test_bad_expanded_rows_are_refused(b, kw, code):
    lib, a = b.load(), rows(b, **({"ldk": 1 << 20, "ldv": 1 << 20} if "H" in kw else {}), **kw)
    assert lib.us_attn_rows(ref(a), P, 1 << 20, 2, 3, P, P, 2, 0.1, P, 1 << 20, P, 1 << 40, None) == code


def test_expanded_calls(b):
    lib, a, n = b.load(), rows(b), ctypes.c_size_t()
    at = lambda Q=P, ldq=768, B=2, T=3, off=P, kv=P, mx=2, scale=0.1, O=P, ldo=512, ws=P, wsb=1 << 40: lib.us_attn_rows(  # noqa: E731
        ref(a), Q, ldq, B, T, off, kv, mx, scale, O, ldo, ws, wsb, None)
    for kw in (dict(Q=None), dict(ldq=760), dict(B=0), dict(T=-1), dict(off=None), dict(kv=None), dict(kv=P + 4), dict(mx=0),
               dict(scale=float("nan")), dict(O=P + 8), dict(ldo=504)):
        assert at(**kw) == 1, kw
    assert at(B=1025) == 3 and at(mx=1 << 28) == 3 and at(ws=None) == 4 and at(wsb=1000) == 4 and at(T=0) == 0
    assert lib.us_attn_rows(None, P, 768, 2, 3, P, P, 2, 0.1, P, 512, P, 1 << 40, None) == 1
    assert lib.us_attn_rows_workspace_bytes(ref(a), 2, 2, None) == 1
    assert lib.us_attn_rows_workspace_bytes(ref(a), 2, 2, ctypes.byref(n)) == 0 and n.value > 1000


# ---- the binding's checks: CPU tensors stand in for device ones, so calls that pass them are not made
def ints(n):
    return on_gpu(n, dtype=torch.int32)


def objects(b):
    r = b.Rope(0, on_gpu(32, dtype=torch.int64))
    P_ = b.KVPool(16, on_gpu(1, 3, dtype=torch.int32), ints(1), ints(3), ints(1))
    L = b.LatCache(512, 64, on_gpu(3, 16, 576), on_gpu(1, 3, dtype=torch.int32))
    C = b.KVCache(b.US_I8, 64, *(on_gpu(3, 2, 16, 64, dtype=torch.uint8) for _ in range(2)), on_gpu(3, 2, 16, 2), on_gpu(1, 3, dtype=torch.int32))
    return r, P_, L, C


def calls(b, o, x, off, pos, word, ws, stream=None):
    """x: (heads 3 x 2 x 64, rows 3 x 576, queries 3 x 2 x 576, latent outputs 3 x 2 x 512, q 3 x 2 x 128)"""
    r, pl, L, C = o
    h, row, ql, ol, q = x
    yield lambda: b.us_kv_reserve(pl, pos, stream=stream)
    yield lambda: b.us_kv_slots(pl, off, pos, 3, word, stream=stream)
    yield lambda: b.us_norm_rope(r, h, None, h, h, None, h, off, pos, None, 3, stream=stream)
    yield lambda: b.us_kv_append(C, r, h, None, h, h, None, h, off, pos, None, 3, stream=stream)
    yield lambda: b.us_lat_write(L, r, row, None, off, pos, None, 3, stream=stream)
    yield lambda: b.us_lat_read(L, off, pos, 3, row, stream=stream)
    yield lambda: b.us_lat_commit(L, off, ints(3), pos, 3, stream=stream)
    yield lambda: b.us_attn_lat(L, ql, off, pos, word, 3, 0.1, ol, ws, stream=stream)
    yield lambda: b.us_attn_rows(q, h, h[:, 0], h, off, off, 3, 0.1, h, ws, stream=stream)


def inputs(dtype=torch.float16):
    return tuple(on_gpu(*s, dtype=dtype) for s in ((3, 2, 64), (3, 576), (3, 2, 576), (3, 2, 512), (3, 2, 128)))


def test_one_device_for_a_call(b, monkeypatch):
    monkeypatch.setattr(OnGpu, "get_device", lambda t: 0, raising=False)
    o, x, off, pos, word, ws = objects(b), inputs(), ints(2), ints(1), on_gpu(3, dtype=torch.int64), on_gpu(64, dtype=torch.uint8)
    for device, stream in ((1, None), (1, 0), (0, 1)):
        monkeypatch.setattr(b, "_current_device", lambda: device)
        st = None if stream is None else type("Stream", (), {"device_index": stream, "cuda_stream": 0})()
        for call in calls(b, o, x, off, pos, word, ws, st):
            with pytest.raises(AssertionError, match="device"):
                call()
    monkeypatch.setattr(b, "_current_device", lambda: 0)
    away = lambda t: t.as_subclass(OnOther)  # noqa: E731
    for xs, of, ps, wd, w, who in ((x, away(off), pos, word, ws, (1, 2, 3, 4, 5, 6, 7, 8)), (x, off, away(pos), word, ws, (0, 1, 2, 3, 4, 5, 6, 7)),
                                   (x, off, pos, away(word), ws, (1, 7)), (x, off, pos, word, away(ws), (7, 8)),
                                   (tuple(map(away, x)), off, pos, word, ws, (2, 3, 4, 5, 7))):
        made_ = list(calls(b, o, xs, of, ps, wd, w))
        for i in who:
            with pytest.raises(AssertionError, match="device"):
                made_[i]()
    with pytest.raises(AssertionError, match="device"):
        b.LatCache(512, 64, o[2].rows, away(o[2].page_table))
    with pytest.raises(AssertionError, match="device"):
        b.KVPool(16, o[1].page_table, away(o[1].held), o[1].free_pages, o[1].free_count)


def test_types_and_shapes_are_checked(b, monkeypatch):
    monkeypatch.setattr(OnGpu, "get_device", lambda t: 0, raising=False)
    monkeypatch.setattr(b, "_current_device", lambda: 0)
    o, off, pos, word, ws = objects(b), ints(2), ints(1), on_gpu(3, dtype=torch.int64), on_gpu(64, dtype=torch.uint8)
    for i, call in enumerate(calls(b, o, inputs(torch.bfloat16), off, pos, word, ws)):
        if i in (2, 3, 4, 5, 7, 8):
            with pytest.raises(AssertionError, match="fp16"):
                call()
    r, pl, L, C = o
    h, row, ql, ol, q = inputs()
    with pytest.raises(AssertionError, match="int64"):
        b.us_kv_slots(pl, off, pos, 3, ints(3))
    with pytest.raises(AssertionError, match="64-bit"):
        b.us_attn_lat(L, ql, off, pos, ints(3), 3, 0.1, ol, ws)
    with pytest.raises(AssertionError, match="weights"):
        b.us_norm_rope(r, h, on_gpu(63), h, None, None, None, off, pos, None, 3)
    with pytest.raises(AssertionError, match="shape"):
        b.us_norm_rope(r, h, None, on_gpu(3, 1, 64), None, None, None, off, pos, None, 3)
    with pytest.raises(AssertionError, match="int32"):
        b.us_norm_rope(r, h, None, h, None, None, None, off, pos, word, 3)
    with pytest.raises(AssertionError):
        b.us_attn_lat(L, q, off, pos, None, 3, 0.1, ol, ws)
    with pytest.raises(AssertionError, match="same rows"):
        b.us_attn_rows(q, h, on_gpu(4, 64), h, off, off, 3, 0.1, h, ws)
    with pytest.raises(AssertionError, match="rows"):
        b.LatCache(512, 64, on_gpu(3, 16, 512), L.page_table)
    with pytest.raises(AssertionError):
        b.KVPool(16, on_gpu(1, 3, dtype=torch.int64), ints(1), ints(3), ints(1))


def test_frequencies_as_fractions_of_a_turn(b):
    """turns / 2^64 is freq / 2 pi of a turn, to 2^-53 of itself; whole turns fall away."""
    f = [1.0, 0.5, 10000.0 ** -0.9, 1e-12, 0.0, 2 * np.pi * 0.75, 2 * np.pi * 3.25, -1.0]
    t = [int(x) & (1 << 64) - 1 for x in b.rope_freq(torch.tensor(f, dtype=torch.float64)).tolist()]
    for x, u in zip(f, t):
        want = x / (2 * np.pi) % 1.0
        assert abs(u / 2 ** 64 - want) <= 2.0 ** -52
    assert t[4] == 0


# ---- the plain reference by hand
def test_reference_pool_by_hand():
    p = lat.Pool(16, 6, 3, 4)
    assert p.reserve([17, 0, 16]) and p.held == [[0, 1], [], [2]] and p.free == [5, 4, 3]
    assert p.reserve([1, 40, 0]) and p.held == [[0], [2, 1, 3], []]          # 1 and 2 given back, then taken from the top
    assert not p.reserve([16, 64, 16 * 3]) and p.held == [[0], [2, 1, 3, 4], []]
    assert p.slot(1, 20) == 16 + 4 and p.table()[1].tolist() == [2, 1, 3, 4]


def test_reference_norm_and_rotation_by_hand():
    assert np.allclose(lat.norm([[3.0, -4.0]], [1.0, 2.0], 0.0), [[3 / np.sqrt(12.5), -8 / np.sqrt(12.5)]])
    x = lat.rotate(np.array([[1.0, 0.0, 0.0, 1.0, 7.0]]), [1], [np.pi / 2, np.pi], pairs=True)
    assert np.allclose(x, [[0, 1, 0, -1, 7]])
    x = lat.rotate(np.array([[1.0, 0.0, 0.0, 1.0, 7.0]]), [2], [np.pi / 4, 0.0], pairs=False)
    assert np.allclose(x, [[0, 0, 1, 1, 7]])


def test_reference_attention_by_hand():
    q, k = np.zeros((2, 4)), np.ones((3, 4))
    o, mag, big = lat.attend(q, k, np.array([[1.0], [3.0], [np.nan]]), [[1, 1, 0], [0, 0, 0]], 1.0)
    assert np.allclose(o, [[2], [0]]) and np.allclose(mag, o) and (big == 0).all()
